"""Activation checkpoints in 8 bits: the very codes, scales and values of the definition."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import step_util as su  # noqa: E402

DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def randn(shape, dtype, seed, spread=2.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(shape, device=DEV, generator=g) * torch.exp(spread * torch.randn(shape, device=DEV, generator=g))
    return x.clamp(-6e4, 6e4).to(dtype)


def run(x, fmt):
    from powersgd_rank_gradient_gb300 import save_activation

    a = save_activation(x, fmt)
    assert a.shape == x.shape and a.dtype == fmt
    su.check_eight(a.codes, a.scales, x, fmt)
    exact = a.codes.float().double() * su.spread(a.scales.double(), x.shape[-1])
    for t in (F32, F16, BF16):
        want = exact.to(t)  # one rounding from 64 bits; what lies between two values of t is not met by 4 bits and a power of two
        got = a.restore(t)
        assert got.dtype == t and torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    return a


@pytest.mark.parametrize("fmt", [su.E4, su.E5])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (5, 128), (2, 129), (7, 256), (33, 200), (151, 1023), (300, 1024), (9, 1600),
                                      (4, 8191), (2, 20001), (0, 64)])
def test_shapes(rows, dim, dtype, fmt):
    run(randn((rows, dim), dtype, rows + dim), fmt)


@pytest.mark.parametrize("fmt", [su.E4, su.E5])
def test_every_value_around_each_border(fmt):
    """Values at, just under and just over the middle of two neighbours, in a block whose scale is 1; the scale's borders."""
    values = torch.arange(256, dtype=torch.uint8, device=DEV).view(fmt).float()
    values = torch.sort(values[torch.isfinite(values)]).values.unique()
    middle = 0.5 * (values[1:] + values[:-1])
    x = torch.cat([values, middle, middle * (1 + 2.0 ** -23), middle * (1 - 2.0 ** -23)])
    most = su.MOST[fmt]
    x = torch.nn.functional.pad(x, (0, -len(x) % 127)).view(-1, 127)
    x = torch.cat([x, torch.full_like(x[:, :1], most)], 1)
    a = run(x, fmt)
    assert bool((a.scales == 1).all())
    tops = torch.tensor([most, most * (1 + 2.0 ** -23), most * (1 - 2.0 ** -23), 2 * most, 1.0, 2.0 ** -126, 2.0 ** -140, 3.4028234e38,
                         1e-30, 2.0 ** 120], device=DEV)
    run(torch.cat([tops, -tops])[:, None].repeat(1, 130), fmt)


@pytest.mark.parametrize("fmt", [su.E4, su.E5])
@pytest.mark.parametrize("dtype,dim", [(F32, 256), (BF16, 384), (F16, 131)])
def test_infinities_and_nan(fmt, dtype, dim):
    x = randn((9, dim), dtype, 1)
    x[1, 3], x[2, 130], x[3, 5], x[4, 100:128] = torch.nan, torch.inf, -torch.inf, torch.inf
    x[5], x[6] = torch.nan, torch.inf
    x[7] = 0
    x[7, 17] = -torch.nan
    run(x, fmt)


@pytest.mark.parametrize("dtype,dim", [(BF16, 256), (F32, 100), (F16, 131)])
def test_strides_and_places(dtype, dim):
    from powersgd_rank_gradient_gb300 import Activation8, save_activation

    for offset, gap in [(0, 0), (1, 8), (8, 3), (3, 0)]:
        flat = randn((offset + 40 * (dim + gap),), dtype, offset)
        x = flat[offset:].view(40, dim + gap)[:, :dim]
        a = run(x, su.E4)
        place = torch.zeros(40 * dim + 3, dtype=torch.uint8, device=DEV).view(su.E4)[offset % 4:][:40 * dim].view(40, dim)
        b = Activation8(place, torch.empty_like(a.scales))
        assert save_activation(x, out=b) is b and torch.equal(b.codes.view(torch.uint8), a.codes.view(torch.uint8))
        out = torch.full_like(flat, 7.0)
        view = out[offset:].view(40, dim + gap)[:, :dim]
        assert b.restore(out=view) is view and torch.equal(view, a.restore(dtype))
        assert bool((out[:offset] == 7).all()) and bool((out[offset:].view(40, dim + gap)[:, dim:] == 7).all())
    one = run(x[:1].expand(30, dim), su.E5)
    assert torch.equal(one.scales[0], one.scales[29])
    run(randn((2, 3, 4, dim), dtype, 5), su.E4)


def test_offsets_beyond_32_bits():
    from powersgd_rank_gradient_gb300 import save_activation

    rows, dim = 65536 + 3, 1 << 16
    x = torch.zeros((rows, dim), dtype=BF16, device=DEV)  # 8 GB
    x[-1] = randn((dim,), BF16, 1)
    a = save_activation(x)
    su.check_eight(a.codes[-2:], a.scales[-2:], x[-2:], su.E4)
    assert not bool(a.codes.view(torch.uint8)[::4099].any())
    y = a.restore(BF16, out=x)
    want = (a.codes[-1].float() * su.spread(a.scales[-1], dim)).to(BF16)
    assert torch.equal(y[-1], want) and not bool(y[:-1:4099].any())


def test_streams_and_graphs():
    from powersgd_rank_gradient_gb300 import save_activation

    x = randn((500, 640), BF16, 1)
    want = save_activation(x).restore(BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = save_activation(x, stream=side).restore(BF16, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = save_activation(x)
        y = a.restore(BF16)
    x.mul_(2.0)
    graph.replay()
    assert torch.equal(y, 2 * want)
    before = y._version
    a.restore(out=y)
    assert y._version == before + 1


def test_refusals():
    from powersgd_rank_gradient_gb300 import Activation8, save_activation
    from powersgd_rank_gradient_gb300._lib import PsgdError

    x = randn((4, 64), BF16, 1)
    a = save_activation(x)
    for call, words in [
        (lambda: save_activation(x.cpu()), "must be a CUDA tensor"),
        (lambda: save_activation(x.double()), "float32, float16 or bfloat16"),
        (lambda: save_activation(x, torch.int8), "float8"),
        (lambda: save_activation(x, "e4m3"), "torch.dtype"),
        (lambda: save_activation(x[0, 0]), "x must have rows"),
        (lambda: save_activation(x[:, :0]), "last dimension"),
        (lambda: save_activation(x[:, ::2]), "contiguous in its last"),
        (lambda: save_activation(x[:3], out=a), "out must have x's shape"),
        (lambda: a.restore(torch.float64), "float32, float16 or bfloat16"),
        (lambda: a.restore(out=x[:3]), "shape"),
        (lambda: a.restore(out=x.cpu()), "must be on cuda"),
        (lambda: save_activation(x.float().requires_grad_()), "requires a gradient"),
        (lambda: Activation8(a.codes.cpu(), a.scales), "CUDA tensor"),
        (lambda: Activation8(a.codes, a.scales.cpu()), "must be on cuda"),
        (lambda: Activation8(a.codes.view(torch.uint8), a.scales), "float8"),
        (lambda: Activation8(a.codes[:, ::2], a.scales), "contiguous"),
    ]:
        with pytest.raises(ValueError, match=words):
            call()
    with pytest.raises(PsgdError, match="overlap"):
        a.restore(out=a.codes.view(torch.uint8).view(-1)[:256].view(F32).view(1, 64).expand(4, 64))
