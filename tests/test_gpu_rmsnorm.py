"""Root-mean-square norm, forward and backward, against its 64-bit definition."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import step_util as su  # noqa: E402

DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-6


def randn(shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(mean, std, generator=g)


def norm(dim, eps=EPS):
    from powersgd_rank_gradient_gb300 import RMSNorm

    return RMSNorm(dim, eps=eps, device=DEV)


def run_forward(n, x, w, residual, fmt=su.E4, eps=EPS):
    want_s = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    (wy, wr), (ey, er) = su.rms_forward(want_s, w, eps)
    y, s, rstd = n.forward(x, w, residual)
    assert torch.equal(s, want_s) and (residual is not None or s is x)
    su.check(y, wy, su.out_tol(ey, wy, x.dtype))
    su.check(rstd, wr, su.out_tol(er, wr, F32))
    q, s8, rstd8 = n.forward8(x, w, residual, dtype=fmt)
    assert torch.equal(s8, s) and torch.equal(rstd8, rstd)
    su.check_eight_near(q.codes, q.scales, wy, ey + su.TINY[F32], fmt)
    return s, rstd


def run_backward(n, grad, s, rstd, w, add, odtype=F32, accumulate=False, fmt=None, seed=0):
    from powersgd_rank_gradient_gb300 import save_activation

    dim = grad.shape[-1]
    kept = s if fmt is None else save_activation(s, fmt)
    values = s if fmt is None else kept.restore(F32)
    bucket = torch.full((dim + 9,), 7.0, dtype=odtype, device=DEV)
    dw = bucket[3:3 + dim]
    before = randn((dim,), odtype, seed + 4) if accumulate else None
    if accumulate:
        dw.copy_(before)
    dx, gw = n.backward(grad, kept, rstd, w, grad_summed=add, dweight=dw, accumulate=accumulate)
    assert gw is dw
    (wx, ww), (ex, ew) = su.rms_backward(grad, values, rstd, w, add, before)
    su.check(dx, wx, su.out_tol(ex, wx, grad.dtype))
    su.check(dw, ww, su.out_tol(ew, ww, odtype))
    assert bool((bucket[:3] == 7.0).all()) and bool((bucket[3 + dim:] == 7.0).all())
    first = bucket.clone()
    if accumulate:
        dw.copy_(before)
    dx2, _ = n.backward(grad, kept, rstd, w, grad_summed=add, dweight=dw, accumulate=accumulate)
    assert torch.equal(dx, dx2) and torch.equal(first, bucket), "another result from the same inputs"


def run_both(rows, dim, dtype, pdtype, seed, residual=True, fmt=None, odtype=F32, accumulate=False):
    n = norm(dim)
    x = randn((rows, dim), dtype, seed, 1.5, 0.25)
    w = randn((dim,), pdtype, seed + 1, 0.2, 1.0)
    r = randn((rows, dim), dtype, seed + 2) if residual else None
    s, rstd = run_forward(n, x, w, r, fmt or su.E4)
    add = randn((rows, dim), dtype, seed + 5) if residual else None
    run_backward(n, randn((rows, dim), dtype, seed + 3), s, rstd, w, add, odtype, accumulate, fmt, seed)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim", [1, 2, 3, 8, 31, 33, 64, 100, 127, 128, 129, 255, 256, 512, 640, 1000, 1023, 1024, 1600, 2050, 4096,
                                 4800, 6400, 8191, 8192, 8200, 16384, 20001])
def test_widths(dim, dtype):
    run_both(7, dim, dtype, F32, dim, residual=dim % 2 == 0, fmt=(None, su.E4, su.E5)[dim % 3])


@pytest.mark.parametrize("rows", [0, 1, 2, 3, 5, 151, 153, 609, 2435, 4867, 20011])
@pytest.mark.parametrize("dim,dtype,fmt", [(64, F32, None), (129, BF16, su.E4), (1024, BF16, su.E5), (1600, F16, None)])
def test_row_counts(rows, dim, dtype, fmt):
    run_both(rows, dim, dtype, F32, rows, fmt=fmt)


@pytest.mark.parametrize("dtype,pdtype,odtype", [(F32, F32, F32), (F16, F16, F16), (F16, F32, F32), (BF16, BF16, BF16),
                                                 (BF16, F32, F16), (F32, BF16, BF16)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_types(dtype, pdtype, odtype, accumulate):
    run_both(37, 200, dtype, pdtype, 11, odtype=odtype, accumulate=accumulate)


def test_without_weight_and_leading_shapes():
    n = norm(96)
    x = randn((3, 5, 7, 96), BF16, 1)
    s, rstd = run_forward(n, x, None, x * 0.5)
    assert s.shape == x.shape and rstd.shape == (3, 5, 7)
    run_backward(n, randn((3, 5, 7, 96), BF16, 2), s, rstd, None, None)
    y, s, rstd = n.forward(x[0, 0, 0])
    assert y.shape == (96,) and rstd.shape == () and torch.equal(y, n.forward(x)[0][0, 0, 0])


@pytest.mark.parametrize("dtype,dim", [(BF16, 256), (F32, 100), (F16, 131)])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_strides_and_places(dtype, dim, offset):
    n = norm(dim)

    def rows(seed, gap):
        flat = randn((offset + 40 * (dim + gap),), dtype, seed)
        return flat[offset:].view(40, dim + gap)[:, :dim]

    x, r, g, add = rows(1, 8), rows(2, 3), rows(3, 0), rows(4, 16)
    w = randn((dim + 1,), dtype, 5)[1:]
    out, summed, dx = rows(6, 5), rows(7, 8), rows(8, 24)
    y, s, rstd = n.forward(x, w, r, out=out, summed=summed)
    assert y is out and s is summed
    wy, ws, wr = n.forward(x.contiguous(), w.clone(), r.contiguous())
    assert torch.equal(y, wy) or offset or dim % 8  # the order of a row's sum goes by alignment
    (ey, er), (ty, tr) = su.rms_forward(ws, w, EPS)
    su.check(y, ey, su.out_tol(ty, ey, dtype))
    assert torch.equal(s, ws)
    run_backward(n, g, s, rstd, w, add)
    got, _ = n.backward(g, s, rstd, w, grad_summed=add, dx=dx)
    assert got is dx
    (wx, _), (ex, _) = su.rms_backward(g, s, rstd, w, add)
    su.check(dx, wx, su.out_tol(ex, wx, dtype))
    # one residual row for all
    y1, s1, _ = n.forward(x, w, r[:1].expand(40, dim))
    assert torch.equal(s1, (x.float() + r[:1].float()).to(dtype))


@pytest.mark.parametrize("dim", [256, 131, 9000])
def test_in_place(dim):
    n = norm(dim)
    x, r, w = randn((50, dim), BF16, 1), randn((50, dim), BF16, 2), randn((dim,), BF16, 3)
    y, s, rstd = n.forward(x, w, r)
    for place in (0, 1):
        ops = [x.clone(), r.clone()]
        y2, s2, rstd2 = n.forward(ops[0], w, ops[1], summed=ops[place])
        assert s2 is ops[place] and torch.equal(s2, s) and torch.equal(y2, y) and torch.equal(rstd2, rstd)
    g, add = randn((50, dim), BF16, 4), randn((50, dim), BF16, 5)
    dx, dw = n.backward(g, s, rstd, w, grad_summed=add)
    for place in (0, 1):
        ops = [g.clone(), add.clone()]
        dx2, dw2 = n.backward(ops[0], s, rstd, w, grad_summed=ops[1], dx=ops[place])
        assert dx2 is ops[place] and torch.equal(dx2, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("dim", [256, 131, 9000])
def test_nan_and_infinity_stay_in_their_rows(dim):
    n = norm(dim)
    x, g = randn((6, dim), F32, 1), randn((6, dim), F32, 2)
    want, s, rstd = n.forward(x)
    wx, _ = n.backward(g, s, rstd)
    x[1, 5], x[4, 7] = torch.nan, torch.inf
    y, s, rstd = n.forward(x)
    q, _, _ = n.forward8(x)
    dx, _ = n.backward(g, s, rstd)
    keep = [0, 2, 3, 5]
    assert torch.equal(y[keep], want[keep]) and torch.equal(dx[keep], wx[keep])
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(q.restore(F32)[1]).all())
    assert float(rstd[4]) == 0.0 and bool(torch.isnan(y[4, 7])) and int(torch.isnan(y[4]).sum()) == 1


def test_rows_of_zeros():
    n = norm(300)
    x = torch.zeros((3, 300), device=DEV, dtype=F16)
    y, s, rstd = n.forward(x)
    q, _, _ = n.forward8(x)
    assert not bool(y.any()) and bool((q.scales == 1).all()) and not bool(q.codes.float().any())
    assert float((rstd - EPS ** -0.5).abs().max()) < 1e-3


def test_offsets_beyond_32_bits():
    stride = (1 << 30) + 8
    flat = torch.zeros(2 * stride + 640, device=DEV, dtype=F16)
    x = torch.as_strided(flat, (3, 640), (stride, 1))
    x.copy_(randn((3, 640), F16, 1))
    n = norm(640)
    y, s, rstd = n.forward(x, residual=randn((3, 640), F16, 2), summed=x)
    (wy, _), (ey, _) = su.rms_forward(s.clone(), None, EPS)
    su.check(y, wy, su.out_tol(ey, wy, F16))
    g = randn((3, 640), F16, 3)
    dx, _ = n.backward(g, x, rstd, dx=x.new_empty(3, 640))
    (wx, _), (ex, _) = su.rms_backward(g, s.clone(), rstd, None)
    su.check(dx, wx, su.out_tol(ex, wx, F16))


def test_gradient_against_differences():
    """dx and dw against central differences of the forward definition in 64 bits."""
    n, dim = norm(48), 48
    x, w, c = randn((4, dim), F32, 1), randn((dim,), F32, 2, 0.3, 1.0), randn((4, dim), F32, 3)
    _, s, rstd = n.forward(x, w)
    dx, dw = n.backward(c, s, rstd, w)

    def loss(x, w):
        return float((su.rms_forward(x, w, EPS)[0][0] * c.double()).sum())

    h = 1e-4
    for k in range(5):
        vx, vw = randn((4, dim), F32, 10 + k).double(), randn((dim,), F32, 20 + k).double()
        slope = (loss(x.double() + h * vx, w.double() + h * vw) - loss(x.double() - h * vx, w.double() - h * vw)) / (2 * h)
        got = float((dx.double() * vx).sum() + (dw.double() * vw).sum())
        # third derivatives leave h^2 of the slope's scale, fp32 some 1e-6 of the terms' size
        size = float((dx.double() * vx).abs().sum() + (dw.double() * vw).abs().sum())
        assert abs(got - slope) <= 1e-5 * size


def test_streams_and_graphs():
    n = norm(512)
    x, r, w, g = randn((300, 512), BF16, 1), randn((300, 512), BF16, 2), randn((512,), BF16, 3), randn((300, 512), BF16, 4)

    def step(**kw):
        q, s, rstd = n.forward8(x, w, r, **kw)
        return (q.codes, q.scales, *n.backward(g, s, rstd, w, grad_summed=r, **kw))

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    side.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        x.copy_(torch.roll(x, 1, 0)), r.copy_(torch.roll(r, 1, 0)), g.copy_(torch.roll(g, 1, 0))
        graph.replay()
        assert torch.equal(got[2], torch.roll(want[2], 1, 0))
        want[2] = got[2].clone()


def test_refusals():
    from powersgd_rank_gradient_gb300 import Activation8
    from powersgd_rank_gradient_gb300._lib import PsgdError

    n = norm(64)
    x = randn((4, 64), BF16, 1)
    y, s, rstd = n.forward(x)
    q = n.forward8(x)[0]
    for call, words in [
        (lambda: n.forward(x[:, :32]), "last dimension of 64"),
        (lambda: n.forward(x.t().contiguous().t()), "contiguous in its last"),
        (lambda: n.forward(x.int()), "float32, float16 or bfloat16"),
        (lambda: n.forward(x.cpu()), "must be on cuda:0"),
        (lambda: n.forward(x, residual=x[:3]), "residual must have x's shape and type"),
        (lambda: n.forward(x, residual=x.float()), "residual must have x's shape and type"),
        (lambda: n.forward(x, torch.ones(63, device=DEV)), "weight must be a contiguous vector of 64"),
        (lambda: n.forward8(x, dtype=torch.bfloat16), "float8_e4m3fn or float8_e5m2"),
        (lambda: n.forward8(x, out=Activation8(q.codes[:2], q.scales[:2])), "out must have x's shape"),
        (lambda: n.backward(x, s, rstd[:3]), "rstd must be"),
        (lambda: n.backward(x, s.float(), rstd), "summed must have grad's shape and type"),
        (lambda: n.backward(x, Activation8(q.codes[:2], q.scales[:2]), rstd), "must have grad's shape"),
        (lambda: n.backward(x, s, rstd, accumulate=True), "accumulate needs"),
        (lambda: n.forward(x.float().requires_grad_()), "x requires a gradient"),
        (lambda: Activation8(q.codes, q.scales[:, :0]), "scales must be"),
        (lambda: Activation8(q.codes.float(), q.scales), "float8"),
        (lambda: Activation8(q.codes, q.scales.half()), "scales must be float32"),
    ]:
        with pytest.raises(ValueError, match=words):
            call()
    for call in [lambda: n.forward(x, out=x), lambda: n.forward(x[1:], residual=x[:3], summed=x[:3]),
                 lambda: n.forward(x, out=y, summed=y), lambda: n.backward(x, s, rstd, dx=s),
                 lambda: n.backward(x[1:], y[1:], rstd[1:], dx=x[:3])]:
        with pytest.raises(PsgdError, match="overlap"):
            call()
    n.close()
    with pytest.raises(PsgdError, match="NULL"):
        n.forward(x)
