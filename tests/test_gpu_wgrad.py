"""The weight gradient from an 8-bit checkpoint against its 64-bit definition."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import step_util as su  # noqa: E402

DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def randn(shape, dtype, seed, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0, std, generator=g)


def handle(outs, ins, rows):
    from powersgd_rank_gradient_gb300 import LinearWeightGrad

    return LinearWeightGrad(outs, ins, rows, device=DEV)


def run(rows, outs, ins, dtype, odtype=F32, fmt=su.E4, accumulate=False, grad=None, h=None, seed=0):
    from powersgd_rank_gradient_gb300 import save_activation

    h = h or handle(outs, ins, rows)
    kept = save_activation(randn((rows, ins), dtype, seed + 1), fmt)
    grad = randn((rows, outs), dtype, seed + 2) if grad is None else grad
    bucket = torch.full((outs * ins + 9,), 7.0, dtype=odtype, device=DEV)
    out = bucket[3:3 + outs * ins].view(outs, ins)
    before = randn((outs, ins), odtype, seed + 3) if accumulate else None
    first = None
    for _ in range(2):
        if accumulate:
            out.copy_(before)
        assert h.backward(grad, kept, out=out, accumulate=accumulate) is out
        h.status()
        if first is None:
            first = bucket.clone()
    assert torch.equal(first, bucket), "another result from the same inputs"
    want, err = su.product(grad, kept.restore(F32), before=before)
    su.check(out, want, su.out_tol(err, want, odtype))
    assert bool((bucket[:3] == 7.0).all()) and bool((bucket[3 + outs * ins:] == 7.0).all())
    return h


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,outs,ins", [(64, 256, 256), (1, 8, 8), (16, 64, 64), (64, 128, 128), (65, 64, 136), (100, 300, 520),
                                           (512, 1024, 512)])
def test_small(rows, outs, ins, dtype):
    run(rows, outs, ins, dtype)


@pytest.mark.parametrize("rows,outs,ins", [(0, 40, 72), (1, 1, 1), (3, 1, 300), (7, 301, 1), (513, 257, 255), (1000, 100, 1601),
                                           (2049, 1023, 77), (63, 2000, 1992)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_odd_sizes(rows, outs, ins, accumulate):
    run(rows, outs, ins, BF16, accumulate=accumulate, fmt=su.E5)


@pytest.mark.parametrize("rows,outs,ins", [(16384, 256, 256), (5000, 1024, 1024), (4096, 2560, 2304), (1024, 3000, 4600), (8192, 300, 5000)])
def test_tiles_that_are_cut(rows, outs, ins):
    run(rows, outs, ins, F16)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("odtype", [F32, F16, BF16])
@pytest.mark.parametrize("accumulate", [False, True])
def test_types(dtype, odtype, accumulate):
    run(333, 264, 200, dtype, odtype, accumulate=accumulate)


@pytest.mark.parametrize("outs", [256, 100])
def test_gradients_of_any_layout(outs):
    h = handle(outs, 128, 300)
    for offset, gap in [(0, 8), (1, 0), (8, 3), (4, 4)]:
        flat = randn((offset + 300 * (outs + gap),), BF16, offset)
        run(300, outs, 128, BF16, grad=flat[offset:].view(300, outs + gap)[:, :outs], h=h)
    run(300, outs, 128, BF16, grad=randn((1, outs), BF16, 5).expand(300, outs), h=h)
    run(1, outs, 128, BF16, grad=randn((outs,), BF16, 6)[None], h=h)
    run(7, outs, 128, BF16, h=h)


def test_leading_shapes_and_a_strided_out():
    from powersgd_rank_gradient_gb300 import save_activation

    h = handle(72, 40, 24)
    kept, grad = save_activation(randn((2, 3, 4, 40), BF16, 1)), randn((2, 3, 4, 72), BF16, 2)
    want, err = su.product(grad.view(24, 72), kept.restore(F32).view(24, 40))
    new = h.backward(grad, kept)
    assert new.dtype == F32
    su.check(new, want, su.out_tol(err, want, F32))
    wide = torch.full((72, 50), 7.0, device=DEV)
    h.backward(grad, kept, out=wide[:, 5:45])
    assert torch.equal(wide[:, 5:45], new) and bool((wide[:, :5] == 7).all()) and bool((wide[:, 45:] == 7).all())


def test_rows_of_zeros_and_nan_stay_where_they_belong():
    from powersgd_rank_gradient_gb300 import save_activation

    h = handle(300, 200, 100)
    x, g = randn((100, 200), BF16, 1), randn((100, 300), BF16, 2)
    x[5, 17], g[9, 33] = torch.nan, torch.inf
    x[9] = x[9].abs() + 1
    d = h.backward(g, save_activation(x))
    bad = torch.isnan(d)
    assert bool(bad[:, 17].all()) and bool(torch.isinf(d[33]).sum() == 199) and int(bad.sum()) == 300


def test_streams_and_graphs():
    from powersgd_rank_gradient_gb300 import save_activation

    h = handle(520, 264, 1000)
    kept, grad = save_activation(randn((1000, 264), BF16, 1)), randn((1000, 520), BF16, 2)
    want = h.backward(grad, kept)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = h.backward(grad, kept, stream=side)
    h.status(stream=side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    out = torch.zeros_like(want)
    with torch.cuda.graph(graph):
        h.backward(grad, kept, out=out)
    for factor in (2.0, 0.5):
        grad.mul_(factor)
        graph.replay()
        want = want * factor
        assert torch.equal(out, want)
    before = out._version
    h.backward(grad, kept, out=out)
    assert out._version == before + 1


def test_refusals():
    from powersgd_rank_gradient_gb300 import save_activation
    from powersgd_rank_gradient_gb300._lib import PsgdError

    h = handle(64, 32, 10)
    kept, grad = save_activation(randn((10, 32), BF16, 1)), randn((10, 64), BF16, 2)
    for call, words in [
        (lambda: h.backward(grad.float(), kept), "grad must be float16 or bfloat16"),
        (lambda: h.backward(grad[:, :32], kept), "last dimension of 64"),
        (lambda: h.backward(grad[:5], kept), "the checkpoint must be"),
        (lambda: h.backward(grad, save_activation(grad)), "the checkpoint must be"),
        (lambda: h.backward(grad.cpu(), kept), "must be on cuda"),
        (lambda: h.backward(grad, kept, accumulate=True), "accumulate needs"),
        (lambda: h.backward(grad, kept, out=torch.zeros(32, 64, device=DEV)), "out must be"),
        (lambda: h.backward(grad, kept, out=torch.zeros(32, 64, device=DEV).t()), "contiguous in its last"),
    ]:
        with pytest.raises(ValueError, match=words):
            call()
    with pytest.raises(PsgdError, match="max_rows"):
        h.backward(torch.cat([grad, grad]), save_activation(randn((20, 32), BF16, 1)))
    with pytest.raises(PsgdError, match="rows overlap"):
        h.backward(grad, kept, out=torch.zeros(1, 32, device=DEV).expand(64, 32))
    with pytest.raises(PsgdError, match="overlaps"):
        big = randn((64, 64), BF16, 3)
        h.backward(big[:10], kept, out=big[:, :32])
    h.close()
    with pytest.raises(PsgdError, match="NULL"):
        h.backward(grad, kept)
