"""Layer norm forward and backward against their 64-bit definitions."""

import pytest

import training_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-5


def randn(shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(mean, std, generator=g)


def norm(dim, eps=EPS):
    from powersgd_rank_gradient_gb300 import LayerNorm

    return LayerNorm(dim, eps=eps, device=DEV)


def stats_of(x):
    d = x.double()
    mean = d.mean(-1)
    return mean.float(), ((d - mean[..., None]).square().mean(-1) + EPS).rsqrt().float()


def run_both(rows, dim, dtype, pdtype, seed, x=None, grad=None, odtype=F32, accumulate=False, n=None):
    n = n or norm(dim)
    x = randn((rows, dim), dtype, seed, 1.5, 0.25) if x is None else x
    grad = randn((rows, dim), dtype, seed + 1) if grad is None else grad
    w, b = randn((dim,), pdtype, seed + 2, 0.2, 1.0), randn((dim,), pdtype, seed + 3)
    y, mean, rstd = n.forward(x, w, b)
    (wy, wm, wr), (ey, em, er) = tu.norm_forward(x, w, b, EPS)
    tu.check(y, wy, tu.out_tol(ey, wy, dtype))
    tu.check(mean, wm, tu.out_tol(em, wm, F32))
    tu.check(rstd, wr, tu.out_tol(er, wr, F32))
    bucket = torch.full((2 * dim + 9,), 7.0, dtype=odtype, device=DEV)
    dw, db = bucket[3:3 + dim], bucket[3 + dim:3 + 2 * dim]
    before = None
    if accumulate:
        before = (randn((dim,), odtype, seed + 4), randn((dim,), odtype, seed + 5))
        dw.copy_(before[0])
        db.copy_(before[1])
    dx, gw, gb = n.backward(grad, x, mean, rstd, w, dweight=dw, dbias=db, accumulate=accumulate)
    assert gw is dw and gb is db
    (wx, ww, wb), (ex, ew, eb) = tu.norm_backward(grad, x, mean, rstd, w, before)
    tu.check(dx, wx, tu.out_tol(ex, wx, dtype))
    tu.check(dw, ww, tu.out_tol(ew, ww, odtype))
    tu.check(db, wb, tu.out_tol(eb, wb, odtype))
    assert bool((bucket[:3] == 7.0).all()) and bool((bucket[3 + 2 * dim:] == 7.0).all())
    first = bucket.clone()
    if accumulate:
        dw.copy_(before[0])
        db.copy_(before[1])
    dx2, _, _ = n.backward(grad, x, mean, rstd, w, dweight=dw, dbias=db, accumulate=accumulate)
    assert torch.equal(dx, dx2) and torch.equal(first, bucket), "another result from the same inputs"
    return n


@pytest.mark.parametrize("dtype", tu.DTYPES)
@pytest.mark.parametrize("dim", [1, 2, 3, 8, 31, 32, 33, 64, 100, 255, 256, 512, 640, 1000, 1023, 1024, 1025, 1600, 2050, 4096,
                                 4800, 6400, 8191, 8192, 16384, 20000, 33000])
def test_widths(dim, dtype):
    run_both(7, dim, dtype, F32, dim)


@pytest.mark.parametrize("rows", [0, 1, 2, 3, 4, 5, 151, 152, 153, 607, 609, 1217, 2435, 4867, 20011])
@pytest.mark.parametrize("dim,dtype", [(64, F32), (129, BF16), (1024, BF16)])
def test_row_counts(rows, dim, dtype):
    run_both(rows, dim, dtype, F32, rows)


@pytest.mark.parametrize("dtype,pdtype,odtype", [(F32, F32, F32), (F16, F16, F16), (F16, F32, F32), (BF16, BF16, BF16),
                                                 (BF16, F32, F16), (F32, BF16, BF16)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_types(dtype, pdtype, odtype, accumulate):
    for dim in (96, 333):
        run_both(75, dim, dtype, pdtype, 5, odtype=odtype, accumulate=accumulate)


def test_large():
    run_both(16384, 1024, BF16, F32, 1)
    run_both(3001, 1600, F32, F32, 2)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("dim", [64, 200, 1600])
def test_strides(dtype, dim):
    big = randn((40, dim + 24), dtype, 1, 1.5)
    grads = randn((40, 3 * dim + 5), dtype, 2)
    for x in (big[:, :dim], big[:, 1:dim + 1], big[::2, 16:dim + 16], big[:1, :dim].expand(40, dim)):
        g = grads[:x.shape[0], dim:2 * dim]
        run_both(x.shape[0], dim, dtype, F32, 3, x=x, grad=g)
    run_both(20, dim, dtype, F32, 4, x=big[:20, :dim], grad=grads[:1, :dim].expand(20, dim))


@pytest.mark.parametrize("dim", [1024, 1023])
def test_offsets_beyond_32_bits(dim):
    """More than 2^31 elements; rows from both ends and the middle, and the columns' sums of all of them."""
    rows = 2**31 // dim + 999
    n = norm(dim)
    x, g = torch.zeros((rows, dim), dtype=BF16, device=DEV), torch.zeros((rows, dim), dtype=BF16, device=DEV)
    places = torch.cat([torch.arange(40), torch.arange(rows // 2, rows // 2 + 40), torch.arange(rows - 40, rows)]).to(DEV)
    x[places], g[places] = randn((120, dim), BF16, 1, 1.5), randn((120, dim), BF16, 2)
    w = randn((dim,), F32, 3)
    y, mean, rstd = n.forward(x, w)
    part, pg = x[places], g[places]
    (wy, _, _), (ey, _, _) = tu.norm_forward(part, w, None, EPS)
    tu.check(y[places], wy, tu.out_tol(ey, wy, BF16))
    dx, dw, db = n.backward(g, x, mean, rstd, w, dx=y)
    (wx, ww, wb), (ex, ew, eb) = tu.norm_backward(pg, part, mean[places], rstd[places], w)
    tu.check(dx[places], wx, tu.out_tol(ex, wx, BF16))
    # the other rows add zeros to the columns' sums
    tu.check(dw, ww, tu.out_tol(ew, ww, F32))
    tu.check(db, wb, tu.out_tol(eb, wb, F32))


def test_three_dimensions_and_outputs():
    n = norm(48)
    x = randn((3, 5, 48), BF16, 1)
    w = randn((48,), F32, 2)
    room = torch.full((15, 60), 4.0, dtype=BF16, device=DEV)
    y, mean, rstd = n.forward(x.view(15, 48), w, None, out=room[:, 5:53])
    (wy, _, _), (ey, _, _) = tu.norm_forward(x.view(15, 48), w, None, EPS)
    tu.check(y, wy, tu.out_tol(ey, wy, BF16))
    assert bool((room[:, :5] == 4.0).all()) and bool((room[:, 53:] == 4.0).all())
    y3, mean3, rstd3 = n.forward(x, w)
    assert y3.shape == x.shape and mean3.shape == (3, 5) and torch.equal(mean3.view(15), mean)
    g = randn((3, 5, 48), BF16, 3)
    dx, dw, db = n.backward(g, x, mean3, rstd3, w)
    assert dx.shape == x.shape and dw.dtype == F32 and db.shape == (48,)


def test_without_parameters():
    n = norm(130)
    x, g = randn((9, 130), F32, 1), randn((9, 130), F32, 2)
    y, mean, rstd = n.forward(x)
    (wy, _, _), (ey, _, _) = tu.norm_forward(x, None, None, EPS)
    tu.check(y, wy, tu.out_tol(ey, wy, F32))
    dx, dw, db = n.backward(g, x, mean, rstd)
    (wx, ww, wb), (ex, ew, eb) = tu.norm_backward(g, x, mean, rstd, None)
    tu.check(dx, wx, tu.out_tol(ex, wx, F32))
    tu.check(dw, ww, tu.out_tol(ew, ww, F32))
    tu.check(db, wb, tu.out_tol(eb, wb, F32))


@pytest.mark.parametrize("dim", [64, 1000, 1023])
def test_rows_without_variance_and_far_from_zero(dim):
    n = norm(dim)
    x = randn((12, dim), F32, 1, 0.1, 1000.0)
    x[3] = 5.0
    x[4] = 0.0
    x[5] = -1e-30
    w, b = randn((dim,), F32, 2), randn((dim,), F32, 3)
    y, mean, rstd = n.forward(x, w, b)
    (wy, wm, wr), (ey, em, er) = tu.norm_forward(x, w, b, EPS)
    tu.check(y, wy, tu.out_tol(ey, wy, F32))
    tu.check(rstd, wr, tu.out_tol(er, wr, F32))
    assert torch.equal(y[4], b)


def test_nonfinite_rows_stay_apart():
    n = norm(96)
    x, g = randn((50, 96), F32, 1), randn((50, 96), F32, 2)
    clean = n.forward(x)[0]
    x[7, 3], x[9, 90] = float("inf"), float("nan")
    y, mean, rstd = n.forward(x)
    bad = torch.zeros(50, dtype=torch.bool, device=DEV)
    bad[7] = bad[9] = True
    assert torch.equal(y[~bad], clean[~bad]) and bool(torch.isnan(y[9]).all()) and not bool(torch.isfinite(y[7]).any())
    dx, dw, db = n.backward(g, x, mean, rstd)
    assert bool(torch.isfinite(dx[~bad]).all()) and bool(torch.isnan(dx[9]).all())
    assert bool(torch.isnan(dw).any()) and bool(torch.isfinite(db).all())


@pytest.mark.parametrize("dtype,dim", [(F32, 24), (F32, 133)])
def test_gradient_against_differences(dtype, dim):
    """<dx, u> + <dw, v> + <db, t> is the slope of <c, y> along (u, v, t), taken from the 64-bit forward."""
    n = norm(dim)
    x, c, w, b = (randn(s, dtype, k) for k, s in enumerate([(6, dim), (6, dim), (dim,), (dim,)]))
    du, dv, dt = (randn(s, dtype, 9 + k).double() for k, s in enumerate([(6, dim), (dim,), (dim,)]))
    y, mean, rstd = n.forward(x, w, b)
    dx, dw, db = n.backward(c, x, mean, rstd, w)

    def value(h):
        xx = x.double() + h * du
        m = xx.mean(1, keepdim=True)
        r = ((xx - m).square().mean(1, keepdim=True) + EPS).rsqrt()
        return ((xx - m) * r * (w.double() + h * dv) + b.double() + h * dt).mul(c.double()).sum()

    h = 1e-4
    slope = (value(h) - value(-h)) / (2 * h)
    got = (dx.double() * du).sum() + (dw.double() * dv).sum() + (db.double() * dt).sum()
    _, (ex, ew, eb) = tu.norm_backward(c, x, mean, rstd, w)
    # the kernel's bound; its statistics' roundings (a few u of each row's terms); the difference quotient's own h^2 term
    bound = (ex * du.abs()).sum() + (ew * dv.abs()).sum() + (eb * dt.abs()).sum()
    bound += 200 * tu.u * ((dx.double() * du).abs().sum() + (dw.double() * dv).abs().sum() + (c.double().abs() * rstd[:, None]).sum() * 10)
    bound += h * h * 100 * (c.double().abs() * w.double().abs()).sum()
    assert abs(float(got - slope)) <= float(bound)


def test_side_stream_and_shared_handle():
    n = norm(256)
    s = torch.cuda.Stream()
    cases = [(randn((1000 + 100 * k, 256), F32, k), randn((1000 + 100 * k, 256), F32, 9 + k)) for k in range(4)]
    w = randn((256,), F32, 99)
    s.wait_stream(torch.cuda.current_stream())
    got = []
    for x, g in cases:
        y, mean, rstd = n.forward(x, w, stream=s)
        got.append((mean, rstd) + n.backward(g, x, mean, rstd, w, stream=s))
    s.synchronize()
    for (x, g), (mean, rstd, dx, dw, db) in zip(cases, got):
        (wx, ww, wb), (ex, ew, eb) = tu.norm_backward(g, x, mean, rstd, w)
        tu.check(dx, wx, tu.out_tol(ex, wx, F32))
        tu.check(dw, ww, tu.out_tol(ew, ww, F32))
        tu.check(db, wb, tu.out_tol(eb, wb, F32))


def test_graph_capture():
    n = norm(320)
    x, g, w = randn((500, 320), BF16, 1), randn((500, 320), BF16, 2), randn((320,), F32, 3)
    out = torch.empty_like(x)
    dx, dw, db = torch.empty_like(x), torch.empty(320, device=DEV), torch.empty(320, device=DEV)
    _, mean, rstd = n.forward(x, w, out=out)
    n.backward(g, x, mean, rstd, w, dx=dx, dweight=dw, dbias=db)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, mean, rstd = n.forward(x, w, out=out)
        n.backward(g, x, mean, rstd, w, dx=dx, dweight=dw, dbias=db)
    x.copy_(randn((500, 320), BF16, 7))
    g.copy_(randn((500, 320), BF16, 8))
    graph.replay()
    (wy, _, _), (ey, _, _) = tu.norm_forward(x, w, None, EPS)
    tu.check(out, wy, tu.out_tol(ey, wy, BF16))
    (wx, ww, wb), (ex, ew, eb) = tu.norm_backward(g, x, mean, rstd, w)
    tu.check(dx, wx, tu.out_tol(ex, wx, BF16))
    tu.check(dw, ww, tu.out_tol(ew, ww, F32))
    tu.check(db, wb, tu.out_tol(eb, wb, F32))


def test_refusals():
    from powersgd_rank_gradient_gb300 import LayerNorm
    from powersgd_rank_gradient_gb300._lib import PsgdError

    n = norm(16)
    x, w = randn((8, 16), F32, 1), randn((16,), F32, 2)
    y, mean, rstd = n.forward(x, w)
    with pytest.raises(PsgdError, match="dim"):
        LayerNorm(0, device=DEV)
    with pytest.raises(PsgdError, match="eps"):
        norm(16, eps=-1.0).forward(x)
    with pytest.raises(PsgdError, match="eps"):
        norm(16, eps=float("nan")).forward(x)
    with pytest.raises(ValueError, match="x must"):
        n.forward(x.double())
    with pytest.raises(ValueError, match="last dimension"):
        n.forward(x[:, :8])
    with pytest.raises(ValueError, match="last dimension"):
        n.forward(x.t().contiguous().t())
    with pytest.raises(ValueError, match="cuda"):
        n.forward(x.cpu())
    with pytest.raises(ValueError, match="weight"):
        n.forward(x, w[:8])
    with pytest.raises(ValueError, match="one type"):
        n.forward(x, w, w.half())
    with pytest.raises(ValueError, match="out"):
        n.forward(x, w, out=torch.empty(8, 16, dtype=F16, device=DEV))
    with pytest.raises(PsgdError, match="overlap"):
        n.forward(x, w, out=x)
    with pytest.raises(ValueError, match="grad"):
        n.backward(x[:4], x, mean, rstd, w)
    with pytest.raises(ValueError, match="mean"):
        n.backward(x, x, mean[:4], rstd, w)
    with pytest.raises(ValueError, match="accumulate"):
        n.backward(x, x, mean, rstd, w, accumulate=True)
    with pytest.raises(PsgdError, match="overlap"):
        n.backward(y, x, mean, rstd, w, dx=y)
    with pytest.raises(PsgdError, match="overlap"):
        d = torch.empty(16, device=DEV)
        n.backward(y, x, mean, rstd, w, dweight=d, dbias=d)
    n.close()
    with pytest.raises(PsgdError, match="NULL"):
        n.forward(x)
