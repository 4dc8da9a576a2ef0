"""Distillation from a teacher's top logits against its 64-bit definition."""

import pytest

import training_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def distill(*a, **kw):
    from powersgd_rank_gradient_gb300 import distill_loss

    return distill_loss(*a, **kw)


def inputs(rows, vocab, k, dtype, tdtype, idtype, seed, ragged=True, std=2.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    z = torch.empty((rows, vocab), dtype=dtype, device=DEV).normal_(0, std, generator=g)
    t = torch.empty((rows, k), dtype=tdtype, device=DEV).normal_(3, 2, generator=g)
    at = torch.randint(0, vocab, (rows, k), device=DEV, generator=g)
    if ragged:
        kept = torch.randint(0, k + 1, (rows, 1), device=DEV, generator=g)
        at = torch.where(torch.arange(k, device=DEV) < kept, at, -1)
    return z, t, at.to(idtype)


def verify(z, t, at, temperature=1.0, weights=None, grad_scale=1.0, **kw):
    losses, dz = distill(z, t, at, temperature=temperature, weights=weights, grad_scale=grad_scale, **kw)
    (wl, wz), (el, ez) = tu.distill(z.reshape(-1, z.shape[-1]), t.reshape(-1, t.shape[-1]), at.reshape(-1, at.shape[-1]),
                                    temperature, None if weights is None else weights.reshape(-1), grad_scale)
    tu.check(losses.reshape(-1), wl, tu.out_tol(el, wl, F32))
    tu.check(dz.reshape(-1, z.shape[-1]), wz, tu.out_tol(ez, wz, z.dtype))
    only, none = distill(z, t, at, temperature=temperature, weights=weights, with_grad=False)
    assert none is None and torch.equal(torch.nan_to_num(only), torch.nan_to_num(losses))
    again, dz2 = distill(z, t, at, temperature=temperature, weights=weights, grad_scale=grad_scale)
    assert torch.equal(torch.nan_to_num(again), torch.nan_to_num(losses))
    assert torch.equal(torch.nan_to_num(dz2), torch.nan_to_num(dz)), "another result from the same inputs"
    return losses, dz


@pytest.mark.parametrize("dtype", tu.DTYPES)
@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 8, 9, 31, 100, 255, 1000, 1001, 4099, 30522, 50257, 50304])
def test_vocabularies(vocab, dtype):
    verify(*inputs(9, vocab, min(vocab, 20), dtype, F32, torch.int64, vocab), temperature=2.0, grad_scale=4.0)


@pytest.mark.parametrize("dtype", tu.DTYPES)
@pytest.mark.parametrize("vocab", [65537, 131072, 200003, 500009])
def test_rows_larger_than_shared_memory(vocab, dtype):
    verify(*inputs(3, vocab, 50, dtype, F32, torch.int32, vocab))


@pytest.mark.parametrize("rows", [0, 1, 2, 5, 19, 38, 76, 151, 152, 153, 305, 1000])
@pytest.mark.parametrize("vocab,dtype", [(333, F32), (5001, BF16)])
def test_row_counts(rows, vocab, dtype):
    verify(*inputs(rows, vocab, 8, dtype, F16, torch.int32, rows))


@pytest.mark.parametrize("k", [1, 2, 31, 32, 33, 100, 511, 513, 1024])
def test_entries(k):
    """Up to the largest k; far more entries than vocabulary, so that most indices repeat."""
    verify(*inputs(11, 1500, k, F32, F32, torch.int64, k))
    verify(*inputs(11, 40, k, BF16, F32, torch.int32, k + 1, ragged=False))


@pytest.mark.parametrize("tdtype", tu.DTYPES)
@pytest.mark.parametrize("idtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("temperature", [0.5, 1.0, 7.5])
def test_teacher_types_and_temperatures(tdtype, idtype, temperature):
    z, t, at = inputs(40, 777, 12, F32, tdtype, idtype, 3)
    w = torch.rand(40, device=DEV)
    verify(z, t, at, temperature, w, 128.0)


def test_large():
    verify(*inputs(1200, 50257, 64, BF16, BF16, torch.int32, 1), temperature=1.5, grad_scale=1024.0)
    verify(*inputs(700, 30522, 32, F32, F16, torch.int64, 2), temperature=2.0)


@pytest.mark.parametrize("dtype", tu.DTYPES)
@pytest.mark.parametrize("vocab,width,first", [(1001, 1024, 0), (1000, 1024, 8), (997, 1003, 5), (50257, 50304, 0), (6, 11, 3)])
def test_strides_and_padding_stay(dtype, vocab, width, first):
    """Logits that are the front or the middle of wider rows; the gradient into such rows too, and in place."""
    z, t, at = inputs(10, vocab, 6, dtype, F32, torch.int64, 5)
    room = torch.full((10, width), 3.0, dtype=dtype, device=DEV)
    room[:, first:first + vocab] = z
    grads = torch.full((10, width), 5.0, dtype=dtype, device=DEV)
    wide_t, wide_at = torch.zeros((10, 13), device=DEV), torch.zeros((10, 17), dtype=torch.int64, device=DEV)
    wide_t[:, 2:8], wide_at[:, 9:15] = t, at
    view, out = room[:, first:first + vocab], grads[:, first:first + vocab]
    losses, dz = verify(view, wide_t[:, 2:8], wide_at[:, 9:15], 1.25)
    distill(view, wide_t[:, 2:8], wide_at[:, 9:15], 1.25, dlogits=out)
    assert torch.equal(out, dz)
    l2, same = distill(view, t, at, 1.25, dlogits=view)
    assert same is view and torch.equal(view, dz) and torch.equal(l2, losses)
    for x, fill in ((room, 3.0), (grads, 5.0)):
        assert bool((x[:, :first] == fill).all()) and bool((x[:, first + vocab:] == fill).all())


def test_leading_dimensions():
    z, t, at = inputs(12, 90, 5, F32, F32, torch.int64, 1)
    losses, dz = distill(z.view(3, 4, 90), t.view(3, 4, 5), at.view(3, 4, 5), weights=torch.ones(3, 4, device=DEV))
    l2, d2 = distill(z, t, at)
    assert losses.shape == (3, 4) and torch.equal(losses.view(12), l2) and torch.equal(dz.view(12, 90), d2)
    l3, d3 = distill(z[0], t[0], at[0])
    assert l3.shape == () and torch.equal(l3, l2[0]) and torch.equal(d3, d2[0])


@pytest.mark.parametrize("dtype", tu.DTYPES)
@pytest.mark.parametrize("vocab", [50, 4097])
def test_masked_rows_read_nothing(dtype, vocab):
    """Weight 0, no valid entry, entries of -infinity only: loss and gradient are 0, NaN in the logits or not."""
    z, t, at = inputs(12, vocab, 6, dtype, F32, torch.int64, 5, ragged=False)
    w = torch.ones(12, device=DEV)
    w[2] = 0.0
    at[5] = -1
    at[6, :3], at[6, 3:] = -7, vocab + 3
    t[8] = -torch.inf
    at[9, 1:] = -1
    t[10, ::2] = -torch.inf
    verify(z, t, at, 1.5, w)
    for r in (2, 5, 6, 8):
        z[r] = float("nan")
    losses, dz = distill(z, t, at, 1.5, w)
    for r in (2, 5, 6, 8):
        assert float(losses[r]) == 0.0 and bool((dz[r] == 0).all())
    assert bool(torch.isfinite(dz).all())


@pytest.mark.parametrize("dtype", tu.DTYPES)
def test_masked_vocabulary(dtype):
    """Logits of -infinity and of the type's lowest value, in a few places and in all but one."""
    z, t, at = inputs(8, 515, 4, dtype, F32, torch.int64, 6, ragged=False)
    low = torch.finfo(dtype).min
    z[0, :200], z[1, 300:], z[2, :], z[3, :], z[4, ::2] = -torch.inf, low, -torch.inf, low, -torch.inf
    z[2, 77], z[3, 78] = 1.0, 1.0
    at[0], at[1] = at[0] % 300 + 210, at[1] % 300
    at[2] = 77
    at[3] = 78
    at[4] = at[4] // 2 * 2 % 514 + 1
    losses, dz = verify(z, t, at, 2.0)
    assert bool(torch.isfinite(losses).all()) and bool(torch.isfinite(dz).all())
    at[0, 1] = 5  # the teacher wants a masked entry
    losses, dz = distill(z, t, at, 2.0)
    assert float(losses[0]) == float("inf") and bool(torch.isfinite(dz).all())


def test_nonfinite_logits_make_their_row_nan():
    for vocab in (100, 9001):
        z, t, at = inputs(8, vocab, 4, F32, F32, torch.int64, 7, ragged=False)
        _, clean = distill(z, t, at)
        z[1, 40], z[3, 41], z[5] = float("nan"), float("inf"), -torch.inf
        losses, dz = distill(z, t, at)
        for r in (1, 3, 5):
            assert bool(torch.isnan(losses[r])) and bool(torch.isnan(dz[r]).all())
        for r in (0, 2, 4, 6, 7):
            assert torch.equal(dz[r], clean[r])
        t[2, 1] = float("nan")
        losses, _ = distill(z, t, at)
        assert bool(torch.isnan(losses[2]))


def test_far_logits():
    """Logits of several hundred: the maximum is taken off before any exponential."""
    z, t, at = inputs(20, 3001, 10, F32, F32, torch.int64, 8, std=300.0)
    verify(z, t, at, 1.0)
    z, t, at = inputs(20, 3001, 10, F16, F32, torch.int64, 9, std=3000.0)
    verify(z, t * 50, at, 3.0)


@pytest.mark.parametrize("vocab,rows", [(100, 8), (60001, 8), (60001, 400)])
def test_rows_far_from_zero(vocab, rows):
    """Rows whose largest logit is enormous, on either side, beside ordinary ones."""
    z, t, at = inputs(rows, vocab, 7, F32, F32, torch.int64, 11, ragged=False)
    z[0] += 1e7
    z[1] -= 1e7
    z[2] = torch.finfo(F32).min
    z[3, 1:] -= 3e38
    z[4, ::3] = 1e30
    z[5, 7] = 2.0 ** 20
    z[6] = -torch.inf
    z[6, 9] = -1e9
    at[6] = 9
    at[3, 1:] = 0
    verify(z, t, at, 1.3)


def test_gradient_against_differences():
    """<dz, v> is the slope of the losses' sum along v, taken from the 64-bit losses."""
    z, t, at = inputs(6, 61, 9, F32, F32, torch.int64, 10)
    w = torch.rand(6, device=DEV)
    v = torch.randn(6, 61, device=DEV).double()
    for temperature in (1.0, 3.0):
        _, dz = distill(z, t, at, temperature, w)
        h = 1e-4
        up, down = (tu.distill(z.double() + s * h * v, t, at, temperature, w)[0][0].sum() for s in (1, -1))
        slope = (up - down) / (2 * h)
        _, (_, ez) = tu.distill(z, t, at, temperature, w)
        # the kernel's bound, and the quotient's h^2 term: third derivatives of log sum exp along v are below (2 max |v| / T)^3
        bound = (ez * v.abs()).sum() + tu.u * (dz.double() * v).abs().sum()
        bound += h * h * (w.sum() * temperature ** 2 * (2 * v.abs().max() / temperature) ** 3) + 1e-9
        assert abs(float((dz.double() * v).sum() - slope)) <= float(bound)


def test_offsets_beyond_32_bits():
    """More than 2^31 logits, in place; rows from both ends and the middle."""
    rows, vocab, k = 43001, 50257, 3
    z = torch.zeros((rows, vocab), dtype=BF16, device=DEV)
    part, t, at = inputs(90, vocab, k, BF16, F32, torch.int64, 15, ragged=False)
    places = torch.cat([torch.arange(30), torch.arange(21000, 21030), torch.arange(rows - 30, rows)]).to(DEV)
    z[places] = part
    teacher, index = torch.zeros((rows, k), device=DEV), torch.full((rows, k), -1, device=DEV)
    teacher[places], index[places] = t, at
    losses, dz = distill(z, teacher, index, dlogits=z)
    (wl, wz), (el, ez) = tu.distill(part, t, at, 1.0)
    tu.check(losses[places], wl, tu.out_tol(el, wl, F32))
    tu.check(dz[places], wz, tu.out_tol(ez, wz, BF16))
    others = torch.ones(rows, dtype=torch.bool, device=DEV)
    others[places] = False
    assert bool((losses[others] == 0).all()) and int(torch.count_nonzero(z[others.nonzero()[::400, 0]])) == 0


def test_side_stream():
    s = torch.cuda.Stream()
    z, t, at = inputs(300, 3000, 9, F32, F32, torch.int64, 11)
    s.wait_stream(torch.cuda.current_stream())
    losses, dz = distill(z, t, at, stream=s)
    s.synchronize()
    l2, d2 = distill(z, t, at)
    assert torch.equal(losses, l2) and torch.equal(dz, d2)


def test_graph_capture():
    z, t, at = inputs(100, 5000, 9, BF16, F32, torch.int64, 12)
    dz = torch.empty_like(z)
    distill(z, t, at, dlogits=dz)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        losses, _ = distill(z, t, at, dlogits=dz)
    z2, t2, at2 = inputs(100, 5000, 9, BF16, F32, torch.int64, 13)
    z.copy_(z2), t.copy_(t2), at.copy_(at2)
    graph.replay()
    l2, d2 = distill(z2, t2, at2)
    assert torch.equal(losses, l2) and torch.equal(dz, d2)


def test_refusals():
    from powersgd_rank_gradient_gb300._lib import PSGD_DISTILL_MAX_K, PsgdError

    z, t, at = inputs(4, 50, 6, F32, F32, torch.int64, 1)
    with pytest.raises(ValueError, match="CUDA"):
        distill(z.cpu(), t, at)
    with pytest.raises(ValueError, match="logits"):
        distill(z.double(), t, at)
    with pytest.raises(ValueError, match="teacher"):
        distill(z, t[:3], at)
    with pytest.raises(ValueError, match="teacher"):
        distill(z, t, at[:, :3])
    with pytest.raises(ValueError, match="teacher_indices"):
        distill(z, t, at.float())
    with pytest.raises(ValueError, match="cuda"):
        distill(z, t.cpu(), at)
    with pytest.raises(ValueError, match="last dimension"):
        distill(z.t().contiguous().t(), t, at)
    with pytest.raises(ValueError):
        distill(z, t[:, :0], at[:, :0])
    with pytest.raises(PsgdError, match="k must"):
        distill(z, t[:, :1].expand(4, PSGD_DISTILL_MAX_K + 1).contiguous(),
                at[:, :1].expand(4, PSGD_DISTILL_MAX_K + 1).contiguous())
    for bad in (0.0, -1.0, float("inf"), float("nan"), 1e-39):
        with pytest.raises(PsgdError, match="temperature"):
            distill(z, t, at, temperature=bad)
    with pytest.raises(ValueError, match="weights"):
        distill(z, t, at, weights=torch.ones(3, device=DEV))
    with pytest.raises(ValueError, match="weights"):
        distill(z, t, at, weights=torch.ones(4, device=DEV, dtype=F16))
    with pytest.raises(ValueError, match="dlogits"):
        distill(z, t, at, dlogits=torch.empty(4, 50, dtype=F16, device=DEV))
    with pytest.raises(ValueError, match="dlogits"):
        distill(z, t, at, dlogits=torch.empty_like(z), with_grad=False)
    room = torch.empty(5 * 50, device=DEV)
    with pytest.raises(PsgdError, match="overlap"):
        distill(room[:200].view(4, 50), t, at, dlogits=room[50:].view(4, 50))
    with pytest.raises(PsgdError, match="overlap"):
        distill(z, t, at, dlogits=torch.empty(50, device=DEV).expand(4, 50))
