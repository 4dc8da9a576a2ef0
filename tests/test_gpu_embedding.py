"""Embedding lookup and table gradient against their 64-bit definitions."""

import pytest

import training_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(shape, dtype, seed, std=1.0):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0, std, generator=gen(seed))


def make_ids(shape, vocab, seed, dtype=torch.int64, hot=0.0):
    ids = torch.randint(0, vocab, shape, device=DEV, generator=gen(seed))
    if hot:
        ids = torch.where(torch.rand(shape, device=DEV, generator=gen(seed + 1)) < hot, vocab // 2, ids)
    return ids.to(dtype)


def embedding(vocab, dim, tokens, **kw):
    from powersgd_rank_gradient_gb300 import Embedding

    return Embedding(vocab, dim, tokens, device=DEV, **kw)


def guarded(vocab, dim, dtype, offset, fill=7.0, tail=37):
    """A bucket with a (vocab, dim) view ``offset`` elements in."""
    bucket = torch.full((offset + vocab * dim + tail,), fill, dtype=dtype, device=DEV)
    return bucket, bucket[offset:offset + vocab * dim].view(vocab, dim)


def untouched(bucket, offset, n, fill=7.0):
    assert bool((bucket[:offset] == fill).all()) and bool((bucket[offset + n:] == fill).all())


# -- lookup ------------------------------------------------------------------------

@pytest.mark.parametrize("wdtype", tu.DTYPES)
@pytest.mark.parametrize("odtype", tu.DTYPES)
@pytest.mark.parametrize("dim", [1, 7, 8, 64, 1023, 1600])
def test_lookup_types_and_widths(wdtype, odtype, dim):
    e = embedding(301, dim, 66, scale=0.75)
    w = randn((301, dim), wdtype, dim)
    ids = make_ids((3, 22), 301, 5)
    out = e.forward(w, ids, out_dtype=odtype)
    want = w.double()[ids] * 0.75
    tu.check(out, want, tu.out_tol(tu.u * want.abs(), want, odtype))
    assert out.dtype == odtype and not e.status()


@pytest.mark.parametrize("shape", [(), (1,), (0,), (5,), (1, 1), (4, 0), (2, 3, 5)])
@pytest.mark.parametrize("iddtype", [torch.int32, torch.int64])
def test_lookup_token_shapes(shape, iddtype):
    e = embedding(50, 96, 64, scale=2.0)
    w = randn((50, 96), F32, 1)
    ids = make_ids(shape, 50, 2, iddtype)
    out = e.forward(w, ids)
    assert out.shape == shape + (96,)
    assert torch.equal(out, w[ids.long()] * 2.0)


def test_lookup_strides():
    """Ids, table and output that are views of larger tensors, and an output at an odd element."""
    e = embedding(40, 24, 100)
    big = randn((40, 64), BF16, 3)
    base = make_ids((7, 30), 40, 4)
    for ids in (base[:, :-1][:, :14], base[:, ::3], base.t(), base[2], base[::2, 5:9], base[:1].expand(3, 30)):
        for w in (big[:, :24], big[:, 3:27], big[:, 8:32]):
            out = e.forward(w, ids) if ids.numel() <= 100 else None
            if out is None:
                with pytest.raises(Exception, match="max_tokens"):
                    e.forward(w, ids)
                continue
            assert torch.equal(out, w[ids])
    room = torch.full((7 * 5 * 40 + 11,), 9.0, dtype=BF16, device=DEV)
    view = room[3:3 + 7 * 5 * 40].view(7, 5, 40)[:, :, 1:25]
    e.forward(big[:, :24], base[:, :5], out=view)
    assert torch.equal(view, big[:, :24][base[:, :5]])
    view.fill_(9.0)
    assert bool((room == 9.0).all())


def test_lookup_out_of_range_ids_read_zero_and_are_reported():
    e = embedding(10, 16, 8)
    w = randn((10, 16), F32, 1)
    ids = torch.tensor([3, -1, 9, 10, 2**40, -2**40, 0, 5], device=DEV)
    out = e.forward(w, ids)
    good = (ids >= 0) & (ids < 10)
    assert torch.equal(out, torch.where(good[:, None], w[ids.clamp(0, 9)], 0.0))
    assert e.status() and not e.status()
    e.forward(w, ids[:1])
    assert not e.status()


def test_lookup_one_large_table():
    e = embedding(50257, 1600, 2048)
    w = randn((50257, 1600), F16, 11)
    ids = make_ids((2, 1024), 50257, 12)
    assert torch.equal(e.forward(w, ids), w[ids])
    assert torch.equal(e.forward(w, ids[:1, 77:78]), w[ids[:1, 77:78]])


@pytest.mark.parametrize("dim", [1024, 1031])
@pytest.mark.parametrize("tokens", [100, 3000])
def test_offsets_beyond_32_bits(dim, tokens):
    """A table of more than 2^31 elements, read and written at both ends and in the middle."""
    vocab = 2**31 // dim + 77
    e = embedding(vocab, dim, tokens)
    w = torch.zeros((vocab, dim), dtype=BF16, device=DEV)
    rows = torch.cat([torch.arange(9), torch.arange(vocab // 2, vocab // 2 + 9), torch.arange(vocab - 9, vocab)]).to(DEV)
    w[rows] = randn((27, dim), BF16, 1)
    pick = torch.randint(0, 27, (tokens,), device=DEV, generator=gen(2))
    out = e.forward(w, rows[pick])
    assert torch.equal(out, w[rows][pick])
    grad = randn((tokens, dim), BF16, 3)
    w.fill_(3.0)
    e.backward(rows[pick], grad, out=w)
    dw, mag, count = tu.table_grad(pick, grad, 27, 1.0)
    tu.check(w[rows], dw, tu.table_grad_tol(dw, mag, count, BF16))
    assert int(torch.count_nonzero(w[9:vocab // 2:97])) == 0 and int(torch.count_nonzero(w[vocab // 2 + 9:vocab - 9:97])) == 0
    assert not e.status()


# -- gradient ------------------------------------------------------------------------

def run_grad(vocab, dim, shape, gdtype, odtype, seed, iddtype=torch.int64, hot=0.0, padding=None, scale=1.0, offset=0,
             accumulate=False):
    e = embedding(vocab, dim, max(1, torch.Size(shape).numel()), padding_idx=padding, scale=scale)
    ids = make_ids(shape, vocab, seed, iddtype, hot)
    grad = randn(tuple(shape) + (dim,), gdtype, seed + 2)
    bucket, view = guarded(vocab, dim, odtype, offset)
    before = None
    if accumulate:
        before = randn((vocab, dim), odtype, seed + 3)
        view.copy_(before)
    got = e.backward(ids, grad, out=view, accumulate=accumulate)
    assert got is view
    dw, mag, count = tu.table_grad(ids, grad, vocab, scale, padding, before)
    tu.check(view, dw, tu.table_grad_tol(dw, mag, count, odtype))
    untouched(bucket, offset, vocab * dim)
    assert not e.status()
    first = view.clone()
    if accumulate:
        view.copy_(before)
    else:
        view.fill_(-3.0)
    e.backward(ids, grad, out=view, accumulate=accumulate)
    assert torch.equal(first, view), "another result from the same inputs"


@pytest.mark.parametrize("gdtype", tu.DTYPES)
@pytest.mark.parametrize("odtype", tu.DTYPES)
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_types(gdtype, odtype, accumulate):
    run_grad(97, 136, (3, 71), gdtype, odtype, 1, scale=1.5, accumulate=accumulate)


@pytest.mark.parametrize("tokens", [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 1025, 4097])
@pytest.mark.parametrize("vocab", [1, 2, 300])
def test_grad_token_counts(tokens, vocab):
    """Chunk ends on and beside the token count; tables of one and two rows, whose rows span every chunk."""
    run_grad(vocab, 40, (tokens,), F32, F32, tokens + vocab, iddtype=torch.int32)


@pytest.mark.parametrize("dim,offset", [(1, 0), (3, 1), (8, 0), (8, 4), (64, 3), (255, 0), (257, 2), (1023, 0), (1024, 8),
                                        (1600, 5), (2050, 0)])
@pytest.mark.parametrize("odtype", [F32, BF16])
def test_grad_widths_and_bucket_offsets(dim, offset, odtype):
    run_grad(77, dim, (5, 53), BF16, odtype, dim + offset, offset=offset, hot=0.3)


@pytest.mark.parametrize("vocab", [255, 256, 257, 1023, 1024, 1025, 65535, 65536, 65537, 70001])
@pytest.mark.parametrize("tokens", [700, 2047, 2048, 2049, 9 * 301, 16384, 16385, 20000])
def test_grad_table_sizes(vocab, tokens):
    """One, two and three radix passes, of 8 bits and of 10, on one CTA and on a cluster, in registers and not."""
    run_grad(vocab, 8, (tokens,), F16, F32, vocab, padding=vocab // 3)


@pytest.mark.parametrize("hot", [0.5, 1.0])
@pytest.mark.parametrize("padding", [None, 500])
def test_grad_hot_row(hot, padding):
    """Most tokens name one row (the padding's, or one that counts)."""
    run_grad(1000, 72, (40, 333), BF16, F32, 3, hot=hot, padding=padding)


def test_grad_large():
    run_grad(30522, 1024, (32, 512), F32, F32, 8, hot=0.1, padding=0, scale=32.0)
    run_grad(50257, 1600, (4, 1024), BF16, BF16, 9, iddtype=torch.int32, offset=1)


@pytest.mark.parametrize("vocab", [1, 33, 300, 512, 1217, 2500, 30522, 50257])
@pytest.mark.parametrize("tokens,hot", [(1, 0), (15, 0.5), (17, 1.0), (100, 0.9), (1000, 0.3), (4096, 0.05), (8192, 0.6)])
def test_grad_few_tokens(vocab, tokens, hot):
    """One launch or the sorted list, rows of one token and of most of them."""
    run_grad(vocab, 24, (tokens,), BF16, F32, vocab, hot=hot, padding=vocab - 1 if vocab > 1 else None, offset=3)
    run_grad(vocab, 17, (tokens,), F32, F16, vocab, hot=hot, accumulate=True)


def test_grad_many_tokens():
    run_grad(5000, 8, (300, 1001), F16, F32, 4, hot=0.05)
    run_grad(1000, 4, (300, 1001), F16, F32, 5, hot=0.9)
    run_grad(777, 8, (262, 1001), F16, F32, 6, hot=0.5, padding=5)
    run_grad(2, 8, (1, 200001), F32, F32, 7)


@pytest.mark.parametrize("tokens", [3000, 65536, 65537, 150000])
def test_grad_of_tall_tables(tokens):
    """Tables of far more rows than tokens, and rows of one element: every row that no token names is zero."""
    run_grad(200003, 1, (tokens,), F32, F32, 1, offset=1)
    run_grad(70001, 3, (tokens,), BF16, F16, 2, offset=3, hot=0.4, padding=0)
    run_grad(30522, 40, (tokens,), F32, F32, 3, iddtype=torch.int32)


def test_grad_of_padding_only():
    run_grad(300, 24, (3, 50), F32, F32, 1, hot=1.0, padding=150)
    run_grad(300, 24, (3000,), F32, F32, 1, hot=1.0, padding=150)
    run_grad(30000, 24, (3000,), F32, F32, 1, hot=1.0, padding=15000, accumulate=True)


def test_grad_strides_and_broadcast():
    e = embedding(60, 32, 400, scale=0.5)
    base = make_ids((8, 41), 60, 1)
    big = randn((8, 41, 80), F32, 2)
    odd = randn((8, 41, 33), F32, 3)
    for ids, grad in ((base[:, :-1], big[:, 1:, :32]), (base[:, ::2], big[:, ::2, 40:72]), (base, odd[:, :, 1:]),
                      (base, big[:1, :1, :32].expand(8, 41, 32)), (base.t(), big.transpose(0, 1)[:, :, 4:36])):
        room = torch.full((60, 50), 5.0, device=DEV)
        out = e.backward(ids, grad, out=room[:, 7:39])
        dw, mag, count = tu.table_grad(ids, grad, 60, 0.5)
        tu.check(out, dw, tu.table_grad_tol(dw, mag, count, F32))
        assert bool((room[:, :7] == 5.0).all()) and bool((room[:, 39:] == 5.0).all())


@pytest.mark.parametrize("vocab", [513, 1025, 66000])
@pytest.mark.parametrize("tokens", [8192, 8193, 32768, 32769, 100000])
def test_grad_sort_sizes(vocab, tokens):
    run_grad(vocab, 12, (tokens,), F32, F32, 1, hot=0.1, padding=3)


@pytest.mark.parametrize("gdtype", tu.DTYPES)
@pytest.mark.parametrize("dim", [5, 33, 513, 1025, 2100])
@pytest.mark.parametrize("tokens", [1300, 12000])
def test_grad_rows_between_other_values(gdtype, dim, tokens):
    """Gradient rows of every alignment, as columns of an array whose other columns are NaN."""
    e = embedding(1500, dim, tokens)
    ids = make_ids((tokens,), 1500, 1, hot=0.1)
    for first in (1, 7):
        room = torch.full((tokens + 1, dim + 10), float("nan"), dtype=gdtype, device=DEV)
        grad = room[1:, first:first + dim]
        grad.copy_(randn((tokens, dim), gdtype, 2 + first))
        bucket, view = guarded(1500, dim, F32, 1)
        e.backward(ids, grad, out=view)
        dw, mag, count = tu.table_grad(ids, grad, 1500, 1.0)
        tu.check(view, dw, tu.table_grad_tol(dw, mag, count, F32))
        untouched(bucket, 1, 1500 * dim)
    flat = torch.full((tokens * dim + 9,), float("nan"), dtype=gdtype, device=DEV)
    grad = flat[1:1 + tokens * dim].view(tokens, dim)  # the first row begins within the first granule
    grad.copy_(randn((tokens, dim), gdtype, 5))
    dw, mag, count = tu.table_grad(ids, grad, 1500, 1.0)
    tu.check(e.backward(ids, grad), dw, tu.table_grad_tol(dw, mag, count, F32))


def test_grad_out_of_range_ids_add_nothing_and_are_reported():
    e = embedding(10, 16, 100)
    ids = torch.tensor([3, -1, 9, 10, 2**33 + 3, -2**31 - 1, 0, 3], device=DEV)
    grad = randn((8, 16), F32, 1)
    out = e.backward(ids, grad)
    dw, mag, count = tu.table_grad(ids, grad, 10, 1.0)
    tu.check(out, dw, tu.table_grad_tol(dw, mag, count, F32))
    assert e.status() and not e.status()


@pytest.mark.parametrize("bad", [-1, 10, 2**32, -2**31])
@pytest.mark.parametrize("tokens", [9, 5000])
def test_grad_reports_a_single_bad_id(bad, tokens):
    for padding in (None, 4):
        e = embedding(10, 8, tokens, padding_idx=padding)
        ids = make_ids((tokens,), 10, 1)
        grad = randn((tokens, 8), F32, 2)
        e.backward(ids, grad)
        assert not e.status()
        ids[tokens // 2] = bad
        out = e.backward(ids, grad)
        dw, mag, count = tu.table_grad(ids, grad, 10, 1.0, padding)
        tu.check(out, dw, tu.table_grad_tol(dw, mag, count, F32))
        assert e.status()


def test_grad_keeps_nonfinite_rows_apart():
    """An infinity or NaN in one token's gradient reaches that token's row only; in padding it reaches none."""
    e = embedding(20, 24, 400, padding_idx=7)
    ids = make_ids((400,), 20, 3)
    ids[5], ids[6], ids[7] = 2, 11, 7
    grad = randn((400, 24), F32, 4)
    grad[5, 3], grad[6, 20] = float("inf"), float("nan")
    grad[ids == 7] = float("nan")
    out = e.backward(ids, grad)
    dw, mag, count = tu.table_grad(ids, grad, 20, 1.0, padding=7)
    tu.check(out, dw, torch.nan_to_num(tu.table_grad_tol(dw, mag, count, F32), posinf=0.0))
    assert bool((out[7] == 0).all())


def test_grad_against_differences():
    """<dW, V> is the change of <g, lookup(W)> along V (linear in W, so exact up to rounding)."""
    e = embedding(31, 12, 90, scale=3.0)
    ids = make_ids((90,), 31, 1)
    g = randn((90, 12), F32, 2)
    w, v = randn((31, 12), F32, 3), randn((31, 12), F32, 4)
    h = 2.0 ** -6
    up, down = e.forward(w + h * v, ids).double(), e.forward(w - h * v, ids).double()
    slope = ((up - down) / (2 * h) * g.double()).sum()
    dw = e.backward(ids, g).double()
    # each value carries a few roundings of its size, divided by the step
    bound = (4 * tu.u * (up.abs() + down.abs()) / (2 * h) * g.double().abs()).sum() + 100 * tu.u * (dw * v.double()).abs().sum()
    assert abs(float((dw * v.double()).sum() - slope)) <= float(bound)


def test_side_stream_and_alternating_inputs():
    e = embedding(500, 64, 3000)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs, wants = [], []
    for k in range(4):
        ids, grad = make_ids((3000 - 700 * k,), 500, k), randn((3000 - 700 * k, 64), F32, 50 + k)
        s.wait_stream(torch.cuda.current_stream())
        outs.append(e.backward(ids, grad, stream=s))
        wants.append((ids, grad))
    s.synchronize()
    for out, (ids, grad) in zip(outs, wants):
        dw, mag, count = tu.table_grad(ids, grad, 500, 1.0)
        tu.check(out, dw, tu.table_grad_tol(dw, mag, count, F32))


def test_graph_capture():
    e = embedding(300, 64, 2000)
    ids, grad = make_ids((2000,), 300, 1), randn((2000, 64), F32, 2)
    out = torch.empty((300, 64), device=DEV)
    e.backward(ids, grad, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e.backward(ids, grad, out=out)
    for k in range(2):
        ids.copy_(make_ids((2000,), 300, 10 + k))
        grad.copy_(randn((2000, 64), F32, 20 + k))
        out.fill_(1.0)
        graph.replay()
        dw, mag, count = tu.table_grad(ids, grad, 300, 1.0)
        tu.check(out, dw, tu.table_grad_tol(dw, mag, count, F32))


def test_refusals():
    from powersgd_rank_gradient_gb300 import Embedding
    from powersgd_rank_gradient_gb300._lib import PsgdError

    e = embedding(10, 16, 8)
    w = randn((10, 16), F32, 1)
    ids = make_ids((8,), 10, 2)
    g = randn((8, 16), F32, 3)
    with pytest.raises(ValueError, match="padding_idx"):
        embedding(10, 16, 8, padding_idx=10)
    with pytest.raises(PsgdError, match="vocab"):
        Embedding(0, 16, 8, device=DEV)
    with pytest.raises(PsgdError, match="dim"):
        Embedding(10, 0, 8, device=DEV)
    with pytest.raises(ValueError, match="CUDA"):
        Embedding(10, 16, 8, device="cpu")
    with pytest.raises(ValueError, match="ids"):
        e.forward(w, ids.float())
    with pytest.raises(ValueError, match="weight"):
        e.forward(w.double(), ids)
    with pytest.raises(ValueError, match="weight"):
        e.forward(w[:, :8], ids)
    with pytest.raises(ValueError, match="weight"):
        e.forward(w.t().contiguous().t(), ids)
    with pytest.raises(ValueError, match="cuda"):
        e.forward(w.cpu(), ids)
    with pytest.raises(ValueError, match="out"):
        e.forward(w, ids, out=torch.empty(7, 16, device=DEV))
    with pytest.raises(PsgdError, match="max_tokens"):
        e.forward(w, torch.zeros(9, dtype=torch.int64, device=DEV))
    with pytest.raises(PsgdError, match="max_tokens"):
        e.backward(torch.zeros(9, dtype=torch.int64, device=DEV), randn((9, 16), F32, 4))
    with pytest.raises(PsgdError, match="overlap"):
        e.forward(w, ids, out=w[:8])
    with pytest.raises(PsgdError, match="overlap"):
        e.forward(w, ids, out=torch.empty(16, device=DEV).expand(8, 16))
    with pytest.raises(PsgdError, match="overlap"):
        big = torch.empty(10 * 16 + 40, device=DEV)
        e.backward(ids, big[40:168].view(8, 16), out=big[:160].view(10, 16))
    with pytest.raises(ValueError, match="grad"):
        e.backward(ids, g[:, :8])
    with pytest.raises(ValueError, match="accumulate"):
        e.backward(ids, g, accumulate=True)
    assert not e.status()
    e.close()
    with pytest.raises(PsgdError, match="NULL"):
        e.forward(w, ids)
