"""Layer norm's C calls with the outputs a caller chooses (the Python face passes all of them)."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
CODES = {F32: 0, F16: 1, BF16: 2}


def randn(shape, seed, dtype=F32, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0, std, generator=g)


def at(t):
    return None if t is None else t.data_ptr()


def forward(n, x, w, b, y, mean, rstd):
    from powersgd_rank_gradient_gb300 import _lib

    return _lib.lib().psgd_layernorm_forward(n._h, at(x), CODES[x.dtype], x.shape[1], x.shape[0], at(w), at(b), 0, n.eps, at(y),
                                             x.shape[1], at(mean), at(rstd), torch.cuda.current_stream().cuda_stream)


def test_statistics_overlap_nothing():
    from powersgd_rank_gradient_gb300 import LayerNorm, _lib

    n = LayerNorm(16, device=DEV)
    x, w, b = randn((8, 16), 1), randn((16,), 2), randn((16,), 3)
    y, stats = torch.empty((8, 16), device=DEV), torch.empty(16, device=DEV)
    mean, rstd = stats[:8], stats[8:]
    assert forward(n, x, w, b, y, mean, rstd) == _lib.PSGD_OK
    want = n.forward(x, w, b)
    assert torch.equal(y, want[0]) and torch.equal(mean, want[1]) and torch.equal(rstd, want[2])
    before = [t.clone() for t in (x, w, b)]
    for m, r in ((mean, stats[7:]), (stats[4:], mean), (mean, mean), (x[3], rstd), (mean, x[7]), (w, rstd), (mean, w[9:]),
                 (b, rstd), (mean, b), (y[2], rstd), (mean, y[7])):
        assert forward(n, x, w, b, y, m, r) == _lib.PSGD_EINVAL
        assert "overlap" in _lib.lib().psgd_last_error().decode()
    assert all(torch.equal(s, t) for s, t in zip(before, (x, w, b)))


def backward(n, grad, x, mean, rstd, w, dx, dw, db):
    from powersgd_rank_gradient_gb300 import _lib

    dim = x.shape[1]
    return _lib.lib().psgd_layernorm_backward(n._h, at(grad), dim, at(x), CODES[x.dtype], dim, x.shape[0], at(mean), at(rstd), at(w),
                                              0, at(dx), dim, at(dw), at(db), 0, 0, torch.cuda.current_stream().cuda_stream)


# rows of whole 16-byte units, of any length, and too long for registers
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim", [64, 1600, 333, 1023, 20000])
@pytest.mark.parametrize("rows", [0, 1, 3, 1300])
def test_outputs_that_are_left_out(dtype, dim, rows):
    """Whatever is left out, the others are the same bits."""
    from powersgd_rank_gradient_gb300 import LayerNorm, _lib

    n = LayerNorm(dim, device=DEV)
    x, g, w, b = randn((rows, dim), 1, dtype, 1.5), randn((rows, dim), 2, dtype), randn((dim,), 3), randn((dim,), 4)
    want = n.forward(x, w, b)
    for keep in ((0, 0), (1, 0), (0, 1)):
        y = torch.full_like(want[0], 3.0)
        stats = [torch.full_like(want[1 + i], 3.0) if keep[i] else None for i in range(2)]
        assert forward(n, x, w, b, y, *stats) == _lib.PSGD_OK
        assert torch.equal(y, want[0]) and all(s is None or torch.equal(s, want[1 + i]) for i, s in enumerate(stats))
    grads = n.backward(g, x, want[1], want[2], w)
    for keep in range(8):
        outs = [torch.full_like(t, 3.0) if keep >> i & 1 else None for i, t in enumerate(grads)]
        assert backward(n, g, x, want[1], want[2], w, *outs) == _lib.PSGD_OK
        assert all(o is None or torch.equal(o, t) for o, t in zip(outs, grads)), keep
