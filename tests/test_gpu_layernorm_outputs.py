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
