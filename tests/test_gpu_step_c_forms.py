"""Forms of the C interface that leave one of two gradients out: the other is what it is with both."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import step_util as su  # noqa: E402
from powersgd_rank_gradient_gb300 import _lib  # noqa: E402

DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
CODE = {F32: _lib.PSGD_F32, F16: _lib.PSGD_F16, BF16: _lib.PSGD_BF16}


def randn(*shape, dtype=F32, seed=0):
    return torch.randn(*shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed + sum(shape))).to(dtype)


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("rows,dim", [(1, 64), (700, 1600), (3001, 264), (700, 1601), (37, 6405), (9, 16384), (5, 20001)])
def test_norm(rows, dim, add, saved, dtype):
    from powersgd_rank_gradient_gb300 import RMSNorm, save_activation

    n = RMSNorm(dim, device=DEV)
    x, g, w = randn(rows, dim, dtype=dtype), randn(rows, dim, dtype=dtype, seed=1), randn(dim, seed=2)
    gs = randn(rows, dim, dtype=dtype, seed=3) if add else None
    rstd = (x.float() ** 2).mean(1).rsqrt()
    kept = save_activation(x) if saved else x
    want_dx, _ = n.backward(g, kept, rstd, w, grad_summed=gs)
    before = randn(dim, seed=4)
    # (how many rows a turn takes, and with it the order of dweight's sum, may hang on what else there is)
    s = kept.restore(F32) if saved else x
    (_, want_dw), (_, err) = su.rms_backward(g, s, rstd, w)
    (_, want_more), (_, err_more) = su.rms_backward(g, s, rstd, w, before=before)

    def call(dx, dw, accumulate):
        ptr = [None if t is None else t.data_ptr() for t in (None if saved else x, kept.codes if saved else None, kept.scales if saved else None)]
        assert n._lib.psgd_rmsnorm_backward(
            n._h, g.data_ptr(), CODE[dtype], dim, rows, ptr[0], dim, ptr[1], 0, ptr[2], rstd.data_ptr(), w.data_ptr(), CODE[F32],
            None if gs is None else gs.data_ptr(), dim, None if dx is None else dx.data_ptr(), dim,
            None if dw is None else dw.data_ptr(), CODE[F32], int(accumulate), stream()) == _lib.PSGD_OK

    dx, dw, more = torch.full_like(g, 7.0), torch.full((dim,), 7.0, device=DEV), before.clone()
    call(dx, None, False)
    call(None, dw, False)
    call(None, more, True)
    call(None, None, False)
    assert torch.equal(dx, want_dx)
    su.check_out(dw, want_dw, err, F32)
    su.check_out(more, want_more, err_more, F32)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tokens,vocab,dim", [(0, 300, 72), (3, 300, 72), (40, 1000, 201), (700, 900, 136), (6000, 40000, 64)])
def test_loss(tokens, vocab, dim, dtype):
    """6000 tokens: in pieces of the vocabulary."""
    from powersgd_rank_gradient_gb300 import LinearCrossEntropy

    c = LinearCrossEntropy(vocab, dim, tokens, device=DEV)
    hidden, weight = randn(tokens, dim, dtype=dtype), (randn(vocab, dim, seed=1) * dim ** -0.5).to(dtype)
    targets = torch.randint(-1, vocab, (tokens,), device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))
    _, lse = c.forward(hidden, weight, targets)
    want_dh, want_dw = c.backward(hidden, weight, targets, lse)
    before = randn(vocab, dim, seed=4)
    _, want_more = c.backward(hidden, weight, targets, lse, dweight=before.clone(), accumulate=True)

    def call(dh, dw, accumulate):
        assert c._lib.psgd_linear_ce_backward(
            c._h, hidden.data_ptr(), CODE[dtype], dim, tokens, weight.data_ptr(), dim, targets.data_ptr(), 64, lse.data_ptr(), None, 1.0,
            None if dh is None else dh.data_ptr(), dim, None if dw is None else dw.data_ptr(), CODE[F32], dim, int(accumulate),
            stream()) == _lib.PSGD_OK

    dh, dw, more = torch.full_like(hidden, 7.0), torch.full((vocab, dim), 7.0, device=DEV), before.clone()
    call(dh, None, False)
    call(None, dw, False)
    call(None, more, True)
    call(None, None, False)
    c.status()
    assert torch.equal(dh, want_dh) and torch.equal(dw, want_dw) and torch.equal(more, want_more)
