"""What the product handles hold: nothing of the size of a table or a gradient that is read where it lies."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import step_util as su  # noqa: E402

DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
MB = 1 << 20


def sums():
    """Partial sums of products: two tiles of 256 x 256 for every pair of SMs."""
    return torch.cuda.get_device_properties(0).multi_processor_count * 256 * 1024


@pytest.mark.parametrize("vocab,dim,tokens", [(50257, 1600, 1), (50257, 1600, 4), (128256, 8192, 1), (128256, 8192, 64), (30522, 1024, 499)])
def test_a_loss_holds_no_table(vocab, dim, tokens):
    from powersgd_rank_gradient_gb300 import LinearCrossEntropy

    rows, wide = -(-tokens // 64) * 64, (dim // 64 + 2) * 64
    # the tokens that count (three times, and a few numbers each), their logits' gradient, a copied piece, entries of tiles
    most = rows * (wide * 8 + 32) + rows * (vocab + 512) * 2 + 32 * MB + sums() + (vocab / 128 + 200) * rows * 8
    h = LinearCrossEntropy(vocab, dim, tokens, device=DEV)
    assert h.workspace_bytes() <= most < vocab * dim * 2 + sums() + rows * vocab * 2
    h.close()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("vocab,dim,tokens", [(20001, 1024, 20), (9000, 4104, 70)])
def test_tables_that_are_copied_in_pieces(vocab, dim, tokens, dtype):
    """Rows of whole units that begin between two of them: more than 32 MB."""
    from powersgd_rank_gradient_gb300 import LinearCrossEntropy

    gen = torch.Generator(device=DEV).manual_seed(vocab)
    flat = torch.zeros(vocab * dim + 1, dtype=dtype, device=DEV)
    weight = flat[1:].view(vocab, dim)
    weight.copy_(torch.randn((vocab, dim), device=DEV, generator=gen) * dim ** -0.5)
    targets = torch.randint(-1, vocab, (tokens,), device=DEV, generator=gen)
    hidden = (torch.randn((tokens, dim), device=DEV, generator=gen) + 5 * weight[targets.clamp(min=0)].float()).to(dtype)
    h = LinearCrossEntropy(vocab, dim, tokens, device=DEV)
    assert h.workspace_bytes() < weight.numel() * 2 + 60 * MB
    losses, lse = h.forward(hidden, weight, targets)
    dh, dw = h.backward(hidden, weight, targets, lse)
    h.status()
    (wl, ws), (el, es) = su.loss_forward(hidden, weight, targets, None)
    su.check(losses, wl, el)
    su.check(lse, ws, es)
    (wh, ww), (eh, ew) = su.loss_backward(hidden, weight, targets, lse, None)
    su.check_out(dh, wh, eh, dtype)
    su.check_out(dw, ww, ew, F32)


@pytest.mark.parametrize("tokens", [1, 63, 64, 65, 127, 128, 129, 191, 193, 320])
def test_a_handle_of_just_so_many_tokens(tokens):
    """Workspaces end at a multiple of 64 tokens, tiles at one of 256."""
    from powersgd_rank_gradient_gb300 import LinearCrossEntropy

    gen = torch.Generator(device=DEV).manual_seed(tokens)
    weight = (torch.randn((1111, 136), device=DEV, generator=gen) * 136 ** -0.5).to(BF16)
    hidden = torch.randn((tokens, 136), device=DEV, generator=gen).to(BF16)
    targets = torch.randint(0, 1111, (tokens,), device=DEV, generator=gen)
    h = LinearCrossEntropy(1111, 136, tokens, device=DEV)
    for n in (tokens, max(1, tokens - 33), tokens):
        losses, lse = h.forward(hidden[:n], weight, targets[:n])
        dh, dw = h.backward(hidden[:n], weight, targets[:n], lse)
        h.status()
        (wl, ws), (el, es) = su.loss_forward(hidden[:n], weight, targets[:n], None)
        su.check(losses, wl, el)
        su.check(lse, ws, es)
        (wh, ww), (eh, ew) = su.loss_backward(hidden[:n], weight, targets[:n], lse, None)
        su.check_out(dh, wh, eh, BF16)
        su.check_out(dw, ww, ew, F32)


@pytest.mark.parametrize("outs,ins,rows", [(6400, 1600, 16384), (1024, 1024, 509), (2048, 64, 300000)])
def test_a_weight_gradient_holds_no_gradient(outs, ins, rows):
    from powersgd_rank_gradient_gb300 import LinearWeightGrad

    h = LinearWeightGrad(outs, ins, rows, device=DEV)
    # the checkpoint restored, a copied piece (256 columns at least), partial sums
    assert h.workspace_bytes() <= rows * ins * 2 + max(32 * MB, rows * 512) + sums() + 64
    h.close()


@pytest.mark.parametrize("odtype,accumulate", [(F32, False), (BF16, True)])
@pytest.mark.parametrize("rows,outs,ins", [(9000, 3000, 72), (30000, 1096, 200)])
def test_gradients_that_are_copied_in_pieces(rows, outs, ins, odtype, accumulate):
    """Rows of whole units that begin between two of them: more than 32 MB."""
    from powersgd_rank_gradient_gb300 import LinearWeightGrad, save_activation

    gen = torch.Generator(device=DEV).manual_seed(outs)
    grad = torch.randn(rows * outs + 3, device=DEV, generator=gen).to(BF16)[3:].view(rows, outs)
    kept = save_activation(torch.randn((rows, ins), device=DEV, generator=gen).to(BF16))
    before = torch.randn((outs, ins), device=DEV, generator=gen).to(odtype)
    h = LinearWeightGrad(outs, ins, rows, device=DEV)
    assert h.workspace_bytes() < rows * ins * 2 + grad.numel() * 2 + sums()
    out = h.backward(grad, kept, out=before.clone(), accumulate=accumulate)
    h.status()
    want, err = su.product(grad, kept.restore(F32), before=before if accumulate else None)
    su.check(out, want, su.out_tol(err, want, odtype))
