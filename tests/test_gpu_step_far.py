"""Operands of the products beyond 2^31 elements: the rows at their ends."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import step_util as su  # noqa: E402

DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("offset", [0, 1])
def test_a_table(offset):
    """All but the last 600 rows are 0, in place and copied in pieces; logits of 0 have their part of lse."""
    from powersgd_rank_gradient_gb300 import LinearCrossEntropy

    vocab, dim, tokens, last = 1400000, 1608, 40, 600
    assert vocab * dim > 2 ** 31
    gen = torch.Generator(device=DEV).manual_seed(1)
    flat = torch.zeros(vocab * dim + offset, dtype=BF16, device=DEV)
    weight = flat[offset:].view(vocab, dim)
    weight[-last:] = (torch.randn((last, dim), device=DEV, generator=gen) * dim ** -0.5).to(BF16)
    targets = vocab - 1 - torch.randint(0, last, (tokens,), device=DEV, generator=gen)
    hidden = (torch.randn((tokens, dim), device=DEV, generator=gen) + 15 * weight[targets].float()).to(BF16)
    c = LinearCrossEntropy(vocab, dim, tokens, device=DEV)
    losses, lse = c.forward(hidden, weight, targets)
    dw = torch.full((vocab, dim), 7.0, dtype=BF16, device=DEV)
    dh, _ = c.backward(hidden, weight, targets, lse, dweight=dw)
    c.status()
    z = torch.cat([torch.zeros((tokens, 1), dtype=torch.float64, device=DEV), hidden.double() @ weight[-last:].double().t()], 1)
    z[:, 0] += torch.log(torch.tensor(float(vocab - last), dtype=torch.float64))
    want = torch.logsumexp(z, 1)
    at = targets - (vocab - last) + 1
    # sums of 1608 products, and of a tile's exponentials and 1400000 / 256 tiles' in 32 runs
    mag = (hidden.double().abs() @ weight[-last:].double().abs().t()).amax(1)
    err = (dim + 4) * su.u * mag + (300 + vocab / 128 / 32) * su.u + 4 * su.u * want
    su.check(lse, want, err)
    su.check(losses, want - z.gather(1, at[:, None])[:, 0], 2 * err + 4 * su.u * z.abs().amax(1))
    # the rows at the end: the definition with lse as it is given
    q = torch.exp(z[:, 1:] - lse.double()[:, None])
    eq = q * torch.expm1((dim + 8) * su.u * mag + 8 * su.u * want)[:, None]
    q[torch.arange(tokens, device=DEV), at - 1] -= 1
    eg = eq + su.U[BF16] * (q.abs() + eq) + 2 * su.u
    h, w = hidden.double(), weight[-last:].double()
    su.check_out(dw[-last:], q.t() @ h, eg.t() @ h.abs() + 80 * su.u * (q.abs() + eg).t() @ h.abs(), BF16)
    su.check_out(dh, q @ w, eg @ w.abs() + (last + vocab / 1024) * su.u * (q.abs() + eg) @ w.abs(), BF16)
    # and a row in front of them: every token's exp(-lse)
    q0 = torch.exp(-lse.double())[:, None].expand(tokens, 1)
    e0 = q0 * (su.U[BF16] + 40 * su.u + 2 * su.u * lse.double()[:, None])
    for row in (0, 2 ** 31 // dim, 2 ** 31 // dim + 1):
        su.check_out(dw[row:row + 1], q0.t() @ h, e0.t() @ h.abs() * 1.01, BF16)


def test_a_weight_gradient():
    from powersgd_rank_gradient_gb300 import LinearWeightGrad, save_activation

    outs, ins, rows = 140000, 16000, 70
    assert outs * ins > 2 ** 31
    gen = torch.Generator(device=DEV).manual_seed(2)
    kept = save_activation(torch.randn((rows, ins), device=DEV, generator=gen).to(BF16))
    grad = torch.randn((rows, outs), device=DEV, generator=gen).to(BF16)
    h = LinearWeightGrad(outs, ins, rows, device=DEV)
    out = h.backward(grad, kept, out=torch.full((outs, ins), 7.0, dtype=BF16, device=DEV))
    h.status()
    x = kept.restore(F32)
    for lo in (0, 2 ** 31 // ins - 200, outs - 300):
        want, err = su.product(grad[:, lo:lo + 300], x)
        su.check(out[lo:lo + 300], want, su.out_tol(err, want, BF16))


@pytest.mark.parametrize("dim", [4096, 4095])
def test_checkpoints_and_norms(dim):
    from powersgd_rank_gradient_gb300 import RMSNorm, save_activation

    rows = 2 ** 31 // dim + 700
    x = torch.zeros((rows, dim), dtype=BF16, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(3)
    ends = (slice(0, 300), slice(rows - 900, rows - 500), slice(rows - 300, rows))
    for e in ends:
        x[e] = torch.randn(x[e].shape, device=DEV, generator=gen).to(BF16)
    kept = save_activation(x)
    back = kept.restore(BF16)
    n = RMSNorm(dim, device=DEV)
    y, _, rstd = n.forward(x, out=back.clone())
    for e in ends:
        su.check_eight(kept.codes[e], kept.scales[e], x[e], su.E4)
        assert torch.equal(back[e].float(), kept.codes[e].float() * su.spread(kept.scales[e], dim))
        (wy, wr), (ey, er) = su.rms_forward(x[e], None, 1e-6)
        su.check_out(y[e], wy, ey, BF16)
        su.check(rstd[e], wr, er)
    del back
    rstd.fill_(1.0)
    grad = y  # a gradient of the same shape; rows of zeros add nothing to dweight
    for s in (x, kept):
        dx, dw = n.backward(grad, s, rstd)
        values = [(x[e] if s is x else kept.codes[e].float() * su.spread(kept.scales[e], dim)) for e in ends]
        for e, v in zip(ends, values):
            (wdx, _), (edx, _) = su.rms_backward(grad[e], v, rstd[e], None)
            su.check_out(dx[e], wdx, edx, BF16)
        g = torch.cat([grad[e] for e in ends])
        (_, wdw), (_, edw) = su.rms_backward(g, torch.cat(values), torch.ones(g.shape[0], device=DEV), None)
        su.check(dw, wdw, edw * (1 + rows / 300 / 32))
        del dx
