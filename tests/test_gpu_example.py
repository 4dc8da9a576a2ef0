"""The training operators together: one step's bucket against 64-bit autograd, and the example's loss."""

import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
DEV = "cuda:0"


def reference(student, ids, top, at, temperature, pad):
    """The same step in 64 bits, differentiated by autograd."""
    flat = student.params.double().requires_grad_()
    table, w1, b1, linear, w2, b2 = student.views(flat)
    live = (ids != pad).double()
    x = table[ids] * math.sqrt(table.shape[1])
    # padding reads its row, but gives it no gradient
    x = torch.where((ids == pad)[..., None], x.detach(), x)
    norm = torch.nn.functional.layer_norm
    y = norm(x, (x.shape[-1],), w1, b1, 1e-5)
    h = torch.nn.functional.gelu(y @ linear.t())
    z = norm(h, (h.shape[-1],), w2, b2, 1e-5)
    logq = torch.log_softmax(z @ table.t() / temperature, -1)
    logp = torch.log_softmax(top.double() / temperature, -1)
    kl = (logp.exp() * (logp - logq.gather(-1, at))).sum(-1) * temperature ** 2
    loss = (kl * live / live.sum()).sum()
    loss.backward()
    return loss.detach(), flat.grad


@pytest.mark.parametrize("vocab,dim,length", [(301, 64, 17), (1003, 136, 40)])
def test_step_against_autograd(vocab, dim, length):
    import distill_step as ex

    student = ex.Student(vocab, dim, 4 * length, DEV, seed=3)
    gen = torch.Generator(device=DEV).manual_seed(5)
    ids = ex.batch(gen, 4, length, vocab, DEV)
    top, at = torch.randn(4, length, vocab, device=DEV, generator=gen).mul_(3).topk(9, dim=-1)
    bucket = torch.full((student.numel,), float("nan"), device=DEV)
    loss = student.gradients(ids, top, at, 2.0, bucket)
    want_loss, want = reference(student, ids, top, at, 2.0, ex.PAD)
    # fp32 throughout: sums of some hundred terms and products of 64-136, a few 1e-6 of the tensor's norm each
    assert abs(float(loss) - float(want_loss)) <= 1e-5 * abs(float(want_loss))
    for got, exp in zip(student.views(bucket), student.views(want)):
        assert float((got.double() - exp).norm()) <= 2e-5 * float(exp.norm())


def test_example_learns():
    import distill_step as ex

    losses = ex.train(steps=30, device=DEV)
    assert all(math.isfinite(x) for x in losses)
    assert sum(losses[-5:]) < 0.8 * sum(losses[:5])
