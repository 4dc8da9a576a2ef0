"""The teacher's softmax: logits far from zero and at the ends of their type."""

import pytest

import training_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32 = torch.float32
# a row in shared memory, a row over a cluster of CTAs, a row read from memory twice
VOCABS = [700, 60001, 500009]


def inputs(rows, vocab, k, seed, offset=0.0, tdtype=F32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    z = torch.empty((rows, vocab), device=DEV).normal_(0, 2, generator=g)
    t = torch.empty((rows, k), device=DEV).normal_(offset, 2, generator=g).to(tdtype)
    at = torch.stack([torch.randperm(vocab, device=DEV, generator=g)[:k] for _ in range(rows)])
    return z, t, at


def verify(z, t, at, temperature):
    from powersgd_rank_gradient_gb300 import distill_loss

    losses, dz = distill_loss(z, t, at, temperature)
    (wl, wz), (el, ez) = tu.distill(z, t, at, temperature)
    tu.check(losses, wl, tu.out_tol(el, wl, F32))
    tu.check(dz, wz, tu.out_tol(ez, wz, z.dtype))
    return losses, dz


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("temperature", [0.7, 1.3])
@pytest.mark.parametrize("offset", [-100.0, 1e3, 1e6])
def test_offset(vocab, temperature, offset):
    """The softmax depends on the logits' distances only, and so does its error."""
    verify(*inputs(8, vocab, 30, 5, offset), temperature)


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("tdtype", tu.DTYPES)
@pytest.mark.parametrize("temperature", [0.5, 2.0])
def test_ends_of_the_type(vocab, tdtype, temperature):
    """Entries of the type's lowest and largest value count as any other; only -infinity has no mass."""
    z, t, at = inputs(6, vocab, 6, 7, tdtype=tdtype)
    low, high = torch.finfo(tdtype).min, torch.finfo(tdtype).max
    t[1], t[2] = low, high
    t[3, :4] = low
    t[4, 0], t[4, 1:] = high, low
    t[5, :5] = -torch.inf
    t[5, 5] = low
    losses, dz = verify(z, t, at, temperature)
    assert bool((losses != 0).all()) and bool(torch.isfinite(dz).all())
