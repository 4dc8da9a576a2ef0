"""The logits' gradient where targets are likely: 1 - p, which is all that is left of exp(z - lse) - 1, against 64 bits."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import step_util as su  # noqa: E402
from training_util import U, u  # noqa: E402

DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
VOCAB = 256


def batch(tokens, dim, dtype, seed, offset=0):
    """hidden, weight, targets.  The weight's last VOCAB columns are the identity and meet zeros in hidden, so that those
    columns of dhidden are the logits' gradient itself; 1 - p goes from 5e-2 to 1e-8."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n = dim - VOCAB
    flat = torch.zeros(VOCAB * dim + offset, dtype=dtype, device=DEV)
    weight = flat[offset:].view(VOCAB, dim)
    weight[:, :n] = (torch.randn((VOCAB, n), device=DEV, generator=gen) * n ** -0.5).to(dtype)
    weight[:, n:] = torch.eye(VOCAB, dtype=dtype, device=DEV)
    targets = torch.randint(0, VOCAB, (tokens,), device=DEV, generator=gen)
    hidden = torch.zeros((tokens, dim), dtype=dtype, device=DEV)
    hidden[:, :n] = (torch.linspace(10, 24, tokens, device=DEV)[:, None] * weight[targets, :n].float()).to(dtype)
    return hidden, weight, targets


def definition(hidden, weight, targets, dtype):
    """(G, its error where lse is the forward pass's own)."""
    h, w = hidden.double(), weight.double()
    z, mag = h @ w.t(), h.abs() @ w.abs().t()
    ez = (h.shape[1] + 4) * u * mag  # sums in fp32, in any order
    lse = torch.logsumexp(z, 1, keepdim=True)
    at = targets[:, None]
    g = torch.exp(z - lse)
    # a logit's error, lse's, an exponential's (4 u and its argument's size) and lse's rounding
    rel = torch.expm1(ez + ez.amax(1, keepdim=True) + 2 * u * (z.abs() + 2 * lse.abs()) + 300 * u)
    eg = rel * g
    # the target's: 1 - p is the others' sum over exp(lse), and where both passes take the same logit, its error
    # is theirs, and lse's rounding once
    g.scatter_(1, at, torch.expm1(z.gather(1, at) - lse))
    eg.scatter_(1, at, rel.amax(1, keepdim=True) * g.gather(1, at).abs() + 1.01 * u * lse.abs())
    low = 2.0 ** -39 if dtype == F16 else 0.0  # G is rounded at 2^14 times its size
    return g, eg + U[dtype] * (g.abs() + eg) + low


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens,dim,offset", [(1, 1600, 0), (3, 1600, 0), (40, 1600, 0), (300, 1600, 0), (300, 1601, 0), (40, 1600, 1),
                                               (2, 8192, 0), (40, 8192, 0)])
def test_likely_targets(tokens, dim, offset, dtype):
    from powersgd_rank_gradient_gb300 import LinearCrossEntropy

    hidden, weight, targets = batch(tokens, dim, dtype, tokens + dim, offset)
    h = LinearCrossEntropy(VOCAB, dim, tokens, device=DEV)
    scale = 2.0 ** 14  # keeps f16's dhidden out of its subnormals; exact
    _, lse = h.forward(hidden, weight, targets)
    dh, _ = h.backward(hidden, weight, targets, lse, grad_scale=scale)
    h.status()
    want, err = definition(hidden, weight, targets, dtype)
    got = dh[:, dim - VOCAB:].double() / scale
    su.check(got, want, err + (2.0 ** -25 / scale if dtype == F16 else 0.0))
    at = targets[:, None]
    assert bool((want.gather(1, at).abs() < 0.1).all())


def test_both_passes_take_the_same_logit():
    """lse - z is 0 where nothing but the target has mass: its gradient is exactly 0, however many tokens a call has and
    wherever the operands lie."""
    from powersgd_rank_gradient_gb300 import LinearCrossEntropy

    for dtype in (BF16, F16):
        for offset in (0, 1):
            hidden, weight, targets = batch(33, 1600, dtype, 5, offset)
            hidden *= 8
            h = LinearCrossEntropy(VOCAB, 1600, 33, device=DEV)
            for lo, hi in ((0, 1), (1, 3), (3, 7), (7, 12), (0, 33)):
                losses, lse = h.forward(hidden[lo:hi], weight, targets[lo:hi])
                dh, _ = h.backward(hidden[lo:hi], weight, targets[lo:hi], lse)
                got = dh[:, 1600 - VOCAB:].gather(1, targets[lo:hi, None])
                assert bool((losses < 1e-20).all()) and not bool(got.any())
