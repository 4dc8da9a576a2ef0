"""Long sums on the tensor cores, which cut off where fp32 rounds: what that loses of a sum stays bounded.  Results of 76
whole tiles, that is, sums that are not shared out among pairs of CTAs."""

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import step_util as su  # noqa: E402
from training_util import U, u  # noqa: E402

DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
# 1024 elements are 64 instructions, of which each may cut the sum off twice, by a step of fp32 (2^-23 of it) at most
CUT = 64 * 2 * 2.0 ** -23


def positive(shape, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (0.5 + 0.5 * torch.rand(shape, device=DEV, generator=g)).to(dtype)


def randn(shape, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, device=DEV, generator=g).to(dtype)


def constant_gradient(dtype, lse=0.3):
    """(G of every column, G at the target) where all logits are 0, as they are rounded to ``dtype``."""
    shift = 2.0 ** 14 if dtype == F16 else 1.0
    out = []
    for exact in (math.exp(-lse), math.expm1(-lse)):
        x = torch.tensor(exact * shift, dtype=torch.float64)
        # far enough from a border between two values that fp32's error (4 u) does not matter
        assert (x * (1 - 8 * u)).to(dtype) == (x * (1 + 8 * u)).to(dtype)
        out.append(float(x.to(dtype)) / shift)
    return out


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens", [1000, 16384])
def test_table_gradient_of_many_tokens(tokens, dtype):
    from powersgd_rank_gradient_gb300 import LinearCrossEntropy

    vocab, dim = 4864, 1024  # 76 whole tiles
    c = LinearCrossEntropy(vocab, dim, tokens, device=DEV)
    hidden, weight = positive((tokens, dim), dtype, 1), torch.zeros((vocab, dim), dtype=dtype, device=DEV)
    targets = torch.randint(0, vocab, (tokens,), device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))
    _, dw = c.backward(hidden, weight, targets, torch.full((tokens,), 0.3, device=DEV))
    c.status()
    q, own = constant_gradient(dtype)
    h = hidden.double()
    at = torch.zeros((vocab, dim), dtype=torch.float64, device=DEV).index_add_(0, targets, h)
    want, mag = (h.sum(0) - at) * q + at * own, (h.sum(0) - at) * q - at * own
    # the pieces that are taken out, and those of a tile that is cut, are added in rounded fp32
    su.check(dw, want, (CUT + (tokens / 1024 + 80) * u) * mag)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("tokens,vocab,dim", [(33, 262144, 64), (512, 131072, 9728)])
def test_hidden_gradient_of_a_long_vocabulary(tokens, vocab, dim, dtype):
    from powersgd_rank_gradient_gb300 import LinearCrossEntropy

    c = LinearCrossEntropy(vocab, dim, tokens, device=DEV)
    hidden, weight = torch.zeros((tokens, dim), dtype=dtype, device=DEV), positive((vocab, dim), dtype, 3)
    targets = torch.randint(0, vocab, (tokens,), device=DEV, generator=torch.Generator(device=DEV).manual_seed(4))
    scale = 2.0 ** -8
    dh, _ = c.backward(hidden, weight, targets, torch.full((tokens,), 0.3, device=DEV), grad_scale=scale,
                       dweight=torch.empty_like(weight))
    c.status()
    q, own = constant_gradient(dtype)
    at = weight[targets].double()
    want = ((sum(w.double().sum(0) for w in weight.split(8192)) - at) * q + at * own) * scale
    # a sum that is not taken out loses an eighth of half a step, 2^-12 or 2^-9 of it
    err = (max(CUT, 2.0 ** (-15 if dtype == F16 else -12)) + (vocab / 1024 + 80) * u) * want.abs()
    su.check(dh, want, err + U[dtype] * (want.abs() + err))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("sign", ["one", "both"])
@pytest.mark.parametrize("rows", [2048, 16384])
def test_weight_gradient_of_many_rows(rows, sign, dtype):
    """The whole matrix: an fp32 library product of these operands is 1e-7 to 4e-7 of its norm off, whole sums of 16384
    rows on the tensor cores are 8e-6."""
    from powersgd_rank_gradient_gb300 import LinearWeightGrad, save_activation

    make = positive if sign == "one" else randn
    kept, grad = save_activation(make((rows, 1024), dtype, 5)), make((rows, 4864), dtype, 6)
    h = LinearWeightGrad(4864, 1024, rows, device=DEV)
    got = h.backward(grad, kept)
    h.status()
    want = grad.double().t() @ kept.restore(F32).double()
    assert float((got.double() - want).norm() / want.norm()) < 1e-6


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dim", [8192, 65536])
def test_logits_of_long_rows(dim, dtype):
    """Losses and lse where no target is likely and all products have one sign."""
    from powersgd_rank_gradient_gb300 import LinearCrossEntropy

    tokens, vocab = 40, 2000
    c = LinearCrossEntropy(vocab, dim, tokens, device=DEV)
    hidden = positive((tokens, dim), dtype, 7)
    weight = (positive((vocab, dim), F32, 8) * (48 / dim)).to(dtype)
    targets = torch.randint(0, vocab, (tokens,), device=DEV, generator=torch.Generator(device=DEV).manual_seed(9))
    losses, lse = c.forward(hidden, weight, targets)
    c.status()
    z = hidden.double() @ weight.double().t()
    want = torch.logsumexp(z, 1)
    ez = (CUT + (dim / 1024 + 4) * u) * float(z.max())
    # a target's own logit: 4 dim / 256 products of a lane in a chain, then 6 additions
    et = (dim / 64 + 6) * u * float(z.max())
    el = ez + (200 + vocab / 128 / 32) * u + 3 * u * want
    su.check(lse, want, el)
    su.check(losses, want - z.gather(1, targets[:, None])[:, 0], el + et + 6 * u * want)
