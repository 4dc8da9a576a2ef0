"""Layer norm backward near the ends of fp32's range."""

import pytest

import training_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32 = torch.float32


def randn(shape, seed, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.empty(shape, device=DEV).normal_(0, 1, generator=g).double().mul_(std).float()


def verify(x, grad, w, mean, rstd, eps):
    from powersgd_rank_gradient_gb300 import LayerNorm

    got = LayerNorm(x.shape[1], eps=eps, device=DEV).backward(grad, x, mean, rstd, w)
    want, err = tu.norm_backward(grad, x, mean, rstd, w)
    for a, b, e in zip(got, want, err):
        assert bool(torch.isfinite(b).all())
        tu.check(a, b, tu.out_tol(e, b, F32))


# rows of whole 16-byte units (one, two and four vectors a thread), of any length, and too long for registers
@pytest.mark.parametrize("dim", [64, 1600, 4096, 8192, 133, 1023, 4099, 9001])
@pytest.mark.parametrize("std", [1e-30, 1e-21, 1e-19, 1e15, 1e18])
def test_deviations_of_any_size(dim, std):
    """Statistics without an eps, of rows with tiny and with huge deviations."""
    x, grad, w = randn((9, dim), 1, std), randn((9, dim), 2), randn((dim,), 3)
    d = x.double()
    mean = d.mean(1)
    rstd = (d - mean[:, None]).square().mean(1).rsqrt()
    verify(x, grad, w, mean.float(), rstd.float(), 0.0)


@pytest.mark.parametrize("dim", [64, 1600, 133, 9001])
def test_large_gradients_of_large_activations(dim):
    """The product of a gradient and a deviation is beyond fp32, the normalised one's is not."""
    x, grad, w = randn((9, dim), 1, 1e15), randn((9, dim), 2, 1e25), randn((dim,), 3)
    d = x.double()
    mean = d.mean(1)
    rstd = ((d - mean[:, None]).square().mean(1) + 1e-5).rsqrt()
    verify(x, grad, w, mean.float(), rstd.float(), 1e-5)


@pytest.mark.parametrize("dim", [64, 1000, 1023, 9001])
def test_rows_far_from_zero_and_without_variance(dim):
    from powersgd_rank_gradient_gb300 import LayerNorm

    x, grad, w = randn((12, dim), 1, 0.1) + 1000.0, randn((12, dim), 2), randn((dim,), 3)
    x[3], x[4], x[5] = 5.0, 0.0, -1e-30
    _, mean, rstd = LayerNorm(dim, device=DEV).forward(x, w)
    verify(x, grad, w, mean, rstd, 1e-5)
