"""Distillation of rows longer than a cluster's shared memory, which are read from memory twice."""

import pytest

import training_util as tu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("vocab,dtype", [(500009, F32), (1000003, BF16), (1000003, F16)])
def test_masks_far_rows_and_in_place(vocab, dtype):
    from powersgd_rank_gradient_gb300 import distill_loss

    g = torch.Generator(device=DEV).manual_seed(vocab)
    rows, k = 10, 600
    z = torch.empty((rows, vocab), dtype=dtype, device=DEV).normal_(0, 2, generator=g)
    t = torch.empty((rows, k), device=DEV).normal_(0, 2, generator=g)
    at = torch.randint(0, vocab, (rows, k), device=DEV, generator=g)
    w = torch.rand(rows, device=DEV, generator=g) + 0.5
    w[2], at[5], t[6], at[7, ::2], at[9, 300:] = 0.0, -1, -torch.inf, -3, at[9, :300]
    if dtype == F32:  # the largest logits enormous, on either side
        z[0] += 1e7
        z[1] -= 1e7
        z[3, 1:] -= 3e38
        at[3] = 0
    losses, dz = distill_loss(z, t, at, 1.5, w, 8.0)
    (wl, wz), (el, ez) = tu.distill(z, t, at, 1.5, w, 8.0)
    tu.check(losses, wl, tu.out_tol(el, wl, F32))
    tu.check(dz, wz, tu.out_tol(ez, wz, dtype))
    only, _ = distill_loss(z, t, at, 1.5, w, with_grad=False)
    assert torch.equal(only, losses)
    copy = z.clone()
    l2, same = distill_loss(copy, t, at, 1.5, w, 8.0, dlogits=copy)
    assert same is copy and torch.equal(l2, losses) and torch.equal(copy, dz)
    # rows that do not count may hold anything; a NaN or nothing but -infinity is NaN in its own row only
    z[2] = z[5] = z[6] = float("nan")
    z[8], z[4, 77] = -torch.inf, float("nan")
    l3, d3 = distill_loss(z, t, at, 1.5, w, 8.0)
    for r in range(rows):
        if r in (2, 5, 6):
            assert float(l3[r]) == 0.0 and bool((d3[r] == 0).all())
        elif r in (4, 8):
            assert bool(torch.isnan(l3[r])) and bool(torch.isnan(d3[r]).all())
        else:
            assert torch.equal(l3[r], losses[r]) and torch.equal(d3[r], dz[r])
