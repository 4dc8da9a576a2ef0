"""The operators that keep a step small, and autograd and threads: nothing is passed by in silence."""

import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16 = torch.bfloat16


def randn(*shape, dtype=torch.float32):
    return torch.randn(*shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(sum(shape))).to(dtype)


def operands():
    """(call, its tensors by argument, those that it writes) of every operator."""
    from powersgd_rank_gradient_gb300 import Activation8, LinearCrossEntropy, LinearWeightGrad, RMSNorm, save_activation

    n, g, c = RMSNorm(64, device=DEV), LinearWeightGrad(24, 64, 16, device=DEV), LinearCrossEntropy(40, 64, 16, device=DEV)
    x = randn(16, 64)
    kept = save_activation(x)
    targets = torch.randint(0, 40, (16,), device=DEV)
    hidden, weight = randn(16, 64, dtype=BF16), randn(40, 64, dtype=BF16)
    out8 = save_activation(x)
    return [
        (lambda **kw: n.forward(**kw), dict(x=x, weight=randn(64), residual=randn(16, 64), out=randn(16, 64), summed=randn(16, 64)),
         ["out", "summed"]),
        (lambda x, weight, residual: n.forward8(x, weight, residual, out=out8), dict(x=x, weight=randn(64), residual=randn(16, 64)), []),
        (lambda **kw: n.backward(**kw),
         dict(grad=randn(16, 64), summed=x, rstd=randn(16).abs(), weight=randn(64), grad_summed=randn(16, 64), dx=randn(16, 64),
              dweight=randn(64)), ["dx", "dweight"]),
        (lambda scales, out: Activation8._made(kept.codes, scales).restore(out=out), dict(scales=kept.scales, out=randn(16, 64)), ["out"]),
        (lambda x: save_activation(x, out=out8), dict(x=x), []),
        (lambda grad, out: g.backward(grad, kept, out=out), dict(grad=randn(16, 24, dtype=BF16), out=randn(24, 64)), ["out"]),
        (lambda **kw: c.forward(targets=targets, **kw), dict(hidden=hidden, weight=weight, weights=randn(16).abs()), []),
        (lambda **kw: c.backward(targets=targets, **kw),
         dict(hidden=hidden, weight=weight, lse=randn(16).abs() + 4, weights=randn(16).abs(), dhidden=randn(16, 64, dtype=BF16),
              dweight=randn(40, 64)), ["dhidden", "dweight"]),
    ]


@pytest.mark.parametrize("which", range(8))
def test_operands_that_require_a_gradient(which):
    """Refused while autograd records, each of them; taken under no_grad and in inference mode."""
    call, tensors, written = operands()[which]
    call(**tensors)
    want = [tensors[k].clone() for k in written]
    for name in tensors:
        with_grad = dict(tensors, **{name: tensors[name].detach().requires_grad_()})
        with pytest.raises(ValueError, match=f"^{name} requires a gradient"):
            call(**with_grad)
        before = with_grad[name]._version
        with torch.no_grad():
            call(**with_grad)
        assert with_grad[name]._version == before + (name in written)
        assert all(torch.equal(with_grad[k], w) for k, w in zip(written, want))
    with torch.inference_mode():
        inference = {k: v.clone() for k, v in tensors.items()}
        call(**inference)
        assert all(torch.equal(inference[k], w) for k, w in zip(written, want))


@pytest.mark.parametrize("which", range(8))
def test_written_tensors_advance_their_version(which):
    call, tensors, written = operands()[which]
    before = {k: t._version for k, t in tensors.items()}
    call(**tensors)
    assert {k: t._version - before[k] for k, t in tensors.items()} == {k: int(k in written) for k in tensors}


def test_written_checkpoints_advance_their_version():
    from powersgd_rank_gradient_gb300 import RMSNorm, save_activation

    x = randn(8, 64)
    a = save_activation(x)
    before = a.codes._version, a.scales._version
    save_activation(x, out=a)
    RMSNorm(64, device=DEV).forward8(x, out=a)
    assert (a.codes._version, a.scales._version) == (before[0] + 2, before[1] + 2)


def test_handles_of_two_threads():
    """Two host threads with handles and streams of their own, the products' pairs of CTAs among each other."""
    from powersgd_rank_gradient_gb300 import LinearCrossEntropy, LinearWeightGrad, RMSNorm

    done, failed = {}, []

    def work(seed):
        try:
            gen = torch.Generator(device=DEV).manual_seed(seed)
            with torch.cuda.stream(torch.cuda.Stream()):
                n, g = RMSNorm(200, device=DEV), LinearWeightGrad(300, 200, 900, device=DEV)
                c = LinearCrossEntropy(1500, 200, 900, device=DEV)
                x, w = (torch.randn(r, 200, device=DEV, generator=gen).to(BF16) for r in (900, 1500))
                grad = torch.randn(900, 300, device=DEV, generator=gen).to(BF16)
                targets = torch.randint(0, 1500, (900,), device=DEV, generator=gen)
                results = []
                for _ in range(15):
                    kept, s, rstd = n.forward8(x, residual=x)
                    losses, lse = c.forward(s, w, targets)
                    results.append((kept.restore(), g.backward(grad, kept), losses, *c.backward(s, w, targets, lse), *n.backward(x, s, rstd)))
                g.status(), c.status()
                assert all(torch.equal(a, b) for r in results[1:] for a, b in zip(r, results[0]))
                done[seed] = True
        except Exception as e:  # shown by the main thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and done == {0: True, 1: True}
