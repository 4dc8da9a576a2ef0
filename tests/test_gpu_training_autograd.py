"""The training operators and autograd: nothing is passed by in silence."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def randn(*shape):
    return torch.randn(*shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(sum(shape)))


def operands():
    """(call, its tensors by argument) of every operator; the call takes them by name."""
    from powersgd_rank_gradient_gb300 import Embedding, LayerNorm, distill_loss

    e, n = Embedding(20, 8, 6, device=DEV), LayerNorm(8, device=DEV)
    ids = torch.randint(0, 20, (6,), device=DEV)
    x, z = randn(6, 8), randn(6, 20)
    at = torch.randint(0, 20, (6, 3), device=DEV)
    return [
        (lambda weight, out: e.forward(weight, ids, out=out), dict(weight=randn(20, 8), out=randn(6, 8)), ["out"]),
        (lambda grad, out: e.backward(ids, grad, out=out), dict(grad=randn(6, 8), out=randn(20, 8)), ["out"]),
        (lambda x, weight, bias, out: n.forward(x, weight, bias, out=out),
         dict(x=x, weight=randn(8), bias=randn(8), out=randn(6, 8)), ["out"]),
        (lambda **kw: n.backward(**kw),
         dict(grad=randn(6, 8), x=x, mean=randn(6), rstd=randn(6).abs(), weight=randn(8), dx=randn(6, 8), dweight=randn(8),
              dbias=randn(8)), ["dx", "dweight", "dbias"]),
        (lambda **kw: distill_loss(teacher_indices=at, **kw),
         dict(logits=z, teacher_logits=randn(6, 3), weights=randn(6).abs(), dlogits=randn(6, 20)), ["dlogits"]),
    ]


@pytest.mark.parametrize("which", range(5))
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
        derived = dict(tensors, **{name: tensors[name].detach().requires_grad_() * 1})  # not a leaf
        with pytest.raises(ValueError, match=f"^{name} requires a gradient"):
            call(**derived)
    with torch.inference_mode():
        inference = {k: v.clone() for k, v in tensors.items()}
        call(**inference)
        call(**tensors)
        assert all(torch.equal(inference[k], w) and torch.equal(tensors[k], w) for k, w in zip(written, want))


@pytest.mark.parametrize("which", range(5))
def test_written_tensors_advance_their_version(which):
    call, tensors, written = operands()[which]
    before = {k: t._version for k, t in tensors.items()}
    call(**tensors)
    assert {k: t._version - before[k] for k, t in tensors.items()} == {k: int(k in written) for k in tensors}
    bucket = torch.zeros(4000, device=DEV)  # a view's writes are its base's too
    at, views = 0, {}
    for k in written:
        views[k] = bucket[at:at + tensors[k].numel()].view(tensors[k].shape)
        at += tensors[k].numel()
    version = bucket._version
    call(**dict(tensors, **views))
    assert bucket._version == version + len(written)


def test_a_saved_value_that_is_overwritten_is_noticed():
    from powersgd_rank_gradient_gb300 import distill_loss

    w = randn(4, 30).requires_grad_()
    logits = torch.exp(w)  # saves its own result
    with torch.no_grad():
        distill_loss(logits, randn(4, 3), torch.randint(0, 30, (4, 3), device=DEV), dlogits=logits)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        logits.sum().backward()


def test_a_refused_call_writes_and_advances_nothing():
    from powersgd_rank_gradient_gb300._lib import PsgdError

    call, tensors, _ = operands()[0]
    before = tensors["weight"].clone()
    version = tensors["weight"]._version
    with pytest.raises(PsgdError, match="overlap"):
        call(weight=tensors["weight"], out=tensors["weight"][:6])
    assert tensors["weight"]._version == version and torch.equal(tensors["weight"], before)
