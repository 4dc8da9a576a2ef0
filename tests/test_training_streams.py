"""CPU checks of the training operators' ``stream=``: a stream of another device than the operands' is refused."""

import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def training(monkeypatch):
    """The module, its compiled calls replaced by one that must not be reached."""
    from powersgd_rank_gradient_gb300 import training

    def reached(*a):
        raise AssertionError("called on another device's stream")

    calls = ("embedding_forward", "embedding_backward", "layernorm_forward", "layernorm_backward", "distill")
    monkeypatch.setattr(training, "_bind", types.SimpleNamespace(**{c: reached for c in calls}))
    return training


def handle(cls):
    h = cls.__new__(cls)
    h.device, h._spec, h._h = torch.device("cuda", 0), None, None
    h._lib = types.SimpleNamespace(psgd_embedding_status=lambda *a: 0)
    return h


@pytest.mark.parametrize("call", [
    lambda t, s: handle(t.Embedding).forward(None, None, stream=s),
    lambda t, s: handle(t.Embedding).backward(None, None, stream=s),
    lambda t, s: handle(t.Embedding).status(stream=s),
    lambda t, s: handle(t.LayerNorm).forward(None, stream=s),
    lambda t, s: handle(t.LayerNorm).backward(None, None, None, None, stream=s),
])
def test_handles(training, call):
    with pytest.raises(ValueError, match="stream must be on cuda:0"):
        call(training, types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0))


def test_distill_loss(training):
    class Logits(torch.Tensor):
        is_cuda = property(lambda self: True)

        def get_device(self):
            return 0

    with pytest.raises(ValueError, match="stream must be on cuda:0"):
        training.distill_loss(torch.zeros(2, 3).as_subclass(Logits), None, None,
                              stream=types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0))
