"""CPU checks of ``stream=``: a stream of another device than the operands' is refused."""

import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def training(monkeypatch):
    """The module, its compiled calls replaced by one that must not be reached."""
    from powersgd_rank_gradient_gb300 import training

    def reached(*a):
        raise AssertionError("called on another device's stream")

    calls = ("activation_save", "activation_restore", "rmsnorm_forward", "rmsnorm_backward", "wgrad_backward", "linear_ce_forward",
             "linear_ce_backward")
    monkeypatch.setattr(training, "_bind", types.SimpleNamespace(**{c: reached for c in calls}))
    return training


class OnCuda(torch.Tensor):
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def cuda_tensor():
    return torch.zeros(2, 3).as_subclass(OnCuda)


def handle(cls):
    h = cls.__new__(cls)
    h.device, h._spec, h._h = torch.device("cuda", 0), None, None
    h._lib = types.SimpleNamespace(psgd_wgrad_status=lambda *a: 0, psgd_linear_ce_status=lambda *a: 0)
    return h


@pytest.mark.parametrize("call", [
    lambda t, s: handle(t.RMSNorm).forward(None, stream=s),
    lambda t, s: handle(t.RMSNorm).forward8(None, stream=s),
    lambda t, s: handle(t.RMSNorm).backward(None, None, None, stream=s),
    lambda t, s: t.save_activation(cuda_tensor(), stream=s),
    lambda t, s: t.Activation8._made(cuda_tensor(), None).restore(stream=s),
    lambda t, s: handle(t.LinearWeightGrad).backward(None, t.Activation8._made(None, None), stream=s),
    lambda t, s: handle(t.LinearWeightGrad).status(stream=s),
    lambda t, s: handle(t.LinearCrossEntropy).forward(None, None, None, stream=s),
    lambda t, s: handle(t.LinearCrossEntropy).backward(None, None, None, None, stream=s),
    lambda t, s: handle(t.LinearCrossEntropy).status(stream=s),
])
def test_streams_of_another_device(training, call):
    with pytest.raises(ValueError, match="stream must be on cuda:0"):
        call(training, types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0))


@pytest.mark.parametrize("call,what", [
    (lambda t, x: t.save_activation(x, out=x), "out"),
    (lambda t, x: handle(t.RMSNorm).forward8(x, out=x), "out"),
    (lambda t, x: handle(t.LinearWeightGrad).backward(x, x), "activation"),
    (lambda t, x: handle(t.LinearWeightGrad).backward(x, None), "activation"),
])
def test_what_is_no_checkpoint_is_refused(training, call, what):
    with pytest.raises(ValueError, match=f"^{what} must be an Activation8"):
        call(training, cuda_tensor())
