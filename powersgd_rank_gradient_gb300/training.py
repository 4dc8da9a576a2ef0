"""Training operators: what fills the gradient buckets.

``Embedding`` (lookup with scaling, and the dense gradient of its table),
``LayerNorm`` (forward, and backward with the reduction of the parameters'
gradients) and ``distill_loss`` (losses and logits' gradient of distillation
from a teacher's top logits).  Parameter gradients are written into tensors
the caller passes, typically views of a flat replica bucket at any element
offset and in the bucket's type, so that ``powerSGD_hook`` takes the bucket as
it is.  torch is used for device memory and streams; the arithmetic runs in the
CUDA kernels of libpsgd.so.

Autograd does not see these calls: each gradient is a call of its own.  While
autograd records (outside ``torch.no_grad()``), an operand that requires a
gradient raises ValueError in place of giving a result without one.
"""

from __future__ import annotations

import ctypes
import os

import torch

from . import _lib
from ._lib import PSGD_BAD_TOKEN, check

_lib.lib()  # the library itself; raises with how to build it where it is missing
if not os.path.exists(os.path.join(_lib.HERE, "_bind.so")):
    raise RuntimeError(f"{_lib.HERE}/_bind.so is missing: build it with "
                       "`python -c 'import __graft_entry__ as g; g.build()'` "
                       "(it needs a CUDA build of torch, Python's headers and g++)")
from . import _bind  # noqa: E402  (argument checks and calls, compiled: psgd_bind.cpp)


def _check_binding(built_with, library, torch_version):
    """The binding calls the library and torch through their headers: both must be the ones it was compiled against."""
    for what, built, found in zip(("library", "torch"), built_with, (library, torch_version)):
        if built != found:
            raise RuntimeError(f"_bind.so was built against another {what} ({built}) than the one loaded ({found}): build it again "
                               "with `python -c 'import __graft_entry__ as g; g.build()'`")


_check_binding(_bind.built_with(), _lib.lib().psgd_build_id().decode(), str(torch.__version__))


def _device(device):
    if device is None:
        device = torch.cuda.current_device()
    device = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
    if device.type != "cuda":
        raise ValueError("device must be a CUDA device")
    return torch.device("cuda", torch.cuda.current_device()) if device.index is None else device


def _of_device(stream, index):
    """``stream``, which must belong to CUDA device ``index``."""
    if stream.device.index != index:
        raise ValueError(f"stream must be on cuda:{index}, got {stream.device}")
    return stream


def _on(stream, index):
    return torch.cuda.stream(_of_device(stream, index))


class Embedding:
    """A table of ``num_embeddings`` rows of ``embedding_dim`` elements: lookup
    times ``scale``, and the gradient of the table.

    ``max_tokens`` bounds the tokens of one call (the handle holds the
    gradient's workspace).  Tokens equal to ``padding_idx`` give the table no
    gradient.  An id outside the table reads as a row of zeros, adds nothing to
    the gradient, and makes the next ``status()`` True.  Calls on one handle
    must not overlap on the GPU."""

    def __init__(self, num_embeddings, embedding_dim, max_tokens, padding_idx=None, scale=1.0, device=None):
        self.num_embeddings, self.embedding_dim = int(num_embeddings), int(embedding_dim)
        self.max_tokens = int(max_tokens)
        self.padding_idx = None if padding_idx is None else int(padding_idx)
        if self.padding_idx is not None and not 0 <= self.padding_idx < self.num_embeddings:
            raise ValueError("padding_idx must be a row of the table")
        self.scale = float(scale)
        self.device = _device(device)
        self._lib = _lib.lib()
        handle = ctypes.c_void_p()
        check(self._lib.psgd_embedding_create(self.num_embeddings, self.embedding_dim, self.max_tokens,
                                              self.device.index, ctypes.byref(handle)))
        self._h = handle
        self._spec = _bind.spec(handle.value, self.num_embeddings, self.embedding_dim, self.scale,
                                -1 if self.padding_idx is None else self.padding_idx, self.device.index)

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            if getattr(self, "_spec", None) is not None:
                _bind.closed(self._spec)
            self._lib.psgd_embedding_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, weight, ids, out=None, out_dtype=None, stream=None):
        """``scale * weight[ids]``, of shape ids.shape + (embedding_dim,), in
        ``out`` or a new tensor of ``out_dtype`` (default: the weight's)."""
        if stream is None:
            return _bind.embedding_forward(self._spec, weight, ids, out, out_dtype)
        with _on(stream, self.device.index):
            return _bind.embedding_forward(self._spec, weight, ids, out, out_dtype)

    def backward(self, ids, grad, out=None, accumulate=False, stream=None):
        """The table's gradient, ``scale`` times each row's sum of ``grad``
        (ids.shape + (embedding_dim,)) over its tokens, into ``out`` (default: a
        new fp32 tensor), over what it holds or, with ``accumulate``, added to it."""
        if stream is None:
            return _bind.embedding_backward(self._spec, ids, grad, out, accumulate)
        with _on(stream, self.device.index):
            return _bind.embedding_backward(self._spec, ids, grad, out, accumulate)

    def status(self, stream=None):
        """Synchronises; True when an id outside the table was met since the last status()."""
        index = self.device.index
        stream = torch.cuda.current_stream(index) if stream is None else _of_device(stream, index)
        return check(self._lib.psgd_embedding_status(self._h, stream.cuda_stream)) == PSGD_BAD_TOKEN

    def workspace_bytes(self):
        return int(self._lib.psgd_embedding_workspace_bytes(self._h))


class LayerNorm:
    """Layer norm over a last dimension of ``normalized_size`` elements.  The
    handle holds the partial sums of the parameters' gradients; backward calls
    on one handle must not overlap on the GPU."""

    def __init__(self, normalized_size, eps=1e-5, device=None):
        self.dim, self.eps = int(normalized_size), float(eps)
        self.device = _device(device)
        self._lib = _lib.lib()
        handle = ctypes.c_void_p()
        check(self._lib.psgd_layernorm_create(self.dim, self.device.index, ctypes.byref(handle)))
        self._h = handle
        self._spec = _bind.spec(handle.value, 0, self.dim, self.eps, -1, self.device.index)

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            if getattr(self, "_spec", None) is not None:
                _bind.closed(self._spec)
            self._lib.psgd_layernorm_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, x, weight=None, bias=None, out=None, stream=None):
        """(y, mean, rstd); mean and rstd (fp32, one a row) are what backward takes."""
        if stream is None:
            return _bind.layernorm_forward(self._spec, x, weight, bias, out)
        with _on(stream, self.device.index):
            return _bind.layernorm_forward(self._spec, x, weight, bias, out)

    def backward(self, grad, x, mean, rstd, weight=None, dx=None, dweight=None, dbias=None, accumulate=False,
                 stream=None):
        """(dx, dweight, dbias).  ``dweight`` and ``dbias`` (default: new fp32
        vectors) are overwritten or, with ``accumulate``, added to."""
        if stream is None:
            return _bind.layernorm_backward(self._spec, grad, x, mean, rstd, weight, dx, dweight, dbias, accumulate)
        with _on(stream, self.device.index):
            return _bind.layernorm_backward(self._spec, grad, x, mean, rstd, weight, dx, dweight, dbias, accumulate)

    def workspace_bytes(self):
        return int(self._lib.psgd_layernorm_workspace_bytes(self._h))


def distill_loss(logits, teacher_logits, teacher_indices, temperature=1.0, weights=None, grad_scale=1.0, dlogits=None,
                 with_grad=True, stream=None):
    """(losses, dlogits) of distillation from a teacher's top logits.

    ``logits`` (..., V); ``teacher_logits`` and ``teacher_indices`` (..., k),
    filled up with index -1 where a row has fewer than k; ``weights`` (...) in
    fp32, multiplied into loss and gradient (a row of weight 0 has neither,
    whatever its logits hold); ``grad_scale`` multiplies the gradient only (a
    loss scale).  ``dlogits`` (default: a new tensor) may be ``logits``
    itself.  with_grad=False: (losses, None)."""
    if stream is None:
        return _bind.distill(logits, teacher_logits, teacher_indices, temperature, weights, grad_scale, dlogits, with_grad)
    index = logits.get_device() if isinstance(logits, torch.Tensor) and logits.is_cuda else stream.device.index
    with _on(stream, index):
        return _bind.distill(logits, teacher_logits, teacher_indices, temperature, weights, grad_scale, dlogits, with_grad)
