"""Training operators: what fills the gradient buckets.

``Embedding`` (lookup with scaling, and the dense gradient of its table),
``LayerNorm`` (forward, and backward with the reduction of the parameters'
gradients), ``distill_loss`` (losses and logits' gradient of distillation
from a teacher's top logits), and what keeps a step's memory small: ``RMSNorm``
(with the residual's addition, an output in 8 bits, a backward pass that reads
one), activation checkpoints in 8 bits (``save_activation``, ``Activation8``)
with the weight gradient of a linear layer from one (``LinearWeightGrad``), and
``LinearCrossEntropy`` (losses and gradients of an output layer without its
logits).  Parameter gradients are written into tensors
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


class Activation8:
    """An activation kept in 8 bits: ``codes`` (float8_e4m3fn or float8_e5m2, of the
    activation's shape) and ``scales`` (float32, one for each 128 elements of a
    row: (..., ceil(dim / 128))), both contiguous.  Scales that this package makes
    are powers of two; it stands for codes times scales."""

    __slots__ = ("codes", "scales")

    def __init__(self, codes, scales):
        _bind.activation_check(codes, scales)
        self.codes, self.scales = codes, scales

    @classmethod
    def _made(cls, codes, scales):
        a = cls.__new__(cls)
        a.codes, a.scales = codes, scales
        return a

    @property
    def shape(self):
        return self.codes.shape

    @property
    def dtype(self):
        return self.codes.dtype

    @property
    def device(self):
        return self.codes.device

    def restore(self, dtype=torch.bfloat16, out=None, stream=None):
        """The values it stands for, in ``out`` or a new tensor of ``dtype`` (float32, float16 or bfloat16)."""
        if stream is None:
            return _bind.activation_restore(self.codes, self.scales, dtype, out)
        with _on(stream, self.codes.get_device()):
            return _bind.activation_restore(self.codes, self.scales, dtype, out)


def _eight(a, what):
    """(codes, scales) of ``a``, which must be an ``Activation8`` (or None: None of each)."""
    if a is None:
        return None, None
    if not isinstance(a, Activation8):
        raise ValueError(f"{what} must be an Activation8, got {type(a).__name__}")
    return a.codes, a.scales


def _index_of(t, stream):
    return t.get_device() if isinstance(t, torch.Tensor) and t.is_cuda else stream.device.index


def save_activation(x, dtype=torch.float8_e4m3fn, out=None, stream=None):
    """``x`` (..., dim) as an ``Activation8`` of ``dtype`` (float8_e4m3fn or
    float8_e5m2), a new one or ``out``.

    A block of 128 elements of a row has one scale, the least power of two that
    brings its largest value within the format; a code is its element, rounded
    once.  Infinities and NaN become NaN (e5m2 keeps infinities)."""
    codes, scales = _eight(out, "out")
    if stream is None:
        codes, scales = _bind.activation_save(x, dtype, codes, scales)
    else:
        with _on(stream, _index_of(x, stream)):
            codes, scales = _bind.activation_save(x, dtype, codes, scales)
    return Activation8._made(codes, scales) if out is None else out


class RMSNorm:
    """Root-mean-square norm over a last dimension of ``normalized_size`` elements,
    with the residual's addition.  The handle holds the partial sums of the weight's
    gradient; backward calls on one handle must not overlap on the GPU."""

    def __init__(self, normalized_size, eps=1e-6, device=None):
        self.dim, self.eps = int(normalized_size), float(eps)
        self.device = _device(device)
        self._lib = _lib.lib()
        handle = ctypes.c_void_p()
        check(self._lib.psgd_rmsnorm_create(self.dim, self.device.index, ctypes.byref(handle)))
        self._h = handle
        self._spec = _bind.spec(handle.value, 0, self.dim, self.eps, -1, self.device.index)

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            if getattr(self, "_spec", None) is not None:
                _bind.closed(self._spec)
            self._lib.psgd_rmsnorm_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, x, weight=None, residual=None, out=None, summed=None, stream=None):
        """(y, summed, rstd): ``summed`` is x + residual in x's type (a new tensor, the
        one given, which may be ``x`` or ``residual`` itself, or without a residual x),
        rstd = (mean(summed^2) + eps)^-1/2 in fp32, y = summed * rstd * weight.
        backward takes summed and rstd."""
        if stream is None:
            return _bind.rmsnorm_forward(self._spec, x, weight, residual, out, summed, None, None, None)
        with _on(stream, self.device.index):
            return _bind.rmsnorm_forward(self._spec, x, weight, residual, out, summed, None, None, None)

    def forward8(self, x, weight=None, residual=None, dtype=torch.float8_e4m3fn, out=None, summed=None, stream=None):
        """(y, summed, rstd) with y an ``Activation8`` of ``dtype`` (a new one, or ``out``)."""
        codes, scales = _eight(out, "out")
        if stream is None:
            codes, scales, summed, rstd = _bind.rmsnorm_forward(self._spec, x, weight, residual, None, summed, dtype, codes, scales)
        else:
            with _on(stream, self.device.index):
                codes, scales, summed, rstd = _bind.rmsnorm_forward(self._spec, x, weight, residual, None, summed, dtype, codes,
                                                                    scales)
        return (Activation8._made(codes, scales) if out is None else out), summed, rstd

    def backward(self, grad, summed, rstd, weight=None, grad_summed=None, dx=None, dweight=None, accumulate=False, stream=None):
        """(dx, dweight).  ``summed``: as forward gave it, or an ``Activation8`` of it.
        ``grad_summed``: the gradient that reaches the sum past the norm, added to dx
        (which is the gradient of both x and the residual); ``dx`` may be ``grad`` or
        ``grad_summed`` itself.  ``dweight`` (default: a new fp32 vector) is overwritten
        or, with ``accumulate``, added to."""
        codes = scales = None
        if isinstance(summed, Activation8):
            summed, codes, scales = None, summed.codes, summed.scales
        if stream is None:
            return _bind.rmsnorm_backward(self._spec, grad, summed, codes, scales, rstd, weight, grad_summed, dx, dweight, accumulate)
        with _on(stream, self.device.index):
            return _bind.rmsnorm_backward(self._spec, grad, summed, codes, scales, rstd, weight, grad_summed, dx, dweight, accumulate)

    def workspace_bytes(self):
        return int(self._lib.psgd_rmsnorm_workspace_bytes(self._h))


class LinearWeightGrad:
    """The weight gradient of a linear layer ``y = x W^T``, W of ``out_features`` rows
    of ``in_features`` elements, from an 8-bit checkpoint of x.

    ``max_tokens`` bounds the rows of one call (the handle holds the restored
    checkpoint, a bounded piece of a gradient that begins between two 16-byte units and a
    product's partial sums; layers of one shape may share it).
    Calls on one handle must not overlap on the GPU."""

    def __init__(self, out_features, in_features, max_tokens, device=None):
        self.out_features, self.in_features, self.max_tokens = int(out_features), int(in_features), int(max_tokens)
        self.device = _device(device)
        self._lib = _lib.lib()
        handle = ctypes.c_void_p()
        check(self._lib.psgd_wgrad_create(self.out_features, self.in_features, self.max_tokens, self.device.index,
                                          ctypes.byref(handle)))
        self._h = handle
        self._spec = _bind.spec(handle.value, self.out_features, self.in_features, 0.0, -1, self.device.index)

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            if getattr(self, "_spec", None) is not None:
                _bind.closed(self._spec)
            self._lib.psgd_wgrad_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def backward(self, grad, activation, out=None, accumulate=False, stream=None):
        """``grad^T x`` with grad (..., out_features) in float16 or bfloat16 and x the values of
        ``activation`` (an ``Activation8`` of (..., in_features)) in grad's type, into ``out``
        (default: a new fp32 tensor), over what it holds or, with ``accumulate``, added to it."""
        if activation is None:
            raise ValueError("activation must be an Activation8, got NoneType")
        codes, scales = _eight(activation, "activation")
        if stream is None:
            return _bind.wgrad_backward(self._spec, grad, codes, scales, out, accumulate)
        with _on(stream, self.device.index):
            return _bind.wgrad_backward(self._spec, grad, codes, scales, out, accumulate)

    def status(self, stream=None):
        """Synchronises; raises PsgdError if a bounded wait on the GPU gave up since the last status()."""
        index = self.device.index
        stream = torch.cuda.current_stream(index) if stream is None else _of_device(stream, index)
        check(self._lib.psgd_wgrad_status(self._h, stream.cuda_stream))

    def workspace_bytes(self):
        return int(self._lib.psgd_wgrad_workspace_bytes(self._h))


class LinearCrossEntropy:
    """Softmax cross entropy of an output layer ``hidden @ weight.t()`` over a vocabulary
    of ``vocab`` rows of ``dim`` elements, without the logits: they are made tile by
    tile and used where they are made, in the backward pass again.

    ``max_tokens`` bounds the tokens of one call (the handle holds them, bounded pieces of the
    logits' gradient and of a weight that begins between two 16-byte units, and partial sums: see
    ``workspace_bytes()``).  Calls on one handle must not overlap on the GPU.

    ``hidden`` (..., dim) and ``weight`` (vocab, dim) are float16 or bfloat16, of one
    type; ``targets`` (...) int32 or int64; ``weights`` (...) float32, multiplied into
    losses and gradients.  A token whose target is outside the vocabulary (-100, say) or
    whose weight is 0 does not count: loss, lse and gradient are 0 whatever its row
    holds, and it costs no arithmetic."""

    def __init__(self, vocab, dim, max_tokens, device=None):
        self.vocab, self.dim, self.max_tokens = int(vocab), int(dim), int(max_tokens)
        self.device = _device(device)
        self._lib = _lib.lib()
        handle = ctypes.c_void_p()
        check(self._lib.psgd_linear_ce_create(self.vocab, self.dim, self.max_tokens, self.device.index, ctypes.byref(handle)))
        self._h = handle
        self._spec = _bind.spec(handle.value, self.vocab, self.dim, 0.0, -1, self.device.index)

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            if getattr(self, "_spec", None) is not None:
                _bind.closed(self._spec)
            self._lib.psgd_linear_ce_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, hidden, weight, targets, weights=None, stream=None):
        """(losses, lse), fp32, of targets' shape: lse = log sum exp of a token's logits, loss = weight * (lse - its
        target's logit).  backward takes lse."""
        if stream is None:
            return _bind.linear_ce_forward(self._spec, hidden, weight, targets, weights)
        with _on(stream, self.device.index):
            return _bind.linear_ce_forward(self._spec, hidden, weight, targets, weights)

    def backward(self, hidden, weight, targets, lse, weights=None, grad_scale=1.0, dhidden=None, dweight=None, accumulate=False,
                 stream=None):
        """(dhidden, dweight), the gradients of the sum of the losses times ``grad_scale``.
        ``dhidden`` (default: a new tensor) has hidden's type; ``dweight`` (default: a new
        fp32 tensor) is overwritten or, with ``accumulate``, added to."""
        if stream is None:
            return _bind.linear_ce_backward(self._spec, hidden, weight, targets, lse, weights, grad_scale, dhidden, dweight, accumulate)
        with _on(stream, self.device.index):
            return _bind.linear_ce_backward(self._spec, hidden, weight, targets, lse, weights, grad_scale, dhidden, dweight, accumulate)

    def status(self, stream=None):
        """Synchronises; raises PsgdError if a bounded wait on the GPU gave up since the last status()."""
        index = self.device.index
        stream = torch.cuda.current_stream(index) if stream is None else _of_device(stream, index)
        check(self._lib.psgd_linear_ce_status(self._h, stream.cuda_stream))

    def workspace_bytes(self):
        return int(self._lib.psgd_linear_ce_workspace_bytes(self._h))
