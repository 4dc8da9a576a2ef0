"""Training operators: what fills the gradient buckets.

``Embedding`` (lookup with scaling, and the dense gradient of its table),
``LayerNorm`` (forward, and backward with the reduction of the parameters'
gradients) and ``distill_loss`` (losses and logits' gradient of distillation
from a teacher's top logits).  Parameter gradients are written into tensors
the caller passes, typically views of a flat replica bucket at any element
offset and in the bucket's type, so that ``powerSGD_hook`` takes the bucket as
it is.  torch is used for device memory and streams; the arithmetic runs in the
CUDA kernels of libpsgd.so.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import PSGD_BAD_TOKEN, PSGD_BF16, PSGD_F16, PSGD_F32, check

_DTYPE = {torch.float32: PSGD_F32, torch.float16: PSGD_F16, torch.bfloat16: PSGD_BF16}
_ID_BITS = {torch.int32: 32, torch.int64: 64}


def _device(device):
    if device is None:
        device = torch.cuda.current_device()
    device = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
    if device.type != "cuda":
        raise ValueError("device must be a CUDA device")
    return torch.device("cuda", torch.cuda.current_device()) if device.index is None else device


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _new(shape, dtype, device, stream):
    """A new tensor, from the memory of the stream that writes it first."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _dtype(t, what):
    try:
        return _DTYPE[t.dtype]
    except KeyError:
        raise ValueError(f"{what} must be float32, float16 or bfloat16, got {t.dtype}") from None


def _on(t, device, what):
    if t.device != device:
        raise ValueError(f"{what} must be on {device}, got {t.device}")


def _layout(t, lead, what):
    """(outer, inner, outer stride, inner stride) of the first ``lead``
    dimensions of ``t``, which must be expressible as two."""
    shape, stride = t.shape[:lead], t.stride()[:lead]
    if lead == 0:
        return 1, 1, 0, 0
    if lead == 1:
        return 1, shape[0], 0, stride[0]
    if lead == 2:
        return shape[0], shape[1], stride[0], stride[1]
    # more than two: all but the last must collapse into one
    outer = 1
    for d in range(lead - 1):
        outer *= shape[d]
    if outer == 0 or shape[lead - 1] == 0:
        return 0, 0, 0, 0
    step = None
    run = 1
    for d in range(lead - 2, -1, -1):
        if shape[d] != 1:
            if step is None:
                step = stride[d] // run if run else 0
            if stride[d] != step * run:
                raise ValueError(f"{what}: its leading dimensions must be contiguous among themselves")
        run *= shape[d]
    return outer, shape[lead - 1], step or 0, stride[lead - 1]


def _rows(t, dim, what):
    """(rows, row stride) of a tensor of rows of ``dim`` elements."""
    if dim < 1 or t.dim() < 1 or t.shape[-1] != dim:
        raise ValueError(f"{what} must have a last dimension of {max(dim, 1)}, got {tuple(t.shape)}")
    if dim > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what} must be contiguous in its last dimension")
    if t.is_contiguous():
        return t.numel() // dim, dim
    if t.dim() == 2:
        return t.shape[0], t.stride(0)
    outer, inner, os, is_ = _layout(t, t.dim() - 1, what)
    if outer > 1 and inner > 1 and os != inner * is_:
        raise ValueError(f"{what}: its rows must be one stride apart")
    return outer * inner, is_ if inner > 1 else os


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

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            self._lib.psgd_embedding_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _ids(self, ids):
        if ids.dtype not in _ID_BITS:
            raise ValueError(f"ids must be int32 or int64, got {ids.dtype}")
        _on(ids, self.device, "ids")
        return _layout(ids, ids.dim(), "ids")

    def _table(self, t, what):
        if t.dim() != 2 or t.shape[0] != self.num_embeddings or t.shape[1] != self.embedding_dim:
            raise ValueError(f"{what} must be ({self.num_embeddings}, {self.embedding_dim}), got {tuple(t.shape)}")
        if self.embedding_dim > 1 and t.stride(1) != 1:
            raise ValueError(f"{what} must be contiguous in its last dimension")
        _on(t, self.device, what)
        return _dtype(t, what), t.stride(0) if self.num_embeddings > 1 else self.embedding_dim

    def _token_rows(self, t, ids, what):
        if t.dim() != ids.dim() + 1 or t.shape[:-1] != ids.shape or t.shape[-1] != self.embedding_dim:
            raise ValueError(f"{what} must be {tuple(ids.shape) + (self.embedding_dim,)}, got {tuple(t.shape)}")
        if self.embedding_dim > 1 and t.stride(-1) != 1:
            raise ValueError(f"{what} must be contiguous in its last dimension")
        _on(t, self.device, what)
        return _dtype(t, what), *_layout(t, t.dim() - 1, what)[2:]

    def forward(self, weight, ids, out=None, out_dtype=None, stream=None):
        """``scale * weight[ids]``, of shape ids.shape + (embedding_dim,), in
        ``out`` or a new tensor of ``out_dtype`` (default: the weight's)."""
        wd, ws = self._table(weight, "weight")
        outer, inner, os, is_ = self._ids(ids)
        if out is None:
            out = _new(ids.shape + (self.embedding_dim,), out_dtype or weight.dtype, self.device, stream)
        od, oos, ois = self._token_rows(out, ids, "out")
        check(self._lib.psgd_embedding_forward(
            self._h, weight.data_ptr(), wd, ws, ids.data_ptr(), _ID_BITS[ids.dtype], outer, inner, os, is_, self.scale,
            out.data_ptr(), od, oos, ois, _stream(stream, self.device)))
        return out

    def backward(self, ids, grad, out=None, accumulate=False, stream=None):
        """The table's gradient, ``scale`` times each row's sum of ``grad``
        (ids.shape + (embedding_dim,)) over its tokens, into ``out`` (default: a
        new fp32 tensor), over what it holds or, with ``accumulate``, added to it."""
        outer, inner, os, is_ = self._ids(ids)
        gd, gos, gis = self._token_rows(grad, ids, "grad")
        if out is None:
            if accumulate:
                raise ValueError("accumulate needs an out to add to")
            out = _new((self.num_embeddings, self.embedding_dim), torch.float32, self.device, stream)
        wd, ws = self._table(out, "out")
        check(self._lib.psgd_embedding_backward(
            self._h, ids.data_ptr(), _ID_BITS[ids.dtype], outer, inner, os, is_, grad.data_ptr(), gd, gos, gis,
            self.scale, -1 if self.padding_idx is None else self.padding_idx, int(accumulate), out.data_ptr(), wd, ws,
            _stream(stream, self.device)))
        return out

    def status(self, stream=None):
        """Synchronises; True when an id outside the table was met since the last status()."""
        return check(self._lib.psgd_embedding_status(self._h, _stream(stream, self.device))) == PSGD_BAD_TOKEN

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

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            self._lib.psgd_layernorm_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _param(self, t, what):
        if t.dim() != 1 or t.shape[0] != self.dim or (self.dim > 1 and t.stride(0) != 1):
            raise ValueError(f"{what} must be a contiguous vector of {self.dim} elements")
        _on(t, self.device, what)
        return _dtype(t, what)

    def _pair(self, a, b, names):
        """dtype and addresses of two optional vectors of one type."""
        da = None if a is None else self._param(a, names[0])
        db = None if b is None else self._param(b, names[1])
        if da is not None and db is not None and da != db:
            raise ValueError(f"{names[0]} and {names[1]} must have one type")
        return (da if da is not None else db if db is not None else PSGD_F32,
                None if a is None else a.data_ptr(), None if b is None else b.data_ptr())

    def _stat(self, t, rows, what):
        if t.dtype != torch.float32 or t.numel() != rows or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous float32 tensor of {rows} elements")
        _on(t, self.device, what)

    def forward(self, x, weight=None, bias=None, out=None, stream=None):
        """(y, mean, rstd); mean and rstd (fp32, one a row) are what backward takes."""
        xd = _dtype(x, "x")
        _on(x, self.device, "x")
        rows, xs = _rows(x, self.dim, "x")
        pd, w, b = self._pair(weight, bias, ("weight", "bias"))
        if out is None:
            out = _new(x.shape, x.dtype, self.device, stream)
        elif out.shape != x.shape or out.dtype != x.dtype:
            raise ValueError("out must have x's shape and type")
        else:
            _on(out, self.device, "out")
        _, ys = _rows(out, self.dim, "out")
        stats = _new((2,) + x.shape[:-1], torch.float32, self.device, stream)
        mean, rstd = stats[0], stats[1]
        check(self._lib.psgd_layernorm_forward(
            self._h, x.data_ptr(), xd, xs, rows, w, b, pd, self.eps, out.data_ptr(), ys, mean.data_ptr(),
            rstd.data_ptr(), _stream(stream, self.device)))
        return out, mean, rstd

    def backward(self, grad, x, mean, rstd, weight=None, dx=None, dweight=None, dbias=None, accumulate=False,
                 stream=None):
        """(dx, dweight, dbias).  ``dweight`` and ``dbias`` (default: new fp32
        vectors) are overwritten or, with ``accumulate``, added to."""
        xd = _dtype(x, "x")
        _on(x, self.device, "x")
        if grad.shape != x.shape or grad.dtype != x.dtype:
            raise ValueError("grad must have x's shape and type")
        _on(grad, self.device, "grad")
        rows, xs = _rows(x, self.dim, "x")
        _, gs = _rows(grad, self.dim, "grad")
        self._stat(mean, rows, "mean")
        self._stat(rstd, rows, "rstd")
        pd, w, _ = self._pair(weight, None, ("weight", ""))
        if dx is None:
            dx = _new(x.shape, x.dtype, self.device, stream)
        elif dx.shape != x.shape or dx.dtype != x.dtype:
            raise ValueError("dx must have x's shape and type")
        else:
            _on(dx, self.device, "dx")
        _, ds = _rows(dx, self.dim, "dx")
        if accumulate and (dweight is None or dbias is None):
            raise ValueError("accumulate needs a dweight and a dbias to add to")
        if dweight is None:
            dweight = _new(self.dim, torch.float32 if dbias is None else dbias.dtype, self.device, stream)
        if dbias is None:
            dbias = _new(self.dim, dweight.dtype, self.device, stream)
        od, dw, db = self._pair(dweight, dbias, ("dweight", "dbias"))
        check(self._lib.psgd_layernorm_backward(
            self._h, grad.data_ptr(), gs, x.data_ptr(), xd, xs, rows, mean.data_ptr(), rstd.data_ptr(), w, pd,
            dx.data_ptr(), ds, dw, db, od, int(accumulate), _stream(stream, self.device)))
        return dx, dweight, dbias

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
    if logits.device.type != "cuda":
        raise ValueError("logits must be a CUDA tensor")
    device = logits.device
    if logits.dim() < 1:
        raise ValueError("logits must have a vocabulary dimension")
    vocab = logits.shape[-1]
    zd = _dtype(logits, "logits")
    lead = logits.shape[:-1]
    rows, zs = _rows(logits, vocab, "logits")
    if teacher_logits.dim() < 1 or teacher_logits.shape != teacher_indices.shape or teacher_logits.shape[:-1] != lead:
        raise ValueError("teacher_logits and teacher_indices must have the logits' leading shape and one k")
    k = teacher_logits.shape[-1]
    td = _dtype(teacher_logits, "teacher_logits")
    if teacher_indices.dtype not in _ID_BITS:
        raise ValueError(f"teacher_indices must be int32 or int64, got {teacher_indices.dtype}")
    _on(teacher_logits, device, "teacher_logits")
    _on(teacher_indices, device, "teacher_indices")
    _, ts = _rows(teacher_logits, k, "teacher_logits")
    _, ns = _rows(teacher_indices, k, "teacher_indices")
    w = None
    if weights is not None:
        if weights.dtype != torch.float32 or weights.shape != lead or not weights.is_contiguous():
            raise ValueError("weights must be a contiguous float32 tensor of the logits' leading shape")
        _on(weights, device, "weights")
        w = weights.data_ptr()
    ds = 0
    if with_grad:
        if dlogits is None:
            dlogits = _new(logits.shape, logits.dtype, device, stream)
        elif dlogits.shape != logits.shape or dlogits.dtype != logits.dtype:
            raise ValueError("dlogits must have the logits' shape and type")
        else:
            _on(dlogits, device, "dlogits")
        _, ds = _rows(dlogits, vocab, "dlogits")
    elif dlogits is not None:
        raise ValueError("dlogits given with with_grad=False")
    losses = _new(lead, torch.float32, device, stream)
    lib = _lib.lib()
    with torch.cuda.device(device):
        check(lib.psgd_distill(
            logits.data_ptr(), zd, zs, rows, vocab, teacher_logits.data_ptr(), td, ts, teacher_indices.data_ptr(),
            _ID_BITS[teacher_indices.dtype], ns, k, float(temperature), w, float(grad_scale), losses.data_ptr(),
            dlogits.data_ptr() if with_grad else None, ds, _stream(stream, device)))
    return losses, dlogits
