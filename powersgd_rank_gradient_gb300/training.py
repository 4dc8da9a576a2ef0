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


# The current stream's handle without a Stream object around it, where this torch has the call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, index):
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _new(shape, dtype, device, stream):
    """A new tensor, from the memory of the stream that writes it first."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _new_like(t, stream):
    """A new contiguous tensor of ``t``'s shape and type."""
    return torch.empty_like(t) if stream is None and t.is_contiguous() else _new(t.shape, t.dtype, t.device, stream)


def _dtype(t, index, what):
    """The library's name of the type of ``t``, which must be on CUDA device ``index``."""
    d = _DTYPE.get(t.dtype)
    if d is None:
        raise ValueError(f"{what} must be float32, float16 or bfloat16, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{what} must be on cuda:{index}, got {t.device}")
    return d


def _id_bits(t, index, what):
    bits = _ID_BITS.get(t.dtype)
    if bits is None:
        raise ValueError(f"{what} must be int32 or int64, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{what} must be on cuda:{index}, got {t.device}")
    return bits


def _layout(shape, stride, what):
    """(outer, inner, outer stride, inner stride) of the given dimensions, which
    must be expressible as two."""
    lead = len(shape)
    if lead == 2:
        return shape[0], shape[1], stride[0], stride[1]
    if lead == 1:
        return 1, shape[0], 0, stride[0]
    if lead == 0:
        return 1, 1, 0, 0
    # more than two: all but the last must collapse into one
    outer = 1
    for d in range(lead - 1):
        outer *= shape[d]
    if outer == 0 or shape[lead - 1] == 0:
        return 0, 0, 0, 0
    step, run = None, 1
    for d in range(lead - 2, -1, -1):
        if shape[d] != 1:
            if step is None:
                step = stride[d]
            if stride[d] != step * run:
                raise ValueError(f"{what}: its leading dimensions must be contiguous among themselves")
            run *= shape[d]
    return outer, shape[lead - 1], step or 0, stride[lead - 1]


def _rows(t, dim, what):
    """(rows, row stride) of a tensor of rows of ``dim`` elements."""
    shape = t.shape
    if dim < 1 or len(shape) < 1 or shape[-1] != dim:
        raise ValueError(f"{what} must have a last dimension of {max(dim, 1)}, got {tuple(shape)}")
    if t.is_contiguous():
        return t.numel() // dim, dim
    stride = t.stride()
    if dim > 1 and stride[-1] != 1:
        raise ValueError(f"{what} must be contiguous in its last dimension")
    if len(shape) == 2:
        return shape[0], stride[0]
    outer, inner, os, is_ = _layout(shape[:-1], stride[:-1], what)
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
        self._index = self.device.index
        self._shape = (self.num_embeddings, self.embedding_dim)
        self._padding = -1 if self.padding_idx is None else self.padding_idx
        self._lib = _lib.lib()
        handle = ctypes.c_void_p()
        check(self._lib.psgd_embedding_create(self.num_embeddings, self.embedding_dim, self.max_tokens,
                                              self.device.index, ctypes.byref(handle)))
        self._h = handle
        self._forward, self._backward = self._lib.psgd_embedding_forward, self._lib.psgd_embedding_backward

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            self._lib.psgd_embedding_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _table(self, t, what):
        """(type, row stride) of a table."""
        if t.shape != self._shape:
            raise ValueError(f"{what} must be {self._shape}, got {tuple(t.shape)}")
        s0, s1 = t.stride()
        if s1 != 1 and self.embedding_dim > 1:
            raise ValueError(f"{what} must be contiguous in its last dimension")
        return _dtype(t, self._index, what), s0 if self.num_embeddings > 1 else self.embedding_dim

    def _token_rows(self, t, shape, what):
        """(type, outer stride, inner stride) of one row per token."""
        if t.shape != shape:
            raise ValueError(f"{what} must be {tuple(shape)}, got {tuple(t.shape)}")
        stride = t.stride()
        if stride[-1] != 1 and self.embedding_dim > 1:
            raise ValueError(f"{what} must be contiguous in its last dimension")
        d = _dtype(t, self._index, what)
        if len(shape) == 3:
            return d, stride[0], stride[1]
        return d, *_layout(shape[:-1], stride[:-1], what)[2:]

    def forward(self, weight, ids, out=None, out_dtype=None, stream=None):
        """``scale * weight[ids]``, of shape ids.shape + (embedding_dim,), in
        ``out`` or a new tensor of ``out_dtype`` (default: the weight's)."""
        wd, ws = self._table(weight, "weight")
        bits = _id_bits(ids, self._index, "ids")
        shape = ids.shape
        outer, inner, os, is_ = _layout(shape, ids.stride(), "ids")
        shape = (*shape, self.embedding_dim)
        if out is None:
            out = _new(shape, out_dtype or weight.dtype, self.device, stream)
            od, oos, ois = _DTYPE.get(out.dtype), inner * self.embedding_dim, self.embedding_dim
            if od is None:
                raise ValueError(f"out_dtype must be float32, float16 or bfloat16, got {out.dtype}")
        else:
            od, oos, ois = self._token_rows(out, shape, "out")
        rc = self._forward(
            self._h, weight.data_ptr(), wd, ws, ids.data_ptr(), bits, outer, inner, os, is_, self.scale,
            out.data_ptr(), od, oos, ois, _stream(stream, self._index))
        if rc:
            check(rc)
        return out

    def backward(self, ids, grad, out=None, accumulate=False, stream=None):
        """The table's gradient, ``scale`` times each row's sum of ``grad``
        (ids.shape + (embedding_dim,)) over its tokens, into ``out`` (default: a
        new fp32 tensor), over what it holds or, with ``accumulate``, added to it."""
        bits = _id_bits(ids, self._index, "ids")
        shape = ids.shape
        outer, inner, os, is_ = _layout(shape, ids.stride(), "ids")
        gd, gos, gis = self._token_rows(grad, (*shape, self.embedding_dim), "grad")
        if out is None:
            if accumulate:
                raise ValueError("accumulate needs an out to add to")
            out = _new(self._shape, torch.float32, self.device, stream)
        wd, ws = self._table(out, "out")
        rc = self._backward(
            self._h, ids.data_ptr(), bits, outer, inner, os, is_, grad.data_ptr(), gd, gos, gis, self.scale,
            self._padding, 1 if accumulate else 0, out.data_ptr(), wd, ws, _stream(stream, self._index))
        if rc:
            check(rc)
        return out

    def status(self, stream=None):
        """Synchronises; True when an id outside the table was met since the last status()."""
        return check(self._lib.psgd_embedding_status(self._h, _stream(stream, self._index))) == PSGD_BAD_TOKEN

    def workspace_bytes(self):
        return int(self._lib.psgd_embedding_workspace_bytes(self._h))


class LayerNorm:
    """Layer norm over a last dimension of ``normalized_size`` elements.  The
    handle holds the partial sums of the parameters' gradients; backward calls
    on one handle must not overlap on the GPU."""

    def __init__(self, normalized_size, eps=1e-5, device=None):
        self.dim, self.eps = int(normalized_size), float(eps)
        self._shape = (self.dim,)
        self.device = _device(device)
        self._index = self.device.index
        self._lib = _lib.lib()
        handle = ctypes.c_void_p()
        check(self._lib.psgd_layernorm_create(self.dim, self.device.index, ctypes.byref(handle)))
        self._h = handle
        self._forward, self._backward = self._lib.psgd_layernorm_forward, self._lib.psgd_layernorm_backward

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            self._lib.psgd_layernorm_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _pair(self, a, b, name_a, name_b):
        """(type, addresses) of two optional vectors of one type."""
        d = pa = pb = None
        if a is not None:
            if a.shape != self._shape or not a.is_contiguous():
                raise ValueError(f"{name_a} must be a contiguous vector of {self.dim} elements")
            d, pa = _dtype(a, self._index, name_a), a.data_ptr()
        if b is not None:
            if b.shape != self._shape or not b.is_contiguous():
                raise ValueError(f"{name_b} must be a contiguous vector of {self.dim} elements")
            e, pb = _dtype(b, self._index, name_b), b.data_ptr()
            if d is not None and d != e:
                raise ValueError(f"{name_a} and {name_b} must have one type")
            d = e
        return PSGD_F32 if d is None else d, pa, pb

    def _stat(self, t, rows, what):
        if t.dtype != torch.float32 or t.numel() != rows or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous float32 tensor of {rows} elements")
        if t.get_device() != self._index:
            raise ValueError(f"{what} must be on {self.device}, got {t.device}")
        return t.data_ptr()

    def _like(self, t, x, what):
        """The row stride of a tensor that must match ``x``."""
        if t.shape != x.shape or t.dtype != x.dtype:
            raise ValueError(f"{what} must have x's shape and type")
        if t.get_device() != self._index:
            raise ValueError(f"{what} must be on {self.device}, got {t.device}")
        return _rows(t, self.dim, what)[1]

    def forward(self, x, weight=None, bias=None, out=None, stream=None):
        """(y, mean, rstd); mean and rstd (fp32, one a row) are what backward takes."""
        index, device = self._index, self.device
        xd = _dtype(x, index, "x")
        rows, xs = _rows(x, self.dim, "x")
        pd, w, b = self._pair(weight, bias, "weight", "bias")
        if out is None:
            out, ys = _new_like(x, stream), self.dim
        else:
            ys = self._like(out, x, "out")
        shape = x.shape
        lead = (shape[0],) if len(shape) == 2 else shape[:-1]
        if stream is None:
            mean, rstd = (torch.empty(lead, dtype=torch.float32, device=device),
                          torch.empty(lead, dtype=torch.float32, device=device))
        else:
            mean, rstd = _new(lead, torch.float32, device, stream), _new(lead, torch.float32, device, stream)
        rc = self._forward(
            self._h, x.data_ptr(), xd, xs, rows, w, b, pd, self.eps, out.data_ptr(), ys, mean.data_ptr(),
            rstd.data_ptr(), _stream(stream, index))
        if rc:
            check(rc)
        return out, mean, rstd

    def backward(self, grad, x, mean, rstd, weight=None, dx=None, dweight=None, dbias=None, accumulate=False,
                 stream=None):
        """(dx, dweight, dbias).  ``dweight`` and ``dbias`` (default: new fp32
        vectors) are overwritten or, with ``accumulate``, added to."""
        xd = _dtype(x, self._index, "x")
        rows, xs = _rows(x, self.dim, "x")
        gs = self._like(grad, x, "grad")
        m, r = self._stat(mean, rows, "mean"), self._stat(rstd, rows, "rstd")
        pd, w, _ = self._pair(weight, None, "weight", "")
        if dx is None:
            dx, ds = _new_like(x, stream), self.dim
        else:
            ds = self._like(dx, x, "dx")
        if dweight is None or dbias is None:
            if accumulate:
                raise ValueError("accumulate needs a dweight and a dbias to add to")
            given = dweight if dweight is not None else dbias
            dtype = torch.float32 if given is None else given.dtype
            if dweight is None:
                dweight = _new((self.dim,), dtype, self.device, stream)
            if dbias is None:
                dbias = _new((self.dim,), dtype, self.device, stream)
        od, dw, db = self._pair(dweight, dbias, "dweight", "dbias")
        rc = self._backward(
            self._h, grad.data_ptr(), gs, x.data_ptr(), xd, xs, rows, m, r, w, pd, dx.data_ptr(), ds, dw, db, od,
            1 if accumulate else 0, _stream(stream, self._index))
        if rc:
            check(rc)
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
    index = logits.get_device()
    if index < 0:
        raise ValueError("logits must be a CUDA tensor")
    shape = logits.shape
    if len(shape) < 1:
        raise ValueError("logits must have a vocabulary dimension")
    vocab, lead = shape[-1], shape[:-1]
    zd = _dtype(logits, index, "logits")
    rows, zs = _rows(logits, vocab, "logits")
    tshape = teacher_logits.shape
    if len(tshape) < 1 or tshape != teacher_indices.shape or tshape[:-1] != lead:
        raise ValueError("teacher_logits and teacher_indices must have the logits' leading shape and one k")
    k = tshape[-1]
    td = _dtype(teacher_logits, index, "teacher_logits")
    bits = _id_bits(teacher_indices, index, "teacher_indices")
    ts = _rows(teacher_logits, k, "teacher_logits")[1]
    ns = _rows(teacher_indices, k, "teacher_indices")[1]
    w = None
    if weights is not None:
        if weights.dtype != torch.float32 or weights.shape != lead or not weights.is_contiguous():
            raise ValueError("weights must be a contiguous float32 tensor of the logits' leading shape")
        if weights.get_device() != index:
            raise ValueError(f"weights must be on {logits.device}, got {weights.device}")
        w = weights.data_ptr()
    dz, ds = None, 0
    if with_grad:
        if dlogits is None:
            dlogits, ds = _new_like(logits, stream), vocab
        else:
            if dlogits.shape != shape or dlogits.dtype != logits.dtype:
                raise ValueError("dlogits must have the logits' shape and type")
            if dlogits.get_device() != index:
                raise ValueError(f"dlogits must be on {logits.device}, got {dlogits.device}")
            ds = _rows(dlogits, vocab, "dlogits")[1]
        dz = dlogits.data_ptr()
    elif dlogits is not None:
        raise ValueError("dlogits given with with_grad=False")
    losses = _new(lead, torch.float32, logits.device, stream)
    check(_lib.lib().psgd_distill(
        logits.data_ptr(), zd, zs, rows, vocab, teacher_logits.data_ptr(), td, ts, teacher_indices.data_ptr(), bits, ns,
        k, temperature, w, grad_scale, losses.data_ptr(), dz, ds, index, _stream(stream, index)))
    return losses, dlogits
