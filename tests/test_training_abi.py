"""CPU checks of the training operators' C entry points: bad arguments are
refused with a message before any CUDA call."""

import ctypes

import pytest

from powersgd_rank_gradient_gb300 import _lib

F32 = _lib.PSGD_F32


def message():
    return _lib.lib().psgd_last_error().decode()


@pytest.mark.parametrize("vocab,dim,tokens,device", [(0, 8, 8, 0), (2**31 - 1, 8, 8, 0), (8, 0, 8, 0), (8, 2**20 + 1, 8, 0),
                                                     (8, 8, -1, 0), (8, 8, 2**31, 0), (8, 8, 8, 64), (8, 8, 8, -1)])
def test_embedding_create_refuses(vocab, dim, tokens, device):
    L = _lib.lib()
    h = ctypes.c_void_p(1)
    assert L.psgd_embedding_create(vocab, dim, tokens, device, ctypes.byref(h)) == _lib.PSGD_EINVAL
    assert not h.value and "psgd_embedding_create" in message()


@pytest.mark.parametrize("dim,device", [(0, 0), (2**20 + 1, 0), (8, 64), (8, -1)])
def test_layernorm_create_refuses(dim, device):
    L = _lib.lib()
    h = ctypes.c_void_p(1)
    assert L.psgd_layernorm_create(dim, device, ctypes.byref(h)) == _lib.PSGD_EINVAL
    assert not h.value and "psgd_layernorm_create" in message()


def test_null_handles():
    L = _lib.lib()
    assert L.psgd_embedding_create(8, 8, 8, 0, None) == _lib.PSGD_EINVAL
    assert L.psgd_layernorm_create(8, 0, None) == _lib.PSGD_EINVAL
    assert L.psgd_embedding_forward(None, None, F32, 8, None, 32, 1, 1, 1, 1, 1.0, None, F32, 8, 8, None) == _lib.PSGD_EINVAL
    assert L.psgd_embedding_backward(None, None, 32, 1, 1, 1, 1, None, F32, 8, 8, 1.0, -1, 0, None, F32, 8,
                                     None) == _lib.PSGD_EINVAL
    assert L.psgd_embedding_status(None, None) == _lib.PSGD_EINVAL
    assert L.psgd_layernorm_forward(None, None, F32, 8, 1, None, None, F32, 0.0, None, 8, None, None,
                                    None) == _lib.PSGD_EINVAL
    assert L.psgd_layernorm_backward(None, None, 8, None, F32, 8, 1, None, None, None, F32, None, 8, None, None, F32, 0,
                                     None) == _lib.PSGD_EINVAL
    assert L.psgd_embedding_workspace_bytes(None) == 0 and L.psgd_layernorm_workspace_bytes(None) == 0
    L.psgd_embedding_destroy(None)
    L.psgd_layernorm_destroy(None)


def distill(dtype=F32, stride=50, rows=4, vocab=50, tdtype=F32, bits=64, k=6, t=1.0, null=(), dz=False, dz_at=1 << 24,
            dz_stride=50, device=0):
    """psgd_distill with made-up addresses, which only calls that are refused (or have no rows) may be given."""
    at = dict(logits=1 << 20, teacher=1 << 21, index=1 << 22, losses=1 << 23)
    at.update({n: None for n in null})
    return _lib.lib().psgd_distill(at["logits"], dtype, stride, rows, vocab, at["teacher"], tdtype, 6, at["index"], bits, 6, k,
                                   t, None, 1.0, at["losses"], dz_at if dz else None, dz_stride, device, None)


@pytest.mark.parametrize("kw,words", [
    (dict(dtype=9), "dtype"), (dict(tdtype=-1), "dtype"), (dict(bits=16), "index_bits"), (dict(rows=-1), "rows"),
    (dict(rows=2**31), "rows"), (dict(vocab=0), "vocab"), (dict(vocab=2**30 + 1), "vocab"), (dict(k=0), "k must"), (dict(device=64), "device"), (dict(device=-1), "device"),
    (dict(k=_lib.PSGD_DISTILL_MAX_K + 1), "k must"), (dict(t=0.0), "temperature"), (dict(t=float("nan")), "temperature"),
    (dict(null=["logits"]), "NULL"), (dict(null=["teacher"]), "NULL"), (dict(null=["index"]), "NULL"),
    (dict(null=["losses"]), "NULL"), (dict(stride=-1), "stride"), (dict(stride=2**60), "stride"),
    (dict(dz=True, dz_stride=49), "overlap"), (dict(dz=True, dz_at=(1 << 20) + 4), "overlap"),
    (dict(dz=True, dz_at=1 << 23), "overlap"), (dict(dz=True, dz_at=1 << 20, stride=60), "overlap"),
])
def test_distill_refuses(kw, words):
    assert distill(**kw) == _lib.PSGD_EINVAL
    assert words in message()


def test_distill_without_rows_does_nothing():
    assert distill(rows=0) == _lib.PSGD_OK
