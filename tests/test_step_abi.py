"""CPU checks of the C entry points of the norm and the 8-bit checkpoints: bad
arguments are refused with a message before any CUDA call."""

import ctypes

import pytest

from powersgd_rank_gradient_gb300 import _lib

F32 = _lib.PSGD_F32


def message():
    return _lib.lib().psgd_last_error().decode()


@pytest.mark.parametrize("dim,device", [(0, 0), (2**20 + 1, 0), (8, 64), (8, -1)])
def test_rmsnorm_create_refuses(dim, device):
    h = ctypes.c_void_p(1)
    assert _lib.lib().psgd_rmsnorm_create(dim, device, ctypes.byref(h)) == _lib.PSGD_EINVAL
    assert not h.value and "psgd_rmsnorm_create" in message()


def test_null_handles():
    L = _lib.lib()
    assert L.psgd_rmsnorm_create(8, 0, None) == _lib.PSGD_EINVAL
    assert L.psgd_rmsnorm_forward(None, None, F32, 8, 1, None, 8, None, F32, 0.0, None, 8, None, 0, None, None, 8, None,
                                  None) == _lib.PSGD_EINVAL
    assert L.psgd_rmsnorm_backward(None, None, F32, 8, 1, None, 8, None, 0, None, None, None, F32, None, 8, None, 8, None, F32, 0,
                                   None) == _lib.PSGD_EINVAL
    assert L.psgd_rmsnorm_workspace_bytes(None) == 0
    L.psgd_rmsnorm_destroy(None)


def save(dtype=F32, stride=50, rows=4, dim=50, code=0, device=0, x=1 << 20, codes=1 << 21, scales=1 << 22):
    """psgd_activation_save with made-up addresses, which only calls that are refused (or have no rows) may be given."""
    return _lib.lib().psgd_activation_save(x, dtype, stride, rows, dim, codes, code, scales, device, None)


def restore(dtype=F32, stride=50, rows=4, dim=50, code=0, device=0, x=1 << 20, codes=1 << 21, scales=1 << 22):
    return _lib.lib().psgd_activation_restore(codes, code, scales, rows, dim, x, dtype, stride, device, None)


@pytest.mark.parametrize("call", [save, restore])
@pytest.mark.parametrize("kw,words", [
    (dict(dtype=9), "dtype"), (dict(code=2), "8-bit"), (dict(rows=-1), "rows"), (dict(rows=2**31), "rows"), (dict(dim=0), "dim"),
    (dict(dim=2**31), "dim"), (dict(device=64), "device"), (dict(device=-1), "device"), (dict(stride=-1), "stride"),
    (dict(stride=2**60), "stride"), (dict(rows=2**29, dim=2**29, stride=0), "stride"), (dict(x=None), "NULL"), (dict(codes=None), "NULL"),
    (dict(scales=None), "NULL"), (dict(codes=(1 << 20) + 4), "overlap"), (dict(scales=(1 << 21) + 8), "overlap"),
])
def test_activation_refuses(call, kw, words):
    assert call(**kw) == _lib.PSGD_EINVAL
    assert words in message()


def test_restore_refuses_rows_that_overlap():
    assert restore(stride=49) == _lib.PSGD_EINVAL and "overlap" in message()


@pytest.mark.parametrize("call", [save, restore])
def test_no_rows_do_nothing(call):
    assert call(rows=0, x=None, codes=None, scales=None) == _lib.PSGD_OK


@pytest.mark.parametrize("outs,ins,rows,device", [(0, 8, 8, 0), (8, 0, 8, 0), (2**20 + 1, 8, 8, 0), (8, 2**20 + 1, 8, 0), (8, 8, -1, 0),
                                                  (8, 8, 2**24 + 1, 0), (8, 8, 8, 64), (8, 8, 8, -1)])
def test_wgrad_create_refuses(outs, ins, rows, device):
    h = ctypes.c_void_p(1)
    assert _lib.lib().psgd_wgrad_create(outs, ins, rows, device, ctypes.byref(h)) == _lib.PSGD_EINVAL
    assert not h.value and "psgd_wgrad_create" in message()


@pytest.mark.parametrize("vocab,dim,tokens,device", [(0, 8, 8, 0), (2**24 + 1, 8, 8, 0), (8, 0, 8, 0), (8, 2**20 + 1, 8, 0), (8, 8, -1, 0),
                                                     (8, 8, 2**20 + 1, 0), (8, 8, 8, 64), (8, 8, 8, -1)])
def test_linear_ce_create_refuses(vocab, dim, tokens, device):
    h = ctypes.c_void_p(1)
    assert _lib.lib().psgd_linear_ce_create(vocab, dim, tokens, device, ctypes.byref(h)) == _lib.PSGD_EINVAL
    assert not h.value and "psgd_linear_ce_create" in message()


def test_null_product_handles():
    L = _lib.lib()
    bf16 = _lib.PSGD_BF16
    assert L.psgd_wgrad_create(8, 8, 8, 0, None) == _lib.PSGD_EINVAL
    assert L.psgd_linear_ce_create(8, 8, 8, 0, None) == _lib.PSGD_EINVAL
    assert L.psgd_wgrad_backward(None, None, bf16, 8, 1, None, 0, None, None, F32, 8, 0, None) == _lib.PSGD_EINVAL
    assert L.psgd_linear_ce_forward(None, None, bf16, 8, 1, None, 8, None, 64, None, None, None, None) == _lib.PSGD_EINVAL
    assert L.psgd_linear_ce_backward(None, None, bf16, 8, 1, None, 8, None, 64, None, None, 1.0, None, 8, None, F32, 8, 0,
                                     None) == _lib.PSGD_EINVAL
    assert L.psgd_wgrad_status(None, None) == _lib.PSGD_EINVAL and L.psgd_linear_ce_status(None, None) == _lib.PSGD_EINVAL
    assert L.psgd_wgrad_workspace_bytes(None) == 0 and L.psgd_linear_ce_workspace_bytes(None) == 0
    L.psgd_wgrad_destroy(None)
    L.psgd_linear_ce_destroy(None)
