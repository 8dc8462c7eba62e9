"""Refusals of the 4-bit floating-point cache's and the windowed
verification's entry points, on the CPU: the C checks run before any CUDA
call (the pointers are fake addresses that nothing dereferences), the
binding's before the library is called."""

import ctypes

import pytest
import torch

from lossless_draft_verify_vc_b200 import vc

A = 0x100000  # aligned fake device address
M = 0x100008  # 8 bytes off a 16-byte boundary
INVALID = -1
WS = 1 << 40


@pytest.fixture(scope="module")
def L():
    return vc.lib()


def _refused(L, status, who):
    assert status == INVALID, status
    assert who in L.vc_last_error().decode(), L.vc_last_error()


def _fc(**kw):
    f = dict(records=A, T_cap=1024, T=1000, lens=0, k_exp=0, v_exp=0)
    f.update(kw)
    return vc.vc_fp4_cache(*f.values())


@pytest.mark.parametrize("shape,cache,args", [
    ((0, 4, 1, 128), {}, {}),
    ((70000, 4, 1, 128), {}, {}),                # B * Hkv > 65535
    ((1, 4, 1, 96), {}, {}),                     # head dim
    ((1, 4, 1, 128), dict(T_cap=1000), {}),      # not whole records
    ((1, 4, 1, 128), dict(T_cap=0), {}),
    ((1, 4, 1, 128), dict(T_cap=1 << 31), {}),
    ((1, 4, 1, 128), dict(records=0), {}),
    ((1, 4, 1, 128), dict(records=M), {}),
    ((1, 4, 1, 128), {}, dict(k=0)),
    ((1, 4, 1, 128), {}, dict(v=M)),
    ((1, 4, 1, 128), {}, dict(n=-1)),
    ((1, 4, 1, 128), {}, dict(n=1 << 31)),
    ((1, 4, 1, 128), {}, dict(pos0=-1)),
    ((1, 4, 1, 128), {}, dict(pos0=1025)),
    ((1, 4, 1, 128), {}, dict(dtype=9)),
    ((1, 4, 1, 128), {}, dict(ws=0)),
    ((1, 4, 1, 128), {}, dict(ws_bytes=16)),
])
def test_write_and_read_refuse(L, shape, cache, args):
    a = dict(k=A, v=A, dtype=vc.VC_BF16, n=4, pos=0, pos0=0, counts=0, ws=A, ws_bytes=WS, stream=0)
    a.update(args)
    for f in (L.vc_fp4_cache_write, L.vc_fp4_cache_read):
        st = f(ctypes.byref(vc.shape(*shape)), ctypes.byref(_fc(**cache)), *a.values())
        _refused(L, st, f.__name__)


def test_write_takes_16_bit_inputs_only(L):
    st = L.vc_fp4_cache_write(ctypes.byref(vc.shape(1, 4, 1, 128)), ctypes.byref(_fc()), A, A, vc.VC_F32, 4, 0, 0, 0,
                              A, WS, 0)
    _refused(L, st, "vc_fp4_cache_write")


def test_no_rows_is_no_work(L):
    for f in (L.vc_fp4_cache_write, L.vc_fp4_cache_read):
        assert f(ctypes.byref(vc.shape(1, 4, 1, 128)), ctypes.byref(_fc()), 0, 0, vc.VC_BF16, 0, 0, 0, 0, A, WS, 0) == 0


@pytest.mark.parametrize("shape,cache,args", [
    ((1, 4, 3, 128), {}, {}),                    # Hq not a multiple of Hkv
    ((1, 16, 1, 128), {}, {}),                   # g > 8
    ((1, 4, 1, 80), {}, {}),
    ((1, 4, 1, 128), dict(T=1025), {}),          # more than the capacity
    ((1, 4, 1, 128), dict(T=-1), {}),
    ((1, 4, 1, 128), dict(T_cap=24), {}),
    ((1, 4, 1, 128), dict(records=M), {}),
    ((1, 4, 1, 128), {}, dict(window=-1)),
    ((1, 4, 1, 128), {}, dict(n_sink=-1)),
    ((1, 4, 1, 128), {}, dict(q=0)),
    ((1, 4, 1, 128), {}, dict(out=M)),
    ((1, 4, 1, 128), {}, dict(ws=0)),
    ((1, 4, 1, 128), {}, dict(ws_bytes=8)),
])
def test_draft_refuses(L, shape, cache, args):
    a = dict(window=0, n_sink=0, q=A, out=A, lse=0, ws=A, ws_bytes=WS, stream=0)
    a.update(args)
    st = L.vc_draft_attn_fp4(ctypes.byref(vc.shape(*shape)), ctypes.byref(_fc(**cache)), *a.values())
    _refused(L, st, "vc_draft_attn_fp4")


@pytest.mark.parametrize("shape,args", [
    ((1, 4, 1, 128), dict(nq=0)),
    ((1, 4, 1, 128), dict(nq=33)),
    ((1, 4, 1, 128), dict(T=0)),
    ((1, 4, 1, 128), dict(T=1 << 31)),
    ((1, 4, 1, 128), dict(window=-1)),
    ((1, 4, 1, 128), dict(n_sink=-1)),
    ((1, 4, 1, 96), {}),
    ((1, 9, 1, 128), {}),
    ((70000, 1, 1, 128), {}),
    ((1, 4, 1, 128), dict(q=0)),
    ((1, 4, 1, 128), dict(k=M)),
    ((1, 4, 1, 128), dict(out=0)),
])
def test_windowed_verification_refuses(L, shape, args):
    a = dict(q=A, k=A, v=A, T=100, lens=0, nq=5, window=10, n_sink=4, out=A, lse=0, ws=A, ws_bytes=WS, stream=0)
    a.update(args)
    st = L.vc_verify_attn_window(ctypes.byref(vc.shape(*shape)), *a.values())
    _refused(L, st, "vc_verify_attn_window")


def test_workspace_sizes_are_zero_for_refused_shapes(L):
    ok, bad = vc.shape(1, 4, 1, 128), vc.shape(1, 4, 1, 100)
    assert L.vc_draft_attn_fp4_workspace_size(ctypes.byref(bad), ctypes.byref(_fc())) == 0
    assert L.vc_draft_attn_fp4_workspace_size(ctypes.byref(ok), ctypes.byref(_fc(T=-5))) == 0
    for a in ((0, 4, 8, 0), (100, 40, 8, 0), (100, 4, -1, 0), (100, 4, 8, -1)):
        assert L.vc_verify_attn_window_workspace_size(ctypes.byref(ok), *a) == 0


def test_binding_checks_its_tensors():
    rec = torch.zeros(1, 2, 4, 18 * 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="current CUDA device"):
        vc.fp4_cache(rec)  # host memory
    with pytest.raises(ValueError, match="18"):
        vc.fp4_cache(torch.zeros(1, 2, 4, 100, dtype=torch.uint8))
    with pytest.raises(ValueError, match="uint8"):
        vc.fp4_cache(rec.float())
    fc = vc.vc_fp4_cache(A, 64, 64, 0, 0, 0)
    fc._dims = (1, 2, 64)
    ws = torch.zeros(256, dtype=torch.uint8)
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="shape says"):
        vc.vc_fp4_cache_write(vc.shape(1, 4, 4, 64), fc, x, x, 3, ws)
    with pytest.raises(ValueError, match="same dtype"):
        vc.vc_fp4_cache_write(vc.shape(1, 4, 2, 64), fc, x, x.half(), 3, ws)
    with pytest.raises(ValueError, match="elements"):
        vc.vc_fp4_cache_write(vc.shape(1, 4, 2, 64), fc, x, x, 4, ws)
    with pytest.raises(ValueError, match="contiguous"):
        vc.vc_fp4_cache_read(vc.shape(1, 4, 2, 64), fc, 3, x.transpose(1, 2), x, ws)
    with pytest.raises(ValueError, match="q must be"):
        vc.vc_draft_attn_fp4(vc.shape(1, 4, 2, 64), fc, torch.zeros(4, 64), torch.zeros(4, 64), ws)
    with pytest.raises(ValueError, match="missing"):
        vc.vc_verify_attn_window(vc.shape(1, 4, 2, 64), None, x, x, 3, 1, x, None, ws)
