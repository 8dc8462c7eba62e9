"""Refusals of the two entry points that force a give-up (CPU only: the checks
run before any CUDA call, the pointers are never dereferenced)."""

import ctypes

import pytest

from lossless_draft_verify_vc_b200 import vc

A = 0x100000


def refused(status, who):
    assert status == vc.VC_ERR_INVALID_ARG and who in vc.lib().vc_last_error().decode()


@pytest.mark.parametrize("kw", [dict(stuck=-1), dict(stuck=16), dict(limit=999), dict(limit=100_000_001), dict(q=0),
                                dict(window=-1), dict(ws_bytes=8)])
def test_draft(kw):
    a = dict(window=0, n_sink=0, q=A, out=A, lse=0, ws=A, ws_bytes=1 << 40, stuck=0, limit=1_000_000, stream=0)
    a.update(kw)
    fc = vc.vc_fp4_cache(A, 1024, 1000, 0, 0, 0)
    refused(vc.lib().vc_debug_draft_fp4_abort(ctypes.byref(vc.shape(1, 4, 1, 128)), ctypes.byref(fc), *a.values()),
            "vc_debug_draft_fp4_abort")


@pytest.mark.parametrize("kw", [dict(skip=-1), dict(limit=999), dict(limit=100_000_001), dict(nq=2), dict(nq=0), dict(T=0)])
def test_windowed_verification(kw):
    a = dict(q=A, k=A, v=A, T=100, lens=0, nq=5, window=10, n_sink=4, out=A, lse=0, ws=A, ws_bytes=1 << 40, skip=0,
             limit=1_000_000, stream=0)
    a.update(kw)
    st = vc.lib().vc_debug_verify_window_abort(ctypes.byref(vc.shape(1, 4, 1, 128)), *a.values())
    # (more than 32 or no rows are refused by the operator itself)
    refused(st, "vc_")
