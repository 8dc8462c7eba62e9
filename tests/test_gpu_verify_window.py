"""Windowed block verification against the oracle.

Tolerance, per output element (derived): a score of D exact products summed
in fp32 is off by at most (D + 4) 2^-23 peak; the exponential adds 2^-21, the
split of a weight into two bf16 parts 2^-17; sums of n terms n 2^-23 of the
sum of magnitudes (amp)."""

import numpy as np
import pytest
import torch

from lossless_draft_verify_vc_b200 import synth, vc
from oracle import fp4 as F
from tests.vcutil import ATTN_TOL, np32, row_rel_err

pytestmark = pytest.mark.gpu
dev = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def run(q, k, v, window, sinks, lens=None, with_lse=True, sm_scale=0.0):
    B, Hkv, T, D = k.shape
    nq, Hq = q.shape[1:3]
    sh = vc.shape(B, Hq, Hkv, D, sm_scale)
    ws = vc.workspace(vc.vc_verify_attn_window_workspace_size(sh, T, nq, window, sinks))
    out = torch.full((B, nq, Hq, D), float("nan"), device=dev)
    lse = torch.full((B, nq, Hq), float("nan"), device=dev) if with_lse else None
    vc.vc_verify_attn_window(sh, q.to(dev), k.to(dev), v.to(dev), T, nq, out, lse, ws, window=window, n_sink=sinks,
                             lens=None if lens is None else ints(lens))
    return np32(out), np32(lse) if with_lse else None, vc.vc_workspace_flags(ws)


def check(o, l, q, k, v, lens, window, sinks, sm_scale=None):
    D, nq = q.shape[-1], q.shape[1]
    wo, wl, amp, peak = F.window_attention(np32(q), np32(k), np32(v), lens, window, sinks, sm_scale)
    n = np.array([min(x, window + sinks + nq) if window else x for x in lens])[:, None, None]
    eps = (D + 4) * 2.0 ** -23 * peak + 2.0 ** -21 + 2.0 ** -17
    assert np.isfinite(o).all()
    assert (np.abs(o - wo) <= (2 * eps + n * 2.0 ** -23)[..., None] * amp + 1e-30).all()
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(l), empty) and not o[empty].any()
    d, m = np.where(empty, 0, l) - np.where(empty, 0, wl), np.where(empty, 0, np.abs(wl))
    assert (np.abs(d) <= eps + n * 2.0 ** -23 + 2.0 ** -22 * m).all()
    assert row_rel_err(o[~empty], wo[~empty]) <= ATTN_TOL


def make(B, Hkv, T, D, nq, Hq, seed, lens=None):
    """Rows past a request's length are NaN (keys) and infinite (values)."""
    k, v = synth.kv_full(B, Hkv, T, D, seed=seed)
    for b, n in enumerate(lens or []):
        k[b, :, max(n, 0):] = float("nan")
        v[b, :, max(n, 0):] = float("inf")
    return synth.normal((B, nq, Hq, D), seed=seed + 1), k, v


@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (63, 0), (64, 4), (65, 64), (100, 130), (257, 7), (600, 0),
                                          (0, 0), (0, 5), (2000, 3), (5, 1000)])
@pytest.mark.parametrize("B,nq,Hq,Hkv,D,T", [
    (1, 1, 4, 1, 128, 700),      # one row
    (2, 31, 8, 2, 128, 700),     # one row tile
    (1, 31, 10, 2, 64, 700),     # g = 5: two row tiles in one block
    (1, 32, 8, 8, 64, 500),      # g = 1
])
def test_windows_and_first_tokens(window, sinks, B, nq, Hq, Hkv, D, T):
    q, k, v = make(B, Hkv, T, D, nq, Hq, seed=window + sinks)
    o, l, flags = run(q, k, v, window, sinks)
    assert flags == 0
    check(o, l, q, k, v, [T] * B, window, sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 0), (64, 3), (130, 70), (10, 600)])
@pytest.mark.parametrize("nq,Hq,Hkv,D", [(1, 4, 2, 64), (7, 16, 2, 128), (31, 16, 2, 128), (31, 40, 20, 64)])
def test_ragged_requests_and_garbage_behind_them(window, sinks, nq, Hq, Hkv, D):
    """Lengths below nq leave rows without a key; rows past a length hold NaN and infinities."""
    lens = [0, 1, 20, 64, 65, 500, 611]
    B, T = len(lens), 611
    q, k, v = make(B, Hkv, T, D, nq, Hq, seed=nq, lens=lens)
    o, l, flags = run(q, k, v, window, sinks, lens=lens)
    assert flags == 0
    check(o, l, q, k, v, lens, window, sinks)


def test_garbage_between_the_first_tokens_and_the_window():
    B, Hkv, T, D, nq, Hq, window, sinks = 1, 2, 900, 128, 6, 8, 200, 10
    q, k, v = make(B, Hkv, T, D, nq, Hq, seed=3)
    w = F.window_attention(np32(q), np32(k), np32(v), [T], window, sinks)
    k[:, :, sinks:T - nq + 1 - window] = float("nan")
    v[:, :, sinks:T - nq + 1 - window] = float("nan")
    o, l, _ = run(q, k, v, window, sinks)
    assert row_rel_err(o, w[0]) <= ATTN_TOL and np.abs(l - w[1]).max() <= 1e-3


def test_lengths_outside_the_cache_are_empty_and_flagged():
    lens = [100, -3, 201]
    q, k, v = make(3, 2, 200, 64, 4, 4, seed=5)
    o, l, flags = run(q, k, v, 32, 2, lens=lens)
    assert flags == vc.VC_FLAG_BAD_LENGTH
    check(o, l, q, k, v, [100, 0, 0], 32, 2)


@pytest.mark.parametrize("nq,Hq", [(31, 32), (31, 64), (1, 32)])
def test_without_a_window_it_equals_plain_verification(nq, Hq):
    """window 0, or one that hides nothing: the same numbers as vc_verify_attn
    within both calls' own error (their splits of the context may differ)."""
    B, Hkv, T, D = 1, 8, 3000, 128
    q, k, v = make(B, Hkv, T, D, nq, Hq, seed=6)
    sh = vc.shape(B, Hq, Hkv, D)
    ws = vc.workspace(vc.vc_verify_attn_workspace_size(sh, T, nq))
    base = torch.empty(B, nq, Hq, D, device=dev)
    vc.vc_verify_attn(sh, q.to(dev), k.to(dev), v.to(dev), T, nq, base, None, ws)
    for window in (0, T, 1 << 40):
        o, _, _ = run(q, k, v, window, 0)
        assert row_rel_err(o, np32(base)) <= 2.0 ** -14


def test_many_chunks_explicit_scale_no_lse_and_repeatability():
    B, Hkv, T, D, nq, Hq = 1, 2, 20000, 128, 9, 16
    q, k, v = make(B, Hkv, T, D, nq, Hq, seed=7)
    o, l, _ = run(q, k, v, 12345, 100, sm_scale=0.125)
    check(o, l, q, k, v, [T], 12345, 100, 0.125)
    o2, _, _ = run(q, k, v, 12345, 100, with_lse=False, sm_scale=0.125)
    assert np.array_equal(o, o2)


def test_captured_calls_follow_the_lengths_on_the_device():
    B, Hkv, T, D, nq, Hq, window, sinks = 2, 2, 800, 128, 5, 8, 150, 4
    q, k, v = make(B, Hkv, T, D, nq, Hq, seed=8)
    qd, kd, vd, lens = q.to(dev), k.to(dev), v.to(dev), ints([800, 3])
    sh = vc.shape(B, Hq, Hkv, D)
    ws = vc.workspace(vc.vc_verify_attn_window_workspace_size(sh, T, nq, window, sinks))
    out, lse = torch.empty(B, nq, Hq, D, device=dev), torch.empty(B, nq, Hq, device=dev)
    call = lambda: vc.vc_verify_attn_window(sh, qd, kd, vd, T, nq, out, lse, ws, window=window, n_sink=sinks, lens=lens)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for now in ([800, 3], [77, 512], [0, 800]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        check(np32(out), np32(lse), q, k, v, now, window, sinks)
