"""Draft attention over the 4-bit floating-point cache against the oracle.

Tolerance, per output element (derived, not fitted): products of q and k_hat
are exact in fp32, so a score is off by at most (D + 4) 2^-23 peak (peak =
the largest sum of |q k| * scale); an exponential adds 2^-21 and the split of
a weight into two fp16 parts 2^-20; numerator and denominator both carry
that, and each sum of n terms in fp32 up to n 2^-23 of the sum of magnitudes
(amp = sum p |v|).  lse: the score's error plus that of its sum.

Weights far below the row's largest are held in steps: the parts' last place
is 2^-24, so a weight is off by at most 2^-25 where the largest is at least
2^10 (the reference is set 11 below the ceiling of the maximum and moves up
only) -- 2^-35 of the largest, hence of the denominator.  n of them add at
most n 2^-35 max |v|, which shows where the heavy tokens' values are exactly
0, as 4-bit values often are."""

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


def make_cache(B, H, T, D, lens, seed, exp=None, poison=True):
    """Records of random rows; every byte of tokens past a request's length is 0xFF (a NaN scale)."""
    k, v = synth.kv_full(B, H, T, D, seed=seed)
    kc, ks = F.quantise(np32(k), exp)
    vc_, vs = F.quantise(np32(v), exp)
    fill = np.full((B, H, -(-T // 16), 18 * D), 0xFF if poison else 0, np.uint8)
    rec = F.pack(kc, ks, vc_, vs, fill, np.zeros(B, int), np.clip(lens, 0, T))
    return rec, F.values(kc, ks, exp), F.values(vc_, vs, exp)


def check(o, l, q, kh, vh, lens, window, sinks, sm_scale=None):
    D = q.shape[-1]
    wo, wl, amp, peak = F.window_attention(np32(q)[:, None], kh, vh, lens, window, sinks, sm_scale)
    wo, wl, amp, peak = wo[:, 0], wl[:, 0], amp[:, 0], peak[:, 0]
    n = np.array([min(x, window + sinks) if window else x for x in lens])[:, None]
    eps = (D + 4) * 2.0 ** -23 * peak + 2.0 ** -21 + 2.0 ** -20
    assert np.isfinite(o).all()
    floor = n[..., None] * 2.0 ** -35 * np.abs(vh).max()
    assert (np.abs(o - wo) <= (2 * eps + n * 2.0 ** -23)[..., None] * amp + floor + 1e-30).all()
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(l), empty) and not o[empty].any()
    d, m = np.where(empty, 0, l) - np.where(empty, 0, wl), np.where(empty, 0, np.abs(wl))
    assert (np.abs(d) <= eps + n * 2.0 ** -23 + 2.0 ** -22 * m).all()
    assert row_rel_err(o[~empty], wo[~empty]) <= ATTN_TOL if (~empty).any() else True


def run(rec, q, T=None, lens=None, window=0, sinks=0, exp=None, sm_scale=0.0, ws=None):
    B, H, _, nb = rec.shape
    Hq, D = q.shape[1:]
    sh = vc.shape(B, Hq, H, D, sm_scale)
    e = None if exp is None else ints(exp)
    fc = vc.fp4_cache(torch.from_numpy(rec).to(dev), T=T, lens=None if lens is None else ints(lens), k_exp=e, v_exp=e)
    ws = vc.workspace(vc.vc_draft_attn_fp4_workspace_size(sh, fc)) if ws is None else ws
    out = torch.full((B, Hq, D), float("nan"), device=dev)
    lse = torch.full((B, Hq), float("nan"), device=dev)
    vc.vc_draft_attn_fp4(sh, fc, q.to(dev), out, ws, lse=lse, window=window, n_sink=sinks)
    return np32(out), np32(lse), vc.vc_workspace_flags(ws)


@pytest.mark.parametrize("B,Hq,Hkv,D,T", [
    (1, 1, 1, 64, 1),
    (1, 8, 1, 128, 1),
    (2, 4, 4, 128, 15),          # g = 1
    (1, 6, 3, 64, 16),
    (3, 6, 2, 128, 17),          # g = 3
    (1, 32, 8, 128, 100),        # g = 4
    (2, 10, 2, 64, 333),         # g = 5
    (1, 14, 2, 128, 1000),       # g = 7
    (2, 16, 2, 64, 2047),        # g = 8
    (1, 8, 1, 128, 9001),
    (40, 16, 8, 64, 40),         # more units than blocks
])
def test_shapes_and_lengths(B, Hq, Hkv, D, T):
    lens = [T] * B
    rec, kh, vh = make_cache(B, Hkv, T, D, lens, seed=T + D)
    q = synth.normal((B, Hq, D), seed=T)
    o, l, flags = run(rec, q, T=T)
    assert flags == 0
    check(o, l, q, kh, vh, lens, 0, 0)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (20, 3), (64, 4), (100, 17), (300, 64), (5000, 4),
                                          (700, 700), (31, 1000)])
@pytest.mark.parametrize("D,g", [(64, 2), (128, 4), (128, 8)])
def test_windows_and_first_tokens_over_ragged_requests(window, sinks, D, g):
    lens = [0, 1, 16, 83, 500, 777]
    B, Hkv, T = len(lens), 2, 777
    rec, kh, vh = make_cache(B, Hkv, T, D, lens, seed=window + D)
    q = synth.normal((B, g * Hkv, D), seed=sinks)
    o, l, flags = run(rec, q, lens=lens, window=window, sinks=sinks)
    assert flags == 0
    check(o, l, q, kh, vh, lens, window, sinks)


def test_lengths_outside_the_cache_are_empty_and_flagged():
    lens = [40, -1, 65, 64]
    rec, kh, vh = make_cache(4, 2, 64, 64, lens, seed=3, poison=False)
    q = synth.normal((4, 4, 64), seed=4)
    o, l, flags = run(rec, q, lens=lens)
    assert flags == vc.VC_FLAG_BAD_LENGTH
    check(o, l, q, kh, vh, [40, 0, 0, 64], 0, 0)


def test_all_requests_empty():
    rec, kh, vh = make_cache(2, 2, 32, 128, [0, 0], seed=3)
    q = synth.normal((2, 4, 128), seed=4)
    for kw in (dict(T=0), dict(lens=[0, 0]), dict(lens=[0, 0], window=4, sinks=2)):
        o, l, flags = run(rec, q, **kw)
        assert flags == 0 and not o.any() and np.isneginf(l).all()


@pytest.mark.parametrize("scale", [0.0, 0.25, 1e-3])
def test_explicit_scale_and_head_exponents(scale):
    B, Hkv, D, T, exp = 2, 3, 128, 260, [3, -9, 0]
    rec, kh, vh = make_cache(B, Hkv, T, D, [T] * B, seed=9, exp=exp)
    # the exponents only move the stored scales; keep the scores moderate
    q = (synth.normal((B, 12, D), seed=5).float() / 8).to(torch.bfloat16)
    o, l, flags = run(rec, q, T=T, exp=exp, sm_scale=scale)
    assert flags == 0
    check(o, l, q, kh, vh, [T] * B, 0, 0, scale or None)


def test_one_dominant_key_and_very_large_scores():
    B, Hkv, D, T = 1, 1, 64, 500
    rec, kh, vh = make_cache(B, Hkv, T, D, [T], seed=12)
    q = torch.zeros(1, 2, D)
    q[0, 0] = torch.from_numpy(kh[0, 0, 321]).float() * 30  # one key far above the rest
    q[0, 1] = -3e4
    q = q.to(torch.bfloat16)
    o, l, flags = run(rec, q, T=T)
    check(o, l, q, kh, vh, [T], 0, 0)


def test_scores_that_grow_along_the_context_rescale_often():
    """Keys whose score rises by several units per token: the running maximum
    moves at every tile, in both directions of the split."""
    B, Hkv, D, T = 1, 2, 128, 700
    k = torch.zeros(B, Hkv, T, D)
    k[0, 0, :, 0] = torch.linspace(0, 400, T)
    k[0, 1, :, 0] = torch.linspace(400, 0, T)
    v = synth.normal((B, Hkv, T, D), seed=2)
    kc, ks = F.quantise(np32(k))
    vc_, vs = F.quantise(np32(v))
    rec = F.pack(kc, ks, vc_, vs, np.zeros((B, Hkv, 44, 18 * D), np.uint8), np.zeros(1, int), np.array([T]))
    q = torch.zeros(B, 4, D)
    q[..., 0] = 40.0
    q = q.to(torch.bfloat16)
    o, l, _ = run(rec, q, T=T)
    check(o, l, q, F.values(kc, ks), F.values(vc_, vs), [T], 0, 0)


def test_repeated_calls_reuse_a_workspace_and_give_the_same_bits():
    B, Hkv, D, T = 3, 4, 128, 3000
    lens = [3000, 1, 1777]
    rec, kh, vh = make_cache(B, Hkv, T, D, lens, seed=13)
    q = synth.normal((B, 16, D), seed=14)
    sh = vc.shape(B, 16, Hkv, D)
    fc = vc.fp4_cache(torch.from_numpy(rec).to(dev), lens=ints(lens))
    ws = vc.workspace(vc.vc_draft_attn_fp4_workspace_size(sh, fc))
    first = run(rec, q, lens=lens, ws=ws)
    run(rec, q, lens=lens, window=100, sinks=3, ws=ws)
    again = run(rec, q, lens=lens, ws=ws)
    assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_without_lse_on_another_stream():
    B, Hkv, D, T = 2, 2, 64, 400
    rec, kh, vh = make_cache(B, Hkv, T, D, [T] * B, seed=15)
    q = synth.normal((B, 8, D), seed=16)
    o, l, _ = run(rec, q, T=T)
    sh = vc.shape(B, 8, Hkv, D)
    fc = vc.fp4_cache(torch.from_numpy(rec).to(dev), T=T)
    ws = vc.workspace(vc.vc_draft_attn_fp4_workspace_size(sh, fc))
    out, qd = torch.empty(B, 8, D, device=dev), q.to(dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    vc.vc_draft_attn_fp4(sh, fc, qd, out, ws, stream=s)
    torch.cuda.synchronize()
    assert np.array_equal(np32(out), o)


def test_captured_calls_follow_the_lengths_on_the_device():
    B, Hkv, D, T = 2, 2, 128, 900
    rec, kh, vh = make_cache(B, Hkv, T, D, [T] * B, seed=17)
    q = synth.normal((B, 8, D), seed=18)
    lens = ints([1, 700])
    sh = vc.shape(B, 8, Hkv, D)
    fc = vc.fp4_cache(torch.from_numpy(rec).to(dev), lens=lens)
    ws = vc.workspace(vc.vc_draft_attn_fp4_workspace_size(sh, fc))
    qd = q.to(dev)
    out, lse = torch.empty(B, 8, D, device=dev), torch.empty(B, 8, device=dev)
    vc.vc_draft_attn_fp4(sh, fc, qd, out, ws, lse=lse, window=128, n_sink=4)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vc.vc_draft_attn_fp4(sh, fc, qd, out, ws, lse=lse, window=128, n_sink=4)
    for now in ([1, 700], [900, 0], [333, 16]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        check(np32(out), np32(lse), q, kh, vh, now, 128, 4)


def test_byte_offsets_past_32_bits():
    H, D, T = 8, 128, 1 << 22
    rec = torch.zeros(1, H, T // 16, 18 * D, dtype=torch.uint8, device=dev)  # 4.8 GB
    k, v = synth.kv_full(1, H, 40, D, seed=19)
    sh, fc = vc.shape(1, 8, H, D), vc.fp4_cache(rec)
    ws = vc.workspace(vc.vc_draft_attn_fp4_workspace_size(sh, fc))
    vc.vc_fp4_cache_write(sh, fc, k.to(dev), v.to(dev), 40, ws, pos0=T - 40)
    q = synth.normal((1, 8, D), seed=20)
    out, lse = torch.empty(1, 8, D, device=dev), torch.empty(1, 8, device=dev)
    vc.vc_draft_attn_fp4(sh, fc, q.to(dev), out, ws, lse=lse, window=40)
    kh, vh = F.values(*F.quantise(np32(k))), F.values(*F.quantise(np32(v)))
    check(np32(out), np32(lse), q, kh, vh, [40], 0, 0)
