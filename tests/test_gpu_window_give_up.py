"""Waits that run out in windowed verification and in the 4-bit draft: the call
ends, raises VC_FLAG_WAIT_TIMEOUT and leaves the workspace and the context as
usable as before.  Nothing here faults or hangs a GPU: a copy is left out, or a
barrier expects one arrival more, and the waits on it give up after 20 ms."""

import time

import pytest
import torch

from lossless_draft_verify_vc_b200 import synth, vc
from oracle import fp4 as F
from tests import test_gpu_draft_fp4 as D4
from tests import test_gpu_verify_window as VW
from tests.vcutil import np32

pytestmark = pytest.mark.gpu
dev = "cuda"
LIMIT = 20_000_000


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def ends_flagged(call, ws, flag=vc.VC_FLAG_WAIT_TIMEOUT):
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    assert vc.vc_workspace_flags(ws) == flag
    assert took < 5.0, f"the aborted call took {took:.1f} s"


@pytest.mark.parametrize("nq,g,Hkv,D,lens,window,sinks,skip", [
    (31, 4, 2, 128, [1500, 1500], 0, 0, 1),     # a cluster: every block gives up
    (31, 4, 2, 128, [1500, 100], 0, 0, 2),      # blocks of the short request finish
    (31, 4, 2, 64, [1500, 0], 700, 70, 0),      # before the tile loop; chunks without tiles
    (9, 1, 2, 128, [1400, 900], 600, 4, 1),     # warps without rows; dead values behind the lengths
    (31, 5, 4, 128, [1500, 40], 0, 0, 1),       # two row tiles
    (31, 4, 1, 128, [20000, 70], 0, 0, 1),      # partials and a second launch
    (31, 4, 32, 64, [200] * 10, 60, 0, 1),      # one chunk per unit
])
def test_windowed_verification_gives_up(nq, g, Hkv, D, lens, window, sinks, skip):
    B, T = len(lens), max(lens) + 9
    q, k, v = VW.make(B, Hkv, T, D, nq, g * Hkv, seed=nq + D, lens=lens)
    qd, kd, vd, ld = q.to(dev), k.to(dev), v.to(dev), ints(lens)
    sh = vc.shape(B, g * Hkv, Hkv, D)
    n = vc.vc_verify_attn_window_workspace_size(sh, T, nq, window, sinks)
    used, fresh = vc.workspace(n), vc.workspace(n)
    out, lse = torch.empty(B, nq, g * Hkv, D, device=dev), torch.empty(B, nq, g * Hkv, device=dev)
    ends_flagged(lambda: vc.vc_debug_verify_window_abort(sh, qd, kd, vd, T, nq, out, lse, used, skip, LIMIT, window=window,
                                                         n_sink=sinks, lens=ld), used)
    got = []
    for ws in (used, fresh):
        out.fill_(float("nan"))
        vc.vc_verify_attn_window(sh, qd, kd, vd, T, nq, out, lse, ws, window=window, n_sink=sinks, lens=ld)
        assert vc.vc_workspace_flags(ws) == 0
        got.append(out.clone())
    assert torch.equal(*got)
    some = [b for b in range(B) if b < 2]
    VW.check(np32(out)[some], np32(lse)[some], q[some], k[some], v[some], [lens[b] for b in some], window, sinks)


@pytest.mark.parametrize("stuck", [0, 15])
@pytest.mark.parametrize("g,Hkv,D,lens,window,sinks,busy", [
    (4, 2, 128, [24000, 9000], 0, 0, 16),    # equal shares: merges by the block that finishes last
    (8, 1, 64, [60001], 0, 0, 16),           # one unit over every block
    # clusters of 2 blocks: 2 records of first tokens (1 stage) and 44 or 45 of the window (22 or 23), 12 stages a block
    (3, 8, 128, [4000, 3999], 700, 40, 12),
    (1, 8, 64, [1500] * 25, 0, 0, 16),       # several units per block: later copies in flight
])
def test_the_draft_gives_up(stuck, g, Hkv, D, lens, window, sinks, busy):
    """busy: warps of a block that have copies to wait for; another one that is stuck is not noticed."""
    B, T = len(lens), max(lens)
    k, v = synth.kv_full(B, Hkv, T, D, seed=len(lens))
    sh, fc = vc.shape(B, g * Hkv, Hkv, D), vc.fp4_cache(vc.fp4_records(B, Hkv, T, D), lens=ints(lens))
    n = vc.vc_draft_attn_fp4_workspace_size(sh, fc)
    used, fresh = vc.workspace(n), vc.workspace(n)
    vc.vc_fp4_cache_write(sh, fc, k.to(dev), v.to(dev), T, vc.workspace(256))
    q = synth.normal((B, g * Hkv, D), seed=3)
    qd = q.to(dev)
    out, lse = torch.empty(B, g * Hkv, D, device=dev), torch.empty(B, g * Hkv, device=dev)
    ends_flagged(lambda: vc.vc_debug_draft_fp4_abort(sh, fc, qd, out, lse, used, stuck, LIMIT, window=window, n_sink=sinks),
                 used, vc.VC_FLAG_WAIT_TIMEOUT if stuck < busy else 0)
    assert torch.isfinite(out).all()
    got = []
    for ws in (used, fresh, used):
        out.fill_(float("nan"))
        vc.vc_draft_attn_fp4(sh, fc, qd, out, ws, lse=lse, window=window, n_sink=sinks)
        assert vc.vc_workspace_flags(ws) == 0
        got.append(out.clone())
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    kh, vh = (torch.empty(B, Hkv, T, D, device=dev) for _ in range(2))
    vc.vc_fp4_cache_read(sh, fc, T, kh, vh, vc.workspace(256))
    some = [b for b in range(B) if b < 2]
    D4.check(np32(out)[some], np32(lse)[some], q[some], np32(kh)[some], np32(vh)[some], [lens[b] for b in some], window, sinks)


def test_a_warp_that_gave_up_adds_nothing():
    """One unit, one block per share: rows are the softmax over the other warps' tokens."""
    D, T = 128, 64  # a cluster of one block with two stages of 32 tokens: warps 0 and 1
    k, v = synth.kv_full(1, 1, T, D, seed=1)
    sh, fc = vc.shape(1, 2, 1, D), vc.fp4_cache(vc.fp4_records(1, 1, T, D))
    ws = vc.workspace(vc.vc_draft_attn_fp4_workspace_size(sh, fc))
    vc.vc_fp4_cache_write(sh, fc, k.to(dev), v.to(dev), T, ws)
    q = synth.normal((1, 2, D), seed=2)
    out, lse = torch.empty(1, 2, D, device=dev), torch.empty(1, 2, device=dev)
    ends_flagged(lambda: vc.vc_debug_draft_fp4_abort(sh, fc, q.to(dev), out, lse, ws, 0, LIMIT), ws)
    kh, vh = F.values(*F.quantise(np32(k[:, :, 32:]))), F.values(*F.quantise(np32(v[:, :, 32:])))
    D4.check(np32(out), np32(lse), q, kh, vh, [32], 0, 0)
