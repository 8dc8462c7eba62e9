"""The 4-bit draft cache and windowed verification as a program uses them
together, and every way the work is split: a cluster per (request, KV head),
equal shares of all requests' stages, more units than blocks, shared
workspaces, rows that are only 16-byte aligned, two streams at once.

Tolerances: those derived in test_gpu_draft_fp4 and test_gpu_verify_window."""

import numpy as np
import pytest
import torch

from lossless_draft_verify_vc_b200 import synth, vc
from oracle import fp4 as F
from tests import test_gpu_draft_fp4 as D4
from tests import test_gpu_verify_window as VW
from tests.vcutil import np32

pytestmark = pytest.mark.gpu
dev = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("Hq,Hkv,D,window,sinks", [(8, 2, 128, 0, 0), (6, 3, 64, 40, 3)])
def test_two_rounds_of_drafting_and_verification(Hq, Hkv, D, window, sinks):
    """Prompt rows written at once, K drafted tokens appended and attended to one
    by one, the block verified against the full cache, the accepted part kept
    and the rest overwritten by the next round: one workspace throughout."""
    B, K, T = 2, 5, 160
    lens, accepted = np.array([70, 33]), [[2, 5], [0, 3]]
    sh = vc.shape(B, Hq, Hkv, D)
    rec = vc.fp4_records(B, Hkv, T, D)
    lens_d = ints(lens.tolist())
    fc = vc.fp4_cache(rec, lens=lens_d)
    ws = vc.workspace(max(vc.vc_draft_attn_fp4_workspace_size(sh, fc), vc.vc_compress_workspace_size(),
                          vc.vc_verify_attn_window_workspace_size(sh, T, K + 1, window, sinks)))
    full_k, full_v = (torch.zeros(B, Hkv, T, D, dtype=torch.bfloat16) for _ in range(2))
    want = np.zeros(tuple(rec.shape), np.uint8)

    def put(k, v, pos, counts):  # the full cache, the 4-bit cache and the oracle's copy of it
        nonlocal want
        for b in range(B):
            full_k[b, :, pos[b]:pos[b] + counts[b]] = k[b, :, :counts[b]]
            full_v[b, :, pos[b]:pos[b] + counts[b]] = v[b, :, :counts[b]]
        vc.vc_fp4_cache_write(sh, fc, k.to(dev), v.to(dev), k.shape[2], ws, pos=ints(list(pos)), counts=ints(list(counts)))
        want = F.pack(*F.quantise(np32(k)), *F.quantise(np32(v)), want, np.array(pos), np.array(counts))

    k, v = synth.kv_full(B, Hkv, int(lens.max()), D, seed=1)
    put(k, v, [0, 0], lens.tolist())
    out, lse = torch.empty(B, Hq, D, device=dev), torch.empty(B, Hq, device=dev)
    for rnd, accept in enumerate(accepted):
        start = lens.copy()
        for i in range(K + 1):
            k, v = synth.kv_full(B, Hkv, 1, D, seed=100 * rnd + 2 * i)
            put(k, v, (start + i).tolist(), [1, 1])
            lens_d.copy_(torch.tensor((start + i + 1).tolist(), dtype=torch.int32))
            q = synth.normal((B, Hq, D), seed=50 * rnd + i)
            vc.vc_draft_attn_fp4(sh, fc, q.to(dev), out, ws, lse=lse, window=window, n_sink=sinks)
            kc, ks, vc_, vs = F.unpack(want)
            D4.check(np32(out), np32(lse), q, F.values(kc, ks), F.values(vc_, vs), (start + i + 1).tolist(), window, sinks)
        q = synth.normal((B, K + 1, Hq, D), seed=rnd)
        vo, vl = torch.empty(B, K + 1, Hq, D, device=dev), torch.empty(B, K + 1, Hq, device=dev)
        vc.vc_verify_attn_window(sh, q.to(dev), full_k.to(dev), full_v.to(dev), T, K + 1, vo, vl, ws, window=window,
                                 n_sink=sinks, lens=lens_d)
        VW.check(np32(vo), np32(vl), q, full_k, full_v, (start + K + 1).tolist(), window, sinks)
        lens = start + np.array(accept) + 1
    assert np.array_equal(rec.cpu().numpy(), want)
    assert vc.vc_workspace_flags(ws) == 0


@pytest.mark.parametrize("Hkv,g,D,lens,window,sinks", [
    (2, 4, 128, [24000, 7, 0, 15001], 0, 0),      # equal shares: parts of units, whole ones
    (1, 8, 64, [60001], 0, 0),                    # one unit over every block
    (3, 5, 128, [9000, 40000], 30000, 1000),      # first tokens and windows as two lists
    (8, 3, 128, [4000, 3999, 17], 700, 40),       # clusters
    (8, 1, 64, [1500] * 25, 0, 0),                # more units than blocks
    (1, 2, 64, [(i * 37) % 80 for i in range(3000)], 20, 1),  # many requests, some empty
])
def test_every_split_of_the_draft(Hkv, g, D, lens, window, sinks):
    B, T = len(lens), max(lens)
    k, v = synth.kv_full(B, Hkv, T, D, seed=len(lens))
    kd, vd = k.to(dev), v.to(dev)
    sh, fc = vc.shape(B, g * Hkv, Hkv, D), vc.fp4_cache(vc.fp4_records(B, Hkv, T, D), lens=ints(lens))
    ws = vc.workspace(vc.vc_draft_attn_fp4_workspace_size(sh, fc))
    vc.vc_fp4_cache_write(sh, fc, kd, vd, T, ws)
    kh, vh = (torch.empty(B, Hkv, T, D, device=dev) for _ in range(2))
    vc.vc_fp4_cache_read(sh, fc, T, kh, vh, ws)  # (compared with the oracle in test_gpu_fp4_cache)
    q = synth.normal((B, g * Hkv, D), seed=3)
    out, lse = torch.empty(B, g * Hkv, D, device=dev), torch.empty(B, g * Hkv, device=dev)
    for _ in range(2):  # the second call finds the workspace that the first one left
        out.fill_(float("nan"))
        vc.vc_draft_attn_fp4(sh, fc, q.to(dev), out, ws, lse=lse, window=window, n_sink=sinks)
        some = list(range(B)) if B < 100 else list(range(0, B, 59))
        D4.check(np32(out)[some], np32(lse)[some], q[some], np32(kh)[some], np32(vh)[some], [lens[b] for b in some],
                 window, sinks)
    assert torch.isfinite(out).all() and vc.vc_workspace_flags(ws) == 0


@pytest.mark.parametrize("nq,g,Hkv,D,lens,window,sinks", [
    (1, 1, 2, 64, [1, 0, 300], 0, 0),
    (1, 8, 1, 128, [50000], 0, 0),                # equal shares, one unit
    (1, 4, 2, 128, [30000, 5, 20000], 12345, 70),
    (1, 3, 3, 64, [700, 699], 100, 130),
    (2, 4, 2, 128, [1, 2, 3, 16, 17, 400], 33, 5),
    (8, 1, 2, 64, [3, 8, 9, 200], 16, 2),
    (4, 2, 1, 128, [130], 1, 0),
    (2, 3, 25, 64, [90] * 8, 64, 4),              # more units than blocks
])
def test_few_rows_of_windowed_verification(nq, g, Hkv, D, lens, window, sinks):
    B, T = len(lens), max(lens)
    q, k, v = VW.make(B, Hkv, T, D, nq, g * Hkv, seed=nq, lens=lens)
    if window and B == 1:  # keys between the first tokens and the windows
        lo = max(sinks, lens[0] - nq + 1 - window)
        k[0, :, sinks:lo], v[0, :, sinks:lo] = float("nan"), float("-inf")
    o, l, flags = VW.run(q, k, v, window, sinks, lens=lens)
    assert flags == 0
    if window and B == 1:
        k[0, :, sinks:lo], v[0, :, sinks:lo] = 0, 0
    VW.check(o, l, q, k, v, lens, window, sinks)


def shifted(x):
    """The same tensor 16 bytes past a 32-byte boundary."""
    n = 16 // x.element_size()
    buf = torch.empty(x.numel() + 2 * n, dtype=x.dtype, device=dev)
    at = n if buf.data_ptr() % 32 == 0 else 0
    y = buf[at:at + x.numel()].view(x.shape)
    y.copy_(x)
    assert y.data_ptr() % 32 == 16
    return y


@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_are_only_16_byte_aligned(D):
    B, Hkv, n, g = 2, 2, 50, 2
    k, v = synth.kv_full(B, Hkv, n, D, seed=5)
    sh = vc.shape(B, g * Hkv, Hkv, D)
    ws = vc.workspace(vc.vc_compress_workspace_size())
    recs, outs = [], []
    for put in (lambda x: x.to(dev), lambda x: shifted(x)):
        fc = vc.fp4_cache(vc.fp4_records(B, Hkv, n, D))
        vc.vc_fp4_cache_write(sh, fc, put(k), put(v), n, ws)
        recs.append(fc._keep[0])
        for dt in (torch.bfloat16, torch.float32):
            ko, vo = put(torch.zeros(B, Hkv, n, D, dtype=dt)), put(torch.zeros(B, Hkv, n, D, dtype=dt))
            vc.vc_fp4_cache_read(sh, fc, n, ko, vo, ws)
            outs += [ko, vo]
        q = synth.normal((B, 1, g * Hkv, D), seed=6)
        o = put(torch.zeros(B, 1, g * Hkv, D))
        w2 = vc.workspace(vc.vc_verify_attn_window_workspace_size(sh, n, 1, 20, 2))
        vc.vc_verify_attn_window(sh, put(q), put(k), put(v), n, 1, o, None, w2, window=20, n_sink=2)
        outs.append(o)
    assert torch.equal(*recs)
    for a, b in zip(outs[:5], outs[5:]):
        assert torch.equal(a, b) and a.any()


def test_one_workspace_for_calls_of_different_shapes():
    """Partials of a wide call must not be left where a later call of more
    (request, head) pairs keeps its counters."""
    sizes = []
    calls = []
    for B, g, Hkv, D, T, nq, window in ((1, 8, 1, 128, 40000, 1, 0), (1, 4, 4, 64, 30000, 31, 0), (70, 2, 6, 64, 64, 2, 9),
                                        (3, 8, 2, 128, 6000, 7, 4000)):
        sh = vc.shape(B, g * Hkv, Hkv, D)
        k, v = (x.to(dev) for x in synth.kv_full(B, Hkv, T, D, seed=T))
        fc = vc.fp4_cache(vc.fp4_records(B, Hkv, T, D))
        vc.vc_fp4_cache_write(sh, fc, k, v, T, vc.workspace(256))
        q = synth.normal((B, nq, g * Hkv, D), seed=nq).to(dev)
        out = torch.empty(B, nq, g * Hkv, D, device=dev)
        calls.append(lambda ws, a=(sh, q, k, v, T, nq, out, None), w=window: vc.vc_verify_attn_window(*a, ws, window=w) or a[6].clone())
        calls.append(lambda ws, a=(sh, fc, q[:, 0].contiguous(), torch.empty_like(out[:, 0])), w=window: vc.vc_draft_attn_fp4(*a, ws, window=w) or a[3].clone())
        sizes += [vc.vc_verify_attn_window_workspace_size(sh, T, nq, window), vc.vc_draft_attn_fp4_workspace_size(sh, fc)]
    alone = [c(vc.workspace(n)) for c, n in zip(calls, sizes)]
    ws = vc.workspace(max(sizes))
    for order in (range(8), reversed(range(8)), (0, 4, 1, 4, 2, 5, 3, 5, 6, 4, 7)):
        for i in order:
            assert torch.equal(calls[i](ws), alone[i])


def test_two_streams_at_once():
    B, Hkv, g, D, T = 2, 2, 4, 128, 30000
    sh = vc.shape(B, g * Hkv, Hkv, D)
    runs = []
    for s in range(2):
        k, v = (x.to(dev) for x in synth.kv_full(B, Hkv, T, D, seed=s))
        fc = vc.fp4_cache(vc.fp4_records(B, Hkv, T, D), lens=ints([T, 9000 + s]))
        vc.vc_fp4_cache_write(sh, fc, k, v, T, vc.workspace(256))
        q = synth.normal((B, g * Hkv, D), seed=s).to(dev)
        runs.append((fc, q, torch.empty(B, g * Hkv, D, device=dev), vc.workspace(vc.vc_draft_attn_fp4_workspace_size(sh, fc)),
                     torch.cuda.Stream()))
    want = []
    for fc, q, out, ws, _ in runs:
        vc.vc_draft_attn_fp4(sh, fc, q, out, ws)
        want.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for fc, q, out, ws, stream in runs:
            vc.vc_draft_attn_fp4(sh, fc, q, out, ws, stream=stream)
            vc.vc_draft_attn_fp4(sh, fc, q, out, ws, window=500, stream=stream)
            vc.vc_draft_attn_fp4(sh, fc, q, out, ws, stream=stream)
    torch.cuda.synchronize()
    for (_, _, out, ws, _), w in zip(runs, want):
        assert torch.equal(out, w) and vc.vc_workspace_flags(ws) == 0


def test_raw_pointers_take_their_dtype():
    B, Hkv, n, D = 1, 2, 20, 64
    k, v = (x.to(dev) for x in synth.kv_full(B, Hkv, n, D, seed=7, dtype=torch.float16))
    sh = vc.shape(B, Hkv, Hkv, D)
    a, b = vc.fp4_cache(vc.fp4_records(B, Hkv, n, D)), vc.fp4_cache(vc.fp4_records(B, Hkv, n, D))
    ws = vc.workspace(256)
    vc.vc_fp4_cache_write(sh, a, k, v, n, ws)
    vc.vc_fp4_cache_write(sh, b, k.data_ptr(), v.data_ptr(), n, ws.data_ptr(), dtype=torch.float16)
    torch.cuda.synchronize()
    assert torch.equal(a._keep[0], b._keep[0])
    with pytest.raises(ValueError, match="dtype"):
        vc.vc_fp4_cache_write(sh, b, k.data_ptr(), v.data_ptr(), n, ws)
