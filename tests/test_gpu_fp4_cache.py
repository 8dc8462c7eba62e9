"""The 4-bit floating-point cache's write and read against the oracle: records
byte for byte, values exactly (their only rounding is to fp16 outputs)."""

import numpy as np
import pytest
import torch

from lossless_draft_verify_vc_b200 import synth, vc
from oracle import fp4 as F
from tests.vcutil import np32

pytestmark = pytest.mark.gpu
dev = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def rand_records(B, H, T, D, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 256, (B, H, -(-T // 16), 18 * D), generator=g, dtype=torch.int32).to(torch.uint8)


def write(rec, k, v, pos, counts=None, k_exp=None, v_exp=None, Hq=None):
    B, H, n, D = k.shape
    r = rec.to(dev)
    fc = vc.fp4_cache(r, k_exp=k_exp, v_exp=v_exp)
    ws = vc.workspace(vc.vc_compress_workspace_size())
    vc.vc_fp4_cache_write(vc.shape(B, Hq or H, H, D), fc, k.to(dev), v.to(dev), n, ws, pos=pos, counts=counts)
    return r, vc.vc_workspace_flags(ws)


def want_write(rec, k, v, pos, counts, k_exp=None, v_exp=None):
    kc, ks = F.quantise(np32(k), k_exp)
    vc_, vs = F.quantise(np32(v), v_exp)
    return F.pack(kc, ks, vc_, vs, rec.numpy(), np.array(pos), np.array(counts))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,pos,counts", [
    (1, [0, 15], [1, 1]),           # single tokens at a record's ends
    (1, [16, 37], [1, 0]),          # one request without a row
    (7, [13, 3], [7, 5]),           # across a record's border; inside one
    (33, [0, 47], [33, 17]),        # whole records and both kinds of edge
    (100, [1, 28], [100, 99]),
])
def test_records_equal_the_oracle_and_other_bytes_stay(D, dtype, n, pos, counts):
    B, H, T = 2, 3, 128
    k, v = synth.kv_full(B, H, n, D, seed=n + D, dtype=dtype)
    rec = rand_records(B, H, T, D, seed=7)
    got, flags = write(rec, k, v, ints(pos), ints(counts))
    assert flags == 0
    assert np.array_equal(got.cpu().numpy(), want_write(rec, k, v, pos, counts))


def test_every_16_bit_pattern():
    """Blocks of raw bf16 and fp16 patterns (subnormals, infinities, NaN, both
    zeros): each pattern appears among random ones of nearby exponents, so that
    it meets many scales; ties are constructed in a second tensor."""
    D, n = 128, 1024
    for dtype in (torch.bfloat16, torch.float16):
        bits = np.arange(65536, dtype=np.uint16).reshape(1, 1, 512, D)
        rng = np.random.default_rng(3)
        mant = {torch.bfloat16: 7, torch.float16: 10}[dtype]
        # a second half: blocks whose values stay within 4 binades of each other
        e = rng.integers(4, {torch.bfloat16: 250, torch.float16: 26}[dtype], (1, 1, 512, D // 16, 1))
        near = ((e + rng.integers(-3, 2, (1, 1, 512, D // 16, 16))) << mant) + rng.integers(0, 1 << mant, (1, 1, 512, D // 16, 16))
        near = (near | (rng.integers(0, 2, near.shape) << 15)).astype(np.uint16).reshape(1, 1, 512, D)
        x = torch.from_numpy(np.concatenate([bits, near], 2).astype(np.int16)).view(dtype)
        rec = rand_records(1, 1, n, D, seed=1)
        got, flags = write(rec, x, x.flip(2), ints([0]))
        assert flags == vc.VC_FLAG_RANGE  # NaN and infinities are among them
        assert np.array_equal(got.cpu().numpy(), want_write(rec, x, x.flip(2), [0], [n]))


def test_exact_ties_between_codes_and_between_scales():
    """x = border * s for every e4m3 scale s of a bf16-sized block maximum: the
    quotient lies exactly between two codes."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for s in F.e4m3_table()[1:]:
        for m in (6.0 * s, 5.75 * s, 6.25 * s):
            x = np.zeros(64)
            x[:7], x[7:14] = mids * s, -mids * s
            x[14], x[15] = m, -m
            x[16:32] = x[:16] * (1 + 2.0 ** -7)
            x[32:48] = x[:16] * (1 - 2.0 ** -8)
            rows.append(x)
    x = torch.from_numpy(np.array(rows)[None, None]).to(torch.float16)
    n = x.shape[2]
    rec = rand_records(1, 1, n, 64, seed=2)
    got, flags = write(rec, x, -x, ints([0]))
    assert np.array_equal(got.cpu().numpy(), want_write(rec, x, -x, [0], [n]))
    assert flags == vc.VC_FLAG_RANGE  # 6.25 * 448 is past the range


def test_range_and_nan_are_flagged_and_stored_as_documented():
    x = synth.normal((1, 1, 4, 64), seed=1).float()
    fine = x.clone()
    for bad in (3e3, float("inf"), float("nan"), float("-inf")):
        x = fine.clone()
        x[0, 0, 2, 5] = bad
        rec = rand_records(1, 1, 16, 64, seed=3)
        got, flags = write(rec, x.to(torch.bfloat16), fine.to(torch.bfloat16), ints([3]))
        assert flags == vc.VC_FLAG_RANGE
        assert np.array_equal(got.cpu().numpy(), want_write(rec, x.to(torch.bfloat16), fine.to(torch.bfloat16), [3], [4]))


@pytest.mark.parametrize("exp", [[0, 3], [-60, 60], [-100, 100], [-7, 1]])
def test_head_exponents(exp):
    B, H, n, D = 1, 2, 20, 64
    k, v = synth.kv_full(B, H, n, D, seed=4)
    k = (k.float() * torch.tensor([2.0 ** max(-60, min(60, e)) for e in exp])[None, :, None, None]).to(torch.bfloat16)
    rec = rand_records(B, H, 32, D, seed=5)
    e = ints(exp)
    got, flags = write(rec, k, v, ints([5]), k_exp=e)
    assert flags == 0 and np.array_equal(got.cpu().numpy(), want_write(rec, k, v, [5], [n], k_exp=exp))
    ws = vc.workspace(vc.vc_compress_workspace_size())
    ko, vo = (torch.empty(B, H, n, D, device=dev) for _ in range(2))
    vc.vc_fp4_cache_read(vc.shape(B, H, H, D), vc.fp4_cache(got, k_exp=e, v_exp=e), n, ko, vo, ws, pos0=5)
    kc, ks, vc_, vs = (a[:, :, 5:5 + n] for a in F.unpack(got.cpu().numpy()))
    assert np.array_equal(ko.cpu().numpy(), F.values(kc, ks, exp)) and np.array_equal(vo.cpu().numpy(), F.values(vc_, vs, exp))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_read_gives_the_stored_values_and_leaves_other_rows(D, dtype):
    B, H, T, n = 3, 2, 96, 41
    k, v = synth.kv_full(B, H, T, D, seed=6)
    rec, _ = write(rand_records(B, H, T, D, 1), k, v, ints([0] * B))
    pos, counts = [0, 30, 55], [41, 0, 23]
    ko = torch.full((B, H, n, D), -7.0, dtype=dtype, device=dev)
    vo = torch.full_like(ko, -9.0)
    ws = vc.workspace(vc.vc_compress_workspace_size())
    vc.vc_fp4_cache_read(vc.shape(B, H, H, D), vc.fp4_cache(rec), n, ko, vo, ws, pos=ints(pos), counts=ints(counts))
    kc, ks, vc_, vs = F.unpack(rec.cpu().numpy())
    wk, wv = F.values(kc, ks), F.values(vc_, vs)
    for b in range(B):
        for out, want, fill in ((ko, wk, -7.0), (vo, wv, -9.0)):
            w = torch.from_numpy(want[b, :, pos[b]:pos[b] + counts[b]]).to(dtype)
            assert torch.equal(out[b, :, :counts[b]].cpu(), w)
            assert (out[b, :, counts[b]:] == fill).all()
    assert vc.vc_workspace_flags(ws) == 0


def test_requests_that_do_not_fit_are_skipped_and_flagged():
    B, H, n, D = 5, 2, 4, 64
    k, v = synth.kv_full(B, H, n, D, seed=8)
    rec = rand_records(B, H, 32, D, seed=9)
    pos, counts = [-1, 29, 28, 0, 2], [4, 4, 4, 5, -1]
    got, flags = write(rec, k, v, ints(pos), ints(counts))
    assert flags == vc.VC_FLAG_BAD_LENGTH
    ok = [0, 0, 4, 0, 0]  # only request 2 fits
    assert np.array_equal(got.cpu().numpy(), want_write(rec, k, v, [0, 0, 28, 0, 0], ok))
    out = torch.full((B, H, n, D), 3.0, device=dev)
    ws = vc.workspace(vc.vc_compress_workspace_size())
    vc.vc_fp4_cache_read(vc.shape(B, H, H, D), vc.fp4_cache(got), n, out, out.clone(), ws, pos=ints(pos), counts=ints(counts))
    assert vc.vc_workspace_flags(ws) == vc.VC_FLAG_BAD_LENGTH
    assert (out[[0, 1, 3, 4]] == 3.0).all() and not (out[2] == 3.0).all()
    # nothing fits: pos0 + n past the capacity
    got2, flags = write(rec, k, v, ints([30] * B))
    assert flags == vc.VC_FLAG_BAD_LENGTH and torch.equal(got2.cpu(), rec)


def test_byte_offsets_past_32_bits():
    B, H, D, T = 1, 8, 128, 1 << 22
    rec = torch.empty(B, H, T // 16, 18 * D, dtype=torch.uint8, device=dev)  # 4.8 GB
    rec[:, :, -2:] = 0
    k, v = synth.kv_full(B, H, 9, D, seed=10)
    ws = vc.workspace(vc.vc_compress_workspace_size())
    fc, sh = vc.fp4_cache(rec), vc.shape(B, 8, H, D)
    vc.vc_fp4_cache_write(sh, fc, k.to(dev), v.to(dev), 9, ws, pos0=T - 12)
    want = want_write(torch.zeros(B, H, 2, 18 * D, dtype=torch.uint8), k, v, [20], [9])
    assert np.array_equal(rec[:, :, -2:].cpu().numpy(), want)
    ko, vo = (torch.empty(B, H, 9, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    vc.vc_fp4_cache_read(sh, fc, 9, ko, vo, ws, pos0=T - 12)
    kc, ks, vc_, vs = (a[:, :, 20:29] for a in F.unpack(want))
    assert np.array_equal(np32(ko), F.values(kc, ks)) and np.array_equal(np32(vo), F.values(vc_, vs))


def test_a_long_write_on_another_stream_then_the_same_rows_token_by_token():
    B, H, n, D = 2, 4, 700, 128
    k, v = synth.kv_full(B, H, n, D, seed=11)
    kd, vd = k.to(dev), v.to(dev)
    recs = [vc.fp4_records(B, H, n, D) for _ in range(2)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ws = vc.workspace(vc.vc_compress_workspace_size())
    torch.cuda.synchronize()
    sh = vc.shape(B, 4 * H, H, D)
    vc.vc_fp4_cache_write(sh, vc.fp4_cache(recs[0]), kd, vd, n, ws, stream=s)
    one = vc.fp4_cache(recs[1])
    for i in range(n):
        vc.vc_fp4_cache_write(sh, one, kd[:, :, i:i + 1].contiguous(), vd[:, :, i:i + 1].contiguous(), 1, ws, pos0=i)
    torch.cuda.synchronize()
    assert torch.equal(recs[0], recs[1])
