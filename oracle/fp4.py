"""Reference of the 4-bit floating-point draft cache and of windowed
attention (oracle; test infrastructure only).

What the pages fix: a compressed cache is known by its bits per element
([P2] "Key Contributions"); drafting reads it one token at a time, the
verifier checks a block of rows against the full cache ([P1] "The Core
Idea").  The number format (e2m1 codes, an e4m3 scale per 16 channels of a
token, an optional power of two per KV head), the record layout and the
visibility rule (a sliding window that includes the row's own token, and
first tokens that stay visible) are readings: the pages are silent.

Everything is float64 and written element by element from the definition.
"""

from __future__ import annotations

import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_table() -> np.ndarray:
    """Values of the finite non-negative e4m3 codes 0 .. 126."""
    out = []
    for i in range(127):
        e, m = divmod(i, 8)
        out.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(out)


def nearest(x: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Index of the entry of an ascending table nearest to x >= 0, ties to the
    even index, values past the last entry saturating."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(table, x), 0, len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    with np.errstate(invalid="ignore"):
        dl, dh = x - table[lo], table[hi] - x
    take_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    return np.where(np.isinf(x), len(table) - 1, np.where(take_lo, lo, hi))


def quantise(x: np.ndarray, exp: np.ndarray | None = None):
    """x [B, H, T, D] -> (codes [B, H, T, D] in 0..15, scale codes
    [B, H, T, D/16]); exp [H] powers of two."""
    with np.errstate(invalid="ignore"):
        x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), 0.0, x)
    if exp is not None:
        x = x * np.array([2.0 ** -int(np.clip(e, -60, 60)) for e in exp])[None, :, None, None]
    xb = x.reshape(*x.shape[:-1], -1, 16)
    scales = nearest(np.abs(xb).max(-1) / 6.0, e4m3_table())
    s = e4m3_table()[scales][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        mag = nearest(np.where(s > 0, np.abs(xb) / np.where(s > 0, s, 1.0), 0.0), E2M1)
    codes = np.where(s > 0, mag + 8 * np.signbit(xb), 0)
    return codes.reshape(x.shape).astype(np.uint8), scales.astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray, exp: np.ndarray | None = None) -> np.ndarray:
    """x_hat [B, H, T, D] of codes and scale codes."""
    v = np.where(codes >= 8, -1.0, 1.0) * E2M1[codes & 7]
    v = v * np.repeat(e4m3_table()[scales], 16, axis=-1)
    if exp is not None:
        v = v * np.array([2.0 ** int(np.clip(e, -60, 60)) for e in exp])[None, :, None, None]
    return v


def addresses(D: int):
    """Byte addresses inside a record: key code bytes and value code bytes
    [16][D/2] (byte i holds channels 2i, 2i + 1), key and value scales
    [16][D/16]."""
    kc = np.zeros((16, D // 2), int)
    vc = np.zeros((16, D // 2), int)
    ks = np.zeros((16, D // 16), int)
    vs = np.zeros((16, D // 16), int)
    for t in range(16):
        for i in range(D // 2):
            c = 2 * i
            gr, x = c // (D // 8), c % (D // 8) // 2
            kc[t, i] = t * (D // 2) + i
            if D == 128:
                vc[t, i] = 8 * D + (t // 8) * 512 + gr * 64 + (t % 8 // 2) * 16 + (t % 2) * 8 + x
            else:
                vc[t, i] = 8 * D + gr * 64 + (t % 8 // 2) * 16 + (t // 8) * 8 + (t % 2) * 4 + x
        for j in range(D // 16):
            ks[t, j] = 16 * D + ((t % 8) * 16 + (j // 2) * 4 + (t // 8) * 2 + j % 2 if D == 128
                                 else (t % 8) * 8 + j * 2 + t // 8)
            vs[t, j] = 17 * D + j * 16 + (t % 8 // 2) * 4 + (t // 8) * 2 + t % 2
    return kc, vc, ks, vs


def pack(kc, ks, vc, vs, records: np.ndarray, pos: np.ndarray, counts: np.ndarray) -> np.ndarray:
    """Writes rows i < counts[b] of codes and scales (as from quantise) as tokens
    pos[b] + i into a copy of records [B, H, T_cap/16, 18 D]."""
    out = records.copy()
    D = out.shape[-1] // 18
    a = addresses(D)
    for b in range(out.shape[0]):
        for i in range(int(counts[b])):
            r, t = divmod(int(pos[b]) + i, 16)
            for codes, at in ((kc, a[0]), (vc, a[1])):
                c = codes[b, :, i]
                out[b, :, r, at[t]] = (c[:, 0::2] | (c[:, 1::2] << 4)).T
            for sc, at in ((ks, a[2]), (vs, a[3])):
                out[b, :, r, at[t]] = sc[b, :, i].T
    return out


def unpack(records: np.ndarray):
    """records [B, H, R, 18 D] -> (kc, ks, vc, vs) with tokens in order [B, H, 16 R, ..]."""
    B, H, n, nb = records.shape
    D = nb // 18
    a = addresses(D)

    def codes(at):
        byte = records[..., at.reshape(-1)].reshape(B, H, n * 16, D // 2)
        return np.stack([byte & 15, byte >> 4], -1).reshape(B, H, n * 16, D)

    def scale(at):
        return records[..., at.reshape(-1)].reshape(B, H, n * 16, D // 16)

    return codes(a[0]), scale(a[2]), codes(a[1]), scale(a[3])


def window_attention(q, k, v, lens, window: int = 0, n_sink: int = 0, sm_scale: float | None = None):
    """q [B, nq, Hq, D]; k, v [B, Hkv, T, D]; lens [B].  Row i of request b sits
    at p = lens[b] - nq + i and sees t <= p with t > p - window (window > 0)
    or t < n_sink.  Returns (o, lse, amp, peak): amp = sum_t p_t |v_t| and
    peak = max_t sum_c |q_c k_tc| * scale bound what rounding can do to a row."""
    q = np.asarray(q, np.float64)
    B, nq, Hq, D = q.shape
    Hkv = k.shape[1]
    g = Hq // Hkv
    scale = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
    o = np.zeros((B, nq, Hq, D))
    amp = np.zeros((B, nq, Hq, D))
    lse = np.full((B, nq, Hq), -np.inf)
    peak = np.zeros((B, nq, Hq))
    for b in range(B):
        for i in range(nq):
            p = int(lens[b]) - nq + i
            t = np.arange(max(p + 1, 0))
            t = t[((t > p - window) | (t < n_sink)) if window > 0 else np.ones(len(t), bool)]
            if not len(t):
                continue
            for hq in range(Hq):
                kk = np.asarray(k[b, hq // g, t], np.float64)
                vv = np.asarray(v[b, hq // g, t], np.float64)
                s = kk @ q[b, i, hq] * scale
                w = np.exp(s - s.max())
                l = w.sum()
                o[b, i, hq] = w @ vv / l
                amp[b, i, hq] = w @ np.abs(vv) / l
                lse[b, i, hq] = s.max() + math.log(l)
                peak[b, i, hq] = (np.abs(kk) @ np.abs(q[b, i, hq])).max() * scale
    return o, lse, amp, peak
