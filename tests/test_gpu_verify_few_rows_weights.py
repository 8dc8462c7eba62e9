"""At most 8 rows per KV head: a softmax weight keeps all 24 bits of fp32.

Two visible keys.  Their scores are single products of 16-bit numbers times
the scale, so they are exact up to the scale's own rounding: a weight is off
by at most 2^-22 (the exponential), 2^-24 (its argument's rounding) and
3 * 2^-24 of |s| <= 2 (the scale's roundings): eps = 2^-21.  The second key's
score is picked so that bits 17 to 24 of its weight are nearly all ones, and
the values are 1 and -1: a sum that dropped those bits would be off by about
2^-17 of a weight.  Each of the two sums and the quotient adds at most 2^-23:
the bound is 2 eps + 3 * 2^-23 of amp = 1."""

import numpy as np
import pytest
import torch

from lossless_draft_verify_vc_b200 import vc
from oracle import fp4 as F
from tests.vcutil import np32

pytestmark = pytest.mark.gpu
dev = "cuda"
BOUND = 2 * 2.0 ** -21 + 3 * 2.0 ** -23


def low_bits(w):
    """Share of bits 17 to 24 of w's significand that are set, of 1."""
    m = np.frexp(w)[0] * 2.0 ** 16
    return m - np.floor(m)


def scores(n, seed):
    """n scores in (-2, -1) with 8 significant bits whose weights have high low bits."""
    s = -(1 + np.arange(1, 128) / 128)
    s = s[np.argsort(-low_bits(np.exp(s)))][:40]
    return np.random.default_rng(seed).choice(s[low_bits(np.exp(s)) > 0.8], n)


@pytest.mark.parametrize("B,Hkv,g,D,nq,T", [(1, 1, 1, 128, 1, 2), (3, 2, 4, 128, 1, 500), (2, 4, 8, 64, 1, 4000), (1, 25, 2, 64, 1, 60),
                                            (2, 2, 4, 128, 2, 3), (1, 1, 1, 64, 8, 9)])
def test_weights_keep_24_bits(B, Hkv, g, D, nq, T):
    window = 2
    s = scores(Hkv * B, seed=D + T).reshape(B, Hkv)
    # every row sees the last two keys up to its own: scores 0 and s in turn
    k, v = torch.zeros(B, Hkv, T, D), torch.zeros(B, Hkv, T, D)
    odd = torch.arange(T) % 2 == 1
    k[..., 3] = torch.where(odd, torch.from_numpy(s).float()[..., None], torch.zeros(()))
    v[:] = torch.where(odd, -1.0, 1.0)[:, None]
    q = torch.zeros(B, nq, g * Hkv, D)
    q[..., 3] = 1.0
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    assert np.array_equal(np32(k)[..., 3].min(-1), s)
    wo, wl, amp, _ = F.window_attention(np32(q), np32(k), np32(v), [T] * B, window, 0, 1.0)
    # without the last 8 bits of a weight (planted in the oracle) the bound is missed
    w = np.exp(s)
    lost = w - low_bits(w) * 2.0 ** -16 * 2.0 ** np.frexp(w)[1]
    assert (np.abs((1 - lost) / (1 + w) - (1 - w) / (1 + w)) > BOUND).all()
    sh = vc.shape(B, g * Hkv, Hkv, D, 1.0)
    ws = vc.workspace(vc.vc_verify_attn_window_workspace_size(sh, T, nq, window, 0))
    out, lse = torch.empty(B, nq, g * Hkv, D, device=dev), torch.empty(B, nq, g * Hkv, device=dev)
    vc.vc_verify_attn_window(sh, q.to(dev), k.to(dev), v.to(dev), T, nq, out, lse, ws, window=window)
    assert (np.abs(np32(out) - wo) <= BOUND * amp).all()
    assert (np.abs(np32(lse) - wl) <= BOUND + 2.0 ** -23).all()
