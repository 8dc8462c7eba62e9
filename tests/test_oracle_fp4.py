"""Pins of the 4-bit floating-point cache's oracle (CPU only): hand-worked
values and ties, the record layout as a bijection, and closed forms of the
visibility rule."""

import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import fp4 as F


def _block(first):
    x = np.zeros((1, 1, 1, 64))
    x[0, 0, 0, : len(first)] = first
    return x


def test_hand_worked_block_ties_go_to_the_even_code():
    # largest 6 -> scale 1 (e4m3 code 56); halfway values: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1,
    # 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4, and just past a tie rounds up
    x = _block([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -5, 0.26, 5.01, -6, 0.1, -0.0, 3])
    codes, s = F.quantise(x)
    assert s[0, 0, 0].tolist() == [56, 0, 0, 0]
    assert codes[0, 0, 0, :16].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 14, 1, 7, 15, 0, 8, 5]
    assert not codes[0, 0, 0, 16:].any()
    assert F.values(codes, s)[0, 0, 0, :8].tolist() == [6, 0, 1, 1, 2, 2, 4, 4]


def test_scale_rounding_saturation_and_tiny_blocks():
    t = F.e4m3_table()
    assert t[56] == 1.0 and t[126] == 448.0 and t[1] == 2.0 ** -9
    # max 6.375 -> 1.0625, halfway between 1 (code 56, even) and 1.125 -> 56
    assert F.quantise(_block([6.375]))[1][0, 0, 0, 0] == 56
    assert F.quantise(_block([6.4]))[1][0, 0, 0, 0] == 57
    c, s = F.quantise(_block([1e6, 1.0, np.inf]))
    assert s[0, 0, 0, 0] == 126 and c[0, 0, 0, :3].tolist() == [7, 0, 7]
    c, s = F.quantise(_block([6 * 2.0 ** -10, -1e-3]))  # scale halfway to the smallest: even = 0, all codes 0
    assert s[0, 0, 0, 0] == 0 and not c.any()
    assert F.quantise(_block([np.nan, 6.0]))[0][0, 0, 0, :2].tolist() == [0, 7]


def test_head_exponent_moves_small_values_into_range():
    x = np.random.default_rng(0).standard_normal((1, 2, 3, 64))
    a = F.values(*F.quantise(x), None)
    e = np.array([-20, -20])
    b = F.values(*F.quantise(x * 2.0 ** -20, e), e)
    assert np.array_equal(a * 2.0 ** -20, b)


def test_scale_table_agrees_with_torch():
    f8 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(f8, F.e4m3_table())


@pytest.mark.parametrize("D", [64, 128])
def test_layout_is_a_bijection_and_pack_unpack_agree(D):
    at = np.concatenate([a.reshape(-1) for a in F.addresses(D)])
    assert sorted(at.tolist()) == list(range(18 * D))
    rng = np.random.default_rng(D)
    rec = rng.integers(0, 256, (2, 3, 4, 18 * D), dtype=np.uint8)
    kc, ks, vc, vs = (x[:, :, 5:30] for x in F.unpack(rec))
    again = F.pack(kc, ks, vc, vs, rec, np.array([5, 5]), np.array([25, 25]))
    assert np.array_equal(rec, again)
    moved = F.pack(kc, ks, vc, vs, rec, np.array([20, 39]), np.array([25, 0]))
    assert np.array_equal(F.unpack(moved)[0][0, :, 20:45], kc[0]) and np.array_equal(moved[1], rec[1])
    assert np.array_equal(F.unpack(moved)[3][0, :, :20], F.unpack(rec)[3][0, :, :20])


def test_window_attention_reduces_to_known_forms():
    rng = np.random.default_rng(5)
    B, nq, Hq, Hkv, D, T = 2, 4, 4, 2, 16, 30
    q, k, v = (rng.standard_normal(s) for s in ((B, nq, Hq, D), (B, Hkv, T, D), (B, Hkv, T, D)))
    want, wl = A.verify_attention(q, k, v)
    for window, sinks in ((0, 0), (T, 0), (3, T)):  # nothing hidden
        o, l, _, _ = F.window_attention(q, k, v, [T, T], window, sinks)
        assert np.allclose(o, want, atol=1e-13) and np.allclose(l, wl, atol=1e-13)
    o, l, _, _ = F.window_attention(q, k, v, [T, T], 1, 0)  # only its own key
    assert np.allclose(o[:, 2, 1], v[:, 0, T - 2], atol=1e-14)
    k1 = np.zeros_like(k)  # equal keys: the mean of what is visible
    o, _, _, _ = F.window_attention(q, k1, v, [T, 2], 5, 3)
    seen = [0, 1, 2] + list(range(T - nq + 1 - 4, T - nq + 2))
    assert np.allclose(o[0, 1, 0], v[0, 0, seen].mean(0), atol=1e-14)
    # a request of 2 rows with a block of 4: the first two rows see nothing
    o, l, _, _ = F.window_attention(q, k, v, [T, 2], 5, 3)
    assert not o[1, :2].any() and np.isneginf(l[1, :2]).all() and np.allclose(o[1, 2], np.repeat(v[1, :, 0], 2, 0))
