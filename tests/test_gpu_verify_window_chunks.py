"""Windowed verification where a request's keys are cut into many chunks whose
partials meet in a second launch, with requests of different lengths: chunks
without tiles, requests without keys and with fewer keys than rows, garbage
behind every length; both head sizes, one and two row tiles.

Tolerance: derived in test_gpu_verify_window."""

import pytest

from lossless_draft_verify_vc_b200 import vc
from tests import test_gpu_verify_window as VW

pytestmark = pytest.mark.gpu

# header and tickets, then nothing of a size: what a call without partials asks for
SMALL = 300_000


@pytest.mark.parametrize("nq,g,Hkv,D,lens,window,sinks,partials", [
    (31, 4, 1, 128, [20000, 0, 70], 0, 0, True),        # 79 chunks
    (31, 4, 1, 64, [20000, 0, 20], 12345, 70, True),    # 98 chunks, fewer keys than rows
    (10, 1, 8, 128, [20000, 0, 70], 0, 0, True),        # 12 chunks: the merge of few partials
    (10, 1, 8, 64, [20000, 9000, 5], 15000, 40, True),
    (31, 5, 2, 128, [9000], 8000, 130, True),           # two row tiles, 65 chunks
    (31, 5, 2, 128, [6000, 3100], 5000, 130, True),     # two row tiles, 28 chunks
    (31, 5, 2, 64, [6000, 17], 0, 0, True),
    (31, 5, 8, 128, [2950, 40], 2000, 130, False),      # two row tiles, a cluster of 7
    (31, 8, 4, 128, [1500, 0], 700, 0, False),
])
def test_ragged_requests_over_many_chunks(nq, g, Hkv, D, lens, window, sinks, partials):
    B, T = len(lens), max(lens) + 7
    size = vc.vc_verify_attn_window_workspace_size(vc.shape(B, g * Hkv, Hkv, D), T, nq, window, sinks)
    assert (size > SMALL) == partials
    q, k, v = VW.make(B, Hkv, T, D, nq, g * Hkv, seed=nq + D, lens=lens)
    if window and B == 1:  # keys between the first tokens and the windows
        lo = lens[0] - nq + 1 - window
        k[0, :, sinks:lo], v[0, :, sinks:lo] = float("nan"), float("-inf")
    o, l, flags = VW.run(q, k, v, window, sinks, lens=lens)
    assert flags == 0
    if window and B == 1:
        k[0, :, sinks:lo], v[0, :, sinks:lo] = 0, 0
    VW.check(o, l, q, k, v, lens, window, sinks)
