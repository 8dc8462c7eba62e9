"""The 4-bit cache stores a negative zero, and negative numbers that round to
zero, as code 8 under every scale: records byte for byte as the oracle's."""

import numpy as np
import pytest
import torch

from lossless_draft_verify_vc_b200 import vc
from oracle import fp4 as F
from tests.test_gpu_fp4_cache import ints, rand_records, want_write, write

pytestmark = pytest.mark.gpu


def rows(D, dtype):
    """One token per e4m3 scale; every block of 16 holds its maximum, zeros of
    both signs and small numbers of both signs, at places that move."""
    out = []
    for s in F.e4m3_table()[1:]:
        blk = np.array([6 * s, -0.0, 0.0, -0.2 * s, 0.2 * s, -0.0, -1e-7, 0.0, -0.0, 0.5 * s, -0.5 * s, -0.0, 0.0, -0.0, -3 * s, -0.0])
        out.append(np.concatenate([np.roll(blk, i) for i in range(D // 16)]))
    return torch.from_numpy(np.array(out)[None, None]).to(dtype)


@pytest.mark.parametrize("exp", [None, [-3], [-60]])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
def test_zeros_keep_their_sign_under_every_scale(D, dtype, exp):
    x = rows(D, dtype)
    n = x.shape[2]
    e = None if exp is None else ints(exp)
    rec = rand_records(1, 1, n, D, seed=D)
    got, flags = write(rec, x, -x, ints([0]), k_exp=e, v_exp=e)
    want = want_write(rec, x, -x, [0], [n], exp, exp)
    assert np.array_equal(got.cpu().numpy(), want)
    if exp is None:
        assert flags == 0
        kc = F.unpack(want)[0][:, :, :n]
        assert (kc[torch.signbit(x).numpy() & (x == 0).numpy()] == 8).all()
