"""Threads that wait on an mbarrier are ordered behind its initialisation by
another thread: in every kernel file, a warp or block barrier stands between
mbar_init and the first wait that follows.  (A missing one cannot be shown by
running: a warp's shared-memory accesses happen to issue in order.)"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "lossless_draft_verify_vc_b200", "csrc")


def code(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


FILES = sorted(p for p in glob.glob(os.path.join(CSRC, "*.cu")) if "mbar_init(&" in code(p))


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_a_barrier_stands_between_initialisation_and_waits(path):
    events = re.findall(r"mbar_init\(&|__syncwarp\(|__syncthreads\(|mbar_\w*wait\w*\(", code(path))
    ready = True
    for e in events:
        if e.startswith("mbar_init"):
            ready = False
        elif e.startswith("__sync"):
            ready = True
        else:
            assert ready, f"{e[:-1]} follows mbar_init without a barrier"


def test_the_files_with_barriers_of_their_own_are_covered():
    assert {"vc_draft_fp4.cu", "vc_draft_quant.cu", "vc_draft_sparse.cu", "vc_verify.cu"} <= {os.path.basename(p) for p in FILES}
