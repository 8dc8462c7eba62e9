"""A changed header rebuilds its users: every header that a source file of the
library includes from the tree counts (CPU only, nothing is compiled)."""
import glob
import os
import re

from lossless_draft_verify_vc_b200 import build as B


def included(path, seen):
    for name in re.findall(r'#include "([^"]+)"', open(path).read()):
        p = os.path.normpath(os.path.join(os.path.dirname(path), name))
        if p not in seen:
            seen.add(p)
            included(p, seen)
    return seen


def test_every_included_header_counts():
    used = set()
    for src in glob.glob(os.path.join(B.CSRC, "*.cu")):
        included(src, used)
    assert used and all(os.path.exists(p) for p in used)
    assert used <= {os.path.normpath(p) for p in B._headers()}
