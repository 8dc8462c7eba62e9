"""Kernels launched as programmatic dependents wait for the grid before them
before they let the next one start: a caller of the quantised draft with
VC_CACHE_STATIC promises something about its direct predecessor only, so that
predecessor must not be resident while an older grid still writes.  They also
read nothing through the read-only path, which a grid may use only for memory
that nobody writes while it is resident."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "lossless_draft_verify_vc_b200", "csrc")
WAIT, LAUNCH = "griddepcontrol.wait", "griddepcontrol.launch_dependents"
FILES = ["vc_fp4.cu", "vc_draft_fp4.cu", "vc_verify_rows.cu"]


def code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


@pytest.mark.parametrize("name", FILES)
def test_wait_precedes_launch(name):
    order = re.findall(rf'asm volatile\("({WAIT}|{LAUNCH})', code(name))
    kernels = len(re.findall(r"__global__", code(name)))
    assert order == [WAIT, LAUNCH] * kernels


@pytest.mark.parametrize("name", FILES + ["vc_stream.cuh", "vc_fp4.cuh"])
def test_no_read_only_loads(name):
    assert not re.search(r"__ldg\(|ld\.global\.nc", code(name))
