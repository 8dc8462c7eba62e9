"""Kernels that are resident while the call before them still writes what they
will read name the instruction of every load from such memory: a plain
dereference leaves the compiler free to take the read-only path as soon as it
can prove that the kernel itself does not write there."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "lossless_draft_verify_vc_b200", "csrc")


def code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


@pytest.mark.parametrize("name", ["vc_stream.cuh", "vc_draft_fp4.cu", "vc_verify_rows.cu", "vc_fp4.cu"])
def test_lengths_positions_and_rows_are_loaded_by_name(name):
    src = code(name)
    assert not re.search(r"\b(lens|pos|counts|k_exp|v_exp|part_o|part_ml)\[", src)
    assert not re.search(r"[=?] *\*?src\[", src)
