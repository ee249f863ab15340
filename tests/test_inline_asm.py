"""Inline assembly in the kernels' sources: what it writes is named as written."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mamba_selective_scan_04_amd", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.hpp")) + glob.glob(os.path.join(CSRC, "*.hip")))


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_m0_is_named(path):
    """The address of loads into LDS goes into M0; unnamed, the compiler may keep a value of its own there."""
    text = open(path).read()
    for stmt in re.findall(r"\basm\b(?:\s+volatile)?\s*\((.*?)\);", text, re.S):
        code, _, rest = stmt.partition("::")
        if re.search(r"\b(s_mov_b32|s_add_u32|s_movk_i32)\s+m0\b", code):
            assert '"m0"' in rest, stmt
