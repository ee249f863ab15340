"""The compiler's resource report of the hybrid's kernels, both stream types:
no vector registers spilled, but for the gradients of fp32 streams at heads of
128 by 128, whose operands in three parts leave some for scratch."""
import csv
import glob
import os
import re

import pytest

BUILD = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mamba_selective_scan_04_amd", "_build")
ROWS = []
for path in glob.glob(os.path.join(BUILD, "launch_*.resources.tsv")):
    with open(path) as f:
        ROWS += [r for r in csv.DictReader(f, delimiter="\t") if re.search(r"\d(delta|kv)_\w+_kernel", r["kernel"])]
pytestmark = pytest.mark.skipif(not ROWS, reason="no resource report (run the build first)")

SPILLING = {"delta_grad_kernelIfLi128ELi128ELb0E": 10, "delta_grad_kernelIfLi128ELi128ELb1E": 43}


def test_both_stream_types_are_covered():
    for kernel in ("delta_prep", "delta_chain", "delta_adjoint", "delta_grad", "delta_step", "kv_commit", "kv_attn", "kv_join"):
        for stream in "tf":
            assert any("%s_kernelI%s" % (kernel, stream) in r["kernel"] for r in ROWS), (kernel, stream)


def test_vector_registers():
    over = {}
    for r in ROWS:
        may = max((n for k, n in SPILLING.items() if k in r["kernel"]), default=0)
        if int(r["vgpr_spill"] or 0) > may:
            over[r["kernel"]] = r["vgpr_spill"]
    assert not over, over


def test_scalar_registers_are_reported():
    """Scalars spilled go to lanes of a vector register, counted in the report; not to memory."""
    assert all(r["sgpr_spill"] != "" for r in ROWS)
    for r in ROWS:
        if int(r["vgpr_spill"] or 0) == 0:
            assert int(r["scratch"] or 0) == 0, r["kernel"]
