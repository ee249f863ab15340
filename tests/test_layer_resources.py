"""The compiler's resource report of the kernels around the scans and of the
cache's upkeep, both stream types: no vector registers spilled, no scratch."""
import csv
import glob
import os
import re

import pytest

BUILD = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mamba_selective_scan_04_amd", "_build")
ROWS = []
for path in glob.glob(os.path.join(BUILD, "launch_*.resources.tsv")):
    with open(path) as f:
        ROWS += [r for r in csv.DictReader(f, delimiter="\t") if re.search(r"\d(conv|norm|kv_weights|kv_evict|parts)_\w*kernel", r["kernel"])]
pytestmark = pytest.mark.skipif(not ROWS, reason="no resource report (run the build first)")


@pytest.mark.parametrize("kernel", ["conv_kernelI[tf]", "conv_bwd_kernelI[tf]", "norm_kernelI(tt|tf|ff)", "norm_bwd_kernelI(tt|tf|ff)",
                                    "norm_wide_kernelI(tt|tf|ff)", "norm_wide_bwd_kernelI(tt|tf|ff)", "kv_weights_kernelI[tf]", "kv_evict_kernel",
                                    "parts_sum_kernel"])
def test_nothing_spills(kernel):
    got = [r for r in ROWS if re.search(r"\d" + kernel, r["kernel"])]
    assert got
    over = {r["kernel"]: (r["vgpr_spill"], r["scratch"]) for r in got if int(r["vgpr_spill"] or 0) or int(r["scratch"] or 0)}
    assert not over, over
