"""Register and scratch budgets of the linear layer's and AdamW's kernels (CPU; reads the compiler's resource report that
the build writes)."""
import json
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RES = os.path.join(ROOT, "int6_weight_export_amd", "_build", "resources.json")

pytestmark = pytest.mark.skipif(not os.path.exists(RES), reason="library not built here (no resource report)")


def kernels(pattern):
    with open(RES) as f:
        return {k: v for k, v in json.load(f).items() if re.search(pattern, k)}


def test_no_kernel_spills():
    every = kernels(r"pgq_mm_|pgq_linear_|pgq_adamw_")
    assert len(every) > 40
    bad = {k: v for k, v in every.items() if v["scratch"] or v["vgpr_spill"]}
    assert not bad, bad


@pytest.mark.parametrize("pattern,count,vgprs,occupancy", [
    (r"pgq_mm_nt_kernelI", 14, 256, 2),         # (two wavefronts a SIMD: 256 registers each)
    (r"pgq_mm_tt_kernelI", 4, 256, 2),
    (r"pgq_mm_both_kernelI", 10, 256, 2),
    (r"pgq_mm_\w\w_reduce_kernelI", 11, 64, 8),
    (r"pgq_linear_skinny_kernelI", 3, 128, 4),
    (r"pgq_linear_prep_kernel", 1, 96, 5),
    (r"pgq_adamw_kernelILi\d+ELi[01]E", 4, 104, 4),
    (r"pgq_adamw_kernelILi\d+ELi2E", 2, 128, 4),
    (r"pgq_adamw_decode_kernel", 1, 64, 8),
])
def test_budgets(pattern, count, vgprs, occupancy):
    got = kernels(pattern)
    assert len(got) == count, sorted(got)
    bad = {k: v for k, v in got.items() if v["vgprs"] > vgprs or v["occupancy"] < occupancy}
    assert not bad, bad
