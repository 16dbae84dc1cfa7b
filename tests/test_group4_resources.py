"""Register and scratch budgets of the 4-bit kernels and of the gradient norm (CPU; reads the compiler's resource report that the
build writes)."""
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
    every = kernels(r"pgq_linear4_|_groups_kernel|pgq_grad_")
    assert len(every) > 30
    bad = {k: v for k, v in every.items() if v["scratch"] or v["vgpr_spill"]}
    assert not bad, bad


@pytest.mark.parametrize("pattern,count,vgprs,occupancy", [
    (r"pgq_linear4_stream_kernelILi[12]ELi1E", 2, 136, 3),
    (r"pgq_linear4_stream_kernelILi[34]ELi1E", 2, 184, 2),
    (r"pgq_linear4_stream_kernelILi[12]ELi2E", 2, 168, 3),
    (r"pgq_linear4_rows_kernelILi1ELi1E", 3, 104, 4),
    (r"pgq_linear4_rows_kernelILi1ELi2E", 3, 144, 3),
    (r"pgq_linear4_rows_kernelILi2ELi1E", 3, 144, 3),
    (r"pgq_linear4_rows_kernelILi4ELi1E", 3, 232, 2),
    (r"pgq_linear4_shared_kernelILi[12]ELi1E", 6, 128, 4),
    (r"pgq_linear4_shared_kernelILi[12]ELi2E", 6, 184, 2),
    (r"pgq_linear4_shared_kernelILi4ELi[12]E", 6, 256, 2),
    (r"pgq_quantize_groups_kernelI", 6, 48, 8),
    (r"pgq_dequant_groups_kernelI", 2, 32, 8),
    (r"pgq_grad_norm_kernel", 1, 72, 7),
    (r"pgq_grad_scale_kernel", 1, 64, 8),
    (r"pgq_grad_clip_small_kernel", 1, 128, 4),
])
def test_budgets(pattern, count, vgprs, occupancy):
    got = kernels(pattern)
    assert len(got) == count, sorted(got)
    bad = {k: v for k, v in got.items() if v["vgprs"] > vgprs or v["occupancy"] < occupancy}
    assert not bad, bad
