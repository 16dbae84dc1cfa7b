"""GPU tests of the linear layer over 4-bit weights on whole numbers, equal to the last bit (group4_exact.py): sizes that bring every
kernel, tile and way of cutting K into use, the longest streamed rows among them."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int6_weight_export_amd import ops  # noqa: E402
from tests import group4_exact as ex  # noqa: E402

# tokens x outputs x inputs
STREAM = [(1, 5, 25), (1, 6, 31), (1, 40, 2048), (1, 33, 2079), (1, 33, 4101), (1, 100, 4096), (1, 70, 6001), (1, 33, 6144), (1, 20, 8190), (1, 70, 8192),
          (1, 9, 14001), (1, 20, 16384), (1, 35, 26656), (1, 70, 30031), (1, 9, 32766), (1, 9, 32768), (1, 66000, 6176), (2, 50, 2048), (2, 90, 4064),
          (2, 40, 8192), (2, 9, 16384), (2, 33, 14016), (2, 70000, 32)]
TILES = [(1, 300, 24), (1, 9, 32770), (2, 33, 4101), (3, 4100, 520), (6, 48, 16392), (9, 16000, 300), (10, 8100, 1030), (5, 20000, 4500), (4, 8100, 4500),
         (16, 130, 9000), (16, 4096, 4096), (16, 9000, 12300), (16, 28672, 2100), (12, 1000, 30000), (3, 66000, 1030), (17, 500, 30000), (20, 4100, 520),
         (24, 9000, 12300), (32, 8192, 4000), (32, 20000, 4500), (30, 48, 16392), (30, 28672, 2100), (33, 30000, 520), (50, 520, 4100), (50, 4100, 14500),
         (64, 80, 16392), (64, 8200, 1030), (64, 14400, 4100), (64, 8192, 8192), (129, 300, 4100), (129, 4100, 4100)]


@pytest.mark.parametrize("M,N,K", STREAM + TILES)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_whole_numbers(M, N, K, group):
    print(f"[case] linear4 whole numbers {M}x{N}x{K} group {group}", flush=True)
    sys.stdout.flush()
    x, code, e = ex.layer(M, N, K, group, M + N + K, "cuda")
    got = ops.qlinear4(x.bfloat16(), ex.pack(code), torch.exp2(e.double()).half(), group=group, out_dtype=torch.float32)
    want = ex.product(x, ex.weights(code, e, group))
    assert torch.equal(got.double(), want)
