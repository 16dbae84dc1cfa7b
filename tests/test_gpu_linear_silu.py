"""GPU tests of the SiLU at arguments whose exponential is next to the ends of binary32: it must not vanish while it and
its value are still normal numbers.

Bounds, u = 2^-24.  exp, a sum, a reciprocal and two products: within 8 u of the value (as in linear_ref).  Below -87.3
e^z is subnormal, off by up to 2^-149 (rounded, and the exponential's own last place), which |z| multiplies: 2 |z| 2^-149.
The derivative's factor of e^z is below 1 + |z| there.  Stored as bf16 a value adds 2^-8 of itself and 2^-134."""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int6_weight_export_amd import ops  # noqa: E402
from tests import linear_ref as ref  # noqa: E402
from tests.test_gpu_linear import T, f64, within  # noqa: E402

Z = np.unique(np.concatenate([np.linspace(-104, -80, 193), np.linspace(-20, 20, 81), np.linspace(80, 104, 25)])).astype(np.float32)


def say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", [(3, 0), (3, 16), (40, 64), (70, 64), (300, 24)])
def test_values(M, K, y):
    """X = 0, so that the bias is Z: the few-token, element-load and matrix kernels."""
    say(f"silu of {len(Z)} arguments, {M} tokens, K = {K}, {y}")
    bias = torch.from_numpy(Z).cuda()
    codes = torch.ones(len(Z), K, dtype=torch.int8, device="cuda")
    scales = torch.ones(len(Z), dtype=torch.float16, device="cuda")
    got = ops.qlinear(torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"), codes, scales, bias=bias, act="silu", out_dtype=T[y])
    torch.cuda.synchronize()
    z = Z.astype(np.float64)
    want = z / (1 + np.exp(-z))
    bound = ref.stored(want, 8 * ref.U * np.abs(want) + 2 * np.abs(z) * 2.0 ** -149, y)
    within(got, np.broadcast_to(want, (M, len(Z))), np.broadcast_to(bound, (M, len(Z))), "silu")


@pytest.mark.parametrize("M", [3, 70])
def test_slopes(M):
    """db of M equal rows of Z and dY = 1: M times the derivative, the sum of M equal terms exact or off by M u."""
    say(f"slope of silu, {M} tokens")
    zt = torch.from_numpy(Z).bfloat16()
    z = zt.double().numpy()
    got = ops.qlinear_backward(torch.ones(M, len(Z), device="cuda"), None, None, z=zt.cuda().expand(M, -1).contiguous(), act="silu",
                               want_dx=False, want_dw=False, want_dbias=True)["dbias"]
    torch.cuda.synchronize()
    s = 1 / (1 + np.exp(-z))
    want = s * (1 + z * (1 - s))
    # the two terms of the factor cancel near z = -1.278; 1 - s is off by 2 u for z > 0
    e = 8 * ref.U * np.abs(s) * (1 + np.abs(z)) + 2 * (1 + np.abs(z)) * 2.0 ** -149
    within(got, M * want, M * e + M * ref.U * M * (np.abs(want) + e), "slope")
