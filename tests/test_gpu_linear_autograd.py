"""GPU test: qlinear is no autograd function; a caller who expects a gradient is told."""
import warnings

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int6_weight_export_amd import ops  # noqa: E402


def test_arguments_that_require_a_gradient_are_warned_about():
    print("[case] qlinear on tensors that require a gradient", flush=True)
    codes = torch.ones(8, 16, dtype=torch.int8, device="cuda")
    scales = torch.full((8,), 0.5, dtype=torch.float16, device="cuda")
    x = torch.randn(3, 16, device="cuda").bfloat16()
    b, r = torch.randn(8, device="cuda"), torch.randn(3, 8, device="cuda")
    want = ops.qlinear(x, codes, scales, bias=b, residual=r)
    for k in range(3):
        a = [t.clone().requires_grad_(i == k) for i, t in enumerate((x, b, r))]
        with pytest.warns(UserWarning, match="qlinear_backward"):
            y = ops.qlinear(a[0], codes, scales, bias=a[1], residual=a[2])
        assert not y.requires_grad and torch.equal(y, want)
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with torch.no_grad():
                assert torch.equal(ops.qlinear(a[0], codes, scales, bias=a[1], residual=a[2]), want)
            assert torch.equal(ops.qlinear(x, codes, scales, bias=b, residual=r), want)
    torch.cuda.synchronize()
