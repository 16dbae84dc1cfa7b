"""GPU tests of every tile of the linear layer's matrix kernels, whole and in parts, in both output types, against 64
bits: outputs sampled at the tiles' edges and at random.  Bounds as derived in linear_ref and in the tests of dZ's
precision."""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int6_weight_export_amd import ops  # noqa: E402
from tests import linear_ref as ref, linear_tiles as lt  # noqa: E402
from tests.test_gpu_linear import T, f64, within  # noqa: E402
from tests.test_gpu_linear_precision import bounds  # noqa: E402


def say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def layer(M, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(-31, 32, (N, K), generator=g, device="cuda", dtype=torch.int8)
    scales = (torch.rand(N, generator=g, device="cuda") * 0.002 + 0.001).half()
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    return g, codes, scales, (codes.float() * scales.float()[:, None]).bfloat16(), x


def sample(n, rng, most=24):
    """Indices at the edges of tiles and of the matrix, and some at random."""
    edge = [0, 1, 31, 32, 63, 64, 127, 128, 191, 192, 255, 256, n - 257, n - 65, n - 33, n - 2, n - 1]
    return np.unique([i for i in edge if 0 <= i < n] + list(rng.integers(0, n, most)))


@pytest.mark.parametrize("args,plan", lt.FORWARD)
def test_forward_tile(args, plan):
    M, N, K, y, res = args
    say(f"forward tile {plan} {M}x{N}x{K}")
    assert lt.forward_plan(*args) == plan
    g, codes, scales, what, x = layer(M, N, K, M)
    bias = torch.randn(N, generator=g, device="cuda")
    r = None if not res else torch.randn(M, N, generator=g, device="cuda").to(T[res])
    out, z = ops.qlinear(x, codes, scales, bias=bias, act="silu", residual=r, want_z=True, out_dtype=T[y])
    again = ops.qlinear(x, codes, scales, bias=bias, act="silu", residual=r, out_dtype=T[y])
    torch.cuda.synchronize()
    assert again.shape == out.shape and bool(out.isfinite().all()) and bool(z.isfinite().all())
    rng = np.random.default_rng(M)
    i, j = sample(M, rng), sample(N, rng)
    zr, ez, yr, ey = ref.forward(f64(x[i]), f64(what[j]), f64(bias[j]), "silu", 0.0, None if r is None else f64(r[i][:, j]), y)
    within(z[i][:, j], zr, ez, "z")
    within(out[i][:, j], yr, ey, "y")


@pytest.mark.parametrize("args,plan", lt.BACKWARD)
def test_backward_tile(args, plan):
    M, N, K, want, t, act = args
    say(f"backward tile {plan} {M}x{N}x{K}")
    assert lt.backward_plan(*args) == plan
    g, codes, scales, what, x = layer(M, N, K, M + 1)
    dy = torch.randn(M, N, generator=g, device="cuda").bfloat16()
    z = torch.randn(M, N, generator=g, device="cuda").bfloat16()
    bits = torch.rand(N, (K + 7) // 8 * 8, generator=g, device="cuda") > 0.2
    mask = (bits.view(N, -1, 8).int() << torch.arange(8, device="cuda", dtype=torch.int32)).sum(2).to(torch.uint8)
    kw = dict(x=x, z=z, act=act, mask=mask, want_dx="dx" in want, want_dw="dw" in want, want_dbias="dbias" in want,
              dx_dtype=T[t], dw_dtype=T[t])
    got = ops.qlinear_backward(dy, codes, scales, **kw)
    again = ops.qlinear_backward(dy, codes, scales, **kw)
    torch.cuda.synchronize()
    assert set(got) == set(want.split())
    for k, v in got.items():
        assert torch.equal(v, again[k]) and bool(v.isfinite().all()), k
    rng = np.random.default_rng(M)
    m, n, k = sample(M, rng), sample(N, rng), sample(K, rng)

    def dz(rows, cols):
        d = f64(dy[rows][:, cols])
        s = ref.act_grad(f64(z[rows][:, cols]), act, 0.0) if act != "none" else np.ones_like(d)
        return d * s, (np.zeros_like(d) if act == "none" else 16 * ref.U * np.abs(d) * np.maximum(np.abs(s), 1.0))

    every = slice(None)
    if "dx" in got:
        d, ed = dz(m, every)
        v, e = bounds(d, ed, f64(what[:, k]), np.zeros((len(m), 1)), None, t, t)["dx"]
        within(got["dx"][m][:, k], v, e, "dx")
    if "dw" in got:
        d, ed = dz(every, n)
        v, e = bounds(d, ed, np.zeros((len(n), 1)), f64(x[:, k]), bits[n][:, k].cpu().numpy(), t, t)["dw"]
        within(got["dw"][n][:, k], v, e, "dw")
        if "dbias" in got:
            within(got["dbias"][n], d.sum(0), ed.sum(0) + (M + 1) * ref.U * (np.abs(d) + ed).sum(0) + ref.TINY["f32"], "dbias")
