"""GPU tests of the precision and the infinities of the linear layer's gradient: dZ = dY act'(Z) is a binary32
value, and what enters the products stands for it more closely than the outputs' own rounding does.

Bounds, u = 2^-24.  For a bf16 output dZ enters as two bf16 values, its upper 8 bits and 8 bits of the rest: the
rest is below 2^-7 |dZ|, and what its 8 bits leave, cut off or rounded, below 2^-7 of that: 2^-14 |dZ|.  For an
fp32 output the parts' sum is dZ.  (A part that would be zero is 2^-40 dZ, which 2^-39 |dZ| covers.)  P parts make P times as many terms of the same total magnitude: (P L + 1) u sum |a b|.
dZ itself is formed in binary32, 16 u |dY| max(|act'|, 1) off as in linear_ref.
"""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int6_weight_export_amd import ops  # noqa: E402
from tests import linear_ref as ref  # noqa: E402
from tests.test_gpu_linear import T, f64, grads, weights, within  # noqa: E402


def say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def bounds(d, ed, w, x, mask, dx, dw):
    """{name: (value, bound)} of dx and dw for the 64-bit dZ d, off by at most ed."""
    out = {}
    for name, a, b, t in (("dx", d, w, dx), ("dw", d.T, x, dw)):
        e = (ed if name == "dx" else ed.T) + (2.0 ** -39 if t == "f32" else 2.0 ** -14) * np.abs(a)
        v = a @ b
        e = e @ np.abs(b) + (3 * a.shape[1] + 1) * ref.U * ((np.abs(a) + e) @ np.abs(b))
        e = ref.stored(v, e, t)
        if name == "dw" and mask is not None:
            v, e = np.where(mask, v, 0.0), np.where(mask, e, 0.0)
        out[name] = (v, e)
    return out


@pytest.mark.parametrize("M,N,K", [(1, 7, 33), (3, 130, 65), (65, 200, 176), (200, 513, 528), (300, 72, 40), (777, 129, 264),
                                   (2049, 65, 130), (1000, 1000, 24)])
@pytest.mark.parametrize("act,slope", [("none", 0.0), ("relu", 0.5), ("relu", 0.3), ("relu2", 0.5), ("relu2", -0.7), ("silu", 0.0)])
@pytest.mark.parametrize("dy_t,dx,dw", [("bf16", "bf16", "bf16"), ("f32", "bf16", "bf16"), ("f32", "f32", "f32"),
                                        ("bf16", "f32", "f32"), ("f32", "bf16", "f32"), ("f32", "f32", "bf16")])
def test_gradients_of_unrounded_dz(M, N, K, act, slope, dy_t, dx, dw):
    say(f"unrounded dZ {M}x{N}x{K} {act} {slope} dy={dy_t} dx={dx} dw={dw}")
    codes, scales, w, x, dy, z, mask, keep = grads(M, N, K, act, slope, True, M + N, dy_t)
    g = ref.act_grad(f64(z), act, slope) if z is not None else np.ones((M, N))
    d = f64(dy) * g
    ed = np.zeros_like(d) if act == "none" else 16 * ref.U * np.abs(f64(dy)) * np.maximum(np.abs(g), 1.0)
    want = bounds(d, ed, w, f64(x), keep, dx, dw)
    kw = dict(z=z, act=act, slope=slope)
    both = ops.qlinear_backward(dy, codes, scales, x=x, mask=mask, want_dbias=True, dx_dtype=T[dx], dw_dtype=T[dw], **kw)
    alone = {**ops.qlinear_backward(dy, codes, scales, want_dw=False, dx_dtype=T[dx], **kw),
             **ops.qlinear_backward(dy, None, None, x=x, mask=mask, want_dx=False, dw_dtype=T[dw], **kw)}
    torch.cuda.synchronize()
    for got in (both, alone):
        for name, (v, e) in want.items():
            within(got[name], v, e, name)


def test_unrounded_dz_through_the_element_loads():
    """Rows of 2^21 inputs go through the element-load kernel; N = 3, so that dX has few terms, and X and the
    codes are zero but for 200 columns, whose sums over M are compared."""
    say("unrounded dZ with K past 2^21")
    M, N, K, live = 70, 3, (1 << 21) + 24, 200
    g = torch.Generator(device="cuda").manual_seed(3)
    at = torch.cat([torch.arange(live - 30, device="cuda") * 10007, torch.arange(K - 30, K, device="cuda")])
    codes = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    codes[:, at] = torch.randint(-31, 32, (N, live), generator=g, device="cuda", dtype=torch.int8)
    scales = torch.full((N,), 0.0123, device="cuda", dtype=torch.float16)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[:, at] = torch.randn(M, live, generator=g, device="cuda").bfloat16()
    dy = torch.randn(M, N, generator=g, device="cuda")
    z = torch.randn(M, N, generator=g, device="cuda").bfloat16()
    w = f64((codes[:, at].float() * scales.float()[:, None]).bfloat16())
    gr = ref.act_grad(f64(z), "silu", 0.0)
    d = f64(dy) * gr
    ed = 16 * ref.U * np.abs(f64(dy)) * np.maximum(np.abs(gr), 1.0)
    for t in ("f32", "bf16"):
        got = ops.qlinear_backward(dy, codes, scales, x=x, z=z, act="silu", dx_dtype=T[t], dw_dtype=T[t])
        torch.cuda.synchronize()
        want = bounds(d, ed, w, f64(x[:, at]), None, t, t)
        for name, (v, e) in want.items():
            within(got[name][:, at], v, e, name)
        rest = torch.ones(K, dtype=torch.bool, device="cuda")
        rest[at] = False
        assert not bool(got["dx"][:, rest].any()) and not bool(got["dw"][:, rest].any())


@pytest.mark.parametrize("dy_t,dx,dw", [("f32", "f32", "f32"), ("f32", "bf16", "bf16"), ("bf16", "bf16", "f32")])
@pytest.mark.parametrize("M,N,K", [(5, 24, 40), (200, 264, 136), (1030, 70, 300)])
def test_infinities_follow_the_formula(M, N, K, dy_t, dx, dw):
    """An infinite weight, input or dY makes an infinity of the product's sign, NaN only where the formula has
    one (0 * infinity, infinities of both signs), also for a dZ that fewer bits hold exactly."""
    say(f"infinities in backward {M}x{N}x{K} dy={dy_t} dx={dx} dw={dw}")
    codes, scales, w, x, dy, z, mask, keep = grads(M, N, K, "silu", 0.0, False, 7, dy_t)
    z.uniform_(0.5, 4.0, generator=torch.Generator(device="cuda").manual_seed(1))     # act' > 0
    dy[0, :] = dy[0, :].abs() + 1.0
    dy[:, 3] = 1.0                                                                     # (one bit)
    dy[1, 5] = float("inf")
    codes[7, :] = codes[7, :].abs() + 1
    scales[7] = float("inf")
    x[2, 9] = float("inf")
    x[4, 9] = 1.0
    got = ops.qlinear_backward(dy, codes, scales, x=x, z=z, act="silu", dx_dtype=T[dx], dw_dtype=T[dw])
    torch.cuda.synchronize()
    s = ref.act_grad(f64(z), "silu", 0.0)
    with np.errstate(all="ignore"):
        d = f64(dy) * s
        wd = f64((codes.float() * scales.float()[:, None]).bfloat16())
        xd = f64(x)
        # column 7 of dZ meets the infinite weights, everything else is finite but dZ[1, 5] and X[2, 9]
        for name, a, b in (("dx", d, wd), ("dw", d.T, xd)):
            want = np.zeros((a.shape[0], b.shape[1]))
            for l in range(a.shape[1]):
                want = want + a[:, l:l + 1] * b[l:l + 1, :]
            out = f64(got[name])
            assert np.array_equal(np.isnan(want), np.isnan(out)), name
            inf = np.isinf(want)
            assert inf.any() and np.array_equal(inf, np.isinf(out)) and np.array_equal(np.sign(want[inf]), np.sign(out[inf])), name


def test_largest_and_smallest_dz():
    """dZ next to the largest binary32 number does not overflow on its way into the products; subnormal dZ leave
    no NaN."""
    say("largest and smallest dZ")
    M, N, K = 130, 24, 40
    codes, scales, w, x, dy, z, mask, keep = grads(M, N, K, "none", 0.0, False, 9, "f32")
    big = float(np.float32(3.4028235e38))
    dy.zero_()
    dy[0, 0], dy[1, 1], dy[2, 2] = big, -big, 1e-41
    scales.fill_(2.0 ** -10)
    codes.fill_(1)
    x.fill_(2.0 ** -10)
    got = ops.qlinear_backward(dy, codes, scales, x=x, dx_dtype=torch.float32, dw_dtype=torch.float32)
    torch.cuda.synchronize()
    want = big * 2.0 ** -10
    assert np.all(np.abs(f64(got["dx"])[0] - want) <= 2.0 ** -22 * want) and np.all(np.abs(f64(got["dx"])[1] + want) <= 2.0 ** -22 * want)
    assert np.all(np.abs(f64(got["dw"])[0] - want) <= 2.0 ** -22 * want)
    assert bool((got["dx"][2:].abs() <= 1e-43).all()) and bool(got["dx"].isfinite().all())
    # nothing of a row of zeros, not even of the parts
    assert not bool(got["dx"][3:].any()) and not bool(got["dw"][3:].any())
