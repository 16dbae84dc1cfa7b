"""GPU tests of the quantized linear layer (bias, activation, residual) and its gradient against the
definitions in 64 bits; the bounds are derived in linear_ref.py."""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import oracle  # noqa: E402
from int6_weight_export_amd import ops, pgq  # noqa: E402
from tests import linear_ref as ref  # noqa: E402

T = {"f32": torch.float32, "bf16": torch.bfloat16}


def say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def weights(N, K, seed, pad=0):
    """Device codes (row stride K + pad) and scales, and the bf16 weights they stand for in float64."""
    rng = np.random.default_rng(seed)
    w = oracle.f32_to_bf16((rng.standard_normal((N, max(K, 1))) * 0.05).astype(np.float32))
    fq = oracle.fakequant_rows(w, 31)
    codes, scales = fq["codes"][:, :K], fq["scales"]
    buf = torch.full((N, K + pad), 77, dtype=torch.int8)
    buf[:, :K] = torch.from_numpy(np.ascontiguousarray(codes))
    sc = torch.from_numpy(scales.view(np.int16).copy()).view(torch.float16)
    what = (torch.from_numpy(codes.astype(np.float32)) * sc.float()[:, None]).bfloat16().double().numpy()
    return buf.cuda()[:, :K], sc.cuda(), what


def randn(shape, seed, dtype, std=1.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    t = torch.full((shape[0], shape[1] + pad), float("nan"))
    t[:, :shape[1]] = torch.randn(shape, generator=g) * std
    return t.to(dtype).cuda()[:, :shape[1]]


def within(got, want, bound, what):
    got = f64(got)
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off; worst {np.nanmax(err / np.maximum(bound, 1e-300)):.3g} bounds"


# sizes around the tiles of every kernel variant (skinny, 16-byte rows or not, one tile and several)
SHAPES = [(1, 1, 1), (1, 16, 1), (1, 7, 33), (2, 1584, 528), (3, 130, 65), (15, 64, 96), (16, 48, 512), (17, 33, 1040),
          (31, 257, 100), (33, 96, 32), (63, 129, 72), (64, 128, 64), (65, 200, 176), (100, 7, 1000), (127, 131, 257),
          (128, 256, 128), (129, 255, 63), (200, 513, 528), (257, 1, 80), (300, 1584, 40), (520, 390, 1032)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("y", ["bf16", "f32"])
def test_forward_shapes(M, N, K, y):
    say(f"linear forward {M}x{N}x{K} {y}")
    codes, scales, w = weights(N, K, M + N + K)
    x = randn((M, K), 1, torch.bfloat16)
    bias = randn((1, N), 2, torch.float32)[0]
    got, z = ops.qlinear(x, codes, scales, bias=bias, act="relu2", slope=0.5, want_z=True, out_dtype=T[y])
    torch.cuda.synchronize()
    zr, ez, yr, ey = ref.forward(f64(x), w, f64(bias), "relu2", 0.5, y=y)
    within(z, zr, ez, "z")
    within(got, yr, ey, "y")


@pytest.mark.parametrize("act,slope", [("none", 0.0), ("relu", 0.0), ("relu", 0.25), ("relu2", 0.0), ("relu2", 0.5),
                                       ("relu2", -0.5), ("silu", 0.0)])
@pytest.mark.parametrize("M", [1, 40, 200])
@pytest.mark.parametrize("y,res,bias", [("bf16", "", ""), ("f32", "f32", "bf16"), ("bf16", "bf16", "f32"),
                                        ("f32", "bf16", "f32"), ("bf16", "f32", "")])
def test_forward_epilogues(act, slope, M, y, res, bias):
    say(f"linear forward epilogue {act} {slope} M={M} y={y} residual={res} bias={bias}")
    N, K = 136, 112
    codes, scales, w = weights(N, K, 5)
    x = randn((M, K), 3, torch.bfloat16, std=4.0)
    b = randn((1, N), 4, T[bias])[0] if bias else None
    r = randn((M, N), 6, T[res], std=2.0) if res else None
    got = ops.qlinear(x, codes, scales, bias=b, act=act, slope=slope, residual=r, out_dtype=T[y])
    torch.cuda.synchronize()
    _, _, yr, ey = ref.forward(f64(x), w, None if b is None else f64(b), act, slope, None if r is None else f64(r), y)
    within(got, yr, ey, "y")


@pytest.mark.parametrize("M", [1, 50, 300])
@pytest.mark.parametrize("padx,padc", [(8, 16), (1, 3), (2, 4), (0, 5)])
@pytest.mark.parametrize("K", [96, 101])
def test_forward_strided_views_write_nothing_else(M, padx, padc, K):
    say(f"linear forward strided M={M} K={K} padx={padx} padc={padc}")
    N = 150
    codes, scales, w = weights(N, K, 7, pad=padc)
    x = randn((M, K), 8, torch.bfloat16, pad=padx)         # NaN in the padding: must not be read into a sum
    for y, off, more in (("f32", 1, 3), ("bf16", 1, 2), ("bf16", 0, 8)):
        buf = torch.full((M, N + more), 7.0, dtype=T[y], device="cuda")
        ops.qlinear(x, codes, scales, act="relu", slope=0.1, out=buf[:, off:off + N], out_dtype=T[y])
        torch.cuda.synchronize()
        _, _, yr, ey = ref.forward(f64(x), w, None, "relu", 0.1, y=y)
        within(buf[:, off:off + N], yr, ey, "y")
        assert bool((buf[:, :off] == 7.0).all()) and bool((buf[:, off + N:] == 7.0).all())


@pytest.mark.parametrize("M", [2, 130])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_forward_residual_in_place(M, t):
    say(f"linear forward into its own residual M={M} {t}")
    N, K = 200, 64
    codes, scales, w = weights(N, K, 9)
    x, r = randn((M, K), 10, torch.bfloat16), randn((M, N), 11, T[t])
    r0 = f64(r)
    got = ops.qlinear(x, codes, scales, residual=r, out=r, out_dtype=T[t])
    torch.cuda.synchronize()
    assert got is r
    _, _, yr, ey = ref.forward(f64(x), w, None, "none", 0.0, r0, t)
    within(r, yr, ey, "y")


def test_forward_empty_and_k_zero():
    say("linear forward M = 0, N = 0, K = 0")
    codes, scales, _ = weights(5, 16, 1)
    assert ops.qlinear(randn((0, 16), 1, torch.bfloat16), codes, scales).shape == (0, 5)
    assert ops.qlinear(randn((3, 16), 1, torch.bfloat16), codes[:0], scales[:0]).shape == (3, 0)
    b, r = randn((1, 5), 2, torch.float32)[0], randn((3, 5), 3, torch.float32)
    for M in (3, 200):
        r = randn((M, 5), 3, torch.float32)
        y, z = ops.qlinear(torch.empty(M, 0, dtype=torch.bfloat16, device="cuda"),
                           torch.empty(5, 0, dtype=torch.int8, device="cuda"), scales, bias=b, act="relu", slope=0.5,
                           residual=r, want_z=True, out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert torch.equal(z, b.bfloat16().expand(M, 5))
        assert torch.equal(y, torch.where(b > 0, b, b * 0.5) + r)


def test_forward_infinities_and_nan_stay_in_their_rows():
    say("linear forward with NaN and infinity in single rows of X")
    for M in (4, 150):
        codes, scales, w = weights(70, 80, 3)
        x = randn((M, 80), 5, torch.bfloat16)
        clean = ops.qlinear(x, codes, scales, act="silu", out_dtype=torch.float32)
        x2 = x.clone()
        x2[1, 7] = float("nan")
        x2[3, 0] = float("inf")
        got = ops.qlinear(x2, codes, scales, act="silu", out_dtype=torch.float32)
        torch.cuda.synchronize()
        rows = [i for i in range(M) if i not in (1, 3)]
        assert torch.equal(got[rows], clean[rows])
        assert bool(got[1].isnan().all()) and not bool(got[3].isfinite().all())


def test_forward_is_repeatable_and_matches_qgemm():
    say("linear forward twice, and beside the bare GEMM")
    M, N, K = 2000, 1584, 528
    codes, scales, w = weights(N, K, 12)
    x = randn((M, K), 13, torch.bfloat16)
    a = ops.qlinear(x, codes, scales, act="silu", out_dtype=torch.float32)
    b = ops.qlinear(x, codes, scales, act="silu", out_dtype=torch.float32)
    c = ops.qlinear(x, codes, scales, out_dtype=torch.float32)
    d = ops.qgemm(x, codes, scales.view(torch.int16))
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    mag = np.abs(f64(x)) @ np.abs(w).T
    assert np.all(np.abs(f64(c) - f64(d)) <= 2 * (K + 1) * ref.U * mag)


def grads(M, N, K, act, slope, masked, seed, dy_t="bf16", padx=0, padc=0):
    codes, scales, w = weights(N, K, seed, pad=padc)
    x = randn((M, K), seed + 1, torch.bfloat16, pad=padx)
    dy = randn((M, N), seed + 2, T[dy_t], std=0.1, pad=padx)
    z = randn((M, N), seed + 3, torch.bfloat16) if act != "none" else None
    mask = keep = None
    if masked:
        bits = torch.rand(N, (K + 7) // 8 * 8, generator=torch.Generator().manual_seed(seed)) > 0.2
        keep = bits[:, :K].numpy()
        mask = (bits.view(N, -1, 8).int() << torch.arange(8, dtype=torch.int32)).sum(2).to(torch.uint8).cuda()
    return codes, scales, w, x, dy, z, mask, keep


def check_grads(got, dy, z, x, w, act, slope, keep, dy_t="bf16", dx="bf16", dw="bf16"):
    want = ref.backward(f64(dy), f64(z) if z is not None else None, f64(x), w, act, slope, keep, dy_t, dx, dw)
    for k, t in got.items():
        within(t, *want[k], k)


@pytest.mark.parametrize("M,N,K", SHAPES + [(1000, 40, 24), (2049, 65, 130)])
@pytest.mark.parametrize("act,masked", [("none", False), ("relu2", True)])
def test_backward_shapes(M, N, K, act, masked):
    say(f"linear backward {M}x{N}x{K} {act} masked={masked}")
    codes, scales, w, x, dy, z, mask, keep = grads(M, N, K, act, 0.5, masked, M + K)
    got = ops.qlinear_backward(dy, codes, scales, x=x, z=z, act=act, slope=0.5, mask=mask, want_dbias=True)
    torch.cuda.synchronize()
    assert set(got) == {"dx", "dw", "dbias"}
    check_grads(got, dy, z, x, w, act, 0.5, keep)


@pytest.mark.parametrize("act,slope", [("none", 0.0), ("relu", 0.25), ("relu2", -0.5), ("silu", 0.0)])
@pytest.mark.parametrize("dy_t,dx,dw", [("bf16", "f32", "f32"), ("f32", "bf16", "f32"), ("f32", "f32", "bf16")])
@pytest.mark.parametrize("padx,padc", [(0, 0), (8, 16), (1, 3)])
def test_backward_types_and_strides(act, slope, dy_t, dx, dw, padx, padc):
    say(f"linear backward {act} dy={dy_t} dx={dx} dw={dw} pad={padx},{padc}")
    codes, scales, w, x, dy, z, mask, keep = grads(140, 88, 72, act, slope, True, 21, dy_t, padx, padc)
    got = ops.qlinear_backward(dy, codes, scales, x=x, z=z, act=act, slope=slope, mask=mask, want_dbias=True,
                               dx_dtype=T[dx], dw_dtype=T[dw])
    torch.cuda.synchronize()
    check_grads(got, dy, z, x, w, act, slope, keep, dy_t, dx, dw)


def test_backward_each_gradient_alone():
    say("linear backward, one gradient at a time beside all at once")
    codes, scales, w, x, dy, z, mask, keep = grads(300, 120, 200, "silu", 0.0, True, 30)
    kw = dict(z=z, act="silu")
    every = ops.qlinear_backward(dy, codes, scales, x=x, mask=mask, want_dbias=True, **kw)
    again = ops.qlinear_backward(dy, codes, scales, x=x, mask=mask, want_dbias=True, **kw)
    dx = ops.qlinear_backward(dy, codes, scales, want_dw=False, **kw)
    dw = ops.qlinear_backward(dy, None, None, x=x, mask=mask, want_dx=False, **kw)
    db = ops.qlinear_backward(dy, None, None, want_dx=False, want_dw=False, want_dbias=True, **kw)
    torch.cuda.synchronize()
    assert set(dx) == {"dx"} and set(dw) == {"dw"} and set(db) == {"dbias"}
    for got in (dx, dw, db):                  # (the tiles, and so the order of the sums, may differ from the joint call's)
        check_grads(got, dy, z, x, w, "silu", 0.0, keep)
    assert all(torch.equal(again[k], every[k]) for k in every)
    assert torch.equal(db["dbias"], every["dbias"])


def test_backward_empty_sums_are_zero():
    say("linear backward with M = 0, N = 0, K = 0")
    codes, scales, *_ = weights(6, 16, 1)
    got = ops.qlinear_backward(randn((0, 6), 1, torch.bfloat16), codes, scales, x=randn((0, 16), 2, torch.bfloat16),
                               want_dbias=True)
    torch.cuda.synchronize()
    assert got["dx"].shape == (0, 16) and not bool(got["dw"].view(torch.int16).any()) and not bool(got["dbias"].any())
    got = ops.qlinear_backward(randn((3, 0), 1, torch.bfloat16), codes[:0], scales[:0], x=randn((3, 16), 2, torch.bfloat16),
                               want_dbias=True)
    torch.cuda.synchronize()
    assert not bool(got["dx"].view(torch.int16).any()) and got["dw"].shape == (0, 16) and got["dbias"].shape == (0,)
    dy = randn((3, 6), 1, torch.bfloat16)
    got = ops.qlinear_backward(dy, codes[:, :0], scales, x=randn((3, 16), 2, torch.bfloat16)[:, :0], want_dbias=True)
    torch.cuda.synchronize()
    assert got["dx"].shape == (3, 0) and got["dw"].shape == (6, 0)
    assert torch.allclose(got["dbias"], dy.float().sum(0), rtol=1e-6, atol=1e-6)


def test_backward_masked_nan_gives_zero():
    say("linear backward: NaN in a row of X and of dY reaches only unmasked weights")
    codes, scales, w, x, dy, z, mask, keep = grads(64, 48, 40, "none", 0.0, True, 40)
    x2 = x.clone()
    x2[5, 3] = float("nan")
    got = ops.qlinear_backward(dy, codes, scales, x=x2, mask=mask, want_dx=False)["dw"]
    torch.cuda.synchronize()
    col = got[:, 3].float().cpu().numpy()
    assert np.isnan(col[keep[:, 3]]).all() and (col[~keep[:, 3]] == 0).all()
    rest = np.delete(got.float().cpu().numpy(), 3, 1)
    assert np.isfinite(rest).all()


@pytest.mark.parametrize("act,slope", [("none", 0.0), ("relu2", 0.5), ("silu", 0.0)])
def test_backward_against_differences(act, slope):
    """Central differences of L = sum(Y * dY) in 64 bits, h = 2^-12: their own error is at most
    h^2 / 6 times the third derivative (bounded by 2 sum |dY| |a|^3 for these activations on
    |z| < 8) plus rounding 2^-50 L / h; Z reaches backward as bf16, which moves act' by at most
    2 * 2^-8 |z|."""
    say(f"linear backward against differences, {act}")
    M, N, K = 6, 9, 16
    codes, scales, w = weights(N, K, 50)
    x = randn((M, K), 51, torch.bfloat16)
    bias = randn((1, N), 52, torch.float32)[0]
    dy = randn((M, N), 53, torch.bfloat16)
    _, z = ops.qlinear(x, codes, scales, bias=bias, act=act, slope=slope, want_z=True)
    got = ops.qlinear_backward(dy, codes, scales, x=x, z=z, act=act, slope=slope, want_dbias=True,
                               dx_dtype=torch.float32, dw_dtype=torch.float32)
    torch.cuda.synchronize()
    X, W, B, D = f64(x), w.copy(), f64(bias), f64(dy)

    def loss(X, W, B):
        return float((ref.act(X @ W.T + B, act, slope) * D).sum())

    h = 2.0 ** -12
    want = ref.backward(D, f64(z), X, W, act, slope, None, "bf16", "f32", "f32")
    dz_off = 0 if act == "none" else 2 * 2.0 ** -8 * np.abs(X @ W.T + B) * np.abs(D) * 1.1
    zero = np.zeros((M, N)) + dz_off
    slack = {"dx": zero @ np.abs(W), "dw": zero.T @ np.abs(X), "dbias": zero.sum(0)}
    third = h * h / 6 * 2 * np.abs(D).sum() * max(1.0, np.abs(X).max(), np.abs(W).max()) ** 3
    noise = 2.0 ** -50 * np.abs(ref.act(X @ W.T + B, act, slope) * D).sum() / h
    for name, arr in (("dx", X), ("dw", W), ("dbias", B)):
        num = np.zeros_like(arr)
        for i in np.ndindex(arr.shape):
            old = arr[i]
            arr[i] = old + h
            up = loss(X, W, B)
            arr[i] = old - h
            num[i] = (up - loss(X, W, B)) / (2 * h)
            arr[i] = old
        within(got[name], num, want[name][1] + slack[name] + third + noise, name)


def test_streams_and_graph():
    """Forward and backward recorded into one graph on a side stream and replayed between eager work
    on new inputs: every replay equals the eager result."""
    say("linear forward + backward captured and replayed")
    M, N, K = 400, 264, 136
    codes, scales, w = weights(N, K, 60)
    xs = [randn((M, K), 61 + i, torch.bfloat16) for i in range(3)]
    dys = [randn((M, N), 71 + i, torch.bfloat16) for i in range(3)]
    x, dy = xs[0].clone(), dys[0].clone()

    def step(x, dy):
        y, z = ops.qlinear(x, codes, scales, act="silu", want_z=True)
        return [y, z, *ops.qlinear_backward(dy, codes, scales, x=x, z=z, act="silu", want_dbias=True).values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, dy)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(x, dy)
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        dy.copy_(dys[i])
        graph.replay()
        eager = step(xs[i], dys[i])
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a, b)


def test_large_sampled_rows():
    say("linear 16384 x 1584 x 528 forward and backward, sampled")
    M, N, K = 16384, 1584, 528
    codes, scales, w, x, dy, z, mask, keep = grads(M, N, K, "relu2", 0.5, True, 80)
    y, zz = ops.qlinear(x, codes, scales, act="relu2", slope=0.5, want_z=True)
    got = ops.qlinear_backward(dy, codes, scales, x=x, z=z, act="relu2", slope=0.5, mask=mask, want_dbias=True)
    torch.cuda.synchronize()
    rows = np.r_[0:2, 127:129, 255:257, 8000:8002, 16382:16384]
    X, D, Z = f64(x), f64(dy), f64(z)
    zr, ez, yr, ey = ref.forward(X[rows], w, None, "relu2", 0.5)
    within(zz[rows], zr, ez, "z")
    within(y[rows], yr, ey, "y")
    want = ref.backward(D[rows], Z[rows], X[rows], w, "relu2", 0.5)
    within(got["dx"][rows], *want["dx"], "dx")
    cols = np.r_[0:2, 127:129, 800:802, 1582:1584]
    want = ref.backward(D[:, cols], Z[:, cols], X, w[cols], "relu2", 0.5, keep[cols])
    within(got["dw"][cols], *want["dw"], "dw")
    within(got["dbias"][cols], *want["dbias"], "dbias")


def test_contractions_and_strides_past_the_matrix_kernels():
    """Rows of 2^21 elements and more (32-bit byte offsets within a tile end there), and row strides that
    long: against 64-bit products on the device, bounds as in linear_ref."""
    say("linear with K, N or strides of 2^21 and more")
    big = (1 << 21) + 24
    g = torch.Generator(device="cuda").manual_seed(1)

    def rand(*s, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()

    def layer(N, K):
        codes = torch.randint(-31, 32, (N, K), generator=g, device="cuda", dtype=torch.int8)
        scales = torch.rand(N, generator=g, device="cuda").half() * 0.01 + 0.001
        return codes, scales, (codes.float() * scales.float()[:, None]).bfloat16().double()

    def near(got, a, b, L, half_step):
        want, mag = a @ b, a.abs() @ b.abs()
        bound = (L + 1) * ref.U * mag
        bound = bound + half_step * (want.abs() + bound) + 2.0 ** -133
        assert bool(((got.double() - want).abs() <= bound).all())

    for M in (2, 66):                                      # few-token kernel; element-load kernel
        codes, scales, w = layer(3, big)
        x = rand(M, big)
        near(ops.qlinear(x, codes, scales, out_dtype=torch.float32), x.double(), w.t(), big, ref.U)
        del x
    x, dy = rand(3, big), rand(3, 3)
    got = ops.qlinear_backward(dy, codes, scales, x=x, want_dbias=True)
    near(got["dx"], dy.double(), w, 3, 2.0 ** -8)
    near(got["dw"], dy.double().t(), x.double(), 3, 2.0 ** -8)
    codes, scales, w = layer(big, 5)
    x, dy = rand(2, 5), rand(2, big)
    got = ops.qlinear_backward(dy, codes, scales, x=x, want_dbias=True)
    near(got["dx"], dy.double(), w, big, 2.0 ** -8)
    near(got["dw"], dy.double().t(), x.double(), 2, 2.0 ** -8)
    assert torch.allclose(got["dbias"], dy.float().sum(0), rtol=1e-6, atol=0)
    # row strides: X in a buffer of rows 2^21 + 24 apart, 70 rows; codes and dY likewise
    wide = torch.full((70, big), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = wide[:, 8:72]
    x.copy_(rand(70, 64))
    cwide = torch.zeros((40, big), dtype=torch.int8, device="cuda")
    codes, scales, w = layer(40, 64)
    cwide[:, 16:80] = codes
    y = ops.qlinear(x, cwide[:, 16:80], scales, out_dtype=torch.float32)
    near(y, x.double(), w.t(), 64, ref.U)
    dwide = torch.full((70, big), float("nan"), dtype=torch.bfloat16, device="cuda")
    dy = dwide[:, 64:104]
    dy.copy_(rand(70, 40))
    got = ops.qlinear_backward(dy, cwide[:, 16:80], scales, x=x)
    torch.cuda.synchronize()
    near(got["dx"], dy.double(), w, 40, 2.0 ** -8)
    near(got["dw"], dy.double().t(), x.double(), 70, 2.0 ** -8)


@pytest.mark.parametrize("M,N,K", [(40, 96, 4096), (96, 64, 8192), (300, 48, 4160), (640, 4096, 1024), (2048, 1024, 520),
                                   (4096, 1536, 512), (8192, 264, 96)])
def test_every_tile_and_its_parts(M, N, K):
    """Sizes that the plan gives to each tile, from codes and from laid-out weights (K not a multiple of 16), whole
    and in parts: the outputs sampled, in both types."""
    say(f"linear tiles {M}x{N}x{K}")
    codes, scales, w = weights(N, K, M)
    x = randn((M, K), 5, torch.bfloat16)
    r = randn((M, N), 6, torch.float32)
    b = randn((1, N), 7, torch.bfloat16)[0]
    rows = np.unique(np.r_[0:3, M // 2:M // 2 + 3, M - 3:M, np.arange(0, M, max(1, M // 40))])
    for y, res in (("f32", r), ("bf16", None)):
        got, z = ops.qlinear(x, codes, scales, bias=b, act="silu", residual=res, want_z=True, out_dtype=T[y])
        torch.cuda.synchronize()
        zr, ez, yr, ey = ref.forward(f64(x)[rows], w, f64(b), "silu", 0.0, None if res is None else f64(res)[rows], y)
        within(z[rows], zr, ez, "z")
        within(got[rows], yr, ey, "y")
    dy = randn((M, N), 8, torch.bfloat16, std=0.1)
    got = ops.qlinear_backward(dy, codes, scales, x=x, dx_dtype=torch.float32, dw_dtype=torch.float32)
    torch.cuda.synchronize()
    want = ref.backward(f64(dy)[rows], None, f64(x)[rows], w, dx="f32", dw="f32")
    within(got["dx"][rows], *want["dx"], "dx")
    cols = np.unique(np.r_[0:2, N // 2, N - 2:N, np.arange(0, N, max(1, N // 20))])
    want = ref.backward(f64(dy)[:, cols], None, f64(x), w[cols], dx="f32", dw="f32")
    within(got["dw"][cols], *want["dw"], "dw")


@pytest.mark.parametrize("M,N,K", [(3, 40, 128), (40, 24, 200), (96, 64, 1024), (96, 64, 1040), (700, 264, 152), (64, 96, 2048)])
def test_infinite_and_nan_scales(M, N, K):
    """code * infinity is an infinity of the code's sign, NaN for code 0, on every path; a row's neighbours
    are untouched.  Codes and x of one sign, so that no sum mixes infinities."""
    say(f"linear infinite scales {M}x{N}x{K}")
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.randint(1, 32, (N, K), generator=g, device="cuda", dtype=torch.int8)
    codes[5] *= -1
    codes[7, 3] = 0
    scales = torch.full((N,), 0.01, device="cuda", dtype=torch.float16)
    clean = (torch.rand(M, K, generator=g, device="cuda") + 0.5).bfloat16()
    base = ops.qlinear(clean, codes, scales, out_dtype=torch.float32)
    scales[4], scales[5], scales[6], scales[7] = float("inf"), float("inf"), float("nan"), float("inf")
    y = ops.qlinear(clean, codes, scales, out_dtype=torch.float32)
    dx = ops.qlinear_backward(torch.ones(M, N, device="cuda"), codes[:, :16].contiguous(), scales, want_dw=False)["dx"]
    torch.cuda.synchronize()
    assert bool((y[:, 4] == float("inf")).all()) and bool((y[:, 5] == -float("inf")).all())
    assert bool(y[:, 6:8].isnan().all()) and bool(dx.isnan().all())
    rest = [n for n in range(N) if n not in (4, 5, 6, 7)]
    assert torch.equal(y[:, rest], base[:, rest])


@pytest.mark.parametrize("M,N,K,pad", [(1, 7, 40000, 0), (5, 40, 8192, 0), (16, 64, 6176, 3), (33, 20, 8200, 1), (19, 224, 6176, 1),
                                       (2, 100, 4160, 16), (64, 16, 16384, 8)])
@pytest.mark.parametrize("act,y,res", [("none", "f32", None), ("relu2", "bf16", "f32"), ("silu", "f32", "bf16")])
def test_few_tokens_long_rows(M, N, K, pad, act, y, res):
    """Few weight rows of long K go in parts; padding around the rows holds NaN and codes that must not count."""
    say(f"linear few tokens in parts {M}x{N}x{K} pad {pad} {act} {y}")
    codes, scales, w = weights(N, K, M)
    cw = torch.full((N, K + pad), 77, dtype=torch.int8, device="cuda")
    cw[:, :K] = codes
    xw = torch.full((M, K + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    xw[:, :K] = randn((M, K), 5, torch.bfloat16)
    x = xw[:, :K]
    b = randn((1, N), 7, torch.float32)[0]
    r = None if res is None else randn((M, N), 6, T[res])
    got, z = ops.qlinear(x, cw[:, :K], scales, bias=b, act=act, slope=0.5, residual=r, want_z=True, out_dtype=T[y])
    again, _ = ops.qlinear(x, cw[:, :K], scales, bias=b, act=act, slope=0.5, residual=r, want_z=True, out_dtype=T[y])
    torch.cuda.synchronize()
    zr, ez, yr, ey = ref.forward(f64(x), w, f64(b), act, 0.5, None if r is None else f64(r), y)
    within(z, zr, ez, "z")
    within(got, yr, ey, "y")
    assert torch.equal(got, again)


def test_in_place_and_shared_memory():
    """Y over X is refused; Y and X, and Y and Z, as columns of one buffer are not."""
    say("linear shared memory")
    codes, scales, w = weights(64, 64, 2)
    buf = torch.zeros(100, 192, dtype=torch.bfloat16, device="cuda")
    x = buf[:, :64]
    x.copy_(randn((100, 64), 1, torch.bfloat16))
    with pytest.raises(pgq.PgqError):
        ops.qlinear(x, codes, scales, out=x)
    with pytest.raises(pgq.PgqError):
        ops.qlinear(x, codes, scales, out=buf[:, 63:127])
    want = ops.qlinear(x.contiguous(), codes, scales)
    ops.qlinear(x, codes, scales, out=buf[:, 64:128])
    torch.cuda.synchronize()
    assert torch.equal(buf[:, 64:128], want) and not bool(buf[:, 128:].any())


def test_wrapper_refusals():
    say("linear wrappers refuse wrong operands")
    codes, scales, _ = weights(8, 16, 1)
    x = randn((3, 16), 1, torch.bfloat16)
    dy = randn((3, 8), 1, torch.bfloat16)
    for bad in (lambda: ops.qlinear(x.float(), codes, scales), lambda: ops.qlinear(x[:, :8], codes, scales),
                lambda: ops.qlinear(x, codes, scales[:4]), lambda: ops.qlinear(x, codes, scales, residual=x),
                lambda: ops.qlinear(x, codes, scales, bias=scales), lambda: ops.qlinear(x, codes, scales, act="gelu"),
                lambda: ops.qlinear(x, codes, scales, out_dtype=torch.float16),
                lambda: ops.qlinear(x.cpu(), codes, scales),
                lambda: ops.qlinear(x.t().contiguous().t(), codes, scales),
                lambda: ops.qlinear(x[:1].expand(3, 16), codes, scales),
                lambda: ops.qlinear(x, codes, scales, act="relu", slope=float("nan")),
                lambda: ops.qlinear_backward(dy, codes, scales, x=x, act="silu"),
                lambda: ops.qlinear_backward(dy, codes, scales), lambda: ops.qlinear_backward(dy, None, None, x=x),
                lambda: ops.qlinear_backward(dy, codes, scales, x=x, mask=codes),
                lambda: ops.qlinear_backward(dy[:, :4], codes, scales, x=x)):
        with pytest.raises((ValueError, TypeError, KeyError, pgq.PgqError)):
            bad()
