"""GPU tests of the 4-bit group quantizer and decode, bit for bit against the oracle's row quantizer applied to every
group, and of the linear layer over such weights against the definition in 64 bits (bounds: linear_ref.py; the sum of K
terms below runs as a tree of K - 1 additions, and the multiply-add that brings in a group's scale rounds once, where the
tree's addition would)."""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int6_weight_export_amd import ops, pgq  # noqa: E402
from tests import group4_ref as g4, linear_ref as ref  # noqa: E402
from tests.gpu_util import same_bits  # noqa: E402

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def f64(t):
    return t.detach().double().cpu().numpy()


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def randn(shape, seed, dtype=torch.float32, std=1.0, pad=0, fill=float("nan")):
    """Rows in a wider buffer whose padding is NaN: it must not be read into anything."""
    g = torch.Generator().manual_seed(seed)
    t = torch.full((shape[0], shape[1] + pad), fill)
    t[:, :shape[1]] = torch.randn(shape, generator=g) * std
    return t.to(dtype).cuda()[:, :shape[1]]


def check_quantize(w, group, dq):
    got = ops.quantize_groups(w, group=group, dq_dtype=dq)
    torch.cuda.synchronize()
    codes, scales, values, _ = g4.quantize(w.float().cpu().numpy(), group)
    same_bits(got["codes"].cpu().numpy(), g4.pack(codes), "codes")
    same_bits(bits(got["scales"]), scales, "scales")
    if dq is not None:
        want = torch.from_numpy(values).to(dq)
        same_bits(got["dq"].view(torch.int32 if dq == torch.float32 else torch.int16).cpu().numpy(),
                  want.view(torch.int32 if dq == torch.float32 else torch.int16).numpy(), "dq")
    back = ops.dequant_groups(got["codes"], got["scales"], w.shape[1], group=group)
    torch.cuda.synchronize()
    same_bits(back.cpu().numpy(), values, "decoded")
    half = ops.dequant_groups(got["codes"], got["scales"].view(torch.float16), w.shape[1], group=group, out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    same_bits(bits(half), bits(torch.from_numpy(values).bfloat16()), "decoded to bf16")
    return got


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 8), (2, 31), (5, 32), (4, 33), (7, 64), (2, 65), (3, 100), (9, 127), (6, 128),
                                       (5, 129), (33, 200), (2, 1000), (3, 4096), (300, 257), (1025, 40)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_quantize_shapes(rows, cols, group, t):
    say(f"quantize groups {rows}x{cols} group {group} {t}")
    got = check_quantize(randn((rows, cols), rows + cols, T[t], 0.05), group, {"f32": None, "bf16": torch.bfloat16, "f16": torch.float32}[t])
    assert int(got["status"].item()) == 0


@pytest.mark.parametrize("pad", [1, 2, 3, 8, 13])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [96, 101])
def test_quantize_strided_rows(pad, t, cols):
    say(f"quantize groups strided pad {pad} {t} cols {cols}")
    check_quantize(randn((37, cols), pad, T[t], 0.05, pad=pad), 32, torch.float32)


def test_quantize_hard_values():
    """Ties and their neighbours, zeros, signed zeros, subnormal scales, scales that round to zero, the largest finite scale."""
    say("quantize groups hard values")
    for group in (32, 64, 128):
        rng = np.random.default_rng(group)
        rows = []
        for s in (np.float16(0.01), np.float16(6e-8), np.float16(1.5e-5), np.float16(1.0), np.float16(9000.0)):
            w = (rng.integers(-15, 16, group) * np.float32(0.5)).astype(np.float32) * np.float32(s)
            w[0] = np.float32(7) * np.float32(s)
            rows += [w, np.nextafter(w, np.float32(np.inf)), np.nextafter(w, np.float32(-np.inf))]
        rows += [np.zeros(group, np.float32), np.full(group, -0.0, np.float32), np.full(group, 1e-9, np.float32),
                 np.full(group, 1e-40, np.float32), np.full(group, -65504.0 * 7, np.float32)]
        w = np.stack(rows).astype(np.float32)
        got = check_quantize(torch.from_numpy(w).cuda(), group, torch.float32)
        assert int(got["status"].item()) == 0
        assert not np.signbit(got["dq"].cpu().numpy()[got["dq"].cpu().numpy() == 0]).any()


def test_quantize_status_bits():
    say("quantize groups status")
    w = randn((8, 256), 3, std=0.05)
    for bad, want in ((float("nan"), pgq.PGQ_DEV_NONFINITE), (float("-inf"), pgq.PGQ_DEV_NONFINITE), (65520.0 * 7, pgq.PGQ_DEV_SCALE_OVF)):
        x = w.clone()
        x[5, 200] = bad
        st = ops.new_status()
        got = ops.quantize_groups(x, group=64, status=st)
        torch.cuda.synchronize()
        assert got["status"] is st and int(st.item()) == want
        # the other groups are not touched by it
        codes, scales, _, _ = g4.quantize(w.cpu().numpy(), 64)
        keep = np.ones((8, 4), bool)
        keep[5, 3] = False
        assert np.array_equal(bits(got["scales"])[keep], scales[keep])
        k = np.repeat(keep, 32, axis=1)
        assert np.array_equal(got["codes"].cpu().numpy()[k], g4.pack(codes)[k])


def test_outputs_in_strided_buffers_leave_the_rest():
    say("quantize and decode into strided rows")
    rows, cols, group = 19, 101, 32
    w = randn((rows, cols), 5, std=0.05)
    codes, scales, values, _ = g4.quantize(w.cpu().numpy(), group)
    cb = torch.full((rows, 52 + 5), 0xA5, dtype=torch.uint8, device="cuda")
    sb = torch.full((rows, 4 + 3), 0x1234, dtype=torch.int16, device="cuda")
    db = torch.full((rows, cols + 2), 3.0, device="cuda")
    st = ops.new_status()
    rc = pgq.pgq_quantize_groups(w.data_ptr(), pgq.PGQ_F32, rows, cols, cols, group, cb.data_ptr() + 1, 57, sb.data_ptr() + 2, 7,
                                 db.data_ptr() + 4, pgq.PGQ_F32, cols + 2, st.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == pgq.PGQ_OK
    torch.cuda.synchronize()
    c, s, d = cb.cpu().numpy(), sb.cpu().numpy(), db.cpu().numpy()
    assert np.array_equal(c[:, 1:53], g4.pack(codes)) and (c[:, 0] == 0xA5).all() and (c[:, 53:] == 0xA5).all()
    assert np.array_equal(s[:, 1:5].view(np.uint16), scales) and (s[:, 0] == 0x1234).all() and (s[:, 5:] == 0x1234).all()
    assert np.array_equal(d[:, 1:102], values) and (d[:, 0] == 3).all() and (d[:, 102:] == 3).all()
    for t in ("f32", "bf16"):
        ob = torch.full((rows, cols + 3), 5.0, dtype=T[t], device="cuda")
        ops.dequant_groups(cb[:, 1:53], sb[:, 1:5], cols, group=group, out_dtype=T[t], out=ob[:, 1:cols + 1])
        torch.cuda.synchronize()
        assert torch.equal(ob[:, 1:cols + 1].float().cpu(), torch.from_numpy(values).to(T[t]).float())
        assert bool((ob[:, 0] == 5).all()) and bool((ob[:, cols + 1:] == 5).all())


def test_more_than_2_32_lanes():
    """Rows of one column take a whole group of lanes each: places past 2^32 are right."""
    say("quantize 2^27 + 3 rows of one column")
    rows = (1 << 27) + 3
    w = (torch.arange(rows, dtype=torch.int32, device="cuda") % 1999 - 999).float()[:, None] * 0.125
    got = ops.quantize_groups(w, group=128)
    torch.cuda.synchronize()
    a = w[:, 0].abs()
    s = (a / torch.full_like(a, 7)).half()
    s = torch.where(s == 0, torch.ones_like(s), s)
    assert torch.equal(got["scales"][:, 0], s.view(torch.int16))
    code = torch.where(a == 0, 0, torch.where(w[:, 0] < 0, 15, 7)).to(torch.uint8)
    assert torch.equal(got["codes"][:, 0], code) and not bool(got["codes"][:, 1:].any()) and int(got["status"].item()) == 0


def test_decode_takes_every_code():
    """Bytes that no quantizer writes decode as the layout says: 1000 is +0."""
    say("decode every byte")
    b = np.arange(256, dtype=np.uint8).reshape(8, 32)
    s = np.full((8, 2), 0x3800, np.uint16)
    out = ops.dequant_groups(torch.from_numpy(b).cuda(), torch.from_numpy(s.view(np.int16)).cuda(), 64, group=32)
    torch.cuda.synchronize()
    want = (g4.unpack(b, 64).astype(np.float32) * np.float32(0.5)) + np.float32(0)
    same_bits(out.cpu().numpy(), want, "values")


# ---- the linear layer ---------------------------------------------------------------------------------


def weights(N, K, group, seed, pads=0, padc=0):
    """Device codes (row stride padded by `padc` bytes of ones) and scales (by `pads` NaNs), the values in float64."""
    rng = np.random.default_rng(seed)
    w = (rng.standard_normal((N, max(K, 1))) * 0.05).astype(np.float32)[:, :K]
    if K == 0:
        return torch.empty(N, 0, dtype=torch.uint8, device="cuda"), torch.empty(N, 0, dtype=torch.float16, device="cuda"), np.zeros((N, 0))
    codes, scales, values, _ = g4.quantize(w, group)
    packed = g4.pack(codes)
    if K % 8:                                             # the filling codes of a row's last bytes need not be zero
        rest = np.full((N, packed.shape[1] * 2), 5, np.int8)
        rest[:, :K] = codes
        packed = g4.pack(rest)
    cb = torch.full((N, packed.shape[1] + padc), 255, dtype=torch.uint8)
    cb[:, :packed.shape[1]] = torch.from_numpy(packed)
    sb = torch.full((N, scales.shape[1] + pads), float("nan"), dtype=torch.float16)
    sb[:, :scales.shape[1]] = torch.from_numpy(scales.view(np.float16))
    return cb.cuda()[:, :packed.shape[1]], sb.cuda()[:, :scales.shape[1]], values.astype(np.float64)


def within(got, want, bound, what):
    err = np.abs(f64(got) - want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off; worst {np.nanmax(err / np.maximum(bound, 1e-300)):.3g} bounds"


SHAPES = [(1, 1, 1), (1, 16, 8), (1, 7, 33), (1, 1536, 512), (2, 130, 65), (3, 64, 127), (4, 17, 128), (5, 717, 1031), (8, 33, 129),
          (15, 96, 96), (16, 48, 512), (17, 33, 1040), (31, 257, 100), (32, 40, 264), (33, 96, 32), (48, 130, 260), (63, 129, 72),
          (64, 128, 640), (65, 70, 176), (100, 7, 1000), (130, 131, 257), (1, 16, 8192), (1, 300, 5000), (2, 16, 16392), (20, 24, 4100),
          (64, 16, 2048)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_linear_shapes(M, N, K, group):
    say(f"linear4 {M}x{N}x{K} group {group}")
    codes, scales, w = weights(N, K, group, M + N + K)
    x = randn((M, K), 1, torch.bfloat16)
    bias = randn((1, N), 2)[0]
    for y in ("f32", "bf16"):
        got = ops.qlinear4(x, codes, scales, group=group, bias=bias, act="relu2", slope=0.5, out_dtype=T[y])
        torch.cuda.synchronize()
        _, _, yr, ey = ref.forward(f64(x), w, f64(bias), "relu2", 0.5, y=y)
        within(got, yr, ey, "y")


# sizes that bring every kernel, tile and way of cutting K into use: rows streamed by one, two and four wavefronts with one to four
# slabs each; 16, 32 and 64 rows a workgroup; tokens through LDS; parts of K
KERNELS = [(1, 5, 25), (1, 6, 31), (1, 300, 24), (1, 33, 4101), (1, 70, 6001), (1, 20, 8190), (1, 9, 14001), (1, 70, 30031), (1, 9, 32766), (1, 9, 32770),
           (1, 40, 2048), (1, 100, 4096), (1, 33, 6144), (1, 70, 8192), (1, 20, 16384), (1, 35, 26656), (2, 50, 2048), (2, 90, 4064),
           (2, 40, 8192), (2, 9, 16384), (1, 70000, 64), (1, 66000, 6176), (2, 70000, 32),
           (1, 4100, 520), (3, 4100, 520), (16, 8200, 520), (10, 8100, 1030), (4, 8100, 4500), (9, 16000, 300), (6, 48, 16392), (16, 130, 9000), (20, 4100, 520), (32, 8192, 4000), (25, 14400, 520),
           (16, 30000, 520), (5, 20000, 4500), (16, 9000, 12300), (3, 66000, 1030), (12, 1000, 30000),
           (20, 30000, 520), (32, 20000, 4500), (24, 9000, 12300), (17, 500, 30000), (16, 28672, 2100), (30, 28672, 2100), (16, 8192, 20000), (32, 8192, 20000),
           (30, 48, 16392), (40, 4100, 520), (64, 30000, 300), (33, 30000, 520), (64, 14400, 4100), (50, 4100, 14500), (129, 4100, 4100), (64, 80, 16392), (50, 520, 4100), (64, 8200, 1030), (129, 300, 4100)]


@pytest.mark.parametrize("M,N,K", KERNELS)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_linear_kernels(M, N, K, group):
    say(f"linear4 kernels {M}x{N}x{K} group {group}")
    rng = np.random.default_rng(M + N + K)
    code = rng.integers(-7, 8, (N, K)).astype(np.int8)
    scale = (rng.random((N, -(-K // group))) * 0.02).astype(np.float16)
    x = randn((M, K), 1, torch.bfloat16)
    r = randn((M, N), 2)
    got = ops.qlinear4(x, torch.from_numpy(g4_pack_fast(code)).cuda(), torch.from_numpy(scale).cuda(), group=group, residual=r,
                       out_dtype=torch.float32)
    torch.cuda.synchronize()
    # (in 64 bits on the GPU: the largest of these have 10^9 products)
    w = torch.from_numpy(code).cuda().double() * torch.from_numpy(scale).cuda().double().repeat_interleave(group, 1)[:, :K]
    z, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    want = z + r.double()
    # (K - 1 additions and a scale's rounding, the residual's addition, the store: linear_ref.forward's terms)
    bound = K * ref.U * mag
    bound = bound + 2 * ref.U * (want.abs() + bound) + ref.TINY["f32"]
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("act,slope", [("none", 0.0), ("relu", 0.0), ("relu", 0.25), ("relu2", 0.0), ("relu2", -0.5), ("silu", 0.0)])
@pytest.mark.parametrize("M", [1, 20, 64])
@pytest.mark.parametrize("y,res,bias", [("bf16", "", ""), ("f32", "f32", "bf16"), ("bf16", "bf16", "f32"), ("f32", "bf16", "f32"),
                                        ("bf16", "f32", "")])
def test_linear_epilogues(act, slope, M, y, res, bias):
    say(f"linear4 epilogue {act} {slope} M={M} y={y} residual={res} bias={bias}")
    N, K = 136, 208
    codes, scales, w = weights(N, K, 64, 5)
    x = randn((M, K), 3, torch.bfloat16, std=4.0)
    b = randn((1, N), 4, T[bias])[0] if bias else None
    r = randn((M, N), 6, T[res], std=2.0) if res else None
    got = ops.qlinear4(x, codes, scales, group=64, bias=b, act=act, slope=slope, residual=r, out_dtype=T[y])
    torch.cuda.synchronize()
    _, _, yr, ey = ref.forward(f64(x), w, None if b is None else f64(b), act, slope, None if r is None else f64(r), y)
    within(got, yr, ey, "y")


@pytest.mark.parametrize("M", [1, 3, 50])
@pytest.mark.parametrize("padx,padc,pads", [(8, 16, 8), (1, 3, 1), (2, 4, 2), (0, 5, 0), (3, 0, 3)])
@pytest.mark.parametrize("K", [256, 101, 8])
@pytest.mark.parametrize("group", [32, 128])
def test_linear_strided_views_write_nothing_else(M, padx, padc, pads, K, group):
    say(f"linear4 strided M={M} K={K} padx={padx} padc={padc} pads={pads} group {group}")
    N = 150
    codes, scales, w = weights(N, K, group, 7, pads, padc)
    x = randn((M, K), 8, torch.bfloat16, pad=padx)
    for y, off, more in (("f32", 1, 3), ("bf16", 1, 2), ("bf16", 0, 8)):
        buf = torch.full((M, N + more), 7.0, dtype=T[y], device="cuda")
        ops.qlinear4(x, codes, scales, group=group, act="relu", slope=0.1, out=buf[:, off:off + N], out_dtype=T[y])
        torch.cuda.synchronize()
        _, _, yr, ey = ref.forward(f64(x), w, None, "relu", 0.1, y=y)
        within(buf[:, off:off + N], yr, ey, "y")
        assert bool((buf[:, :off] == 7.0).all()) and bool((buf[:, off + N:] == 7.0).all())


@pytest.mark.parametrize("offset", [1, 2, 4, 6])
def test_linear_operands_at_odd_addresses(offset):
    say(f"linear4 operands {offset} elements into their buffers")
    M, N, K, group = 3, 40, 512, 128
    codes, scales, w = weights(N, K, group, 11)
    cb = torch.zeros(codes.numel() + offset, dtype=torch.uint8, device="cuda")
    cb[offset:] = codes.reshape(-1)
    sb = torch.zeros(scales.numel() + offset, dtype=torch.float16, device="cuda")
    sb[offset:] = scales.reshape(-1)
    x = randn((M, K), 12, torch.bfloat16)
    xb = torch.zeros(x.numel() + offset, dtype=torch.bfloat16, device="cuda")
    xb[offset:] = x.reshape(-1)
    got = ops.qlinear4(xb[offset:].view(M, K), cb[offset:].view(N, -1), sb[offset:].view(N, -1), group=group, out_dtype=torch.float32)
    torch.cuda.synchronize()
    _, _, yr, ey = ref.forward(f64(x), w, None, "none", 0.0, y="f32")
    within(got, yr, ey, "y")


@pytest.mark.parametrize("M", [1, 2, 40, 70])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_linear_residual_in_place(M, t):
    say(f"linear4 into its own residual M={M} {t}")
    codes, scales, w = weights(200, 64, 32, 9)
    x, r = randn((M, 64), 10, torch.bfloat16), randn((M, 200), 11, T[t])
    r0 = f64(r)
    got = ops.qlinear4(x, codes, scales, group=32, residual=r, out=r, out_dtype=T[t])
    torch.cuda.synchronize()
    assert got is r
    _, _, yr, ey = ref.forward(f64(x), w, None, "none", 0.0, r0, t)
    within(r, yr, ey, "y")


@pytest.mark.parametrize("M", [5, 16, 27, 40, 64, 90])
@pytest.mark.parametrize("K", [264, 512, 301])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_linear_wide_layers(M, K, group):
    """Layers so wide that the tokens go through LDS: strided operands, every epilogue argument, Y between other columns."""
    say(f"linear4 wide M={M} K={K} group {group}")
    N = 6000
    codes, scales, w = weights(N, K, group, 41, 3, 5)
    x, b, r = randn((M, K), 42, torch.bfloat16, pad=3), randn((1, N), 43)[0], randn((M, N), 44, torch.bfloat16, pad=1)
    for y in ("f32", "bf16"):
        buf = torch.full((M, N + 3), 7.0, dtype=T[y], device="cuda")
        ops.qlinear4(x, codes, scales, group=group, bias=b, act="silu", residual=r, out=buf[:, 1:1 + N], out_dtype=T[y])
        torch.cuda.synchronize()
        _, _, yr, ey = ref.forward(f64(x), w, f64(b), "silu", 0.0, f64(r), y)
        within(buf[:, 1:1 + N], yr, ey, "y")
        assert bool((buf[:, :1] == 7.0).all()) and bool((buf[:, 1 + N:] == 7.0).all())


@pytest.mark.parametrize("M", [5, 16, 27, 40, 64])
@pytest.mark.parametrize("K", [512, 330])
def test_linear_wide_layers_infinities_and_nan(M, K):
    """An infinite token value, a NaN and a scale that is not finite stay in their token's and output's elements."""
    say(f"linear4 wide infinities M={M} K={K}")
    N, group = 6000, 64
    codes, scales, w = weights(N, K, group, 45)
    x = randn((M, K), 46, torch.bfloat16)
    clean = ops.qlinear4(x, codes, scales, group=group, out_dtype=torch.float32)
    x[1, 100], x[M - 1, 7] = float("inf"), float("nan")
    got = ops.qlinear4(x, codes, scales, group=group, out_dtype=torch.float32)
    torch.cuda.synchronize()
    rows = [m for m in range(M) if m not in (1, M - 1)]
    v = torch.from_numpy(w[:, 100])
    inf = got[1].cpu()
    assert torch.equal(got[rows], clean[rows]) and bool(torch.isnan(got[M - 1]).all())
    assert bool(torch.isnan(inf[v == 0]).all()) and bool((inf[v > 0] == float("inf")).all()) and bool((inf[v < 0] == float("-inf")).all())
    s = scales.clone()
    s[3009, scales.shape[1] - 1] = float("inf")
    got = ops.qlinear4(randn((M, K), 46, torch.bfloat16), codes, s, group=group, out_dtype=torch.float32)
    torch.cuda.synchronize()
    cols = [n for n in range(N) if n != 3009]
    assert torch.equal(got[:, cols], clean[:, cols]) and not bool(torch.isfinite(got[:, 3009]).any())


def test_linear_empty_and_k_zero():
    say("linear4 M = 0, N = 0, K = 0")
    codes, scales, _ = weights(5, 16, 32, 1)
    assert ops.qlinear4(randn((0, 16), 1, torch.bfloat16), codes, scales, group=32).shape == (0, 5)
    assert ops.qlinear4(randn((3, 16), 1, torch.bfloat16), codes[:0], scales[:0], group=32).shape == (3, 0)
    codes, scales, _ = weights(5, 0, 32, 1)
    b = randn((1, 5), 2)[0]
    for M in (1, 3, 100):
        r = randn((M, 5), 3)
        y = ops.qlinear4(torch.empty(M, 0, dtype=torch.bfloat16, device="cuda"), codes, scales, group=32, bias=b, act="relu", slope=0.5,
                         residual=r, out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert torch.equal(y, torch.where(b > 0, b, b * 0.5) + r)
    assert ops.dequant_groups(torch.empty(3, 0, dtype=torch.uint8, device="cuda"), torch.empty(3, 0, dtype=torch.int16, device="cuda"), 0,
                              group=32).shape == (3, 0)
    got = ops.quantize_groups(torch.empty(0, 40, device="cuda"), group=32)
    assert got["codes"].shape == (0, 20) and got["scales"].shape == (0, 2)


@pytest.mark.parametrize("M,K,group", [(1, 4096, 128), (3, 1000, 32), (16, 8192, 64), (64, 2048, 128), (100, 512, 32)])
def test_linear_sums_of_whole_numbers_are_exact(M, K, group):
    """Tokens and scales that are small powers of two and whole numbers: every sum is a whole number below 2^24, so any
    order gives the same fp32, equal to the last bit."""
    say(f"linear4 exact M={M} K={K} group {group}")
    rng = np.random.default_rng(K)
    N = 50
    codes = rng.integers(-7, 8, (N, K)).astype(np.int8)
    scales = (2.0 ** rng.integers(0, 4, (N, -(-K // group)))).astype(np.float16)
    x = rng.integers(-16, 17, (M, K)).astype(np.float32)
    got = ops.qlinear4(torch.from_numpy(x).bfloat16().cuda(), torch.from_numpy(g4.pack(codes)).cuda(), torch.from_numpy(scales).cuda(),
                       group=group, out_dtype=torch.float32)
    torch.cuda.synchronize()
    want = x.astype(np.float64) @ g4.values(codes, scales.view(np.uint16), group).T
    assert np.abs(want).max() < 2 ** 24
    assert np.array_equal(got.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("M,K", [(1, 512), (2, 512), (5, 512), (20, 501), (40, 512), (64, 4096)])
@pytest.mark.parametrize("e", [-130, -124])
def test_linear_subnormal_tokens(M, K, e):
    """Tokens 2^e times whole numbers, below binary32's normal range, with scales of 1; then larger ones with scales of 2^-18 to
    2^-15, which are subnormal in fp16.  Every sum is a power of two times a whole number below 2^20 and a binary32 value, so
    equal to the last bit, unless a multiplication takes subnormal numbers for zeros."""
    say(f"linear4 subnormal tokens M={M} K={K} 2^{e}")
    rng = np.random.default_rng(K + M)
    N = 40
    codes = rng.integers(-7, 8, (N, K)).astype(np.int8)
    scales = (2.0 ** rng.integers(-18, -14, (N, -(-K // 64)))).astype(np.float16)
    x = rng.integers(-3, 4, (M, K)) * 2.0 ** e
    xt = torch.from_numpy(x.astype(np.float32)).bfloat16()
    assert np.array_equal(xt.double().numpy(), x)
    ones = np.ones_like(scales)
    for s, up in ((ones, 1.0), (scales, 2.0 ** 30)):
        got = ops.qlinear4((xt.double() * up).bfloat16().cuda(), torch.from_numpy(g4.pack(codes)).cuda(), torch.from_numpy(s).cuda(),
                           group=64, out_dtype=torch.float32)
        torch.cuda.synchronize()
        want = (x * up) @ g4.values(codes, s.view(np.uint16), 64).T
        assert np.array_equal(got.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("M,K", [(1, 320), (2, 320), (1, 4096), (5, 320), (20, 320), (40, 320), (40, 4096), (70, 330)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_linear_infinities_and_nan(M, K, group):
    """An infinite token value gives the formula's infinity or NaN in its own row and leaves the other rows alone; so does a
    bad scale in its own column."""
    say(f"linear4 infinities M={M} K={K} group {group}")
    N = 40
    codes, scales, w = weights(N, K, group, 21)
    x = randn((M, K), 22, torch.bfloat16)
    clean = ops.qlinear4(x, codes, scales, group=group, out_dtype=torch.float32)
    bad, nan = M // 2, M - 1 if M > 1 else None
    x[bad, 100] = float("inf")
    if nan is not None:
        x[nan, 7] = float("nan")
    got = ops.qlinear4(x, codes, scales, group=group, out_dtype=torch.float32)
    torch.cuda.synchronize()
    rows = [m for m in range(M) if m not in (bad, nan)]
    assert torch.equal(got[rows], clean[rows])
    assert nan is None or bool(torch.isnan(got[nan]).all())
    if bad != nan:
        v = torch.from_numpy(w[:, 100])
        inf = got[bad].cpu()
        assert bool(torch.isnan(inf[v == 0]).all()) and bool((inf[v > 0] == float("inf")).all()) and bool((inf[v < 0] == float("-inf")).all())
    x = randn((M, K), 22, torch.bfloat16)
    for value in (float("inf"), float("nan")):
        s = scales.clone()
        s[9, scales.shape[1] - 1] = value
        got = ops.qlinear4(x, codes, s, group=group, out_dtype=torch.float32)
        torch.cuda.synchronize()
        cols = [n for n in range(N) if n != 9]
        assert torch.equal(got[:, cols], clean[:, cols]) and not bool(torch.isfinite(got[:, 9]).any())


@pytest.mark.parametrize("M", [1, 2, 16, 33, 64])
def test_linear_same_bits_each_time_and_on_two_streams(M):
    say(f"linear4 repeated and on two streams M={M}")
    N, K, group = 400, 4096, 128
    codes, scales, _ = weights(N, K, group, 31)
    x = randn((M, K), 32, torch.bfloat16)
    first = ops.qlinear4(x, codes, scales, group=group)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(6):
        with torch.cuda.stream(s[i % 2]):
            outs.append(ops.qlinear4(x, codes, scales, group=group))
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)


@pytest.mark.parametrize("M,K", [(1, 1024), (4, 1000), (4, 16384), (30, 1000), (64, 8192)])
def test_captured_calls_replay(M, K):
    say(f"quantize, decode and linear4 in a graph, M={M} K={K}")
    N, group = 200, 64
    w, x = randn((N, K), 41, std=0.05), randn((M, K), 42, torch.bfloat16)
    w2, x2 = randn((N, K), 43, std=0.05), randn((M, K), 44, torch.bfloat16)
    st = ops.new_status()
    torch.cuda.synchronize()

    def chain():
        q = ops.quantize_groups(w, group=group, status=st)
        return ops.dequant_groups(q["codes"], q["scales"], K, group=group), ops.qlinear4(x, q["codes"], q["scales"], group=group)

    chain()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dq, y = chain()
    for i in range(4):
        w.copy_(w2 * (i + 1))
        x.copy_(x2 * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        a, b = chain()
        torch.cuda.synchronize()
        assert torch.equal(a, dq) and torch.equal(b, y), i
    assert int(st.item()) == 0


def test_long_rows():
    """Two rows of 2^21 + 9 columns of whole numbers: every sum, equal to the last bit."""
    say("linear4 K = 2^21 + 9")
    K, group = (1 << 21) + 9, 128
    rng = np.random.default_rng(1)
    codes = rng.integers(-7, 8, (2, K)).astype(np.int8)
    scales = np.full((2, -(-K // group)), 0.25, np.float16)
    x = rng.integers(-1, 2, (1, K)).astype(np.float32)
    packed = torch.from_numpy(g4_pack_fast(codes)).cuda()
    got = ops.qlinear4(torch.from_numpy(x).bfloat16().cuda(), packed, torch.from_numpy(scales).cuda(), group=group, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy().astype(np.float64), x.astype(np.float64) @ (codes.astype(np.float64) * 0.25).T)


def g4_pack_fast(codes):
    rows, cols = codes.shape
    full = np.zeros((rows, -(-cols // 8) * 8), np.int8)
    full[:, :cols] = codes
    nib = np.where(full < 0, 8 - full, full).astype(np.uint8).reshape(rows, -1, 2, 4)
    return (nib[:, :, 0] | nib[:, :, 1] << 4).reshape(rows, -1)


def test_codes_past_two_gib():
    """A matrix whose codes and values lie past 2^31 bytes from their first: the last rows are right."""
    say("quantize, decode and linear4 past 2^31 bytes")
    rows, cols, group = 65536 + 3, 65536 + 32, 128
    w = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = randn((3, cols), 51, torch.bfloat16, 0.05)
    w[-3:] = tail
    got = ops.quantize_groups(w, group=group)
    codes, scales, values, _ = g4.quantize(tail.float().cpu().numpy(), group)
    torch.cuda.synchronize()
    assert got["codes"].numel() > 1 << 31
    assert np.array_equal(got["codes"][-3:].cpu().numpy(), g4_pack_fast(codes)) and np.array_equal(bits(got["scales"][-3:]), scales)
    assert not bool(got["codes"][:-3].any())
    x = randn((1, cols), 52, torch.bfloat16)
    y = ops.qlinear4(x, got["codes"], got["scales"], group=group, out_dtype=torch.float32)
    torch.cuda.synchronize()
    _, _, yr, ey = ref.forward(f64(x), values.astype(np.float64), None, "none", 0.0, y="f32")
    within(y[:, -3:], yr, ey, "y")
    assert not bool(y[:, :-3].any())
    ops.dequant_groups(got["codes"], got["scales"], cols, group=group, out_dtype=torch.bfloat16, out=w)
    torch.cuda.synchronize()
    assert torch.equal(w[-3:].float().cpu(), torch.from_numpy(values).bfloat16().float()) and not bool(w[:-3].any())


def test_wrapper_refusals():
    say("group wrappers refuse wrong arguments")
    w = randn((8, 64), 1)
    q = ops.quantize_groups(w, group=32)
    c, s = q["codes"], q["scales"]
    x = randn((2, 64), 2, torch.bfloat16)
    for bad in (lambda: ops.quantize_groups(w[0]), lambda: ops.quantize_groups(w.t()), lambda: ops.quantize_groups(w, group=16),
                lambda: ops.quantize_groups(w.int()), lambda: ops.quantize_groups(w.cpu()), lambda: ops.quantize_groups(w, dq_dtype=torch.float16),
                lambda: ops.quantize_groups(w, status=torch.zeros(1, device="cuda")),
                lambda: ops.dequant_groups(c, s, 64, group=64), lambda: ops.dequant_groups(c, s, 65, group=32),
                lambda: ops.dequant_groups(c.view(torch.int8), s, 64, group=32), lambda: ops.dequant_groups(c, s.float(), 64, group=32),
                lambda: ops.dequant_groups(c, s, 64, group=32, out_dtype=torch.float16), lambda: ops.dequant_groups(c, s.cpu(), 64, group=32),
                lambda: ops.dequant_groups(c, s, 64, group=32, out=torch.empty(8, 65, device="cuda")),
                lambda: ops.qlinear4(x.float(), c, s, group=32), lambda: ops.qlinear4(x[:, :56], c, s, group=32),
                lambda: ops.qlinear4(x, c, s, group=64), lambda: ops.qlinear4(x, c[:, :-4], s, group=32), lambda: ops.qlinear4(x, c.cpu(), s, group=32),
                lambda: ops.qlinear4(x, c, s, group=32, act="gelu"), lambda: ops.qlinear4(x, c, s, group=32, bias=w[0, :7]),
                lambda: ops.qlinear4(x, c, s, group=32, out_dtype=torch.float16), lambda: ops.qlinear4(x[0], c, s, group=32),
                lambda: ops.qlinear4(x, c, s, group=32, residual=x[:, :8].float(), out=x[:, :8])):
        with pytest.raises((ValueError, TypeError, KeyError, pgq.PgqError)):
            bad()
    with pytest.warns(UserWarning, match="records no gradient"):
        ops.qlinear4(x.clone().requires_grad_(), c, s, group=32)
    torch.cuda.synchronize()
