"""GPU tests of the global gradient norm, clipping, and the optimizer step that clips on the way.

Bounds.  The squares are exact in 64 bits (48 significant bits) and every addition errs by 2^-53 of its result, so a sum of n
terms of one sign is off by less than n 2^-53 of itself and the norm by half of that; its store to binary32 adds 2^-24.
For the sizes here (below 2^24) that is (1 + 2^-6) 2^-24 of the norm in all; the factor's quotient alike.  The gradients
that clipping leaves are fl32(g * factor) rounded to their type, which the tests form from the factor on the device, bit for
bit."""
import math
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int6_weight_export_amd import ops, pgq  # noqa: E402

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
REL = (1 + 2.0 ** -6) * 2.0 ** -24


def say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def rand(n, seed, std=1.0, t="f32"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, generator=g) * std).to(T[t]).cuda()


def exact_norm(grads):
    return math.sqrt(math.fsum(float((g.double().cpu().numpy().astype(np.longdouble) ** 2).sum()) for g in grads))


def check(grads, max_norm, scale=1.0, gn=None):
    gn = gn or ops.GradNorm(grads)
    norm, factor = gn.norm(max_norm, scale)
    torch.cuda.synchronize()
    want = abs(float(np.float32(scale))) * exact_norm(grads)
    assert abs(float(norm) - want) <= REL * want + 2.0 ** -150, (float(norm), want)
    most = float(np.float32(max_norm))
    f = 1.0 if want <= most else most / want
    if abs(want - most) > 1e-12 * want:
        assert abs(float(factor) - f) <= REL * f + 2.0 ** -150 and (f < 1 or float(factor) == 1.0)
    assert int(gn.status.item()) == 0
    return float(norm), float(factor)


SIZES = [[1], [2], [3, 5], [255], [256, 1], [4095], [4096], [4097], [16383], [16384], [16385], [3 * 16384 + 5, 7], [100003, 1, 64, 0, 31],
         [0], [0, 0, 5], [1 << 20, 3], [(1 << 22) + 13] * 3]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_norm(sizes, t):
    say(f"grad norm {sizes} {t}")
    grads = [rand(n, i + n, 0.01, t) for i, n in enumerate(sizes)]
    check(grads, 1e-3)
    check(grads, 1e9)
    check(grads, float("inf"))


@pytest.mark.parametrize("offset", [1, 2, 3, 5])
@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_unaligned_views_of_one_buffer(offset, t):
    say(f"grad norm and clip at offset {offset} {t}")
    buf = rand(60000, 3, 0.1, t)
    sizes, grads, at = [1, 17, 20000, 333, 16384, 5], [], offset
    for n in sizes:
        grads.append(buf[at:at + n])
        at += n + 1                                         # one element between two tensors that belongs to none
    check(grads, 1.0)
    before = buf.clone()
    gn = ops.GradNorm(grads)
    gn.clip_(1.0)
    torch.cuda.synchronize()
    factor = float(gn.result[1])
    assert factor < 1
    mine = torch.zeros_like(buf, dtype=torch.bool)
    at = offset
    for n in sizes:
        mine[at:at + n] = True
        at += n + 1
    assert torch.equal(buf, torch.where(mine, (before.float() * np.float32(factor)).to(T[t]), before))


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sizes", [[1], [7, 4096], [50000, 1, 0, 16385], [(1 << 21) + 3, 11]], ids=str)
def test_clip(sizes, t):
    say(f"grad clip {sizes} {t}")
    grads = [rand(n, n, 0.5, t) for n in sizes]
    before = [g.clone() for g in grads]
    want = exact_norm(grads)
    gn = ops.GradNorm(grads)
    norm = gn.clip_(1e6)                                    # nothing to clip: nothing written
    torch.cuda.synchronize()
    assert abs(float(norm) - want) <= REL * want and all(torch.equal(a, b) for a, b in zip(grads, before))
    norm = gn.clip_(want / 3)
    torch.cuda.synchronize()
    factor = np.float32(float(gn.result[1]))
    assert abs(float(norm) - want) <= REL * want and abs(float(factor) - 1 / 3) <= 2 * REL
    for a, b in zip(grads, before):
        assert torch.equal(a, (b.float() * torch.tensor(factor)).to(T[t]))
    gn.clip_(0.0)
    torch.cuda.synchronize()
    assert all(not bool(g.any()) for g in grads)
    gn.clip_(0.0)                                           # a norm of 0 is within a bound of 0
    torch.cuda.synchronize()
    assert gn.result.tolist() == [0.0, 1.0] and int(gn.status.item()) == 0


# either side of what one launch takes (8192 pieces of 16 bytes in 128 tensors): the last full one, one more piece, one more tensor
EDGES = [[0], [0, 0, 3], [8], [9], [1, 0, 1023, 4096, 5], [3] * 128, [3] * 129, [0] * 5 + [7] * 127 + [0, 2], [0] * 5 + [7] * 128 + [0, 2],
         [32768], [32767, 1], [32769], [65536], [65535, 9], [65528, 8], [65537], [256] * 128, [257] * 127]


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sizes", EDGES, ids=lambda s: f"{len(s)}x{s[0]}-{sum(s)}")
def test_clip_of_small_lists(sizes, t):
    say(f"grad clip, {len(sizes)} tensors of {sum(sizes)} elements {t}")
    buf = torch.full((sum(sizes) + 3 * len(sizes) + 3,), 9.0).to(T[t]).cuda()      # neighbours that no tensor holds
    mine, grads, at = torch.zeros(buf.numel(), dtype=torch.bool), [], 1
    for n in sizes:
        grads.append(buf[at:at + n])
        mine[at:at + n] = True
        at += n + 3
    buf[mine.cuda()] = rand(sum(sizes), 3, 0.5, t)
    before, want = buf.clone(), exact_norm(grads)
    gn = ops.GradNorm(grads)
    for most, clipped in ((1e6, False), (want / 3, True)):
        norm = gn.clip_(most)
        torch.cuda.synchronize()
        assert abs(float(norm) - want) <= REL * want
        f = float(gn.result[1])
        if not clipped or want == 0:
            assert f == 1.0 and torch.equal(buf, before)
        else:
            assert abs(f - 1 / 3) <= 2 * REL
            assert torch.equal(buf, torch.where(mine.cuda(), (before.float() * torch.tensor(f, device="cuda")).to(T[t]), before))
    assert int(gn.status.item()) == 0


def test_clip_of_small_lists_in_mixed_types_captured():
    say("grad clip of a small list, mixed types, captured and replayed")
    grads = [rand(n, n, 1.0, t) for n, t in ((700, "f32"), (33, "bf16"), (1, "f16"), (4095, "bf16"), (2, "f32"))]
    gn = ops.GradNorm(grads)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gn.clip_(1.5)
    for i in range(4):
        bad = i == 2
        new = [rand(g.numel(), 10 * i + j, 1.0).to(g.dtype) for j, g in enumerate(grads)]
        if bad:
            new[3][4094] = float("nan")
        for g, x in zip(grads, new):
            g.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        f = float(gn.result[1])
        if bad:
            assert math.isnan(f) and int(gn.status.item()) == pgq.PGQ_DEV_NONFINITE
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(grads, new))
            gn.status.zero_()
            continue
        want = exact_norm(new)
        assert abs(float(gn.result[0]) - want) <= REL * want and abs(f - 1.5 / want) <= REL * f
        assert all(torch.equal(a, (b.float() * torch.tensor(f, device="cuda")).to(a.dtype)) for a, b in zip(grads, new))
    assert int(gn.status.item()) == 0


def test_mixed_types_and_many_tensors():
    say("grad norm and clip over 700 tensors of mixed types")
    grads = [rand((37 * i) % 211, i, 0.3, ["f32", "bf16", "f16"][i % 3]) for i in range(700)]
    check(grads, 1.0)
    before = [g.clone() for g in grads]
    gn = ops.GradNorm(grads)
    gn.clip_(1.0)
    torch.cuda.synchronize()
    f = torch.tensor(float(gn.result[1]), dtype=torch.float32)
    assert all(torch.equal(a, (b.float() * f.cuda()).to(a.dtype)) for a, b in zip(grads, before))


def test_magnitudes_whose_squares_leave_binary32():
    say("grad norm of huge and tiny values")
    for v in (1e-38, 1e-30, 1e-42, 1e20, 1e37):
        grads = [torch.full((1000,), v, device="cuda"), torch.full((24,), -v, device="cuda")]
        check(grads, 1.0)
    check([torch.full((1 << 16,), 65504.0, dtype=torch.float16, device="cuda")], 1.0)
    check([rand(1000, 1)], 1.0, scale=1.0 / 65536)
    check([rand(1000, 1)], 1.0, scale=-3.0)


def test_more_than_2_31_elements():
    """Ones: the sum of squares is the number of elements, exact in 64 bits; the last elements are scaled like the first."""
    say("grad norm of 2^31 + 5 bf16 elements")
    n = (1 << 31) + 5
    g = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    gn = ops.GradNorm([g, rand(3, 1)[:0]])
    gn.clip_(math.sqrt(n) / 4)
    torch.cuda.synchronize()
    assert abs(float(gn.result[0]) - math.sqrt(n)) <= REL * math.sqrt(n) and abs(float(gn.result[1]) - 0.25) <= 2.0 ** -25
    assert int((g != 0.25).sum()) == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), "overflow"])
def test_not_finite(bad):
    say(f"grad norm with {bad}")
    grads = [rand(40000, 1), rand(300, 2, t="bf16")]
    if bad == "overflow":
        grads[0].fill_(3e38)
    else:
        grads[0][31234] = bad
    before = [g.clone() for g in grads]
    gn = ops.GradNorm(grads)
    gn.clip_(1.0)
    torch.cuda.synchronize()
    assert int(gn.status.item()) == pgq.PGQ_DEV_NONFINITE
    assert not math.isfinite(float(gn.result[0])) and math.isnan(float(gn.result[1]))
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(grads, before))
    grads[0].fill_(0.0)                                     # the next call is not touched by it
    check(grads, 1e9, gn=None)
    gn.norm(1e9)
    torch.cuda.synchronize()
    assert float(gn.result[1]) == 1.0


def test_same_bits_each_time():
    say("grad norm repeated")
    grads = [rand(n, n) for n in (1 << 20, 12345, 7, 300000)]
    gn, other = ops.GradNorm(grads), ops.GradNorm(grads)
    seen = set()
    for _ in range(20):
        seen.add(tuple(gn.norm(1.0)[i].item() for i in range(2)))
    seen.add(tuple(other.norm(1.0)[i].item() for i in range(2)))
    assert len(seen) == 1


def test_two_streams_at_once():
    say("two norms on two streams")
    a, b = [rand(1 << 21, 1)], [rand(1 << 21, 2, 3.0)]
    ga, gb = ops.GradNorm(a), ops.GradNorm(b)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(sa):
            ga.norm(1.0)
        with torch.cuda.stream(sb):
            gb.norm(1.0)
    torch.cuda.synchronize()
    for g, grads in ((ga, a), (gb, b)):
        want = exact_norm(grads)
        assert abs(float(g.result[0]) - want) <= REL * want


def test_graph_replays():
    say("captured norm and clip, replayed over new gradients")
    grads = [rand(n, n) for n in (5000, 16384 * 3 + 1, 3)]
    gn, eager = ops.GradNorm(grads), None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gn.clip_(2.0)
    for i in range(4):
        new = [rand(g.numel(), 50 * i + j, 0.001 if i == 2 else 1.0) for j, g in enumerate(grads)]
        for g, x in zip(grads, new):
            g.copy_(x)
        graph.replay()
        eager = ops.GradNorm(new)
        eager.clip_(2.0)
        torch.cuda.synchronize()
        assert torch.equal(gn.result, eager.result), i
        assert all(torch.equal(a, b) for a, b in zip(grads, new)), i
        assert (float(gn.result[1]) == 1.0) == (i == 2)


def test_bind_takes_other_tensors():
    say("grad norm bound to other tensors")
    gn = ops.GradNorm([rand(100, 1), rand(7, 2)])
    other = [rand(100, 3, t="bf16"), rand(7, 4)]
    gn.bind(other)
    check(other, 1.0, gn=gn)
    for bad in ([other[0]], [other[1], other[0]], [other[0].cpu(), other[1]], [other[0].int(), other[1]]):
        with pytest.raises((ValueError, TypeError)):
            gn.bind(bad)
    check(other, 1.0, gn=gn)                                # a refused list changes nothing


def test_made_under_other_defaults():
    say("grad norm and optimizer made under another default type and device")
    g = [rand(1000, 1)]
    torch.set_default_dtype(torch.bfloat16)
    torch.set_default_device("cuda")
    try:
        gn, opt = ops.GradNorm(g), ops.AdamW([torch.zeros(1000, dtype=torch.float32)], lr=1e-3)
    finally:
        torch.set_default_device(None)
        torch.set_default_dtype(torch.float32)
    assert gn.result.dtype == torch.float32 and opt.norm_result.dtype == torch.float32
    check(g, 1.0, gn=gn)
    norm = opt.step(g, max_norm=1.0)
    torch.cuda.synchronize()
    assert torch.equal(norm, gn.result[0])


def test_refusals():
    say("grad norm refuses wrong arguments")
    g = rand(100, 1)
    for bad in (lambda: ops.GradNorm([]), lambda: ops.GradNorm([g.cpu()]), lambda: ops.GradNorm([g[::2]]), lambda: ops.GradNorm([g.int()]),
                lambda: ops.GradNorm([g]).norm(-1.0), lambda: ops.GradNorm([g]).norm(float("nan")),
                lambda: ops.GradNorm([g]).norm(1.0, float("inf")), lambda: ops.GradNorm([g, g]).clip_(1.0),
                lambda: ops.GradNorm([g[:60], g[50:]]).clip_(1.0)):
        with pytest.raises((ValueError, TypeError, pgq.PgqError)):
            bad()
    ops.GradNorm([g, g]).norm(1.0)                          # (twice the same tensor counts twice)
    torch.cuda.synchronize()


# ---- the optimizer step that clips -----------------------------------------------------------------------


def optimizer(sizes, bits, seed=1):
    return ops.AdamW([rand(n, seed + i, 0.1) for i, n in enumerate(sizes)], lr=0.01, state_bits=bits, seed=5,
                     copies=[torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in sizes])


def same(a, b):
    torch.cuda.synchronize()
    for x, y in zip(a.weights + a.copies + [t for s in a.states for t in s], b.weights + b.copies + [t for s in b.states for t in s]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1.0, 0.25])
def test_clipped_step_is_the_step_with_the_factor(bits, t, scale):
    say(f"clipped adamw step {bits}-bit states {t} scale {scale}")
    sizes = [4096, 700, 3, 20001]
    a, b = optimizer(sizes, bits), optimizer(sizes, bits)
    for i in range(3):
        grads = [rand(n, 10 * i + j, 0.5, t) for j, n in enumerate(sizes)]
        most = 1e9 if i == 1 else 2.0
        norm = a.step(grads, grad_scale=scale, max_norm=most)
        torch.cuda.synchronize()
        want = scale * exact_norm(grads)
        assert abs(float(norm) - want) <= REL * want
        factor = np.float32(float(a.norm_result[1]))
        assert (factor == 1) == (i == 1) and abs(float(factor) - min(1, most / want)) <= REL
        assert b.step(grads, grad_scale=float(np.float32(scale) * factor)) is None
        same(a, b)
    assert a.step_count == 3 and int(a.status.item()) == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_step_with_a_bad_gradient_changes_nothing(bits):
    say(f"clipped adamw step with a NaN gradient, {bits}-bit states")
    sizes = [500, 20000]
    a, b = optimizer(sizes, bits), optimizer(sizes, bits)
    good = [rand(n, n) for n in sizes]
    a.step(good, max_norm=1.0)
    b.step(good, max_norm=1.0)
    bad = [g.clone() for g in good]
    bad[1][777] = float("nan")
    a.step(bad, max_norm=1.0)
    same(a, b)
    assert int(a.status.item()) == pgq.PGQ_DEV_NONFINITE
    a.step_count = b.step_count
    a.step(good, max_norm=1.0)
    b.step(good, max_norm=1.0)
    same(a, b)


def test_clipped_step_captured():
    say("clipped adamw step captured, constants from the device")
    sizes = [4096, 700, 3]
    for bits in (32, 8):
        a, b = optimizer(sizes, bits), optimizer(sizes, bits)
        grads = [rand(n, n) for n in sizes]
        a.step(grads, max_norm=1.0)
        b.step(grads, max_norm=1.0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norm = a.step(grads, device_hyper=True, max_norm=1.0)
        for i in range(4):
            scale = [1.0, 0.5, 1e-4, 2.0][i]
            for j, g in enumerate(grads):
                g.copy_(rand(g.numel(), 100 * i + j))
            a.load_hyper(lr=0.01 / (i + 1), grad_scale=scale)
            graph.replay()
            want = b.step(grads, lr=0.01 / (i + 1), grad_scale=scale, max_norm=1.0)
            torch.cuda.synchronize()
            assert torch.equal(norm, want)
            same(a, b)


def test_clipped_step_refusals():
    say("clipped adamw step refuses wrong bounds")
    a = optimizer([100], 32)
    g = [rand(100, 1)]
    for bad in (-1.0, float("nan")):
        with pytest.raises(pgq.PgqError):
            a.step(g, max_norm=bad)
    assert a.step_count == 0
    a.step(g, max_norm=float("inf"))
    torch.cuda.synchronize()
    assert a.step_count == 1 and float(a.norm_result[1]) == 1.0
