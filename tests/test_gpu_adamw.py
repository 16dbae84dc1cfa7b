"""GPU tests of the AdamW step: bit for bit against the binary32 steps of include/pgq.h, and against
64 bits within bounds derived here."""
import ctypes
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int6_weight_export_amd import ops, pgq  # noqa: E402
from tests import adamw_ref as ref  # noqa: E402
from tests.gpu_util import same_bits  # noqa: E402

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = [1, 3, 63, 64, 65, 255, 256, 257, 1000, 4095, 4096, 4097, 8192, 20011]


def say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def host(t):
    return t.detach().float().cpu().numpy().reshape(-1)


def rand(n, seed, std, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, generator=g) * std).to(dtype).cuda()


def bf16_bits(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().view(torch.int16).numpy()


class Model:
    """The reference beside an ops.AdamW over tensors of the given sizes."""

    def __init__(self, sizes, bits, w="f32", copy=False, lr_scale=1.0, wd=0.01, **kw):
        self.sizes, self.bits = sizes, bits
        self.w = [rand(n, 10 + i, 0.05, T[w]) for i, n in enumerate(sizes)]
        self.copies = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in sizes] if copy else None
        self.lr_scale = lr_scale if isinstance(lr_scale, list) else [lr_scale] * len(sizes)
        self.wd = wd if isinstance(wd, list) else [wd] * len(sizes)
        self.opt = ops.AdamW(self.w, weight_decay=wd, lr_scale=lr_scale, state_bits=bits, copies=self.copies, **kw)
        self.rw = [host(t) for t in self.w]
        self.rm = [np.zeros(n, np.float32) for n in sizes]
        self.rv = [np.zeros(n, np.float32) for n in sizes]
        self.codes = [[np.zeros(n, np.uint8), np.zeros(n, np.uint8), np.zeros((n + 63) // 64, np.uint8),
                       np.zeros((n + 63) // 64, np.uint8)] for n in sizes]

    def step(self, grads, **kw):
        o = self.opt
        o.step(grads, **kw)
        h = ref.hyper(kw.get("lr") or o.lr, o.betas, o.eps, o.step_count, kw.get("grad_scale", 1.0))
        for i, g in enumerate(grads):
            r = None
            if self.bits == 8:
                c = self.codes[i]
                self.rm[i], r = ref.decode(c[0], c[2], 3), ref.decode(c[1], c[3], 4)
            w, m, v, r1, _ = ref.step32(self.rw[i], host(g), self.rm[i], self.rv[i], h, self.lr_scale[i], self.wd[i], r)
            if self.w[i].dtype == torch.bfloat16:
                w = torch.from_numpy(w).bfloat16().float().numpy()
            self.rw[i] = w
            if self.bits == 8:
                um, ur = ref.random16(i, len(w), (o.seed + o.step_count) & 0xFFFFFFFF)
                cm, bm = ref.encode(m, um, 3)
                cr, br = ref.encode(r1, ur, 4)
                self.codes[i] = [cm, cr, bm, br]
            else:
                self.rm[i], self.rv[i] = m, v

    def check(self, what=""):
        torch.cuda.synchronize()
        for i, n in enumerate(self.sizes):
            tag = f"{what} tensor {i} ({n})"
            same_bits(host(self.w[i]), self.rw[i], tag + " w")
            if self.copies:
                same_bits(self.copies[i].view(torch.int16).cpu().numpy(), bf16_bits(self.rw[i]), tag + " copy")
            got = [t.cpu().numpy() for t in self.opt.states[i]]
            want = self.codes[i] if self.bits == 8 else [self.rm[i], self.rv[i]]
            for name, a, b in zip(("m", "v", "m_scale", "v_scale"), got, want):
                same_bits(a, b, f"{tag} {name}")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("w,g,copy", [("f32", "f32", False), ("f32", "bf16", True), ("f32", "f16", False),
                                      ("bf16", "bf16", False), ("bf16", "f32", False)])
def test_steps_bit_for_bit(bits, w, g, copy):
    say(f"adamw {bits} bits w={w} g={g} copy={copy}")
    mod = Model(SIZES, bits, w, copy, lr_scale=[1.0 + 0.25 * (i % 3) for i in range(len(SIZES))],
                wd=[0.1 * (i % 2) for i in range(len(SIZES))], lr=0.01, seed=5)
    for s in range(4):
        mod.step([rand(n, 100 * s + i, 0.02 * (s + 1), T[g]) for i, n in enumerate(SIZES)],
                 **({"lr": 0.002, "grad_scale": 0.5} if s == 2 else {}))
        mod.check(f"step {s + 1}")
    assert int(mod.opt.status.item()) == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_mixed_gradient_types_and_odd_offsets(bits):
    say(f"adamw {bits} bits, mixed types, views at odd offsets")
    sizes = [5000, 4096, 700]
    mod = Model(sizes, bits, lr=0.01)
    for s in range(2):
        for off in (0, 1):
            grads = []
            for i, (n, t) in enumerate(zip(sizes, ("f32", "bf16", "f16"))):
                grads.append(rand(n + off, s * 10 + i, 0.1, T[t])[off:])
            mod.step(grads)
            mod.check(f"step {s} offset {off}")


def test_unaligned_weights_and_states():
    say("adamw, weights and states at odd offsets of one buffer")
    n = 5003
    for bits in (32, 8):
        buf = rand(n + 1, 3, 0.1)
        w = buf[1:]
        if bits == 32:
            st = [(torch.zeros(n + 1, device="cuda")[1:], torch.zeros(n + 1, device="cuda")[1:])]
        else:
            st = [tuple(torch.zeros(k + 1, dtype=torch.uint8, device="cuda")[1:] for k in (n, n, (n + 63) // 64, (n + 63) // 64))]
        first = float(buf[0])
        a, b = w.clone(), None
        o1 = ops.AdamW([w], state_bits=bits, states=st)
        o2 = ops.AdamW([a], state_bits=bits)
        for s in range(3):
            g = rand(n, 50 + s, 0.1)
            o1.step([g])
            o2.step([g])
        torch.cuda.synchronize()
        assert torch.equal(w, a) and float(buf[0]) == first
        for x, y in zip(o1.states[0], o2.states[0]):
            assert torch.equal(x, y)


@pytest.mark.parametrize("bits", [32, 8])
def test_nonfinite_gradients_leave_their_elements(bits):
    say(f"adamw {bits} bits with NaN, infinite and overflowing gradients")
    n = 4500
    mod = Model([n, 64], bits, copy=True)
    mod.step([rand(n, 1, 0.1), rand(64, 2, 0.1)])
    mod.check("finite")
    assert int(mod.opt.status.item()) == 0
    g = rand(n, 3, 0.1)
    g[0], g[70], g[4100], g[4499] = float("nan"), float("inf"), -float("inf"), 1e30
    before = host(mod.w[0])[[0, 70, 4100, 4499]]
    mod.step([g, rand(64, 4, 0.1)])
    mod.check("non-finite")
    assert np.array_equal(host(mod.w[0])[[0, 70, 4100, 4499]], before)
    assert int(mod.opt.status.item()) == pgq.PGQ_DEV_NONFINITE


def test_extreme_magnitudes_in_8_bits():
    """Blocks whose largest value is huge, tiny or subnormal, and blocks with a wide spread: codes as the
    reference's, r never falls to zero."""
    say("adamw 8 bits, extreme magnitudes")
    n = 64 * 12
    mod = Model([n], 8, lr=1e-4)
    for s in range(3):
        g = host(rand(n, 20 + s, 1.0)).copy()
        for b, scale in enumerate([1e18, 1e-18, 1e-30, 1e-38, 1e-42, 0.0, 1.0, 1e10, 1e-10, 1e5]):
            g[64 * b:64 * b + 64] *= scale
        g[640:704] *= 10.0 ** np.linspace(-12, 12, 64)
        mod.step([torch.from_numpy(g.astype(np.float32)).cuda()])
        mod.check(f"step {s}")
    c = mod.codes[0]
    nz = np.abs(g.astype(np.float64)) > 1e-18
    assert (c[1][nz] > 0).all()


def test_decode_states():
    say("adamw decode of 8-bit states")
    sizes = [1, 63, 64, 65, 4096, 9001]
    mod = Model(sizes, 8)
    mod.step([rand(n, 7 + i, 0.1) for i, n in enumerate(sizes)])
    mod.check()
    outs = mod.opt.decode_states()
    odd = [torch.zeros(n + 1, dtype=torch.bfloat16, device="cuda")[1:] for n in sizes]
    mod.opt.decode_states(odd, [torch.empty(n, dtype=torch.bfloat16, device="cuda") for n in sizes])
    torch.cuda.synchronize()
    for i, c in enumerate(mod.codes):
        m, r = ref.decode(c[0], c[2], 3), ref.decode(c[1], c[3], 4)
        same_bits(host(outs[0][i]), m, "m")
        same_bits(host(outs[1][i]), r, "r")
        assert torch.equal(odd[i], outs[0][i])


def test_against_64_bits():
    """One step against 64 bits.  With u = 2^-24: m' and v' have two rounded terms and a sum and constants
    off by u each: 5 u of the terms' magnitudes; the update m' / (root ib2 + eps) ib1 lr is off by at most
    16 u of itself plus m's own error over the same denominator; w' adds 4 u |w|."""
    say("adamw 32 bits against 64 bits")
    n, t = 50000, 7
    w, m, v = rand(n, 1, 0.05), rand(n, 2, 0.01), rand(n, 3, 0.01).square()
    g = rand(n, 4, 0.02)
    w0, m0, v0, g0 = (host(x).astype(np.float64) for x in (w, m, v, g))
    opt = ops.AdamW([w], lr=0.003, weight_decay=0.1, states=[(m, v)], step_count=t - 1)
    opt.step([g], grad_scale=0.75)
    torch.cuda.synchronize()
    rw, rm, rv = ref.step64(w0, g0, m0, v0, 0.003, (0.9, 0.999), 1e-8, t, wd=0.1, grad_scale=0.75)
    u = 2.0 ** -24
    em = 5 * u * (np.abs(0.9 * m0) + np.abs(0.1 * 0.75 * g0))
    ev = 6 * u * (0.999 * v0 + 0.001 * (0.75 * g0) ** 2)
    assert np.all(np.abs(host(m) - rm) <= em) and np.all(np.abs(host(v) - rv) <= ev)
    den = np.sqrt(rv / (1 - 0.999 ** t)) + 1e-8
    upd = 0.003 * np.abs(rm) / (1 - 0.9 ** t) / den
    assert np.all(np.abs(host(w) - rw) <= 16 * u * upd + 0.003 * em / (1 - 0.9 ** t) / den + 4 * u * np.abs(w0))


def test_stochastic_rounding_is_unbiased():
    """A constant gradient: v follows the exact average.  Each element's r^2 after rounding has relative
    standard deviation at most 2 * 2^-5 (r moves by less than one step, 2^-4 of its value or less) for each
    step; over 40 steps the errors add to at most sqrt(40) times that, and the mean over 2^16 elements is
    256 times steadier: 3 sigma below 0.5%.  E[r^2] exceeds E[r]^2 by the variance, below 2^-10 a step and
    so 40 * 2^-10 = 4% in all, which is the drift allowed upward."""
    say("adamw 8 bits, drift of v under stochastic rounding")
    n = 1 << 16
    w = torch.zeros(n, device="cuda")
    opt = ops.AdamW([w], lr=0.0, weight_decay=0.0, betas=(0.9, 0.99), state_bits=8)
    g = torch.full((n,), 0.01, device="cuda")
    for _ in range(40):
        opt.step([g])
    m, r = opt.decode_states()
    torch.cuda.synchronize()
    v, want = float(r[0].double().square().mean()), 1e-4 * (1 - 0.99 ** 40)
    assert want * 0.995 <= v <= want * 1.045
    mean_m, want_m = float(m[0].double().mean()), 0.01 * (1 - 0.9 ** 40)
    assert abs(mean_m - want_m) <= 0.005 * want_m


def test_many_tensors_split_into_several_launches():
    say("adamw over 600 tensors")
    sizes = [(37 * i) % 130 for i in range(600)]          # empty tensors among them
    for bits in (32, 8):
        mod = Model(sizes, bits)
        for s in range(2):
            mod.step([rand(n, i + s, 0.1) for i, n in enumerate(sizes)])
        mod.check()


def test_graph_replay_with_device_hyper():
    say("adamw captured once, replayed with each step's constants")
    sizes = [4096, 700, 3]
    for bits in (32, 8):
        mod, other = Model(sizes, bits, seed=3), Model(sizes, bits, seed=3)
        grads = [torch.zeros(n, device="cuda") for n in sizes]
        mod.opt.decode_states() if bits == 8 else None
        warm = ops.AdamW([torch.zeros(4, device="cuda")])
        warm.step([torch.zeros(4, device="cuda")])
        opt = mod.opt
        if bits == 32:                                     # the upload happens outside the capture
            zero = [torch.zeros(n, device="cuda") for n in sizes]
            keep = [w.clone() for w in mod.w]
            opt.step(zero, lr=0.0)
            opt.step_count = 0
            for w, k in zip(mod.w, keep):
                w.copy_(k)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            opt.step(grads, device_hyper=True)
        for s in range(4):
            new = [rand(n, 30 * s + i, 0.1) for i, n in enumerate(sizes)]
            for a, b in zip(grads, new):
                a.copy_(b)
            opt.load_hyper(lr=0.01 / (s + 1))
            graph.replay()
            other.step(new, lr=0.01 / (s + 1))
            torch.cuda.synchronize()
            other.check(f"eager {s}")
            for a, b in zip(mod.w, other.w):
                assert torch.equal(a, b), s
            for a, b in zip(opt.states, other.opt.states):
                assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_upload_refused_under_capture_and_stale_table_reported():
    say("adamw: first step under capture refused; changed descriptors with a resident table write nothing")
    w = rand(100, 1, 0.1)
    opt = ops.AdamW([w])
    g = rand(100, 2, 0.1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        keep = torch.zeros(1, device="cuda")
        with pytest.raises(pgq.PgqError):
            opt.step([g])
        keep += 1
    assert opt.step_count == 0
    opt.step([g])
    torch.cuda.synchronize()
    before = w.clone()
    opt._arr[0].weight_decay = 0.5
    opt.step([g])
    torch.cuda.synchronize()
    assert torch.equal(w, before) and int(opt.status.item()) == pgq.PGQ_DEV_STALE_TABLE


def test_wrapper_refusals():
    say("adamw wrapper refuses wrong tensors")
    w = rand(100, 1, 0.1)
    opt = ops.AdamW([w])
    for bad in (lambda: ops.AdamW([]), lambda: ops.AdamW([w.half()]), lambda: ops.AdamW([w[::2]]),
                lambda: ops.AdamW([w], state_bits=16), lambda: ops.AdamW([w], lr_scale=[1.0, 2.0]),
                lambda: ops.AdamW([w], states=[(w, w)], state_bits=8), lambda: ops.AdamW([w], copies=[w]),
                lambda: ops.AdamW([w.bfloat16()], copies=[w.bfloat16()]).step([w]),
                lambda: opt.step([]), lambda: opt.step([w[:50]]), lambda: opt.step([w.cpu()]),
                lambda: opt.step([w.int()]), lambda: opt.decode_states(), lambda: opt.step([w], lr=-1.0),
                lambda: opt.step([w], lr=float("nan"))):
        with pytest.raises((ValueError, TypeError, pgq.PgqError)):
            bad()


def test_shared_memory_and_captured_constants_refused():
    say("adamw: the same weight twice, overlapping views, a captured step with host constants")
    w = torch.zeros(1000, device="cuda")
    c = torch.zeros(1000, dtype=torch.bfloat16, device="cuda")
    for weights, copies in (([w, w], None), ([w[:600], w[500:]], None), ([w, w.clone()], [c, c])):
        with pytest.raises(ValueError, match="share"):
            ops.AdamW(weights, copies=copies)
    opt = ops.AdamW([w[:500], w[500:]], lr=0.1)
    grads = [torch.ones(500, device="cuda") for _ in range(2)]
    opt.step(grads)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(pgq.PgqError, match="device_hyper"):
            opt.step(grads)
        opt.step(grads, device_hyper=True)
    assert opt.step_count == 1
    torch.cuda.synchronize()
