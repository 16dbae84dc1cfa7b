"""The AdamW entry points on the CPU: constants, sizes and argument errors (nothing is enqueued)."""
import ctypes

import numpy as np
import pytest

from tests import adamw_ref as ref

pgq = pytest.importorskip("int6_weight_export_amd.pgq")

FAKE = 0x10000


def tensor(**kw):
    a = dict(w=FAKE, m=FAKE, v=FAKE, m_scale=FAKE, v_scale=FAKE, numel=100, w_dtype=pgq.PGQ_F32, g_dtype=pgq.PGQ_F32,
             lr_scale=1.0)
    a.update(kw)
    return (pgq.pgq_adamw_tensor * 1)(pgq.pgq_adamw_tensor(**a))


def step(t, n=1, bits=32, grad=FAKE, h=True, h_dev=None, ws=None, ws_bytes=0, flags=0):
    g = (ctypes.c_void_p * 1)(grad)
    hy = pgq.pgq_adamw_hyper()
    return pgq.pgq_adamw_step(t, n, bits, g, ctypes.byref(hy) if h else None, h_dev, ws, ws_bytes, flags, None, None)


@pytest.mark.parametrize("kw,bits,want", [
    (dict(numel=-1), 32, pgq.PGQ_ERR_SHAPE), (dict(numel=(1 << 40) + 1), 32, pgq.PGQ_ERR_SHAPE),
    (dict(w_dtype=pgq.PGQ_F16), 32, pgq.PGQ_ERR_DTYPE), (dict(g_dtype=5), 32, pgq.PGQ_ERR_DTYPE),
    (dict(w_dtype=pgq.PGQ_BF16, copy=FAKE), 32, pgq.PGQ_ERR_DTYPE), (dict(lr_scale=float("nan")), 32, pgq.PGQ_ERR_PARAM),
    (dict(weight_decay=float("inf")), 32, pgq.PGQ_ERR_PARAM), (dict(), 16, pgq.PGQ_ERR_PARAM),
    (dict(w=None), 32, pgq.PGQ_ERR_NULL), (dict(m=None), 32, pgq.PGQ_ERR_NULL), (dict(v_scale=None), 8, pgq.PGQ_ERR_NULL),
    (dict(w=FAKE + 2), 32, pgq.PGQ_ERR_ALIGN), (dict(m=FAKE + 2), 32, pgq.PGQ_ERR_ALIGN),
    (dict(copy=FAKE + 1), 32, pgq.PGQ_ERR_ALIGN), (dict(), 32, pgq.PGQ_ERR_WORKSPACE),
    (dict(m=FAKE + 1, m_scale=FAKE + 3), 8, pgq.PGQ_ERR_WORKSPACE),      # codes may sit at any byte
])
def test_step_argument_errors(kw, bits, want):
    assert step(tensor(**kw), bits=bits) == want


def test_other_errors():
    t = tensor()
    assert step(t, n=-1) == pgq.PGQ_ERR_SHAPE
    assert step(None) == pgq.PGQ_ERR_NULL
    assert step(t, h=False) == pgq.PGQ_ERR_NULL
    assert step(t, grad=None) == pgq.PGQ_ERR_NULL
    assert step(t, grad=FAKE + 2) == pgq.PGQ_ERR_ALIGN
    assert step(t, h_dev=FAKE + 2) == pgq.PGQ_ERR_ALIGN
    assert step(t, ws=FAKE, ws_bytes=64) == pgq.PGQ_ERR_WORKSPACE
    assert step(t, ws=FAKE + 4, ws_bytes=1 << 20) == pgq.PGQ_ERR_ALIGN
    assert step(tensor(numel=0, w=None, m=None, v=None), grad=None) == pgq.PGQ_OK
    out = (ctypes.c_void_p * 1)(FAKE)
    none = (ctypes.c_void_p * 1)(None)
    assert pgq.pgq_adamw_decode(t, 1, out, none, None, 0, 0, None, None) == pgq.PGQ_ERR_NULL
    assert pgq.pgq_adamw_decode(t, 1, out, None, None, 0, 0, None, None) == pgq.PGQ_ERR_NULL
    assert pgq.pgq_adamw_decode(t, 1, out, out, None, 0, 0, None, None) == pgq.PGQ_ERR_WORKSPACE
    n = ctypes.c_size_t(0)
    assert pgq.pgq_adamw_workspace(t, 1, None) == pgq.PGQ_ERR_NULL
    assert pgq.pgq_adamw_workspace(t, 1, ctypes.byref(n)) == pgq.PGQ_OK and n.value >= 64
    assert pgq.pgq_adamw_workspace(None, 0, ctypes.byref(n)) == pgq.PGQ_OK


@pytest.mark.parametrize("bad", [dict(lr=-1.0), dict(lr=float("nan")), dict(lr=float("inf")), dict(beta1=1.0),
                                 dict(beta2=-0.1), dict(beta2=float("nan")), dict(eps=-1e-8), dict(step=0)])
def test_hyper_errors(bad):
    a = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1)
    a.update(bad)
    h = pgq.pgq_adamw_hyper()
    assert pgq.pgq_adamw_hyper_at(a["lr"], a["beta1"], a["beta2"], a["eps"], a["step"], 1.0, 0, ctypes.byref(h)) == pgq.PGQ_ERR_PARAM


@pytest.mark.parametrize("step_no", [1, 2, 10, 1000, 10 ** 7])
def test_hyper_constants(step_no):
    h = pgq.pgq_adamw_hyper()
    assert pgq.pgq_adamw_hyper_at(3e-4, 0.9, 0.95, 1e-8, step_no, 0.5, 7, ctypes.byref(h)) == pgq.PGQ_OK
    want = ref.hyper(3e-4, (0.9, 0.95), 1e-8, step_no, 0.5)
    for k, v in want.items():
        assert np.float32(getattr(h, k)) == v, k
    assert h.seed == 7
    assert pgq.pgq_adamw_hyper_at(1e-3, 0.9, 0.9, 1e-8, 1, 1.0, 0, None) == pgq.PGQ_ERR_NULL


def test_reference_codes_hold_their_values():
    """encode/decode of the reference: a value on the grid of its block is kept whatever the random bits, others
    go to a neighbour, up with the right frequency."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(64 * 20) * np.exp(rng.standard_normal(64 * 20) * 3)).astype(np.float32)
    for mant in (3, 4):
        v = np.abs(x) if mant == 4 else x
        c, b = ref.encode(v, rng.integers(0, 65536, len(x)), mant)
        d = ref.decode(c, b, mant)
        c2, b2 = ref.encode(d, rng.integers(0, 65536, len(x)), mant)
        same = ref.scale_bytes(d).repeat(64) == b.repeat(64)
        assert np.array_equal(c2[same], c[same])
        lo, _ = ref.encode(v, np.zeros(len(x), np.int64), mant)
        hi, _ = ref.encode(v, np.full(len(x), 65535), mant)
        assert np.all((c == lo) | (c == hi)) and np.all(hi.astype(int) - lo <= 1)
        step = np.abs(ref.decode(hi, b, mant) - ref.decode(lo, b, mant))
        if mant == 4:               # r below the first code is raised to it: off by less than that code
            step = np.maximum(step, np.where(c == 1, ref.decode(np.ones_like(c), b, 4), 0))
        assert np.all(np.abs(d - v) <= step)


def test_formula_against_an_independent_adamw():
    """The binary32 steps follow torch's AdamW (CPU, 64-bit reference of the same formula)."""
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(1)
    w = rng.standard_normal(500).astype(np.float32) * np.float32(0.1)
    p = torch.nn.Parameter(torch.from_numpy(w.astype(np.float64)))
    opt = torch.optim.AdamW([p], lr=0.01, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    m = v = np.zeros(500, np.float32)
    for s in range(1, 6):
        g = rng.standard_normal(500).astype(np.float32)
        p.grad = torch.from_numpy(g.astype(np.float64))
        opt.step()
        w, m, v, _, ok = ref.step32(w, g, m, v, ref.hyper(0.01, (0.9, 0.95), 1e-8, s), wd=0.1)
        assert ok.all()
    # five steps, each off by at most 32 u of the step (0.01) and of the weight
    assert np.max(np.abs(w - p.detach().numpy())) <= 5 * 32 * 2.0 ** -24 * (0.01 + np.abs(w).max())
