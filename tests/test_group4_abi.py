"""The 4-bit group entry points' C ABI on the CPU: argument errors come back before anything is enqueued, and the
reference that the GPU tests compare with agrees with the definition."""
import ctypes

import numpy as np
import pytest

from tests import group4_ref as ref

pgq = pytest.importorskip("int6_weight_export_amd.pgq")

FAKE = 0x10000      # aligned, never dereferenced: every call here fails its checks or has nothing to do


def quantize(**kw):
    a = dict(w=FAKE, w_dtype=pgq.PGQ_F32, rows=4, cols=40, ld=40, group=32, codes=FAKE + 0x1000, ldc=20, scales=FAKE + 0x2000, lds=2,
             dq=None, dq_dtype=pgq.PGQ_F32, ldq=40, dev_status=None, stream=None)
    a.update(kw)
    return pgq.pgq_quantize_groups(**a)


def dequant(**kw):
    a = dict(codes=FAKE, ldc=20, scales=FAKE + 0x1000, lds=2, rows=4, cols=40, group=32, out=FAKE + 0x2000, out_dtype=pgq.PGQ_F32,
             ldo=40, stream=None)
    a.update(kw)
    return pgq.pgq_dequant_groups(**a)


def linear(**kw):
    a = dict(M=2, N=8, K=40, x=FAKE, ldx=40, codes=FAKE + 0x1000, ldc=20, scales=FAKE + 0x2000, lds=2, y=FAKE + 0x3000, ldy=8,
             y_dtype=pgq.PGQ_BF16, act=pgq.PGQ_ACT_NONE, group=32)
    a.update(kw)
    return pgq.pgq_linear4_fwd(**a)


@pytest.mark.parametrize("args,want", [
    (dict(rows=-1), pgq.PGQ_ERR_SHAPE), (dict(cols=-1), pgq.PGQ_ERR_SHAPE), (dict(ld=39), pgq.PGQ_ERR_SHAPE),
    (dict(ldc=19), pgq.PGQ_ERR_SHAPE), (dict(lds=1), pgq.PGQ_ERR_SHAPE), (dict(dq=FAKE + 0x3000, ldq=39), pgq.PGQ_ERR_SHAPE),
    (dict(cols=1 << 31, ld=1 << 31, ldc=1 << 30, lds=1 << 26), pgq.PGQ_ERR_SHAPE),
    (dict(group=16), pgq.PGQ_ERR_PARAM), (dict(group=0), pgq.PGQ_ERR_PARAM), (dict(group=256), pgq.PGQ_ERR_PARAM),
    (dict(w_dtype=3), pgq.PGQ_ERR_DTYPE), (dict(dq=FAKE + 0x3000, dq_dtype=pgq.PGQ_F16), pgq.PGQ_ERR_DTYPE),
    (dict(w=None), pgq.PGQ_ERR_NULL), (dict(codes=None), pgq.PGQ_ERR_NULL), (dict(scales=None), pgq.PGQ_ERR_NULL),
    (dict(w=FAKE + 2), pgq.PGQ_ERR_ALIGN), (dict(w=FAKE + 1, w_dtype=pgq.PGQ_BF16), pgq.PGQ_ERR_ALIGN),
    (dict(scales=FAKE + 0x2001), pgq.PGQ_ERR_ALIGN), (dict(dq=FAKE + 0x3002), pgq.PGQ_ERR_ALIGN),
    (dict(codes=FAKE), pgq.PGQ_ERR_PARAM), (dict(dq=FAKE), pgq.PGQ_ERR_PARAM), (dict(scales=FAKE + 0x1000), pgq.PGQ_ERR_PARAM),
    (dict(rows=1 << 30, cols=1 << 10, ld=1 << 10, ldc=1 << 9, lds=1 << 5, codes=FAKE + (1 << 50), scales=FAKE + (1 << 51)),
     pgq.PGQ_ERR_SHAPE),                                      # 2^37 threads
    (dict(rows=1 << 29, cols=1, ld=1, group=128, ldc=4, lds=1, codes=1 << 40, scales=1 << 41), pgq.PGQ_ERR_SHAPE),   # a group a row: 2^33 threads
    (dict(rows=0), pgq.PGQ_OK), (dict(cols=0, ldc=0, lds=0), pgq.PGQ_OK), (dict(rows=0, w=None, codes=None, scales=None), pgq.PGQ_OK),
])
def test_quantize_argument_errors(args, want):
    assert quantize(**args) == want


@pytest.mark.parametrize("args,want", [
    (dict(rows=-1), pgq.PGQ_ERR_SHAPE), (dict(ldc=19), pgq.PGQ_ERR_SHAPE), (dict(lds=1), pgq.PGQ_ERR_SHAPE),
    (dict(ldo=39), pgq.PGQ_ERR_SHAPE), (dict(group=48), pgq.PGQ_ERR_PARAM), (dict(out_dtype=pgq.PGQ_F16), pgq.PGQ_ERR_DTYPE),
    (dict(codes=None), pgq.PGQ_ERR_NULL), (dict(out=None), pgq.PGQ_ERR_NULL), (dict(scales=FAKE + 0x1001), pgq.PGQ_ERR_ALIGN),
    (dict(out=FAKE + 0x2002), pgq.PGQ_ERR_ALIGN), (dict(out=FAKE), pgq.PGQ_ERR_PARAM), (dict(rows=0), pgq.PGQ_OK),
])
def test_dequant_argument_errors(args, want):
    assert dequant(**args) == want


@pytest.mark.parametrize("args,want", [
    (dict(M=-1), pgq.PGQ_ERR_SHAPE), (dict(ldx=39), pgq.PGQ_ERR_SHAPE), (dict(ldc=19), pgq.PGQ_ERR_SHAPE),
    (dict(lds=1), pgq.PGQ_ERR_SHAPE), (dict(ldy=7), pgq.PGQ_ERR_SHAPE), (dict(N=1 << 31, ldy=1 << 31), pgq.PGQ_ERR_SHAPE),
    (dict(residual=FAKE + 0x4000, ldr=7, residual_dtype=pgq.PGQ_F32), pgq.PGQ_ERR_SHAPE),
    (dict(group=0), pgq.PGQ_ERR_PARAM), (dict(group=96), pgq.PGQ_ERR_PARAM), (dict(act=4), pgq.PGQ_ERR_PARAM),
    (dict(act=pgq.PGQ_ACT_RELU, slope=float("nan")), pgq.PGQ_ERR_PARAM), (dict(y_dtype=pgq.PGQ_F16), pgq.PGQ_ERR_DTYPE),
    (dict(bias=FAKE, bias_dtype=7), pgq.PGQ_ERR_DTYPE), (dict(residual=FAKE + 0x4000, ldr=8, residual_dtype=7), pgq.PGQ_ERR_DTYPE),
    (dict(x=None), pgq.PGQ_ERR_NULL), (dict(codes=None), pgq.PGQ_ERR_NULL), (dict(scales=None), pgq.PGQ_ERR_NULL),
    (dict(y=None), pgq.PGQ_ERR_NULL), (dict(x=FAKE + 1), pgq.PGQ_ERR_ALIGN), (dict(y=FAKE + 0x3001), pgq.PGQ_ERR_ALIGN),
    (dict(scales=FAKE + 0x2001), pgq.PGQ_ERR_ALIGN), (dict(bias=FAKE + 0x4002, bias_dtype=pgq.PGQ_F32), pgq.PGQ_ERR_ALIGN),
    (dict(y=FAKE), pgq.PGQ_ERR_PARAM), (dict(y=FAKE + 0x1000), pgq.PGQ_ERR_PARAM), (dict(y=FAKE + 0x2000), pgq.PGQ_ERR_PARAM),
    (dict(residual=FAKE + 0x3000, ldr=8, residual_dtype=pgq.PGQ_F32), pgq.PGQ_ERR_PARAM),        # y as residual of another type
    (dict(M=0), pgq.PGQ_OK), (dict(N=0, ldy=0), pgq.PGQ_OK),
])
def test_linear_argument_errors(args, want):
    p, n = linear(**args), ctypes.c_size_t(0)
    assert pgq.pgq_linear4_forward(ctypes.byref(p), None, 0, None) == want
    assert pgq.pgq_linear4_forward_workspace(ctypes.byref(p), ctypes.byref(n)) == want


def test_sizes_past_one_launch_are_refused():
    n = ctypes.c_size_t(0)
    p = linear(N=(1 << 31) - 1, M=1 << 20, ldy=(1 << 31) - 1, codes=1 << 52, scales=1 << 53, y=1 << 54)
    assert pgq.pgq_linear4_forward(ctypes.byref(p), None, 0, None) == pgq.PGQ_ERR_SHAPE
    assert pgq.pgq_linear4_forward_workspace(ctypes.byref(p), ctypes.byref(n)) == pgq.PGQ_ERR_SHAPE


@pytest.mark.parametrize("M,N,K", [(6, 48, 16392), (30, 48, 16392), (64, 48, 16392), (64, 8192, 8192)])
def test_workspace_is_required_when_k_is_cut(M, N, K):
    n = ctypes.c_size_t(0)
    p = linear(M=M, N=N, K=K, ldx=K, ldc=(K + 7) // 8 * 4, lds=(K + 31) // 32, ldy=N, x=1 << 40, codes=1 << 41, scales=1 << 42, y=1 << 43)
    assert pgq.pgq_linear4_forward_workspace(ctypes.byref(p), ctypes.byref(n)) == pgq.PGQ_OK
    assert n.value > 0 and n.value % 256 == 0
    assert pgq.pgq_linear4_forward(ctypes.byref(p), None, 0, None) == pgq.PGQ_ERR_WORKSPACE
    assert pgq.pgq_linear4_forward(ctypes.byref(p), FAKE, n.value - 1, None) == pgq.PGQ_ERR_WORKSPACE
    assert pgq.pgq_linear4_forward(ctypes.byref(p), FAKE + 128, n.value, None) == pgq.PGQ_ERR_ALIGN


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (2, 28672, 8192), (16, 4096, 4096), (5, 717, 1031)])
def test_no_workspace_otherwise(M, N, K):
    n = ctypes.c_size_t(7)
    p = linear(M=M, N=N, K=K, ldx=K, ldc=(K + 7) // 8 * 4, lds=(K + 31) // 32, ldy=N, x=1 << 40, codes=1 << 41, scales=1 << 42, y=1 << 43)
    assert pgq.pgq_linear4_forward_workspace(ctypes.byref(p), ctypes.byref(n)) == pgq.PGQ_OK and n.value == 0


def test_null_descriptors():
    n, p = ctypes.c_size_t(0), linear()
    assert pgq.pgq_linear4_forward(None, None, 0, None) == pgq.PGQ_ERR_NULL
    assert pgq.pgq_linear4_forward_workspace(ctypes.byref(p), None) == pgq.PGQ_ERR_NULL
    assert pgq.pgq_linear4_forward_workspace(None, ctypes.byref(n)) == pgq.PGQ_ERR_NULL


def test_packed_descriptor_matches_the_struct():
    torch = pytest.importorskip("torch")  # noqa: F841  (ops imports it)
    from int6_weight_export_amd import ops

    vals = list(range(1, 19)) + [0.5, 7]
    names = [f[0] for f in pgq.pgq_linear4_fwd._fields_]
    p = pgq.pgq_linear4_fwd.from_buffer_copy(ops._FWD4.pack(*vals))
    assert ops._FWD4.size == ctypes.sizeof(pgq.pgq_linear4_fwd)
    assert [getattr(p, n) for n in names] == vals


def test_struct_layout_matches_the_header(tmp_path):
    """Offsets of pgq_linear4_fwd as a C compiler sees them."""
    import os
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = [f[0] for f in pgq.pgq_linear4_fwd._fields_]
    src = tmp_path / "o.c"
    src.write_text('#include "pgq.h"\n#include <stdio.h>\nint main(void){' + "".join(
        f'printf("%zu\\n", offsetof(pgq_linear4_fwd, {n}));' for n in names) + 'printf("%zu\\n", sizeof(pgq_linear4_fwd));return 0;}')
    exe = tmp_path / "o"
    subprocess.check_call(["gcc", "-I", os.path.join(root, "include"), "-o", str(exe), str(src)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    assert got == [getattr(pgq.pgq_linear4_fwd, n).offset for n in names] + [ctypes.sizeof(pgq.pgq_linear4_fwd)]


@pytest.mark.parametrize("cols,group", [(1, 32), (31, 32), (33, 32), (200, 64), (129, 128), (256, 128)])
def test_reference_against_the_definition(cols, group):
    """Scale and code of every group from exact arithmetic: s the fp16 nearest to the binary32 quotient, the code the
    whole number nearest to w / s (ties to even)."""
    rng = np.random.default_rng(cols)
    w = (rng.standard_normal((5, cols)) * 0.05).astype(np.float32)
    w[1] = 0
    w[2, 0] = 3.5 * np.float32(np.float16(0.01))              # a tie of its group if 0.01 becomes its scale
    codes, scales, dq, status = ref.quantize(w, group)
    assert status == 0
    for r in range(5):
        for g in range(scales.shape[1]):
            part = w[r, g * group:(g + 1) * group]
            s = np.float16(np.float32(np.abs(part).max()) / np.float32(7))
            s = np.float16(1) if s == 0 else s
            assert scales[r, g] == s.view(np.uint16)
            want = np.clip(np.rint(part.astype(np.float64) / np.float64(s)), -7, 7)
            assert np.array_equal(codes[r, g * group:(g + 1) * group], want)
    assert np.array_equal(ref.values(codes, scales, group).astype(np.float32), dq)
    assert np.array_equal(ref.unpack(ref.pack(codes), cols), codes)
    assert ref.pack(codes).shape == (5, -(-cols // 8) * 4)


def test_layout_by_hand():
    codes = np.array([[1, -2, 3, -4, 5, -6, 7, 0, -7]], np.int8)
    assert ref.pack(codes).tolist() == [[0x51, 0xEA, 0x73, 0x0C, 0x0F, 0, 0, 0]]
