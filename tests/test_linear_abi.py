"""The linear layer's C ABI on the CPU: argument errors come back before anything is enqueued."""
import ctypes

import pytest

pgq = pytest.importorskip("int6_weight_export_amd.pgq")

FAKE = 0x10000      # aligned, never dereferenced: every call here fails its checks or has nothing to do


def fwd(**kw):
    a = dict(M=4, N=8, K=16, x=FAKE, ldx=16, codes=FAKE, ldc=16, scales=FAKE, y=FAKE, ldy=8, y_dtype=pgq.PGQ_BF16,
             act=pgq.PGQ_ACT_NONE)
    a.update(kw)
    return pgq.pgq_linear_fwd(**a)


def bwd(**kw):
    a = dict(M=4, N=8, K=16, dy=FAKE, lddy=8, dy_dtype=pgq.PGQ_BF16, x=FAKE, ldx=16, codes=FAKE, ldc=16, scales=FAKE,
             dx=FAKE, lddx=16, dx_dtype=pgq.PGQ_BF16, dw=FAKE, lddw=16, dw_dtype=pgq.PGQ_BF16, dbias=FAKE)
    a.update(kw)
    return pgq.pgq_linear_bwd(**a)


FWD_ERRORS = [
    (dict(M=-1), pgq.PGQ_ERR_SHAPE), (dict(N=1 << 31, ldy=1 << 31), pgq.PGQ_ERR_SHAPE), (dict(ldx=15), pgq.PGQ_ERR_SHAPE),
    (dict(ldc=15), pgq.PGQ_ERR_SHAPE), (dict(ldy=7), pgq.PGQ_ERR_SHAPE),
    (dict(residual=FAKE, ldr=7, residual_dtype=pgq.PGQ_F32), pgq.PGQ_ERR_SHAPE), (dict(z=FAKE, ldz=7), pgq.PGQ_ERR_SHAPE),
    (dict(y_dtype=pgq.PGQ_F16), pgq.PGQ_ERR_DTYPE), (dict(bias=FAKE, bias_dtype=pgq.PGQ_F16), pgq.PGQ_ERR_DTYPE),
    (dict(residual=FAKE, ldr=8, residual_dtype=9), pgq.PGQ_ERR_DTYPE),
    (dict(act=4), pgq.PGQ_ERR_PARAM), (dict(act=-1), pgq.PGQ_ERR_PARAM), (dict(reserved=1), pgq.PGQ_ERR_PARAM),
    (dict(act=pgq.PGQ_ACT_RELU, slope=float("nan")), pgq.PGQ_ERR_PARAM),
    (dict(act=pgq.PGQ_ACT_RELU2, slope=float("inf")), pgq.PGQ_ERR_PARAM),
    (dict(residual=FAKE, ldr=8, residual_dtype=pgq.PGQ_F32), pgq.PGQ_ERR_PARAM),        # y as residual of another type
    (dict(residual=FAKE, ldr=9, residual_dtype=pgq.PGQ_BF16), pgq.PGQ_ERR_PARAM),
    (dict(x=None), pgq.PGQ_ERR_NULL), (dict(codes=None), pgq.PGQ_ERR_NULL), (dict(scales=None), pgq.PGQ_ERR_NULL),
    (dict(y=None), pgq.PGQ_ERR_NULL), (dict(y=FAKE + 1), pgq.PGQ_ERR_ALIGN), (dict(x=FAKE + 1), pgq.PGQ_ERR_ALIGN),
    (dict(bias=FAKE + 2, bias_dtype=pgq.PGQ_F32), pgq.PGQ_ERR_ALIGN), (dict(z=FAKE + 1, ldz=8), pgq.PGQ_ERR_ALIGN),
    (dict(scales=FAKE + 1), pgq.PGQ_ERR_ALIGN),
]

BWD_ERRORS = [
    (dict(K=-1), pgq.PGQ_ERR_SHAPE), (dict(lddy=7), pgq.PGQ_ERR_SHAPE), (dict(ldx=15), pgq.PGQ_ERR_SHAPE),
    (dict(ldc=15), pgq.PGQ_ERR_SHAPE), (dict(lddx=15), pgq.PGQ_ERR_SHAPE), (dict(lddw=15), pgq.PGQ_ERR_SHAPE),
    (dict(act=pgq.PGQ_ACT_SILU, z=FAKE, ldz=7), pgq.PGQ_ERR_SHAPE),
    (dict(dy_dtype=pgq.PGQ_F16), pgq.PGQ_ERR_DTYPE), (dict(dx_dtype=pgq.PGQ_F16), pgq.PGQ_ERR_DTYPE),
    (dict(dw_dtype=7), pgq.PGQ_ERR_DTYPE), (dict(act=9), pgq.PGQ_ERR_PARAM), (dict(reserved=3), pgq.PGQ_ERR_PARAM),
    (dict(act=pgq.PGQ_ACT_SILU, ldz=8), pgq.PGQ_ERR_NULL), (dict(dy=None), pgq.PGQ_ERR_NULL),
    (dict(x=None), pgq.PGQ_ERR_NULL), (dict(codes=None), pgq.PGQ_ERR_NULL), (dict(scales=None), pgq.PGQ_ERR_NULL),
    (dict(dy=FAKE + 2, dy_dtype=pgq.PGQ_F32), pgq.PGQ_ERR_ALIGN), (dict(dx=FAKE + 1), pgq.PGQ_ERR_ALIGN),
    (dict(dw=FAKE + 2, dw_dtype=pgq.PGQ_F32), pgq.PGQ_ERR_ALIGN), (dict(dbias=FAKE + 2), pgq.PGQ_ERR_ALIGN),
]


@pytest.mark.parametrize("args,want", FWD_ERRORS)
def test_forward_argument_errors(args, want):
    p, n = fwd(**args), ctypes.c_size_t(0)
    assert pgq.pgq_linear_forward(ctypes.byref(p), None, 0, None) == want
    assert pgq.pgq_linear_forward_workspace(ctypes.byref(p), ctypes.byref(n)) == want


@pytest.mark.parametrize("args,want", BWD_ERRORS)
def test_backward_argument_errors(args, want):
    p, n = bwd(**args), ctypes.c_size_t(0)
    assert pgq.pgq_linear_backward(ctypes.byref(p), None, 0, None) == want
    assert pgq.pgq_linear_backward_workspace(ctypes.byref(p), ctypes.byref(n)) == want


def test_null_descriptors_and_empty_calls():
    n = ctypes.c_size_t(0)
    assert pgq.pgq_linear_forward(None, None, 0, None) == pgq.PGQ_ERR_NULL
    assert pgq.pgq_linear_backward(None, None, 0, None) == pgq.PGQ_ERR_NULL
    assert pgq.pgq_linear_forward_workspace(ctypes.byref(fwd()), None) == pgq.PGQ_ERR_NULL
    assert pgq.pgq_linear_backward_workspace(ctypes.byref(bwd()), None) == pgq.PGQ_ERR_NULL
    assert pgq.pgq_linear_forward(ctypes.byref(fwd(M=0)), None, 0, None) == pgq.PGQ_OK
    assert pgq.pgq_linear_forward(ctypes.byref(fwd(N=0, y=None, ldy=0)), None, 0, None) == pgq.PGQ_OK
    nothing = bwd(dx=None, dw=None, dbias=None)
    assert pgq.pgq_linear_backward(ctypes.byref(nothing), None, 0, None) == pgq.PGQ_OK
    assert pgq.pgq_linear_backward_workspace(ctypes.byref(nothing), ctypes.byref(n)) == pgq.PGQ_OK and n.value == 0


def test_packed_descriptors_match_the_structs():
    """The wrappers pack descriptors with struct; the layout has to be the C structs'."""
    import struct as st

    for fmt, cls in (("15q4ifi", pgq.pgq_linear_fwd), ("18q4ifi", pgq.pgq_linear_bwd)):
        assert st.calcsize(fmt) == ctypes.sizeof(cls)
        names = [n for n, _ in cls._fields_]
        vals = [i + 1 if n != "slope" else 0.5 for i, n in enumerate(names)]
        p = cls.from_buffer_copy(st.pack(fmt, *vals))
        for n, v in zip(names, vals):
            got = getattr(p, n)
            assert got == v, n
    src = open(__import__("os").path.join(__import__("os").path.dirname(pgq.LIB_PATH), "ops.py")).read()
    assert 'struct.Struct("15q4ifi")' in src and 'struct.Struct("18q4ifi")' in src


def test_workspace_is_required_when_the_call_needs_one():
    n = ctypes.c_size_t(0)
    at = {n: FAKE + (i << 32) for i, n in enumerate(("x", "codes", "scales", "y", "dy", "dx", "dw", "dbias"))}
    p = fwd(M=4096, N=1024, K=520, ldx=520, ldc=520, ldy=1024, **{k: at[k] for k in ("x", "codes", "scales", "y")})
    assert pgq.pgq_linear_forward_workspace(ctypes.byref(p), ctypes.byref(n)) == pgq.PGQ_OK and n.value > 0
    assert pgq.pgq_linear_forward(ctypes.byref(p), None, 0, None) == pgq.PGQ_ERR_WORKSPACE
    assert pgq.pgq_linear_forward(ctypes.byref(p), FAKE, n.value - 1, None) == pgq.PGQ_ERR_WORKSPACE
    assert pgq.pgq_linear_forward(ctypes.byref(p), FAKE + 64, n.value, None) == pgq.PGQ_ERR_ALIGN
    b = bwd(M=512, **{k: at[k] for k in at if k != "y"})
    assert pgq.pgq_linear_backward_workspace(ctypes.byref(b), ctypes.byref(n)) == pgq.PGQ_OK and n.value > 0
    assert pgq.pgq_linear_backward(ctypes.byref(b), None, 0, None) == pgq.PGQ_ERR_WORKSPACE
    assert pgq.pgq_linear_backward(ctypes.byref(b), FAKE + 8, n.value, None) == pgq.PGQ_ERR_ALIGN
    # few tokens need none
    assert pgq.pgq_linear_forward_workspace(ctypes.byref(fwd(M=1, **{k: at[k] for k in ("x", "codes", "scales", "y")})),
                                            ctypes.byref(n)) == pgq.PGQ_OK and n.value == 0


def _status(p):
    size = pgq.pgq_linear_forward_workspace if isinstance(p, pgq.pgq_linear_fwd) else pgq.pgq_linear_backward_workspace
    return size(ctypes.byref(p), ctypes.byref(ctypes.c_size_t(0)))


def test_outputs_share_no_memory_with_other_arguments():
    """4 tokens, 8 outputs, 16 inputs; an output whose bytes meet another argument's is refused."""
    names = ("x", "codes", "scales", "y", "z", "bias", "residual", "dy", "dx", "dw", "dbias", "mask")
    at = {n: FAKE + (i << 16) for i, n in enumerate(names)}

    def f(**kw):
        a = {k: at[k] for k in ("x", "codes", "scales", "y", "z", "bias", "residual")}
        a.update(ldz=8, ldr=8, bias_dtype=pgq.PGQ_F32, residual_dtype=pgq.PGQ_F32)
        a.update(kw)
        return _status(fwd(**a))

    def b(**kw):
        a = {k: at[k] for k in ("x", "codes", "scales", "z", "dy", "dx", "dw", "dbias", "mask")}
        a.update(ldz=8, act=pgq.PGQ_ACT_SILU)
        a.update(kw)
        return _status(bwd(**a))

    assert f() == pgq.PGQ_OK and b() == pgq.PGQ_OK
    for k in ("x", "codes", "scales", "z", "bias", "residual"):
        assert f(y=at[k]) == pgq.PGQ_ERR_PARAM, k
        if k != "z":
            assert f(z=at[k]) == pgq.PGQ_ERR_PARAM, k
    for o in ("dx", "dw", "dbias"):
        for k in ("x", "codes", "scales", "z", "dy", "dx", "dw", "mask"):
            if k != o:
                assert b(**{o: at[k]}) == pgq.PGQ_ERR_PARAM, (o, k)
    # the last byte of x and the one behind it
    assert f(y=at["x"] + 4 * 16 * 2 - 2) == pgq.PGQ_ERR_PARAM and f(y=at["x"] + 4 * 16 * 2) == pgq.PGQ_OK
    # Y in place of its residual; columns of one buffer; the same with one column shared; another stride
    assert f(residual=at["y"], residual_dtype=pgq.PGQ_BF16) == pgq.PGQ_OK
    assert f(y=at["x"] + 32, ldx=24, ldy=24) == pgq.PGQ_OK
    assert f(y=at["x"], x=at["x"] + 16, ldx=24, ldy=24) == pgq.PGQ_OK
    assert f(y=at["x"] + 30, ldx=24, ldy=24) == pgq.PGQ_ERR_PARAM
    assert f(y=at["x"], x=at["x"] + 14, ldx=24, ldy=24) == pgq.PGQ_ERR_PARAM
    assert f(y=at["x"] + 32, ldx=24, ldy=28) == pgq.PGQ_ERR_PARAM
    # an argument that the call does not use may lie anywhere
    assert b(dw=None, x=at["dx"], mask=at["dx"]) == pgq.PGQ_OK and b(dx=None, codes=at["dw"], scales=at["dw"]) == pgq.PGQ_OK
    assert b(act=pgq.PGQ_ACT_NONE, z=at["dx"]) == pgq.PGQ_OK
    assert _status(fwd(M=0)) == pgq.PGQ_OK
