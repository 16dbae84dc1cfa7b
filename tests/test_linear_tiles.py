"""Which tile a size gets (CPU): the sizes that the GPU tests run still get the tiles they are listed for, and the
list holds every tile, whole and in parts, that sizes of a wide range get."""
import ctypes
import math
import random

import pytest

pgq = pytest.importorskip("int6_weight_export_amd.pgq")

from tests import linear_tiles as lt  # noqa: E402


@pytest.mark.parametrize("args,want", lt.FORWARD)
def test_forward_sizes_get_their_tiles(args, want):
    assert lt.forward_plan(*args) == want


@pytest.mark.parametrize("args,want", lt.BACKWARD)
def test_backward_sizes_get_their_tiles(args, want):
    assert lt.backward_plan(*args) == want


def sizes(n, seed):
    rng = random.Random(seed)
    for _ in range(n):
        M, N, K = (int(round(math.exp(rng.uniform(math.log(a), math.log(b))))) for a, b in ((17, 16384), (16, 8192), (16, 8192)))
        if rng.random() < 0.5:
            N, K = max(16, N // 16 * 16), max(16, K // 16 * 16)
        yield M, N, K, rng.choice(["bf16", "f32"]), rng.choice(["", "f32", "bf16"]), rng.choice(["none", "silu"])


def test_every_tile_that_sizes_get_is_listed():
    fwd = {w[:4] for _, w in lt.FORWARD}
    bwd = {w[:7] for _, w in lt.BACKWARD}
    for M, N, K, t, res, act in sizes(12000, 2):
        got = lt.forward_plan(M, N, K, t, res)
        assert got is None or got[:4] in fwd, (M, N, K, t, res, got)
        for want in ("dx", "dw", "dx dw dbias"):
            got = lt.backward_plan(M, N, K, want, t, act)
            assert got is None or got[:7] in bwd, (M, N, K, t, act, got)


def test_both_output_types_of_every_tile_are_listed():
    for key in {w[:3] for _, w in lt.FORWARD}:
        assert {w[4] for _, w in lt.FORWARD if w[:3] == key} == {"bf16", "f32"}, key
    for key in {(w[0], *w[1:3], *w[4:6]) for _, w in lt.BACKWARD}:
        assert {w[7] for _, w in lt.BACKWARD if (w[0], *w[1:3], *w[4:6]) == key} == {"bf16", "f32"}, key
    # and some of both with bias, activation and residual, and with dZ in one, two and three parts (run by the GPU test)
    assert {r for (_, _, _, _, r), _ in lt.FORWARD} == {"", "f32", "bf16"}
    assert {(t, a) for (*_, t, a), _ in lt.BACKWARD} == {(t, a) for t in ("bf16", "f32") for a in ("none", "silu")}


@pytest.mark.parametrize("M,K,path,parts", [(1, 512, pgq.PGQ_LINEAR_FEW, False), (16, 8192, pgq.PGQ_LINEAR_FEW, True),
                                            (0, 512, pgq.PGQ_LINEAR_EMPTY, False), (200, 1 << 21, pgq.PGQ_LINEAR_ELEMENTS, False)])
def test_paths(M, K, path, parts):
    p = pgq.pgq_linear_fwd(M=M, N=64, K=K, x=lt.AT["x"], ldx=K, codes=lt.AT["codes"], ldc=K, scales=lt.AT["scales"], y=lt.AT["y"],
                           ldy=64)
    o = pgq.pgq_linear_plan()
    assert pgq.pgq_linear_forward_plan(ctypes.byref(p), ctypes.byref(o)) == pgq.PGQ_OK
    assert (o.path, o.parts > 1) == (path, parts)
    assert pgq.pgq_linear_forward_plan(ctypes.byref(p), None) == pgq.PGQ_ERR_NULL
    assert pgq.pgq_linear_forward_plan(None, ctypes.byref(o)) == pgq.PGQ_ERR_NULL
    p.ldx = K - 1
    assert pgq.pgq_linear_forward_plan(ctypes.byref(p), ctypes.byref(o)) == pgq.PGQ_ERR_SHAPE


@pytest.mark.parametrize("act,slope,dy,t,parts", [
    (0, 0.0, "bf16", "f32", 1), (0, 0.0, "f32", "bf16", 2), (0, 0.0, "f32", "f32", 3), (1, 0.0, "bf16", "f32", 1),
    (1, -0.25, "bf16", "bf16", 1), (1, 0.3, "bf16", "bf16", 2), (1, 0.3, "bf16", "f32", 3), (1, 0.5, "f32", "f32", 3),
    (2, 0.5, "bf16", "bf16", 2), (2, 0.5, "bf16", "f32", 2), (2, 0.3, "bf16", "f32", 3), (3, 0.0, "bf16", "bf16", 2),
    (3, 0.0, "bf16", "f32", 3)])
def test_parts_of_dz(act, slope, dy, t, parts):
    p = pgq.pgq_linear_bwd(M=100, N=64, K=48, dy=lt.AT["dy"], lddy=64, dy_dtype=lt.TYPE[dy], z=lt.AT["z"], ldz=64, x=lt.AT["x"], ldx=48,
                           codes=lt.AT["codes"], ldc=48, scales=lt.AT["scales"], dx=lt.AT["dx"], lddx=48, dx_dtype=lt.TYPE[t],
                           dw=lt.AT["dw"], lddw=48, dw_dtype=lt.TYPE[t], act=act, slope=slope)
    o = pgq.pgq_linear_plan()
    assert pgq.pgq_linear_backward_plan(ctypes.byref(p), ctypes.byref(o)) == pgq.PGQ_OK
    assert (o.dz_dx, o.dz_dw, o.joint) == (parts, parts, 1)
    p.dx = None
    assert pgq.pgq_linear_backward_plan(ctypes.byref(p), ctypes.byref(o)) == pgq.PGQ_OK
    assert (o.dz_dx, o.dz_dw, o.joint) == (0, parts, 0)
