"""Sizes of the linear layer and AdamW past what one launch holds, on the CPU: refused by the size query and by the
call, before anything is enqueued."""
import ctypes

import pytest

pgq = pytest.importorskip("int6_weight_export_amd.pgq")

AT = {n: (i + 1) << 44 for i, n in enumerate(("x", "codes", "scales", "y", "dy", "dx", "dw", "dbias", "z"))}


def fwd(M, N, K):
    return pgq.pgq_linear_fwd(M=M, N=N, K=K, x=AT["x"], ldx=K, codes=AT["codes"], ldc=K, scales=AT["scales"], y=AT["y"], ldy=N,
                              y_dtype=pgq.PGQ_BF16)


def bwd(M, N, K, want):
    p = pgq.pgq_linear_bwd(M=M, N=N, K=K, dy=AT["dy"], lddy=N, dy_dtype=pgq.PGQ_BF16, x=AT["x"], ldx=K, codes=AT["codes"], ldc=K,
                           scales=AT["scales"], lddx=K, dx_dtype=pgq.PGQ_BF16, lddw=K, dw_dtype=pgq.PGQ_BF16)
    for k in want:
        setattr(p, k, AT[k])
    return p


def both(p):
    """(size query, call): the call is made only where the query refuses."""
    n = ctypes.c_size_t(0)
    f = isinstance(p, pgq.pgq_linear_fwd)
    size, call = ((pgq.pgq_linear_forward_workspace, pgq.pgq_linear_forward) if f
                  else (pgq.pgq_linear_backward_workspace, pgq.pgq_linear_backward))
    rc = size(ctypes.byref(p), ctypes.byref(n))
    if rc == pgq.PGQ_OK:
        return rc, n.value
    return rc, call(ctypes.byref(p), None, 0, None)


@pytest.mark.parametrize("M,N,K", [(1, 1 << 27, 1), (16, (1 << 31) - 1, 1), (1, 1 << 27, 64), (100, 1 << 24, 4099),
                                   (1 << 24, 100, 4099), (1 << 22, 1 << 18, 1 << 21)])
def test_forward_past_a_launch(M, N, K):
    assert both(fwd(M, N, K)) == (pgq.PGQ_ERR_SHAPE, pgq.PGQ_ERR_SHAPE)


@pytest.mark.parametrize("M,N,K", [(100, 1 << 24, 4096),      # (tiles straight from the codes)
                                   (1, (1 << 27) - 16, 1), (16, 1 << 26, 8), (1 << 22, 4096, 4096), (1 << 20, 100, 4099)])
def test_forward_below_the_limits(M, N, K):
    assert both(fwd(M, N, K))[0] == pgq.PGQ_OK


@pytest.mark.parametrize("M,N,K,want", [(1, 1 << 28, 8, ("dbias",)), (1, 1 << 30, 1, ("dx", "dw", "dbias")),
                                        (1 << 24, 64, 4099, ("dw",)), (64, 1 << 20, 1 << 17, ("dx",)),
                                        (1 << 26, 8, 1 << 22, ("dx",))])
def test_backward_past_a_launch(M, N, K, want):
    assert both(bwd(M, N, K, want)) == (pgq.PGQ_ERR_SHAPE, pgq.PGQ_ERR_SHAPE)


@pytest.mark.parametrize("M,N,K,want", [(1, (1 << 28) - 64, 8, ("dbias",)), (1 << 20, 4096, 4096, ("dx", "dw", "dbias")),
                                        (1 << 18, 64, 4099, ("dw",)), (1, 1, 1, ("dx", "dw", "dbias"))])
def test_backward_below_the_limits(M, N, K, want):
    assert both(bwd(M, N, K, want))[0] == pgq.PGQ_OK


def test_adamw_past_a_launch():
    n = ctypes.c_size_t(0)
    for numel, want in ((1 << 36, pgq.PGQ_ERR_SHAPE), ((1 << 36) - (1 << 13), pgq.PGQ_OK), (1 << 40, pgq.PGQ_ERR_SHAPE)):
        t = (pgq.pgq_adamw_tensor * 1)(pgq.pgq_adamw_tensor(w=AT["x"], m=AT["y"], v=AT["z"], numel=numel, lr_scale=1.0))
        assert pgq.pgq_adamw_workspace(t, 1, ctypes.byref(n)) == want, numel
