"""Host checks of AdamW's constants (CPU; nothing is enqueued)."""
import ctypes

import pytest

pgq = pytest.importorskip("int6_weight_export_amd.pgq")

FAKE = 0x10000


def step(h):
    t = (pgq.pgq_adamw_tensor * 1)(pgq.pgq_adamw_tensor(w=FAKE, m=FAKE + 4096, v=FAKE + 8192, numel=100, lr_scale=1.0))
    g = (ctypes.c_void_p * 1)(FAKE + 12288)
    return pgq.pgq_adamw_step(t, 1, 32, g, ctypes.byref(h), None, FAKE, 1 << 20, 0, None, None)


@pytest.mark.parametrize("kw", [dict(), dict(ib1=1.0), dict(ib2=1.0), dict(ib1=-1.0, ib2=1.0),
                                dict(ib1=float("nan"), ib2=1.0), dict(ib1=1.0, ib2=float("nan"))])
def test_constants_of_no_step_are_refused(kw):
    """Zeroed constants would make every weight 0 / 0 and clear the states."""
    assert step(pgq.pgq_adamw_hyper(lr=0.1, **kw)) == pgq.PGQ_ERR_PARAM


@pytest.mark.parametrize("kw", [dict(lr=3.5e38), dict(lr=1e300), dict(eps=1e39)])
def test_constants_that_binary32_cannot_hold_are_refused(kw):
    """Finite numbers that round to a binary32 infinity would make every weight NaN."""
    a = dict(lr=1e-3, eps=1e-8)
    a.update(kw)
    h = pgq.pgq_adamw_hyper()
    assert pgq.pgq_adamw_hyper_at(a["lr"], 0.9, 0.999, a["eps"], 1, 1.0, 0, ctypes.byref(h)) == pgq.PGQ_ERR_PARAM
    assert pgq.pgq_adamw_hyper_at(3.4e38, 0.9, 0.999, 1e-8, 1, 1.0, 0, ctypes.byref(h)) == pgq.PGQ_OK
