"""ops.GradNorm's and ops.AdamW's handling of tensors and of the norm's buffers, on the CPU: the library is replaced by a stand-in
that writes down which addresses, sizes and types a call was given, and nothing is launched."""
import ctypes
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")
pgq = pytest.importorskip("int6_weight_export_amd.pgq")
from int6_weight_export_amd import ops  # noqa: E402


@pytest.fixture
def calls(monkeypatch):
    """The calls that reach the library, in order: (entry point, addresses, sizes, types)."""
    made, real = [], pgq._lib

    def record(name):
        def call(ptrs, numel, dtype, n, *rest):
            made.append((name, [p or 0 for p in ptrs], list(numel), list(dtype)))
            assert n == len(ptrs)
            return pgq.PGQ_OK
        return call

    monkeypatch.setattr(pgq, "_lib", SimpleNamespace(pgq_grad_norm_workspace=real.pgq_grad_norm_workspace,
                                                     pgq_grad_norm=record("norm"), pgq_grad_clip=record("clip")))
    monkeypatch.setattr(ops, "_gpu_of", lambda name, t: t.get_device())
    monkeypatch.setattr(ops, "_current_device", lambda: -1)
    monkeypatch.setattr(ops, "_stream_of", lambda index: 0)
    return made


def where(grads):
    return [g.data_ptr() for g in grads]


@pytest.mark.parametrize("name", ["norm", "clip"])
def test_a_gradient_whose_data_was_replaced_is_taken_where_it_lies(calls, name):
    grads = [torch.randn(n) for n in (100, 7, 33)]
    gn = ops.GradNorm(grads)
    run = {"norm": gn.norm, "clip": gn.clip_}[name]
    run(1.0)
    assert calls[-1] == (name, where(grads), [100, 7, 33], [pgq.PGQ_F32] * 3)
    old = where(grads)
    keep = grads[1].untyped_storage()                       # (so that the new memory is elsewhere)
    grads[1].data = torch.randn(7).bfloat16() if name == "norm" else torch.randn(7)
    assert where(grads) != old and keep.data_ptr() == old[1]
    run(1.0)
    assert calls[-1][1] == where(grads) and calls[-1][3][1] == ops._dtype_code(grads[1].dtype)
    run(1.0)
    assert calls[-1][1] == where(grads) and len(calls) == 3


def test_a_gradient_whose_storage_was_reallocated_is_taken_where_it_lies(calls):
    grads = [torch.randn(5), torch.randn(1 << 20)]
    gn = ops.GradNorm(grads)
    st, old = grads[1].untyped_storage(), where(grads)
    st.resize_(0)
    other = torch.zeros(1 << 20)                            # (may take the freed memory)
    st.resize_(4 << 20)
    gn.clip_(1.0)
    assert calls[-1][1] == where(grads) and other.data_ptr() not in calls[-1][1] and old[0] == calls[-1][1][0]


def test_a_gradient_that_changed_its_size_is_refused(calls):
    grads = [torch.randn(100), torch.randn(7)]
    gn = ops.GradNorm(grads)
    for bad in (torch.randn(8), torch.randn(6), torch.randn(14)[::2], torch.zeros(7, dtype=torch.int32)):
        grads[1].data = bad
        for call in (gn.norm, gn.clip_):
            with pytest.raises((ValueError, TypeError)):
                call(1.0)
    assert calls == []
    grads[1].data = torch.randn(7)
    gn.norm(1.0)
    assert calls[-1][1] == where(grads)


def test_memory_of_a_bound_gradient_is_not_given_away(calls):
    """A replaced storage stays allocated until the next bind(), so no smaller one can lie at its address."""
    g = torch.randn(1 << 16)
    gn, old = ops.GradNorm([g]), g.data_ptr()
    for n in (1 << 16, 1 << 15, 64):
        g.data = torch.randn(n)
        assert g.data_ptr() != old
    with pytest.raises(ValueError):
        gn.clip_(1.0)
    assert calls == []
