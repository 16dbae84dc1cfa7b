"""ops.GradNorm's and ops.AdamW's handling of tensors and of the norm's buffers, on the CPU: the library is replaced by a stand-in
that writes down which addresses, sizes and types a call was given, and nothing is launched."""
import ctypes
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")
pgq = pytest.importorskip("int6_weight_export_amd.pgq")
from int6_weight_export_amd import ops  # noqa: E402

REAL = pgq._lib


@pytest.fixture
def calls(monkeypatch):
    """The calls that reach the library, in order: (entry point, addresses, sizes, types)."""
    made = []

    def record(name):
        def call(ptrs, numel, dtype, n, *rest):
            made.append((name, [p or 0 for p in ptrs], list(numel), list(dtype)))
            assert n == len(ptrs)
            return pgq.PGQ_OK
        return call

    monkeypatch.setattr(pgq, "_lib", SimpleNamespace(pgq_grad_norm_workspace=REAL.pgq_grad_norm_workspace,
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


# ---- the optimizer's norm buffers ------------------------------------------------------------------------


@pytest.fixture
def opt_calls(calls, monkeypatch):
    """The optimizer's calls: (entry point, workspace, result or factor, whether the workspace was clear); and what torch says about
    capturing, with the number of times that the workspace's size was asked for."""
    lib, made, state = pgq._lib, [], SimpleNamespace(capturing=False, sizes=0)
    size_of = lib.pgq_grad_norm_workspace

    def size(*a):
        state.sizes += 1
        return size_of(*a)

    def norm(ptrs, numel, dtype, n, scale, scale_dev, max_norm, result, workspace, nbytes, status, stream):
        clear = all(b == 0 for b in (ctypes.c_uint8 * nbytes).from_address(workspace))
        made.append(("norm", workspace, result, clear))
        return pgq.PGQ_OK

    def step(arr, n, bits, ptrs, h, h_dev, factor, *rest):
        made.append(("step", None, factor, True))
        return pgq.PGQ_OK

    lib.pgq_grad_norm_workspace, lib.pgq_grad_norm, lib.pgq_adamw_step_clipped = size, norm, step
    for name in ("pgq_adamw_workspace", "pgq_adamw_hyper_at"):
        setattr(lib, name, getattr(REAL, name))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state.capturing)
    return made, state


def optimizer():
    return ops.AdamW([torch.randn(100), torch.randn(7)], lr=0.01), [torch.randn(100), torch.randn(7)]


def test_an_optimizer_that_never_clips_makes_no_norm_buffers(opt_calls, monkeypatch):
    made, state = opt_calls
    copies = []
    monkeypatch.setattr(ops, "_norm_result", lambda *a: copies.append(a))
    state.capturing = True
    opt, grads = optimizer()
    state.capturing = False
    for _ in range(2):
        assert opt.step(grads) is None
    assert state.sizes == 0 and copies == [] and [c[0] for c in made] == ["step", "step"] and made[0][2] is None


def test_clipped_steps_share_the_buffers_of_the_first(opt_calls):
    made, state = opt_calls
    opt, grads = optimizer()
    norms = [opt.step(grads, max_norm=1.0) for _ in range(2)]
    state.capturing = True
    norms.append(opt.step(grads, max_norm=1.0, device_hyper=True))
    at = opt.norm_result.data_ptr()
    assert [c[:3] for c in made] == [("norm", opt.norm_workspace.data_ptr(), at), ("step", None, at + 4)] * 3 and state.sizes == 1
    assert all(c[3] for c in made) and all(n.data_ptr() == at for n in norms) and opt.grad_norm.data_ptr() == at


def test_steps_captured_before_the_first_clipped_one_have_buffers_of_their_own(opt_calls):
    made, state = opt_calls
    opt, grads = optimizer()
    opt.step(grads)
    state.capturing = True
    kept = []
    for _ in range(2):
        norm = opt.step(grads, max_norm=1.0, device_hyper=True)
        kept.append((opt.norm_workspace, opt.norm_result))
        assert norm.data_ptr() == opt.norm_result.data_ptr() == opt.grad_norm.data_ptr()
    state.capturing = False
    opt.step(grads, max_norm=1.0)
    kept.append((opt.norm_workspace, opt.norm_result))
    norms = [c for c in made if c[0] == "norm"]
    assert [(c[1], c[2]) for c in norms] == [(w.data_ptr(), r.data_ptr()) for w, r in kept] and all(c[3] for c in norms)
    assert len({c[1] for c in norms}) == len({c[2] for c in norms}) == 3
    state.capturing = True                                  # from now on captured steps take the kept ones, as eager steps do
    opt.step(grads, max_norm=1.0, device_hyper=True)
    assert (made[-2][1], made[-2][2]) == (kept[2][0].data_ptr(), kept[2][1].data_ptr())


def test_the_result_can_be_read_before_a_clipped_step(opt_calls):
    _, state = opt_calls
    opt, grads = optimizer()
    assert opt.norm_result.tolist() == [0.0, 0.0] and opt.norm_result.dtype == torch.float32
    at = opt.norm_result.data_ptr()
    assert opt.step(grads, max_norm=1.0).data_ptr() == at and state.sizes == 1
