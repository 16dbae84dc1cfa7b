"""GPU tests of AdamW steps that read their constants from device memory, before any were written there and
after some were refused: nothing may change, and the caller is told."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int6_weight_export_amd import ops, pgq  # noqa: E402


def say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def make(bits, seed=0, sizes=(5000, 64, 3)):
    g = torch.Generator().manual_seed(seed)
    w = [torch.randn(n, generator=g).cuda() for n in sizes]
    copies = [torch.randn(n, generator=g).bfloat16().cuda() for n in sizes]
    grads = [torch.randn(n, generator=g).cuda() for n in sizes]
    opt = ops.AdamW(w, lr=0.01, state_bits=bits, copies=copies, seed=4)
    return opt, grads


def everything(opt):
    torch.cuda.synchronize()
    return [t.clone() for t in (*opt.weights, *opt.copies, *(s for st in opt.states for s in st))]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("bits", [32, 8])
def test_eager_step_without_loaded_constants_is_refused(bits):
    say(f"adamw {bits} bits: device_hyper before load_hyper")
    opt, grads = make(bits)
    before = everything(opt)
    with pytest.raises(pgq.PgqError, match="load_hyper"):
        opt.step(grads, device_hyper=True)
    assert same(before, everything(opt)) and opt.step_count == 0
    opt.step(grads)
    before = everything(opt)
    with pytest.raises(pgq.PgqError, match="load_hyper"):
        opt.step(grads, device_hyper=True)
    assert same(before, everything(opt)) and opt.step_count == 1
    opt.load_hyper()
    opt.step(grads, device_hyper=True)
    other, _ = make(bits)
    other.step(grads)
    other.step(grads)
    assert same(everything(opt), everything(other)) and opt.step_count == 2 and int(opt.status.item()) == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_replay_before_loaded_constants_changes_nothing(bits):
    say(f"adamw {bits} bits: a replay before load_hyper")
    opt, grads = make(bits)
    opt.step(grads)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(grads, device_hyper=True)
    before = everything(opt)
    for _ in range(2):
        graph.replay()
        assert same(before, everything(opt))
        assert int(opt.status.item()) == pgq.PGQ_DEV_NO_HYPER
    opt.status.zero_()
    other, _ = make(bits)
    other.step(grads)
    for k in range(3):
        opt.load_hyper(lr=0.02 / (k + 1))
        graph.replay()
        other.step(grads, lr=0.02 / (k + 1))
        assert same(everything(opt), everything(other)), k
    assert int(opt.status.item()) == 0 and opt.step_count == other.step_count == 4


def test_refused_constants_count_no_step():
    say("adamw: refused learning rates leave the step number")
    opt, grads = make(32)
    for lr in (float("nan"), -1.0, float("inf")):
        with pytest.raises(pgq.PgqError):
            opt.load_hyper(lr=lr)
        with pytest.raises(pgq.PgqError):
            opt.step(grads, lr=lr)
    with pytest.raises(Exception):
        opt.step(grads, lr="high")
    assert opt.step_count == 0
    with pytest.raises(pgq.PgqError, match="load_hyper"):
        opt.step(grads, device_hyper=True)
    opt.load_hyper()
    opt.step(grads)
    assert opt.step_count == 2
