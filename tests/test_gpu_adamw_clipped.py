"""GPU tests of the optimizer step that clips on the way: an optimizer made while a graph is captured, clipped steps that are captured
before the first eager one, types of weights and gradients, lists of several launches, two streams.  A clipped step is compared, bit
for bit, with an unclipped one whose grad_scale is fl32(grad_scale * factor), the factor being read back from the device; the norm
with the sum in 64 bits (bound as in test_gpu_gradnorm.py)."""
import math
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int6_weight_export_amd import ops  # noqa: E402

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
REL = (1 + 2.0 ** -6) * 2.0 ** -24


def say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def rand(n, seed, std=1.0, t="f32"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, generator=g) * std).to(T[t]).cuda()


def exact_norm(grads):
    return math.sqrt(math.fsum(float((g.double().cpu().numpy().astype(np.longdouble) ** 2).sum()) for g in grads))


def tensors(opt):
    return opt.weights + [c for c in opt.copies if c is not None] + [t for s in opt.states for t in s]


def same(a, b):
    torch.cuda.synchronize()
    for x, y in zip(tensors(a), tensors(b)):
        assert torch.equal(x, y)


def optimizer(sizes, bits, types=("f32",), seed=1):
    weights = [rand(n, seed + i, 0.1, types[i % len(types)]) for i, n in enumerate(sizes)]
    copies = [torch.zeros(w.numel(), dtype=torch.bfloat16, device="cuda") if w.dtype == torch.float32 else None for w in weights]
    return ops.AdamW(weights, lr=0.01, state_bits=bits, seed=5, copies=copies)


def unclipped(opt, grads, norm_result, scale):
    """The step that opt takes with these gradients and the factor that the clipped step found."""
    opt.step(grads, grad_scale=float(np.float32(scale) * np.float32(float(norm_result[1]))))


def test_made_while_a_graph_is_captured():
    say("adamw made while a graph is captured")
    sizes = [4096, 700]
    weights, other = [rand(n, n, 0.1) for n in sizes], [rand(n, n, 0.1) for n in sizes]
    states = [tuple(torch.zeros(n, device="cuda") for _ in range(2)) for n in sizes]
    x = torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt = ops.AdamW(weights, lr=0.01, states=states, seed=5)
        x.add_(1.0)
    graph.replay()                                          # (which clears the status word)
    torch.cuda.synchronize()
    ref = ops.AdamW(other, lr=0.01, seed=5)
    for i in range(3):
        grads = [rand(n, 10 * i + n) for n in sizes]
        for o in (opt, ref):
            o.step(grads, max_norm=None if i == 0 else 1.0)
        same(opt, ref)
    assert int(opt.status.item()) == 0 and float(x[0]) == 1.0


@pytest.mark.parametrize("bits", [32, 8])
def test_clipped_step_captured_before_the_first_eager_one(bits):
    """Two graphs, each with its own workspace, and eager steps between their replays."""
    say(f"adamw: clipped steps captured before the first eager one, {bits}-bit states")
    sizes = [4096, 700, 3, 70000]
    a, b = optimizer(sizes, bits), optimizer(sizes, bits)
    grads = [rand(n, n) for n in sizes]
    a.step(grads)
    b.step(grads)
    graphs = []
    for most in (1.0, 5.0):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norm = a.step(grads, device_hyper=True, max_norm=most)
        graphs.append((graph, norm, a.norm_result, most))
    for turn in range(5):
        graph, norm, result, most = graphs[turn % 2]
        for j, g in enumerate(grads):
            g.copy_(rand(g.numel(), 100 * turn + j))
        a.load_hyper(lr=0.01 / (turn + 1))
        graph.replay()
        torch.cuda.synchronize()
        want = exact_norm(grads)
        assert abs(float(norm) - want) <= REL * want and abs(float(result[1]) - most / want) <= 2 * REL
        b.step(grads, lr=0.01 / (turn + 1), grad_scale=float(np.float32(float(result[1]))))
        same(a, b)
        a.step(grads, max_norm=2.0)                         # eager, with the optimizer's own buffers
        torch.cuda.synchronize()
        assert abs(float(a.grad_norm) - want) <= REL * want
        unclipped(b, grads, a.norm_result, 1.0)
        same(a, b)
    assert int(a.status.item()) == 0


KINDS = {"bf16 weights": (("bf16",), ("bf16",)), "fp16 gradients": (("f32",), ("f16",)), "mixed": (("f32", "bf16"), ("f16", "f32", "bf16"))}
LISTS = {"few": [4096, 700, 3, 20001], "several launches": [37 * i % 211 + 1 for i in range(300)], "large last": [9] * 130 + [3000001, 5]}


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sizes", LISTS)
def test_types_and_long_lists(kind, sizes, bits):
    say(f"clipped adamw step: {kind}, {sizes}, {bits}-bit states")
    (types, gtypes), sizes = KINDS[kind], LISTS[sizes]
    a, b = optimizer(sizes, bits, types), optimizer(sizes, bits, types)
    for turn in range(3):
        grads = [rand(n, 10 * turn + j, 0.5, gtypes[(j + turn) % len(gtypes)]) for j, n in enumerate(sizes)]      # (types change by the step)
        want = 0.5 * exact_norm(grads)
        most = 2 * want if turn == 1 else want / 3
        norm = a.step(grads, grad_scale=0.5, max_norm=most)
        torch.cuda.synchronize()
        assert abs(float(norm) - want) <= REL * want and abs(float(a.norm_result[1]) - min(1, most / want)) <= 2 * REL
        unclipped(b, grads, a.norm_result, 0.5)
        same(a, b)
    assert a.step_count == 3 and int(a.status.item()) == 0


def test_two_optimizers_on_two_streams():
    say("clipped adamw steps of two optimizers on two streams")
    sizes = [300000, 17, 70001]
    pair, alone = [optimizer(sizes, 32, seed=s) for s in (1, 50)], [optimizer(sizes, 32, seed=s) for s in (1, 50)]
    grads = [[[rand(n, 1000 * k + 10 * turn + n % 7, 1.0 + k) for n in sizes] for turn in range(6)] for k in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for turn in range(6):
        for opt, stream, g in zip(pair, streams, grads):
            with torch.cuda.stream(stream):
                opt.step(g[turn], max_norm=1.0)
    torch.cuda.synchronize()
    for opt, other, g in zip(pair, alone, grads):
        for turn in range(6):
            other.step(g[turn], max_norm=1.0)
        same(opt, other)
        assert torch.equal(opt.grad_norm, other.grad_norm) and int(opt.status.item()) == 0
