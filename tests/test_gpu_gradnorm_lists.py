"""GPU tests of the gradient norm and clipping over lists: tensors whose memory was replaced between two
calls, no tensors at all, and lists that take several launches.  Bounds as in test_gpu_gradnorm.py."""
import ctypes
import math
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int6_weight_export_amd import ops, pgq  # noqa: E402

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


@pytest.mark.parametrize("sizes", [[40, 300], [200000, 70000]], ids=str)
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_replaced_data_is_clipped_where_it_lies(sizes, t):
    """Memory that a gradient left is another tensor's and stays as it is."""
    say(f"grad clip of replaced data {sizes} {t}")
    grads = [rand(n, n, 1.0, t) for n in sizes]
    gn = ops.GradNorm(grads)
    gn.clip_(1e9)
    for turn in range(3):
        new = [rand(n, 10 * turn + n, 2.0, t) for n in sizes]
        want = exact_norm(new)
        left = [g.data for g in grads]
        kept = [x.clone() for x in left]
        for g, x in zip(grads, new):
            g.data = x.clone()
        norm = gn.clip_(want / 2)
        torch.cuda.synchronize()
        f = torch.tensor(float(gn.result[1]), device="cuda")
        assert abs(float(norm) - want) <= REL * want and abs(float(f) - 0.5) <= 2 * REL
        assert all(torch.equal(g, (x.float() * f).to(T[t])) for g, x in zip(grads, new))
        assert all(torch.equal(a, b) for a, b in zip(left, kept))
        now = exact_norm(grads)
        assert abs(float(gn.norm(1.0)[0]) - now) <= REL * now


def test_no_tensors_through_the_c_abi():
    """The norm of nothing is 0; lists of empty tensors likewise, NULL pointers among them."""
    say("grad norm and clip of no tensors")
    stream = torch.cuda.current_stream().cuda_stream
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    st = ops.new_status()
    torch.cuda.synchronize()
    for n in (0, 1, 300):
        p, m, d = (ctypes.c_void_p * n)(), (ctypes.c_int64 * n)(), (ctypes.c_int32 * n)()
        for call in ("norm", "clip"):
            for _ in range(2):
                r = torch.full((2,), 9.0, device="cuda")
                tail = (r.data_ptr(), ws.data_ptr(), ws.numel(), st.data_ptr(), stream)
                if call == "norm":
                    rc = pgq.pgq_grad_norm(p, m, d, n, 1.0, None, 0.0, *tail)
                else:
                    rc = pgq.pgq_grad_clip(p, m, d, n, 0.0, *tail)
                torch.cuda.synchronize()
                assert rc == pgq.PGQ_OK and r.tolist() == [0.0, 1.0], (n, call)
    assert int(st.item()) == 0 and not bool(ws[:17 * 256].any())


# lists of several launches of 128 tensors: the first large and the last small, the last with more workgroups (over 256) than one
# counter takes, both, and three launches with empty tensors between
LISTS = [[100000] * 128 + [5] * 3, [5] * 128 + [5000003, 7], [70001] * 130 + [3000000], [17] * 128 + [0] * 9 + [40000] * 128 + [1 << 20] * 6]


@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{s[0]}-{sum(s)}")
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_lists_of_several_launches(sizes, t):
    say(f"grad norm and clip of {len(sizes)} tensors, {sum(sizes)} elements {t}")
    buf = rand(sum(sizes), len(sizes), 0.5, t)
    grads, at = [], 0
    for n in sizes:
        grads.append(buf[at:at + n])
        at += n
    before, want = buf.clone(), exact_norm([buf])
    gn = ops.GradNorm(grads)
    for _ in range(3):
        norm, factor = gn.norm(want / 4)
        torch.cuda.synchronize()
        assert abs(float(norm) - want) <= REL * want and abs(float(factor) - 0.25) <= 2 * REL
    gn.clip_(want / 4)
    torch.cuda.synchronize()
    f = torch.tensor(float(gn.result[1]), device="cuda")
    assert abs(float(f) - 0.25) <= 2 * REL and torch.equal(buf, (before.float() * f).to(T[t]))
    assert int(gn.status.item()) == 0 and not bool(gn.workspace[:17 * 256].any())
