"""GPU tests of the gradient norm and clipping over lists that change under them: tensors whose memory was replaced between two
calls.  Bounds as in test_gpu_gradnorm.py."""
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
