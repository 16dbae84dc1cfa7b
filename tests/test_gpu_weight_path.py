"""One weight's way through the operators, as a training run with an export at its end uses them: bf16 gradients of a
two-layer MLP over fake-quantized weights, clipped on the way into AdamW, for some steps; the fp32 masters then quantized to
4-bit groups, decoded, and served token by token.  Every stage is checked against its definition on what the stage before
it left on the device."""
import math
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from int6_weight_export_amd import ops, pgq  # noqa: E402
from tests import adamw_ref, group4_ref as g4, linear_ref as ref  # noqa: E402
from tests.gpu_util import same_bits  # noqa: E402


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("M,D,H,group", [(96, 64, 200, 32), (130, 136, 264, 64), (64, 256, 384, 128)])
def test_train_clip_export_serve(M, D, H, group):
    print(f"[case] train, clip, export, serve M={M} D={D} H={H} group {group}", flush=True)
    sys.stdout.flush()
    gen = torch.Generator().manual_seed(M)
    masters = [(torch.randn(s, generator=gen) * 0.05).cuda() for s in ((H, D), (D, H))]
    bias = (torch.randn(H, generator=gen) * 0.1).cuda()
    copies = [m.bfloat16() for m in masters]
    opt = ops.AdamW(masters + [bias], lr=0.01, copies=copies + [None], seed=9)
    fq = ops.FakeQuant(copies, want_codes=True)
    for step in range(3):
        x = torch.randn(M, D, generator=gen).bfloat16().cuda()
        target = torch.randn(M, D, generator=gen).cuda()
        fq.run(pgq.PGQ_FQ_FWD)
        h, z = ops.qlinear(x, fq.codes[0], fq.scales[0], bias=bias, act="relu2", slope=0.5, want_z=True)
        dy = ops.qlinear(h, fq.codes[1], fq.scales[1], residual=x, out_dtype=torch.float32) - target
        g2 = ops.qlinear_backward(dy, fq.codes[1], fq.scales[1], x=h, mask=fq.mask[1])
        g1 = ops.qlinear_backward(g2["dx"], fq.codes[0], fq.scales[0], x=x, z=z, act="relu2", slope=0.5, mask=fq.mask[0],
                                  want_dbias=True, want_dx=False)
        grads = [g1["dw"], g2["dw"], g1["dbias"]]
        before = [w.clone() for w in opt.weights]
        states = [[t.clone() for t in s] for s in opt.states]
        norm = opt.step(grads, max_norm=1.0)
        torch.cuda.synchronize()
        want = math.sqrt(sum(float((f64(g) ** 2).sum()) for g in grads))
        assert want > 1.0 and abs(float(norm) - want) <= 2.0 ** -23 * want
        factor = float(opt.norm_result[1])
        assert abs(factor - 1 / want) <= 2.0 ** -23 * factor
        hy = adamw_ref.hyper(0.01, (0.9, 0.999), 1e-8, step + 1, factor)
        for i, (w, g) in enumerate(zip(opt.weights, grads)):
            m, v = (t.cpu().numpy() for t in states[i])
            w1, m1, v1, _, _ = adamw_ref.step32(before[i].cpu().numpy().reshape(-1), g.float().cpu().numpy().reshape(-1), m, v, hy, 1.0, 0.01)
            same_bits(w.cpu().numpy().reshape(-1), w1, f"step {step} weight {i}")
            same_bits(opt.states[i][0].cpu().numpy(), m1, "m")
            same_bits(opt.states[i][1].cpu().numpy(), v1, "v")
        # the same gradients clipped in place give the same step, through bf16 gradients rounded once more
        gn = ops.GradNorm(grads)
        kept = [g.clone() for g in grads]
        gn.clip_(1.0)
        torch.cuda.synchronize()
        assert float(gn.result[1]) == factor
        for a, b in zip(grads, kept):
            assert torch.equal(a, (b.float() * torch.tensor(factor, device="cuda")).to(a.dtype))

    stored, values = [], []
    for m in masters:
        q = ops.quantize_groups(m, group=group)
        dq = ops.dequant_groups(q["codes"], q["scales"], m.shape[1], group=group)
        torch.cuda.synchronize()
        codes, scales, v, _ = g4.quantize(m.cpu().numpy(), group)
        assert np.array_equal(q["codes"].cpu().numpy(), g4.pack(codes)) and int(q["status"].item()) == 0
        same_bits(dq.cpu().numpy(), v, "decoded masters")
        # no weight is further from its master than half a step of its group's scale, where the scale was not rounded down
        s = np.repeat(scales.view(np.float16).astype(np.float64), group, axis=1)[:, :m.shape[1]]
        assert (np.abs(v - f64(m)) <= s * (0.5 + 7 * 2.0 ** -11) * (1 + 2.0 ** -20)).all()
        stored.append(q)
        values.append(v.astype(np.float64))
    for tokens in (1, 7, 64):
        x = torch.randn(tokens, D, generator=gen).bfloat16().cuda()
        h = ops.qlinear4(x, stored[0]["codes"], stored[0]["scales"], group=group, bias=bias, act="relu2", slope=0.5)
        y = ops.qlinear4(h, stored[1]["codes"], stored[1]["scales"], group=group, residual=x, out_dtype=torch.float32)
        torch.cuda.synchronize()
        _, _, hr, eh = ref.forward(f64(x), values[0], f64(bias), "relu2", 0.5)
        assert np.all(np.abs(f64(h) - hr) <= eh)
        _, _, yr, ey = ref.forward(f64(h), values[1], None, "none", 0.0, f64(x), "f32")
        assert np.all(np.abs(f64(y) - yr) <= ey)
    assert int(opt.status.item()) == 0 and int(fq.status.item()) == 0
