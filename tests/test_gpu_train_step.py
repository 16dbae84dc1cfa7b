"""The training-step operators together, as a quantization-aware training loop uses them: fp32 masters,
their bf16 copies through fake quantization, a two-layer MLP forward and backward over the codes, the
straight-through mask, AdamW writing the next copies, an EMA of the masters.  Every stage is checked against
its definition on what the stage before it left on the device, over several steps."""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import oracle  # noqa: E402
from int6_weight_export_amd import ops, pgq  # noqa: E402
from tests import adamw_ref, linear_ref as ref  # noqa: E402
from tests.gpu_util import same_bits  # noqa: E402


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def within(got, want, bound, what):
    err = np.abs(f64(got) - want)
    assert np.all(err <= bound), f"{what}: worst {np.max(err / np.maximum(bound, 1e-300)):.3g} bounds"


def mask_bits(fq, i, cols):
    return np.unpackbits(fq.mask[i].cpu().numpy(), axis=1, bitorder="little")[:, :cols].astype(bool)


@pytest.mark.parametrize("state_bits", [32, 8])
@pytest.mark.parametrize("M,D,H", [(96, 64, 200), (257, 72, 133)])
def test_qat_steps(state_bits, M, D, H):
    print(f"[case] QAT steps M={M} D={D} H={H} {state_bits}-bit states", flush=True)
    sys.stdout.flush()
    gen = torch.Generator().manual_seed(M)
    shapes = [(H, D), (D, H)]
    masters = [(torch.randn(s, generator=gen) * 0.05).cuda() for s in shapes]
    bias = (torch.randn(H, generator=gen) * 0.1).cuda()
    copies = [m.bfloat16() for m in masters]
    opt = ops.AdamW(masters + [bias], lr=0.01, weight_decay=[0.1, 0.1, 0.0], lr_scale=[1.0, 1.0, 2.0],
                    state_bits=state_bits, copies=copies + [None], seed=9)
    # a clip below the maximum leaves mask zeros, so the straight-through mask does something
    fq = ops.FakeQuant(copies, pct=(9, 10), want_codes=True)
    ema = ops.Ema(masters)
    ema.update(masters, init=True)
    for step in range(3):
        x = torch.randn(M, D, generator=gen).bfloat16().cuda()
        target = torch.randn(M, D, generator=gen).cuda()
        fq.run(pgq.PGQ_FQ_FWD)
        h, z = ops.qlinear(x, fq.codes[0], fq.scales[0], bias=bias, act="relu2", slope=0.5, want_z=True)
        y = ops.qlinear(h, fq.codes[1], fq.scales[1], residual=x, out_dtype=torch.float32)
        dy = y - target
        g2 = ops.qlinear_backward(dy, fq.codes[1], fq.scales[1], x=h, mask=fq.mask[1])
        g1 = ops.qlinear_backward(g2["dx"], fq.codes[0], fq.scales[0], x=x, z=z, act="relu2", slope=0.5,
                                  mask=fq.mask[0], want_dbias=True, want_dx=False)
        before = [m.clone() for m in masters] + [bias.clone()]
        states = [[t.clone() for t in s] for s in opt.states]
        grads = [g1["dw"], g2["dw"], g1["dbias"]]
        ema_before = [e.clone() for e in ema.avg]
        opt.step(grads)
        ema.update(masters)
        torch.cuda.synchronize()

        # the layer on the codes that fake quantization left
        ws = [f64(fq.dq[i]) for i in range(2)]
        for i in range(2):
            o = oracle.fakequant_rows(bf16_bits(before[i]), 31, 9, 10)
            assert np.array_equal(fq.codes[i].cpu().numpy(), o["codes"])
        zr, ez, hr, eh = ref.forward(f64(x), ws[0], f64(before[2]), "relu2", 0.5)
        within(z, zr, ez, "z")
        within(h, hr, eh, "h")
        _, _, yr, ey = ref.forward(f64(h), ws[1], None, "none", 0.0, f64(x), "f32")
        within(y, yr, ey, "y")
        keep = [mask_bits(fq, i, shapes[i][1]) for i in range(2)]
        assert all(0 < k.sum() < k.size for k in keep)
        want = ref.backward(f64(dy), None, f64(h), ws[1], mask=keep[1], dy_type="f32")
        within(g2["dx"], *want["dx"], "dh")
        within(g2["dw"], *want["dw"], "dw2")
        want = ref.backward(f64(g2["dx"]), f64(z), f64(x), ws[0], "relu2", 0.5, keep[0])
        within(g1["dw"], *want["dw"], "dw1")
        within(g1["dbias"], *want["dbias"], "dbias")
        assert not bool(g1["dw"][torch.from_numpy(~keep[0]).cuda()].any())

        # the optimizer, bit for bit, and the copies that the next step quantizes
        hy = adamw_ref.hyper(0.01, (0.9, 0.999), 1e-8, step + 1)
        for i, (w, g) in enumerate(zip(masters + [bias], grads)):
            n = w.numel()
            s = [t.cpu().numpy() for t in states[i]]
            if state_bits == 8:
                m, r, v = adamw_ref.decode(s[0], s[2], 3), adamw_ref.decode(s[1], s[3], 4), None
            else:
                m, v, r = s[0], s[1], None
            w1, m1, v1, r1, _ = adamw_ref.step32(before[i].cpu().numpy().reshape(-1), f64(g).reshape(-1).astype(np.float32), m, v,
                                                 hy, opt_lr_scale(i), [0.1, 0.1, 0.0][i], r)
            same_bits(w.cpu().numpy().reshape(-1), w1, f"step {step} weight {i}")
            if state_bits == 8:
                um, ur = adamw_ref.random16(i, n, 9 + step + 1)
                same_bits(opt.states[i][0].cpu().numpy(), adamw_ref.encode(m1, um, 3)[0], "m")
                same_bits(opt.states[i][1].cpu().numpy(), adamw_ref.encode(r1, ur, 4)[0], "r")
            else:
                same_bits(opt.states[i][0].cpu().numpy(), m1, "m")
                same_bits(opt.states[i][1].cpu().numpy(), v1, "v")
        for c, w in zip(copies, masters):
            assert torch.equal(c, w.bfloat16())
        for e0, e1, w in zip(ema_before, ema.avg, masters):
            d = np.float32(0.997)
            want = (d * e0.cpu().numpy()) + (np.float32(1) - d) * w.cpu().numpy()
            same_bits(e1.cpu().numpy(), want.astype(np.float32), "ema")
    assert int(opt.status.item()) == 0 and int(fq.status.item()) == 0 and int(ema.status.item()) == 0


def bf16_bits(master):
    return master.bfloat16().view(torch.int16).cpu().numpy().view(np.uint16)


def opt_lr_scale(i):
    return [1.0, 1.0, 2.0][i]


def test_two_streams_at_once():
    """Two layers' forward and backward on two streams, interleaved, equal the same calls one after another."""
    print("[case] two streams at once", flush=True)
    jobs = []
    for k in range(2):
        g = torch.Generator().manual_seed(k)
        M, N, K = (700, 264, 152) if k else (513, 200, 264)
        w = oracle.f32_to_bf16((np.random.default_rng(k).standard_normal((N, K)) * 0.05).astype(np.float32))
        o = oracle.fakequant_rows(w, 31)
        jobs.append(dict(codes=torch.from_numpy(o["codes"]).cuda(), scales=torch.from_numpy(o["scales"].view(np.int16)).cuda(),
                         x=torch.randn(M, K, generator=g).bfloat16().cuda(), dy=torch.randn(M, N, generator=g).bfloat16().cuda()))

    def run(j):
        y, z = ops.qlinear(j["x"], j["codes"], j["scales"], act="silu", want_z=True)
        b = ops.qlinear_backward(j["dy"], j["codes"], j["scales"], x=j["x"], z=z, act="silu", want_dbias=True)
        return [y, z, b["dx"], b["dw"], b["dbias"]]

    alone = [run(j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        outs = [None, None]
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                for _ in range(4):
                    outs[k] = run(jobs[k])
        torch.cuda.synchronize()
        for a, b in zip(alone, outs):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
