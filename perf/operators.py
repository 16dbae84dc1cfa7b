"""Measured cases of the training-step and serving operators: the linear layer over quantized
weights (forward and backward) and the AdamW step over many tensors.

Each case is one call (or the calls of one pass) as a training step or a decoder makes it.  Where
`own` is false, run() computes the operators from elementary torch operations in 32 bits; where it
is true, it calls the library.  exact() computes the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

# ---- cases ------------------------------------------------------------------------------------------
# Linear layer: M tokens, K inputs, N outputs; act and slope (leaky slope of the ReLU kinds); bias
# and residual types ("" for none); y: output type; save: the pre-activation is stored for backward;
# pad: extra elements in the row stride of X and the codes (a view into a wider buffer).
# AdamW: layout names the list of tensors; bits: 32 or 8 bit states; grad: gradient type; copy: a
# bf16 copy of the weights is written.


def _fwd(name, M, K, N, act="none", slope=0.0, bias="", residual="", y="bf16", save=False, pad=0):
    return {"name": name, "op": "linear", "M": M, "K": K, "N": N, "act": act, "slope": slope, "bias": bias,
            "residual": residual, "y": y, "save": save, "pad": pad}


def _bwd(name, M, K, N, act="none", slope=0.0, bias=False, mask=False, dw="bf16", pad=0):
    return {"name": name, "op": "backward", "M": M, "K": K, "N": N, "act": act, "slope": slope, "bias": bias,
            "mask": mask, "dw": dw, "pad": pad}


def _adam(name, layout, bits, grad="f32", copy=False, size=0):
    return {"name": name, "op": "adamw", "layout": layout, "bits": bits, "grad": grad, "copy": copy, "size": size}


def listed():
    return [
        # one generated token through the 512-wide MLP's up projection: pure latency
        _fwd("token", 1, 512, 1536, act="relu2", slope=0.5, bias="bf16"),
        # a batch of 16 generated tokens through a generic 4096-wide layer added to the residual stream
        _fwd("tokens 16", 16, 4096, 4096, residual="bf16"),
        # the 11-layer d=528 model's MLP at 16384 tokens: up projection, LeakyReLU^2, kept for backward
        _fwd("up 528", 16384, 528, 1584, act="relu2", slope=0.5, bias="f32", save=True),
        # and its down projection into an fp32 residual stream
        _fwd("down 528", 16384, 1584, 528, residual="f32", y="f32"),
        # a ragged batch, odd sizes, rows that are not 16-byte aligned
        _fwd("odd", 1009, 1031, 717, act="relu", bias="f32", y="f32", pad=3),
        # a large prefill or training batch through a generic wide gate projection
        _fwd("wide", 8192, 4096, 8192, act="silu", bias="bf16"),
        # backward of the d=528 up projection: activation, bias gradient, straight-through mask
        _bwd("up 528 backward", 16384, 528, 1584, act="relu2", slope=0.5, bias=True, mask=True),
        # backward of a generic wide layer without an activation
        _bwd("wide backward", 8192, 4096, 4096),
        # a ragged batch, odd sizes
        _bwd("odd backward", 777, 519, 1023, act="silu", bias=True, mask=True, pad=1),
        # the optimizer step over the 9-layer d=512 model: fp32 masters, fp32 states
        _adam("adamw 9 layers", "gpt9", 32),
        # the same step for the 11-layer d=528 model's matrices with 8-bit states, bf16 gradients and
        # the bf16 weights that the next forward pass reads
        _adam("adamw 8 bit 11 layers", "gpt11", 8, grad="bf16", copy=True),
        # the vectors alone (norms, scales, biases of odd sizes): many tiny tensors, latency
        _adam("adamw vectors", "vectors", 32, size=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mkn(rng, most):
    while True:
        M = rng.choice([_log(rng, 1, 64), _log(rng, 64, 16384)])
        K, N = _log(rng, 32, 8192), _log(rng, 32, 8192)
        if rng.random() < 0.5:      # widths are more often round than not
            K, N = max(16, K // 16 * 16), max(16, N // 16 * 16)
        if M * K * N <= most:
            return M, K, N


def draw(rng):
    op = rng.choice(["linear", "linear", "backward", "backward", "adamw"])
    act = rng.choice(["none", "relu", "relu2", "silu"])
    slope = rng.choice([0.0, 0.5]) if act in ("relu", "relu2") else 0.0
    pad = rng.choice([0, 0, 0, 1, 8, 16])
    if op == "linear":
        M, K, N = _mkn(rng, 8192 * 4096 * 8192)
        c = _fwd("", M, K, N, act=act, slope=slope, bias=rng.choice(["", "f32", "bf16"]),
                 residual=rng.choice(["", "", "f32", "bf16"]), y=rng.choice(["bf16", "bf16", "f32"]),
                 save=rng.random() < 0.3, pad=pad)
    elif op == "backward":
        M, K, N = _mkn(rng, 8192 * 4096 * 4096)
        c = _bwd("", M, K, N, act=act, slope=slope, bias=rng.random() < 0.5, mask=rng.random() < 0.5,
                 dw=rng.choice(["bf16", "f32"]) if act == "none" else "bf16", pad=pad)
    else:
        c = _adam("", rng.choice(["mixed", "vectors"]), rng.choice([32, 8]), grad=rng.choice(["f32", "bf16"]),
                  copy=rng.random() < 0.5, size=_log(rng, 64, 2048))
    del c["name"]
    return c


_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _shapes(case):
    """Elements of each tensor of an AdamW case."""
    lay, d = case["layout"], case["size"]
    if lay == "gpt9":       # tied embedding, per layer four attention and two MLP matrices, two vectors
        return [1024 * 512] + [512 * 512, 256 * 512, 256 * 512, 512 * 512, 1536 * 512, 512 * 1536, 512, 512] * 9
    if lay == "gpt11":      # unified Q/K/V projection, attention output, MLP up and down
        return [1584 * 528, 528 * 528, 1584 * 528, 528 * 1584] * 11
    if lay == "mixed":      # a few layers of any width with odd heads, vectors and a scalar
        return [d * 1000 + 1, d * d, d * (d + 7), 3 * d * d // 2, d, d + 1, 1] * 2
    return [d, d, d // 2 + 1, 3, 1] * 9


# ---- inputs -----------------------------------------------------------------------------------------


def _weights(N, K, pad, g, dev):
    """int6 codes (N x K, row stride K + pad), fp16 row scales."""
    w = torch.randn(N, K, generator=g, device=dev) * 0.02
    s = (w.abs().amax(1) / 31).half()
    codes = torch.empty(N, K + pad, dtype=torch.int8, device=dev)
    codes.random_(-31, 32, generator=g)
    codes[:, :K] = (w / s.float()[:, None]).round().clamp(-31, 31).to(torch.int8)
    return codes[:, :K], s


def _activations(M, K, pad, std, g, dev):
    return (torch.randn(M, K + pad, generator=g, device=dev) * std).bfloat16()[:, :K]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    if case["op"] == "adamw":
        return _prepare_adam(case, g, dev)
    M, K, N, pad = case["M"], case["K"], case["N"], case["pad"]
    codes, scales = _weights(N, K, pad, g, dev)
    s = {"case": case, "codes": codes, "scales": scales, "x": _activations(M, K, pad, 1.0, g, dev)}
    spread = 0.02 * math.sqrt(K)     # of the pre-activation
    if case["op"] == "linear":
        s["bias"] = s["residual"] = None
        if case["bias"]:
            s["bias"] = (torch.randn(N, generator=g, device=dev) * 0.1).to(_TYPES[case["bias"]])
        if case["residual"]:
            s["residual"] = torch.randn(M, N, generator=g, device=dev).to(_TYPES[case["residual"]])
        return s
    s["dy"] = _activations(M, N, 0, 0.01, g, dev)
    s["z"] = _activations(M, N, 0, spread, g, dev) if case["act"] != "none" else None
    s["mask"] = None
    if case["mask"]:                 # rare zeros, as clipping by the absolute maximum or a percentile leaves
        keep = torch.rand(N, (K + 7) // 8 * 8, generator=g, device=dev) > 0.01
        s["mask"] = (keep.view(N, -1, 8).to(torch.int32) << torch.arange(8, device=dev, dtype=torch.int32)).sum(2).to(torch.uint8)
    return s


# ---- the linear layer -------------------------------------------------------------------------------


def _act(z, kind, slope):
    if kind == "none":
        return z
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    r = torch.where(z > 0, z, z * slope)
    return r if kind == "relu" else r * r


def _act_grad(z, kind, slope):
    if kind == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    d = torch.where(z > 0, torch.ones_like(z), torch.full_like(z, slope))
    return d if kind == "relu" else 2 * z * d * d


def _what(s):
    """The layer's weights: bf16 of code * scale, as the quantization-aware forward uses them."""
    return (s["codes"].float() * s["scales"].float()[:, None]).bfloat16()


def _linear(s):
    c = s["case"]
    z = s["x"].float() @ _what(s).float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"], c["slope"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(_TYPES[c["y"]])}
    if c["save"]:
        out["z"] = z.bfloat16()
    return out


def _backward(s):
    c = s["case"]
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_grad(s["z"].float(), c["act"], c["slope"])
    dw = dz.t() @ s["x"].float()
    if s["mask"] is not None:
        bits = (s["mask"][:, :, None] >> torch.arange(8, device=dw.device, dtype=torch.uint8)) & 1
        dw = torch.where(bits.view(c["N"], -1)[:, :c["K"]] != 0, dw, torch.zeros_like(dw))
    out = {"dx": (dz @ _what(s).float()).bfloat16(), "dw": dw.to(_TYPES[c["dw"]])}
    if c["bias"]:
        out["dbias"] = dz.sum(0)
    return out


# ---- AdamW ------------------------------------------------------------------------------------------
# States in 8 bits: per 64 consecutive elements of a tensor one power of two 2^e (a byte, e + 127), m
# as a sign, four exponent and three mantissa bits, r = sqrt(v) as four exponent and four mantissa
# bits; a code with magnitude bits c stands for the binary32 number whose exponent and leading
# mantissa bits are c, times 2^(120 + e).  Rounding is up or down at random, from 16 bits of a hash
# of the seed, the tensor and the element; r > 0 is never rounded to zero.

_LR, _BETAS, _EPS, _WD, _STEP, _SEED = 1e-3, (0.9, 0.999), 1e-8, 0.01, 10, 77
_U32 = 0xFFFFFFFF


def _round_up(n, m):
    return (n + m - 1) // m * m


def _prepare_adam(case, g, dev):
    sizes = _shapes(case)
    off, total = [], 0
    for n in sizes:                  # one arena for all tensors, each at a multiple of 64 elements
        off.append(total)
        total += _round_up(n, 64)
    owner = torch.full((total,), -1, dtype=torch.int64, device=dev)
    index = torch.zeros(total, dtype=torch.int64, device=dev)
    for i, (o, n) in enumerate(zip(off, sizes)):
        owner[o:o + n] = i
        index[o:o + n] = torch.arange(n, device=dev)
    live = owner >= 0

    def arena(t):
        return torch.where(live, t, torch.zeros_like(t))

    s = {"case": case, "owner": owner.clamp(min=0), "index": index, "live": live, "t": _STEP,
         "w": arena(torch.randn(total, generator=g, device=dev) * 0.02),
         "grad": arena(torch.randn(total, generator=g, device=dev) * 0.001).to(_TYPES[case["grad"]]),
         "lr_scale": torch.tensor([1.0 if n > 4096 else 2.0 for n in sizes], device=dev),
         "wd": torch.tensor([_WD if n > 4096 else 0.0 for n in sizes], device=dev),
         "copy": torch.zeros(total, dtype=torch.bfloat16, device=dev) if case["copy"] else None}
    m = arena(torch.randn(total, generator=g, device=dev) * 0.0005)
    r = arena((torch.randn(total, generator=g, device=dev) * 0.0007).abs() + 0.0003)
    if case["bits"] == 8:
        half = torch.full_like(owner, 0x8000)
        s["m"], s["m_scale"] = _encode(m, half, 3)
        s["v"], s["v_scale"] = _encode(r, half, 4)
        s["m_out"] = torch.zeros(total, dtype=torch.bfloat16, device=dev)
        s["r_out"] = torch.zeros(total, dtype=torch.bfloat16, device=dev)
    else:
        s["m"], s["v"] = m, r * r
    if own:
        s["step"] = _plan(s, off, sizes)
    return s


def _plan(s, off, sizes):
    """What a training program keeps: the optimizer over its list of tensors."""
    from int6_weight_export_amd import ops

    def views(key, per=1):
        return [s[key][o // per:o // per + (n + per - 1) // per] for o, n in zip(off, sizes)]

    eight = s["case"]["bits"] == 8
    states = list(zip(views("m"), views("v"), *([views("m_scale", 64), views("v_scale", 64)] if eight else [])))
    opt = ops.AdamW(views("w"), lr=_LR, betas=_BETAS, eps=_EPS, weight_decay=s["wd"].tolist(),
                    lr_scale=s["lr_scale"].tolist(), state_bits=s["case"]["bits"], states=states,
                    copies=views("copy") if s["copy"] is not None else None, step_count=_STEP, seed=_SEED)
    grads = views("grad")
    if not eight:
        return lambda: opt.step(grads)
    m_out, r_out = views("m_out"), views("r_out")

    def step():
        opt.step(grads)
        opt.decode_states(m_out, r_out)

    return step


def _hash16(s, t):
    """Two 16-bit random numbers for each element at step t."""
    seed = (_SEED + t) & _U32
    x = (s["owner"] + 1) * 0x9E3779B1 + seed
    x = _mix(x & _U32)
    x = _mix(x ^ (s["index"] & _U32))
    return x >> 16, x & 0xFFFF


def _mix(x):
    x = ((x ^ (x >> 16)) * 0x6A09E667) & _U32
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & _U32
    return x ^ (x >> 16)


def _encode(x, rnd, mant):
    """Codes (uint8) and scale bytes of the arena x with `mant` mantissa bits; rnd: 16 random bits."""
    a = x.abs()
    top = a.view(-1, 64).amax(1)
    byte = ((top.view(torch.int32) >> 23) - 7).clamp(min=0)
    e = (byte - 127).repeat_interleave(64)
    y = (a.double() * torch.exp2(-(120 + e).double())).float()
    c = (y.view(torch.int32).long() + (rnd << (7 - mant))) >> (23 - mant)
    if mant == 4:
        c = torch.where((x > 0) & (c == 0), torch.ones_like(c), c)
    else:
        c = c | ((x.view(torch.int32) < 0).long() << 7)
    return c.to(torch.uint8), byte.to(torch.uint8)


def _decode(code, byte, mant):
    c = code.int()
    e = (byte.int() - 127).repeat_interleave(64)
    mag = c if mant == 4 else c & 0x7F
    v = ((mag << (23 - mant)).view(torch.float32).double() * torch.exp2((120 + e).double())).float()
    return v if mant == 4 else torch.where(c >= 128, -v, v)


def _adamw(s):
    c = s["case"]
    s["t"] += 1
    t, (b1, b2) = s["t"], _BETAS
    lr = s["lr_scale"] * _LR
    step = (lr * (1 / (1 - b1 ** t)))[s["owner"]]
    keep = (1 - lr * s["wd"])[s["owner"]]
    if c["bits"] == 8:
        m, r = _decode(s["m"], s["m_scale"], 3), _decode(s["v"], s["v_scale"], 4)
        v = r * r
    else:
        m, v = s["m"], s["v"]
    gr = s["grad"].float()
    m1 = m * b1 + gr * (1 - b1)
    v1 = v * b2 + (gr * gr) * (1 - b2)
    ok = torch.isfinite(m1) & torch.isfinite(v1) & s["live"]
    root = torch.sqrt(v1)
    w1 = s["w"] * keep - (m1 / (root * (1 / math.sqrt(1 - b2 ** t)) + _EPS)) * step
    s["w"].copy_(torch.where(ok, w1, s["w"]))
    out = {"w": s["w"]}
    if c["copy"]:
        s["copy"].copy_(s["w"])
        out["copy"] = s["copy"]
    m1 = torch.where(ok, m1, m)
    if c["bits"] == 8:
        r1 = torch.where(ok, root, r)
        um, ur = _hash16(s, t)
        for key, x, u, mant in (("m", m1, um, 3), ("v", r1, ur, 4)):
            code, byte = _encode(x, u, mant)
            s[key].copy_(code)
            s[key + "_scale"].copy_(byte)
        s["m_out"].copy_(_decode(s["m"], s["m_scale"], 3))
        s["r_out"].copy_(_decode(s["v"], s["v_scale"], 4))
        return {**out, "m": s["m_out"], "r": s["r_out"]}
    s["m"].copy_(m1)
    s["v"].copy_(torch.where(ok, v1, v))
    return {**out, "m": s["m"], "v": s["v"]}


# ---- one pass ---------------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    return _linear(state) if op == "linear" else _backward(state) if op == "backward" else _adamw(state)


def _run_own(s, op):
    from int6_weight_export_amd import ops

    c = s["case"]
    if op == "linear":
        got = ops.qlinear(s["x"], s["codes"], s["scales"], bias=s["bias"], act=c["act"], slope=c["slope"],
                          residual=s["residual"], out_dtype=_TYPES[c["y"]], want_z=c["save"])
        return {"y": got[0], "z": got[1]} if c["save"] else {"y": got}
    if op == "backward":
        return ops.qlinear_backward(s["dy"], s["codes"], s["scales"], x=s["x"], z=s["z"], act=c["act"],
                                    slope=c["slope"], mask=s["mask"], want_dbias=c["bias"],
                                    dw_dtype=_TYPES[c["dw"]])
    s["step"]()
    out = {"w": s["w"]}
    if c["copy"]:
        out["copy"] = s["copy"]
    return {**out, "m": s["m_out"], "r": s["r_out"]} if c["bits"] == 8 else {**out, "m": s["m"], "v": s["v"]}


def work(case):
    if case["op"] == "adamw":
        n = sum(_shapes(case))
        g = 4 if case["grad"] == "f32" else 2
        # weight, gradient and states in, weight and states out; 8 bits: a byte a state each way, a
        # scale byte for 64, and the decoded states
        states = 16 if case["bits"] == 32 else 4 + 4 / 64 + 4
        return {"bytes": n * (8 + g + states + (2 if case["copy"] else 0)), "flops": 12 * n}
    M, K, N = case["M"], case["K"], case["N"]
    if case["op"] == "linear":
        y = 4 if case["y"] == "f32" else 2
        b = {"": 0, "f32": 4, "bf16": 2}
        return {"bytes": 2 * M * K + N * K + 2 * N + b[case["bias"]] * N + b[case["residual"]] * M * N + y * M * N
                + (2 * M * N if case["save"] else 0), "flops": 2 * M * N * K}
    return {"bytes": 2 * M * N * (2 if case["act"] != "none" else 1) + 4 * M * K + N * K + 2 * N
            + (N * K // 8 if case["mask"] else 0) + (4 if case["dw"] == "f32" else 2) * N * K
            + (4 * N if case["bias"] else 0), "flops": 4 * M * N * K}


# ---- the definitions in 64 bits ---------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adam(s)
    # code * scale is exact in 64 bits; its bf16 is the weight
    w = torch.mul(s["codes"].double(), s["scales"].double().unsqueeze(1)).to(torch.bfloat16).double()
    x = s["x"].double()
    if case["op"] == "linear":
        z = torch.matmul(x, w.transpose(0, 1))
        if case["bias"]:
            z += s["bias"].double()
        k = case["slope"]
        a = {"none": lambda: z, "silu": lambda: z * torch.sigmoid(z),
             "relu": lambda: z.clamp(min=0) + k * z.clamp(max=0),
             "relu2": lambda: z.clamp(min=0) ** 2 + (k * z.clamp(max=0)) ** 2}[case["act"]]()
        if case["residual"]:
            a = a + s["residual"].double()
        return {"y": a, "z": z} if case["save"] else {"y": a}
    d = s["dy"].double()
    if case["act"] != "none":
        z, k = s["z"].double(), case["slope"]
        sg = torch.sigmoid(z)
        d = d * {"silu": lambda: sg + z * sg * (1 - sg),
                 "relu": lambda: (z > 0).double() + k * (z <= 0).double(),
                 "relu2": lambda: 2 * z.clamp(min=0) + 2 * k * k * z.clamp(max=0)}[case["act"]]()
    dw = torch.matmul(d.transpose(0, 1), x)
    if case["mask"]:
        m = torch.stack([(s["mask"] & (1 << b)) != 0 for b in range(8)], 2).flatten(1)[:, :case["K"]]
        dw = dw * m.double()
    out = {"dx": torch.matmul(d, w), "dw": dw}
    if case["bias"]:
        out["dbias"] = torch.sum(d, dim=0)
    return out


def _exact_adam(s):
    c, t = s["case"], _STEP + 1
    (b1, b2), o = _BETAS, s["owner"]
    lr = _LR * s["lr_scale"].double()[o]

    def value(code, byte, bits):     # (-1)^sign 2^(E - 7 + e) (1 + F), or F 2^(-6 + e) where E = 0
        full = code.double()
        neg = full >= 128 if bits == 3 else torch.zeros_like(full, dtype=torch.bool)
        mag = torch.where(neg, full - 128, full)
        E = torch.floor(mag / 2 ** bits)
        F = mag / 2 ** bits - E
        e = byte.double().repeat_interleave(64) - 127
        v = torch.where(E > 0, torch.exp2(E - 7 + e) * (1 + F), torch.exp2(e - 6) * F)
        return torch.where(neg, -v, v)

    g, w = s["grad"].double(), s["w"].double()
    if c["bits"] == 8:
        m, r = value(s["m"], s["m_scale"], 3), value(s["v"], s["v_scale"], 4)
        v = r * r
    else:
        m, v = s["m"].double(), s["v"].double()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    w = w - lr * ((m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + _EPS) + s["wd"].double()[o] * w)
    out = {"w": w}
    if c["copy"]:
        out["copy"] = w
    if c["bits"] == 32:
        return {**out, "m": m, "v": v}

    def held(x, u, bits):            # the grid value below or above, by the random number
        top = x.abs().view(-1, 64).amax(1)
        e = (torch.floor(torch.log2(top.clamp(min=1e-300))) - 7).clamp(min=-127).repeat_interleave(64)
        a = x.abs() * torch.exp2(-e)
        step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - bits)
        k = torch.floor(a / step + u.double() / 65536)
        if bits == 4:
            k = torch.where((x > 0) & (k == 0), torch.ones_like(k), k)
        return torch.sign(x) * k * step * torch.exp2(e)

    seed = (_SEED + t) % 2 ** 32
    h = _scramble(_scramble(((o + 1) * 0x9E3779B1 + seed) % 2 ** 32) ^ (s["index"] % 2 ** 32))
    return {**out, "m": held(m, h // 65536, 3), "r": held(torch.sqrt(v), h % 65536, 4)}


def _scramble(x):
    for shift, factor in ((16, 0x6A09E667), (15, 0xBB67AE85)):
        x = torch.bitwise_and(torch.bitwise_xor(x, x // 2 ** shift) * factor, 0xFFFFFFFF)
    return torch.bitwise_xor(x, x // 2 ** 16)
