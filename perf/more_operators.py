"""Measured cases of the global gradient norm with clipping and of 4-bit weights with group scales: their
quantizer, their decode and the linear layer over them for few tokens.

Each case is one call as a training step, an export or a decoder makes it.  Where `own` is false, run()
computes the operators from elementary torch operations; where it is true, it calls the library.  exact()
computes the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

# ---- cases ------------------------------------------------------------------------------------------
# norm, clip: layout names the list of gradient tensors, size its width; type: of the gradients; loose: the
# norm lies below the bound (nothing to clip); packed: the tensors lie one behind the other in a flat
# buffer, else each begins at a multiple of 64 elements.
# quantize, decode: a rows x cols matrix in groups of `group` columns; type: of the weights or of the
# decoded values; dq: type of the values that quantize writes beside the codes; pad: extra elements in the
# row stride of the weights, extra bytes in that of the codes.
# linear: M tokens, K inputs, N outputs; the rest as in perf/operators.py; pad: extra elements in the row
# stride of X and extra bytes in that of the codes.


def _grads(name, op, layout, type="f32", size=0, loose=False, packed=False):
    return {"name": name, "op": op, "layout": layout, "type": type, "size": size, "loose": loose, "packed": packed}


def _quantize(name, rows, cols, group, type="f32", dq="bf16", pad=0):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "group": group, "type": type, "dq": dq, "pad": pad}


def _decode(name, rows, cols, group, type="bf16", pad=0):
    return {"name": name, "op": "decode", "rows": rows, "cols": cols, "group": group, "type": type, "pad": pad}


def _linear(name, M, K, N, group, act="none", slope=0.0, bias="", residual="", y="bf16", pad=0):
    return {"name": name, "op": "linear", "M": M, "K": K, "N": N, "group": group, "act": act, "slope": slope,
            "bias": bias, "residual": residual, "y": y, "pad": pad}


def listed():
    return [
        # the vectors of a model alone (norms, scales, biases of odd sizes) in one flat buffer: latency
        _grads("clip vectors", "clip", "vectors", size=512, packed=True),
        # the fp32 gradients of the 9-layer d=512 model, clipped in place
        _grads("clip 9 layers", "clip", "gpt9"),
        # the bf16 gradients of the 11-layer d=528 model's matrices: norm and factor, which the optimizer step reads
        _grads("norm 11 layers", "norm", "gpt11", type="bf16"),
        # one MLP matrix of the 9-layer model in fine groups
        _quantize("quantize 1536x512", 1536, 512, 32),
        # a generic wide layer exported from bf16 weights
        _quantize("quantize wide", 8192, 8192, 128, type="bf16"),
        # a ragged matrix with rows that are not 16-byte aligned, decoded to fp32
        _decode("decode odd", 717, 1031, 64, type="f32", pad=3),
        # a generic wide layer decoded for a long prompt's library product
        _decode("decode wide", 14336, 4096, 128),
        # one generated token through the 512-wide MLP's up projection: pure latency
        _linear("token", 1, 512, 1536, 64, act="relu2", slope=0.5, bias="bf16"),
        # one token through the widest layer: the stream of the codes
        _linear("token wide", 1, 8192, 28672, 128, act="silu"),
        # a batch of 16 tokens through a generic layer added to the residual stream
        _linear("tokens 16", 16, 4096, 4096, 128, residual="bf16"),
        # a few tokens, odd sizes, unaligned rows, fine groups
        _linear("tokens odd", 5, 1031, 717, 32, act="relu", bias="f32", y="f32", pad=3),
        # the largest batch through a generic wide projection
        _linear("tokens 64", 64, 8192, 8192, 128, act="silu", bias="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    n = _log(rng, lo, hi)           # widths are more often round than not
    return max(lo, n // 32 * 32) if rng.random() < 0.6 else n


_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def draw(rng):
    op = rng.choice(["norm", "clip", "quantize", "decode", "linear", "linear", "linear"])
    group = rng.choice([32, 64, 128])
    pad = rng.choice([0, 0, 0, 1, 8, 16])
    if op in ("norm", "clip"):
        c = _grads("", op, rng.choice(["mixed", "vectors"]), type=rng.choice(["f32", "f32", "bf16", "f16"]),
                   size=_log(rng, 64, 2048), loose=rng.random() < 0.25, packed=rng.random() < 0.5)
    elif op in ("quantize", "decode"):
        rows, cols = _log(rng, 16, 16384), _width(rng, 32, 16384)
        while rows * cols > 8192 * 8192:
            rows, cols = _log(rng, 16, 16384), _width(rng, 32, 16384)
        if op == "quantize":
            c = _quantize("", rows, cols, group, type=rng.choice(["f32", "bf16", "f16"]), dq=rng.choice(["bf16", "f32"]), pad=pad)
        else:
            c = _decode("", rows, cols, group, type=rng.choice(["bf16", "f32"]), pad=pad)
    else:
        while True:
            M = rng.choice([1, _log(rng, 1, 64)])
            K, N = _width(rng, 64, 16384), _width(rng, 16, 28672)
            if N * K <= 8192 * 28672 and M * N * K <= 64 * 8192 * 8192:
                break
        act = rng.choice(["none", "relu", "relu2", "silu"])
        c = _linear("", M, K, N, group, act=act, slope=rng.choice([0.0, 0.5]) if act in ("relu", "relu2") else 0.0,
                    bias=rng.choice(["", "f32", "bf16"]), residual=rng.choice(["", "", "f32", "bf16"]),
                    y=rng.choice(["bf16", "bf16", "f32"]), pad=pad)
    del c["name"]
    return c


def _shapes(case):
    """Elements of each gradient tensor."""
    lay, d = case["layout"], case["size"]
    if lay == "gpt9":       # tied embedding, per layer four attention and two MLP matrices, two vectors
        return [1024 * 512] + [512 * 512, 256 * 512, 256 * 512, 512 * 512, 1536 * 512, 512 * 1536, 512, 512] * 9
    if lay == "gpt11":      # unified Q/K/V projection, attention output, MLP up and down
        return [1584 * 528, 528 * 528, 1584 * 528, 528 * 1584] * 11
    if lay == "mixed":      # a few layers of any width with odd heads, vectors and a scalar
        return [d * 1000 + 1, d * d, d * (d + 7), 3 * d * d // 2, d, d + 1, 1] * 2
    return [d, d, d // 2 + 1, 3, 1] * 9


# ---- inputs -----------------------------------------------------------------------------------------
# Eight codes of a row take four bytes: byte j holds code j in its low and code j + 4 in its high half, each
# a sign bit (8) and the magnitude 0 .. 7.  A row's last bytes are filled up with zero codes.


def _pack(code):
    n, k = code.shape
    nib = code.abs().to(torch.uint8) + 8 * (code < 0).to(torch.uint8)
    nib = torch.nn.functional.pad(nib, (0, (k + 7) // 8 * 8 - k)).view(n, -1, 2, 4)
    return (nib[:, :, 0] + 16 * nib[:, :, 1]).view(n, -1)


def _codes(rows, cols, group, pad, g, dev):
    """Packed codes (row stride that many bytes and pad more) and fp16 group scales of normal weights."""
    w = torch.randn(rows, (cols + group - 1) // group * group, generator=g, device=dev) * 0.02
    w[:, cols:] = 0
    w = w.view(rows, -1, group)
    s = (w.abs().amax(2) / 7).half()
    code = torch.round(w / s.float().unsqueeze(2)).clamp_(-7, 7).to(torch.int8).view(rows, -1)[:, :cols]
    del w
    packed = _pack(code)
    buf = torch.zeros(rows, packed.shape[1] + pad, dtype=torch.uint8, device=dev)
    buf[:, :packed.shape[1]] = packed
    return buf[:, :packed.shape[1]], s


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case}
    if op in ("norm", "clip"):
        sizes = _shapes(case)
        step = 1 if case["packed"] else 64
        off, total = [], 0
        for n in sizes:
            off.append(total)
            total += (n + step - 1) // step * step
        live = torch.zeros(total, dtype=torch.bool, device=dev)
        for o, n in zip(off, sizes):
            live[o:o + n] = True
        # a norm of about 2, as early training has it, against a bound of 1 (or 10)
        v = torch.randn(total, generator=g, device=dev) * (2 / math.sqrt(sum(sizes)))
        s["grads"] = torch.where(live, v, torch.zeros_like(v)).to(_TYPES[case["type"]])
        s["max"] = 10.0 if case["loose"] else 1.0
        if own:
            from int6_weight_export_amd import ops

            s["norm"] = ops.GradNorm([s["grads"][o:o + n] for o, n in zip(off, sizes)])
        return s
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        s["w"] = (torch.randn(rows, cols + case["pad"], generator=g, device=dev) * 0.02).to(_TYPES[case["type"]])[:, :cols]
        if own:
            from int6_weight_export_amd import ops

            s["status"] = ops.new_status()
        return s
    if op == "decode":
        s["codes"], s["scales"] = _codes(case["rows"], case["cols"], case["group"], case["pad"], g, dev)
        return s
    M, K, N, pad = case["M"], case["K"], case["N"], case["pad"]
    s["codes"], s["scales"] = _codes(N, K, case["group"], pad, g, dev)
    s["x"] = torch.randn(M, K + pad, generator=g, device=dev).bfloat16()[:, :K]
    s["bias"] = s["residual"] = None
    if case["bias"]:
        s["bias"] = (torch.randn(N, generator=g, device=dev) * 0.1).to(_TYPES[case["bias"]])
    if case["residual"]:
        s["residual"] = torch.randn(M, N, generator=g, device=dev).to(_TYPES[case["residual"]])
    return s


# ---- plain forms ------------------------------------------------------------------------------------


def _falling(s):
    """This pass's bound: a little lower each time, so that gradients clipped in place are clipped again."""
    s["max"] *= 0.9999
    return s["max"]


def _norm_factor(grads, most):
    d = grads.double()
    norm = torch.sqrt((d * d).sum())
    factor = torch.where(norm > most, most / norm, torch.ones_like(norm))
    return norm.float(), torch.where(torch.isfinite(norm), factor, torch.full_like(norm, math.nan)).float()


def _clip(s):
    norm, factor = _norm_factor(s["grads"], _falling(s))
    keep = torch.isfinite(factor)
    s["grads"].copy_(torch.where(keep, s["grads"].float() * factor, s["grads"].float()))
    return {"norm": norm, "grads": s["grads"]}


def _plain_quantize(s):
    c = s["case"]
    rows, cols, group = c["rows"], c["cols"], c["group"]
    w = torch.nn.functional.pad(s["w"].float(), (0, -cols % group)).view(rows, -1, group)
    top = w.abs().amax(2)
    scale = (top / torch.full_like(top, 7)).half()      # (a quotient by a number may be a product with its inverse)
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    code = torch.round(w / scale.float().unsqueeze(2)).clamp(-7, 7)
    value = (code * scale.float().unsqueeze(2)).view(rows, -1)[:, :cols]
    return {"dq": value.to(_TYPES[c["dq"]]), "scales": scale}


def _values(s, rows, cols, group):
    """fp32 weights of packed codes: code * scale, exact."""
    b = s["codes"].view(rows, -1, 4)
    nib = torch.cat([b & 15, b >> 4], 2).view(rows, -1)[:, :cols]
    v = (nib & 7).float()
    v = torch.where(nib >= 8, -v, v)
    return v * s["scales"].float().repeat_interleave(group, 1)[:, :cols]


def _act(z, kind, slope):
    if kind == "none":
        return z
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    r = torch.where(z > 0, z, z * slope)
    return r if kind == "relu" else r * r


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ _values(s, c["N"], c["K"], c["group"]).t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"], c["slope"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(_TYPES[c["y"]])}


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        return _run_own(state, c, op)
    if op == "norm":
        norm, factor = _norm_factor(state["grads"], state["max"])
        return {"norm": norm, "factor": factor}
    if op == "clip":
        return _clip(state)
    if op == "quantize":
        return _plain_quantize(state)
    if op == "decode":
        return {"value": _values(state, c["rows"], c["cols"], c["group"]).to(_TYPES[c["type"]])}
    return _plain_linear(state)


def _run_own(s, c, op):
    from int6_weight_export_amd import ops

    if op == "norm":
        norm, factor = s["norm"].norm(max_norm=s["max"])
        return {"norm": norm, "factor": factor}
    if op == "clip":
        return {"norm": s["norm"].clip_(_falling(s)), "grads": s["grads"]}
    if op == "quantize":
        got = ops.quantize_groups(s["w"], group=c["group"], dq_dtype=_TYPES[c["dq"]], status=s["status"])
        return {"dq": got["dq"], "scales": got["scales"].view(torch.float16)}
    if op == "decode":
        return {"value": ops.dequant_groups(s["codes"], s["scales"], c["cols"], group=c["group"], out_dtype=_TYPES[c["type"]])}
    return {"y": ops.qlinear4(s["x"], s["codes"], s["scales"], group=c["group"], bias=s["bias"], act=c["act"], slope=c["slope"],
                              residual=s["residual"], out_dtype=_TYPES[c["y"]])}


_SIZE = {"": 0, "f32": 4, "bf16": 2, "f16": 2}


def work(case):
    op = case["op"]
    if op in ("norm", "clip"):
        n = sum(_shapes(case))
        written = op == "clip" and not case["loose"]
        return {"bytes": n * _SIZE[case["type"]] * (2 if written else 1), "flops": n * (3 if written else 2)}
    group = case["group"]
    rows, cols = (case["N"], case["K"]) if op == "linear" else (case["rows"], case["cols"])
    held = rows * ((cols + 7) // 8 * 4 + (cols + group - 1) // group * 2)       # codes and scales
    if op == "quantize":
        return {"bytes": rows * cols * (_SIZE[case["type"]] + _SIZE[case["dq"]]) + held, "flops": 5 * rows * cols}
    if op == "decode":
        return {"bytes": rows * cols * _SIZE[case["type"]] + held, "flops": rows * cols}
    M = case["M"]
    return {"bytes": held + 2 * M * cols + _SIZE[case["bias"]] * rows + (_SIZE[case["residual"]] + _SIZE[case["y"]]) * M * rows,
            "flops": 2 * M * rows * cols}


# ---- the definitions in 64 bits ---------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "clip"):
        g = s["grads"].double()
        most = s["max"] * (0.9999 if op == "clip" else 1.0)
        norm = torch.linalg.vector_norm(g)
        factor = torch.clamp(most / norm, max=1.0)
        return {"norm": norm, "factor": factor} if op == "norm" else {"norm": norm, "grads": torch.mul(g, factor)}
    if op == "quantize":
        return _exact_quantize(case, s)
    if op == "decode":
        return {"value": _exact_values(s["codes"], s["scales"], case["cols"], case["group"])}
    w = _exact_values(s["codes"], s["scales"], case["K"], case["group"])
    z = torch.matmul(s["x"].double(), w.transpose(0, 1))
    if case["bias"]:
        z += s["bias"].double()
    k = case["slope"]
    y = {"none": lambda: z, "silu": lambda: z * torch.sigmoid(z), "relu": lambda: z.clamp(min=0) + k * z.clamp(max=0),
         "relu2": lambda: z.clamp(min=0) ** 2 + (k * z.clamp(max=0)) ** 2}[case["act"]]()
    return {"y": y + s["residual"].double() if case["residual"] else y}


def _exact_quantize(case, s):
    """Per group of columns, one after the other: the scale, an fp16 of the binary32 quotient by its definition, and
    the multiples of it that the weights are rounded to."""
    w, group = s["w"].double(), case["group"]
    scales, values = [], []
    for k in range(0, case["cols"], group):
        part = w[:, k:k + group]
        top = part.abs().max(dim=1).values
        sc = torch.div(top, torch.full_like(top, 7)).to(torch.float32).to(torch.float16).double()
        sc[sc == 0] = 1.0
        scales.append(sc)
        values.append(torch.div(part, sc[:, None]).round().clamp(min=-7, max=7) * sc[:, None])
    return {"dq": torch.hstack(values), "scales": torch.stack(scales, dim=1)}


def _exact_values(codes, scales, cols, group):
    out = torch.empty(codes.shape[0], cols, dtype=torch.float64, device=codes.device)
    for e in range(8):              # code e of every eight: four bits of byte e mod 4
        nib = torch.div(codes[:, e % 4::4], 16 ** (e // 4), rounding_mode="floor") % 16
        mag = (nib % 8).double()
        k = torch.arange(e, cols, 8, device=codes.device)
        out[:, e::8] = ((1 - 2 * (nib // 8).double()) * mag)[:, :len(k)] * scales.double()[:, k // group]
    return out
