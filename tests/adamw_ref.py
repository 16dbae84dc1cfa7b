"""The AdamW step as include/pgq.h spells it out, in numpy: one binary32 operation at a time (bit for
bit what the kernel must give), and in 64 bits."""
import numpy as np

F = np.float32


def hyper(lr, betas, eps, step, grad_scale=1.0):
    b1, b2 = betas
    return {"lr": F(lr), "beta1": F(b1), "c1": F(1 - b1), "beta2": F(b2), "c2": F(1 - b2),
            "ib1": F(1 / (1 - b1 ** step)), "ib2": F(1 / np.sqrt(1 - b2 ** step)), "eps": F(eps),
            "grad_scale": F(grad_scale)}


def step32(w, g, m, v, h, lr_scale=1.0, wd=0.0, r=None):
    """(w', m', v', r', ok) in binary32; r: the held square root of 8-bit states, or None."""
    with np.errstate(all="ignore"):
        lr = F(lr_scale) * h["lr"]
        step, keep = lr * h["ib1"], F(1) - lr * F(wd)
        if r is not None:
            v = r * r
        gs = h["grad_scale"] * g
        m1 = m * h["beta1"] + gs * h["c1"]
        v1 = v * h["beta2"] + (gs * gs) * h["c2"]
        root = np.sqrt(v1)
        w1 = w * keep - (m1 / (root * h["ib2"] + h["eps"])) * step
        ok = np.isfinite(m1) & np.isfinite(v1)
    for x in (m1, v1, root, w1):
        assert x.dtype == F
    return (np.where(ok, w1, w), np.where(ok, m1, m), np.where(ok, v1, v), np.where(ok, root, r if r is not None else root),
            ok)


def mix(x):
    x = x.astype(np.uint64) & 0xFFFFFFFF
    for shift, factor in ((16, 0x6A09E667), (15, 0xBB67AE85)):
        x = ((x ^ (x >> np.uint64(shift))) * np.uint64(factor)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def random16(tensor, numel, seed):
    t = mix(np.array([(0x9E3779B1 * (tensor + 1) + seed) & 0xFFFFFFFF], np.uint64))
    x = mix(t ^ (np.arange(numel, dtype=np.uint64) & np.uint64(0xFFFFFFFF)))
    return (x >> np.uint64(16)).astype(np.int64), (x & np.uint64(0xFFFF)).astype(np.int64)


def scale_bytes(x):
    pad = np.zeros((len(x) + 63) // 64 * 64, F)
    pad[:len(x)] = np.abs(x)
    top = pad.reshape(-1, 64).max(1) if len(pad) else pad.reshape(0, 64).sum(1)
    return np.maximum((top.view(np.int32) >> 23) - 7, 0).astype(np.uint8)


def encode(x, u, mant):
    b = scale_bytes(x)
    e = b.astype(np.int64).repeat(64)[:len(x)]
    y = np.ldexp(np.abs(x).astype(np.float64), (7 - e).astype(np.int64)).astype(F)
    c = (y.view(np.int32).astype(np.int64) + (u << (7 - mant))) >> (23 - mant)
    if mant == 4:
        c = np.where((x > 0) & (c == 0), 1, c)
    else:
        c = c | (np.signbit(x).astype(np.int64) << 7)
    assert c.min(initial=0) >= 0 and c.max(initial=0) <= 255
    return c.astype(np.uint8), b


def decode(c, b, mant):
    e = b.astype(np.int64).repeat(64)[:len(c)]
    mag = (c if mant == 4 else c & 0x7F).astype(np.int32)
    v = np.ldexp((mag << (23 - mant)).view(F).astype(np.float64), e - 7).astype(F)
    return v if mant == 4 else np.where(c >= 128, -v, v)


def step64(w, g, m, v, lr, betas, eps, step, lr_scale=1.0, wd=0.0, grad_scale=1.0):
    """(w', m', v') in 64 bits."""
    w, g, m, v = (np.asarray(t, np.float64) for t in (w, g, m, v))
    b1, b2 = betas
    g = g * grad_scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    upd = (m / (1 - b1 ** step)) / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return w - lr * lr_scale * (upd + wd * w), m, v
