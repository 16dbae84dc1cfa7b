"""The linear layer and its gradient in 64 bits (numpy), with error bounds for a binary32 computation
of each output, for the GPU tests.

Bounds.  u = 2^-24.  A product of two bf16 values is exact in binary32, so a sum of L of them in any
order errs by at most (L - 1) u sum |a b|; one more u each covers the bias and the residual.  An
activation multiplies the error of its argument by its slope and adds the error of its own few
operations, taken as 8 u of its value (exp and a division are within 2 u each).  A store to type t
adds eps(t) / 2 of the value, and half the smallest subnormal.  In backward, dZ is rounded to bf16
(2^-8) before the products whenever it is not a bf16 value already.
"""
import numpy as np

U = 2.0 ** -24
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -134}


def act(z, kind, slope):
    if kind == "none":
        return z
    if kind == "silu":
        return z / (1 + np.exp(-z))
    r = np.where(z > 0, z, z * slope)
    return r if kind == "relu" else r * r


def act_grad(z, kind, slope):
    if kind == "none":
        return np.ones_like(z)
    if kind == "silu":
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    d = np.where(z > 0, 1.0, slope)
    return d if kind == "relu" else 2 * z * d * d


def _act_error(z, e, kind, slope):
    """Bound on the error of act(z) when its argument is off by at most e."""
    big = max(1.0, abs(slope))
    if kind == "none":
        return e
    if kind == "relu":
        return big * e + 8 * U * big * np.abs(z)
    if kind == "silu":                                  # |silu'| < 1.1
        return 1.1 * e + 8 * U * np.abs(act(z, kind, slope))
    m = big * (np.abs(z) + e)
    return 2 * m * big * e + 8 * U * m * m


def stored(v, e, t):
    return e + HALF_STEP[t] * (np.abs(v) + e) + TINY[t]


def forward(x, w, bias=None, kind="none", slope=0.0, residual=None, y="bf16"):
    """(z, bound of the stored bf16 z, y, bound of the stored y); x, w in float64."""
    z = x @ w.T
    mag = np.abs(x) @ np.abs(w).T
    if bias is not None:
        z = z + bias
        mag = mag + np.abs(bias)
    e = (x.shape[1] + 1) * U * mag
    a = act(z, kind, slope)
    ea = _act_error(z, e, kind, slope)
    if residual is not None:
        a = a + residual
        ea = ea + U * (np.abs(a) + ea)
    return z, stored(z, e, "bf16"), a, stored(a, ea, y)


def backward(dy, z, x, w, kind="none", slope=0.0, mask=None, dy_type="bf16", dx="bf16", dw="bf16"):
    """{name: (value, bound)} of dx, dw, dbias; mask: boolean N x K."""
    d = dy * (act_grad(z, kind, slope) if kind != "none" else 1.0)
    exact = kind == "none"
    ed = np.zeros_like(d) if exact else 16 * U * np.abs(dy) * np.maximum(np.abs(act_grad(z, kind, slope)), 1.0)
    er = ed if exact and dy_type == "bf16" else ed + HALF_STEP["bf16"] * (np.abs(d) + ed) + TINY["bf16"]
    M, N = d.shape
    out = {}
    v = d @ w
    out["dx"] = (v, stored(v, er @ np.abs(w) + (N + 1) * U * ((np.abs(d) + er) @ np.abs(w)), dx))
    v = d.T @ x
    e = er.T @ np.abs(x) + (M + 1) * U * ((np.abs(d) + er).T @ np.abs(x))
    if mask is not None:
        v, e = np.where(mask, v, 0.0), np.where(mask, e, 0.0)
    out["dw"] = (v, np.where(e > 0, stored(v, e, dw), 0.0) if mask is not None else stored(v, e, dw))
    out["dbias"] = (d.sum(0), ed.sum(0) + (M + 1) * U * (np.abs(d) + ed).sum(0) + TINY["f32"])
    return out
