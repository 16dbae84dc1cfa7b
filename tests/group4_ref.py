"""4-bit codes with group scales as include/pgq.h defines them, in numpy, for the tests."""
import numpy as np

import oracle


def quantize(w, group):
    """(codes int8 [rows, cols], scales uint16 [rows, groups], values float32 [rows, cols], status) of a float32 matrix.

    A group is a row of its own to the oracle's row quantizer with Q = 7; zeros that fill up a row's last group change
    neither its maximum nor its codes."""
    rows, cols = w.shape
    groups = -(-cols // group)
    full = np.zeros((rows, groups * group), np.float32)
    full[:, :cols] = w
    o = oracle.quantize_rows(full.reshape(-1, group), 7)
    return (o["codes"].reshape(rows, -1)[:, :cols], o["scales"].reshape(rows, groups),
            o["dq"].reshape(rows, -1)[:, :cols], o["status"])


def pack(codes):
    """Stored bytes [rows, 4 ceil(cols / 8)] of int8 codes in [-7, 7]."""
    rows, cols = codes.shape
    out = np.zeros((rows, -(-cols // 8) * 4), np.uint8)
    for k in range(cols):
        c = codes[:, k].astype(np.int64)
        nib = np.where(c < 0, 8 - c, c).astype(np.uint8)
        out[:, k // 8 * 4 + k % 4] |= nib << (4 * (k % 8 // 4))
    return out


def unpack(packed, cols):
    rows = packed.shape[0]
    out = np.empty((rows, cols), np.int8)
    for k in range(cols):
        nib = (packed[:, k // 8 * 4 + k % 4] >> (4 * (k % 8 // 4))) & 15
        out[:, k] = np.where(nib & 8, -(nib & 7).astype(np.int8), (nib & 7).astype(np.int8))
    return out


def values(codes, scales, group):
    """code * scale in float64 (exact)."""
    s = scales.view(np.float16).astype(np.float64)
    return codes.astype(np.float64) * np.repeat(s, group, axis=1)[:, :codes.shape[1]]
