"""The 4-bit formats in float64, from their definitions (no GPU code shared):
E2M1 codes with an E4M3 scale per 16 values and a tensor scale ("nvfp4"), or an
E8M0 scale per 32 ("mxfp4"), and the place of each scale byte."""
from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# every E4M3 magnitude by its byte (0x7f is NaN)
E4M3 = np.array([(b & 7) * 2.0 ** -9 if b < 8 else (8 + (b & 7)) * 2.0 ** ((b >> 3) - 10) for b in range(127)])
BLOCK = {"nvfp4": 16, "mxfp4": 32}


def nearest(values, table):
    """Index in the ascending table of the value nearest to each, the even
    index of two as near; above the table its last."""
    v = np.minimum(np.abs(values), table[-1])
    hi = np.searchsorted(table, v)                # table[hi - 1] < v <= table[hi]
    lo = np.maximum(hi - 1, 0)
    up, down = table[hi] - v, v - table[lo]
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return np.where(take_hi, hi, lo)


def quantize(x, fmt, t=1.0):
    """x [..., K] -> (codes 0..15 [..., K], scale bytes [..., K / block])."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // BLOCK[fmt], BLOCK[fmt]))
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    if fmt == "nvfp4":
        s = nearest(amax / (6 * t), E4M3)
        d = E4M3[s] * t
        byte = np.where(bad, 0x7F, s)
    else:
        with np.errstate(divide="ignore"):
            e = np.where(amax > 0, np.frexp(amax)[1] - 3, -127)
        e = np.maximum(e, -127)
        d = 2.0 ** e.astype(np.float64)
        byte = np.where(bad, 0xFF, e + 127)
    with np.errstate(divide="ignore", invalid="ignore"):
        u = np.where(d[..., None] > 0, b / d[..., None], 0.0)
    code = nearest(u, MAGNITUDES) + 8 * np.signbit(b)
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def scale_values(byte, fmt):
    byte = np.asarray(byte)
    if fmt == "nvfp4":
        return np.where(byte == 0x7F, np.nan, E4M3[np.minimum(byte, 126)])
    return np.where(byte == 0xFF, np.nan, 2.0 ** (byte.astype(np.float64) - 127))


def code_values(code):
    code = np.asarray(code)
    return np.where(code & 8, -1.0, 1.0) * MAGNITUDES[code & 7]


def values(code, byte, fmt, t=1.0):
    code = np.asarray(code)
    v = code_values(code).reshape(code.shape[:-1] + (code.shape[-1] // BLOCK[fmt], BLOCK[fmt]))
    return (v * scale_values(byte, fmt)[..., None] * t).reshape(code.shape)


def unpack(q):
    """Bytes [..., K / 2] -> codes [..., K]."""
    q = np.asarray(q)
    return np.stack([q & 15, q >> 4], -1).reshape(q.shape[:-1] + (2 * q.shape[-1],))


def chunks(K, fmt):
    return K // 64 if fmt == "nvfp4" else -(-K // 128)


def scale_bytes(rows, E, K, fmt):
    return (rows // 128 + E) * chunks(K, fmt) * 512


def scale_place(offsets, K, fmt):
    """Byte index of each row's scales [rows below the last offset, K / block]
    (-1: the row is in no expert)."""
    offsets = [int(o) for o in offsets]
    nb, C = K // BLOCK[fmt], chunks(K, fmt)
    at = np.full((offsets[-1], nb), -1, np.int64)
    b = np.arange(nb)
    for e in range(len(offsets) - 1):
        for row in range(offsets[e], offsets[e + 1]):
            r = row - offsets[e]
            tile = offsets[e] // 128 + e + r // 128
            at[row] = (tile * C + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
    return at


def tensor_scale(x):
    """The smallest power of two t with max|x| <= 2688 t over the finite x."""
    x = np.abs(np.asarray(x, np.float64))
    top = np.where(np.isfinite(x), x, 0.0).max(initial=0.0)
    if top == 0:
        return 1.0
    m, e = np.frexp(top / 2688)
    return float(2.0 ** min(127, max(-126, e - (m == 0.5))))
