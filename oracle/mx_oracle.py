"""CPU oracle of the microscaled 4-bit formats (test infrastructure only): the
E2M1 quantization with E8M0 scales per 32 values or E4M3 scales per 16, the
scales' tile layout, and the block-scaled product in float64.  Shares no code
with the CUDA path.
"""
from __future__ import annotations

import numpy as np

MXFP4, NVFP4 = 0, 1
LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
# values of the 128 non-negative E4M3 bytes (0x7F is NaN)
E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)])
E4M3[127] = np.nan


def block(fmt):
    return 32 if fmt == MXFP4 else 16


def nearest(values, table):
    """Index of the nearest entry of an ascending table; ties go to the even index."""
    v = np.asarray(values, np.float64)
    hi = np.clip(np.searchsorted(table, v, side="left"), 1, len(table) - 1)
    lo = hi - 1
    dlo, dhi = v - table[lo], table[hi] - v
    pick = np.where(dlo < dhi, lo, np.where(dhi < dlo, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(v >= table[-1], len(table) - 1, pick)


def quant(x, fmt, g=None):
    """fp16 [R, K] -> (codes uint8 [R, K] in 0..15, scale bytes uint8 [R, K / block])."""
    b = block(fmt)
    xf = np.asarray(x, np.float16).astype(np.float32)
    r, k = xf.shape
    xb = xf.reshape(r, k // b, b)
    finite = np.isfinite(xb).all(-1)
    xb = np.where(finite[..., None], xb, np.float32(0))
    amax = np.abs(xb).max(-1)
    if fmt == MXFP4:
        e = np.frexp(amax)[1].astype(np.int64) - 1 - 2
        e = np.where(amax == 0, -127, e)
        sb = (e + 127).astype(np.uint8)
        d = np.ldexp(1.0, e)
        v = xb.astype(np.float64) / d[..., None]
        nan = 0xFF
    else:
        gs = np.float32(1.0 if g is None else g)
        t = (amax / np.float32(np.float32(6.0) * gs)).astype(np.float32)
        sb = nearest(t, E4M3[:127]).astype(np.uint8)
        d = (E4M3[sb].astype(np.float32) * gs).astype(np.float32)
        with np.errstate(divide="ignore", invalid="ignore"):
            v = np.where(d[..., None] != 0, (xb / d[..., None]).astype(np.float32), np.float32(0)).astype(np.float64)
        nan = 0x7F
    code = nearest(np.abs(v), LEVELS).astype(np.uint8)
    code |= (np.signbit(v) << 3).astype(np.uint8)
    code[~finite] = 0
    sb = np.where(finite, sb, nan).astype(np.uint8)
    return code.reshape(r, k), sb


def pack(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    out = np.empty((q.shape[0], q.shape[1] * 2), np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def scale_value(sb, fmt):
    """Float64 values of scale bytes (NaN where they hold NaN)."""
    sb = np.asarray(sb)
    if fmt == MXFP4:
        return np.where(sb == 255, np.nan, np.ldexp(1.0, sb.astype(np.int64) - 127))
    return np.where(sb & 128, np.nan, E4M3[sb & 127])


def to_tiles(sb, fill=0):
    """Scale bytes [R, B] -> the tiled bytes (rows padded with `fill`)."""
    r, b = sb.shape
    rt = -(-r // 128)
    out = np.full(rt * 128 * b, fill, np.uint8)
    rr, bb = np.meshgrid(np.arange(r), np.arange(b), indexing="ij")
    out[((rr // 128) * (b // 4) + bb // 4) * 512 + (rr % 32) * 16 + (rr % 128 // 32) * 4 + bb % 4] = sb
    return out


def from_tiles(t, r, b):
    rr, bb = np.meshgrid(np.arange(r), np.arange(b), indexing="ij")
    return np.asarray(t)[((rr // 128) * (b // 4) + bb // 4) * 512 + (rr % 32) * 16 + (rr % 128 // 32) * 4 + bb % 4]


def values(code, sb, fmt):
    """Float64 code values times block scales (without the tensor scale)."""
    v = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    return v * np.repeat(scale_value(sb, fmt), block(fmt), axis=1)


def product(xc, xs, wc, ws, fmt):
    """Float64 (acc [M, N], sum of the terms' magnitudes)."""
    x, w = values(xc, xs, fmt), values(wc, ws, fmt)
    return x @ w.T, np.abs(x) @ np.abs(w).T
