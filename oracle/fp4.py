"""Float64 oracle of the microscaled 4-bit formats (MXFP4, NVFP4): quantiser,
stored layout, values and products.  Shares no code with the kernels.

Decisions are those of exact arithmetic.  Float64 quotients decide them
exactly: x and the tensor scale g have 24 significant bits, a block scale at
most 4 and a rounding border at most 5, so a quotient that is not itself a
border differs from it by more than 2^-40 relative, and one that is a border
is exact.
"""
from __future__ import annotations

import numpy as np

MX, NV = 0, 1
BLOCK = {MX: 32, NV: 16}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_table():
    """Values of the bytes 0 .. 126 (127 is NaN), float64."""
    b = np.arange(127)
    e, mant = b >> 3, (b & 7).astype(np.float64)
    return np.where(e == 0, mant * 2.0 ** -9, (1.0 + mant / 8.0) * 2.0 ** (e - 7.0))


def code_row_bytes(n):
    return -(-(-(-n // 2)) // 16) * 16


def scale_row_bytes(fmt, n):
    return -(-(-(-n // BLOCK[fmt])) // 16) * 16


def _nearest_even(y, table):
    """Index of the nearest table entry (ascending), ties to the even index, saturating."""
    hi = np.clip(np.searchsorted(table, y), 1, len(table) - 1)
    mid = (table[hi - 1] + table[hi]) / 2.0
    up = (y > mid) | ((y == mid) & (hi % 2 == 0))
    return np.where(up, hi, hi - 1)


def tensor_scale(x):
    """float32(largest finite |x| / 2688), at least 2^-126; 1 for zeros."""
    a = np.abs(np.asarray(x, np.float64))
    a = a[np.isfinite(a)].max(initial=0.0)
    return np.float32(1.0) if a == 0 else max(np.float32(a / 2688.0), np.float32(2.0 ** -126))


def quantize(x, fmt, g=None):
    """(codes rows x n in 0..15, scale bytes rows x blocks, g) of float x (rows x n)."""
    x = np.asarray(x, np.float64)
    rows, n = x.shape
    bs = BLOCK[fmt]
    nb = -(-n // bs)
    wide = np.zeros((rows, nb * bs))
    wide[:, :n] = x
    b = wide.reshape(rows, nb, bs)
    bad = ~np.isfinite(b).all(axis=2)
    mag = np.where(bad[:, :, None], 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)))
    amax = mag.max(axis=2)
    if fmt == MX:
        _, e = np.frexp(amax)                      # amax = f 2^e, f in [0.5, 1)
        e = np.where(amax > 0, np.clip(e - 3, -127, 127), -127)
        scale, sbytes = 2.0 ** e.astype(np.float64), e + 127
    else:
        g = tensor_scale(x) if g is None else np.float32(g)
        if not (np.isfinite(g) and g >= np.float32(2.0 ** -126)):
            bad = np.ones_like(bad)
            scale, sbytes = np.zeros_like(amax), np.zeros_like(amax, dtype=np.int64)
        else:
            table = e4m3_table()
            sbytes = _nearest_even(amax / (6.0 * np.float64(g)), table)
            scale = table[sbytes] * np.float64(g)
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(scale[:, :, None] > 0, mag / scale[:, :, None], 0.0)
    codes = _nearest_even(y, E2M1) + 8 * np.signbit(b)
    codes = np.where(bad[:, :, None], 0, codes)
    sbytes = np.where(bad, 255 if fmt == MX else 127, sbytes)
    return codes.reshape(rows, -1)[:, :n].astype(np.uint8), sbytes.astype(np.uint8), g


def store(codes, sbytes, fmt):
    """The stored arrays: codes two per byte, rows padded with zeros."""
    rows, n = codes.shape
    c = np.zeros((rows, 2 * code_row_bytes(n)), np.uint8)
    c[:, :n] = codes
    s = np.zeros((rows, scale_row_bytes(fmt, n)), np.uint8)
    s[:, : sbytes.shape[1]] = sbytes
    return c[:, 0::2] | (c[:, 1::2] << 4), s


def values(codes, sbytes, fmt):
    """code * scale in float64 (no tensor scale) of unpacked codes (rows x n) and scale bytes."""
    n = codes.shape[1]
    q = np.where(codes >= 8, -1.0, 1.0) * E2M1[codes & 7]
    if fmt == MX:
        s = np.where(sbytes == 255, np.nan, 2.0 ** (sbytes.astype(np.float64) - 127.0))
    else:
        s = np.append(e4m3_table(), np.nan)[sbytes]
    return q * np.repeat(s, BLOCK[fmt], axis=1)[:, :n]


def values_f32(codes, sbytes, fmt, g=None):
    """(code * scale) * g with float32 roundings: what the dequantiser returns in float32."""
    v = values(codes, sbytes, fmt).astype(np.float32)   # exact
    return v if g is None else v * np.float32(g)


def product(xv, wv, xg=None, wg=None):
    """(y, bound): X W^T in float64 and sum |x w|, the scale of its rounding errors."""
    f = (1.0 if xg is None else np.float64(xg)) * (1.0 if wg is None else np.float64(wg))
    return xv @ wv.T * f, np.abs(xv) @ np.abs(wv).T * f


def group_bounds(offsets, T):
    """The offsets as taken: each at least its predecessor, within [0, T]."""
    return np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, T))
