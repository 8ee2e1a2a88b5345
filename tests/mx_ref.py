"""The MX formats in fp64 on the CPU, from the definition in
include/dense_gemm.h: rounding a matrix to blocks of 32, the stored form, and
the values that a stored form stands for.  Shares no code with the library."""
from __future__ import annotations

import numpy as np

EMAX = {"mxfp4": 2, "mxfp8": 8, "mxint8": 0}


def _table(exp_bits, frac_bits, bias):
    """Value of every code of a small float without infinities."""
    n = 1 << (1 + exp_bits + frac_bits)
    out = np.empty(n)
    for c in range(n):
        sign = -1.0 if c >> (exp_bits + frac_bits) else 1.0
        e, f = (c >> frac_bits) & ((1 << exp_bits) - 1), c & ((1 << frac_bits) - 1)
        out[c] = sign * (f * 2.0 ** (1 - bias - frac_bits) if e == 0 else (1 + f / 2 ** frac_bits) * 2.0 ** (e - bias))
    return out


FP4 = _table(2, 1, 1)
FP8 = _table(4, 3, 7)
FP8[0x7f] = FP8[0xff] = np.nan
INT8 = np.arange(256).astype(np.uint8).view(np.int8) / 64.0
TABLE = {"mxfp4": FP4, "mxfp8": FP8, "mxint8": INT8}


def groups(cols):
    return -(-cols // 256)


def row_bytes(fmt, cols):
    return groups(cols) * (128 if fmt == "mxfp4" else 256)


def _nearest_code(u, fmt):
    """Code of the nearest element to each u (ties to the even code), with the
    sign kept, by search over the sorted magnitudes."""
    if fmt == "mxint8":
        return np.clip(np.rint(u * 64), -127, 127).astype(np.int64) & 255
    t = TABLE[fmt]
    half = len(t) // 2
    mags = t[:half][np.isfinite(t[:half])]           # increasing with the code
    m = np.minimum(np.abs(u), mags[-1])
    hi = np.clip(np.searchsorted(mags, m), 1, len(mags) - 1)
    lo = hi - 1
    dl, dh = m - mags[lo], mags[hi] - m
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return code | np.where(np.signbit(u), half, 0)


def quantize(x, fmt):
    """(codes [rows, groups * 256], scale bytes [rows, groups * 8]) of fp64 x."""
    rows, cols = x.shape
    g = groups(cols)
    full = np.zeros((rows, g * 256))
    full[:, :cols] = x
    b = full.reshape(rows, g * 8, 32)
    bad = ~np.isfinite(b).all(-1)
    top = np.where(bad, 1.0, np.abs(np.where(np.isfinite(b), b, 0)).max(-1))
    e = np.where(top > 0, np.frexp(np.where(top > 0, top, 1.0))[1] - 1 - EMAX[fmt], -127)
    e = np.maximum(e, -127)
    u = np.where(bad[..., None], 0.0, b) / np.exp2(e.astype(np.float64))[..., None]
    code = np.where(bad[..., None], 0, _nearest_code(u, fmt))
    byte = np.where(bad, 255, e + 127)
    # blocks wholly past the last column are written as zero
    byte[:, -(-cols // 32):] = 0
    return code.reshape(rows, -1), byte.astype(np.uint8)


def pack(code, fmt):
    if fmt == "mxfp4":
        return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)
    return code.astype(np.uint8)


def scales_to_s(byte):
    """[rows, groups * 8] -> [groups, rows, 8]."""
    return np.ascontiguousarray(byte.reshape(byte.shape[0], -1, 8).transpose(1, 0, 2))


def values(q, s, fmt, cols):
    """fp64 values of a stored matrix: q [rows, bytes], s [groups, rows, 8]."""
    rows = q.shape[0]
    code = q[:, :row_bytes(fmt, cols)]
    if fmt == "mxfp4":
        code = np.stack([code & 15, code >> 4], -1).reshape(rows, -1)
    byte = s.transpose(1, 0, 2).reshape(rows, -1).astype(np.float64)
    sc = np.where(byte == 255, np.nan, np.exp2(byte - 127))
    return (TABLE[fmt][code] * np.repeat(sc, 32, axis=1))[:, :cols]


def random_stored(rng, rows, cols, fmt, spread=2, whole=False):
    """A random stored matrix (q, s) with zeros past cols; scales 2^-spread ..
    2^spread.  whole: elements are small multiples of 1/2, so that sums of
    products stay exact."""
    rb = row_bytes(fmt, cols)
    n = groups(cols) * 256
    if fmt == "mxfp4":
        code = rng.integers(0, 16, (rows, n))
    elif fmt == "mxfp8":
        if whole:
            small = np.flatnonzero(np.isfinite(FP8) & (np.abs(FP8) <= 8) & (FP8 == np.rint(FP8)))
            code = small[rng.integers(0, len(small), (rows, n))]
        else:
            code = _nearest_code(rng.standard_normal((rows, n)) * 100, "mxfp8")
    else:
        code = rng.integers(-127, 128, (rows, n)) & 255
        if whole:
            code = (rng.integers(-3, 4, (rows, n)) * 32) & 255
    code[:, cols:] = 0
    byte = rng.integers(127 - spread, 128 + spread, (rows, groups(cols) * 8)).astype(np.uint8)
    q = pack(code, fmt)
    assert q.shape[1] == rb
    return q, scales_to_s(byte)
