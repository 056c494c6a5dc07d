"""Plain 64-bit reference of the fp8 matrices with a scale for each block of 128.

Written from the definitions of the formats (OCP e4m3: 4 exponent bits, bias 7,
3 fraction bits, largest 448, no infinity; e5m2: 5 exponent bits, bias 15, 2
fraction bits, largest 57344) and of the scale rule, in numpy.  Used by tests only.
"""
import numpy as np

GROUP = 128
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
_FRACTION, _LOWEST = {"e4m3": 3, "e5m2": 2}, {"e4m3": -6, "e5m2": -14}


def decode(codes, fmt):
    """float64 value of every code byte."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    f = _FRACTION[fmt]
    sign = np.where(c & 0x80, -1.0, 1.0)
    e, m = (c & 0x7F) >> f, c & ((1 << f) - 1)
    v = np.where(e == 0, m * 2.0 ** (_LOWEST[fmt] - f), (m + (1 << f)) * 2.0 ** (e + _LOWEST[fmt] - 1.0 - f))
    if fmt == "e4m3":
        v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    else:
        v = np.where(e == 31, np.where(m == 0, np.inf, np.nan), v)
    return sign * v


def round_to(x, fmt):
    """x rounded to the format's grid, nearest even (|x| at most TOP; infinities as the format has them)."""
    x = np.asarray(x, np.float64)
    finite = np.where(np.isfinite(x), x, 0.0)
    _, e = np.frexp(finite)
    step = 2.0 ** (np.maximum(e - 1, _LOWEST[fmt]) - float(_FRACTION[fmt]))
    out = np.rint(finite / step) * step
    return np.where(np.isfinite(x), out, np.nan if fmt == "e4m3" else x)


def scale_exponent(amax, fmt):
    """Smallest e >= -126 with amax <= TOP 2^e; 0 for amax = 0."""
    if amax == 0:
        return 0
    e = -126
    while amax > TOP[fmt] * 2.0 ** e:
        e += 1
    return e


def quantize(x, fmt, block_rows=1):
    """(values of the codes before scaling [rows][cols rounded up], exponents [rows][groups])."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    q = np.zeros((rows, groups * GROUP))
    ex = np.zeros((rows, groups), np.int64)
    for r in range(0, rows, block_rows):
        for g in range(groups):
            part = x[r:r + block_rows, g * GROUP:(g + 1) * GROUP]
            mag = np.abs(part[np.isfinite(part)])
            e = scale_exponent(mag.max() if mag.size else 0.0, fmt)
            ex[r:r + block_rows, g] = e
            q[r:r + block_rows, g * GROUP:g * GROUP + part.shape[1]] = round_to(part * 2.0 ** -e, fmt)
    return q, ex


def pack_scales(ex):
    """Scale bytes [words][rows rounded up to 4][4] of exponents [rows][groups], 127 where unused."""
    rows, groups = ex.shape
    out = np.full((-(-groups // 4), -(-rows // 4) * 4, 4), 127, np.uint8)
    for g in range(groups):
        out[g // 4, :rows, g % 4] = ex[:, g] + 127
    return out


def unpack_scales(s, rows, groups):
    """2^e as float64 [rows][groups]."""
    return np.stack([2.0 ** (s[g // 4, :rows, g % 4].astype(np.float64) - 127.0) for g in range(groups)], axis=1)


def values(codes, s, fmt):
    """float64 matrix that codes [rows][K] and scale bytes stand for."""
    rows, K = codes.shape
    return decode(codes, fmt) * np.repeat(unpack_scales(s, rows, K // GROUP), GROUP, axis=1)


def gemm(A, B, C, alpha, beta):
    """beta C + alpha A B^T (C is not read where beta is 0)."""
    return alpha * (A @ B.T) + (beta * C if beta != 0 else 0.0)
