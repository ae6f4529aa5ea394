"""NumPy oracle of the microscaled 4-bit floating-point operators (MXFP4, NVFP4).

Everything is taken from the definition in 64 bits: nearest entries by distance with ties to
the even code, scales by exact powers of two and by search in the table of E4M3 values. No
code or table is shared with the CUDA library.
"""
from __future__ import annotations

import numpy as np

MX, NV = 0, 1
BLOCK = {MX: 32, NV: 16}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_table() -> np.ndarray:
    """Values of the bytes 0..0x7E, ascending."""
    b = np.arange(127)
    e, m = b >> 3, b & 7
    return np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))


def nearest(v, table) -> np.ndarray:
    """Index of the nearest entry of an ascending table (ties to the even index)."""
    v = np.asarray(v, np.float64)
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = v - table[lo], table[hi] - v
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(v >= table[-1], len(table) - 1, np.where(v <= table[0], 0, pick))


def floor_log2(a) -> np.ndarray:
    """floor(log2 a) of positive values, exactly."""
    return np.frexp(a)[1] - 1


def gscale(top) -> np.ndarray:
    """The smallest power of two 2^e, e >= -126, with top <= 2688 * 2^e; 1 for top = 0."""
    top = np.asarray(top, np.float64)
    m, e = np.frexp(np.where(top > 0, top, 1.0) / 2688.0)
    e = np.maximum(np.where(m > 0.5, e, e - 1), -126)
    return np.where(top > 0, 2.0 ** e.astype(np.float64), 1.0)


def _scales(amax, bad, fmt, g):
    """(byte, value) of block scales from finite maxima; bad: blocks with a NaN or infinity."""
    if fmt == MX:
        e = np.where(amax > 0, floor_log2(np.where(amax > 0, amax, 1.0)) - 2, -127)
        e = np.clip(e, -127, 127)
        byte, val = e + 127, 2.0 ** e.astype(np.float64)
        return np.where(bad, 255, byte).astype(np.uint8), np.where(bad, np.nan, val)
    t = e4m3_table()
    byte = nearest(amax / g / 6.0, t)
    return np.where(bad, 0x7F, byte).astype(np.uint8), np.where(bad, np.nan, t[byte])


def _codes(x, val, fmt, g):
    """E2M1 codes of x (blocks in the last axes broadcast against val)."""
    ok = np.isfinite(val) & (val > 0)
    q = np.where(ok, x / g / np.where(ok, val, 1.0), 0.0)
    q = np.where(np.isfinite(q), q, 0.0)
    return (nearest(np.abs(q), E2M1) | (np.signbit(q).astype(np.int64) << 3)).astype(np.uint8)


def quantize(X, fmt):
    """Row-wise form: dict of codes [rows, cols] (one per byte), bytes [rows, blocks], g [rows]."""
    X = np.asarray(X, np.float64)
    R, C = X.shape
    x = X.reshape(R, C // BLOCK[fmt], BLOCK[fmt])
    fin = np.isfinite(x)
    amax = np.abs(np.where(fin, x, 0.0)).max(2)
    g = gscale(amax.max(1)) if fmt == NV else np.ones(R)
    byte, val = _scales(amax, ~fin.all(2), fmt, g[:, None])
    codes = _codes(x, val[:, :, None], fmt, g[:, None, None]).reshape(R, C)
    return {"codes": codes, "bytes": byte, "g": g, "fmt": fmt}


def quantize_weight(W, fmt):
    """Square-block form of W [N, K] and of its transpose."""
    W = np.asarray(W, np.float64)
    N, K = W.shape
    b = BLOCK[fmt]
    x = W.reshape(N // b, b, K // b, b)
    fin = np.isfinite(x)
    amax = np.abs(np.where(fin, x, 0.0)).max((1, 3))
    g = gscale(amax.max()) if fmt == NV else np.float64(1.0)
    byte, val = _scales(amax, ~fin.all((1, 3)), fmt, g)
    codes = _codes(x, val[:, None, :, None], fmt, g).reshape(N, K)
    w = {"codes": codes, "bytes": byte.repeat(b, 0), "g": np.array([g]), "fmt": fmt}
    wt = {"codes": codes.T.copy(), "bytes": byte.T.repeat(b, 0), "g": np.array([g]), "fmt": fmt}
    return w, wt


def dequant(q) -> np.ndarray:
    """Values, fp64."""
    c, fmt = q["codes"], q["fmt"]
    if fmt == MX:
        val = np.where(q["bytes"] == 255, np.nan, 2.0 ** (q["bytes"].astype(np.float64) - 127))
    else:
        val = np.append(e4m3_table(), np.nan)[q["bytes"]]
    v = np.where(c >= 8, -E2M1[c & 7], E2M1[c & 7]) * val.repeat(BLOCK[fmt], 1)
    return v * np.asarray(q["g"], np.float64).reshape(-1, 1)


def pack(codes) -> np.ndarray:
    """Stored code bytes: the even column in the low nibble."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def scale_index(rows, blocks) -> np.ndarray:
    """Position of the scale byte of (row, block) in the stored array."""
    r, b = np.arange(rows)[:, None], np.arange(blocks)[None]
    return (r // 128 * -(-blocks // 4) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4


def store_scales(byte) -> np.ndarray:
    """The stored scale array (zeros where no block is)."""
    R, B = byte.shape
    out = np.zeros(-(-R // 128) * -(-B // 4) * 512, np.uint8)
    out[scale_index(R, B)] = byte
    return out


def linear_forward(X, w, A, B, scale):
    """Y and T = X A in fp64, q(X) through the rounding of the weight's format."""
    X, A, B = (np.asarray(a, np.float64) for a in (X, A, B))
    T = X @ A
    return dequant(quantize(X, w["fmt"])) @ dequant(w).T + scale * (T @ B), T


def linear_backward(dY, X, w, A, B, scale):
    """dX, dA, dB in fp64."""
    dY, X, A, B = (np.asarray(a, np.float64) for a in (dY, X, A, B))
    G = dY @ B.T
    dX = dequant(quantize(dY, w["fmt"])) @ dequant(w) + scale * (G @ A.T)
    return dX, scale * (X.T @ G), scale * ((X @ A).T @ dY)
