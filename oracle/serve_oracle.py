"""Float64 restatement of the serving operators: microscaled 4-bit floating point, products of such
operands, and the layer for a few tokens. NumPy, from the definitions; test infrastructure only."""
from __future__ import annotations

import numpy as np

MX, NV = 0, 1
BLOCK = {MX: 32, NV: 16}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)) for e in range(16) for m in range(8)][:127])


def _nearest(v, table):
    """Index of the nearest number of an increasing table, the even index on a tie; the last at most."""
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    lo = hi - 1
    below, above = v - table[lo], table[hi] - v
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return np.where(v >= table[-1], len(table) - 1, np.where(up, hi, lo))


def scale_columns(K, fmt):
    return (K // BLOCK[fmt] + 15) // 16 * 16


def quantize(x, fmt, g=None):
    """x float64 [rows, K] -> (codes uint8 [rows, K / 2], scales uint8 [rows, S]). g: a number (NV)."""
    rows, K = x.shape
    b = x.reshape(rows, -1, BLOCK[fmt])
    bad = ~np.isfinite(b).all(2)
    b = np.where(bad[:, :, None], 0.0, b)
    top = np.abs(b).max(2)
    if fmt == MX:
        e = np.arange(-127, 128)
        byte = np.searchsorted(6.0 * 2.0 ** e.astype(np.float64), top)      # the least with top <= 6 2^e
        unit = 2.0 ** (byte - 127.0)
    else:
        g = 1.0 if g is None else float(g)
        byte = _nearest(top / (6.0 * g), E4M3)
        unit = E4M3[byte] * g
    z = np.abs(b) / np.where(unit > 0, unit, np.inf)[:, :, None]
    code = (_nearest(z, E2M1) + 8 * np.signbit(b)).astype(np.uint8)
    code[bad] = 0
    byte = np.where(bad, 255 if fmt == MX else 127, byte)
    code = code.reshape(rows, K // 2, 2)
    scales = np.zeros((rows, scale_columns(K, fmt)), np.uint8)
    scales[:, :byte.shape[1]] = byte
    return code[:, :, 0] | code[:, :, 1] << 4, scales


def dequantize(codes, scales, fmt, g=None):
    """The values of codes [rows, K / 2]."""
    rows, half = codes.shape
    both = np.stack([codes & 15, codes >> 4], 2).reshape(rows, -1)
    v = np.where(both >= 8, -1.0, 1.0) * E2M1[both & 7]
    sc = scales[:, :2 * half // BLOCK[fmt]]
    if fmt == MX:
        s = np.where(sc == 255, np.nan, 2.0 ** (sc.astype(np.float64) - 127))
    else:
        s = np.where(sc == 127, np.nan, np.append(E4M3, np.nan)[np.minimum(sc, 127)]) * (1.0 if g is None else float(g))
    return v * np.repeat(s, BLOCK[fmt], 1)


def swiglu(gu):
    I = gu.shape[1] // 2
    with np.errstate(over="ignore"):
        return gu[:, :I] / (1 + np.exp(-gu[:, :I])) * gu[:, I:]


def experts_matmul(x, w, offsets):
    """y[r] = x[r] . w[e]^T for the rows of expert e, 0 elsewhere."""
    y = np.zeros((x.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        y[a:b] = x[a:b] @ w[e].T
    return y
