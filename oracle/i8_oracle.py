"""Plain CPU definitions of the 8-bit quantisers and of their product: numpy, f64,
exact rational arithmetic where a value lies next to the border between two codes.
Test infrastructure only.

codes(v): M = max |v|, code = 127 v / M to the nearest integer, ties away from zero.
"""
from fractions import Fraction

import numpy as np

NEAR = 1e-9  # f64 quotients of at most 127 are off by less than 1e-13


def row_bytes(k):
    return -(-k // 16) * 16


def _code_exact(factors, top):
    """Code magnitude of |v| = the product of `factors` (f64 numbers taken as they are), with the maximum `top` likewise."""
    v, m = Fraction(1), Fraction(1)
    for f in factors:
        v *= abs(Fraction(float(f)))
    for f in top:
        m *= abs(Fraction(float(f)))
    return int((254 * v + m) // (2 * m))


def quantise(*factors):
    """(codes int8 [rows][row_bytes(k)], M f64[rows]) of v = the elementwise product of the f64 arrays `factors`. M is NaN
    for a row with a value that is not finite."""
    with np.errstate(all="ignore"):
        v = np.ones_like(factors[0], dtype=np.float64)
        for f in factors:
            v = v * np.asarray(f, np.float64)
    rows, k = v.shape
    out, top = np.zeros((rows, row_bytes(k)), np.int8), np.zeros(rows)
    for r in range(rows):
        if not all(np.isfinite(np.broadcast_to(f, v.shape)[r]).all() for f in factors) or not np.isfinite(v[r]).all():
            top[r] = np.nan
            continue
        mag = np.abs(v[r])
        at = int(np.argmax(mag))
        top[r] = mag[at]
        if top[r] == 0:
            continue
        t = 127.0 * (mag / top[r])
        q = np.floor(t + 0.5)
        for i in np.flatnonzero(np.abs(t - np.floor(t) - 0.5) < NEAR):
            q[i] = _code_exact([np.broadcast_to(f, v.shape)[r, i] for f in factors],
                               [np.broadcast_to(f, v.shape)[r, at] for f in factors])
        out[r, :k] = (q * np.sign(v[r])).astype(np.int8)
    return out, top


def rows_quant(x):
    """(codes, scale f32) of the rows of x (any float array)."""
    codes, top = quantise(np.asarray(x, np.float64))
    return codes, (top / 127.0).astype(np.float32)


def norm_quant(h, g, eps):
    """(codes, scale f64) of the RMSNorm of the stored rows h."""
    h, g = np.asarray(h, np.float64), np.asarray(g, np.float64)
    codes, top = quantise(h, np.broadcast_to(g, h.shape))
    with np.errstate(all="ignore"):
        return codes, np.where(top == 0, 0.0, top / np.sqrt((h * h).mean(1) + eps) / 127.0)


def silu_quant(gate, up):
    """(codes, scale f64) of silu(gate) * up. silu in extended precision, where the platform has it."""
    gate, up = np.asarray(gate, np.longdouble), np.asarray(up, np.longdouble)
    with np.errstate(all="ignore"):
        v = np.where(np.isfinite(gate) & np.isfinite(up), gate / (1 + np.exp(-gate)) * up, np.nan)
    codes, top = quantise(v.astype(np.float64))
    return codes, top / 127.0


def q8_0_values(blocks, k):
    """The values d * q of Q8_0 blocks uint8 [rows][k / 32 * 34]."""
    b = np.ascontiguousarray(blocks).reshape(blocks.shape[0], k // 32, 34)
    d = b[..., :2].copy().view("<f2").astype(np.float64)
    return (d * b[..., 2:].view(np.int8)).reshape(blocks.shape[0], k)


def matmul(a, sa, w, sw, k):
    """y f64 = (codes a . codes w) * scales, the sums exact."""
    s = a[:, :k].astype(np.float64) @ w[:, :k].astype(np.float64).T  # below 2^31: exact in f64
    return s * np.asarray(sa, np.float64)[:, None] * np.asarray(sw, np.float64)[None, :]
