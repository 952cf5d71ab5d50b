"""Block-scaled e4m3 matrices: quantizer, norm, product and gated projection.

Oracle (test infrastructure only), fp64.  e4m3 is the 8-bit floating-point
format without infinities (1 sign, 4 exponent bits with bias 7, 3 mantissa
bits; 0x7F and 0xFF are NaN, the largest value is 448).  A matrix is codes
and one scale per block of 128 columns and 1 or 128 rows:

    scale = max(fl32(amax/448), 2^-126),  code = rne_e4m3(x/scale)

and a block with a NaN or an infinity has a NaN scale and NaN codes.
Matrices here are (values [rows x cols] of the codes, scales); ``decode``
turns stored bytes into values.
"""
from __future__ import annotations

import numpy as np
from scipy import special

BLOCK = 128
_c = np.arange(127)
#: the values of the codes 0x00..0x7E
GRID = np.where(_c < 8, _c / 8 * 2.0 ** -6, (1 + _c % 8 / 8) * 2.0 ** (_c // 8 - 7.0))
_MID = (GRID[1:] + GRID[:-1]) / 2


def decode(codes) -> np.ndarray:
    """Values of e4m3 bytes."""
    c = np.asarray(codes, dtype=np.uint8)
    v = np.append(GRID, np.nan)[c & 0x7F]
    return np.where(c & 0x80, -v, v)


def nearest(q) -> np.ndarray:
    """The e4m3 value nearest to q (|q| <= 464), ties to the even code."""
    a = np.abs(q)
    low, high = np.searchsorted(_MID, a, "left"), np.searchsorted(_MID, a, "right")
    code = np.where(low % 2 == 0, low, high)
    return np.copysign(GRID[code], q)


def border_distance(q) -> np.ndarray:
    """Distance of |q| to the nearest border between two codes, relative to |q|."""
    a = np.abs(np.asarray(q, dtype=np.float64))
    i = np.clip(np.searchsorted(_MID, a), 1, len(_MID) - 1)
    d = np.minimum(np.abs(a - _MID[i]), np.abs(a - _MID[i - 1]))
    return d / np.maximum(a, 2.0 ** -10)


def expand(scales, block_rows: int, rows: int, cols: int) -> np.ndarray:
    i, j = np.arange(rows) // block_rows, np.arange(cols) // BLOCK
    return np.asarray(scales, dtype=np.float64)[i][:, j]


def quantize(x, block_rows: int):
    """(values of the codes, fp32 scales) of x."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    rb, kb = -(-rows // block_rows), -(-cols // BLOCK)
    a = np.zeros((rb * block_rows, kb * BLOCK))
    a[:rows, :cols] = np.where(np.isfinite(x), np.abs(x), np.inf)
    amax = a.reshape(rb, block_rows, kb, BLOCK).max((1, 3))
    with np.errstate(over="ignore"):
        s = np.maximum((amax / 448).astype(np.float32), np.float32(2.0 ** -126))
    s = np.where(np.isfinite(amax), s, np.float32(np.nan)).astype(np.float32)
    e = expand(s, block_rows, rows, cols)
    v = np.full(x.shape, np.nan)
    ok = np.isfinite(e)
    v[ok] = nearest(x[ok] / e[ok])
    return v, s


def values(m, block_rows: int) -> np.ndarray:
    v, s = m
    return v * expand(s, block_rows, *v.shape)


def rmsnorm(h, gamma, eps: float) -> np.ndarray:
    h = np.asarray(h, dtype=np.float64)
    return h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * np.asarray(gamma, dtype=np.float64)


def matmul(a, b):
    """(A·Bᵀ, Σ|a||b|) of block-scaled activations and weights: the exact
    product, and what its rounding errors are measured by."""
    x, w = values(a, 1), values(b, BLOCK)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def accumulation_bound(mag, K: int, grouped: bool = False) -> np.ndarray:
    """Error bound of the fp32 sum: inside a block of 128 every addition may
    lose one unit in the last place (2^-23 of the running magnitude: an
    instruction that truncates is covered), the blocks' sums add one fma
    each, the scales' product one rounding.  grouped: the instruction that
    adds eight products in fixed point, at 2^-13 of the power of two below
    the largest: the seven others lose up to 2^-13 of it each."""
    u = 2.0 ** -23 * min(K, BLOCK) + 2.0 ** -24 * (-(-K // BLOCK) + 2)
    return mag * (u + (7 * 2.0 ** -13 if grouped else 0.0))


def dropped_spread(a, b) -> np.ndarray:
    """Spread σ of what the fp8 matrix instruction cuts off A·Bᵀ.  It aligns
    every eight neighbouring products to the power of two of the largest,
    2^e <= max|p|, and cuts the seven others (toward zero) below 2^(e-13): an
    error below one step each, with a second moment of at most step²/3.  For
    products of independent signs the errors add in squares,
    σ² = Σ_eights 7/3·(2^-13·max|p|)², and max|p|² is at most the eight's sum
    of squares.  Magnitudes of codes count as 2^-6 at least, the lowest
    exponent that the format holds."""
    (x, s), (w, t) = a, b
    x = np.maximum(np.abs(x), 2.0 ** -6) * expand(s, 1, *x.shape)
    w = np.maximum(np.abs(w), 2.0 ** -6) * expand(t, BLOCK, *w.shape)
    return 2.0 ** -13 * np.sqrt(7 / 3 * ((x * x) @ (w * w).T))


def activation(x, kind: str) -> np.ndarray:
    if kind == "silu":
        return x * special.expit(x)
    if kind == "gelu":
        return x * special.ndtr(x)
    return x * special.expit(2 * np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3))


def gated(a, g, u, kind: str, grouped: bool = False):
    """(act(A·Gᵀ)·(A·Uᵀ), bound of its fp32 error): the activations' slopes
    stay below 1.13; their fp32 evaluation is given eight units, and the
    exponent of gelu_tanh, rounded before exp, |x| + |x|³/8 more."""
    K = a[0].shape[1]
    cg, mg = matmul(a, g)
    cu, mu = matmul(a, u)
    eg, eu = accumulation_bound(mg, K, grouped), accumulation_bound(mu, K, grouped)
    f = activation(cg, kind)
    z = np.minimum(np.abs(cg) + np.abs(cg) ** 3 / 8, 100.0)
    ef = 1.13 * eg + np.abs(f) * 2.0 ** -24 * (8 + 4 * z) + 1e-37
    return f * cu, ef * (np.abs(cu) + eu) + np.abs(f) * eu + np.abs(f * cu) * 2.0 ** -23
