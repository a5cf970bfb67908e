"""Plain implementations in 64 bits of the 8-bit path (CPU, numpy): e4m3 rows with a
scale for each 128 columns, the norm, the product, the activation, the layer."""
from __future__ import annotations

import numpy as np

BLK = 128
TINY = 2.0 ** -126


def e4m3_table() -> np.ndarray:
    """Value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 fraction bits;
    0x7F / 0xFF are NaN, there is no infinity."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e.astype(np.float64) - 10))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


TABLE = e4m3_table()


def e4m3_round(v: np.ndarray) -> np.ndarray:
    """The nearest e4m3 value, ties to even (|v| <= 448 up to rounding)."""
    v = np.asarray(v, np.float64)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(v)
        ulp = np.exp2(np.maximum(e - 1, -6) - 3.0)
        return np.clip(np.rint(v / ulp) * ulp, -448.0, 448.0)


def encode(v: np.ndarray) -> np.ndarray:
    """Codes of values that e4m3 holds."""
    pos = TABLE[:127]
    c = np.searchsorted(pos, np.abs(v)).astype(np.uint8)
    return c | (np.signbit(v).astype(np.uint8) << 7)


def groups(C: int) -> int:
    return -(-C // BLK)


def quant(v: np.ndarray):
    """(values q, scales s) of rows v; s rounded to fp32."""
    R, C = v.shape
    q, s = np.empty((R, C)), np.empty((R, groups(C)))
    for g in range(groups(C)):
        p = v[:, g * BLK:(g + 1) * BLK]
        amax = np.abs(p).max(axis=1) if p.size else np.zeros(R)
        s[:, g] = np.maximum((amax / 448.0).astype(np.float32).astype(np.float64), TINY)
        with np.errstate(invalid="ignore"):
            q[:, g * BLK:(g + 1) * BLK] = e4m3_round(p / s[:, g:g + 1])
    return q, s


def spread(s: np.ndarray, C: int) -> np.ndarray:
    return np.repeat(s, BLK, axis=1)[:, :C]


def block_values(codes: np.ndarray, s: np.ndarray) -> np.ndarray:
    """Values of one matrix [N][K] with scales [ceil(N/128)][ceil(K/128)]."""
    N, K = codes.shape
    return TABLE[codes] * np.repeat(np.repeat(s.astype(np.float64), BLK, 0)[:N], BLK, 1)[:, :K]


def norm(x, residual, gamma, eps, store):
    """store: rounds to the residual's type (fp32 sum first)."""
    h = x.astype(np.float64)
    if residual is not None:
        h = store((x.astype(np.float32) + residual.astype(np.float32))).astype(np.float64)
    y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + np.float64(np.float32(eps))) * gamma.astype(np.float64)
    return h, y


def rows_of(perm, topk, gather, r0, r1):
    r = np.arange(r0, r1)
    return perm[r] // topk if gather else r


def product(xv, wv, perm, offsets, topk, gather):
    """(out, magnitude): out[r] = xv[src] . wv[e], and the same of the magnitudes."""
    R, N = int(offsets[-1]), wv[0].shape[0]
    out, mag = np.zeros((R, N)), np.zeros((R, N))
    for e in range(len(wv)):
        r0, r1 = int(offsets[e]), int(offsets[e + 1])
        if r1 > r0:
            s = rows_of(perm, topk, gather, r0, r1)
            out[r0:r1] = xv[s] @ wv[e].T
            mag[r0:r1] = np.abs(xv[s]) @ np.abs(wv[e]).T
    return out, mag


def silu(z):
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z))
