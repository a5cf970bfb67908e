"""Plain implementations in 64 bits of the paged key-value cache (CPU, numpy): the order
inside a page, the rotation, the cache write, attention with a window and first tokens."""
from __future__ import annotations

import numpy as np
import torch

import fp8_ref

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SMALLEST = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half the spacing at zero


def round16(v: np.ndarray, t: str) -> np.ndarray:
    """The nearest value of type t, ties to even, rounded once (fp64 -> t through fp32 is
    rounded twice)."""
    bits, low, top = (11, -14, 65504.0) if t == "f16" else (8, -126, 2.0 ** 128 - 2.0 ** 120)
    v = np.asarray(v, np.float64)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(v)
        ulp = np.exp2(np.maximum(e - 1, low) - (bits - 1.0))
        r = np.rint(v / ulp) * ulp
    return np.where(np.abs(r) > top, np.copysign(np.inf, r), r)


def place(kind: str, page: int, D: int, size: int) -> np.ndarray:
    """[page][D] index of each token's columns among the elements of a head of a page."""
    t, d = np.arange(page)[:, None], np.arange(D)[None, :]
    if kind == "k":
        c = 16 // size
        return ((t // 16 * (D // c) + d // c) * 16 + t % 16) * c + d % c
    return ((t // 32 * 4 + t % 16 // 4) * D + d) * 8 + t % 32 // 16 * 4 + t % 4


class Cache:
    """A pool on the CPU: elements as values (16-bit types) or e4m3 codes."""

    def __init__(self, n_pages, page, heads, D, t, c8, fill=np.nan):
        self.n_pages, self.page, self.heads, self.D, self.t, self.c8 = n_pages, page, heads, D, t, c8
        n = (n_pages, heads, page * D)
        self.data = {x: np.full(n, 0x7F, np.uint8) if c8 else np.full(n, fill) for x in "kv"}
        self.scale = {x: np.full((n_pages, heads, page), fill) if c8 else None for x in "kv"}

    def put(self, kind, pg, at, rows):
        """rows [heads][D] of one token."""
        idx = place(kind, self.page, self.D, 1 if self.c8 else 2)[at]
        if self.c8:
            with np.errstate(invalid="ignore"):
                s = np.abs(rows).max(axis=1) / 448.0
                s = np.where(s < fp8_ref.TINY, fp8_ref.TINY, s.astype(np.float32).astype(np.float64))
                q = fp8_ref.e4m3_round(rows / s[:, None])
            codes = np.where(np.isnan(q), 0x7F, fp8_ref.encode(q)).astype(np.uint8)
            self.data[kind][pg][:, idx] = codes
            self.scale[kind][pg][:, at] = s
        else:
            self.data[kind][pg][:, idx] = round16(rows, self.t)

    def rows(self, kind, pages, n):
        """[heads][n][D] values of a sequence's first n tokens; NaN on no page."""
        idx = place(kind, self.page, self.D, 1 if self.c8 else 2)
        out = np.full((self.heads, max(1, -(-n // self.page)) * self.page, self.D), np.nan)
        for i in range(-(-n // self.page)):
            p = int(pages[i])
            if 0 <= p < self.n_pages:
                v = self.data[kind][p][:, idx]
                v = fp8_ref.TABLE[v] * self.scale[kind][p][:, :, None] if self.c8 else v
                out[:, i * self.page:(i + 1) * self.page] = v
        return out[:, :n]

    def torch(self, device):
        """(k, v, k_scale, v_scale) tensors."""
        out = []
        for x in "kv":
            d = torch.from_numpy(self.data[x])
            out.append((d if self.c8 else d.to(TORCH[self.t])).to(device))
        for x in "kv":
            out.append(None if not self.c8 else torch.from_numpy(self.scale[x].astype(np.float32)).to(device))
        return out


def rope_table(n_pos: int, rot: int, theta: float = 1e4) -> np.ndarray:
    a = np.arange(n_pos)[:, None] * theta ** (-np.arange(0, rot, 2) / max(rot, 1))
    return np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)


def rotate(x: np.ndarray, row: np.ndarray, rot: int, interleaved: bool) -> np.ndarray:
    """x [heads][D]; row: the position's cosines and sines."""
    x, h = np.asarray(x, np.float64).copy(), rot // 2
    a, b = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(h), np.arange(h, rot))
    c, s = row[:h].astype(np.float64), row[h:].astype(np.float64)
    u, w = x[:, a] * c - x[:, b] * s, x[:, a] * s + x[:, b] * c
    x[:, a], x[:, b] = u, w
    return x


def tokens(lens, offsets, T):
    """(row, sequence, position) of each row that belongs to a sequence."""
    if offsets is None:
        return [(b, b, int(n) - 1) for b, n in enumerate(lens)]
    out = []
    for b, n in enumerate(lens):
        new = int(offsets[b + 1] - offsets[b])
        out += [(int(offsets[b]) + i, b, int(n) - new + i) for i in range(new)]
    return [x for x in out if x[0] < T]


def append(cache: Cache, table, lens, offsets, q, k, v, rope, rot, interleaved, q_out, limit):
    """q [T][Hq][D], k, v [T][Hkv][D] values; writes cache and q_out (values)."""
    for row, b, pos in tokens(lens, offsets, k.shape[0]):
        if pos < 0 or pos >= limit or (rot and pos >= rope.shape[0]):
            continue
        p = int(table[b, pos // cache.page])
        if not 0 <= p < cache.n_pages:
            continue
        turn = (lambda x: rotate(x, rope[pos], rot, interleaved)) if rot else (lambda x: x.astype(np.float64))
        if q is not None:
            q_out[row] = round16(turn(q[row]), cache.t)
        cache.put("k", p, pos % cache.page, turn(k[row]))
        cache.put("v", p, pos % cache.page, v[row].astype(np.float64))


def attention(cache: Cache, table, lens, offsets, q, scale, window, sinks, limit, p_err, out_t, floor=2.0 ** -24):
    """(out [T][Hq][D], bound of the error, rows that belong to a sequence), for q values
    [T][Hq][D].

    The bound: a score is an fp32 sum of D exact products in any order, D 2^-23 of the
    magnitudes, scaled, with at most four more roundings of the score (its scale, the cache's
    scale, the maximum's subtraction) and 2^-21 for the exponential: relative errors of the
    probabilities of at most d = 2 x that.  They are normalised by their own sum, so the
    output is off by 2 d sum p |v|; their rounding for the second product p_err, and its
    fp32 sum (also over parts and waves) (n + 64) 2^-23 of sum p |v|.  Probabilities below
    fp16's normal range are off by `floor` of the largest.  Then half a step of the type."""
    T, Hq, D = q.shape
    G = Hq // cache.heads
    out, bound = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    live = np.zeros(T, bool)
    memo = {}
    for row, b, pos in tokens(lens, offsets, T):
        live[row] = True
        n = max(0, min(int(lens[b]), table.shape[1] * cache.page, limit))
        j = np.arange(n)
        here = np.array([0 <= int(table[b, i]) < cache.n_pages for i in range(-(-n // cache.page))], bool)
        m = (j <= pos) & here[j // cache.page]
        if window:
            m &= (pos - j < window) | (j < sinks)
        if not m.any():
            continue
        if b not in memo:
            memo[b] = cache.rows("k", table[b], n), cache.rows("v", table[b], n)
        K, V = (x[:, m] for x in memo[b])
        for h in range(Hq):
            k, v, x = K[h // G], V[h // G], q[row, h]
            with np.errstate(all="ignore"):
                s = k @ x * scale
                mag = np.abs(k) @ np.abs(x) * abs(scale)
                top = s.max()
                if top == -np.inf:
                    continue
                p = np.exp(s - top)
                L = p.sum()
                out[row, h] = o = p @ v / L
                d = 2 * ((D + 4) * 2.0 ** -23 * mag.max() + 2.0 ** -21)
                size = p @ np.abs(v) / L
                bound[row, h] = (np.abs(o) + size * 2 * d) * HALF_STEP[out_t] + SMALLEST[out_t] + size * (
                    2 * d + p_err + (m.sum() + 64) * 2.0 ** -23) + np.abs(v).sum(axis=0) * floor / L
    return out, bound, live
