"""Attention over the paged cache at the ends of the types: scores that are NaN, scores at and
past fp32's range, many small probabilities, large and small values."""
import numpy as np
import pytest
import torch

import any_precision_weight_amd as apw
import attn_ref as ref
from gpu_util import ctx
from test_gpu_attn import Batch, attend, check, np64, queries, rng_of, same

pytestmark = pytest.mark.gpu

BOTH = [apw.attn_decode, apw.attn_prefill]


# ------------------------------------------------------------------ scores that are NaN

def put_nan_keys(bt, rng, b, positions, heads=None):
    """Keys with a NaN (all heads, or one) at these positions of sequence b."""
    for p in positions:
        row = rng.standard_normal((bt.Hkv, bt.D))
        row[slice(None) if heads is None else heads, 3] = np.nan
        bt.cache.put("k", bt.table[b, p // bt.page], p % bt.page, row)


# whole in one launch (8 waves, 4 waves, another width), and in parts
NAN_CASES = [("f16", 64, 2, 2, [33, 40, 1, 200]), ("bf16", 128, 8, 2, [129, 33, 700]), ("bf16", 256, 4, 2, [65, 300]),
             ("f16", 128, 6, 1, [3000, 33]), ("bf16", 64, 4, 4, [2500, 900])]


@pytest.mark.parametrize("c8", [False, True])
@pytest.mark.parametrize("t,D,Hq,Hkv,lens", NAN_CASES)
@pytest.mark.parametrize("fn", BOTH)
def test_a_query_with_a_nan_gives_nan(fn, t, D, Hq, Hkv, lens, c8):
    """In its own head's row, and in no other."""
    rng = rng_of("nan query", t, D, Hq, Hkv, lens, c8)
    bt = Batch(rng, lens, None if fn is apw.attn_decode else [min(n, 5) for n in lens], Hkv, D, 32, t, c8)
    q = queries(rng, bt.T, Hq, D, t)
    q[0, 7] = float("nan")
    q[bt.T - 1, (Hq - 1) * D + 5] = float("nan")
    g = np64(check(fn, bt, q, Hq)).reshape(bt.T, Hq, D)
    assert np.isnan(g[0, 0]).all() and np.isnan(g[-1, -1]).all() and np.isfinite(g[0, 1:]).all()


@pytest.mark.parametrize("c8", [False, True])
@pytest.mark.parametrize("fn", BOTH)
def test_a_key_with_a_nan_gives_nan_wherever_it_lies(fn, c8):
    """Alone in its tile, and so in its wave; beside finite ones; in one head of two; first and last."""
    rng = rng_of("nan key", c8)
    lens = [33, 65, 40, 161, 32, 900]
    bt = Batch(rng, lens, None if fn is apw.attn_decode else [1] * 6, 2, 128, 32, "f16", c8)
    for b, p in enumerate((32, 64, 3, 160, 31, 897)):
        put_nan_keys(bt, rng, b, [p], heads=b % 2)
    q = queries(rng, bt.T, 4, 128, "f16")
    g = np64(check(fn, bt, q, 4)).reshape(6, 2, 2, 128)
    for b in range(6):
        assert np.isnan(g[b, b % 2]).all() and np.isfinite(g[b, 1 - b % 2]).all()
    # out of the window, and out of mind
    assert np.isfinite(np64(check(fn, bt, q, 4, window=2, sinks=1))[2]).all()


@pytest.mark.parametrize("c8", [False, True])
@pytest.mark.parametrize("fn", BOTH)
def test_a_part_of_nothing_but_nan_keys_gives_nan(fn, c8):
    """Whole tiles, waves and parts of them, beside finite ones, and nothing else at all."""
    rng = rng_of("nan part", c8)
    lens = [5000, 3000, 400, 64]
    bt = Batch(rng, lens, None if fn is apw.attn_decode else [2, 1, 3, 1], 1, 64, 64, "bf16", c8)
    put_nan_keys(bt, rng, 0, range(2048, 4096))
    put_nan_keys(bt, rng, 1, range(3000))
    put_nan_keys(bt, rng, 2, range(128, 160))
    put_nan_keys(bt, rng, 3, range(64))
    q = queries(rng, bt.T, 2, 64, "bf16")
    assert np.isnan(np64(check(fn, bt, q, 2))).all()
    # a window of 200 with 100 first tokens sees none of them in sequences 0 and 2
    g = np64(check(fn, bt, q, 2, window=200, sinks=100)).reshape(bt.T, -1)
    assert np.isfinite(g[0]).all()


@pytest.mark.parametrize("fn", BOTH)
def test_8_bit_rows_of_nan(fn):
    rng = rng_of("nan out8")
    for lens in ([40, 7], [3000, 7]):
        bt = Batch(rng, lens, None if fn is apw.attn_decode else [1, 1], 1, 128, 32, "bf16", False)
        q = queries(rng, 2, 2, 128, "bf16")
        q[0, 128:] = float("nan")
        _, _, scale = attend(fn, bt, q, 2, out8=True)
        same(np.isnan(np64(scale)), np.array([[False, True], [False, False]]))


# ------------------------------------------------------------------ large scores

def fill_column(bt, rng, keys):
    """Sequence b's key at position p is keys[b][p] in column 0 and zeros; values as always."""
    for b, n in enumerate(bt.lens):
        for p in range(int(n)):
            row = np.zeros((bt.Hkv, bt.D))
            row[:, 0] = keys[b][p]
            pg, at = bt.table[b, p // bt.page], p % bt.page
            bt.cache.put("k", pg, at, row)
            bt.cache.put("v", pg, at, rng.standard_normal((bt.Hkv, bt.D)))


def check_largest(fn, bt, q, Hq, scale):
    """Rows against the mean of the values whose scores are the largest (the others' weights
    are e^-200 and less of theirs), or of all values where the scores differ by less than
    2^-18: equal weights are exact in any type, or off by 2^-18 each and in the sum.  So the
    errors are those of the values' scales (an 8-bit cache: p_err of each), of fp32 sums, and
    half a step."""
    g = np64(attend(fn, bt, q, Hq, scale)[0]).reshape(bt.T, Hq, bt.D)
    q = np64(q).reshape(bt.T, Hq, bt.D)
    p_err = 2.0 ** -8 if bt.c8 and bt.t == "bf16" and fn is apw.attn_prefill else 2.0 ** -15
    rows = [(bt.cache.rows("k", bt.table[b], int(n)), bt.cache.rows("v", bt.table[b], int(n)))
            for b, n in enumerate(bt.lens)]
    for row, b, pos in ref.tokens(bt.lens, bt.offsets, bt.T):
        K, V = (x[:, :pos + 1] for x in rows[b])
        for h in range(Hq):
            s = K[h * bt.Hkv // Hq] @ q[row, h] * scale
            off = s.max() - s
            w = (off < 2.0 ** -18).astype(np.float64)
            assert np.all((off > 200) | (w == 1))  # the case says what it says it does
            v = V[h * bt.Hkv // Hq]
            want, size = w @ v / w.sum(), w @ np.abs(v) / w.sum()
            tol = (np.abs(want) + size * 2.0 ** -7) * ref.HALF_STEP[bt.t] + ref.SMALLEST[bt.t] + size * (
                p_err + 2.0 ** -16 + (len(s) + 64) * 2.0 ** -23)
            d = np.abs(g[row, h] - want)
            assert np.all(d <= tol), (row, h, d.max(), g[row, h][:4], want[:4])


@pytest.mark.parametrize("c8", [False, True])
@pytest.mark.parametrize("t,top", [("f16", 60000.0), ("bf16", 2.0 ** 60)])
@pytest.mark.parametrize("scale", [1.0, 1000.0, 2.0 ** 100, -1.0, -(2.0 ** 90), 0.0, 1e-42])
@pytest.mark.parametrize("fn", BOTH)
def test_the_largest_of_large_scores_has_the_weight(fn, scale, t, top, c8):
    """Scores up to 2^32 (fp16) and 2^120 (bf16), whose product with the scale may pass fp32's
    range: two largest ones, all of them the same, and all of them negative; rows of small
    scores beside those of large ones; whole and in parts."""
    rng = rng_of("large", scale, t, c8)
    for lens, news in (([200, 45, 64], [70, 3, 64]), ([3000], [4])):
        bt = Batch(rng, lens, None if fn is apw.attn_decode else news, 1, 64, 32, t, c8, filled=False)
        q = torch.zeros((bt.T, 2 * 64), dtype=ref.TORCH[t])
        q[:, 0], q[:, 64] = top, 1.0
        mixed = [rng.choice([-top, 0.0, top / 2], n) for n in lens]
        for x in mixed:
            x[[3, -2]] = top
            x[[0, 5]] = -1.5 * top if t == "bf16" else -65504.0
        below = [np.full(n, -top) for n in lens]
        for x in below:
            x[[1, -1]] = -top / 2
        for keys in (mixed, [np.full(n, -top) for n in lens], below):
            fill_column(bt, rng, keys)
            check_largest(fn, bt, q, 2, scale)


# ------------------------------------------------------------------ small probabilities

def first_token_case(n, t, gap, news, rng, D=64):
    """One token a third of the way with exp(gap) times the weight of each of the others."""
    bt = Batch(rng, [n], news, 1, D, 256, t, False, filled=False)
    idx = {x: ref.place(x, 256, D, 2) for x in "kv"}
    keys = np.zeros((n, D))
    keys[n // 3, 0] = gap
    values = 1.0 + rng.standard_normal((n, D)) * 0.1
    values[n // 3] = 0.0
    for x, rows in (("k", ref.round16(keys, t)), ("v", ref.round16(values, t))):
        for i in range(-(-n // 256)):
            part = rows[i * 256:(i + 1) * 256]
            bt.cache.data[x][bt.table[0, i], 0, idx[x][:len(part)].ravel()] = part.ravel()
    q = torch.zeros((bt.T, D), dtype=ref.TORCH[t])
    q[:, 0] = 1.0
    return bt, q


@pytest.mark.parametrize("gap", [14.3, 16.25, 17.3, 18.0, 20.0])
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("n,fn,news", [(20000, apw.attn_decode, None), (20000, apw.attn_prefill, [2]), (700, apw.attn_decode, None),
                                       (700, apw.attn_prefill, [700]), (131072, apw.attn_decode, None)])
def test_many_small_probabilities_beside_a_large_one(n, fn, news, t, gap):
    """Probabilities of 2^-20 to 2^-29 of the largest, whose token's value is zero: the output is theirs alone.

    As the sum of two 16-bit numbers of probabilities up to 2^15 they are off by half of
    fp16's smallest number, 2^-25 of 2^15; prefill's, up to 2^7 and one number, by 2^-32 of the
    largest beside their rounding."""
    rng = rng_of("small", n, t, gap)
    bt, q = first_token_case(n, t, gap, news, rng)
    decode = fn is apw.attn_decode
    p_err = 2.0 ** -15 if decode else ref.HALF_STEP[t]
    floor = 0.0 if t == "bf16" else 2.0 ** -40 if decode else 2.0 ** -32
    got = np64(attend(fn, bt, q, 1, 1.0)[0]).reshape(bt.T, 1, 64)
    want, bound, _ = ref.attention(bt.cache, bt.table, bt.lens, bt.offsets, np64(q).reshape(bt.T, 1, 64), 1.0, 0, 0, 1 << 30,
                                   p_err, t, floor)
    off = np.abs(got - want)
    assert np.all(off <= bound), (off.max(), want.ravel()[-4:], got.ravel()[-4:], bound.ravel()[-4:])


@pytest.mark.parametrize("top", [256.0, 704.0])
@pytest.mark.parametrize("fn,lens,news", [(apw.attn_decode, [600, 90], None), (apw.attn_prefill, [600, 90], [600, 90]),
                                          (apw.attn_decode, [4000], None), (apw.attn_prefill, [4000], [3])])
def test_small_differences_of_large_scores(fn, lens, news, top):
    """Scores of 2^16 and 2^19, exact as fp32 sums of two products, that rise by 20 along the
    sequence: the differences count, so the maximum's own rounding must not.  Beside the
    probabilities' rounding each may be off by 2^-13 (an exponent's rounding below 2^10)."""
    rng = rng_of("differences", lens, top)
    bt = Batch(rng, lens, news, 1, 64, 32, "f16", False, filled=False)
    for b, n in enumerate(lens):
        for p in range(n):
            row = np.zeros((1, 64))
            row[0, 0], row[0, 1] = top, np.rint(p * 160 / n) / 8
            bt.cache.put("k", bt.table[b, p // 32], p % 32, row)
            bt.cache.put("v", bt.table[b, p // 32], p % 32, rng.standard_normal((1, 64)) + p / n)
    q = torch.zeros((bt.T, 64), dtype=torch.float16)
    q[:, 0], q[:, 1] = top, 1.0
    g = np64(attend(fn, bt, q, 1, 1.0)[0])
    p_err = 2.0 ** -15 if fn is apw.attn_decode else 2.0 ** -11
    for row, b, pos in ref.tokens(bt.lens, bt.offsets, bt.T):
        K, V = (bt.cache.rows(x, bt.table[b], pos + 1)[0] for x in "kv")
        s = K[:, 0] * top + K[:, 1]
        assert np.all(s == s.astype(np.float32))
        w = np.exp(s - s.max())
        want, size = w @ V / w.sum(), w @ np.abs(V) / w.sum()
        tol = (np.abs(want) + size * 2.0 ** -8) * 2.0 ** -11 + size * (p_err + 2.0 ** -13 + (pos + 65) * 2.0 ** -23)
        d = np.abs(g[row] - want)
        assert np.all(d <= tol), (row, (d / tol).max(), d.max())


@pytest.mark.parametrize("fn,lens,news", [(apw.attn_decode, [300, 40], None), (apw.attn_prefill, [300, 40], [20, 40]),
                                          (apw.attn_decode, [3000], None), (apw.attn_prefill, [3000], [3])])
@pytest.mark.parametrize("value", [1.0, float("inf"), float("nan")])
def test_nothing_but_scores_of_minus_infinity_is_zeros_whatever_the_values_are(fn, lens, news, value):
    """Head 0's scores are all -infinity; head 1's query is turned, and sees +infinity only."""
    rng = rng_of("minus values", value)
    for t in ("f16", "bf16"):
        bt = Batch(rng, lens, news, 1, 64, 32, t, False, filled=False)
        for b, n in enumerate(lens):
            for p in range(n):
                row = np.zeros((1, 64))
                row[0, 0] = -np.inf
                bt.cache.put("k", bt.table[b, p // 32], p % 32, row)
                row = rng.standard_normal((1, 64))
                row[0, p % 64] = value
                bt.cache.put("v", bt.table[b, p // 32], p % 32, row)
        q = torch.zeros((bt.T, 128), dtype=ref.TORCH[t])
        q[:, 0], q[:, 64] = 1.0, -1.0
        g = np64(attend(fn, bt, q, 2)[0])
        assert np.all(g[:, :64] == 0), np.argwhere(g[:, :64] != 0)[:4]
        assert np.isnan(g[:, 64:]).all()


# ------------------------------------------------------------------ large values

@pytest.mark.parametrize("fn,lens,news", [(apw.attn_decode, [300, 40], None), (apw.attn_prefill, [300, 40], [200, 40]),
                                          (apw.attn_decode, [3000], None), (apw.attn_prefill, [3000], [3])])
@pytest.mark.parametrize("c8", [False, True])
def test_the_largest_bf16_values(fn, lens, news, c8):
    """Sums of many of them, in decode of 16-bit rows the largest there are: their mean is a number.
    (Prefill's probabilities and those times an 8-bit row's scale are off by 2^-8 each, and so a mean of the
    type's largest may come out as its infinity: half of it there.)"""
    rng = rng_of("values", lens, c8)
    top = 2.0 ** 126 if c8 else 2.0 ** 128 - 2.0 ** 120 if fn is apw.attn_decode else 2.0 ** 127
    bt = Batch(rng, lens, news, 1, 128, 32, "bf16", c8, filled=False)
    for b, n in enumerate(lens):
        for p in range(n):
            row = 0.3 * p / n * rng.standard_normal((1, 128))
            bt.cache.put("k", bt.table[b, p // 32], p % 32, row)
            row = np.full((1, 128), top)
            row[0, 1], row[0, 2:] = -top, top * rng.choice([1.0, -1.0, 0.5], 126)
            bt.cache.put("v", bt.table[b, p // 32], p % 32, row)
    q = queries(rng, bt.T, 2, 128, "bf16", 3.0)
    g = np64(check(fn, bt, q, 2)).reshape(bt.T, 2, 128)
    assert np.all(np.abs(g[:, :, 0] - top) <= top * 2.0 ** -6)


@pytest.mark.parametrize("fn,lens,news", [(apw.attn_decode, [300, 40], None), (apw.attn_prefill, [300, 40], [200, 40]),
                                          (apw.attn_decode, [3000], None), (apw.attn_prefill, [3000], [3])])
@pytest.mark.parametrize("c8", [False, True])
def test_small_bf16_values(fn, lens, news, c8):
    """2^-64 and less, with weights down to 2^-20: their products are numbers too."""
    rng = rng_of("small values", lens, c8)
    bt = Batch(rng, lens, news, 1, 128, 32, "bf16", c8, filled=False)
    for b, n in enumerate(lens):
        for p in range(n):
            bt.cache.put("k", bt.table[b, p // 32], p % 32, 0.3 * rng.standard_normal((1, 128)))
            bt.cache.put("v", bt.table[b, p // 32], p % 32, rng.standard_normal((1, 128)) * 2.0 ** -64)
    check(fn, bt, queries(rng, bt.T, 2, 128, "bf16", 3.0), 2)


# ------------------------------------------------------------------ two walks over the same steps

@pytest.mark.parametrize("c8", [False, True])
@pytest.mark.parametrize("t,D,Hq,Hkv", [("f16", 64, 4, 2), ("bf16", 128, 8, 2), ("f16", 128, 6, 1), ("bf16", 256, 2, 2)])
def test_prefill_step_by_step_gives_the_bits_of_the_pipeline(t, D, Hq, Hkv, c8):
    """A value that is not finite where no row sees it (behind a sequence's end) makes a row
    tile walk its steps one after the other, each staged, waited for and used by itself; with
    zeros there the copies run two steps ahead of the products.  The operations are the same."""
    rng = rng_of("walks", t, D, Hq, Hkv, c8)
    lens, news = [1500, 333, 70, 41], [260, 333, 3, 41]
    bt = Batch(rng, lens, news, Hkv, D, 64, t, c8)
    q = queries(rng, bt.T, Hq, D, t, 2.0)
    runs = []
    for bad in (True, False):
        if not bad:  # every page of the pool past the sequences' ends, and those of nobody
            for x in "kv":
                data, scale = bt.cache.data[x], bt.cache.scale[x]
                if c8:
                    data[data == 0x7F] = 0
                    scale[np.isnan(scale)] = 0.0
                else:
                    data[np.isnan(data)] = 0.0
        for window, sinks in ((0, 0), (300, 70)):
            runs.append(check(apw.attn_prefill, bt, q, Hq, window=window, sinks=sinks))
    for a, b in zip(runs[:2], runs[2:]):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("c8", [False, True])
def test_a_context_of_separate_launches_gives_the_same_bits(c8, monkeypatch):
    monkeypatch.setenv("APMOE_UNFUSED", "1")
    other = apw.Context(0)
    monkeypatch.delenv("APMOE_UNFUSED")
    rng = rng_of("separate", c8)
    bt = Batch(rng, [1000, 77], [40, 77], 2, 128, 32, "bf16", c8)
    q = queries(rng, bt.T, 8, 128, "bf16")
    a, b = (attend(apw.attn_prefill, bt, q, 8, out8=True, c=c) for c in (ctx(), other))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    bt.offsets, bt.T = None, 2
    a, b = (attend(apw.attn_decode, bt, q[:2], 8, out8=True, c=c) for c in (ctx(), other))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    other.close()


@pytest.mark.parametrize("fn", BOTH)
def test_lengths_below_zero_are_empty(fn):
    """Their rows are zeros and see nothing, with a window and without; nothing of them is stored."""
    rng = rng_of("negative")
    lens = [-1, -(1 << 31), 40, -5, -(1 << 31) + 3]
    bt = Batch(rng, lens, None if fn is apw.attn_decode else [2, 1, 3, 70, 1], 2, 64, 32, "f16", False)
    q = queries(rng, bt.T, 4, 64, "f16")
    for window, sinks in ((0, 0), (7, 3), (1 << 30, (1 << 31) - 1)):
        g = np64(check(fn, bt, q, 4, window=window, sinks=sinks))
        empty = np.ones(bt.T, bool)
        first = 2 if fn is apw.attn_decode else 3
        empty[first:first + (1 if fn is apw.attn_decode else 3)] = False
        assert np.all(g[empty] == 0) and np.any(g[~empty] != 0)
    kv, batch = bt.upload()
    before = [x.clone() for x in (bt.k, bt.v)]
    x = queries(rng, bt.T, 2, 64, "f16").cuda()
    apw.kv_append(ctx(), kv, batch, None, x, x, 0, None, 0, False, None)
    torch.cuda.synchronize()
    for a, b in zip(before, (bt.k, bt.v)):
        other = [p for p in range(bt.cache.n_pages) if p not in bt.table[2]]
        assert torch.equal(a[other].view(torch.int16), b[other].view(torch.int16))
