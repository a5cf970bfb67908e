"""The paged key-value cache on the GPU, through the C ABI, against plain implementations in
64 bits (attn_ref): the rotation and the cache write bit for bit, both attentions within the
bound derived there, alone and as one decoder layer.

What lies in the cache where a row sees nothing is NaN in every test: places past a
sequence's end, pages of nobody, and in some tests later tokens of the same call."""
import zlib

import numpy as np
import pytest
import torch

import any_precision_weight_amd as apw
import attn_ref as ref
import fp8_ref
from gpu_util import ctx

pytestmark = pytest.mark.gpu

# roundings of the probabilities for the second product
ONE = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TWO = 2.0 ** -15  # two 16-bit numbers, bf16 at worst: 2^-8 of 2^-8, and the remainder's subtraction


def np64(t):
    return t.detach().cpu().double().numpy()


def rng_of(*key):
    return np.random.default_rng([zlib.crc32(str(k).encode()) for k in key])


def same(a, b):
    np.testing.assert_array_equal(a, b)


class Batch:
    """Sequences of given lengths on random pages of a pool, their caches filled with rows
    of the type's values."""

    def __init__(self, rng, lens, news, Hkv, D, page, t, c8, spare=3, filled=True, pad=0):
        self.t, self.c8, self.D, self.Hkv, self.page = t, c8, D, Hkv, page
        self.lens, self.B = np.asarray(lens), len(lens)
        need = [-(-max(0, int(n)) // page) for n in lens]
        n_pages = sum(need) + spare
        order = rng.permutation(n_pages)
        self.table = np.full((self.B, max(1, max(need))), -1)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.offsets = None if news is None else np.concatenate([[0], np.cumsum(news)])
        self.T = (self.B if news is None else int(self.offsets[-1])) + pad
        self.cache = ref.Cache(n_pages, page, Hkv, D, t, c8)
        if filled:
            for b, n in enumerate(lens):
                for p in range(max(0, int(n))):
                    pg, at = self.table[b, p // page], p % page
                    self.cache.put("k", pg, at, rng.standard_normal((Hkv, D)))
                    self.cache.put("v", pg, at, rng.standard_normal((Hkv, D)) * rng.choice([1.0, 1.0, 8.0]))

    def upload(self, max_len=0):
        self.k, self.v, self.ks, self.vs = self.cache.torch("cuda")
        kv = apw.KvCache(self.k, self.v, self.page, self.Hkv, self.D, self.ks, self.vs)
        i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
        return kv, apw.KvBatch(i32(self.table), i32(self.lens), self.T,
                               None if self.offsets is None else i32(self.offsets), max_len)


def queries(rng, T, Hq, D, t, gain=1.0):
    return torch.from_numpy((gain * rng.standard_normal((T, Hq * D))).astype(np.float32)).to(ref.TORCH[t])


def attend(fn, bt, q, Hq, scale=None, window=0, sinks=0, max_len=0, out8=False, c=None):
    """The call's (out, out8, out_scale) as 64-bit arrays; outputs are filled with 7 before."""
    kv, batch = bt.upload(max_len)
    c = c or ctx()
    qd = q.cuda()
    out = torch.full_like(qd, 7.0)[:, :].contiguous()
    o8 = torch.full(out.shape, 0x55, dtype=torch.uint8, device="cuda") if out8 else None
    osc = torch.full((bt.T, Hq * bt.D // 128), -1.0, device="cuda") if out8 else None
    ws = torch.full((apw.attn_workspace(c, kv, batch, Hq),), 0xFF, dtype=torch.uint8, device="cuda")
    fn(c, kv, batch, qd, Hq, bt.D ** -0.5 if scale is None else scale, window, sinks, ws, out, o8, osc)
    torch.cuda.synchronize()
    return out, o8, osc


def check(fn, bt, q, Hq, scale=None, window=0, sinks=0, max_len=0, out8=False):
    got, o8, osc = attend(fn, bt, q, Hq, scale, window, sinks, max_len, out8)
    p_err = TWO if fn is apw.attn_decode or (bt.c8 and bt.t == "f16") else ONE["bf16" if bt.c8 else bt.t]
    want, bound, live = ref.attention(bt.cache, bt.table, bt.lens, bt.offsets, np64(q).reshape(bt.T, Hq, bt.D),
                                      bt.D ** -0.5 if scale is None else scale, window, sinks, max_len or 1 << 30, p_err,
                                      bt.t)
    g = np64(got).reshape(want.shape)
    assert np.all(g[~live] == 7.0)  # rows behind the last sequence
    fine = np.isfinite(want)
    with np.errstate(invalid="ignore"):
        off = np.abs(g - want) - bound
    assert np.all(off[live & np.ones(bt.T, bool)][fine[live]] <= 0), (np.nanmax(off), np.argwhere(~(off <= 0))[:4])
    if not fine.all():
        same(g[live][~fine[live]], want[live][~fine[live]])
    if out8:
        s = np.repeat(np64(osc), 128, axis=1).reshape(want.shape)
        codes = o8.cpu().numpy().reshape(want.shape)
        assert np.all(codes[~live] == 0x55) and np.all(np64(osc)[~live] == -1.0)
        q8 = fp8_ref.TABLE[codes]
        err = bound + np.abs(want) * 2.0 ** -22  # without the 16-bit output's rounding it is smaller still
        top = lambda x: x.reshape(bt.T, -1, 128).max(axis=2)
        lo = np.maximum(top(np.abs(want) - err) / 448, fp8_ref.TINY) * (1 - 2.0 ** -22)
        hi = np.maximum(top(np.abs(want) + err) / 448, fp8_ref.TINY) * (1 + 2.0 ** -22)
        assert np.all((np64(osc) >= lo)[live]) and np.all((np64(osc) <= hi)[live])
        # half a step of e4m3 at the value, which the error may move
        v = (np.abs(want) + err) / s
        half = np.maximum(np.exp2(np.floor(np.log2(np.maximum(v, 2.0 ** -6)))) * 2.0 ** -4, 2.0 ** -10)
        assert np.all((np.abs(q8 * s - want) <= half * s + err)[live])
    return got


# ------------------------------------------------------------------ rotation and cache write

def append_case(rng, bt, Hq, rot, inter, n_pos, fused=True, max_len=0):
    t, D, Hkv, T = ref.TORCH[bt.t], bt.D, bt.Hkv, bt.T
    rows = torch.from_numpy(rng.standard_normal((T, (Hq + 2 * Hkv) * D)).astype(np.float32)).to(t)
    rows[:, -D:] *= torch.from_numpy(np.exp2(rng.integers(-20, 8, (T, 1))).astype(np.float32)).to(t)
    rope = ref.rope_table(n_pos, rot)
    cut = [0, Hq * D, (Hq + Hkv) * D, (Hq + 2 * Hkv) * D]
    dev = rows.cuda()
    parts = [dev[:, a:b] if fused else dev[:, a:b].contiguous() for a, b in zip(cut, cut[1:])]
    kv, batch = bt.upload(max_len)
    q_out = torch.full((T, Hq * D), 7.0, dtype=t, device="cuda")
    apw.kv_append(ctx(), kv, batch, parts[0] if Hq else None, parts[1], parts[2], Hq,
                  torch.from_numpy(rope).cuda() if rot else None, rot, inter, q_out if Hq else None)
    torch.cuda.synchronize()
    v64 = rows.double().numpy()
    q, k, v = (v64[:, a:b].reshape(T, -1, D) for a, b in zip(cut, cut[1:]))
    want_q = np.full((T, Hq, D), 7.0)
    ref.append(bt.cache, bt.table, bt.lens, bt.offsets, q if Hq else None, k, v, rope, rot, inter, want_q,
               max_len or 1 << 30)
    same(np64(q_out).reshape(want_q.shape), want_q)
    for got, x in ((bt.k, "k"), (bt.v, "v")):
        same(got.cpu().numpy() if bt.c8 else np64(got), bt.cache.data[x])
    if bt.c8:
        same(np64(bt.ks), bt.cache.scale["k"])
        same(np64(bt.vs), bt.cache.scale["v"])


@pytest.mark.parametrize("c8", [False, True])
@pytest.mark.parametrize("t,D,page,Hq,Hkv,rot,inter", [
    ("f16", 64, 32, 3, 1, 64, False), ("bf16", 128, 32, 8, 2, 128, False), ("f16", 128, 64, 4, 4, 128, True),
    ("bf16", 256, 128, 5, 1, 64, False), ("f16", 256, 256, 2, 2, 256, True), ("bf16", 64, 64, 1, 1, 16, True),
    ("bf16", 128, 256, 6, 3, 0, False), ("f16", 128, 32, 0, 2, 32, False), ("bf16", 64, 32, 40, 8, 48, False)])
def test_append(t, D, page, Hq, Hkv, rot, inter, c8):
    rng = rng_of("append", t, D, page, Hq, Hkv, rot, inter, c8)
    # one new token of each: pages begun, ended, in the middle; an empty sequence
    append_case(rng, Batch(rng, [1, 16, 17, 32, 33, 0, 100, 257], None, Hkv, D, page, t, c8, filled=False), Hq, rot,
                inter, 300)
    # ragged chunks over tiles and pages, none at all, more than the sequence has, padding behind
    append_case(rng, Batch(rng, [1, 70, 40, 33, 96, 5, 31], [1, 70, 9, 0, 33, 8, 31], Hkv, D, page, t, c8, filled=False,
                           pad=4), Hq, rot, inter, 300, fused=False)


@pytest.mark.parametrize("news", [None, [1, 1, 60, 3, 20]])
def test_append_leaves_out_rows_without_a_place(news):
    """No page, a page out of range, past max_len, past the rotation's table, before the sequence."""
    rng = rng_of("places", news)
    bt = Batch(rng, [40, 64, 50, 2, 90], news, 2, 128, 32, "bf16", True, filled=False)
    bt.table[0, 1] = -1
    bt.table[1, 1] = bt.cache.n_pages
    append_case(rng, bt, 4, 64, False, 45, max_len=80)


def test_append_special_values():
    """Infinities and NaN, largest and smallest numbers; e4m3 rows of zeros."""
    for t in ("f16", "bf16"):
        for c8 in (False, True):
            rng = rng_of("special", t, c8)
            bt = Batch(rng, [9, 3], [9, 3], 1, 64, 32, t, c8, filled=False)
            x = torch.zeros((12, 64), dtype=ref.TORCH[t])
            big = torch.finfo(ref.TORCH[t]).max
            x[1, 3], x[2, 5], x[3, 7], x[4, 9], x[5, 1], x[6, :] = float("nan"), float("inf"), -float("inf"), big, 1e-7, big
            kv, batch = bt.upload()
            apw.kv_append(ctx(), kv, batch, None, x.cuda(), x.cuda(), 0, None, 0, False, None)
            torch.cuda.synchronize()
            v = x.double().numpy().reshape(12, 1, 64)
            for row, b, pos in ref.tokens(bt.lens, bt.offsets, 12):
                if c8 and not np.isfinite(v[row]).all():
                    # stands for NaN: whatever the elements are, times the scale
                    s = np64(bt.ks)[bt.table[b, 0], 0, pos]
                    assert not np.isfinite(s)
                    bt.cache.scale["k"][bt.table[b, 0]][0, pos] = bt.cache.scale["v"][bt.table[b, 0]][0, pos] = s
                    for kind, got in (("k", bt.k), ("v", bt.v)):
                        idx = ref.place(kind, 32, 64, 1)[pos]
                        bt.cache.data[kind][bt.table[b, 0]][:, idx] = got.cpu().numpy()[bt.table[b, 0]][:, idx]
                        with np.errstate(invalid="ignore"):
                            assert np.isnan(fp8_ref.TABLE[got.cpu().numpy()[bt.table[b, 0]][0, idx]] * s).all()
                    continue
                bt.cache.put("k", bt.table[b, 0], pos, v[row])
                bt.cache.put("v", bt.table[b, 0], pos, v[row])
            for got, kind in ((bt.k, "k"), (bt.v, "v")):
                same(got.cpu().numpy() if c8 else np64(got), bt.cache.data[kind])
            if c8:
                same(np64(bt.ks), bt.cache.scale["k"])


# ------------------------------------------------------------------ one new token

LENS = [1, 2, 15, 16, 17, 31, 32, 33, 0, 63, 64, 65, 100, 127, 129, 160, 3]


@pytest.mark.parametrize("c8", [False, True])
@pytest.mark.parametrize("t,D,page,Hq,Hkv", [
    ("f16", 64, 32, 1, 1), ("bf16", 64, 64, 6, 2), ("f16", 128, 32, 8, 2), ("bf16", 128, 64, 16, 1),
    ("bf16", 128, 128, 20, 1), ("f16", 128, 256, 3, 3), ("f16", 256, 32, 10, 2), ("bf16", 256, 64, 33, 1)])
def test_decode(t, D, page, Hq, Hkv, c8):
    rng = rng_of("decode", t, D, page, Hq, Hkv, c8)
    bt = Batch(rng, LENS, None, Hkv, D, page, t, c8)
    q = queries(rng, bt.T, Hq, D, t, 2.0)
    check(apw.attn_decode, bt, q, Hq, out8=D >= 128)
    check(apw.attn_decode, bt, q, Hq, window=20, sinks=3)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 40), (32, 0), (33, 32), (64, 4), (97, 33), (1000, 7),
                                          (1 << 30, 0), (31, 1 << 30)])
def test_decode_window(window, sinks):
    rng = rng_of("window", window, sinks)
    for c8 in (False, True):
        bt = Batch(rng, LENS + [300], None, 2, 64, 32, "bf16", c8)
        check(apw.attn_decode, bt, queries(rng, bt.T, 4, 64, "bf16", 2.0), 4, window=window, sinks=sinks)


@pytest.mark.parametrize("c8", [False, True])
@pytest.mark.parametrize("t,D,page,Hq,Hkv,lens,window,sinks", [
    ("f16", 128, 128, 6, 1, [5000], 0, 0), ("bf16", 128, 32, 8, 2, [3001, 7, 0, 1500, 130], 0, 0),
    ("bf16", 64, 64, 3, 3, [2048, 2047, 2049, 64], 1000, 70), ("f16", 256, 64, 4, 2, [1700, 900], 0, 0),
    ("bf16", 128, 64, 18, 1, [4000, 1], 0, 0)])
def test_decode_in_parts(t, D, page, Hq, Hkv, lens, window, sinks, c8):
    rng = rng_of("parts", t, D, page, Hq, Hkv, lens, window, c8)
    bt = Batch(rng, lens, None, Hkv, D, page, t, c8)
    q = queries(rng, bt.T, Hq, D, t, 2.0)
    a = check(apw.attn_decode, bt, q, Hq, window=window, sinks=sinks, out8=D >= 128)
    b, _, _ = attend(apw.attn_decode, bt, q, Hq, window=window, sinks=sinks)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("c8", [False, True])
def test_decode_of_many_workgroups_in_parts(c8):
    """256 to 1023 workgroups, and more: parts of 16 tiles for the long sequences only."""
    rng = rng_of("many parts", c8)
    lens = list(rng.integers(0, 200, 38)) + [3000, 1400]
    bt = Batch(rng, lens, None, 8, 64, 64, "bf16", c8)
    check(apw.attn_decode, bt, queries(rng, bt.T, 8, 64, "bf16", 2.0), 8)
    lens = list(rng.integers(0, 40, 127)) + [5000, 2100, 600]
    bt = Batch(rng, lens, None, 8, 64, 256, "f16", c8)
    check(apw.attn_decode, bt, queries(rng, bt.T, 8, 64, "f16", 2.0), 8, window=4000, sinks=100)


@pytest.mark.parametrize("c8", [False, True])
def test_decode_of_long_sequences_whole(c8):
    """Many workgroups with up to 4096 tokens in 8 bits, and windows that leave little of a long cache."""
    rng = rng_of("whole", c8)
    lens = list(rng.integers(0, 60, 127)) + [4090, 2500]
    bt = Batch(rng, lens, None, 8, 64, 128, "bf16", c8)
    check(apw.attn_decode, bt, queries(rng, bt.T, 8, 64, "bf16", 2.0), 8)
    for window, sinks in ((700, 68), (700, 69), (1, 0), (0, 0), (3, (1 << 31) - 1)):
        bt = Batch(rng, [5000, 767, 0, 769], None, 2, 128, 64, "f16", c8)
        check(apw.attn_decode, bt, queries(rng, bt.T, 8, 128, "f16", 2.0), 8, window=window, sinks=sinks, out8=True)


@pytest.mark.parametrize("fn", [apw.attn_decode, apw.attn_prefill])
def test_a_long_tail_of_small_probabilities(fn):
    """One token with 2^15 times the weight of each of 20000 others, which have a third of the
    weight together: below fp16's normal numbers, and not to be lost."""
    rng = rng_of("tail")
    n, D = 20000, 64
    bt = Batch(rng, [n], None if fn is apw.attn_decode else [2], 1, D, 256, "f16", False, filled=False)
    idx = {x: ref.place(x, 256, D, 2) for x in "kv"}
    keys, values = np.zeros((n, D)), 1.0 + ref.round16(rng.standard_normal((n, D)) * 0.1, "f16")
    keys[n // 3, 0] = 15.0 * np.log(2.0)
    keys, values = ref.round16(keys, "f16"), ref.round16(values, "f16")
    values[n // 3] = -1.0
    for x, rows in (("k", keys), ("v", values)):
        for i in range(-(-n // 256)):
            part = rows[i * 256:(i + 1) * 256]
            bt.cache.data[x][bt.table[0, i], 0, idx[x][:len(part)].ravel()] = part.ravel()
    q = torch.zeros((bt.T, D), dtype=torch.float16)
    q[:, 0] = 1.0
    check(fn, bt, q, 1, scale=1.0)


def test_decode_of_more_sequences_than_a_wave():
    rng = rng_of("many")
    lens = list(rng.integers(0, 70, 200)) + [900]
    bt = Batch(rng, lens, None, 1, 64, 32, "f16", False)
    check(apw.attn_decode, bt, queries(rng, bt.T, 2, 64, "f16", 2.0), 2)


@pytest.mark.parametrize("fn", [apw.attn_decode, apw.attn_prefill])
def test_missing_pages_hold_nothing(fn):
    """Entries that a window has left behind, out of range, and a sequence with no page at all."""
    for c8 in (False, True):
        rng = rng_of("pages", c8)
        lens, news = [200, 100, 64, 10], None if fn is apw.attn_decode else [90, 100, 2, 10]
        bt = Batch(rng, lens, news, 2, 128, 32, "bf16", c8)
        bt.table[0, 2] = -1
        bt.table[1, 0], bt.table[1, 3] = bt.cache.n_pages, 1 << 30
        bt.table[2, :] = -(1 << 31)
        q = queries(rng, bt.T, 4, 128, "bf16", 2.0)
        check(fn, bt, q, 4)
        check(fn, bt, q, 4, window=50, sinks=33)


@pytest.mark.parametrize("fn", [apw.attn_decode, apw.attn_prefill])
def test_max_len_bounds_what_is_seen(fn):
    rng = rng_of("max_len")
    bt = Batch(rng, [200, 90, 300], None if fn is apw.attn_decode else [150, 90, 1], 1, 64, 32, "f16", False)
    q = queries(rng, bt.T, 2, 64, "f16")
    for n in (1, 95, 128, 129, 300, 1 << 20):
        check(fn, bt, q, 2, max_len=n)
    bt.lens = np.array([1 << 30, 90, (1 << 31) - 1])  # more than the pages hold
    if fn is apw.attn_decode:
        check(fn, bt, q, 2)


# ------------------------------------------------------------------ prompts

@pytest.mark.parametrize("c8", [False, True])
@pytest.mark.parametrize("t,D,page,Hq,Hkv", [
    ("f16", 64, 32, 1, 1), ("bf16", 64, 64, 6, 2), ("f16", 128, 32, 8, 2), ("bf16", 128, 64, 16, 1),
    ("bf16", 128, 128, 20, 1), ("f16", 128, 256, 3, 3), ("f16", 256, 32, 10, 2), ("bf16", 256, 64, 5, 1)])
def test_prefill(t, D, page, Hq, Hkv, c8):
    rng = rng_of("prefill", t, D, page, Hq, Hkv, c8)
    # whole prompts, chunks, one token, none, more rows than tokens, an empty sequence with rows
    lens, news = [1, 130, 70, 65, 200, 40, 5, 0, 64], [1, 130, 9, 1, 66, 0, 8, 2, 64]
    bt = Batch(rng, lens, news, Hkv, D, page, t, c8, pad=3)
    q = queries(rng, bt.T, Hq, D, t, 2.0)
    check(apw.attn_prefill, bt, q, Hq, out8=D >= 128)
    check(apw.attn_prefill, bt, q, Hq, window=20, sinks=3)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 40), (64, 0), (65, 64), (97, 33), (200, 129), (1000, 7),
                                          (1 << 30, 0), (31, 1 << 30)])
def test_prefill_window(window, sinks):
    rng = rng_of("prefill window", window, sinks)
    for c8 in (False, True):
        bt = Batch(rng, [300, 150, 33], [300, 20, 33], 2, 64, 32, "f16", c8)
        check(apw.attn_prefill, bt, queries(rng, bt.T, 2, 64, "f16", 2.0), 2, window=window, sinks=sinks)


@pytest.mark.parametrize("c8", [False, True])
@pytest.mark.parametrize("t,D,page,Hq,Hkv,lens,news,window,sinks", [
    ("f16", 128, 64, 8, 2, [3000], [4], 0, 0), ("bf16", 128, 32, 16, 1, [5000, 70, 0], [33, 70, 2], 0, 0),
    ("bf16", 64, 64, 3, 3, [2048, 1999, 64], [1, 130, 64], 1500, 70), ("f16", 256, 256, 4, 2, [1700, 900], [7, 40], 0, 0),
    ("bf16", 128, 128, 6, 1, [4100, 3], [60, 3], 2000, 600)])
def test_prefill_in_parts(t, D, page, Hq, Hkv, lens, news, window, sinks, c8):
    """Few rows behind long caches: split over the steps and joined."""
    rng = rng_of("prefill parts", t, D, page, Hq, Hkv, lens, news, window, c8)
    bt = Batch(rng, lens, news, Hkv, D, page, t, c8, pad=2)
    q = queries(rng, bt.T, Hq, D, t, 2.0)
    a = check(apw.attn_prefill, bt, q, Hq, window=window, sinks=sinks, out8=D >= 128)
    b, _, _ = attend(apw.attn_prefill, bt, q, Hq, window=window, sinks=sinks)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("c8", [False, True])
def test_prefill_in_parts_with_missing_pages_and_bad_values(c8):
    rng = rng_of("prefill parts, pages", c8)
    bt = Batch(rng, [2000, 1500], [20, 9], 2, 64, 32, "bf16", c8)
    bt.table[0, 10:40] = -1  # a part of nothing
    bt.table[1, 5] = bt.cache.n_pages
    for b, pos in ((0, 1985), (1, 1493)):
        row = rng.standard_normal((2, 64))
        row[1, 5] = np.nan
        bt.cache.put("v", bt.table[b, pos // 32], pos % 32, row)
    q = queries(rng, bt.T, 4, 64, "bf16")
    check(apw.attn_prefill, bt, q, 4)
    check(apw.attn_prefill, bt, q, 4, window=1200, sinks=40)


def test_prefill_without_offsets_is_decode():
    rng = rng_of("one row")
    bt = Batch(rng, LENS, None, 2, 128, 32, "bf16", False)
    q = queries(rng, bt.T, 8, 128, "bf16")
    check(apw.attn_prefill, bt, q, 8)


@pytest.mark.parametrize("c8", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_later_tokens_do_not_reach_earlier_rows(value, c8):
    """Values and keys that are not finite: in rows that see them, and in none before (or
    behind the window)."""
    rng = rng_of("later", value, c8)
    for t in ("f16", "bf16"):
        bt = Batch(rng, [150, 90], [150, 40], 2, 64, 32, t, c8)
        bad = value if not c8 else np.nan  # an e4m3 row with an infinity stands for NaN
        for b, pos in ((0, 77), (0, 140), (1, 70)):
            pg, at = bt.table[b, pos // 32], pos % 32
            row = rng.standard_normal((2, 64))
            row[1, 5] = bad
            bt.cache.put("v", pg, at, row)
        q = queries(rng, bt.T, 4, 64, t)
        check(apw.attn_prefill, bt, q, 4)
        check(apw.attn_prefill, bt, q, 4, window=30, sinks=2)
        # a key that is not finite: its score is a NaN or an infinity for who sees it
        pg, at = bt.table[0, 3], 10  # position 106
        row = rng.standard_normal((2, 64))
        row[0, :] = np.nan
        bt.cache.put("k", pg, at, row)
        check(apw.attn_prefill, bt, q, 4, window=30, sinks=2)


def test_scores_of_minus_infinity_only():
    """Nothing but such scores is nothing."""
    rng = rng_of("minus")
    for fn, news in ((apw.attn_decode, None), (apw.attn_prefill, [40])):
        bt = Batch(rng, [40], news, 1, 64, 32, "f16", False)
        for p in range(40):
            row = np.zeros((1, 64))
            row[0, 0] = -np.inf
            bt.cache.put("k", bt.table[0, p // 32], p % 32, row)
        q = torch.zeros((bt.T, 128), dtype=torch.float16)
        q[:, 0] = 1.0
        q[:, 1:64] = 0.0
        q[:, 64] = 1.0
        assert torch.all(attend(fn, bt, q, 2)[0] == 0)


@pytest.mark.parametrize("fn", [apw.attn_decode, apw.attn_prefill])
def test_large_and_zero_scales(fn):
    """Scores of thousands (one token has all the weight), of zero (all the same), negative."""
    rng = rng_of("scale")
    for t in ("f16", "bf16"):
        bt = Batch(rng, [200, 77], None if fn is apw.attn_decode else [200, 77], 1, 128, 32, t, False)
        q = queries(rng, bt.T, 3, 128, t, 4.0)
        for scale in (0.0, -0.3, 1e-6):
            check(fn, bt, q, 3, scale=scale)
        out, _, _ = attend(fn, bt, q, 3, scale=1000.0)
        assert torch.isfinite(out).all()


# ------------------------------------------------------------------ how they are called

def test_strided_queries_and_padded_rows():
    rng = rng_of("strided")
    bt = Batch(rng, [40, 90, 7], None, 2, 128, 32, "bf16", False)
    kv, batch = bt.upload()
    wide = queries(rng, 5, 12, 128, "bf16").cuda()  # more rows and columns than the call takes
    q = wide[:3, 256:256 + 8 * 128]
    ws = torch.empty(apw.attn_workspace(ctx(), kv, batch, 8), dtype=torch.uint8, device="cuda")
    a, b = (torch.empty((3, 1024), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for fn in (apw.attn_decode, apw.attn_prefill):
        fn(ctx(), kv, batch, q, 8, 0.1, 0, 0, ws, a)
        fn(ctx(), kv, batch, q.contiguous(), 8, 0.1, 0, 0, ws, b)
        assert torch.equal(a, b)


def test_pool_past_32_bits():
    """Pages whose elements lie beyond 2^32 bytes, and beyond 2^32 elements."""
    D, page, Hkv = 256, 256, 4
    n_pages = (1 << 32) // (page * D * Hkv) + 40  # 2^32 elements and some
    for c8 in (False, True):
        rng = rng_of("far", c8)
        bt = Batch(rng, [300, 500], [300, 20], Hkv, D, page, "f16", c8, spare=0, filled=False)
        t = torch.uint8 if c8 else torch.float16
        k, v = (torch.zeros((n_pages, Hkv, page * D), dtype=t, device="cuda") for _ in range(2))
        ks, vs = (torch.zeros((n_pages, Hkv, page), device="cuda") if c8 else None for _ in range(2))
        far = bt.table.copy()
        far[bt.table >= 0] = n_pages - 1 - bt.table[bt.table >= 0] * 7
        i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
        kv = apw.KvCache(k, v, page, Hkv, D, ks, vs)
        batch = apw.KvBatch(i32(far), i32(bt.lens), bt.T, i32(bt.offsets))
        x = torch.from_numpy(rng.standard_normal((2, bt.T, Hkv * D)).astype(np.float32)).half()
        # sequence 1's first 480 tokens, by a call of their own
        old = torch.from_numpy(rng.standard_normal((2, 480, Hkv * D)).astype(np.float32)).half()
        b2 = apw.KvBatch(i32(far[1:]), i32([480]), 480, i32([0, 480]))
        apw.kv_append(ctx(), kv, b2, None, old[0].cuda(), old[1].cuda(), 0, None, 0, False, None)
        apw.kv_append(ctx(), kv, batch, None, x[0].cuda(), x[1].cuda(), 0, None, 0, False, None)
        for lens, off, rows in (([480], [0, 480], old), (bt.lens, bt.offsets, x)):
            a = rows.double().numpy().reshape(2, -1, Hkv, D)
            ref.append(bt.cache, bt.table[1:] if len(lens) == 1 else bt.table, lens, off, None, a[0], a[1], None, 0, False,
                       None, 1 << 30)
        q = queries(rng, bt.T, Hkv, D, "f16", 2.0)
        out = torch.empty((bt.T, Hkv * D), dtype=torch.float16, device="cuda")
        ws = torch.empty(apw.attn_workspace(ctx(), kv, batch, Hkv), dtype=torch.uint8, device="cuda")
        apw.attn_prefill(ctx(), kv, batch, q.cuda(), Hkv, D ** -0.5, 0, 0, ws, out)
        one = apw.KvBatch(i32(far), i32(bt.lens), 2)
        last = q[[299, 319]]
        out1 = torch.empty((2, Hkv * D), dtype=torch.float16, device="cuda")
        apw.attn_decode(ctx(), kv, one, last.cuda(), Hkv, D ** -0.5, 0, 0, ws, out1)
        torch.cuda.synchronize()
        del k, v
        for o, qq, off, p_err in ((out, q, bt.offsets, TWO if c8 else ONE["f16"]), (out1, last, None, TWO)):
            want, bound, _ = ref.attention(bt.cache, bt.table, bt.lens, off, np64(qq).reshape(len(qq), Hkv, D), D ** -0.5,
                                           0, 0, 1 << 30, p_err, "f16")
            assert np.all(np.abs(np64(o).reshape(want.shape) - want) <= bound)
        del kv, ks, vs
        torch.cuda.empty_cache()


def captured(fn):
    fn()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    return g


def test_captured_and_replayed_with_growing_sequences():
    """One graph of append and decode, replayed as the sequences grow over tiles, pages and
    parts, with eager calls between; every replay equals the eager result."""
    rng = rng_of("graph")
    B, Hq, Hkv, D, page = 5, 8, 2, 128, 32
    width = 20
    n_pages = B * width
    kc, vc = (torch.zeros((n_pages, Hkv, page * D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv = apw.KvCache(kc, vc, page, Hkv, D)
    table = torch.from_numpy(rng.permutation(n_pages).astype(np.int32).reshape(B, width)).cuda()
    lens = torch.tensor([1, 30, 31, 0, 500], dtype=torch.int32, device="cuda")
    batch = apw.KvBatch(table, lens, B)
    rope = torch.from_numpy(ref.rope_table(width * page, D)).cuda()
    x = torch.empty((B, (Hq + 2 * Hkv) * D), dtype=torch.bfloat16, device="cuda")
    q, k, v = x[:, :Hq * D], x[:, Hq * D:(Hq + Hkv) * D], x[:, (Hq + Hkv) * D:]
    ws = torch.empty(apw.attn_workspace(ctx(), kv, batch, Hq), dtype=torch.uint8, device="cuda")
    q_out, out = (torch.empty((B, Hq * D), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step():
        apw.kv_append(ctx(), kv, batch, q, k, v, Hq, rope, D, False, q_out)
        apw.attn_decode(ctx(), kv, batch, q_out, Hq, D ** -0.5, 0, 0, ws, out)

    x.copy_(torch.randn_like(x))
    g = captured(step)
    for i in range(6):
        x.copy_(torch.randn_like(x))
        lens += torch.tensor([1, 1, 1, 0, 1], dtype=torch.int32, device="cuda") * (1 if i < 3 else 31)
        lens[4].clamp_(max=width * page)
        g.replay()
        a = out.clone()
        out.fill_(3.0)
        step()
        torch.cuda.synchronize()
        assert torch.equal(a, out)
        assert torch.all(a[3] == 0)


def test_two_streams_with_a_workspace_each():
    rng = rng_of("streams")
    bts = [Batch(rng, [2000, 50], None, 2, 128, 32, "f16", c8) for c8 in (False, True)]
    runs = []
    for bt in bts:
        kv, batch = bt.upload()
        q = queries(rng, 2, 8, 128, "f16").cuda()
        ws = torch.empty(apw.attn_workspace(ctx(), kv, batch, 8), dtype=torch.uint8, device="cuda")
        runs.append((kv, batch, q, ws, torch.empty_like(q), torch.empty_like(q), torch.cuda.Stream()))
    for kv, batch, q, ws, want, _, _ in runs:
        apw.attn_decode(ctx(), kv, batch, q, 8, 0.1, 0, 0, ws, want)
    torch.cuda.synchronize()
    for _ in range(20):
        for kv, batch, q, ws, _, out, st in runs:
            apw.attn_decode(ctx(), kv, batch, q, 8, 0.1, 0, 0, ws, out, stream=st)
    torch.cuda.synchronize()
    for _, _, _, _, want, out, _ in runs:
        assert torch.equal(want, out)


def test_a_context_without_fusion_and_the_drained_build_give_the_same_bits():
    rng = rng_of("safe")
    other = apw.Context(0, library=apw.load_library(apw.SAFE_LIB_PATH))
    for c8 in (False, True):
        bt = Batch(rng, [1000, 77], [40, 77], 2, 128, 32, "bf16", c8)
        q = queries(rng, bt.T, 8, 128, "bf16")
        a, b = (attend(apw.attn_prefill, bt, q, 8, out8=True, c=c) for c in (ctx(), other))
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        bt.offsets, bt.T = None, 2
        a, b = (attend(apw.attn_decode, bt, q[:2], 8, out8=True, c=c) for c in (ctx(), other))
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    other.close()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("c8", [False, True])
def test_a_decoder_layer_prompt_then_token_by_token(c8):
    """norm -> projection -> rotation and cache -> attention -> projection -> norm -> experts, for
    two prompts at once and then one token at a time with the same projected rows (a product of
    few rows may differ from one of many in the last bit): the cache gets the same bits, and
    the attention's rows differ by the roundings of the probabilities and of the output: 2^-11
    of the largest value each for the prompts' probabilities and for either output, and a
    little; 2^-8 covers them."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    c = ctx()
    H, Hq, Hkv, D, page, E, F, topk = 512, 8, 2, 128, 32, 4, 256, 2
    N = (Hq + 2 * Hkv) * D

    def weights(*shape):
        w = rnd(*shape) * shape[-1] ** -0.5
        nb = [-(-n // 128) for n in shape[-2:]]
        s = torch.full((*shape[:-2], *nb), float(w.abs().max() / 448), device="cuda")
        return (w / s[..., :1, :1]).to(torch.float8_e4m3fn).contiguous(), s

    wqkv, sqkv = weights(1, N, H)
    wo, so = weights(1, H, Hq * D)
    gu, gus = weights(E, 2 * F, H)
    gus = gus.view(E, 2, F // 128, H // 128).contiguous()
    dn, dns = weights(E, H, F)
    experts = apw.Fp8Experts(gu, gus, dn, dns)
    router = (rnd(E, H) * 0.05).half()
    gamma = torch.ones(H, dtype=torch.float16, device="cuda")
    prompts, extra = [45, 70], 5
    lens_all = [n + extra for n in prompts]
    width = -(-max(lens_all) // page)
    table = torch.arange(2 * width, dtype=torch.int32, device="cuda").view(2, width)
    rope = torch.from_numpy(ref.rope_table(width * page, D)).cuda()
    if c8:
        pool = lambda: torch.zeros((2 * width, Hkv, page * D), dtype=torch.uint8, device="cuda")
        sc = [torch.zeros((2 * width, Hkv, page), device="cuda") for _ in range(2)]
    else:
        pool = lambda: torch.zeros((2 * width, Hkv, page * D), dtype=torch.float16, device="cuda")
        sc = [None, None]
    kc, vc = pool(), pool()
    kv = apw.KvCache(kc, vc, page, Hkv, D, *sc)

    def layer(x, lens, offsets, decode, rows=None):
        T = x.shape[0]
        batch = apw.KvBatch(table, lens, T, offsets)
        e = lambda *s, dt=torch.float16: torch.empty(s, dtype=dt, device="cuda")
        f8 = lambda n: (e(T, n, dt=torch.uint8), e(T, n // 128, dt=torch.float32))
        x8, xs = f8(H)
        apw.norm(c, x, None, None, gamma, 1e-5, T, H, None, x8, xs)
        qkv = e(T, N)
        apw.gemm_fp8(c, x8, xs, wqkv, sqkv, 1, N, H, False, None, None, T, 1, qkv)
        if rows is not None:
            qkv = rows
        q = e(T, Hq * D)
        apw.kv_append(c, kv, batch, qkv[:, :Hq * D], qkv[:, Hq * D:(Hq + Hkv) * D], qkv[:, (Hq + Hkv) * D:], Hq, rope, D,
                      False, q)
        ws = torch.empty(apw.attn_workspace(c, kv, batch, Hq), dtype=torch.uint8, device="cuda")
        a, (a8, as_) = e(T, Hq * D), f8(Hq * D)
        call = apw.attn_decode if decode else apw.attn_prefill
        call(c, kv, batch, q, Hq, D ** -0.5, 0, 0, ws, a, a8, as_)
        o = e(T, H)
        apw.gemm_fp8(c, a8, as_, wo, so, 1, H, Hq * D, False, None, None, T, 1, o)
        h, y = x.clone(), e(T, H)
        y8, ys = f8(H)
        apw.norm(c, o, h, h, gamma, 1e-5, T, H, y, y8, ys)
        out = e(T, H)
        w2 = torch.empty(apw.moe_workspace_fp8(c, experts, T, topk), dtype=torch.uint8, device="cuda")
        apw.moe_forward_fp8(c, experts, y, y8, ys, router, None, T, topk, True, w2, out)
        torch.cuda.synchronize()
        return qkv, a, a8, as_, out

    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    xs_all = [rnd(n, H).half() for n in lens_all]
    whole = layer(torch.cat(xs_all), i32(lens_all), i32([0, lens_all[0], sum(lens_all)]), False)
    kept = [t.clone() for t in (kc, vc, *sc) if t is not None]
    for t in (kc, vc):
        t.zero_()
    at = [0, lens_all[0]]
    first_rows = torch.cat([torch.arange(at[b], at[b] + n, device="cuda") for b, n in enumerate(prompts)])
    first = layer(torch.cat([x[:n] for x, n in zip(xs_all, prompts)]), i32(prompts), i32([0, prompts[0], sum(prompts)]),
                  False, whole[0][first_rows])
    assert torch.isfinite(first[-1]).all()
    size = float(whole[0][:, (Hq + Hkv) * D:].abs().max())  # the largest value
    for i in range(extra):
        rows = torch.tensor([at[b] + prompts[b] + i for b in range(2)], device="cuda")
        step = layer(torch.cat([x[n + i:n + i + 1] for x, n in zip(xs_all, prompts)]),
                     i32([n + i + 1 for n in prompts]), None, True, whole[0][rows])
        assert float((step[1] - whole[1][rows]).abs().max()) <= size * 2.0 ** -8
        assert torch.isfinite(step[-1]).all()
        # the 8-bit rows stand for the 16-bit ones: half a step of each
        v8 = fp8_ref.TABLE[step[2].cpu().numpy()] * np.repeat(np64(step[3]), 128, axis=1)
        a64 = np64(step[1])
        s64 = np.repeat(np64(step[3]), 128, axis=1)
        assert np.all(np.abs(v8 - a64) <= np.maximum(np.abs(a64) * 2.0 ** -4, s64 * 2.0 ** -10) + np.abs(a64) * 2.0 ** -10)
    assert all(torch.equal(a, b) for a, b in zip(kept, [t for t in (kc, vc, *sc) if t is not None]))
