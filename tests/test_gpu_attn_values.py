"""Attention over the paged cache at the ends of the types: scores that are NaN."""
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
