"""The binding of the paged cache's calls: numbers that do not fit the C ABI's 32 bits are refused
there (ctypes would cut them off, and the call be another one)."""
import pytest
import torch

import any_precision_weight_amd as apw
from test_attn_host import Ctx, small

BIG = [1 << 31, 1 << 32, (1 << 32) + 5, (1 << 40) + 64, -(1 << 31) - 1]


def half(*s):
    return torch.zeros(s, dtype=torch.float16)


def batch(T=2, **kw):
    return apw.KvBatch(torch.zeros((2, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), T, **kw)


@pytest.mark.parametrize("n", BIG)
@pytest.mark.parametrize("name", ["window", "sinks"])
@pytest.mark.parametrize("fn", [apw.attn_decode, apw.attn_prefill])
def test_window_and_first_tokens(fn, name, n):
    a = dict(dict(window=0, sinks=0), **{name: n})
    with pytest.raises(ValueError, match=name):
        fn(Ctx, small(), batch(), half(2, 256), 4, 1.0, a["window"], a["sinks"], torch.zeros(64, dtype=torch.uint8),
           half(2, 256), stream=0)


@pytest.mark.parametrize("n", BIG)
def test_batch(n):
    with pytest.raises(ValueError, match="T="):
        batch(T=n)
    with pytest.raises(ValueError, match="max_len"):
        batch(max_len=n)


@pytest.mark.parametrize("n", BIG)
@pytest.mark.parametrize("name", ["page", "kv_heads", "head_dim"])
def test_cache(name, n):
    a = dict(dict(page=32, kv_heads=2, head_dim=64), **{name: n})
    with pytest.raises(ValueError):
        apw.KvCache(half(0, 4096), half(0, 4096), a["page"], a["kv_heads"], a["head_dim"])


@pytest.mark.parametrize("n", BIG)
def test_heads_and_rotation(n):
    c, b = small(), batch()
    with pytest.raises(ValueError, match="rot"):
        apw.kv_append(Ctx, c, b, half(2, 256), half(2, 128), half(2, 128), 4, None, n, False, half(2, 256), stream=0)
    with pytest.raises(ValueError, match="q_heads"):
        apw.kv_append(Ctx, c, b, None, half(2, 128), half(2, 128), n, None, 0, False, None, stream=0)
    with pytest.raises(ValueError, match="q_heads"):
        apw.attn_workspace(Ctx, c, b, n)
