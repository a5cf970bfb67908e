"""Host-side checks of the paged key-value cache's calls that need no GPU: the C ABI's
refusals (arguments are checked before the context is looked into, so any address stands for
one here), the binding's checks of tensors, and the reference's own pins."""
import ctypes

import numpy as np
import pytest
import torch

import any_precision_weight_amd as apw
import attn_ref as ref

CTX = 0x1000
A = 0x10000000  # 256-byte aligned; never dereferenced


def call(fn, *args):
    return getattr(apw.lib(), fn)(*args)


def cache_desc(**kw):
    d = apw.KvCacheDesc()
    for k, v in dict(dict(dtype=apw.F16, n_pages=9, page=32, kv_heads=2, head_dim=128, k=A, v=A, k_scale=A, v_scale=A),
                     **kw).items():
        setattr(d, k, v)
    return d


def batch_desc(**kw):
    d = apw.KvBatchDesc()
    for k, v in dict(dict(B=3, T=3, max_pages=4, max_len=0, pages=A, lens=A, q_offsets=None), **kw).items():
        setattr(d, k, v)
    return d


def ref_of(d):
    return None if d is None else ctypes.byref(d)


def append_args(cache, batch, **kw):
    a = dict(ctx=CTX, cache=ref_of(cache), batch=ref_of(batch), q=A, qs=1024, k=A, ks=1024, v=A, vs=1024, dt=apw.F16,
             heads=4, rope=A, n_pos=100, rot=64, inter=0, q_out=A + 4096, stream=None)
    a.update(kw)
    return list(a.values())


def attn_args(cache, batch, **kw):
    a = dict(ctx=CTX, cache=ref_of(cache), batch=ref_of(batch), q=A, qs=1024, dt=apw.F16, heads=4, scale=0.1, window=0,
             sinks=0, ws=A, ws_bytes=1 << 40, out=A, out8=None, out_scale=None, stream=None)
    a.update(kw)
    return list(a.values())


CACHE = [(dict(dtype=apw.F32), 2), (dict(dtype=4), 2), (dict(dtype=apw.BF16), 2), (dict(page=16), 1), (dict(page=48), 1),
         (dict(page=512), 1), (dict(head_dim=96), 1), (dict(head_dim=512), 1), (dict(head_dim=0), 1),
         (dict(kv_heads=0), 1), (dict(kv_heads=1025), 1), (dict(n_pages=0), 1), (dict(k=None), 1), (dict(v=None), 1),
         (dict(k=A + 8), 1), (dict(v=A + 8), 1), (dict(dtype=apw.E4M3, k_scale=None), 1),
         (dict(dtype=apw.E4M3, v_scale=None), 1), (dict(dtype=apw.E4M3, v_scale=A + 4), 1)]
BATCH = [(dict(B=-1), 1), (dict(B=65537, T=65537), 1), (dict(T=-1), 1), (dict(T=1 << 24, q_offsets=A), 1), (dict(B=0), 1),
         (dict(max_pages=0), 1), (dict(max_pages=1 << 26), 1), (dict(max_len=-1), 1), (dict(pages=None), 1),
         (dict(lens=None), 1), (dict(T=4), 1), (dict(pages=A + 2), 1), (dict(lens=A + 1), 1), (dict(q_offsets=A + 2), 1)]
FNS = ["apmoe_kv_append", "apmoe_attn_decode", "apmoe_attn_prefill"]


def args_of(fn, cache, batch, **kw):
    return (append_args if fn == "apmoe_kv_append" else attn_args)(cache, batch, **kw)


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("kw,status", CACHE)
def test_cache_refusals(fn, kw, status):
    assert call(fn, *args_of(fn, cache_desc(**kw), batch_desc())) == status
    assert apw.lib().apmoe_last_error()


@pytest.mark.parametrize("fn", FNS)
@pytest.mark.parametrize("kw,status", BATCH)
def test_batch_refusals(fn, kw, status):
    assert call(fn, *args_of(fn, cache_desc(), batch_desc(**kw))) == status


@pytest.mark.parametrize("fn", FNS)
def test_missing_structures(fn):
    assert call(fn, *args_of(fn, None, batch_desc())) == apw.INVALID_ARG
    assert call(fn, *args_of(fn, cache_desc(), None)) == apw.INVALID_ARG


@pytest.mark.parametrize("fn", FNS)
def test_no_rows(fn):
    empty = batch_desc(B=0, T=0, max_pages=0, pages=None, lens=None)
    kw = dict(q=None, k=None, v=None, q_out=None) if fn == "apmoe_kv_append" else dict(q=None, out=None, ws=None)
    assert call(fn, *args_of(fn, cache_desc(), empty, **kw)) == apw.OK
    assert call(fn, *args_of(fn, cache_desc(), batch_desc(T=0, q_offsets=A), **kw)) == apw.OK


@pytest.mark.parametrize("kw,status", [
    (dict(ctx=None), 1), (dict(dt=apw.F32), 2), (dict(dt=apw.E4M3), 2), (dict(dt=-1), 2), (dict(heads=-1), 1),
    (dict(heads=1025), 1), (dict(rot=8), 1), (dict(rot=144), 1), (dict(rot=-16), 1), (dict(n_pos=0), 1),
    (dict(n_pos=-1), 1), (dict(rope=None), 1), (dict(rope=A + 4), 1), (dict(q=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(q_out=None), 1), (dict(q_out=A), 1), (dict(q=A + 2), 1), (dict(k=A + 8), 1),
    (dict(v=A + 8), 1), (dict(q_out=A + 8), 1), (dict(qs=511), 1), (dict(qs=504), 1), (dict(ks=248), 1),
    (dict(vs=1025), 1), (dict(vs=-256), 1), (dict(ks=1 << 60), 1)])
def test_append_refusals(kw, status):
    assert call("apmoe_kv_append", *append_args(cache_desc(), batch_desc(), **kw)) == status


@pytest.mark.parametrize("fn", FNS[1:])
@pytest.mark.parametrize("kw,status", [
    (dict(ctx=None), 1), (dict(dt=apw.F32), 2), (dict(dt=apw.BF16), 2), (dict(dt=apw.E4M3), 2), (dict(heads=0), 1),
    (dict(heads=3), 1), (dict(heads=1026), 1), (dict(heads=-2), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(scale=-1e31), 1), (dict(window=-1), 1), (dict(window=(1 << 30) + 1), 1), (dict(sinks=-1), 1),
    (dict(ws=None), 1), (dict(ws=A + 64), 1), (dict(ws_bytes=100), 1), (dict(q=None), 1), (dict(q=A + 8), 1),
    (dict(qs=508), 1), (dict(qs=504), 1), (dict(out=None), 1), (dict(out=A + 8), 1), (dict(out8=A), 1),
    (dict(out_scale=A), 1), (dict(out8=A + 8, out_scale=A), 1), (dict(out8=A, out_scale=A + 2), 1)])
def test_attention_refusals(fn, kw, status):
    assert call(fn, *attn_args(cache_desc(), batch_desc(), **kw)) == status


@pytest.mark.parametrize("fn", FNS[1:])
def test_8_bit_rows_need_whole_groups(fn):
    a = attn_args(cache_desc(head_dim=64), batch_desc(), out8=A, out_scale=A)
    assert call(fn, *a) == apw.UNSUPPORTED


def test_decode_takes_one_row_a_sequence():
    assert call("apmoe_attn_decode", *attn_args(cache_desc(), batch_desc(q_offsets=A))) == apw.INVALID_ARG


def workspace(cache, batch, heads):
    n = ctypes.c_size_t()
    st = call("apmoe_attn_workspace", CTX, ctypes.byref(cache), ctypes.byref(batch), heads, ctypes.byref(n))
    return st, n.value


def test_workspace():
    st, n = workspace(cache_desc(), batch_desc(), 4)
    assert st == apw.OK and n > 0
    # of a larger batch serves a smaller one, pointers are not looked at
    last = 0
    for B in (0, 1, 2, 7, 300, 65536):
        st, n = workspace(cache_desc(k=None, v=None), batch_desc(B=B, T=B, pages=None, lens=None), 4)
        assert st == apw.OK and n >= last
        last = n
    assert workspace(cache_desc(), batch_desc(), 3)[0] == apw.INVALID_ARG
    assert workspace(cache_desc(page=8), batch_desc(), 4)[0] == apw.INVALID_ARG
    assert call("apmoe_attn_workspace", CTX, ref_of(cache_desc()), ref_of(batch_desc()), 4, None) == apw.INVALID_ARG
    assert call("apmoe_attn_workspace", None, ref_of(cache_desc()), ref_of(batch_desc()), 4,
                ctypes.byref(ctypes.c_size_t())) == apw.INVALID_ARG


# ------------------------------------------------------------------ the binding (no GPU: CPU tensors are on device -1)

class Ctx:
    L, handle, device = apw.lib(), None, -1


def small(dtype=torch.float16, n_pages=3, page=32, heads=2, D=64, scales=False):
    mk = lambda: torch.zeros((n_pages, heads, page * D), dtype=dtype)
    sc = [torch.zeros((n_pages, heads, page)) for _ in range(2)] if scales else (None, None)
    return apw.KvCache(mk(), mk(), page, heads, D, *sc)


def test_binding_cache():
    assert small().desc.dtype == apw.F16 and small(torch.bfloat16).desc.dtype == apw.BF16
    assert small(torch.uint8, scales=True).desc.dtype == apw.E4M3
    with pytest.raises(ValueError, match="k_scale"):
        small(torch.uint8)
    with pytest.raises(ValueError, match="k: need"):
        small(torch.float32)
    with pytest.raises(ValueError, match="v: need"):
        apw.KvCache(torch.zeros(3, 64 * 64, dtype=torch.float16), torch.zeros(3, 64 * 63, dtype=torch.float16), 32, 2, 64)
    with pytest.raises(ValueError, match="k: need"):
        apw.KvCache(torch.zeros(3, 4096, dtype=torch.float16)[:, ::2], torch.zeros(3, 4096, dtype=torch.float16), 32, 1,
                    64)


def test_binding_batch():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    b = apw.KvBatch(i(3, 5), i(3), 3)
    assert (b.desc.B, b.desc.max_pages, b.desc.T) == (3, 5, 3)
    for pages, lens, off in [(i(3, 5), i(2), None), (i(15), i(3), None), (i(3, 5).long(), i(3), None),
                             (i(3, 5), i(3).long(), None), (i(3, 5), i(3), i(3)), (i(3, 10)[:, ::2], i(3), None)]:
        with pytest.raises(ValueError):
            apw.KvBatch(pages, lens, 3, off)


def test_binding_matrices():
    c, b = small(), apw.KvBatch(torch.zeros((2, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 2)
    h = lambda *s: torch.zeros(s, dtype=torch.float16)
    ok = dict(q=h(2, 256), k=h(2, 128), v=h(2, 128), rope=torch.zeros(8, 32), q_out=h(2, 256))
    for bad in [dict(q=h(2, 255)), dict(q=h(1, 256)), dict(k=h(2, 64)), dict(v=h(256)), dict(v=h(128, 2).t()),
                dict(q=h(2, 256).float()), dict(rope=torch.zeros(8, 16)), dict(rope=torch.zeros(8, 32).double()),
                dict(q_out=h(2, 255)), dict(q_out=h(2, 512)[:, ::2])]:
        a = dict(ok, **bad)
        with pytest.raises(ValueError):
            apw.kv_append(Ctx, c, b, a["q"], a["k"], a["v"], 4, a["rope"], 32, False, a["q_out"], stream=0)
    other = type("Other", (), dict(L=apw.lib(), handle=None, device=0))
    with pytest.raises(ValueError, match="the cache is on"):
        apw.kv_append(other, c, b, ok["q"], ok["k"], ok["v"], 4, ok["rope"], 32, False, ok["q_out"], stream=0)
    with pytest.raises(ValueError, match="ws"):
        apw.attn_decode(Ctx, c, b, ok["q"], 4, 1.0, 0, 0, None, h(2, 256), stream=0)


# ------------------------------------------------------------------ the reference

@pytest.mark.parametrize("kind,size", [("k", 1), ("k", 2), ("v", 2)])
@pytest.mark.parametrize("page,D", [(32, 64), (64, 128), (256, 256)])
def test_place_is_a_permutation(kind, size, page, D):
    p = ref.place(kind, page, D, size)
    assert np.array_equal(np.sort(p.ravel()), np.arange(page * D))


def test_rounding_once():
    v = np.random.default_rng(0).standard_normal(20000) * 10.0 ** np.random.default_rng(1).integers(-9, 6, 20000)
    for t in ("f16", "bf16"):
        x = torch.from_numpy(v.astype(np.float32))
        assert np.array_equal(ref.round16(x.double().numpy(), t), x.to(ref.TORCH[t]).double().numpy())
    # next to a border: through fp32 it would fall on the border and go to the even side
    assert ref.round16(1 + 2.0 ** -8 + 2.0 ** -40, "bf16") == 1 + 2.0 ** -7
    assert np.isinf(ref.round16(1e39, "bf16")) and np.isinf(ref.round16(65520.0, "f16"))


def test_attention_of_one_seen_token_is_its_value():
    c = ref.Cache(2, 32, 1, 64, "f16", False)
    rows = np.random.default_rng(2).standard_normal((33, 1, 64))
    table = np.array([[1, 0]])
    for t in range(33):
        c.put("k", table[0, t // 32], t % 32, rows[t])
        c.put("v", table[0, t // 32], t % 32, rows[t])
    out, _, live = ref.attention(c, table, [33], None, rows[:1], 1.0, 1, 0, 1 << 30, 0.0, "f16")
    np.testing.assert_allclose(out[0, 0], ref.round16(rows[32, 0], "f16"), rtol=1e-12)
    assert live[0]
