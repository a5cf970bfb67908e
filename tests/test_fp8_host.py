"""Host-side checks of the 8-bit path that need no GPU: the C ABI's refusals (arguments
are checked before the context is looked into, so any address stands for one here), the
binding's checks of tensors, and the reference's own pins."""
import ctypes

import numpy as np
import pytest
import torch

import any_precision_weight_amd as apw
import fp8_ref as ref
import fp8_tiles as tiles

CTX = 0x1000
A = 0x10000000  # 16-byte aligned; never dereferenced


def call(fn, *args):
    return getattr(apw.lib(), fn)(*args)


def norm_args(**kw):
    a = dict(ctx=CTX, x=A, xt=apw.F16, res=A + 4096, res_out=A + 4096, rt=apw.F32, gamma=A, eps=1e-5, T=4, H=64, y=A,
             y8=A, ys=A, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(ctx=None), 1), (dict(xt=3), 2), (dict(xt=-1), 2), (dict(rt=7), 2), (dict(H=0), 1), (dict(H=12), 1),
    (dict(H=65544), 1), (dict(T=-1), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(res=None), 1), (dict(res_out=None), 1), (dict(y8=None), 1), (dict(ys=None), 1),
    (dict(y=None, y8=None, ys=None), 1), (dict(x=None), 1), (dict(gamma=None), 1), (dict(x=A + 8), 1),
    (dict(gamma=A + 2), 1), (dict(res=A + 4), 1), (dict(res_out=A + 4), 1), (dict(y=A + 2), 1), (dict(y8=A + 8), 1),
    (dict(ys=A + 2), 1)])
def test_norm_refusals(kw, status):
    assert call("apmoe_norm", *norm_args(**kw)) == status
    assert apw.lib().apmoe_last_error()


def test_norm_of_no_rows():
    assert call("apmoe_norm", *norm_args(T=0)) == apw.OK


def gemm_args(**kw):
    a = dict(ctx=CTX, x8=A, xs=A, w8=A, ws=A, E=4, N=100, K=64, gather=1, perm=A, offsets=A, T=4, topk=2, out=A,
             dt=apw.F16, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(ctx=None), 1), (dict(E=0), 1), (dict(E=257), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(K=24), 1), (dict(K=1 << 24), 1),
    (dict(T=-1), 1), (dict(topk=0), 1), (dict(topk=17), 1), (dict(T=1 << 30, topk=2), 1), (dict(offsets=None), 1),
    (dict(perm=None), 1), (dict(x8=None), 1), (dict(xs=None), 1), (dict(w8=None), 1), (dict(ws=None), 1),
    (dict(out=None), 1), (dict(x8=A + 8), 1), (dict(w8=A + 4), 1), (dict(xs=A + 2), 1), (dict(ws=A + 1), 1),
    (dict(perm=A + 2), 1), (dict(offsets=A + 2), 1), (dict(out=A + 8), 1), (dict(dt=3), 2)])
def test_gemm_refusals(kw, status):
    assert call("apmoe_gemm_fp8", *gemm_args(**kw)) == status


def test_gemm_of_too_many_weight_rows():
    assert call("apmoe_gemm_fp8", *gemm_args(N=(1 << 30) + 1)) == apw.INVALID_ARG


@pytest.mark.parametrize("kw", [dict(E=256, N=1 << 30, T=8192, topk=1), dict(N=1 << 30, T=1 << 17), dict(N=1 << 20, T=1 << 29)])
def test_products_of_too_many_tiles(kw):
    assert call("apmoe_gemm_fp8", *gemm_args(**kw)) == apw.INVALID_ARG
    assert b"tiles" in apw.lib().apmoe_last_error()
    assert call("apmoe_gemm_act_fp8", *gemm_args(**dict(kw, E=256, N=(1 << 24) - 128, T=1 << 20, dt=A))) == apw.INVALID_ARG
    assert b"tiles" in apw.lib().apmoe_last_error()


@pytest.mark.parametrize("ex,kw", [
    (dict(E=256, H=16, F=(1 << 24) - 128), dict(T=1 << 18, topk=8)), (dict(E=256, H=(1 << 24) - 128, F=16), dict(T=1 << 22)),
    ({}, dict(T=1 << 24)), (dict(H=1 << 20), dict(T=1 << 15)), ({}, dict(T=1 << 28, topk=1, shared=0))])
def test_layer_size_limits_come_before_the_first_launch(ex, kw):
    """Of the workspace too: sizes that the layer refuses have none."""
    assert call("apmoe_moe_forward_fp8", *layer_args(desc(**ex), ws_bytes=(1 << 63) - 1, **kw)) == apw.INVALID_ARG
    assert b"T=" in apw.lib().apmoe_last_error()
    n = ctypes.c_size_t()
    a = dict(dict(topk=2, shared=1), **kw)
    assert call("apmoe_moe_workspace_fp8", CTX, ctypes.byref(desc(**ex)), a["T"], a["topk"], a["shared"],
                ctypes.byref(n)) == apw.INVALID_ARG


def test_gemm_of_no_rows():
    assert call("apmoe_gemm_fp8", *gemm_args(T=0)) == apw.OK


@pytest.mark.parametrize("kw,status", [
    (dict(ctx=None), 1), (dict(N=0), 1), (dict(N=24), 1), (dict(N=(1 << 30) + 16), 1), (dict(K=8), 1),
    (dict(out=None), 1), (dict(out=A + 8), 1), (dict(dt=None), 1), (dict(dt=A + 2), 1), (dict(offsets=None), 1)])
def test_gemm_act_refusals(kw, status):
    a = gemm_args(**dict(dict(N=64, dt=A), **kw))  # N is F, dt the scales
    assert call("apmoe_gemm_act_fp8", *a) == status


def desc(**kw):
    d = apw.Fp8Desc()
    for k, v in dict(dict(E=5, H=64, F=96, gate_up=A, gate_up_scale=A, down=A, down_scale=A), **kw).items():
        setattr(d, k, v)
    return d


def layer_args(experts=None, **kw):
    a = dict(ctx=CTX, ex=ctypes.byref(experts or desc()), x=A, x8=A, xs=A, wr=A, bias=None, T=3, topk=2, shared=1, renorm=1,
             ws=A, ws_bytes=1 << 30, out=A, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("ex,kw", [
    ({}, dict(ctx=None)), ({}, dict(ex=None)), (dict(E=0), {}), (dict(E=257), {}), (dict(H=24), {}), (dict(F=8), {}),
    (dict(F=100), {}), (dict(gate_up=None), {}), (dict(gate_up_scale=None), {}), (dict(down=None), {}),
    (dict(down_scale=None), {}), (dict(gate_up=A + 4), {}), (dict(down=A + 4), {}), (dict(down_scale=A + 2), {}),
    ({}, dict(T=-1)), ({}, dict(topk=0)), ({}, dict(topk=5)), ({}, dict(topk=9)), ({}, dict(shared=-1)),
    ({}, dict(shared=5)), (dict(E=20), dict(shared=9)), ({}, dict(T=1 << 29)), ({}, dict(x=None)), ({}, dict(x8=None)),
    ({}, dict(xs=None)), ({}, dict(wr=None)), ({}, dict(out=None)), ({}, dict(x=A + 8)), ({}, dict(x8=A + 8)),
    ({}, dict(xs=A + 2)), ({}, dict(wr=A + 8)), ({}, dict(bias=A + 2)), ({}, dict(out=A + 2)), ({}, dict(ws=None)),
    ({}, dict(ws=A + 16)), ({}, dict(ws_bytes=100))])
def test_layer_refusals(ex, kw):
    assert call("apmoe_moe_forward_fp8", *layer_args(desc(**ex), **kw)) == apw.INVALID_ARG


def test_layer_workspace():
    n = ctypes.c_size_t()
    ex = desc()
    sizes = []
    for T in (0, 1, 4, 64, 4096):
        assert call("apmoe_moe_workspace_fp8", CTX, ctypes.byref(ex), T, 2, 1, ctypes.byref(n)) == apw.OK
        sizes.append(n.value)
    assert sizes == sorted(sizes) and all(s % 256 == 0 for s in sizes)
    assert sizes[-1] >= 4096 * 3 * (96 + 4 + 64 * 4)
    for bad in (dict(T=-1), dict(topk=0), dict(topk=5), dict(shared=5)):
        a = dict(dict(T=1, topk=2, shared=1), **bad)
        assert call("apmoe_moe_workspace_fp8", CTX, ctypes.byref(ex), a["T"], a["topk"], a["shared"],
                    ctypes.byref(n)) == apw.INVALID_ARG
    assert call("apmoe_moe_workspace_fp8", CTX, None, 1, 2, 1, ctypes.byref(n)) == apw.INVALID_ARG
    assert call("apmoe_moe_workspace_fp8", CTX, ctypes.byref(ex), 1, 2, 1, None) == apw.INVALID_ARG
    assert call("apmoe_moe_forward_fp8", *layer_args(T=0)) == apw.OK


def test_layer_workspace_of_a_batch_serves_smaller_ones():
    n = ctypes.c_size_t()
    for ex in (desc(), desc(H=96, F=64), desc(E=256, H=16, F=1024)):
        sizes = []
        for T in range(40):
            assert call("apmoe_moe_workspace_fp8", CTX, ctypes.byref(ex), T, 2, 1, ctypes.byref(n)) == apw.OK
            sizes.append(n.value)
        assert sizes == sorted(sizes)


class HostCtx:
    """Stands for a context whose device is the host, to reach the binding's checks."""
    device, handle = -1, CTX

    def __init__(self):
        self.L = apw.lib()


def test_binding_refuses_wrong_tensors():
    c = HostCtx()
    x = torch.zeros((4, 64), dtype=torch.float16)
    gamma, y = torch.ones(64, dtype=torch.float16), torch.empty((4, 64), dtype=torch.float16)
    good = dict(x=x, residual=None, residual_out=None, gamma=gamma, y=y)
    for bad in (dict(x=x.to(torch.float64)), dict(x=x.to(torch.int16)), dict(gamma=gamma.float()), dict(gamma=gamma[:32]),
                dict(y=y.float()), dict(y=y.T), dict(x=torch.zeros((64, 4), dtype=torch.float16).T), dict(y=y[:2]),
                dict(residual=x, residual_out=x.float()), dict(y8=torch.empty((4, 64), dtype=torch.int8))):
        a = dict(dict(good), **bad)
        with pytest.raises(ValueError):
            apw.norm(c, a["x"], a["residual"], a["residual_out"], a["gamma"], 1e-5, 4, 64, a["y"], a.get("y8"),
                     torch.empty((4, 1)), stream=_NoStream())
    other = HostCtx()
    other.device = 0
    with pytest.raises(ValueError, match="context on cuda:0"):
        apw.norm(other, x, None, None, gamma, 1e-5, 4, 64, y, stream=_NoStream())


def test_binding_refuses_what_has_no_type_or_size():
    """Arguments whose type or size is the tensor's own must be tensors; sizes that wrap
    around in 32 bits are refused."""
    c, s = HostCtx(), _NoStream()
    x, gamma = torch.zeros((4, 64), dtype=torch.float16), torch.ones(64, dtype=torch.float16)
    y = torch.empty_like(x)
    for bad in (A, None, [1.0], np.zeros((4, 64), np.float16)):
        with pytest.raises(ValueError, match="x: need a tensor"):
            apw.norm(c, bad, None, None, gamma, 1e-5, 4, 64, y, stream=s)
        with pytest.raises(ValueError, match="out: need a tensor"):
            apw.gemm_fp8(c, A, A, A, A, 1, 64, 64, False, None, None, 4, 1, bad, stream=s)
    with pytest.raises(ValueError, match="residual: need a tensor"):
        apw.norm(c, x, A, A, gamma, 1e-5, 4, 64, y, stream=s)
    for T in (-1, 4 - 2 ** 32):
        with pytest.raises(ValueError, match="x: need"):
            apw.norm(c, x, None, None, gamma, 1e-5, T, 64, y, stream=s)
    gu, dn = torch.zeros((2, 64, 64), dtype=torch.uint8), torch.zeros((2, 64, 32), dtype=torch.uint8)
    ex = apw.Fp8Experts(gu, torch.ones((2, 2, 1, 1)), dn, torch.ones((2, 1, 1)))
    x8, xs, wr = torch.zeros((4, 64), dtype=torch.uint8), torch.ones((4, 1)), torch.zeros((2, 64), dtype=torch.float16)
    ws = torch.empty(1 << 16, dtype=torch.uint8)
    for bad in (A, None):
        with pytest.raises(ValueError, match="ws: need a byte tensor"):
            apw.moe_forward_fp8(c, ex, x, x8, xs, wr, None, 4, 1, True, bad, y, stream=s)
    with pytest.raises(ValueError, match="w_router: need"):
        apw.moe_forward_fp8(c, ex, x, x8, xs, wr, None, 4, 1, True, ws, y, stream=s, n_shared=2 ** 32)


def test_binding_with_no_rows():
    """Empty batches, whose tensors have no address, are calls that do nothing."""
    c, s = HostCtx(), _NoStream()
    e = lambda dt, *shape: torch.empty(shape, dtype=dt)
    f16, u8, f32, i32 = torch.float16, torch.uint8, torch.float32, torch.int32
    x, gamma = e(f16, 0, 64), torch.ones(64, dtype=f16)
    apw.norm(c, x, None, None, gamma, 1e-5, 0, 64, e(f16, 0, 64), stream=s)
    apw.norm(c, x, e(f32, 0, 64), e(f32, 0, 64), gamma, 1e-5, 0, 64, None, e(u8, 0, 64), e(f32, 0, 1), stream=s)
    x8, xs, perm, off = e(u8, 0, 64), e(f32, 0, 1), e(i32, 0), torch.zeros(3, dtype=i32)
    gu, dn = torch.zeros((2, 64, 64), dtype=u8), torch.zeros((2, 64, 32), dtype=u8)
    s1, s2 = torch.ones((2, 2, 1, 1)), torch.ones((2, 1, 1))
    apw.gemm_fp8(c, x8, xs, gu, s1, 2, 64, 64, True, perm, off, 0, 1, e(f16, 0, 64), stream=s)
    apw.gemm_act_fp8(c, x8, xs, gu, s1, 2, 32, 64, True, perm, off, 0, 1, e(u8, 0, 32), e(f32, 0, 1), stream=s)
    ex = apw.Fp8Experts(gu, s1, dn, s2)
    ws = e(u8, apw.moe_workspace_fp8(c, ex, 0, 1))
    apw.moe_forward_fp8(c, ex, x, x8, xs, torch.zeros((2, 64), dtype=f16), None, 0, 1, True, ws, e(f16, 0, 64), stream=s)


class _NoStream:
    cuda_stream = 0


def test_binding_experts():
    E, H, F = 2, 64, 32
    gu, dn = torch.zeros((E, 2 * F, H), dtype=torch.uint8), torch.zeros((E, H, F), dtype=torch.uint8)
    s1, s2 = torch.ones((E, 2, 1, 1)), torch.ones((E, 1, 1))
    ex = apw.Fp8Experts(gu, s1, dn, s2)
    assert (ex.E, ex.H, ex.F) == (E, H, F)
    for bad in ((gu[:, :F], s1, dn, s2), (gu.float(), s1, dn, s2), (gu, s1.double(), dn, s2), (gu, s1[:1], dn, s2),
                (gu, s1, dn, s2[:1]), (gu, s1, dn.transpose(1, 2).contiguous().transpose(1, 2), s2)):
        with pytest.raises(ValueError):
            apw.Fp8Experts(*bad)


# ------------------------------------------------------------------ the reference's own pins

def test_e4m3_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.TABLE, t)


def test_e4m3_round_and_encode():
    fine = ref.TABLE[~np.isnan(ref.TABLE)]
    np.testing.assert_array_equal(ref.e4m3_round(fine), fine)
    np.testing.assert_array_equal(ref.TABLE[ref.encode(fine)], fine)
    v = np.random.default_rng(0).normal(size=4000) * 60
    t = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.e4m3_round(v.astype(np.float32)), t)
    for a, b in zip(ref.TABLE[:126], ref.TABLE[1:127]):  # a tie goes to the even code
        even = a if (int(ref.encode(np.array([a]))[0]) & 1) == 0 else b
        assert ref.e4m3_round(np.array([(a + b) / 2]))[0] == even


def test_quant_of_zeros_and_short_groups():
    q, s = ref.quant(np.zeros((2, 130)))
    assert (q == 0).all() and (s == 2.0 ** -126).all() and s.shape == (2, 2)
    v = np.zeros((1, 130))
    v[0, 129] = -3.5
    q, s = ref.quant(v)
    assert q[0, 129] == -448.0 and s[0, 1] == np.float32(3.5 / 448.0)


# ------------------------------------------------------------------ the tile product's cases

def tile_cases():
    for loads, N, _ in tiles.GEMMS:
        yield loads, N, False, True
        yield loads, N, False, False
    for loads, F, _ in tiles.ACTS:
        yield loads, 2 * F, True, True


def test_tile_cases_cover_every_row_once():
    for loads, N, act, exact in tile_cases():
        off = tiles.offsets_of(loads)
        seen = np.zeros((off[-1], tiles.weight_tiles(N, act)), int)
        for e, r0, rows, nt, _, _ in tiles.forms(off, N, act, exact):
            assert off[e] <= r0 and r0 + rows <= off[e + 1]
            seen[r0:r0 + rows, nt] += 1
        assert (seen == 1).all()


def test_tile_cases_reach_every_form():
    """Every width of each kernel in whole tiles, of a whole round and of a last one, and
    in its parts, with more column blocks than the pipeline has buffers (three at most)."""
    reached = {}
    for loads, N, act, exact in tile_cases():
        off = tiles.offsets_of(loads)
        assert tiles.takes_tiles(len(loads), N, off[-1], 1, act)
        for _, _, rows, _, parts, whole in tiles.forms(off, N, act, exact):
            reached.setdefault((act, exact), set()).add((tiles.width(rows, exact), parts, whole))
    assert {(256, 1, True), (256, 1, False), (128, 1, False), (128, 2, False), (64, 1, True), (64, 1, False),
            (64, 4, False), (64, 2, False)} <= reached[False, False]
    for kernel in ((False, True), (True, True)):
        assert {(128, 1, True), (128, 1, False), (64, 1, True), (64, 1, False), (64, 2, False)} <= reached[kernel]
    assert all(K > 3 * 128 and K % 128 for _, _, K in tiles.GEMMS + tiles.ACTS)
