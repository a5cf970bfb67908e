"""The 8-bit path on the GPU, through the C ABI, against plain implementations in 64
bits (fp8_ref): the norm with the residual's addition and the 8-bit output, the e4m3
product and the gate_up product with the activation, and the whole layer.

Bounds.  The product of one block of 128 columns is an fp32 sum of 128 exact products
(e4m3 x e4m3 has 8 significant bits), scaled with two roundings and added with one per
block: |err| <= (128 + 2 KB + 3) 2^-23 * sum |terms| with KB blocks covers any order and
a matrix unit that cuts off instead of rounding; the split over column parts adds at
most 8 more terms.  16-bit outputs add half a step of their type; where they come from
the e4m3 matrix instruction (calls of more than 32 tokens) each product may be cut off
by 2^-13 of the largest of its group of 8, at most 8 * 2^-13 = 2^-10 of the sum of the
group's magnitudes.

8-bit outputs: the scale has the relative error of the largest magnitude.  Where the
value in 64 bits lies within its error bound of a border between two e4m3 values either
neighbour is right, so a value may be off by half a step of e4m3 (2^-4 relative, 2^-10
below the smallest normal number 2^-6) plus its own error."""
import zlib

import numpy as np
import pytest
import torch

import any_precision_weight_amd as apw
import fp8_ref as ref
import fp8_tiles as tiles
from gpu_util import ctx

pytestmark = pytest.mark.gpu

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SMALLEST = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}  # half the spacing at zero


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def np64(t):
    return t.detach().cpu().double().numpy()


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def rng_of(*key):
    return np.random.default_rng([zlib.crc32(k.encode()) if isinstance(k, str) else int(k) for k in key])


def cast(x, t):
    """fp64 -> type t, as a CPU tensor."""
    return torch.from_numpy(np.asarray(x, np.float32)).to(TORCH[t])


# ------------------------------------------------------------------ norm

def run_norm(x, res, gamma, eps, want_y=True, want_q=True, inplace=False):
    T, H = x.shape
    y = torch.full_like(x, 7.0) if want_y else None
    q = torch.full((T, H), 0x55, dtype=torch.uint8, device="cuda") if want_q else None
    s = torch.full((T, ref.groups(H)), -1.0, device="cuda") if want_q else None
    h = None if res is None else (res if inplace else torch.full_like(res, 7.0))
    apw.norm(ctx(), x, res, h, gamma, eps, T, H, y, q, s)
    torch.cuda.synchronize()
    return h, y, q, s


def check_norm(x, res, gamma, eps, got):
    h, y, q, s = got
    xt = {v: k for k, v in TORCH.items()}[x.dtype]
    store = (lambda v: v) if res is None else (lambda v: torch.from_numpy(v).to(res.dtype).float().numpy())
    resn = None if res is None else res.float().cpu().numpy()
    h64, y64 = ref.norm(x.float().cpu().numpy(), resn, gamma.float().cpu().numpy(), eps, store)
    if h is not None:
        np.testing.assert_array_equal(np64(h), h64)
    if y is not None:
        err = np.abs(np64(y) - y64)
        # one rounding to fp32 and one to the type, of a value known to 2^-50
        assert np.all(err <= np.abs(y64) * (HALF_STEP[xt] + 2.0 ** -24 + 2.0 ** -48) + SMALLEST[xt])
    if q is not None:
        q64, s64 = ref.quant(y64)
        np.testing.assert_allclose(np64(s), s64, rtol=2.0 ** -23, atol=0)
        got_q, s_ = ref.TABLE[codes(q)], ref.spread(np64(s), x.shape[1])
        # the 64-bit quotient by the scale as written; a border between two values may fall
        # either way only where the quotient is within 2^-23 of it (its rounding to fp32)
        with np.errstate(invalid="ignore"):
            v = y64 / s_
        off = np.abs(got_q - v)
        half = np.maximum(np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))) * 2.0 ** -4, 2.0 ** -10)
        assert np.all(off <= half + np.abs(v) * 2.0 ** -23)


NORM_SHAPES = [(1, 8), (1, 128), (3, 136), (5, 504), (2, 520), (7, 704), (4, 1032), (3, 2048), (2, 2056), (3, 4096),
               (2, 4104), (1, 8192), (2, 8200), (1, 32768), (2, 32776), (1, 65536), (333, 264), (1025, 64),
               # above 512 rows
               (515, 8), (515, 520), (517, 1016), (513, 1032), (514, 2056), (519, 4104), (513, 8200)]


@pytest.mark.parametrize("T,H", NORM_SHAPES)
def test_norm_shapes(T, H):
    r = rng_of("norm", T, H)
    x, res = cast(r.normal(size=(T, H)), "f16").cuda(), cast(4 * r.normal(size=(T, H)), "bf16").cuda()
    gamma = cast(1 + 0.2 * r.normal(size=H), "f16").cuda()
    check_norm(x, res, gamma, 1e-5, run_norm(x, res, gamma, 1e-5))


@pytest.mark.parametrize("xt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rt", [None, "f16", "bf16", "f32"])
def test_norm_types_and_outputs(xt, rt):
    r = rng_of("types", xt, str(rt))
    T, H = 37, 712
    x = cast(r.normal(size=(T, H)), xt).cuda()
    gamma = cast(1 + 0.2 * r.normal(size=H), xt).cuda()
    for want_y, want_q, inplace in ((True, True, False), (True, False, True), (False, True, False)):
        res = None if rt is None else cast(3 * r.normal(size=(T, H)), rt).cuda()
        before = None if res is None else res.clone()
        got = run_norm(x, res, gamma, 1e-6, want_y, want_q, inplace)
        check_norm(x, before, gamma, 1e-6, got)
        if res is not None and not inplace:
            assert torch.equal(res, before)


def test_norm_in_place_y():
    r = rng_of("inplace")
    x = cast(r.normal(size=(9, 1048)), "bf16").cuda()
    gamma = cast(1 + 0.2 * r.normal(size=1048), "bf16").cuda()
    _, y, _, _ = run_norm(x, None, gamma, 1e-5, True, False)
    z = x.clone()
    apw.norm(ctx(), z, None, None, gamma, 1e-5, 9, 1048, z)
    assert torch.equal(z.view(torch.int16), y.view(torch.int16))


def test_norm_special_rows():
    """Zeros, huge and tiny rows, NaN and infinities: each row by itself."""
    H = 272
    r = rng_of("special")
    x = r.normal(size=(8, H))
    x[0] = 0.0
    x[1] *= 1e30   # squares leave fp32's range
    x[2] *= 1e-30
    x[3, 5] = np.nan
    x[4, 5] = np.inf
    x[5, :128] = 0.0  # one group of zeros
    x[6, 140] = 3e38
    xd = cast(x, "f32").cuda()
    gamma = cast(np.ones(H), "f32").cuda()
    _, y, q, s = run_norm(xd, None, gamma, 1e-5)
    fine = [0, 1, 2, 5, 6, 7]
    check_norm(xd[fine], None, gamma, 1e-5, (None, y[fine], q[fine], s[fine]))
    assert torch.isnan(y[3]).all() and torch.isnan(y[4, 5])
    values = ref.TABLE[codes(q)] * ref.spread(np64(s), H)
    assert np.isnan(values[3]).all()
    assert np.isnan(values[4, :128]).all() and (values[4, 128:] == 0).all()
    assert (codes(q[0]) & 0x7F == 0).all() and (np64(s[0]) == 2.0 ** -126).all()
    assert (codes(q[5, :128]) & 0x7F == 0).all()
    z = torch.zeros((2, H), device="cuda")  # eps = 0 and a row of zeros: 0 / 0
    _, yz, _, _ = run_norm(z, None, gamma, 0.0)
    assert torch.isnan(yz).all()


def test_norm_many_short_rows():
    """More workgroups than one dimension of the grid holds: the same bits as a call on the
    rows alone."""
    T, H = (1 << 22) + 5, 8
    x = torch.randn((T, H), device="cuda").half()
    gamma = torch.ones(H, device="cuda").half()
    _, y, q, s = run_norm(x, None, gamma, 1e-5)
    for at in (slice(0, 64), slice(1 << 21, (1 << 21) + 64), slice(T - 64, T)):
        _, y1, q1, s1 = run_norm(x[at].clone(), None, gamma, 1e-5)
        assert torch.equal(y[at], y1) and torch.equal(q[at], q1) and torch.equal(s[at], s1)
    assert float((y.float() ** 2).mean(dim=1).sub(1).abs().max()) < 0.1


# ------------------------------------------------------------------ products

def routing(r, T, topk, E, skew=0.0):
    """Distinct experts of each token, perm and offsets."""
    z = r.normal(size=(T, E)) - skew * np.log(np.arange(1, E + 1))
    ids = np.argsort(-z, axis=1)[:, :topk].reshape(-1)
    perm = np.argsort(ids, kind="stable").astype(np.int32)
    off = np.zeros(E + 1, np.int32)
    off[1:] = np.cumsum(np.bincount(ids, minlength=E))
    return perm, off


def random_weights(r, E, halves, rows, K):
    """Random codes (no NaN code) and scales."""
    c = r.integers(0, 256, size=(E, halves * rows, K), dtype=np.uint8)
    c[(c & 0x7F) == 0x7F] ^= 1
    s = np.exp2(r.uniform(-14, -8, size=(E, halves, ref.groups(rows), ref.groups(K)))).astype(np.float32)
    return c, s


def random_rows(r, R, K):
    c = r.integers(0, 256, size=(R, K), dtype=np.uint8)
    c[(c & 0x7F) == 0x7F] ^= 1
    return c, np.exp2(r.uniform(-9, -5, size=(R, ref.groups(K)))).astype(np.float32)


def sum_bound(K):
    return (128 + 2 * ref.groups(K) + 3 + 8) * 2.0 ** -23


# (T, topk, E, N, K): one row, one column block, ragged K and N, many rows, idle experts
GEMMS = [(1, 1, 1, 1, 16), (1, 1, 1, 128, 128), (1, 1, 1, 33, 144), (3, 2, 4, 129, 240), (8, 1, 1, 256, 1024),
         (16, 2, 8, 200, 528), (17, 1, 1, 64, 2048), (33, 1, 1, 130, 400), (40, 4, 6, 384, 1408), (64, 1, 1, 515, 656),
         (65, 1, 2, 256, 512), (130, 2, 3, 300, 1040), (257, 1, 1, 260, 384), (300, 3, 5, 272, 272),
         (513, 1, 1, 520, 912), (700, 2, 9, 128, 128), (1000, 1, 2, 600, 1552),
         # enough tiles for the tile product in each type
         (33, 1, 1, 8720, 144), (300, 1, 1, 8720, 112), (40, 1, 1, 8720, 16), (64, 1, 1, 8452, 656), (130, 2, 3, 4360, 528), (257, 1, 1, 4100, 272),
         (300, 3, 5, 2200, 272), (513, 1, 1, 4099, 1040), (1000, 1, 2, 2600, 912), (2100, 2, 40, 144, 256)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("T,topk,E,N,K", GEMMS)
def test_gemm(T, topk, E, N, K, gather):
    r = rng_of("gemm", T, topk, E, N, K, gather)
    perm, off = routing(r, T, topk, E, 1.0 if T > 100 else 0.0)
    R = T * topk
    x8, xs = random_rows(r, T if gather else R, K)
    w8, ws = random_weights(r, E, 1, N, K)
    xv = ref.TABLE[x8] * ref.spread(xs.astype(np.float64), K)
    wv = [ref.block_values(w8[e], ws[e, 0]) for e in range(E)]
    want, mag = ref.product(xv, wv, perm, off, topk, gather)
    dx, dxs, dw, dws, dp, do = (cuda(v) for v in (x8, xs, w8, ws, perm, off))
    for t in ("f32", "f16", "bf16"):
        out = torch.full((R + 2, N), 7.0, dtype=TORCH[t], device="cuda")
        apw.gemm_fp8(ctx(), dx, dxs, dw, dws, E, N, K, gather, dp, do, T, topk, out)
        torch.cuda.synchronize()
        got = np64(out)
        bound = mag * sum_bound(K)
        if t != "f32":
            bound = bound + mag * (2.0 ** -10 if (R if E == 1 else T) > 32 else 0.0)
        bound = bound + (np.abs(want) + bound) * HALF_STEP[t] + SMALLEST[t]
        err = np.abs(got[:R] - want)
        assert np.all(err <= bound), (t, float((err - bound).max()))
        assert (got[R:] == 7.0).all()  # rows behind the last


def test_gemm_dense_without_offsets():
    r = rng_of("dense")
    T, N, K = 45, 200, 320
    x8, xs = random_rows(r, T, K)
    w8, ws = random_weights(r, 1, 1, N, K)
    d = [cuda(v) for v in (x8, xs, w8, ws)]
    a, b = (torch.empty((T, N), device="cuda") for _ in range(2))
    apw.gemm_fp8(ctx(), *d, 1, N, K, False, None, None, T, 1, a)
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    perm = torch.arange(T, dtype=torch.int32, device="cuda")
    apw.gemm_fp8(ctx(), *d, 1, N, K, True, perm, off, T, 1, b)
    assert torch.equal(a, b)
    # the same rows as 15 tokens of 3 assignments, all of the one expert
    c = torch.empty((T, N), device="cuda")
    apw.gemm_fp8(ctx(), *d, 1, N, K, False, None, None, T // 3, 3, c)
    assert torch.equal(a, c)


@pytest.mark.parametrize("T,E,N", [(20, 3, 144), (200, 3, 144), (200, 3, 2320)])
def test_gemm_rows_behind_the_last_sequence(T, E, N):
    """offsets that end before T * topk rows: the rows behind stay as they were."""
    r = rng_of("behind", T)
    K, used = 272, T - 7
    off = np.array([0, used // 2, used // 2, used], np.int32)
    x8, xs = random_rows(r, T, K)
    w8, ws = random_weights(r, E, 1, N, K)
    perm = np.arange(T, dtype=np.int32)
    out = torch.full((T, N), 7.0, device="cuda")
    apw.gemm_fp8(ctx(), *(cuda(v) for v in (x8, xs, w8, ws)), E, N, K, False, cuda(perm), cuda(off), T, 1, out)
    want, mag = ref.product(ref.TABLE[x8] * ref.spread(xs.astype(np.float64), K),
                            [ref.block_values(w8[e], ws[e, 0]) for e in range(E)], perm, off, 1, False)
    got = np64(out)
    assert (got[used:] == 7.0).all()
    assert np.all(np.abs(got[:used] - want) <= mag * sum_bound(K))


@pytest.mark.parametrize("T,N,K", [(12, 96, 144), (12, 96, 2048), (20, 160, 2048), (30, 64, 272), (200, 2336, 272)])
def test_products_with_a_token_twice_at_an_expert(T, N, K):
    """Every token with both its assignments at one expert, which then has 2 T rows, more
    than the routing's distinct experts give."""
    r = rng_of("twice", T, N, K)
    E, topk, R = 3, 2, 2 * T
    perm, off = r.permutation(R).astype(np.int32), np.array([0, 0, R, R], np.int32)
    x8, xs = random_rows(r, T, K)
    xs = (xs / np.sqrt(K)).astype(np.float32)
    w8, ws = random_weights(r, E, 1, N, K)
    d = [cuda(v) for v in (x8, xs, w8, ws, perm, off)]
    xv = ref.TABLE[x8] * ref.spread(xs.astype(np.float64), K)
    out = torch.full((R + 1, N), 7.0, device="cuda")
    apw.gemm_fp8(ctx(), *d[:4], E, N, K, True, *d[4:], T, topk, out)
    want, mag = ref.product(xv, [ref.block_values(w8[e], ws[e, 0]) for e in range(E)], perm, off, topk, True)
    assert np.all(np.abs(np64(out)[:R] - want) <= mag * sum_bound(K)) and (np64(out)[R] == 7.0).all()
    F = N // 2
    w8, ws = random_weights(r, E, 2, F, K)
    a8 = torch.full((R + 1, F), 0x55, dtype=torch.uint8, device="cuda")
    sc = torch.empty((R + 1, ref.groups(F)), device="cuda")
    apw.gemm_act_fp8(ctx(), d[0], d[1], cuda(w8), cuda(ws), E, F, K, True, *d[4:], T, topk, a8, sc)
    wv = [np.concatenate([ref.block_values(w8[e, h * F:(h + 1) * F], ws[e, h]) for h in (0, 1)]) for e in range(E)]
    a, err = act_bounds(*ref.product(xv, wv, perm, off, topk, True), F, K)
    check_rows8(a, err, a8[:R], sc[:R], F)
    assert (codes(a8[R:]) == 0x55).all()


@pytest.mark.parametrize("T,N", [(5, 96), (70, 96), (70, 8464)])
def test_gemm_nan_stays_in_its_row_and_column(T, N):
    r = rng_of("nan", T)
    K = 400
    x8, xs = random_rows(r, T, K)
    w8, ws = random_weights(r, 1, 1, N, K)
    x8[2, 390] = 0x7F
    w8[0, 40, 3] = 0xFF
    out = torch.empty((T, N), device="cuda")
    apw.gemm_fp8(ctx(), *(cuda(v) for v in (x8, xs, w8, ws)), 1, N, K, False, None, None, T, 1, out)
    nan = np.isnan(np64(out))
    want = np.zeros((T, N), bool)
    want[2], want[:, 40] = True, True
    np.testing.assert_array_equal(nan, want)


def act_bounds(gu, mag, F, K):
    """(a in 64 bits, bound of its error): g and u known to sum_bound, SiLU(g) * u moved by
    at most (1.1 |u| + |s|) times that (the slope of SiLU is below 1.1), and 2^-20 for the
    exponential, the reciprocal and the products."""
    g, u = gu[:, :F], gu[:, F:]
    s = ref.silu(g)
    dg, du = mag[:, :F] * sum_bound(K), mag[:, F:] * sum_bound(K)
    err = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + np.abs(s * u) * 2.0 ** -20
    # e^-g overflows fp32 below about -88: SiLU is below 2^-120 there
    return s * u, err + 2.0 ** -100 * np.abs(u)


def check_rows8(a, err, q, s, C):
    """8-bit rows against 64-bit values with error bounds."""
    got_s = np64(s)
    G = ref.groups(C)
    for g in range(G):
        c = slice(g * ref.BLK, min(C, (g + 1) * ref.BLK))
        amax, e = np.abs(a[:, c]).max(axis=1), err[:, c].max(axis=1)
        want = np.maximum(amax / 448.0, ref.TINY)
        assert np.all(np.abs(got_s[:, g] - want) <= e / 448.0 + want * 2.0 ** -22)
    sv = ref.spread(got_s, C)
    v, got = a / sv, ref.TABLE[codes(q)]
    half = np.maximum(np.exp2(np.floor(np.log2(np.maximum(np.abs(v) + err / sv, 2.0 ** -6)))) * 2.0 ** -4, 2.0 ** -10)
    assert np.all(np.abs(got - v) <= half + err / sv + np.abs(v) * 2.0 ** -22)


ACTS = [(1, 1, 1, 16, 16), (1, 1, 1, 128, 128), (3, 2, 4, 144, 240), (16, 2, 8, 272, 528), (33, 1, 1, 704, 256),
        (40, 4, 6, 384, 400), (130, 2, 3, 208, 1040), (300, 1, 2, 400, 272), (600, 2, 5, 256, 512),
        (50, 1, 1, 32, 16), (300, 1, 1, 144, 112)]


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("T,topk,E,F,K", ACTS)
def test_gemm_act(T, topk, E, F, K, gather):
    r = rng_of("act", T, topk, E, F, K, gather)
    perm, off = routing(r, T, topk, E, 1.0 if T > 100 else 0.0)
    R = T * topk
    x8, xs = random_rows(r, T if gather else R, K)
    w8, ws = random_weights(r, E, 2, F, K)
    xs = (xs / np.sqrt(K)).astype(np.float32)
    xv = ref.TABLE[x8] * ref.spread(xs.astype(np.float64), K)
    wv = [np.concatenate([ref.block_values(w8[e, h * F:(h + 1) * F], ws[e, h]) for h in (0, 1)]) for e in range(E)]
    gu, mag = ref.product(xv, wv, perm, off, topk, gather)
    a8 = torch.full((R + 1, F), 0x55, dtype=torch.uint8, device="cuda")
    sc = torch.full((R + 1, ref.groups(F)), -1.0, device="cuda")
    apw.gemm_act_fp8(ctx(), *(cuda(v) for v in (x8, xs, w8, ws)), E, F, K, gather, cuda(perm), cuda(off), T, topk, a8,
                     sc)
    torch.cuda.synchronize()
    a, err = act_bounds(gu, mag, F, K)
    check_rows8(a, err, a8[:R], sc[:R], F)
    assert (codes(a8[R:]) == 0x55).all() and (np64(sc[R:]) == -1.0).all()


def test_gemm_act_zero_and_nan_groups():
    """A token of zeros gives groups of zeros with the smallest scale; a NaN in a token
    gives NaN for that token alone."""
    r = rng_of("act-special")
    T, F, K = 6, 144, 256
    x8, xs = random_rows(r, T, K)
    w8, ws = random_weights(r, 1, 2, F, K)
    x8[1] = 0
    x8[4, 7] = 0x7F
    a8 = torch.empty((T, F), dtype=torch.uint8, device="cuda")
    sc = torch.empty((T, 2), device="cuda")
    apw.gemm_act_fp8(ctx(), *(cuda(v) for v in (x8, xs, w8, ws)), 1, F, K, False, None, None, T, 1, a8, sc)
    v = ref.TABLE[codes(a8)] * ref.spread(np64(sc), F)
    assert (v[1] == 0).all() and (np64(sc)[1] == 2.0 ** -126).all()
    assert np.isnan(v[4]).all()
    assert np.isfinite(np.delete(v, 4, axis=0)).all()


# ------------------------------------------------------------------ layer

def layer_inputs(r, E, n_shared, H, F, T):
    Et = E + n_shared
    w1, s1 = random_weights(r, Et, 2, F, H)
    w2, s2 = random_weights(r, Et, 1, H, F)
    s1 /= np.float32(np.sqrt(H))
    s2 /= np.float32(np.sqrt(F))
    x = (r.normal(size=(T, H))).astype(np.float16)
    wr = (r.normal(size=(E, H)) * 0.05).astype(np.float16)
    q, s = ref.quant(x.astype(np.float64))
    return dict(w1=w1, s1=s1, w2=w2, s2=s2, x=x, wr=wr, x8=ref.encode(q), xs=s.astype(np.float32))


def layer_ref(d, bias, E, n_shared, H, F, T, topk, renorm):
    """(out, bound).  With more than 32 tokens an expert's down product may come from the
    e4m3 instruction: 2^-10 of the magnitudes (see above)."""
    cut = 2.0 ** -10 if T > 32 else 0.0
    z = d["x"].astype(np.float64) @ d["wr"].astype(np.float64).T + (0 if bias is None else bias.astype(np.float64))
    xv = ref.TABLE[d["x8"]] * ref.spread(d["xs"].astype(np.float64), H)
    out, bound = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        ids = np.argsort(-z[t], kind="stable")[:topk]
        p = np.exp(z[t] - z[t].max())
        w = p[ids] / (p[ids] if renorm else p).sum()
        for e, we in list(zip(ids, w)) + [(E + i, 1.0) for i in range(n_shared)]:
            w1 = np.concatenate([ref.block_values(d["w1"][e, h * F:(h + 1) * F], d["s1"][e, h]) for h in (0, 1)])
            w2 = ref.block_values(d["w2"][e], d["s2"][e, 0])
            gu, mag = xv[t] @ w1.T, np.abs(xv[t]) @ np.abs(w1).T
            a, err = act_bounds(gu[None], mag[None], F, H)
            q, s = ref.quant(a)
            sv = ref.spread(s, F)
            v = a / sv
            # a value near a border of e4m3 may fall either way: a whole step (twice the half) there
            step = 2 * np.maximum(np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))) * 2.0 ** -4, 2.0 ** -10)
            frac = np.abs(v - q)  # distance to the chosen value; a border is half a step away
            flips = frac >= step / 2 - err / sv - np.abs(v) * 2.0 ** -21
            slack = np.where(flips, step, 0.0) * sv + np.abs(q * sv) * 2.0 ** -21 + np.repeat(
                np.array([err[0, g * 128:(g + 1) * 128].max() for g in range(ref.groups(F))]), 128)[None, :F]
            y, ymag = (q * sv) @ w2.T, np.abs(q * sv) @ np.abs(w2).T
            out[t] += we * y[0]
            bound[t] += we * (ymag[0] * (sum_bound(F) + 2.0 ** -22 + cut) + (slack @ np.abs(w2).T)[0])
    return out, bound + (np.abs(out) + bound) * 2.0 ** -11 + 2.0 ** -25


LAYERS = [  # T, E, topk, shared, H, F, renorm, bias
    (1, 4, 2, 0, 256, 512, True, False), (1, 1, 1, 0, 16, 16, True, False), (1, 12, 4, 2, 272, 144, False, True),
    (2, 8, 2, 1, 528, 400, True, True), (3, 60, 8, 4, 256, 208, False, False), (4, 5, 5, 0, 400, 272, True, True),
    (7, 3, 2, 8, 144, 704, False, False), (16, 8, 2, 0, 384, 256, True, False), (17, 8, 2, 1, 384, 256, True, False),
    (33, 6, 3, 0, 272, 272, False, True), (100, 4, 2, 1, 256, 384, True, True), (16, 200, 8, 1, 128, 64, True, False),
    (1, 256, 8, 0, 64, 48, False, True), (4, 248, 8, 8, 80, 16, True, True),
    (16, 8, 8, 8, 64, 272, True, False), (1, 8, 2, 0, 2048, 4096, True, False), (3, 6, 2, 0, 1040, 2064, False, True),
    (100, 4, 2, 1, 1040, 272, True, False),
    # more than 150 rows of an expert: their fp32 rows do not fit LDS at once
    (400, 2, 1, 0, 1552, 272, True, False), (700, 3, 2, 0, 2064, 144, False, True)]


def run_layer(d, bias, E, n_shared, H, F, T, topk, renorm, stream=None):
    ex = apw.Fp8Experts(cuda(d["w1"]), cuda(d["s1"]), cuda(d["w2"]), cuda(d["s2"]))
    n = apw.moe_workspace_fp8(ctx(), ex, T, topk, n_shared=n_shared)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")  # nothing is read before it is written
    out = torch.full((T + 1, H), 7.0, dtype=torch.float16, device="cuda")
    args = [cuda(d["x"]), cuda(d["x8"]), cuda(d["xs"]), cuda(d["wr"]), None if bias is None else cuda(bias)]
    apw.moe_forward_fp8(ctx(), ex, *args, T, topk, renorm, ws, out, n_shared=n_shared)
    torch.cuda.synchronize()
    assert (np64(out[T:]) == 7.0).all()
    return np64(out[:T]), (ex, args, ws, out)


@pytest.mark.parametrize("T,E,topk,shared,H,F,renorm,has_bias", LAYERS)
def test_layer(T, E, topk, shared, H, F, renorm, has_bias):
    r = rng_of("layer", T, E, topk, shared, H, F)
    d = layer_inputs(r, E, shared, H, F, T)
    bias = (r.normal(size=E) * 0.5).astype(np.float32) if has_bias else None
    want, bound = layer_ref(d, bias, E, shared, H, F, T, topk, renorm)
    got, _ = run_layer(d, bias, E, shared, H, F, T, topk, renorm)
    err = np.abs(got - want)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("T,E,topk,H,F", [(5, 256, 8, 128, 272), (6, 256, 1, 64, 48), (15, 160, 2, 80, 144)])
def test_layer_long_selections(T, E, topk, H, F):
    """Near the most comparisons that the few-token launches take (T * E^2 of 384000)."""
    r = rng_of("long", T, E)
    d = layer_inputs(r, E, 0, H, F, T)
    want, bound = layer_ref(d, None, E, 0, H, F, T, topk, True)
    got, _ = run_layer(d, None, E, 0, H, F, T, topk, True)
    assert np.all(np.abs(got - want) <= bound)


@pytest.mark.parametrize("T", [5, 300])
def test_route_with_a_nan_token(T):
    """A token whose logits are all NaN still gets distinct experts (the lowest ones), so
    that perm and inv_perm are permutations; its weights are NaN, the others' are not."""
    r = rng_of("route-nan", T)
    H, E, topk = 64, 6, 2
    x = r.normal(size=(T, H)).astype(np.float16)
    x[T // 2, 5] = np.nan
    wr = r.normal(size=(E, H)).astype(np.float16)
    ids, perm, inv = (torch.full((T * topk,), -1, dtype=torch.int32, device="cuda") for _ in range(3))
    w = torch.empty((T, topk), device="cuda")
    counts, offsets = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E, E + 1))
    apw.route(ctx(), cuda(x), cuda(wr), None, T, H, E, topk, True, ids, w, counts, offsets, perm, inv)
    torch.cuda.synchronize()
    ids, w = ids.view(T, topk).cpu().numpy(), w.cpu().numpy()
    assert ids[T // 2].tolist() == [0, 1]
    assert np.isnan(w[T // 2]).all() and np.isfinite(np.delete(w, T // 2, axis=0)).all()
    for p in (perm, inv):
        assert np.array_equal(np.sort(p.cpu().numpy()), np.arange(T * topk))
    assert int(offsets[-1]) == T * topk


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T", [2, 24, 300])
def test_route_nan_logits(T, renorm):
    """NaN logits of some experts: they are chosen last, the lowest index first, and the
    softmax takes them as they are: a chosen one makes the weights NaN, one that is not
    chosen only the full softmax's."""
    r = rng_of("route-nan-logits", T)
    H, E, topk = 64, 6, 3
    x, wr = r.normal(size=(T, H)).astype(np.float16), r.normal(size=(E, H)).astype(np.float16)
    z = x.astype(np.float64) @ wr.astype(np.float64).T
    for nan in ([4], [1, 2, 4, 5]):
        bias = np.zeros(E, np.float32)
        bias[nan] = np.nan
        ids, perm, inv = (torch.full((T * topk,), -1, dtype=torch.int32, device="cuda") for _ in range(3))
        w = torch.empty((T, topk), device="cuda")
        counts, offsets = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E, E + 1))
        apw.route(ctx(), cuda(x), cuda(wr), cuda(bias), T, H, E, topk, renorm, ids, w, counts, offsets, perm, inv)
        torch.cuda.synchronize()
        ids, w = ids.view(T, topk).cpu().numpy(), w.cpu().numpy()
        zn = z.copy()
        zn[:, nan] = -np.inf
        want = np.argsort(-zn, axis=1, kind="stable")[:, :topk]
        np.testing.assert_array_equal(ids, want)
        if renorm and nan == [4]:
            p = np.exp(np.take_along_axis(z, want, 1) - z[:, [0, 1, 2, 3, 5]].max(axis=1, keepdims=True))
            # fp64 sums of 64 terms and one rounding to fp32
            np.testing.assert_allclose(w, p / p.sum(axis=1, keepdims=True), rtol=2.0 ** -23)
        else:
            assert np.isnan(w).all()


@pytest.mark.parametrize("T", [2, 24, 300])
def test_layer_nan_logits(T):
    """The same rule in the layer, below and above 16 tokens: an expert whose logit is NaN
    and that is not chosen is as one at -infinity; a chosen one makes the output NaN; one
    at -infinity that is chosen has weight 0."""
    r = rng_of("layer-nan-logits", T)
    E, topk, H, F = 6, 3, 272, 144
    d = layer_inputs(r, E, 0, H, F, T)
    low = np.zeros(E, np.float32)
    low[[4]] = -np.inf
    want, bound = layer_ref(d, low, E, 0, H, F, T, topk, True)
    got, _ = run_layer(d, low, E, 0, H, F, T, topk, True)
    assert np.all(np.abs(got - want) <= bound)
    nan = low.copy()
    nan[4] = np.nan
    again, _ = run_layer(d, nan, E, 0, H, F, T, topk, True)
    np.testing.assert_array_equal(again, got)
    assert np.isnan(run_layer(d, nan, E, 0, H, F, T, topk, False)[0]).all()
    low[[1, 2, 5]] = -np.inf
    want, bound = layer_ref(d, low, E, 0, H, F, T, topk, True)
    got, _ = run_layer(d, low, E, 0, H, F, T, topk, True)
    assert np.all(np.abs(got - want) <= bound)
    nan = low.copy()
    nan[1] = np.nan  # the third choice of every token
    assert np.isnan(run_layer(d, nan, E, 0, H, F, T, topk, True)[0]).all()


@pytest.mark.parametrize("T", [1, 3, 20])
def test_layer_with_a_nan_token(T):
    """A NaN in one token leaves the other tokens' outputs as they are."""
    r = rng_of("nan-token", T)
    E, topk, shared, H, F = 6, 2, 1, 272, 144
    d = layer_inputs(r, E, shared, H, F, T + 1)
    d["x"][T, 3] = np.nan
    d["x8"][T, 3] = 0x7F
    got, _ = run_layer(d, None, E, shared, H, F, T + 1, topk, True)
    assert np.isnan(got[T]).all()
    for k in ("x", "x8", "xs"):
        d[k] = d[k][:T]
    want, bound = layer_ref(d, None, E, shared, H, F, T, topk, True)
    assert np.all(np.abs(got[:T] - want) <= bound)


@pytest.mark.parametrize("part", ["gate_up", "down", "down_scale"])
@pytest.mark.parametrize("T,H,F", [(3, 272, 144), (16, 272, 144), (3, 1040, 8208), (24, 272, 144)])
def test_layer_nan_weights_stay_with_their_expert(T, H, F, part):
    """A NaN in an expert's weights is for the tokens that chose it alone: the others' bits
    are those of the call without it.  With 8208 values of F the activation is quantised by
    gate_up, with 144 by down."""
    r = rng_of("nan-expert", T, H, F, part)
    E, topk = 6, 2
    d = layer_inputs(r, E, 0, H, F, T)
    z = d["x"].astype(np.float64) @ d["wr"].astype(np.float64).T
    chosen = np.argsort(-z, axis=1, kind="stable")[:, :topk]
    e = next(e for e in range(E) if 0 < (chosen == e).any(axis=1).sum() < T)
    mine = (chosen == e).any(axis=1)
    before, _ = run_layer(d, None, E, 0, H, F, T, topk, True)
    cols = np.zeros(H, bool)
    if part == "gate_up":  # one value of the activation, and so its group: every output
        d["w1"][e, 5, 7] = 0x7F
        cols[:] = True
    elif part == "down":
        d["w2"][e, 40, F - 3] = 0xFF
        cols[40] = True
    else:
        d["s2"][e, 0, 0, -1] = np.nan
        cols[:128] = True
    got, _ = run_layer(d, None, E, 0, H, F, T, topk, True)
    want = before.copy()
    want[np.ix_(mine, cols)] = np.nan
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("T", [1, 4, 16, 20])
def test_layer_ties_go_to_the_lower_expert(T):
    """Identical router rows: every token takes experts 0 .. topk-1."""
    r = rng_of("ties", T)
    E, topk, H, F = 6, 2, 128, 64
    d = layer_inputs(r, E, 0, H, F, T)
    d["wr"][:] = d["wr"][0]
    want, bound = layer_ref(d, None, E, 0, H, F, T, topk, True)
    got, _ = run_layer(d, None, E, 0, H, F, T, topk, True)
    assert np.all(np.abs(got - want) <= bound)


@pytest.mark.parametrize("T", [1, 5, 40])
def test_layer_graph_replays(T):
    """Captured once, replayed with new rows, with work of the program's own between."""
    r = rng_of("graph", T)
    E, topk, shared, H, F = 8, 2, 1, 256, 384
    d = layer_inputs(r, E, shared, H, F, T)
    _, (ex, args, ws, out) = run_layer(d, None, E, shared, H, F, T, topk, True)
    other = [layer_inputs(rng_of("graph", T, i), E, shared, H, F, T) for i in range(3)]

    def call(stream=None):
        apw.moe_forward_fp8(ctx(), ex, *args, T, topk, True, ws, out, stream=stream, n_shared=shared)

    def put(o):
        for i, k in enumerate(("x", "x8", "xs")):
            args[i].copy_(cuda(o[k]))

    refs = []
    for o in other:
        put(o)
        call()
        torch.cuda.synchronize()
        refs.append(out[:T].clone())
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(s)
    noise = torch.randn(64, 64, device="cuda")
    for rep in range(6):
        put(other[rep % 3])
        out.fill_(float("nan"))
        noise = torch.tanh(noise @ noise)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:T], refs[rep % 3]), rep


def test_layer_on_two_streams_with_a_workspace_and_context_each():
    r = rng_of("streams")
    E, topk, H, F, T = 8, 2, 256, 384, 3
    d = layer_inputs(r, E, 0, H, F, T)
    want, (ex, args, ws, _) = run_layer(d, None, E, 0, H, F, T, topk, True)
    ctxs = [ctx(), apw.Context(0)]
    st = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty((T, H), dtype=torch.float16, device="cuda") for _ in range(2)]
    spaces = [torch.empty_like(ws) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            apw.moe_forward_fp8(ctxs[i], ex, *args, T, topk, True, spaces[i], outs[i], stream=st[i])
    torch.cuda.synchronize()
    for o in outs:
        np.testing.assert_array_equal(np64(o), want)
    ctxs[1].close()


@pytest.mark.parametrize("T,E,topk,H,F", [(8, 256, 4, 64, 64), (16, 8, 8, 64, 13056), (3, 8, 2, 256, 384)])
def test_few_token_layers_at_once_on_one_context(T, E, topk, H, F):
    """Up to 16 tokens two calls, or two captured graphs, may run at the same time on one
    context with a workspace each; with 256 experts, or with scales of the activation that
    LDS does not hold, they route in launches of their own."""
    r = rng_of("one-context", T, E, F)
    d = layer_inputs(r, E, 0, H, F, T)
    ex = apw.Fp8Experts(cuda(d["w1"]), cuda(d["s1"]), cuda(d["w2"]), cuda(d["s2"]))
    n = apw.moe_workspace_fp8(ctx(), ex, T, topk)
    streams, calls, outs, wants = [torch.cuda.Stream() for _ in range(2)], [], [], []
    for i in range(2):
        o = layer_inputs(rng_of("one-context", T, E, F, i), 1, 0, H, 16, T)
        args = [cuda(o["x"]), cuda(o["x8"]), cuda(o["xs"]), cuda(d["wr"]), None]
        ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
        out = torch.empty((T, H), dtype=torch.float16, device="cuda")

        def call(args=args, ws=ws, out=out, s=streams[i]):
            apw.moe_forward_fp8(ctx(), ex, *args, T, topk, True, ws, out, stream=s)
        call()
        torch.cuda.synchronize()
        calls.append(call)
        outs.append(out)
        wants.append(out.clone())
    assert not torch.equal(wants[0], wants[1])
    for _ in range(30):
        calls[0]()
        calls[1]()
    torch.cuda.synchronize()
    for o, w in zip(outs, wants):
        assert torch.equal(o, w)
        o.fill_(float("nan"))
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            calls[i]()
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, wants):
            assert torch.equal(o, w)


@pytest.mark.parametrize("T", [1, 4, 16, 24])
def test_layer_of_an_unfused_context_is_its_steps(T, monkeypatch):
    """A context made under APMOE_UNFUSED=1 runs every step in its own launches, a few
    tokens too: the bits of the route, the two products (to fp32) and the combine."""
    monkeypatch.setenv("APMOE_UNFUSED", "1")
    c = apw.Context(0)
    r = rng_of("unfused", T)
    E, topk, shared, H, F = 8, 2, 1, 272, 400
    Et, kt, R = E + shared, topk + shared, T * (topk + shared)
    d = layer_inputs(r, E, shared, H, F, T)
    w1, s1, w2, s2, x, x8, xs, wr = (cuda(d[k]) for k in ("w1", "s1", "w2", "s2", "x", "x8", "xs", "wr"))
    ex = apw.Fp8Experts(w1, s1, w2, s2)
    ws = torch.empty(apw.moe_workspace_fp8(c, ex, T, topk, n_shared=shared), dtype=torch.uint8, device="cuda")
    out, want = (torch.empty((T, H), dtype=torch.float16, device="cuda") for _ in range(2))
    apw.moe_forward_fp8(c, ex, x, x8, xs, wr, None, T, topk, True, ws, out, n_shared=shared)
    ids, perm, inv = (torch.empty(R, dtype=torch.int32, device="cuda") for _ in range(3))
    w, y = torch.empty((T, kt), device="cuda"), torch.empty((R, H), device="cuda")
    counts, off = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (Et, Et + 1))
    a8, sc = torch.empty((R, F), dtype=torch.uint8, device="cuda"), torch.empty((R, ref.groups(F)), device="cuda")
    apw.route(c, x, wr, None, T, H, E, topk, True, ids, w, counts, off, perm, inv, n_shared=shared)
    apw.gemm_act_fp8(c, x8, xs, w1, s1, Et, F, H, True, perm, off, T, kt, a8, sc)
    apw.gemm_fp8(c, a8, sc, w2, s2, Et, H, F, False, perm, off, T, kt, y)
    apw.combine(c, y, apw.F32, w, inv, T, kt, H, want)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    c.close()


def test_norm_then_layer_then_norm():
    """The calls as a decode step makes them: norm with the residual -> layer on its two
    outputs -> the next norm adds the layer's output to the residual."""
    r = rng_of("chain")
    E, topk, H, F = 8, 2, 256, 384
    for T in (1, 4, 24):
        d = layer_inputs(r, E, 0, H, F, T)
        attn = cast(r.normal(size=(T, H)), "f16").cuda()
        res = cast(3 * r.normal(size=(T, H)), "f32").cuda()
        res0 = res.clone()
        gamma = cast(1 + 0.1 * r.normal(size=H), "f16").cuda()
        x = torch.empty((T, H), dtype=torch.float16, device="cuda")
        x8 = torch.empty((T, H), dtype=torch.float8_e4m3fn, device="cuda")
        xs = torch.empty((T, ref.groups(H)), device="cuda")
        apw.norm(ctx(), attn, res, res, gamma, 1e-5, T, H, x, x8, xs)
        ex = apw.Fp8Experts(cuda(d["w1"]), cuda(d["s1"]), cuda(d["w2"]), cuda(d["s2"]))
        ws = torch.empty(apw.moe_workspace_fp8(ctx(), ex, T, topk), dtype=torch.uint8, device="cuda")
        out = torch.empty((T, H), dtype=torch.float16, device="cuda")
        apw.moe_forward_fp8(ctx(), ex, x, x8, xs, cuda(d["wr"]), None, T, topk, True, ws, out)
        x2 = torch.empty_like(x)
        apw.norm(ctx(), out, res, res, gamma, 1e-5, T, H, x2)
        torch.cuda.synchronize()
        check_norm(attn, res0, gamma, 1e-5, (None, x, x8, xs))
        d.update(x=x.cpu().numpy(), x8=codes(x8), xs=xs.cpu().numpy())
        want, bound = layer_ref(d, None, E, 0, H, F, T, topk, True)
        assert np.all(np.abs(np64(out) - want) <= bound)
        mid = (attn.float() + res0)
        assert torch.equal(res, out.float() + mid)
        check_norm(out, mid, gamma, 1e-5, (None, x2, None, None))



# ------------------------------------------------------------------ the tile product's forms

def tile_operands(r, loads, N, K, halves=1, normal=False):
    """Rows and weights of experts with the given numbers of rows, in any order of tokens
    (gathered).  normal: normally distributed values as e4m3 with their scales."""
    off = np.array(tiles.offsets_of(loads), np.int32)
    R, E = int(off[-1]), len(loads)
    perm = r.permutation(R).astype(np.int32)
    if normal:
        q, xs = ref.quant(r.normal(size=(R, K)))
        x8, xs = ref.encode(q), xs.astype(np.float32)
        w = r.normal(size=(E, N, K)) * 0.02
        nb, kb = ref.groups(N), ref.groups(K)
        ws = np.empty((E, 1, nb, kb), np.float32)
        w8 = np.empty((E, N, K), np.uint8)
        for i in range(nb):
            for j in range(kb):
                b = (slice(None), slice(i * 128, (i + 1) * 128), slice(j * 128, (j + 1) * 128))
                sc = (np.abs(w[b]).max(axis=(1, 2)) / 448.0).astype(np.float32)
                ws[:, 0, i, j] = sc
                w8[b] = ref.encode(ref.e4m3_round(w[b] / sc[:, None, None].astype(np.float64)))
    else:
        x8, xs = random_rows(r, R, K)
        w8, ws = random_weights(r, E, halves, N // halves, K)
        if halves == 2:
            xs = (xs / np.sqrt(K)).astype(np.float32)
    xv = ref.TABLE[x8] * ref.spread(xs.astype(np.float64), K)
    rows = N // halves
    wv = [np.concatenate([ref.block_values(w8[e, h * rows:(h + 1) * rows], ws[e, h]) for h in range(halves)])
          for e in range(E)]
    return R, E, [cuda(v) for v in (x8, xs, w8, ws, perm, off)], ref.product(xv, wv, perm, off, 1, True)


@pytest.mark.parametrize("loads,N,K", tiles.GEMMS)
def test_gemm_tiles(loads, N, K):
    """Every width of the tile product in whole tiles and in the parts of a last round, the
    whole output; the same bits again."""
    R, E, d, (want, mag) = tile_operands(rng_of("tiles", N, K), loads, N, K)
    for t in ("f32", "f16", "bf16"):
        outs = []
        for _ in range(3):
            out = torch.full((R + 1, N), 7.0, dtype=TORCH[t], device="cuda")
            apw.gemm_fp8(ctx(), *d[:4], E, N, K, True, *d[4:], R, 1, out)
            outs.append(out)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
        bound = mag * (sum_bound(K) + (0.0 if t == "f32" else 2.0 ** -10))
        bound = bound + (np.abs(want) + bound) * HALF_STEP[t] + SMALLEST[t]
        assert np.all(np.abs(np64(outs[0][:R]) - want) <= bound), t
        assert bool((outs[0][R:] == 7.0).all())


@pytest.mark.parametrize("loads,F,K", tiles.ACTS)
def test_gemm_act_tiles(loads, F, K):
    R, E, d, (gu, mag) = tile_operands(rng_of("act-tiles", F, K), loads, 2 * F, K, halves=2)
    outs = []
    for _ in range(3):
        a8 = torch.full((R + 1, F), 0x55, dtype=torch.uint8, device="cuda")
        sc = torch.full((R + 1, ref.groups(F)), -1.0, device="cuda")
        apw.gemm_act_fp8(ctx(), *d[:4], E, F, K, True, *d[4:], R, 1, a8, sc)
        outs.append((a8, sc))
    torch.cuda.synchronize()
    for a8, sc in outs[1:]:
        assert torch.equal(a8, outs[0][0]) and torch.equal(sc, outs[0][1])
    a8, sc = outs[0]
    check_rows8(*act_bounds(gu, mag, F, K), a8[:R], sc[:R], F)
    assert (codes(a8[R:]) == 0x55).all() and (np64(sc[R:]) == -1.0).all()


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("loads,N,K", [tiles.GEMMS[0], tiles.GEMMS[2], tiles.GEMMS[3]])
def test_gemm_16_bit_outputs_in_norm(loads, N, K, t):
    """What the e4m3 instruction leaves of normally distributed operands' products: an error
    d of 1.5e-5 of the result in norm.  The output, rounded to a step u, differs from the
    rounded 64-bit value by u with probability |d| / u, so the difference has the mean square
    E[u] E|d| (d and the value independent): u <= 2 HALF_STEP |v|, E|v| = 0.8 and E|d| = 0.8 of
    their norms.  Twice the 1.5e-5 is allowed."""
    R, E, d, (want, _) = tile_operands(rng_of("in-norm", N, K), loads, N, K, normal=True)
    out = torch.empty((R, N), dtype=TORCH[t], device="cuda")
    apw.gemm_fp8(ctx(), *d[:4], E, N, K, True, *d[4:], R, 1, out)
    rounded = torch.from_numpy(want).to(TORCH[t]).double().numpy()
    rel = np.linalg.norm(np64(out) - rounded) / np.linalg.norm(want)
    assert rel <= np.sqrt(2 * HALF_STEP[t] * 0.64 * 3e-5), rel


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("T,N", [(70, 8464), (1100, 8720)])
def test_gemm_16_bit_nan_stays_in_its_row_and_column(T, N, t):
    r = rng_of("nan-16", T, t)
    K = 400
    x8, xs = random_rows(r, T, K)
    w8, ws = random_weights(r, 1, 1, N, K)
    x8[T - 3, 390] = 0x7F
    w8[0, 140, 3] = 0xFF
    out = torch.empty((T, N), dtype=TORCH[t], device="cuda")
    apw.gemm_fp8(ctx(), *(cuda(v) for v in (x8, xs, w8, ws)), 1, N, K, False, None, None, T, 1, out)
    want = torch.zeros((T, N), dtype=torch.bool, device="cuda")
    want[T - 3], want[:, 140] = True, True
    assert torch.equal(out.isnan(), want)


def test_layer_tiles():
    """A layer whose down product runs 256-token tiles to fp32 (their rows leave LDS half by
    half): against 64 bits, and against its steps with fp32 sums, from which the e4m3
    instruction's sums differ as test_gemm_16_bit_outputs_in_norm says."""
    r = rng_of("layer-tiles")
    T, E, H, F = 1100, 2, 8720, 272
    d = layer_inputs(r, E, 0, H, F, T)
    z = d["x"].astype(np.float64) @ d["wr"].astype(np.float64).T
    chosen = np.argmax(z, axis=1)
    loads = np.bincount(chosen, minlength=E).tolist()
    assert any(f[2] > 128 and f[4] == 1 for f in tiles.forms(tiles.offsets_of(loads), H, False, False))
    got, (ex, args, _, out) = run_layer(d, None, E, 0, H, F, T, 1, True)
    xv = ref.TABLE[d["x8"]] * ref.spread(d["xs"].astype(np.float64), H)
    for e in range(E):
        t = np.nonzero(chosen == e)[0]
        w1 = np.concatenate([ref.block_values(d["w1"][e, h * F:(h + 1) * F], d["s1"][e, h]) for h in (0, 1)])
        w2 = ref.block_values(d["w2"][e], d["s2"][e, 0])
        a, err = act_bounds(xv[t] @ w1.T, np.abs(xv[t]) @ np.abs(w1).T, F, H)
        q, s = ref.quant(a)
        sv = ref.spread(s, F)
        step = 2 * np.maximum(np.exp2(np.floor(np.log2(np.maximum(np.abs(a / sv), 2.0 ** -6)))) * 2.0 ** -4, 2.0 ** -10)
        flips = np.abs(a / sv - q) >= step / 2 - err / sv - np.abs(a / sv) * 2.0 ** -21
        top = np.stack([err[:, g * 128:(g + 1) * 128].max(axis=1) for g in range(ref.groups(F))], axis=1)
        slack = np.where(flips, step, 0.0) * sv + np.abs(q * sv) * 2.0 ** -21 + ref.spread(top, F)
        want = (q * sv) @ w2.T
        bound = (np.abs(q * sv) @ np.abs(w2).T) * (sum_bound(F) + 2.0 ** -22 + 2.0 ** -10) + slack @ np.abs(w2).T
        bound += (np.abs(want) + bound) * 2.0 ** -11 + 2.0 ** -25
        assert np.all(np.abs(got[t] - want) <= bound)
    x, x8, xs, wr, _ = args
    w1, s1, w2, s2 = ex.tensors
    ids, perm, inv = (torch.empty(T, dtype=torch.int32, device="cuda") for _ in range(3))
    w, y = torch.empty((T, 1), device="cuda"), torch.empty((T, H), device="cuda")
    counts, off = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E, E + 1))
    a8, sc = torch.empty((T, F), dtype=torch.uint8, device="cuda"), torch.empty((T, ref.groups(F)), device="cuda")
    steps = torch.empty((T, H), dtype=torch.float16, device="cuda")
    apw.route(ctx(), x, wr, None, T, H, E, 1, True, ids, w, counts, off, perm, inv)
    apw.gemm_act_fp8(ctx(), x8, xs, w1, s1, E, F, H, True, perm, off, T, 1, a8, sc)
    apw.gemm_fp8(ctx(), a8, sc, w2, s2, E, H, F, False, perm, off, T, 1, y)
    apw.combine(ctx(), y, apw.F32, w, inv, T, 1, H, steps)
    diff = (out[:T].double() - steps.double()).norm() / steps.double().norm()
    # the codes here are uniform, not normal.  A group of 8 products loses at most 8 * 2^-13 of its
    # largest, a group's largest is no more than its root of squares, and the groups' signs are
    # independent: 2^-10 in norm; the two roundings to fp16 differ by at most 2 * 2^-11
    assert float(diff) <= 2.0 ** -9, float(diff)


# ------------------------------------------------------------------ offsets past 32 bits

def codes_on_gpu(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 255, shape, dtype=torch.uint8, device="cuda", generator=g)
    return c.masked_fill_(c == 0x7F, 0x7E)  # no NaN code


def check_part(x8, xs, w8, ws, got, K):
    """got = rows of x8 times rows of w8 (one 128-row block of scales each) to fp32."""
    x, w = ref.TABLE[codes(x8)] * ref.spread(np64(xs), K), ref.TABLE[codes(w8)] * ref.spread(np64(ws)[None], K)
    assert np.all(np.abs(np64(got) - x @ w.T) <= (np.abs(x) @ np.abs(w).T) * sum_bound(K))


@pytest.mark.parametrize("N", [48, 8720])
def test_gemm_rows_past_32_bits(N):
    """x8 (N = 48) or out (N = 8720) longer than 2^32 elements."""
    R, K = (70016, 65536) if N == 48 else (500032, 16)
    x8, w8 = codes_on_gpu(1, R, K), codes_on_gpu(2, 1, N, K)
    xs = torch.rand((R, ref.groups(K)), device="cuda") * 2.0 ** -9
    ws = torch.rand((1, ref.groups(N), ref.groups(K)), device="cuda") * 2.0 ** -9
    out = torch.empty((R, N), device="cuda")
    apw.gemm_fp8(ctx(), x8, xs, w8, ws, 1, N, K, False, None, None, R, 1, out)
    torch.cuda.synchronize()
    for rows in (slice(0, 8), slice(R - 8, R)):
        check_part(x8[rows], xs[rows], w8[0, N - 16:], ws[0, -1], out[rows, N - 16:], K)


def test_gemm_of_more_tiles_than_a_grid_dimension_holds():
    """2^30 rows, the most that a call takes: 2^23 tiles of 128, each row checked."""
    R, K = 1 << 30, 16
    x8 = torch.empty((R, K), dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    part = 1 << 25
    for r in range(0, R, part):
        x8[r:r + part] = torch.randint(0, 127, (part, K), dtype=torch.uint8, device="cuda", generator=g)
    w8 = codes_on_gpu(6, 1, 1, K)
    xs = torch.empty((R, 1), device="cuda").uniform_(0.5, 1.0, generator=g)
    ws = torch.full((1, 1, 1), 2.0 ** -9, device="cuda")
    out = torch.full((R, 1), float("nan"), device="cuda")
    apw.gemm_fp8(ctx(), x8, xs, w8, ws, 1, 1, K, False, None, None, R, 1, out)
    torch.cuda.synchronize()
    table = torch.from_numpy(ref.TABLE).cuda()
    w = table[w8.view(-1).long()] * 2.0 ** -9
    part = 1 << 22
    for r in range(0, R, part):
        v = table[x8[r:r + part].int()] * xs[r:r + part].double()
        want, mag = (v * w).sum(dim=1), (v * w).abs().sum(dim=1)
        assert bool(((out[r:r + part, 0].double() - want).abs() <= mag * sum_bound(K)).all()), r


@pytest.mark.parametrize("T", [6, 70])
def test_gemm_weights_past_32_bits(T):
    E, N, K = 3, 20096, 73728
    x8, w8 = codes_on_gpu(3, T, K), codes_on_gpu(4, E, N, K)
    xs = torch.rand((T, ref.groups(K)), device="cuda") * 2.0 ** -9
    ws = torch.rand((E, ref.groups(N), ref.groups(K)), device="cuda") * 2.0 ** -9
    off = torch.tensor([0, 1, 2, T], dtype=torch.int32, device="cuda")
    out = torch.empty((T, N), device="cuda")
    apw.gemm_fp8(ctx(), x8, xs, w8, ws, E, N, K, False, torch.arange(T, dtype=torch.int32, device="cuda"), off, T, 1,
                 out)
    torch.cuda.synchronize()
    for e, rows in ((0, slice(0, 1)), (1, slice(1, 2)), (2, slice(T - 4, T))):
        check_part(x8[rows], xs[rows], w8[e, N - 16:], ws[e, -1], out[rows, N - 16:], K)


def most_columns(seed, T, rows, halves=1):
    """Operands with nearly the most columns (the last block short), the rows of x zero but
    for 12 blocks over the whole length, which alone count: (operands, values of x and of w
    in those columns)."""
    K = (1 << 24) - 144
    KB = ref.groups(K)
    blocks = sorted({0, 1, 2, KB - 2, KB - 1} | {(i * KB) // 8 + i for i in range(1, 8)})
    g = torch.Generator(device="cuda").manual_seed(seed)
    x8 = torch.zeros((T, K), dtype=torch.uint8, device="cuda")
    cols = torch.cat([torch.arange(b * 128, min(K, b * 128 + 128), device="cuda") for b in blocks])
    x8[:, cols] = codes_on_gpu(seed, T, cols.numel())
    w8 = torch.empty((1, rows, K), dtype=torch.uint8, device="cuda")
    for r in range(rows):
        w8[0, r] = codes_on_gpu(seed + 1 + r, K)
    xs = torch.rand((T, KB), device="cuda", generator=g) * 2.0 ** -9
    ws = torch.rand((halves, ref.groups(rows // halves), KB), device="cuda", generator=g) * 2.0 ** -9
    b = cols // 128
    x = ref.TABLE[codes(x8[:, cols])] * np64(xs[:, b])
    row = torch.arange(rows, device="cuda")
    w = ref.TABLE[codes(w8[0][:, cols])] * np64(ws[row // (rows // halves), (row % (rows // halves)) // 128][:, b])
    return K, (x8, xs, w8, ws), x, w, (128 + 2 * len(blocks) + 11) * 2.0 ** -23


@pytest.mark.parametrize("T,N,t", [(3, 40, "f32"), (40, 40, "f16"), (1100, 256, "f16"), (1100, 256, "f32")])
def test_gemm_of_the_most_columns(T, N, t):
    K, d, x, w, bound = most_columns(7, T, N)
    out = torch.empty((T, N), dtype=TORCH[t], device="cuda")
    apw.gemm_fp8(ctx(), *d, 1, N, K, False, None, None, T, 1, out)
    want, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    bound = mag * (bound + (2.0 ** -10 if t == "f16" and T > 32 else 0.0))
    assert np.all(np.abs(np64(out) - want) <= bound + (np.abs(want) + bound) * HALF_STEP[t] + SMALLEST[t])


@pytest.mark.parametrize("T", [3, 20, 40])
def test_gemm_act_of_the_most_columns(T):
    F = 16
    K, d, x, w, bound = most_columns(9, T, 2 * F, halves=2)
    a8 = torch.empty((T, F), dtype=torch.uint8, device="cuda")
    sc = torch.empty((T, 1), device="cuda")
    apw.gemm_act_fp8(ctx(), *d, 1, F, K, False, None, None, T, 1, a8, sc)
    gu, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    g, u, s = gu[:, :F], gu[:, F:], ref.silu(gu[:, :F])
    dg, du = mag[:, :F] * bound, mag[:, F:] * bound
    err = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + np.abs(s * u) * 2.0 ** -20 + 2.0 ** -100 * np.abs(u)
    check_rows8(s * u, err, a8, sc, F)


def test_norm_rows_past_32_bits():
    T, H = 70016, 65536
    x = torch.empty((T, H), dtype=torch.float16, device="cuda").normal_()
    gamma = torch.ones(H, dtype=torch.float16, device="cuda")
    _, _, q, s = run_norm(x, None, gamma, 1e-5, want_y=False)
    for at in (slice(0, 4), slice(T - 4, T)):
        _, _, q1, s1 = run_norm(x[at].clone(), None, gamma, 1e-5, want_y=False)
        assert torch.equal(q[at], q1) and torch.equal(s[at], s1)


def test_same_bits_again():
    """No atomics: the same inputs give the same bits."""
    r = rng_of("again")
    T, topk, E, N, K = 90, 2, 4, 256, 1408
    perm, off = routing(r, T, topk, E)
    x8, xs = random_rows(r, T, K)
    w8, ws = random_weights(r, E, 1, N, K)
    d = [cuda(v) for v in (x8, xs, w8, ws, perm, off)]
    outs = []
    for _ in range(3):
        out = torch.empty((T * topk, N), device="cuda")
        apw.gemm_fp8(ctx(), *d[:4], E, N, K, True, d[4], d[5], T, topk, out)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
