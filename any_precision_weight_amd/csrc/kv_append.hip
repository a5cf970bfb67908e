// kv_append.hip -- new tokens into the paged cache: the position rotation of queries and
// keys, the keys and values in the cache's order (attn.h), in 16 bits or as e4m3 rows.
//
// A rotated pair is (x c - y s, x s + y c), in fp64: the products are exact there and a
// value is rounded once, to the type it is stored in.  An e4m3 row is s = max(max |v| / 448,
// 2^-126) in fp32 and v / s, in fp64 too: 16-bit rows have many quotients on or next to a
// border between two e4m3 values.
//
// Bound by memory for many tokens, by the chain of a few dependent loads (length, page,
// rotation's row) for few.
#include <algorithm>

#include "attn.h"

namespace apmoe {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kGridX = 1u << 22;

// A token of the call: its position, and its place in the cache (page < 0: none).
struct Place {
    int pos, page, at;
};

__device__ inline Place place_of(const AppendParams &P, int b, int pos)
{
    Place r{pos, -1, pos & ((1 << P.kv.page_shift) - 1)};
    if (pos >= 0 && pos < P.s.room && !(P.rope && pos >= P.n_pos)) {
        const int p = P.s.pages[(size_t)b * P.s.max_pages + (pos >> P.kv.page_shift)];
        r.page = p >= 0 && p < P.kv.n_pages ? p : -1;
    }
    return r;
}

__device__ inline u32x4 load16(const uint16_t *p) { return *reinterpret_cast<const u32x4 *>(p); }

template <int DT>
__device__ inline double value_of(const u32x4 &x, int i)
{
    const uint32_t w = x[i / 2];
    return (double)(i & 1 ? high16<DT>(w) : low16<DT>(w));
}

// fp64 -> fp32 for a second rounding to few bits: the last bit is set where the value is
// not exact (round to odd), so the second rounding sees on which side of a border it is.
__device__ inline float to_odd(double v)
{
    float f = (float)v;
    const double d = (double)f;
    if (d != v) {
        uint32_t b = __builtin_bit_cast(uint32_t, f);
        if (__builtin_fabs(d) > __builtin_fabs(v))
            b -= 1;  // toward zero
        f = __builtin_bit_cast(float, b | 1u);
    }
    return f;
}

// fp64 -> DT, rounded once: through fp32 only a value that falls on a border there can go
// wrong, and those (2^-13 or 2^-16 of all) are done again.
template <int DT>
__device__ inline u32x4 to16(const double (&v)[8])
{
    constexpr uint32_t kLow = DT == APMOE_F16 ? 0x1FFFu : 0xFFFFu, kBorder = DT == APMOE_F16 ? 0x1000u : 0x8000u;
    // fp16's subnormal numbers have their borders elsewhere
    constexpr uint32_t kNormal = DT == APMOE_F16 ? 0x38800000u : 0x00800000u;
    float f[8];
    bool again = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f[i] = (float)v[i];
        const uint32_t b = __builtin_bit_cast(uint32_t, f[i]);
        again |= ((b & kLow) == kBorder) | (mag(f[i]) < kNormal);
    }
    if (again)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = to_odd(v[i]);
    return u32x4{pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]), pack2<DT>(f[4], f[5]), pack2<DT>(f[6], f[7])};
}

// A head's row is handled as D / 16 pairs of chunks of 8 columns: those of a pair are rotated
// by the same angles (i and i + rot / 2), or lie side by side.
struct Pair {
    int a, b;   // the chunks
    bool turn;  // rotated
};

__device__ inline Pair pair_of(const AppendParams &P, int i)
{
    const int n = P.rot / 16;
    if (i >= n || P.interleaved)
        return Pair{2 * i, 2 * i + 1, i < n};
    return Pair{i, i + n, true};
}

// The angles of a pair: cosines and sines of 8 turns each; with pairs of neighbours the first
// four are chunk a's, the others chunk b's.
struct Turn {
    float4v c[2], s[2];
};

__device__ inline Turn turn_of(const AppendParams &P, int pos, int i)
{
    Turn t;
    const float *row = P.rope + (size_t)pos * P.rot + 8 * i;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        t.c[h] = *reinterpret_cast<const float4v *>(row + 4 * h);
        t.s[h] = *reinterpret_cast<const float4v *>(row + P.rot / 2 + 4 * h);
    }
    return t;
}

template <int DT>
__device__ inline void rotate(const AppendParams &P, const Pair &pr, const Turn &t, const u32x4 &xa, const u32x4 &xb,
                              double (&a)[8], double (&b)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = value_of<DT>(xa, i);
        b[i] = value_of<DT>(xb, i);
    }
    if (!pr.turn)
        return;
    if (P.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            double(&v)[8] = i < 4 ? a : b;
            const double c = (double)t.c[i / 4][i % 4], s = (double)t.s[i / 4][i % 4];
            const double x = v[2 * (i % 4)], y = v[2 * (i % 4) + 1];
            v[2 * (i % 4)] = x * c - y * s;
            v[2 * (i % 4) + 1] = x * s + y * c;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const double c = (double)t.c[i / 4][i % 4], s = (double)t.s[i / 4][i % 4], x = a[i], y = b[i];
            a[i] = x * c - y * s;
            b[i] = x * s + y * c;
        }
    }
}

__device__ inline uint64_t mag64(double v) { return __builtin_bit_cast(uint64_t, v) & 0x7FFFFFFFFFFFFFFFull; }

// Scale of a row from the largest magnitude of each of `lanes` neighbouring lanes.
__device__ inline float row_scale(uint64_t m, int lanes)
{
    for (int d = lanes / 2; d >= 1; d >>= 1) {
        const uint64_t o = (uint64_t)__shfl_xor((unsigned long long)m, d, kWave);
        m = o > m ? o : m;
    }
    const float s = (float)(__builtin_bit_cast(double, m) / (double)kE4m3Max);
    return s < kScaleMin ? kScaleMin : s;  // a NaN stays
}

// v / s from v times r, r = 1 / s rounded: with the remainder added a quotient that fp64 holds
// comes out as it is, and others on their side of every border of e4m3.
__device__ inline float quotient(double v, double s, double r)
{
    const double q = v * r;
    return __builtin_copysignf(to_odd(__builtin_fma(__builtin_fma(-q, s, v), r, q)), (float)v);
}

__device__ inline u32x2 to8(const double (&v)[8], double s, double r)
{
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        q[i] = quotient(v[i], s, r);
    return u32x2{to_e4m3x4(q[0], q[1], q[2], q[3]), to_e4m3x4(q[4], q[5], q[6], q[7])};
}

// Where head h of a page starts, in elements of K or V.
__device__ inline size_t head_base(const KvView &kv, int page, int h)
{
    return ((size_t)page * kv.Hkv + h) * ((size_t)kv.D << kv.page_shift);
}

__device__ inline size_t scale_at(const KvView &kv, int page, int h, int at)
{
    return (((size_t)page * kv.Hkv + h) << kv.page_shift) + at;
}

// A pair of chunks of a key; the D / 16 lanes of a row call it together.
template <int DT, bool C8>
__device__ inline void store_k(const KvView &kv, const Place &pl, int h, int lane, const Pair &pr, const double (&a)[8],
                               const double (&b)[8])
{
    const size_t tile = head_base(kv, pl.page, h) + (size_t)(pl.at / 16) * 16 * kv.D;
    const int t = pl.at % 16;
    if constexpr (C8) {
        uint64_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t x = mag64(a[i]), y = mag64(b[i]);
            m = x > m ? x : m;
            m = y > m ? y : m;
        }
        const float s = row_scale(m, kv.D / 16);
        const double r = 1.0 / (double)s;
        uint8_t *p = static_cast<uint8_t *>(kv.k) + tile;
        *reinterpret_cast<u32x2 *>(p + (pr.a / 2 * 16 + t) * 16 + pr.a % 2 * 8) = to8(a, s, r);
        *reinterpret_cast<u32x2 *>(p + (pr.b / 2 * 16 + t) * 16 + pr.b % 2 * 8) = to8(b, s, r);
        if (lane == 0)
            kv.ks[scale_at(kv, pl.page, h, pl.at)] = s;
    } else {
        uint16_t *p = static_cast<uint16_t *>(kv.k) + tile;
        *reinterpret_cast<u32x4 *>(p + (pr.a * 16 + t) * 8) = to16<DT>(a);
        *reinterpret_cast<u32x4 *>(p + (pr.b * 16 + t) * 8) = to16<DT>(b);
    }
}

template <int DT>
__device__ inline void store_q(const AppendParams &P, uint32_t t, int h, const Pair &pr, const double (&a)[8],
                               const double (&b)[8])
{
    uint16_t *o = P.q_out + ((size_t)t * P.Hq + h) * P.kv.D;
    *reinterpret_cast<u32x4 *>(o + 8 * pr.a) = to16<DT>(a);
    *reinterpret_cast<u32x4 *>(o + 8 * pr.b) = to16<DT>(b);
}

// Bound by the chain of its loads: 1 token of 32 + 16 heads of 128 2.6 us (one kernel launch
// in a graph), 256 tokens of 16 + 8 heads of 256 5.3 us, of 32 + 16 heads of 128 5.6 and to e4m3 5.5
// (one token 3.6).
//
// One row a sequence: a workgroup has some heads of a token, a thread a pair of chunks of a
// query, a key or a value.  Values go to their granules, of 8 tokens each, element by element.
template <int DT, bool C8>
__global__ void __launch_bounds__(kThreads) append_token(const AppendParams P)
{
    const KvView &kv = P.kv;
    const int pairs = kv.D / 16, heads = P.Hq + 2 * kv.Hkv;
    const uint32_t t = blockIdx.x;
    const int i = (int)(blockIdx.y * kThreads + threadIdx.x), h = i / pairs, lane = i % pairs;
    if (h >= heads)
        return;
    const uint16_t *row = h < P.Hq            ? P.q + (size_t)t * P.q_stride + (size_t)h * kv.D
                          : h < P.Hq + kv.Hkv ? P.k + (size_t)t * P.k_stride + (size_t)(h - P.Hq) * kv.D
                                              : P.v + (size_t)t * P.v_stride + (size_t)(h - P.Hq - kv.Hkv) * kv.D;
    Pair pr = pair_of(P, lane);
    if (h >= P.Hq + kv.Hkv)
        pr.turn = false;
    const u32x4 xa = load16(row + 8 * pr.a), xb = load16(row + 8 * pr.b);
    const Place pl = place_of(P, (int)t, P.s.lens[t] - 1);
    if (pl.page < 0)
        return;
    Turn tn;
    if (pr.turn)
        tn = turn_of(P, pl.pos, lane);
    double a[8], b[8];
    rotate<DT>(P, pr, tn, xa, xb, a, b);
    if (h < P.Hq) {
        store_q<DT>(P, t, h, pr, a, b);
    } else if (h < P.Hq + kv.Hkv) {
        store_k<DT, C8>(kv, pl, h - P.Hq, lane, pr, a, b);
    } else {
        const int g = h - P.Hq - kv.Hkv, u = pl.at % kTile;
        const size_t at = head_base(kv, pl.page, g) + (size_t)(pl.at / kTile) * kTile * kv.D +
                          (size_t)(u % 16 / 4) * kv.D * 8 + u / 16 * 4 + u % 4;
        if constexpr (C8) {
            uint64_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint64_t x = mag64(a[j]), y = mag64(b[j]);
                m = x > m ? x : m;
                m = y > m ? y : m;
            }
            const float s = row_scale(m, pairs);
            const double r = 1.0 / (double)s;
            const u32x2 qa = to8(a, s, r), qb = to8(b, s, r);
            uint8_t *p = static_cast<uint8_t *>(kv.v) + at;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                p[(8 * pr.a + j) * 8] = (uint8_t)(qa[j / 4] >> (8 * (j % 4)));
                p[(8 * pr.b + j) * 8] = (uint8_t)(qb[j / 4] >> (8 * (j % 4)));
            }
            if (lane == 0)
                kv.vs[scale_at(kv, pl.page, g, pl.at)] = s;
        } else {
            uint16_t *p = static_cast<uint16_t *>(kv.v) + at;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                p[(8 * pr.a + j) * 8] = (uint16_t)(xa[j / 2] >> (16 * (j % 2)));
                p[(8 * pr.b + j) * 8] = (uint16_t)(xb[j / 2] >> (16 * (j % 2)));
            }
        }
    }
}

// Several rows a sequence: a workgroup has a tile of 32 places of a sequence's cache and one
// key-value head, with every Hkv-th query head.  Threads are (token, pair of chunks), 8 tokens
// x 8 pairs a wave where a row has as many: whole lines of the cache are written, and read.
// The angles are read once for all heads.  Values pass through LDS: a thread gathers 8 tokens
// x 8 columns of a granule's tokens.
//
// 18657 rows of 48 + 16 heads of 128 in fp16: 135 us, 4.6 TB/s of the 4.9 that a copy reaches
// here; written token by token, 16 bytes and 2 bytes at a time, it was 324 us, for a cache line
// of 8 tokens was put together from 8 workgroups on 8 XCDs.  4556 rows of 32 + 16 heads to
// e4m3: 32 us, 3.3 TB/s.  Three waves a SIMD is what the fp64 pairs' registers leave room for, and
// not quite: fp16 rows take 12 to 20 bytes of scratch a lane, e4m3 ones 20 to 48.
template <int DT, bool C8, int D>
__global__ void __launch_bounds__(kThreads, 3) append_tile(const AppendParams P)
{
    constexpr int kPairs = D / 16;
    const KvView &kv = P.kv;
    const uint32_t block = blockIdx.y * kGridX + blockIdx.x;
    const int head = (int)(block % (uint32_t)kv.Hkv);
    const int32_t *off = P.s.q_offsets;
    // tiles that sequence b's new tokens lie in
    auto new_of = [&](int b) { return off ? max(0, off[b + 1] - off[b]) : 1; };
    auto first_of = [&](int b, int n) { return max(0, P.s.lens[b] - n) / kTile; };
    int b, local, tiles;
    if (!find_item(P.s.B, (int)(block / (uint32_t)kv.Hkv), [&](int i) {
            const int n = new_of(i);
            return n > 0 && P.s.lens[i] > 0 ? (P.s.lens[i] - 1) / kTile - first_of(i, n) + 1 : 0;
        }, b, local, tiles))
        return;
    const int n = new_of(b), len = P.s.lens[b], tile = first_of(b, n) + local;
    const int64_t row0 = (int64_t)(off ? off[b] : b) - (len - n);  // row of position 0
    // the tile's tokens that are new and have a place: positions from .. to - 1
    const int from = max(tile * kTile, max(0, len - n));
    int to = min(min(tile * kTile + kTile, len), P.s.room);
    if (P.rope)
        to = min(to, P.n_pos);
    to = (int)min((int64_t)to, (int64_t)P.s.T - row0);
    if (from >= to || row0 + from < 0)
        return;
    const int page = place_of(P, b, from).page;  // of all of them
    if (page < 0)
        return;

    const int tid = threadIdx.x;

    // Values, to LDS.  16 bits: granules, item (g, c) has columns 8 c .. + 7 of granule g's
    // tokens 4 g .. + 3, 16 + 4 g .. + 3; one granule is left out after 8, so that neighbours in
    // c lie in other banks.  The last wave begins: with few tokens the others have the keys and
    // queries meanwhile.  8 bits: rows.
    constexpr int kChunks = D / 8, kSize = C8 ? 8 : 16, kRow = D + 8;
    __shared__ __attribute__((aligned(16))) char lds[C8 ? kTile * kRow : 4 * (D + D / 8) * 16];
    auto slot = [](int g, int d) { return (g * (D + D / 8) + d + d / 8) * 16; };
    auto token = [&](int g, int j) { return j / 4 * 16 + 4 * g + j % 4; };
    auto is_new = [&](int u) { return tile * kTile + u >= from && tile * kTile + u < to; };
    const uint16_t *const values = P.v + (size_t)head * D;
    auto value_row = [&](int u) { return values + (size_t)(row0 + tile * kTile + u) * P.v_stride; };
    if constexpr (C8) {
        for (int i = tid; i < kTile * kChunks; i += kThreads) {
            const int u = i / kChunks, c = i % kChunks;
            if (!is_new(u))
                continue;
            const u32x4 x = load16(value_row(u) + 8 * c);
            double v[8];
            uint64_t m = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[k] = value_of<DT>(x, k);
                const uint64_t y = mag64(v[k]);
                m = y > m ? y : m;
            }
            const float s = row_scale(m, kChunks);
            *reinterpret_cast<u32x2 *>(lds + u * kRow + 8 * c) = to8(v, s, 1.0 / (double)s);
            if (c == 0)
                kv.vs[scale_at(kv, page, head, (tile * kTile + u) & ((1 << kv.page_shift) - 1))] = s;
        }
    } else {
        for (int i = (tid + kWave) % kThreads; i < 4 * kChunks; i += kThreads) {
            const int g = i / kChunks, c = i % kChunks;
            u32x4 x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = u32x4{0, 0, 0, 0};
                if (is_new(token(g, j)))
                    x[j] = load16(value_row(token(g, j)) + 8 * c);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                u32x4 w;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t lo = x[2 * j][k / 2], hi = x[2 * j + 1][k / 2];
                    w[j] = k % 2 ? lo >> 16 | (hi & 0xFFFF0000u) : (lo & 0xFFFFu) | hi << 16;
                }
                *reinterpret_cast<u32x4 *>(lds + slot(g, 8 * c + k)) = w;
            }
        }
    }
    // Keys (head 0 of the list) and queries: the angles are read once for a thread's heads;
    // with few tokens there are threads for several heads at a time.
    {
        const int lane = tid % kPairs, item = tid / kPairs, tokens = to - from;
        const int sets = max(1, kThreads / kPairs / tokens), set = item / tokens;
        const Pair pr = pair_of(P, lane);
        const int heads = 1 + (P.Hq > head ? (P.Hq - head + kv.Hkv - 1) / kv.Hkv : 0);
        for (int pos = from + (sets > 1 ? item % tokens : item); pos < to && set < sets; pos += kThreads / kPairs) {
            const size_t t = (size_t)(row0 + pos);
            const Place pl{pos, page, pos & ((1 << kv.page_shift) - 1)};
            Turn tn;
            if (pr.turn)
                tn = turn_of(P, pos, lane);
            double a[8], v[8];
            int h = set;
            if (h == 0) {
                const uint16_t *x = P.k + t * P.k_stride + (size_t)head * D;
                rotate<DT>(P, pr, tn, load16(x + 8 * pr.a), load16(x + 8 * pr.b), a, v);
                store_k<DT, C8>(kv, pl, head, lane, pr, a, v);
                h = sets;
            }
            const uint16_t *x = P.q + t * P.q_stride;
#pragma unroll 2
            for (; h < heads; h += sets) {
                const int qh = head + (h - 1) * kv.Hkv;
                rotate<DT>(P, pr, tn, load16(x + (size_t)qh * D + 8 * pr.a), load16(x + (size_t)qh * D + 8 * pr.b), a, v);
                store_q<DT>(P, (uint32_t)t, qh, pr, a, v);
            }
            if (sets > 1)
                break;
        }
    }
    __syncthreads();
    char *const out = static_cast<char *>(kv.v) +
                      (head_base(kv, page, head) + (size_t)(tile * kTile & ((1 << kv.page_shift) - 1)) * D) * (kSize / 8);
    for (int i = tid; i < 4 * D; i += kThreads) {
        const int g = i / D, d = i % D;
        uint32_t in = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            in |= is_new(token(g, j)) ? 1u << j : 0u;
        if (in == 0)
            continue;
        char *p = out + (size_t)i * kSize;
        if constexpr (C8) {
            uint8_t x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = in >> j & 1 ? (uint8_t)lds[token(g, j) * kRow + d] : 0;
            if (in == 0xFFu) {
                *reinterpret_cast<u32x2 *>(p) = u32x2{(uint32_t)x[0] | x[1] << 8 | x[2] << 16 | (uint32_t)x[3] << 24,
                                                      (uint32_t)x[4] | x[5] << 8 | x[6] << 16 | (uint32_t)x[7] << 24};
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)  // other tokens' elements stay
                    if (in >> j & 1)
                        p[j] = (char)x[j];
            }
        } else {
            const u32x4 w = *reinterpret_cast<const u32x4 *>(lds + slot(g, d));
            if (in == 0xFFu) {
                *reinterpret_cast<u32x4 *>(p) = w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (in >> j & 1)
                        reinterpret_cast<uint16_t *>(p)[j] = (uint16_t)(w[j / 2] >> (16 * (j % 2)));
            }
        }
    }
}

template <int DT, bool C8>
hipError_t append_launch(const AppendParams &P, hipStream_t s)
{
    if (!P.s.q_offsets) {
        const int items = (P.Hq + 2 * P.kv.Hkv) * (P.kv.D / 16);
        hipLaunchKernelGGL((append_token<DT, C8>), dim3(P.s.T, (items + kThreads - 1) / kThreads), dim3(kThreads), 0, s, P);
        return hipGetLastError();
    }
    // n tokens lie in (n + 62) / 32 tiles at most
    const int64_t tiles = std::min<int64_t>(P.s.T, (int64_t)P.s.T / kTile + 2 * (int64_t)P.s.B);
    const int64_t blocks = tiles * P.kv.Hkv;
    const dim3 grid((uint32_t)std::min<int64_t>(blocks, kGridX), (uint32_t)((blocks + kGridX - 1) / kGridX));
    if (P.kv.D == 64)
        hipLaunchKernelGGL((append_tile<DT, C8, 64>), grid, dim3(kThreads), 0, s, P);
    else if (P.kv.D == 128)
        hipLaunchKernelGGL((append_tile<DT, C8, 128>), grid, dim3(kThreads), 0, s, P);
    else
        hipLaunchKernelGGL((append_tile<DT, C8, 256>), grid, dim3(kThreads), 0, s, P);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const AppendParams &P, hipStream_t s)
{
    if (P.dtype == APMOE_F16)
        return P.kv.c8 ? append_launch<APMOE_F16, true>(P, s) : append_launch<APMOE_F16, false>(P, s);
    return P.kv.c8 ? append_launch<APMOE_BF16, true>(P, s) : append_launch<APMOE_BF16, false>(P, s);
}

}  // namespace apmoe
