// attn_decode.hip -- attention of one new token of each sequence over the paged cache,
// split over the cache's length and joined.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp2(c (q.k_j - m)),  c = scale * log2(e), m the running
// maximum of the scores; parts (m, l, o) and (m', l', o') join as exp2(c (m - M)) and
// exp2(c (m' - M)) times each, M = max(m, m').
//
// Bound by the cache's bytes: 131072 tokens of 8 heads of 128 in fp16 88 us, 6.1 TB/s (4 us of
// them the join); 64 sequences of 160 to 16000 157 us, 5.9; 200 of 870 to 2600 in 8 bits 123 to
// 129 us, 5.2 to 5.4.  Short caches are a chain of loads (length, page, keys) and the waves' join: 100 tokens
// 6.2 us, 601 8.4.
//
// A wave takes one 32-token tile after the other: the scores of 16 query heads of a key-value
// head from two 16-token products, the softmax in registers, the second product on the
// probabilities where they are.  Keys and values go from memory into registers (no LDS: the
// operands of the products are whole lines of the cache); the next tile's keys are asked for
// when this one's are used, its values likewise, so a wave always has 8 to 16 KB on the way.
//
// Every workgroup finds its sequence by a scan of the lengths, 64 a step, so a call's time has a
// part that grows with the square of the batch: sequences of 200 tokens, 32 heads over 8, take 42 us
// for 256 (5.0 TB/s), 190 for 1024 (4.5), 1177 for 4096 (2.9) and 11200 for 16384 (1.2).
//
// Probabilities are given to the second product as the sum of two 16-bit numbers: the
// matrix units have room (16 columns are computed for a group of 1 to 16 heads), and the
// output then has the error of its own rounding only.  In fp16 they are 2^15 times as large, so
// what is lost of one is at most 2^-40 of the largest; in bf16 2^-30 times (kTop, attn.h).
#include <algorithm>

#include "attn.h"

namespace apmoe {
namespace {

constexpr int kCols = 16;  // query heads of one workgroup

// How a call is split, by the workgroups that its sequences have without (a key-value head, 16
// query heads and a sequence each).
//
// Fewer than kFew (a CU each): parts for 512, two a CU in one round, of 4 tiles and more, and
// above 32 parts a row of 8.  131072 tokens of 48 heads over 8 88 us with 512, 97 with 768; one
// sequence of 8192 13.2 us in parts of 8 tiles and 15.9 in parts of 4, of 2000 11.1 and 10.0.
// More: parts of 16 tiles and more for 2048, in several rounds, for even rounds of uneven
// sequences (64 of 160 to 16000 tokens, 32 heads over 8: 158 us; with 1024 162, 512 177; 200 of
// 160 to 8000 292, with 1024 307, 512 334; 24 of 1500 to 30000 with a window of 4096, 16 heads:
// 64, 68 and 79).
// Not at all, and so without the second launch, where no query sees many tokens: up to 768, or
// 2048 with many workgroups (one of 601 8.4 us against 9.0, one of 1000 9.8 against 9.2; 32 of 512
// to 1024 20 against 26, 128 of 167 to 500 30 against 37), or 4096 of an 8-bit cache with kMany
// (as many bytes; 200 of 870 to 2600 123 us against 150; 160 of 30 to 3000 70 against 79; with 16
// bits 200 of 870 to 2600 take 210 against 223, but 128 of 133 to 4000 122 against 110).  These look at
// the bound of the lengths, which the host knows, and not at the lengths: one long sequence among
// short ones is then walked by one workgroup a head (not measured).  Then few
// have eight waves each (16 of 133 to 400 8.0 us against 9.4 with four), many four (128 of 167 to
// 500 30 against 40).
constexpr int kFew = 256, kMany = 1024;
constexpr int kWholeFew = 768, kWholeMany = 2048, kWhole8 = 4096;
constexpr int kPartsOnce = 512, kPartsEven = 2048;
constexpr int kTilesFew = 4, kTilesMany = 16;

// The tiles of one sequence that its query sees: [0, sink) and [first, end).
struct Span {
    int pos, end_tok, sink, first, tiles;
};

__device__ inline Span span_of(const AttnParams &P, int b)
{
    const int len = P.s.lens[b];
    Span r;
    r.pos = len - 1;
    r.end_tok = cached_tokens(P.s, len);
    const int end = (r.end_tok + kTile - 1) / kTile;
    r.first = P.window ? max(0, len - P.window) / kTile : 0;
    r.sink = P.window ? min(r.first, (int)(((int64_t)P.sinks + kTile - 1) / kTile)) : 0;
    r.sink = min(r.sink, end);
    r.tiles = r.sink + max(0, end - r.first);
    return r;
}

// Tiles of a part: every workgroup and the join compute the same number, from the lengths.
__device__ inline int part_tiles(const AttnParams &P)
{
    if (P.slots == P.s.B)  // whole sequences
        return 1 << 30;
    const int lane = threadIdx.x % kWave;
    int64_t mine = 0;
    for (int b = lane; b < P.s.B; b += kWave)
        mine += span_of(P, b).tiles;
    // below 2^35 a lane: in two parts
    const int64_t sum = ((int64_t)wave_sum((int)(mine >> 20)) << 20) + wave_sum((int)(mine & 0xFFFFF));
    const int64_t extra = P.slots - P.s.B;  // sum / ct more parts than sequences at most
    const int64_t ct = (sum + extra - 1) / extra;
    // parts of less than 8 tiles only where they are few (kTilesFew)
    return (int)max(max(ct, min((int64_t)8, 2 * ct)), (int64_t)P.part_tiles);
}

__device__ inline int parts_of(int tiles, int ct) { return max(1, (int)(((uint32_t)tiles + ct - 1) / (uint32_t)ct)); }

// 8-bit rows: a group of 128 columns is D / 128-th of a head.
__device__ inline void store_row(const AttnParams &P, size_t row, int d, const float (&v)[4], float scale)
{
    const size_t at = row * P.kv.D + d;
    if (P.out8) {
        const float inv = 1.0f / scale;
        *reinterpret_cast<uint32_t *>(P.out8 + at) = to_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    }
    if (P.out) {
        const u32x2 w = P.dtype == APMOE_F16 ? u32x2{pack2<APMOE_F16>(v[0], v[1]), pack2<APMOE_F16>(v[2], v[3])}
                                             : u32x2{pack2<APMOE_BF16>(v[0], v[1]), pack2<APMOE_BF16>(v[2], v[3])};
        *reinterpret_cast<u32x2 *>(P.out + at) = w;
    }
}

// ONCE: nothing else reads these bytes, and the caches shall keep other things: 131072 tokens of
// 8 heads 105 -> 91 us, 64 uneven sequences 176 -> 156, 200 in 8 bits 147 -> 135 (5.9 TB/s; a
// cache that fits the 256 MB behind the L2s and is read again and again loses up to 5%).  Where
// more than 16 query heads share a key-value head their workgroups read the same bytes: 64 of
// them 37 us, and 51 this way.
template <int QT, bool C8, int D, bool ONCE>
struct Tile {
    static constexpr int kVT = C8 ? APMOE_BF16 : QT;  // type of the second product (attn.h)
    static constexpr int KL = C8 ? D / 64 : D / 32;   // 1 KB requests of 16 tokens' keys
    u32x4 k[2][KL];
    u32x4 v16[C8 ? 1 : D / 16];
    u32x2 v8[C8 ? D / 16 : 1];
    float4v ks[2], vs[2];

    template <class V>
    __device__ static inline V load(const char *p)
    {
        if constexpr (ONCE)
            return __builtin_nontemporal_load(reinterpret_cast<const V *>(p));
        else
            return *reinterpret_cast<const V *>(p);
    }
    __device__ inline void load_k(const KvView &kv, size_t tile, size_t scale, int lane)
    {
        const char *p = static_cast<const char *>(kv.k) + tile * (C8 ? 1 : 2) + lane * 16;
#pragma unroll
        for (int a = 0; a < 2; ++a) {
#pragma unroll
            for (int s = 0; s < KL; ++s)
                k[a][s] = load<u32x4>(p + a * 16 * D * (C8 ? 1 : 2) + s * 1024);
            if constexpr (C8)
                ks[a] = *reinterpret_cast<const float4v *>(kv.ks + scale + 16 * a + 4 * (lane / 16));
        }
    }
    __device__ inline void load_v(const KvView &kv, size_t tile, size_t scale, int lane)
    {
        const size_t at = ((size_t)(lane / 16) * D + lane % 16) * 8;
        if constexpr (C8) {
            const char *p = static_cast<const char *>(kv.v) + tile + at;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                v8[i] = load<u32x2>(p + i * 128);
#pragma unroll
            for (int a = 0; a < 2; ++a)
                vs[a] = *reinterpret_cast<const float4v *>(kv.vs + scale + 16 * a + 4 * (lane / 16));
        } else {
            const char *p = static_cast<const char *>(kv.v) + (tile + at) * 2;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                v16[i] = load<u32x4>(p + i * 256);
        }
    }
    __device__ inline u32x4 value(int i) const
    {
        if constexpr (C8)
            return from_e4m3x8<kVT>(v8[i][0], v8[i][1]);
        else
            return v16[i];
    }
};

// Grid: x the slots (a part of a sequence each), y key-value heads x groups of 16 query heads.
template <int QT, bool C8, int D, int NW, bool ONCE>
__global__ void __launch_bounds__(NW *kWave, D == 256 ? 1 : 2) decode_kernel(const AttnParams P)
{
    using T = Tile<QT, C8, D, ONCE>;
    constexpr int DT = D / 16;
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int G = P.Hq / P.kv.Hkv, kvh = blockIdx.y % P.kv.Hkv, h0 = blockIdx.y / P.kv.Hkv * kCols;
    const int ct = part_tiles(P);
    int b, part, parts;
    if (!find_item(P.s.B, blockIdx.x, [&](int i) { return parts_of(span_of(P, i).tiles, ct); }, b, part, parts))
        return;
    const Span sp = span_of(P, b);
    const int t0 = part * ct, t1 = min(sp.tiles, t0 + ct);
    const int col = lane % 16, g = lane / 16;
    const bool live = h0 + col < G;
    // the queries: operand column `col`, the same columns of the row as the keys' lanes have
    u32x4 q[D / 32];
    {
        const uint16_t *row = P.q + (size_t)b * P.q_stride + ((size_t)kvh * G + (live ? h0 + col : 0)) * D;
#pragma unroll
        for (int s = 0; s < D / 32; ++s)
            q[s] = *reinterpret_cast<const u32x4 *>(row + (C8 ? 64 * (s / 2) + 16 * g + 8 * (s % 2) : 32 * s + 8 * g)) ^
                   query_sign(P.scale);
    }
    const float c = score_factor(P.scale);
    const int shift = P.kv.page_shift, tshift = shift - 5;
    const size_t head = (size_t)D << shift;
    const int32_t *table = P.s.pages + (size_t)b * P.s.max_pages;

    float m = -INFINITY, l = 0.0f;
    float4v o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i)
        o[i] = float4v{0.f, 0.f, 0.f, 0.f};

    // A wave's tiles are t0 + wave, + NW, ...; lane i has the page of the i-th of 64.
    auto token_tile = [&](int t) { return t < sp.sink ? t : sp.first + t - sp.sink; };
    int ids = 0;
    auto load_ids = [&](int t) {
        const int mine = t + lane * NW;
        ids = mine < t1 ? table[token_tile(mine) >> tshift] : -1;
    };
    T cur;
    size_t tile = 0, scale = 0;
    bool here = false;
    auto locate = [&](int t, int i) {
        const int id = __builtin_amdgcn_readlane(ids, i);
        here = id >= 0 && id < P.kv.n_pages;
        const int at = token_tile(t) & ((1 << tshift) - 1);
        const size_t base = (size_t)(here ? id : 0) * P.kv.Hkv + kvh;
        tile = base * head + (size_t)at * kTile * D;
        scale = (base << shift) + at * kTile;
    };
    int t = t0 + wave, i = 0;
    if (t < t1) {
        load_ids(t);
        locate(t, 0);
        cur.load_k(P.kv, tile, scale, lane);
        cur.load_v(P.kv, tile, scale, lane);
    }
    for (; t < t1; t += NW) {
        const bool on_page = here;
        const int next = t + NW;
        float4v s[2];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            s[a] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                if constexpr (C8) {
                    const u32x4 &w = cur.k[a][j / 2];
                    s[a] = mfma16(QT, from_e4m3x8<QT>(w[j % 2 * 2], w[j % 2 * 2 + 1]), q[j], s[a]);
                } else {
                    s[a] = mfma16(QT, cur.k[a][j], q[j], s[a]);
                }
            }
            if constexpr (C8)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[a][j] *= cur.ks[a][j];
        }
        if (next < t1) {
            if (++i == kWave) {
                i = 0;
                load_ids(next);
            }
            locate(next, i);
            cur.load_k(P.kv, tile, scale, lane);
        }
        // tokens of the tile: 16 a + 4 g + j of lane group g
        const int tok0 = token_tile(t) * kTile;
        const int last = tok0 + kTile - 1;
        const bool whole = on_page && last < sp.end_tok &&
                           (!P.window || sp.pos - tok0 < P.window || last < P.sinks);
        uint32_t seen = 0xFFu;
        if (!whole) {
            seen = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int tok = tok0 + 16 * (e / 4) + 4 * g + e % 4;
                const bool in = on_page && tok < sp.end_tok &&
                                (!P.window || sp.pos - tok < P.window || tok < P.sinks);
                seen |= in ? 1u << e : 0u;
            }
        }
        float x[8], top = -INFINITY;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = s[e / 4][e % 4];
            if (!whole && !(seen >> e & 1))
                x[e] = -INFINITY;
            top = fmaxf(top, x[e]);
        }
        top = fmaxf(top, __shfl_xor(top, 16, kWave));
        top = fmaxf(top, __shfl_xor(top, 32, kWave));
        if (__any(top > m)) {
            const float to = fmaxf(m, top);
            const float f = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m - to) * c);
            m = to;
            l *= f;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[d][j] *= f;
        }
        const float base = m == -INFINITY ? 0.0f : m;
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[e] - base, c, kTop<T::kVT>));
            l += p[e];
        }
        if constexpr (C8)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[e] *= cur.vs[e / 4][e % 4];
                if (!whole && !(seen >> e & 1))
                    p[e] = 0.0f;  // whatever scale lies there
            }
        u32x4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = pack2<T::kVT>(p[2 * e], p[2 * e + 1]);
            lo[e] = pack2<T::kVT>(p[2 * e] - low16<T::kVT>(hi[e]), p[2 * e + 1] - high16<T::kVT>(hi[e]));
        }
        if (whole) {
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const u32x4 v = cur.value(d);
                o[d] = mfma16(T::kVT, v, hi, o[d]);
                o[d] = mfma16(T::kVT, v, lo, o[d]);
            }
        } else {
            // what lies in places that are not seen may be a NaN: no factor makes it vanish
            u32x4 keep;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                keep[e] = (seen >> (2 * e) & 1 ? 0xFFFFu : 0u) | (seen >> (2 * e + 1) & 1 ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const u32x4 v = cur.value(d) & keep;
                o[d] = mfma16(T::kVT, v, hi, o[d]);
                o[d] = mfma16(T::kVT, v, lo, o[d]);
            }
        }
        if (next < t1)
            cur.load_v(P.kv, tile, scale, lane);
    }
    l += __shfl_xor(l, 16, kWave);
    l += __shfl_xor(l, 32, kWave);

    // Join the waves, half of them at a time into the other half.
    __shared__ float ml[NW][2][kCols];
    __shared__ float4v os[NW / 2][DT][kWave];
    if (g == 0) {
        ml[wave][0][col] = m;
        ml[wave][1][col] = l;
    }
    __syncthreads();
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w)
        M = fmaxf(M, ml[w][0][col]);
    float L = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const float lw = ml[w][1][col];
        L += lw * part_factor(ml[w][0][col], lw, M, c);
    }
    {
        const float f = part_factor(m, l, M, c);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[d][j] = l == 0.0f ? 0.0f : o[d][j] * f;
    }
#pragma unroll
    for (int half = NW / 2; half >= 1; half /= 2) {
        if (wave >= half && wave < 2 * half)
#pragma unroll
            for (int d = 0; d < DT; ++d)
                os[wave - half][d][lane] = o[d];
        __syncthreads();
        if (wave < half)
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[d][j] += os[wave][d][lane][j];
        __syncthreads();
    }
    if (wave != 0)
        return;
    const size_t headcol = (size_t)kvh * G + h0 + col;
    if (parts > 1) {
        if (!live)
            return;
        const size_t at = (size_t)blockIdx.x * P.Hq + headcol;
#pragma unroll
        for (int d = 0; d < DT; ++d)
            *reinterpret_cast<float4v *>(P.part_o + at * D + 16 * d + 4 * g) = o[d];
        if (g == 0) {
            P.part_ml[2 * at] = M;
            P.part_ml[2 * at + 1] = L;
        }
        return;
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;  // nothing seen: zeros
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[d][j] *= inv;
    const size_t row = (size_t)b * P.Hq + headcol;
    constexpr int kGroups = D < kBlk ? 1 : D / kBlk;
    float scale8[kGroups] = {};
    if (D >= kBlk && P.out8) {
#pragma unroll
        for (int n = 0; n < kGroups; ++n) {
            uint32_t a = 0;
#pragma unroll
            for (int d = 0; d < DT / kGroups; ++d)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    a = max(a, mag(o[n * (DT / kGroups) + d][j]));
            a = max(a, (uint32_t)__shfl_xor((int)a, 16, kWave));
            a = max(a, (uint32_t)__shfl_xor((int)a, 32, kWave));
            scale8[n] = scale_of(a);
            if (live && g == 0)
                P.out_scale[row * kGroups + n] = scale8[n];
        }
    }
    if (!live)
        return;
#pragma unroll
    for (int d = 0; d < DT; ++d) {
        const float v[4] = {o[d][0], o[d][1], o[d][2], o[d][3]};
        store_row(P, row, 16 * d + 4 * g, v, scale8[d * kGroups / DT]);
    }
}

// Joins the parts of split sequences.  A row of D / 4 threads has the columns; RP rows, whole
// waves, take every RP-th part of one query head of one sequence.
template <int D, int RP>
__global__ void __launch_bounds__(256) join_kernel(const AttnParams P)
{
    constexpr int kLanes = D / 4, kRows = 256 / kLanes, kHeads = kRows / RP;
    static_assert(RP * kLanes % kWave == 0, "a wave has one head");
    const int ct = part_tiles(P);
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, b = blockIdx.x;
    const int n = parts_of(span_of(P, b).tiles, ct);
    if (n <= 1)
        return;
    int first = 0;
    for (int i = lane; i < b; i += kWave)
        first += parts_of(span_of(P, i).tiles, ct);
    first = wave_sum(first);
    const int c = threadIdx.x % kLanes, r = threadIdx.x / kLanes, rp = r % RP;
    const int mine = blockIdx.y * kHeads + r / RP, h = min(mine, P.Hq - 1);
    const float *const ml = P.part_ml + 2 * ((size_t)first * P.Hq + h);
    const float *const po = P.part_o + ((size_t)first * P.Hq + h) * D + 4 * c;
    const size_t step = P.Hq;
    float M = -INFINITY;
    for (int i = lane; i < n; i += kWave)
        M = fmaxf(M, ml[2 * i * step]);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        M = fmaxf(M, __shfl_xor(M, d, kWave));
    __shared__ float fs[4][kWave];
    __shared__ float4v os[kRows][kLanes];
    __shared__ uint32_t top[kHeads][kLanes];
    float L = 0.0f;
    float4v o = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 < n; i0 += kWave) {
        const int i = i0 + lane, end = min(n - i0, kWave);
        float f = 0.0f;
        if (i < n) {
            const float l = ml[2 * i * step + 1];
            f = part_factor(ml[2 * i * step], l, M, score_factor(P.scale));
            L += f * l;
        }
        // the wave's own: its lanes read what they wrote before and after, in order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        fs[wave][lane] = f;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 4
        for (int j = rp; j < end; j += RP) {
            const float4v p = *reinterpret_cast<const float4v *>(po + (size_t)(i0 + j) * step * D);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[k] += fs[wave][j] * p[k];
        }
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        L += __shfl_xor(L, d, kWave);
    os[r][c] = o;
    __syncthreads();
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (rp == 0) {
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        uint32_t a = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int i = 0; i < RP; ++i)
                v[k] += os[r + i][c][k];
            v[k] *= inv;
            a = max(a, mag(v[k]));
        }
        top[r / RP][c] = a;
    }
    __syncthreads();
    if (rp != 0 || mine >= P.Hq)
        return;
    const size_t row = (size_t)b * P.Hq + h;
    float scale = 1.0f;
    if (D >= kBlk && P.out8) {
        uint32_t a = 0;
        for (int i = 0; i < kBlk / 4; ++i)
            a = max(a, top[r / RP][c / (kBlk / 4) * (kBlk / 4) + i]);
        scale = scale_of(a);
        if (c % (kBlk / 4) == 0)
            P.out_scale[row * (D / kBlk) + c / (kBlk / 4)] = scale;
    }
    store_row(P, row, 4 * c, v, scale);
}

template <int D, int RP>
hipError_t join_launch(const AttnParams &P, hipStream_t s)
{
    constexpr int kHeads = 256 / (D / 4) / RP;
    hipLaunchKernelGGL((join_kernel<D, RP>), dim3(P.s.B, (P.Hq + kHeads - 1) / kHeads), dim3(256), 0, s, P);
    return hipGetLastError();
}

template <int QT, bool C8, int D, int NW, bool ONCE>
hipError_t decode_waves(const AttnParams &P, hipStream_t s)
{
    const int G = P.Hq / P.kv.Hkv;
    hipLaunchKernelGGL((decode_kernel<QT, C8, D, NW, ONCE>), dim3(P.slots, P.kv.Hkv * ((G + kCols - 1) / kCols)),
                       dim3(NW * kWave), 0, s, P);
    return hipGetLastError();
}

template <int QT, bool C8, int D>
hipError_t decode_launch(const AttnParams &P, hipStream_t s)
{
    const bool once = P.Hq / P.kv.Hkv <= kCols;
    if constexpr (D <= 128)  // 8 waves leave 256 registers each
        if (P.slots == P.s.B && P.few && once)
            return decode_waves<QT, C8, D, 8, true>(P, s);
    const hipError_t e = once ? decode_waves<QT, C8, D, 4, true>(P, s) : decode_waves<QT, C8, D, 4, false>(P, s);
    if (e != hipSuccess || P.slots == P.s.B)
        return e;
    // few sequences have many parts
    return P.few ? join_launch<D, 1024 / D>(P, s) : join_launch<D, 4>(P, s);
}

template <int QT, bool C8>
hipError_t decode_dim(const AttnParams &P, hipStream_t s)
{
    if (P.kv.D == 64)
        return decode_launch<QT, C8, 64>(P, s);
    if (P.kv.D == 128)
        return decode_launch<QT, C8, 128>(P, s);
    return decode_launch<QT, C8, 256>(P, s);
}

}  // namespace

// How a call is split.  Rows: workgroups that a sequence has anyway; seen: tokens that a query
// sees at most.
DecodePlan decode_plan(int B, int Hkv, int Hq, bool c8, int64_t seen)
{
    const int rows = Hkv * ((Hq / Hkv + kCols - 1) / kCols), all = B * rows;
    DecodePlan p;
    p.few = all < kFew;
    p.part_tiles = p.few ? kTilesFew : kTilesMany;
    const int whole = p.few ? kWholeFew : c8 && all >= kMany ? kWhole8 : kWholeMany;
    p.slots = seen <= whole ? B : B + std::max(1, (p.few ? kPartsOnce : kPartsEven) / rows);
    return p;
}

int decode_slots_most(int B, int Hkv, int Hq)
{
    const int rows = Hkv * ((Hq / Hkv + kCols - 1) / kCols);
    return B + std::max(1, kPartsEven / rows);
}

hipError_t launch_attn_decode(const AttnParams &P, hipStream_t s)
{
    if (P.dtype == APMOE_F16)
        return P.kv.c8 ? decode_dim<APMOE_F16, true>(P, s) : decode_dim<APMOE_F16, false>(P, s);
    return P.kv.c8 ? decode_dim<APMOE_BF16, true>(P, s) : decode_dim<APMOE_BF16, false>(P, s);
}

}  // namespace apmoe
