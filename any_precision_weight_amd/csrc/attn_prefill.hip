// attn_prefill.hip -- causal attention of the new tokens of prompts (or of their chunks) over
// the paged cache, with a sliding window and first tokens that stay visible.
//
// The formulas are attn_decode.hip's.  A row is a (new token, query head) pair; the heads of a
// key-value head's group are neighbours, so a workgroup's 128 rows share their keys and
// values whatever the group's size.  Four waves have 32 rows each and walk over 64 cached
// tokens at a time, staged in LDS in the cache's own order: the operands of the 32 x 32
// products are then 16-byte reads of neighbouring places.
//
// Rows of a key operand: row 16 t + 8 a + 4 h + b of a 32-token product is token 16 a + 8 t +
// 4 h + b.  Lane half h then has, of scores 8t .. 8t+7, the tokens of granule g = 2 t + h of
// V (attn.h), and the probabilities need not move.
#include "attn.h"

namespace apmoe {
namespace {

constexpr int kWaves = 4;
constexpr int kRows = 32 * kWaves;  // rows of a workgroup
constexpr int kStep = 64;           // cached tokens of a step
constexpr uint32_t kGridX = 1u << 22;

__device__ inline int new_tokens(const AttnBatch &S, int b)
{
    return S.q_offsets ? max(0, S.q_offsets[b + 1] - S.q_offsets[b]) : 1;
}

template <int QT, bool C8, int D>
struct Prefill {
    static constexpr int kVT = C8 ? APMOE_BF16 : QT;
    // fp16 queries on an 8-bit cache: probabilities times scales have bf16's range, and two
    // bf16 numbers keep what fp16 would
    static constexpr bool kTwo = C8 && QT == APMOE_F16;
    static constexpr int kBytes = kStep * D * 2;  // of a step's keys, and of its values
    static constexpr int kScales = C8 ? 2 * kStep * 4 : 0;
    static constexpr int kLds = 2 * kBytes + kScales;
};

// One granule (16 bytes of LDS) of values: the non-finite ones become 0, and their signs go
// into two operands: 1 where a value is +infinity or a NaN, 1 where -infinity or a NaN.
template <int DT>
__device__ inline void split_values(u32x4 &v, u32x4 &plus, u32x4 &minus)
{
    constexpr uint32_t kInf = DT == APMOE_F16 ? 0x7C00u : 0x7F80u, kOne = DT == APMOE_F16 ? 0x3C00u : 0x3F80u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t keep = 0, p = 0, n = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t x = v[i] >> (16 * h) & 0xFFFFu, a = x & 0x7FFFu;
            const bool bad = a >= kInf, nan = a > kInf, neg = x >> 15;
            keep |= bad ? 0u : x << (16 * h);
            p |= bad && (nan || !neg) ? kOne << (16 * h) : 0u;
            n |= bad && (nan || neg) ? kOne << (16 * h) : 0u;
        }
        v[i] = keep;
        plus[i] = p;
        minus[i] = n;
    }
}

template <int DT>
__device__ inline bool not_finite(const u32x4 &v)
{
    constexpr uint32_t kInf = DT == APMOE_F16 ? 0x7C00u : 0x7F80u;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bad |= (v[i] & kInf) == kInf || (v[i] >> 16 & kInf) == kInf;
    return bad;
}

__device__ inline u32x4 lds16(const char *base, int at) { return *reinterpret_cast<const u32x4 *>(base + at); }

template <int QT, bool C8, int D>
__global__ void __launch_bounds__(kWaves *kWave) prefill_kernel(const AttnParams P)
{
    using C = Prefill<QT, C8, D>;
    constexpr int VT = C::kVT, KS = D / 16, DB = D / 32;
    __shared__ __attribute__((aligned(16))) char lds[C::kLds];
    char *const k_lds = lds, *const v_lds = lds + C::kBytes;
    float *const ks_lds = reinterpret_cast<float *>(lds + 2 * C::kBytes), *const vs_lds = ks_lds + kStep;

    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int G = P.Hq / P.kv.Hkv, kvh = blockIdx.y;
    const uint32_t block = blockIdx.z * kGridX + blockIdx.x;
    int b, rt, n_rt;
    if (block > 0x7FFFFFFFu || !find_item(P.s.B, (int)block, [&](int i) {
            return (int)(((int64_t)new_tokens(P.s, i) * G + kRows - 1) / kRows);
        }, b, rt, n_rt))
        return;
    rt = n_rt - 1 - rt;  // the rows with the most to see first
    const int nq = new_tokens(P.s, b), row_of_b = P.s.q_offsets ? P.s.q_offsets[b] : b;
    const int len = P.s.lens[b], end_tok = cached_tokens(P.s, len);
    const int64_t rows = (int64_t)nq * G;
    const int64_t r0 = (int64_t)rt * kRows;

    // this lane's row (as a column of the products), and the positions of its wave's
    const int col = lane % 32, h = lane / 32;
    const int64_t r = min(r0 + wave * 32 + col, rows - 1);
    const int qi = (int)(r / G), qh = kvh * G + (int)(r % G);
    const int64_t token = (int64_t)row_of_b + qi;
    const bool live = r0 + wave * 32 + col < rows && token >= 0 && token < P.s.T;
    const int pos = len - nq + qi;
    auto pos_of = [&](int64_t row) { return len - nq + (int)(min(row, rows - 1) / G); };
    const int wave_lo = pos_of(r0 + wave * 32), wave_hi = pos_of(r0 + wave * 32 + 31);
    const int lo = pos_of(r0), hi = pos_of(r0 + kRows - 1);

    // steps that a row of the workgroup sees: [0, sink) and [first, end)
    const int end = (max(0, min(end_tok, hi + 1)) + kStep - 1) / kStep;
    const int first = P.window ? max(0, lo - P.window + 1) / kStep : 0;
    const int sink = P.window ? min(min(first, end), (int)(((int64_t)P.sinks + kStep - 1) / kStep)) : 0;
    const int steps = sink + max(0, end - first);

    u32x4 q[KS];
    {
        const uint16_t *row = P.q + (size_t)(live ? token : 0) * P.q_stride + (size_t)qh * D + 8 * h;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            q[s] = *reinterpret_cast<const u32x4 *>(row + 16 * s);
    }
    const float c = P.scale * kLog2e;
    const int shift = P.kv.page_shift, tshift = shift - 5;
    const int32_t *table = P.s.pages + (size_t)b * P.s.max_pages;

    float m = -INFINITY, l = 0.0f;
    float16v o[DB] = {};

    for (int st = 0; st < steps; ++st) {
        const int step = st < sink ? st : first + st - sink;
        bool here[2];
        size_t base[2], at[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int tt = 2 * step + u;
            const int id = tt * kTile < end_tok ? table[tt >> tshift] : -1;
            here[u] = id >= 0 && id < P.kv.n_pages;
            base[u] = (size_t)(here[u] ? id : 0) * P.kv.Hkv + kvh;
            at[u] = (size_t)(tt & ((1 << tshift) - 1)) * kTile;
        }
        __syncthreads();  // the last step's operands have been read
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const size_t tile = (base[u] << shift) * D + at[u] * D;
            constexpr int kHalf = C::kBytes / 2;
            if constexpr (C8) {
                const char *k = static_cast<const char *>(P.kv.k) + tile;
                const char *v = static_cast<const char *>(P.kv.v) + tile;
                for (int i = tid; i < kTile * D / 16; i += kWaves * kWave) {
                    // 16 columns of one token: chunks 2 c and 2 c + 1
                    const u32x4 w = *reinterpret_cast<const u32x4 *>(k + i * 16);
                    const int a = i / D, ch = i % D / 16, t = i % 16;
                    char *to = k_lds + u * kHalf + a * 16 * D * 2 + (ch * 2 * 16 + t) * 16;
                    *reinterpret_cast<u32x4 *>(to) = from_e4m3x8<QT>(w[0], w[1]);
                    *reinterpret_cast<u32x4 *>(to + 256) = from_e4m3x8<QT>(w[2], w[3]);
                    const u32x4 x = *reinterpret_cast<const u32x4 *>(v + i * 16);
                    char *tv = v_lds + u * kHalf + i * 32;
                    *reinterpret_cast<u32x4 *>(tv) = from_e4m3x8<VT>(x[0], x[1]);
                    *reinterpret_cast<u32x4 *>(tv + 16) = from_e4m3x8<VT>(x[2], x[3]);
                }
                if (tid < kTile) {
                    const size_t sc = (base[u] << shift) + at[u] + tid;
                    ks_lds[u * kTile + tid] = P.kv.ks[sc];
                    vs_lds[u * kTile + tid] = P.kv.vs[sc];
                }
            } else {
                const char *k = static_cast<const char *>(P.kv.k) + tile * 2;
                const char *v = static_cast<const char *>(P.kv.v) + tile * 2;
                for (int i = tid; i < kTile * D / 8; i += kWaves * kWave) {
                    *reinterpret_cast<u32x4 *>(k_lds + u * kHalf + i * 16) = *reinterpret_cast<const u32x4 *>(k + i * 16);
                    *reinterpret_cast<u32x4 *>(v_lds + u * kHalf + i * 16) = *reinterpret_cast<const u32x4 *>(v + i * 16);
                }
            }
        }
        __syncthreads();
        const int tok0 = step * kStep, last = tok0 + kStep - 1;
        if (tok0 > wave_hi)
            continue;
        const bool whole = here[0] && here[1] && last <= wave_lo && last < end_tok &&
                           (!P.window || wave_hi - tok0 < P.window || last < P.sinks);
        float16v s[2];
        const int key_row = ((col >> 3) & 1) * 16 * D * 2 + ((col >> 4) * 8 + (col & 7)) * 16;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            s[u] = float16v{};
#pragma unroll
            for (int j = 0; j < KS; ++j)
                s[u] = mfma32(QT, lds16(k_lds, u * (C::kBytes / 2) + key_row + (2 * j + h) * 256), q[j], s[u]);
        }
        // score 16 u + 8 t + 4 a + b: token 32 u + 16 a + 8 t + 4 h + b
        auto token_at = [&](int i) { return i / 16 * 32 + i % 8 / 4 * 16 + i % 16 / 8 * 8 + 4 * h + i % 4; };
        uint32_t seen = 0xFFFFFFFFu;
        if (!whole) {
            seen = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int tok = tok0 + token_at(i);
                const bool in = here[i / 16] && tok < end_tok && tok <= pos &&
                                (!P.window || pos - tok < P.window || tok < P.sinks);
                seen |= in ? 1u << i : 0u;
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            float x = s[i / 16][i % 16] * c;
            if constexpr (C8)
                x *= ks_lds[token_at(i)];
            if (!whole && !(seen >> i & 1))
                x = -INFINITY;
            s[i / 16][i % 16] = x;
            top = fmaxf(top, x);
        }
        top = fmaxf(top, __shfl_xor(top, 32, kWave));
        if (__any(top > m)) {
            const float to = fmaxf(m, top);
            const float f = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - to);
            m = to;
            l *= f;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    o[d][j] *= f;
        }
        const float zero = m == -INFINITY ? 0.0f : m;
        u32x4 p[4], p2[C::kTwo ? 4 : 1];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = 2 * i + e;
                y[e] = __builtin_amdgcn_exp2f(s[n / 16][n % 16] - zero);
                l += y[e];
                if constexpr (C8) {
                    y[e] *= vs_lds[token_at(n)];
                    if (!whole && !(seen >> n & 1))
                        y[e] = 0.0f;  // whatever scale lies there
                }
            }
            const uint32_t w = pack2<VT>(y[0], y[1]);
            p[i / 4][i % 4] = w;
            if constexpr (C::kTwo)
                p2[i / 4][i % 4] = pack2<VT>(y[0] - low16<VT>(w), y[1] - high16<VT>(w));
        }
        const int value_at = (h * D + col) * 16;
        bool bad = false;
        if (!whole) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int d = 0; d < DB; ++d)
                    bad |= not_finite<VT>(lds16(v_lds, value_at + (2 * j * D + 32 * d) * 16));
            bad = __any(bad);
        }
        if (!bad) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    const u32x4 v = lds16(v_lds, value_at + (2 * j * D + 32 * d) * 16);
                    o[d] = mfma32(VT, v, p[j], o[d]);
                    if constexpr (C::kTwo)
                        o[d] = mfma32(VT, v, p2[j], o[d]);
                }
        } else {
            // A value that is not finite reaches the rows that see it and no others: the
            // product takes 0 for it, and counts of such values that a row sees say
            // which of its sums become infinite.
            u32x4 ones[4];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                ones[i / 4][i % 4] = (seen >> (2 * i) & 1 ? (VT == APMOE_F16 ? 0x3C00u : 0x3F80u) : 0u) |
                                     (seen >> (2 * i + 1) & 1 ? (VT == APMOE_F16 ? 0x3C000000u : 0x3F800000u) : 0u);
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                float16v plus = {}, minus = {};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u32x4 v = lds16(v_lds, value_at + (2 * j * D + 32 * d) * 16), a, z;
                    split_values<VT>(v, a, z);
                    o[d] = mfma32(VT, v, p[j], o[d]);
                    if constexpr (C::kTwo)
                        o[d] = mfma32(VT, v, p2[j], o[d]);
                    plus = mfma32(VT, a, ones[j], plus);
                    minus = mfma32(VT, z, ones[j], minus);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    o[d][j] += plus[j] > 0.0f ? INFINITY : 0.0f;
                    o[d][j] += minus[j] > 0.0f ? -INFINITY : 0.0f;
                }
            }
        }
    }
    l += __shfl_xor(l, 32, kWave);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // nothing seen: zeros
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int j = 0; j < 16; ++j)
            o[d][j] *= inv;
    // column 32 d + 8 (j / 4) + 4 h + j % 4 of the row
    const size_t row = (size_t)token * P.Hq + qh;
    constexpr int kGroups = D < kBlk ? 1 : D / kBlk;
    if (D >= kBlk && P.out8) {
#pragma unroll
        for (int n = 0; n < kGroups; ++n) {
            uint32_t a = 0;
#pragma unroll
            for (int d = 0; d < DB / kGroups; ++d)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    a = max(a, mag(o[n * (DB / kGroups) + d][j]));
            a = max(a, (uint32_t)__shfl_xor((int)a, 32, kWave));
            const float sc = scale_of(a), r8 = 1.0f / sc;
            if (live && h == 0)
                P.out_scale[row * kGroups + n] = sc;
            if (live)
#pragma unroll
                for (int d = 0; d < DB / kGroups; ++d)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float16v &x = o[n * (DB / kGroups) + d];
                        *reinterpret_cast<uint32_t *>(P.out8 + row * D + 128 * n + 32 * d + 8 * j + 4 * h) = to_e4m3x4(
                            x[4 * j] * r8, x[4 * j + 1] * r8, x[4 * j + 2] * r8, x[4 * j + 3] * r8);
                    }
        }
    }
    if (live && P.out)
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<u32x2 *>(P.out + row * D + 32 * d + 8 * j + 4 * h) =
                    u32x2{pack2<QT>(o[d][4 * j], o[d][4 * j + 1]), pack2<QT>(o[d][4 * j + 2], o[d][4 * j + 3])};
}

template <int QT, bool C8, int D>
hipError_t prefill_launch(const AttnParams &P, hipStream_t s)
{
    const int G = P.Hq / P.kv.Hkv;
    // each sequence's last tile may be smaller
    const int64_t all = (int64_t)P.s.T * G, most = all / kRows + P.s.B;
    const uint32_t tiles = (uint32_t)(most < all ? most : all);
    hipLaunchKernelGGL((prefill_kernel<QT, C8, D>),
                       dim3(tiles < kGridX ? tiles : kGridX, P.kv.Hkv, (tiles + kGridX - 1) / kGridX),
                       dim3(kWaves * kWave), 0, s, P);
    return hipGetLastError();
}

template <int QT, bool C8>
hipError_t prefill_dim(const AttnParams &P, hipStream_t s)
{
    if (P.kv.D == 64)
        return prefill_launch<QT, C8, 64>(P, s);
    if (P.kv.D == 128)
        return prefill_launch<QT, C8, 128>(P, s);
    return prefill_launch<QT, C8, 256>(P, s);
}

}  // namespace

hipError_t launch_attn_prefill(const AttnParams &P, hipStream_t s)
{
    if (P.dtype == APMOE_F16)
        return P.kv.c8 ? prefill_dim<APMOE_F16, true>(P, s) : prefill_dim<APMOE_F16, false>(P, s);
    return P.kv.c8 ? prefill_dim<APMOE_BF16, true>(P, s) : prefill_dim<APMOE_BF16, false>(P, s);
}

}  // namespace apmoe
