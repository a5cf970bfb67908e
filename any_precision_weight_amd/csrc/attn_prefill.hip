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
constexpr float kSlack = 8.0f;
constexpr int kAhead = 4;  // operands read ahead of their product

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

// Copies between global memory and LDS of one step: the cache's bytes go there without
// passing registers; an 8-bit cache's pass through them to become 16-bit operands.
template <int QT, bool C8, int D>
struct Stage {
    using C = Prefill<QT, C8, D>;
    static constexpr int kThreads = kWaves * kWave;
    static constexpr int kPieces = kTile * D / 16 / kThreads > 0 ? kTile * D / 16 / kThreads : 1;  // 16 e4m3 bytes each
    const KvView &kv;
    int tid, wave, kvh;
    int ids[2];
    // a step's two V tiles of 32 tokens: their pages' bases and places
    bool here[2];
    size_t base[2], at[2];
    u32x4 k8[C8 ? 2 * kPieces : 1], v8[C8 ? 2 * kPieces : 1];
    float sc[2];

    // Lane i gets the pages of the i-th of 64 steps from st on.
    template <class StepOf>
    __device__ inline void load_ids(const int32_t *table, int st, int steps, const StepOf &step_of, int end_tok)
    {
        const int mine = st + tid % kWave;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int tt = 2 * step_of(mine) + u;
            ids[u] = mine < steps && tt * kTile < end_tok ? table[tt >> (kv.page_shift - 5)] : -1;
        }
    }
    __device__ inline void locate(int st, int step)
    {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int id = __builtin_amdgcn_readlane(ids[u], st % kWave);
            here[u] = id >= 0 && id < kv.n_pages;
            base[u] = (size_t)(here[u] ? id : 0) * kv.Hkv + kvh;
            at[u] = (size_t)((2 * step + u) & ((1 << (kv.page_shift - 5)) - 1)) * kTile;
        }
    }
    // Sends the requests of the located step; `to` is its buffer.
    __device__ inline void fetch(char *to)
    {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const size_t tile = (base[u] << kv.page_shift) * D + at[u] * D;
            if constexpr (C8) {
                const char *k = static_cast<const char *>(kv.k) + tile, *v = static_cast<const char *>(kv.v) + tile;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int piece = tid + i * kThreads;
                    if (kTile * D / 16 >= kThreads || piece < kTile * D / 16) {
                        k8[u * kPieces + i] = *reinterpret_cast<const u32x4 *>(k + piece * 16);
                        v8[u * kPieces + i] = *reinterpret_cast<const u32x4 *>(v + piece * 16);
                    }
                }
                if (tid < 2 * kTile)
                    sc[u] = (tid < kTile ? kv.ks : kv.vs)[(base[u] << kv.page_shift) + at[u] + tid % kTile];
            } else {
                const char *k = static_cast<const char *>(kv.k) + tile * 2, *v = static_cast<const char *>(kv.v) + tile * 2;
#pragma unroll
                for (int i = 0; i < kTile * D / 8 / kThreads; ++i) {
                    const int off = (i * kWaves + wave) * 1024;
                    char *dst = to + u * (C::kBytes / 2) + off;
                    __builtin_amdgcn_global_load_lds(
                        (const __attribute__((address_space(1))) void *)(uintptr_t)(k + off + tid % kWave * 16),
                        (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
                    __builtin_amdgcn_global_load_lds(
                        (const __attribute__((address_space(1))) void *)(uintptr_t)(v + off + tid % kWave * 16),
                        (__attribute__((address_space(3))) void *)(dst + C::kBytes), 16, 0, 0);
                }
            }
        }
    }
    // Writes what fetch left in registers.
    __device__ inline void put(char *to) const
    {
        if constexpr (C8) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int piece = tid + i * kThreads;
                    if (kTile * D / 16 < kThreads && piece >= kTile * D / 16)
                        continue;
                    // 16 columns of one token: chunks 2 c and 2 c + 1 of its row
                    const int a = piece / D, ch = piece % D / 16, t = piece % 16;
                    char *tk = to + u * (C::kBytes / 2) + a * 16 * D * 2 + (ch * 2 * 16 + t) * 16;
                    const u32x4 &w = k8[u * kPieces + i], &x = v8[u * kPieces + i];
                    *reinterpret_cast<u32x4 *>(tk) = from_e4m3x8<QT>(w[0], w[1]);
                    *reinterpret_cast<u32x4 *>(tk + 256) = from_e4m3x8<QT>(w[2], w[3]);
                    char *tv = to + C::kBytes + u * (C::kBytes / 2) + piece * 32;
                    *reinterpret_cast<u32x4 *>(tv) = from_e4m3x8<C::kVT>(x[0], x[1]);
                    *reinterpret_cast<u32x4 *>(tv + 16) = from_e4m3x8<C::kVT>(x[2], x[3]);
                }
                if (tid < 2 * kTile)
                    reinterpret_cast<float *>(to + 2 * C::kBytes)[tid / kTile * kStep + u * kTile + tid % kTile] = sc[u];
            }
        }
    }
};

// The larger of x here and in the lane with the other half of the same column.
__device__ inline float both_halves_max(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false,
                                                    false);
    const uint32_t lo = r[0], hi = r[1];  // a bit cast of a vector's element reads element 0
    return fmaxf(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
}

template <int QT, bool C8, int D>
__global__ void __launch_bounds__(kWaves *kWave, D <= 128 ? 2 : 1) prefill_kernel(const AttnParams P)
{
    using C = Prefill<QT, C8, D>;
    constexpr int VT = C::kVT, KS = D / 16, DB = D / 32;
    __shared__ __attribute__((aligned(16))) char lds[2 * C::kLds];

    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    // heads are neighbours in the grid: workgroups b with the same b % 8 run on one XCD, and
    // with 8 heads each XCD's L2 then has one head's keys and values
    const uint32_t block = blockIdx.y * kGridX + blockIdx.x;
    const int G = P.Hq / P.kv.Hkv, kvh = (int)(block % (uint32_t)P.kv.Hkv);
    int b, rt, n_rt;
    if (!find_item(P.s.B, (int)(block / (uint32_t)P.kv.Hkv), [&](int i) {
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
    auto step_of = [&](int st) { return st < sink ? st : first + st - sink; };

    // a negative scale is the queries' sign, and 0 a number too small to matter: c > 0 keeps
    // the order of the scores, so the maximum is that of the unscaled ones
    u32x4 q[KS];
    {
        const uint16_t *row = P.q + (size_t)(live ? token : 0) * P.q_stride + (size_t)qh * D + 8 * h;
        const uint32_t sign = P.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            q[s] = *reinterpret_cast<const u32x4 *>(row + 16 * s) ^ sign;
    }
    const float c = fmaxf(__builtin_fabsf(P.scale) * kLog2e, 0x1p-126f);
    const int32_t *table = P.s.pages + (size_t)b * P.s.max_pages;

    float m = -INFINITY, l = 0.0f;
    float16v o[DB] = {};

    Stage<QT, C8, D> stage{P.kv, tid, wave, kvh};
    if (steps > 0) {
        stage.load_ids(table, 0, steps, step_of, end_tok);
        stage.locate(0, step_of(0));
        stage.fetch(lds);
        stage.put(lds);
    }
    const int key_at = ((col >> 3) & 1) * 16 * D * 2 + ((col >> 4) * 8 + (col & 7)) * 16 + h * 256;
    const int value_at = (h * D + col) * 16;
    // score 16 u + 8 t + 4 a + b: token 32 u + 16 a + 8 t + 4 h + b
    auto token_at = [&](int i) { return i / 16 * 32 + i % 8 / 4 * 16 + i % 16 / 8 * 8 + 4 * h + i % 4; };
    const char *k_lds = nullptr, *v_lds = nullptr;
    bool here[2];
    int tok0 = 0;

    // Step st's operands are in LDS after this, and the next ones on their way.
    auto open = [&](int st) {
        k_lds = lds + st % 2 * C::kLds;
        v_lds = k_lds + C::kBytes;
        tok0 = step_of(st) * kStep;
        here[0] = stage.here[0];
        here[1] = stage.here[1];
        // this step's copies have landed, everyone's, and the other buffer has been read
        __builtin_amdgcn_s_waitcnt(wait_vm<0>());
        __syncthreads();
        if (st + 1 < steps) {
            if ((st + 1) % kWave == 0)
                stage.load_ids(table, st + 1, steps, step_of, end_tok);
            stage.locate(st + 1, step_of(st + 1));
            stage.fetch(lds + (st + 1) % 2 * C::kLds);
        }
    };
    // whether rows at positions lo .. hi all see the whole step
    auto whole_for = [&](int lo, int hi) {
        const int last = tok0 + kStep - 1;
        return here[0] && here[1] && last <= lo && last < end_tok &&
               (!P.window || hi - tok0 < P.window || last < P.sinks);
    };
    auto body = [&](auto slow_) {
        constexpr bool kSlow = decltype(slow_)::value;
        float16v s[2] = {};
        {
            auto key = [&](int n) { return lds16(k_lds, n % 2 * (C::kBytes / 2) + key_at + n / 2 * 512); };
            u32x4 ring[kAhead];
#pragma unroll
            for (int n = 0; n < kAhead; ++n)
                ring[n] = key(n);
#pragma unroll
            for (int n = 0; n < 2 * KS; ++n) {
                s[n % 2] = mfma32(QT, ring[n % kAhead], q[n / 2], s[n % 2]);
                if (n + kAhead < 2 * KS)
                    ring[n % kAhead] = key(n + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        const float *const ks_lds = reinterpret_cast<const float *>(k_lds + 2 * C::kBytes), *const vs_lds = ks_lds + kStep;
        if constexpr (C8)
#pragma unroll
            for (int i = 0; i < 32; ++i)
                s[i / 16][i % 16] *= ks_lds[token_at(i)];
        const bool whole = whole_for(wave_lo, wave_hi);
        uint32_t seen = 0xFFFFFFFFu;
        if (!whole) {
            seen = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int tok = tok0 + token_at(i);
                const bool in = here[i / 16] && tok < end_tok && tok <= pos &&
                                (!P.window || pos - tok < P.window || tok < P.sinks);
                seen |= in ? 1u << i : 0u;
                s[i / 16][i % 16] = in ? s[i / 16][i % 16] : -INFINITY;
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            top = fmaxf(top, s[i / 16][i % 16]);
        top = both_halves_max(top) * c;
        // The sums are taken to a new maximum only when it is 2^8 times the old one's:
        // probabilities up to 2^8 are as exact, and the sums have room.
        if (__any(top > m + kSlack)) {
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
        const float zero = m == -INFINITY ? 0.0f : -m;
        // Word i of the probabilities: scores 2 i and 2 i + 1; four words are an operand.
        uint32_t p[2][4], p2[2][4];
        auto word = [&](int i) {
            float y[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = 2 * i + e;
                y[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n / 16][n % 16], c, zero));
                l += y[e];
                if constexpr (C8) {
                    y[e] *= vs_lds[token_at(n)];
                    if (!(seen >> n & 1))
                        y[e] = 0.0f;  // whatever scale lies there
                }
            }
            const uint32_t w = pack2<VT>(y[0], y[1]);
            p[i / 4 % 2][i % 4] = w;
            if constexpr (C::kTwo)
                p2[i / 4 % 2][i % 4] = pack2<VT>(y[0] - low16<VT>(w), y[1] - high16<VT>(w));
        };
        auto operand = [](const uint32_t(&w)[4]) { return u32x4{w[0], w[1], w[2], w[3]}; };
        auto value = [&](int n) { return lds16(v_lds, value_at + (n / DB * 2 * D + n % DB * 32) * 16); };
#pragma unroll
        for (int i = 0; i < 4; ++i)
            word(i);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!kSlow) {
            u32x4 ring[kAhead];
#pragma unroll
            for (int n = 0; n < kAhead; ++n)
                ring[n] = value(n);
#pragma unroll
            for (int n = 0; n < 4 * DB; ++n) {
                const int j = n / DB, d = n % DB;
                o[d] = mfma32(VT, ring[n % kAhead], operand(p[j % 2]), o[d]);
                if constexpr (C::kTwo)
                    o[d] = mfma32(VT, ring[n % kAhead], operand(p2[j % 2]), o[d]);
                if (n + kAhead < 4 * DB)
                    ring[n % kAhead] = value(n + kAhead);
                // the next operand's words in the products' time
                if (j < 3)
#pragma unroll
                    for (int i = 4 * d / DB; i < 4 * (d + 1) / DB; ++i)
                        word(4 * (j + 1) + i);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            // A value that is not finite reaches the rows that see it and no others: the
            // product takes 0 for it, and counts of such values that a row sees say which
            // of its sums become infinite.
            constexpr uint32_t kOne = VT == APMOE_F16 ? 0x3C00u : 0x3F80u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u32x4 ones;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ones[i] = (seen >> (8 * j + 2 * i) & 1 ? kOne : 0u) |
                              (seen >> (8 * j + 2 * i + 1) & 1 ? kOne << 16 : 0u);
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    u32x4 v = value(j * DB + d), plus, minus;
                    split_values<VT>(v, plus, minus);
                    o[d] = mfma32(VT, v, operand(p[j % 2]), o[d]);
                    if constexpr (C::kTwo)
                        o[d] = mfma32(VT, v, operand(p2[j % 2]), o[d]);
                    const float16v a = mfma32(VT, plus, ones, float16v{});
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[d][i] += a[i] > 0.0f ? INFINITY : 0.0f;
                    const float16v z = mfma32(VT, minus, ones, float16v{});
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[d][i] += z[i] > 0.0f ? -INFINITY : 0.0f;
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (j < 3)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        word(4 * (j + 1) + i);
            }
        }
    };
    auto close = [&](int st) {
        if (st + 1 < steps)
            stage.put(lds + (st + 1) % 2 * C::kLds);
    };

    int st = 0;
    for (; st < steps; ++st) {
        open(st);
        // Where not every row sees the whole step its values must be finite for the plain
        // product: NaN and infinities times 0 are NaN.
        if (!whole_for(lo, hi)) {
            bool bad = false;
            for (int i = tid; i < C::kBytes / 16; i += kWaves * kWave)
                bad |= not_finite<VT>(lds16(v_lds, i * 16));
            if (__syncthreads_or(bad))
                break;
        }
        if (tok0 <= wave_hi)
            body(std::false_type{});
        close(st);
    }
    for (bool opened = true; st < steps; ++st) {
        if (!opened)
            open(st);
        opened = false;
        if (tok0 <= wave_hi)
            body(std::true_type{});
        close(st);
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
    const int64_t blocks = (most < all ? most : all) * P.kv.Hkv;  // below 2^35 / kRows
    hipLaunchKernelGGL((prefill_kernel<QT, C8, D>),
                       dim3((uint32_t)(blocks < kGridX ? blocks : kGridX), (uint32_t)((blocks + kGridX - 1) / kGridX)),
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
