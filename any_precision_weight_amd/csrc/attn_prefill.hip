// attn_prefill.hip -- causal attention of the new tokens of prompts (or of their chunks) over
// the paged cache, with a sliding window and first tokens that stay visible.
//
// The formulas are attn_decode.hip's.  A row is a (new token, query head) pair; the heads of a
// key-value head's group are neighbours, so a workgroup's 128 rows share their keys and
// values whatever the group's size.  Four waves have 32 rows each and walk over 64 cached
// tokens a step, staged in LDS in the cache's own order (two buffers each of keys and values,
// sent for a step ahead): the operands of the 32 x 32 products are 16-byte reads of
// neighbouring places, without bank conflicts.
//
// A step is the products of the next scores with this step's exponentials between them, then
// the second products with the next maximum between them: a wave's vector instructions run in
// its own matrix instructions' time (5 of them beside each with the exponential, by the
// counters, where one of two waves a SIMD has room for about 6), and two workgroups a CU cover
// each other's barriers.
//
// 8192 tokens, 32 heads over 8 of 128 in bf16 take 511 to 535 us, 1.03 to 1.08 PFLOP/s; 6000 tokens
// of each of three sequences behind up to 14000, with a window, 3.1 to 3.3 ms, 1.03 to 1.09 (a large
// library product reaches 1.50 here).  In the counters' runs the matrix units are busy for 60 and
// 62% of the CUs' cycles, at 1.55 and 1.7 GHz, and waves stand at a wait or a barrier for 30%
// of theirs: neither the units alone nor the clock alone is the bound.  Before the softmax was
// interleaved with the products it took 571 us.  Heads of 64 take 327 to 348 us for two prompts of
// 6000 (0.85 to 0.90; a step's 32 exponentials a lane, at a quarter of the rate, take as long as
// its 16 products), of 256 (one wave a SIMD) 528 to 549 us for two of 5000 of 16 heads (0.75 to
// 0.78); an 8-bit cache, converted on its way into LDS for each row tile, 675 to 695 us for the
// first (0.79 to 0.81), 68 bytes of scratch a lane, and with fp16 queries 950 (0.58), 116 bytes.  64
// rows a wave (half the reads from LDS, one wave a SIMD) took 654 us for it.
//
// Probabilities go into the second product as one 16-bit number (2^-8 of each in bf16), where
// decode gives two: a second number would be half as many matrix instructions again.  The
// output's error against 64 bits in norm is 0.0018 for 8192 tokens; its own rounding alone is 0.0017.
//
// Rows of a key operand: row 16 t + 8 a + 4 h + b of a 32-token product is token 16 a + 8 t +
// 4 h + b.  Lane half h then has, of scores 8t .. 8t+7, the tokens of granule g = 2 t + h of
// V (attn.h), and the probabilities need not move.
#include <algorithm>

#include "attn.h"

namespace apmoe {
namespace {

constexpr int kWaves = 4;
constexpr int kRows = 32 * kWaves;  // rows of a workgroup
static_assert(kRows == kPartRows, "rows of a part");
constexpr int kStep = 64;           // cached tokens of a step
constexpr uint32_t kGridX = 1u << 22;
constexpr float kSlack = 8.0f;
constexpr float kFar = 0x1p10f;
// Calls of few row tiles are split over the steps: up to kSplitBlocks workgroups (of 256 CUs
// that hold two) into parts of kPartSteps steps or more.  512 new tokens behind 32256, 32 heads
// over 8: 796 -> 301 us, 4 of each of 16 sequences of 2700 to 8000 252 -> 93, 64 behind 4000
// 93 -> 29; of 4 steps 316, 96 and 33, of 16 287, 93 and 37.  Not with more workgroups, by
// one case of about 31 steps: 1000 behind 1000, 256 of them, 44.5 us and split in two 51.  Larger
// calls of many steps have not been measured split; unsplit, 4 new tokens of each of 32 and 64
// sequences of 2000 to 8000 take 210 and 269 us.
constexpr int kPartSteps = 8;
constexpr int kSplitBlocks = 192;
constexpr int kMaxParts = 64;

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
    static constexpr float kFirst = kTop<kVT> - kSlack;  // exponent of a maximum (attn.h)
    static constexpr int kBytes = kStep * D * 2;  // of a step's keys, and of its values
    static constexpr int kAhead = D == 64 || C8 ? 3 : 4;  // operands read ahead of their product (registers)
    static constexpr int kBuffer = kBytes + (C8 ? kStep * 4 : 0);  // with their scales
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

// Copies between global memory and LDS: the cache's bytes go there without passing
// registers; an 8-bit cache's pass through them to become 16-bit operands.
template <int QT, bool C8, int D>
struct Stage {
    using C = Prefill<QT, C8, D>;
    static constexpr int kThreads = kWaves * kWave;
    static constexpr int kTileBytes = kTile * D * (C8 ? 1 : 2);  // of 32 tokens' keys in the cache
    static constexpr int kPieces = (kTileBytes / 16 + kThreads - 1) / kThreads;
    static constexpr bool kAll = kTileBytes / 16 % kThreads == 0;
    const KvView &kv;
    int tid, wave, kvh;
    // Lane i has the places of the two tiles of 32 tokens of step base + i, in tokens of all
    // heads; bit i of on[u]: tile u is on a page.
    int base;
    uint32_t lo[2], hi[2];
    uint64_t on[2];
    u32x4 held[C8 ? 2 * kPieces : 1];  // what fetch asked for last, of keys or of values
    float held_scale;

    // The steps from st on; `step` is the lane's own.
    __device__ inline void load_places(const int32_t *table, int st, int step, bool in, int end_tok)
    {
        base = st;
        bool ok[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int tt = 2 * step + u, tshift = kv.page_shift - 5;
            const int id = in && tt * kTile < end_tok ? table[tt >> tshift] : -1;
            ok[u] = id >= 0 && id < kv.n_pages;
            const size_t page = (size_t)(ok[u] ? id : 0) * kv.Hkv + kvh;
            const size_t at = (page << kv.page_shift) + (size_t)(tt & ((1 << tshift) - 1)) * kTile;
            lo[u] = (uint32_t)at;
            hi[u] = (uint32_t)(at >> 32);
        }
        on[0] = __ballot(ok[0]);
        on[1] = __ballot(ok[1]);
    }
    __device__ inline bool here(int st, int u) const { return on[u] >> (st - base) & 1; }
    __device__ inline bool here(int st) const { return (on[0] & on[1]) >> (st - base) & 1; }
    __device__ inline bool knows(int st) const { return st - base < kWave; }
    __device__ inline size_t place(int st, int u) const
    {
        return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)hi[u], st - base) << 32 |
               (uint32_t)__builtin_amdgcn_readlane((int)lo[u], st - base);
    }
    // Sends the requests for the keys (or values) at these places to buffer `to`.
    template <bool V>
    __device__ inline void fetch(const size_t (&at)[2], char *to)
    {
        const char *const src = static_cast<const char *>(V ? kv.v : kv.k);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const char *const p = src + at[u] * (D * (C8 ? 1 : 2));
            if constexpr (C8) {
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
                    if (kAll || tid + i * kThreads < kTileBytes / 16)
                        held[u * kPieces + i] = *reinterpret_cast<const u32x4 *>(p + (tid + i * kThreads) * 16);
                if (tid / kTile == u)
                    held_scale = (V ? kv.vs : kv.ks)[at[u] + tid % kTile];
            } else {
                constexpr int kMine = kTileBytes / kWaves;  // bytes of a wave
                const __amdgpu_buffer_rsrc_t r = make_rsrc(p, kTileBytes);
                char *const dst = to + u * (C::kBytes / 2) + wave * kMine;
#pragma unroll
                for (int i = 0; i < kMine / 1024; ++i)
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)(dst + i * 1024),
                                                             16, wave * kMine + tid % kWave * 16, i * 1024, 0, 0);
            }
        }
    }
    // Writes what fetch left in registers.
    template <bool V>
    __device__ inline void put(char *to) const
    {
        if constexpr (C8) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int piece = tid + i * kThreads;
                    if (!kAll && piece >= kTileBytes / 16)
                        continue;
                    const u32x4 &w = held[u * kPieces + i];
                    char *t = to + u * (C::kBytes / 2);
                    if constexpr (V) {
                        *reinterpret_cast<u32x4 *>(t + piece * 32) = from_e4m3x8<C::kVT>(w[0], w[1]);
                        *reinterpret_cast<u32x4 *>(t + piece * 32 + 16) = from_e4m3x8<C::kVT>(w[2], w[3]);
                    } else {
                        // 16 columns of one token: chunks 2 c and 2 c + 1 of its row
                        t += piece / D * 16 * D * 2 + (piece % D / 16 * 2 * 16 + piece % 16) * 16;
                        *reinterpret_cast<u32x4 *>(t) = from_e4m3x8<QT>(w[0], w[1]);
                        *reinterpret_cast<u32x4 *>(t + 256) = from_e4m3x8<QT>(w[2], w[3]);
                    }
                }
            if (tid < kStep)
                reinterpret_cast<float *>(to + C::kBytes)[tid] = held_scale;
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

// Rows of a workgroup and the steps that they see.  Row i is query head (row0 + i) % G of new
// token q0 + (row0 + i) / G of sequence b; rows past the last one stand for it.
struct RowTile {
    int b, len, nq, row_of_b, end_tok, q0, row0, last_row, lo, hi;
    int first, sink, steps;  // [0, sink) and [first, first + steps - sink)
    int parts, per;          // parts of `per` steps
    int G;

    __device__ inline int token(int i) const { return q0 + (int)((uint32_t)(row0 + i) / (uint32_t)G); }
    __device__ inline int pos(int i) const { return len - nq + token(min(i, last_row)); }
    __device__ inline int step(int st) const { return st < sink ? st : first + st - sink; }
};

__device__ inline bool row_tile(const AttnParams &P, uint32_t tile, RowTile &t)
{
    const int G = P.Hq / P.kv.Hkv;
    int rt, n_rt;
    if (!find_item(P.s.B, (int)tile, [&](int i) {
            return (int)(((int64_t)new_tokens(P.s, i) * G + kRows - 1) / kRows);
        }, t.b, rt, n_rt))
        return false;
    rt = n_rt - 1 - rt;  // the rows with the most to see first
    t.G = G;
    t.nq = new_tokens(P.s, t.b);
    t.row_of_b = P.s.q_offsets ? P.s.q_offsets[t.b] : t.b;
    t.len = P.s.lens[t.b];
    t.end_tok = cached_tokens(P.s, t.len);
    const int64_t r0 = (int64_t)rt * kRows;
    t.q0 = (int)(r0 / G);
    t.row0 = (int)(r0 - (int64_t)t.q0 * G);
    t.last_row = (int)min((int64_t)kRows, (int64_t)t.nq * G - r0) - 1;
    t.lo = t.pos(0);
    t.hi = t.pos(kRows - 1);
    const int end = (max(0, min(t.end_tok, t.hi + 1)) + kStep - 1) / kStep;
    t.first = P.window ? max(0, t.lo - P.window + 1) / kStep : 0;
    t.sink = P.window ? min(min(t.first, end), (int)(((int64_t)P.sinks + kStep - 1) / kStep)) : 0;
    t.steps = t.sink + max(0, end - t.first);
    const int most = min(P.parts, max(1, t.steps / kPartSteps));
    t.per = (t.steps + most - 1) / most;
    t.parts = t.steps > 0 ? (t.steps + t.per - 1) / t.per : 1;
    return true;
}

// 4 columns from d on of a row, with the scale of their group of 128.
template <int QT>
__device__ inline void store_columns(const AttnParams &P, size_t row, int d, const float (&v)[4], float scale)
{
    const size_t at = row * P.kv.D + d;
    if (P.out8) {
        const float r = 1.0f / scale;
        *reinterpret_cast<uint32_t *>(P.out8 + at) = to_e4m3x4(v[0] * r, v[1] * r, v[2] * r, v[3] * r);
    }
    if (P.out)
        *reinterpret_cast<u32x2 *>(P.out + at) = u32x2{pack2<QT>(v[0], v[1]), pack2<QT>(v[2], v[3])};
}

template <int QT, bool C8, int D>
__global__ void __launch_bounds__(kWaves *kWave, D == 64 && !C8 ? 3 : D <= 128 ? 2 : 1) prefill_kernel(const AttnParams P)
{
    using C = Prefill<QT, C8, D>;
    constexpr int VT = C::kVT, KS = D / 16, DB = D / 32;
    __shared__ __attribute__((aligned(16))) char lds[4 * C::kBuffer];
    auto k_buf = [&](int st) { return lds + st % 2 * C::kBuffer; };
    auto v_buf = [&](int st) { return lds + (2 + st % 2) * C::kBuffer; };

    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    // heads are neighbours in the grid: workgroups b with the same b % 8 run on one XCD, and
    // with 8 heads each XCD's L2 then has one head's keys and values
    const uint32_t block = blockIdx.y * kGridX + blockIdx.x, item = block / (uint32_t)P.kv.Hkv;
    const int kvh = (int)(block - item * (uint32_t)P.kv.Hkv), part = (int)(item % (uint32_t)P.parts);
    RowTile t;
    if (!row_tile(P, item / (uint32_t)P.parts, t) || part >= t.parts)
        return;
    const int end_tok = t.end_tok;

    // this lane's row (as a column of the products), and the positions of its wave's
    const int col = lane % 32, h = lane / 32;
    const int mine = wave * 32 + col, last = min(mine, t.last_row), qi = t.token(last);
    const int qh = kvh * t.G + t.row0 + last - (qi - t.q0) * t.G;
    const int64_t token = (int64_t)t.row_of_b + qi;
    const int pos = t.len - t.nq + qi;
    const bool live = mine <= t.last_row && token >= 0 && token < P.s.T;
    const int wave_lo = t.pos(wave * 32), wave_hi = t.pos(wave * 32 + 31);

    // the part's steps, counted from its first one
    const int st0 = part * t.per, steps = min(t.steps - st0, t.per);
    auto step_of = [&](int st) { return t.step(st0 + st); };

    u32x4 q[KS];
    {
        const uint16_t *row = P.q + (size_t)(live ? token : 0) * P.q_stride + (size_t)qh * D + 8 * h;
#pragma unroll
        for (int s = 0; s < KS; ++s)
            q[s] = *reinterpret_cast<const u32x4 *>(row + 16 * s) ^ query_sign(P.scale);
    }
    const float c = score_factor(P.scale), slack = uniform(kSlack / c);
    const int32_t *table = P.s.pages + (size_t)t.b * P.s.max_pages;

    float m, l, top;
    float16v o[DB], sa[2], sb[2];
    const int key_at = ((col >> 3) & 1) * 16 * D * 2 + ((col >> 4) * 8 + (col & 7)) * 16 + h * 256;
    const int value_at = (h * D + col) * 16;
    // score 16 u + 8 t + 4 a + b: token 32 u + 16 a + 8 t + 4 h + b
    auto token_at = [&](int i) { return i / 16 * 32 + i % 8 / 4 * 16 + i % 16 / 8 * 8 + 4 * h + i % 4; };
    auto key = [&](const char *k, int n) { return lds16(k, n % 2 * (C::kBytes / 2) + key_at + n / 2 * 512); };

    Stage<QT, C8, D> stage{P.kv, tid, wave, kvh};
    auto load_places = [&](int st) __attribute__((always_inline)) {
        stage.load_places(table, st, step_of(st + lane), st + lane < steps, end_tok);
    };
    auto turn = [] {  // copies have landed, everyone's, and what they replace next has been read
        __builtin_amdgcn_s_waitcnt(wait_vm<0>());
        __syncthreads();
    };
    // Scores of a step whose keys are in LDS; `between(n)` runs in the time of product n.
    auto scores = [&](float16v(&s)[2], const char *k, const auto &between) __attribute__((always_inline)) {
        u32x4 ring[C::kAhead];
#pragma unroll
        for (int n = 0; n < C::kAhead; ++n)
            ring[n] = key(k, n);
#pragma unroll
        for (int n = 0; n < 2 * KS; ++n) {
            s[n % 2] = mfma32(QT, ring[n % C::kAhead], q[n / 2], n < 2 ? float16v{} : s[n % 2]);
            if (n + C::kAhead < 2 * KS)
                ring[n % C::kAhead] = key(k, n + C::kAhead);
            between(n);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // An 8-bit cache's scales of scores 4 g .. 4 g + 3.
    auto scales = [&](const char *buffer, int g) {
        return *reinterpret_cast<const float4v *>(buffer + C::kBytes + token_at(4 * g) * 4);
    };
    auto top_of = [](const float16v(&s)[2]) __attribute__((always_inline)) {
        float t = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            t = fmaxf(t, s[i / 16][i % 16]);
        return t;
    };

    // Steps that every row of the wave (or of the workgroup) sees whole, if their pages are
    // there: those below `to`, from `from` on or below `sinks`.
    struct Whole {
        int to, from, sinks;
        __device__ inline bool operator()(int st) const { return (st < to) & ((st >= from) | (st < sinks)); }
    };
    auto whole_of = [&](int least, int most) {
        Whole w;
        const int gap = t.sink - t.first, past = max(0, min(least + 1, end_tok)) / kStep;
        w.to = past + gap;  // behind the sinks step = st - gap
        w.from = P.window ? max(t.sink, (max(0, most - P.window + 1) + kStep - 1) / kStep + gap) : 0;
        w.sinks = P.window ? min(min(P.sinks / kStep, t.sink), past) : 0;
        if (w.to < t.sink)  // rows that end among the sinks
            w.to = w.sinks;
        w.to -= st0;
        w.from -= st0;
        w.sinks -= st0;
        return w;
    };
    const Whole whole_wave = whole_of(wave_lo, wave_hi), whole_all = whole_of(t.lo, t.hi);
    // What the rows see of step st.  Score i is of the token tok0 + token_at(i) = tok0 + 4 h + a
    // number known here: seen if that number is below `below` and above `above` (the window)
    // or below `sink_below`.
    struct Sight {
        int below[2], above, sink_below;
    };
    auto sight_of = [&](int st) __attribute__((always_inline)) {
        Sight g;
        const int at = step_of(st) * kStep + 4 * h;
        const bool here0 = stage.here(st, 0), here1 = stage.here(st, 1);
        const int past = min(pos + 1, end_tok) - at;
        g.below[0] = here0 ? past : -1;
        g.below[1] = here1 ? past : -1;
        g.above = P.window ? pos - P.window - at : -kStep;
        g.sink_below = P.sinks - at;
        return g;
    };
    auto sees = [&](const Sight &g, int i) __attribute__((always_inline)) {
        const int n = token_at(i) - 4 * h;
        return (n < g.below[i / 16]) & ((n > g.above) | (n < g.sink_below));
    };
    auto mask = [&](const Sight &g, float16v(&s)[2]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            s[i / 16][i % 16] = sees(g, i) ? s[i / 16][i % 16] : -INFINITY;
        top = top_of(s);
    };
    // The sums are taken to a new maximum m only when a score passes `limit`, where its
    // probability would be 2^8: up to there they are as exact, and the sums have room.  An
    // exponent is then one operation, s c + zero with zero = kFirst - m c.  The rounding of m c is
    // part of it, and another one after each new maximum: 2^-15 at most below |m c| = 2^10, a
    // 16th of what fp16 rounds the probabilities by.  From there on (far; weights of e^710 and
    // more) m is taken from the scores before, and without slack: 3% of 8192 tokens' time.
    float limit, zero;
    bool far;
    auto rescale = [&](float16v(&s)[2]) __attribute__((always_inline)) {
        top = both_halves_max(top);
        if (__any(top > limit)) {
            const float to = fmaxf(m, top);
            const float f = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m - to) * c);
            m = to;
            const float mc = m == -INFINITY ? 0.0f : m * c;
            far = __any(__builtin_fabsf(mc) >= kFar);
            zero = far ? C::kFirst : C::kFirst - mc;
            limit = far || m == -INFINITY ? m : m + slack;
            l *= f;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    o[d][j] *= f;
        }
        if (far) {
            const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                s[i / 16][i % 16] -= base;
        }
    };
    // Word i of the probabilities: scores 2 i and 2 i + 1; four words are an operand.  vq: an
    // 8-bit cache's scales, those of the words after the next ones asked for here.
    uint32_t p[16], p2[C::kTwo ? 16 : 1];
    float4v vq[2];
    auto word = [&](const float16v(&s)[2], const char *v, int i) __attribute__((always_inline)) {
        float y[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int n = 2 * i + e;
            y[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n / 16][n % 16], c, zero));
            l += y[e];
            if constexpr (C8)  // 0 whatever the scale is, where nothing is seen
                y[e] = y[e] == 0.0f ? 0.0f : y[e] * vq[n / 4 % 2][n % 4];
        }
        if constexpr (C8)
            if (i % 2 == 1 && i < 13)
                vq[i / 2 % 2] = scales(v, i / 2 + 2);
        const uint32_t w = pack2<VT>(y[0], y[1]);
        p[i] = w;
        if constexpr (C::kTwo)
            p2[i] = pack2<VT>(y[0] - low16<VT>(w), y[1] - high16<VT>(w));
    };
    auto first_scales = [&](const char *v) __attribute__((always_inline)) {
        if constexpr (C8) {
            vq[0] = scales(v, 0);
            vq[1] = scales(v, 1);
        }
    };
    auto operand = [](const auto &w, int j) __attribute__((always_inline)) {
        return u32x4{w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]};
    };
    auto value = [&](const char *v, int n) { return lds16(v, value_at + (n / DB * 2 * D + n % DB * 32) * 16); };

    // Step st: its values and the next one's keys are in LDS after open, the values behind them
    // and the keys behind those on their way.  What passes registers is sent for and written
    // one after the other: the values in the first half of the step, the keys in the second.
    size_t at_k[2], at_v[2];  // of the keys and values sent for last
    auto more_keys = [&](int st) __attribute__((always_inline)) {
        if (st + 2 < steps) {
            if (!stage.knows(st + 2))
                load_places(st);
            at_k[0] = stage.place(st + 2, 0);
            at_k[1] = stage.place(st + 2, 1);
            stage.template fetch<false>(at_k, k_buf(st));
        }
    };
    auto open = [&](int st) __attribute__((always_inline)) {
        turn();
        at_v[0] = at_k[0];
        at_v[1] = at_k[1];
        if constexpr (!C8)
            more_keys(st);
        if (st + 1 < steps)
            stage.template fetch<true>(at_v, v_buf(st + 1));
    };
    auto half = [&](int st) __attribute__((always_inline)) {
        if constexpr (C8) {
            if (st + 1 < steps)
                stage.template put<true>(v_buf(st + 1));
            more_keys(st);
        }
    };
    auto close = [&](int st) __attribute__((always_inline)) {
        if (st + 2 < steps)
            stage.template put<false>(k_buf(st));
    };
    // One step: s has its scores, next gets those of the step behind it.
    auto body = [&](int st, float16v(&s)[2], float16v(&next)[2]) __attribute__((always_inline)) {
        const char *const v = v_buf(st), *const k = k_buf(st + 1);
        if (!(whole_wave(st) && stage.here(st)))
            mask(sight_of(st), s);
        rescale(s);
        first_scales(v);
        // the first 12 words in the time of the next scores, the last 4 and the next maximum
        // in that of the second product (the next scores of the last step are of keys that
        // have been read before: nothing is done with them)
        constexpr int kEarly = 12;
        scores(next, k, [&](int n) __attribute__((always_inline)) {
#pragma unroll
            for (int i = n * kEarly / (2 * KS); i < (n + 1) * kEarly / (2 * KS); ++i)
                word(s, v, i);
        });
        half(st);
        // ahead of a wave that is at its scores: 529 us against 538 for 8192 tokens
        __builtin_amdgcn_s_setprio(1);
        u32x4 ring[C::kAhead];
#pragma unroll
        for (int n = 0; n < C::kAhead; ++n)
            ring[n] = value(v, n);
        float4v kq[2];
        if constexpr (C8) {
            kq[0] = scales(k, 0);
            kq[1] = scales(k, 1);
        }
        top = -INFINITY;
#pragma unroll
        for (int n = 0; n < 4 * DB; ++n) {
            const int j = n / DB, d = n % DB;
            o[d] = mfma32(VT, ring[n % C::kAhead], operand(p, j), o[d]);
            if constexpr (C::kTwo)
                o[d] = mfma32(VT, ring[n % C::kAhead], operand(p2, j), o[d]);
            if (n + C::kAhead < 4 * DB)
                ring[n % C::kAhead] = value(v, n + C::kAhead);
            if (j < 2)
#pragma unroll
                for (int i = n * (16 - kEarly) / (2 * DB); i < (n + 1) * (16 - kEarly) / (2 * DB); ++i)
                    word(s, v, kEarly + i);
#pragma unroll
            for (int g = n * 8 / (4 * DB); g < (n + 1) * 8 / (4 * DB); ++g) {
                if constexpr (C8) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        next[g / 4][4 * g % 16 + i] *= kq[g % 2][i];
                    if (g < 6)
                        kq[g % 2] = scales(k, g + 2);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top = fmaxf(top, next[g / 4][4 * g % 16 + i]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_setprio(0);
    };
    // Where not every row sees the whole step its values must be finite for the plain
    // product: NaN and infinities times 0 are NaN.
    auto plain = [&](int st) __attribute__((always_inline)) {
        if (whole_all(st) && stage.here(st))
            return true;
        bool bad = false;
        for (int i = tid; i < C::kBytes / 16; i += kWaves * kWave)
            bad |= not_finite<VT>(lds16(v_buf(st), i * 16));
        return !__syncthreads_or(bad);
    };

    auto begin = [&]() __attribute__((always_inline)) {
        m = limit = -INFINITY;
        l = 0.0f;
        zero = C::kFirst;
        far = false;
#pragma unroll
        for (int d = 0; d < DB; ++d)
            o[d] = float16v{};
    };
    auto all_scores = [&]() __attribute__((always_inline)) {
        scores(sa, k_buf(0), [](int) {});
        if constexpr (C8)
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                const float4v f = scales(k_buf(0), g);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sa[g / 4][4 * g % 16 + i] *= f[i];
                __builtin_amdgcn_sched_barrier(0);
            }
    };
    begin();
    int st = 0;
    if (steps > 0) {
        load_places(0);
        at_k[0] = stage.place(0, 0);
        at_k[1] = stage.place(0, 1);
        stage.template fetch<false>(at_k, k_buf(0));
        stage.template put<false>(k_buf(0));
        stage.template fetch<true>(at_k, v_buf(0));
        stage.template put<true>(v_buf(0));
        if (steps > 1) {
            at_k[0] = stage.place(1, 0);
            at_k[1] = stage.place(1, 1);
            stage.template fetch<false>(at_k, k_buf(1));
            stage.template put<false>(k_buf(1));
        }
        turn();
        all_scores();
        top = top_of(sa);
    }
    // two steps a turn of the loop: the scores change places
    while (st < steps) {
        open(st);
        if (!plain(st))
            break;
        body(st, sa, sb);
        close(st);
        if (++st == steps)
            break;
        open(st);
        if (!plain(st))
            break;
        body(st, sb, sa);
        close(st);
        ++st;
    }
    if (st < steps) {
        // All steps again, one after the other.  A value that is not finite reaches the rows
        // that see it and no others: the product takes 0 for it, and counts of such values
        // that a row sees say which of its sums become infinite.
        constexpr uint32_t kOne = VT == APMOE_F16 ? 0x3C00u : 0x3F80u;
        begin();
        turn();
        load_places(0);
        for (st = 0; st < steps; ++st) {
            if (!stage.knows(st))
                load_places(st);
            at_k[0] = stage.place(st, 0);
            at_k[1] = stage.place(st, 1);
            stage.template fetch<false>(at_k, k_buf(0));
            stage.template put<false>(k_buf(0));
            stage.template fetch<true>(at_k, v_buf(0));
            stage.template put<true>(v_buf(0));
            turn();
            const char *const v = v_buf(0);
            const Sight g = sight_of(st);
            all_scores();
            mask(g, sa);
            rescale(sa);
            first_scales(v);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                word(sa, v, i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u32x4 ones;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ones[i] = (sees(g, 8 * j + 2 * i) ? kOne : 0u) | (sees(g, 8 * j + 2 * i + 1) ? kOne << 16 : 0u);
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    u32x4 x = value(v, j * DB + d), plus, minus;
                    split_values<VT>(x, plus, minus);
                    o[d] = mfma32(VT, x, operand(p, j), o[d]);
                    if constexpr (C::kTwo)
                        o[d] = mfma32(VT, x, operand(p2, j), o[d]);
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
            }
            turn();
        }
    }
    l += __shfl_xor(l, 32, kWave);
    // columns 32 d + 8 j + 4 h .. + 3 of the row: o[d][4 j] .. + 3
    if (t.parts > 1) {
        const size_t slot = ((size_t)item * P.kv.Hkv + kvh) * kRows + mine;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float4v *>(P.part_o + slot * D + 32 * d + 8 * j + 4 * h) =
                    float4v{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
        if (h == 0) {
            P.part_ml[2 * slot] = m;
            P.part_ml[2 * slot + 1] = l;
        }
        return;
    }
    const float inv = 1.0f / l;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int j = 0; j < 16; ++j)
            o[d][j] = l == 0.0f ? 0.0f : o[d][j] * inv;  // nothing seen: zeros, whatever lies there
    const size_t row = (size_t)token * P.Hq + qh;
    constexpr int kGroups = D < kBlk ? 1 : D / kBlk, kBlocks = DB / kGroups;
#pragma unroll
    for (int n = 0; n < kGroups; ++n) {
        float scale = 1.0f;
        if (D >= kBlk && P.out8) {
            uint32_t a = 0;
#pragma unroll
            for (int d = 0; d < kBlocks; ++d)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    a = max(a, mag(o[n * kBlocks + d][j]));
            a = max(a, (uint32_t)__shfl_xor((int)a, 32, kWave));
            scale = scale_of(a);
            if (live && h == 0)
                P.out_scale[row * kGroups + n] = scale;
        }
        if (live)
#pragma unroll
            for (int d = n * kBlocks; d < (n + 1) * kBlocks; ++d)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x[4] = {o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
                    store_columns<QT>(P, row, 32 * d + 8 * j + 4 * h, x, scale);
                }
    }
}

// Joins the parts of the row tiles that are split: D / 4 threads a row, 256 a workgroup.
template <int QT, int D>
__global__ void __launch_bounds__(256) join_rows(const AttnParams P)
{
    constexpr int kLanes = D / 4, kGroupLanes = kBlk / 4;
    RowTile t;
    if (!row_tile(P, blockIdx.x, t) || t.parts <= 1)
        return;
    const int kvh = blockIdx.y, c = threadIdx.x % kLanes, i = blockIdx.z * (256 / kLanes) + threadIdx.x / kLanes;
    if (i > t.last_row)
        return;
    const size_t slot0 = ((size_t)blockIdx.x * P.parts * P.kv.Hkv + kvh) * kRows + i;
    const size_t step = (size_t)P.kv.Hkv * kRows;
    float M = -INFINITY;
    for (int n = 0; n < t.parts; ++n)
        M = fmaxf(M, P.part_ml[2 * (slot0 + n * step)]);
    float L = 0.0f, v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int n = 0; n < t.parts; ++n) {
        const size_t slot = slot0 + n * step;
        const float l = P.part_ml[2 * slot + 1], f = part_factor(P.part_ml[2 * slot], l, M, score_factor(P.scale));
        const float4v o = *reinterpret_cast<const float4v *>(P.part_o + slot * D + 4 * c);
        if (l == 0.0f)  // the part saw nothing
            continue;
        L += f * l;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] += f * o[j];
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] *= inv;
        a = max(a, mag(v[j]));
    }
    const int qi = t.token(i), qh = kvh * t.G + t.row0 + i - (qi - t.q0) * t.G;
    const int64_t token = (int64_t)t.row_of_b + qi;
    const bool live = token >= 0 && token < P.s.T;
    const size_t row = (size_t)token * P.Hq + qh;
    float scale = 1.0f;
    if (D >= kBlk && P.out8) {
#pragma unroll
        for (int d = kGroupLanes / 2; d >= 1; d >>= 1)
            a = max(a, (uint32_t)__shfl_xor((int)a, d, kWave));
        scale = scale_of(a);
        if (live && c % kGroupLanes == 0)
            P.out_scale[row * (D / kBlk) + c / kGroupLanes] = scale;
    }
    if (live)
        store_columns<QT>(P, row, 4 * c, v, scale);
}

template <int QT, bool C8, int D>
hipError_t prefill_launch(const AttnParams &P, hipStream_t s)
{
    const int64_t blocks = (int64_t)P.tiles * P.kv.Hkv * P.parts;  // below 2^36 / kRows
    hipLaunchKernelGGL((prefill_kernel<QT, C8, D>),
                       dim3((uint32_t)(blocks < kGridX ? blocks : kGridX), (uint32_t)((blocks + kGridX - 1) / kGridX)),
                       dim3(kWaves * kWave), 0, s, P);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || P.parts == 1)
        return e;
    hipLaunchKernelGGL((join_rows<QT, D>), dim3(P.tiles, P.kv.Hkv, kRows * D / 4 / 256), dim3(256), 0, s, P);
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

int prefill_tiles(int B, int T, int G)
{
    // each sequence's last tile may be smaller
    const int64_t all = (int64_t)T * G, most = all / kRows + B;
    return (int)(most < all ? most : all);
}

int prefill_parts(int tiles, int Hkv, int room)
{
    const int64_t blocks = (int64_t)tiles * Hkv;
    if (blocks == 0 || blocks > kSplitBlocks || room < 2 * kPartSteps * kStep)
        return 1;
    return (int)std::min<int64_t>(kPartBlocks / blocks, kMaxParts);
}

hipError_t launch_attn_prefill(const AttnParams &P, hipStream_t s)
{
    if (P.dtype == APMOE_F16)
        return P.kv.c8 ? prefill_dim<APMOE_F16, true>(P, s) : prefill_dim<APMOE_F16, false>(P, s);
    return P.kv.c8 ? prefill_dim<APMOE_BF16, true>(P, s) : prefill_dim<APMOE_BF16, false>(P, s);
}

}  // namespace apmoe
