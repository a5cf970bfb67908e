// gemm_fp8_tile.hip -- the e4m3 product of calls with many rows: LDS tiles of weights
// and tokens, matrix units fed from them.
//
// Tile: 256 weight rows in two halves of 128 (with the activation: 128 gate rows and the
// 128 matching up rows, so that one workgroup holds the group of 128 values behind a
// scale of a8) x up to 256 tokens, one workgroup of 8 waves.  Wave (wr, wt) multiplies
// rows 32 wr .. + 31 of both halves by token half wt; the sums of a block of 128 columns
// are scaled and added in fp32.
//
// A stage is one block: the 128-byte rows of the weights and tokens and the tokens'
// scales, copied global -> LDS without passing registers, ahead of the products.  A row's
// 16-byte chunk c is stored in slot c ^ ((row / 2) % 8), so 16 lanes reading one chunk of
// 16 consecutive rows hit distinct banks.  Fragments are read ahead too.  When every read
// of a stage has been sent, one barrier (Stages::turn) says that the stage's buffer is
// free and that the next stage has landed; the next stage's first fragments are read
// while the rest of this one multiplies.
//
// Two kernels (block_product has the reason): e4m3 MFMAs for 16-bit outputs (tile_fast),
// fp16 MFMAs on converted operands for sums that stay in fp32 or are quantised again
// (tile_exact).  A vector instruction holds a SIMD for about 4 clocks and an MFMA for 8, so
// beside a 32-clock MFMA there is room for 6 others (they have 6.5 and 7.1).  Measured: 4096
// x 6144 x 4096 to fp16 107 to 115 us, 1.8 to 1.9 PFLOP/s; through fp16 products 8 experts of
// 4096 x 14336 with 4096 rows, unevenly, 518 to 526 us, 0.92, and gate_up of the same layer's
// 8192 rows 1.8 ms, 1.07.
//
// What bounds them is that a CU holds one workgroup, two waves a SIMD, which do not cover
// each other's waits: the matrix units are busy for 37, 50 and 56 % of the SIMDs' cycles in
// these three, a wave stands at a wait or the barrier for 40, 32 and 32 % of its time, and for
// 30, 29 and 28 % it has an instruction ready while the SIMD takes the other wave's.  The
// copies alone are not it: without any the first takes 92 us of 108 and the second 428 of
// 526, with copies that always find their lines in the L2 104 and 462.
#include <algorithm>

#include "gemm_fp8.h"

namespace apmoe {
namespace {

constexpr int kThreads = 512;
constexpr int kHalf = 128;  // weight rows of a half
constexpr int kXcdCus = 32;
constexpr int kGridX = 1 << 20;  // workgroups in x: a dimension has fewer than 2^32 threads
constexpr int kGroup = 8;   // weight tiles that share their token tiles through an XCD's L2
constexpr uint32_t kStageW = 2 * kHalf * kBlk;
// LDS of tiles of TOK tokens: NB buffers, each a stage and its tokens' scales.  A stage is
// multiplied in 1 to 2 us, which a copy may take: three buffers where they fit.
template <int TOK>
struct Lds {
    static constexpr uint32_t kStage = kStageW + TOK * kBlk;
    static constexpr uint32_t kBuffer = kStage + TOK * 4;
    static constexpr int NB = TOK <= 128 ? 3 : 2;
};
constexpr uint32_t kLds = 3 * Lds<128>::kBuffer;
static_assert(kLds >= 2 * Lds<256>::kBuffer && kLds <= 160 * 1024, "LDS of a workgroup");

__device__ const u32x4 kZeros = {0, 0, 0, 0};

struct TileParams {
    Fp8Params p;
    int NT;  // weight tiles of an expert
};

struct Tile {
    int e, r0, m0, M, nt;
};

// Workgroup -> tile, in scalar registers; every wave computes the same answer.  Tiles in
// order: groups of kGroup weight tiles, in a group the token tiles of every
// expert, then the group's weight tiles.  XCD x (workgroups b with b % 8 = x) takes the
// x-th eighth.  Lane l counts the token tiles of experts 4l .. 4l+3.
//
// A CU holds one workgroup, so an XCD works in rounds of kXcdCus tiles.  Where the last
// round would leave half of the CUs idle its tiles are split into 2 or 4 parts of their
// tokens, of not less than 64 (a part of half the tokens takes 0.62 of the time): 4096 x 6144
// x 4096, 1.5 rounds, 120 -> 107 us; 256 rows of it, 24 tiles, 51 -> 26.
__device__ inline bool resolve(const TileParams &T, int tok, Tile &t)
{
    const Fp8Params &P = T.p;
    const int lane = threadIdx.x % kWave;
    int o[5], n[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i)
        o[i] = P.offsets ? P.offsets[min(4 * lane + i, P.E)] : (4 * lane + i == 0 ? 0 : P.R);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = o[i + 1] - o[i];
        n[i] = m > 0 ? (m + tok - 1) / tok : 0;
        sum += n[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int v = __shfl_up(incl, d, kWave);
        incl += lane >= d ? v : 0;
    }
    const int MT = __builtin_amdgcn_readlane(incl, kWave - 1);
    const int total = MT * T.NT, per = (total + kXcds - 1) / kXcds;
    const int block = (int)(blockIdx.y * kGridX + blockIdx.x);
    const int first = (block % kXcds) * per, local = block / kXcds;
    const int mine = max(0, min(per, total - first)), rem = mine % kXcdCus;
    const int parts = tok >= 256 && 4 * rem <= kXcdCus ? 4 : 2 * rem <= kXcdCus ? 2 : 1;
    const int over = local - (mine - rem);  // workgroup of the last round
    if (over >= parts * rem)
        return false;
    const int l = first + (over < 0 ? local : mine - rem + over / parts);
    const int size = over < 0 ? tok : tok / parts, part = over < 0 ? 0 : over % parts;
    const int k = l / (kGroup * MT);
    const int gs = min(kGroup, T.NT - kGroup * k);
    const int at_l = l - k * kGroup * MT;
    const int u = at_l / gs;
    const int at = (int)__builtin_ctzll(__ballot(incl > u));  // the lane with token tile u
    int v = u - __builtin_amdgcn_readlane(incl - sum, at), e = 4 * at;
    int r0 = __builtin_amdgcn_readlane(o[0], at), r1 = __builtin_amdgcn_readlane(o[1], at);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int c = __builtin_amdgcn_readlane(n[i], at);
        if (v >= c && e == 4 * at + i) {
            v -= c;
            ++e;
            r0 = __builtin_amdgcn_readlane(o[i + 1], at);
            r1 = __builtin_amdgcn_readlane(o[i + 2], at);
        }
    }
    const int m0 = v * tok + part * size;
    t = Tile{e, r0, m0, min(size, r1 - r0 - m0), k * kGroup + at_l % gs};
    return t.M > 0;
}

// A pointer that is the same in every lane, in scalar registers.
__device__ inline const uint8_t *scalar_ptr(const uint8_t *p)
{
    const uint64_t v = (uint64_t)(uintptr_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<const uint8_t *>((uintptr_t)((uint64_t)hi << 32 | lo));
}

// The stages of one tile: their copies into LDS, the weights' scales, the turns.
// The copies of a stage are sent one by one between the products: a CU takes about 50
// clocks for each, and a wave whose request finds no room waits with everything behind it.
// Steps are counted from a turn to the next; a step sends EACH requests, every EVERY-th
// step, until all are sent.  POST: steps between a turn and the stage's end.
template <bool ACT, int TOK, int EACH, int EVERY, int POST>
struct Stages {
    static constexpr uint32_t kStage = Lds<TOK>::kStage, kBuffer = Lds<TOK>::kBuffer;
    static constexpr int NB = Lds<TOK>::NB;
    static constexpr int kXi = TOK > 64 ? TOK / 64 : 1;
    static constexpr int kCopies = 4 + kXi + 1;  // requests of a wave for a stage

    char *smem;
    int K, KB, wave, chunk, srow;
    int row[2];          // first row of each half
    const float *ws[2];  // the halves' scales by block
    __amdgpu_buffer_rsrc_t rw[2];
    uint32_t woff[2], xrow[kXi];
    const uint8_t *x8;
    const float *xsp;
    float sw[2], swn[2];  // scales of the stage and the next

    // Copies: wave w, request i: rows 64 i + 8 w + lane / 8, slot lane % 8.
    __device__ __attribute__((always_inline)) inline Stages(const TileParams &T, const Tile &t, char *smem_) : smem(smem_)
    {
        const Fp8Params &P = T.p;
        const int lane = threadIdx.x % kWave;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        K = P.K;
        KB = (K + kBlk - 1) / kBlk;
        const int nb = (P.N + kBlk - 1) / kBlk, fb = (P.F + kBlk - 1) / kBlk;
        const uint8_t *wbase = P.w8 + (size_t)t.e * P.N * K;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int lim = ACT ? (h + 1) * P.F : P.N;
            row[h] = ACT ? h * P.F + t.nt * kHalf : t.nt * 2 * kHalf + h * kHalf;
            const int blk = ACT ? t.nt : min(2 * t.nt + h, nb - 1);
            ws[h] = P.ws + (ACT ? (size_t)(2 * t.e + h) * fb + blk : (size_t)t.e * nb + blk) * KB;
            // rows past the matrix read as zeros
            rw[h] = make_rsrc(scalar_ptr(wbase + (size_t)row[h] * K),
                              __builtin_amdgcn_readfirstlane((uint32_t)max(0, min(kHalf, lim - row[h])) * (uint32_t)K));
        }
        const int crow = 8 * wave + lane / 8;
        chunk = (lane % 8) ^ ((crow / 2) % 8);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            woff[i] = (uint32_t)(64 * i + crow) * (uint32_t)K + 16u * chunk;
#pragma unroll
        for (int i = 0; i < kXi; ++i)
            xrow[i] = (uint32_t)src_row(P, t.r0 + t.m0 + min(64 * i + crow, t.M - 1));
        x8 = scalar_ptr(P.x8);
        // every 64 tokens' scales are copied by one wave of kXi (and again by the others: no
        // branch in the pipeline)
        srow = TOK > 64 ? wave % kXi : 0;
        xsp = P.xs + src_row(P, t.r0 + t.m0 + min(srow * 64 + lane, t.M - 1)) * KB;
        sw[0] = scale(0, 0);
        sw[1] = scale(1, 0);
    }

    // Request i of stage kb into buffer number q.
    __device__ __attribute__((always_inline)) inline void copy(int i, int kb, int q) const
    {
        char *dst = smem + q * kBuffer;
        // K's last block may be shorter: zeros there, for the weights by an offset out of
        // range, for the tokens from kZeros
        const bool in = kb * kBlk + 16 * chunk < K;
        if (i < 4) {
            const int h = i / 2, u = i % 2;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rw[h], (__attribute__((address_space(3))) void *)(dst + h * kHalf * kBlk + (64 * u + 8 * wave) * kBlk), 16,
                in ? woff[u] : 0x80000000u, (uint32_t)kb * kBlk, 0, 0);
        } else if (i < 4 + kXi) {
            const int u = i - 4;
            const uint64_t pick = in ? ~0ull : 0ull, zeros = (uint64_t)(uintptr_t)&kZeros;
            const uint64_t src = (uint64_t)(uintptr_t)(x8 + (uint32_t)kb * kBlk + 16 * chunk) + (uint64_t)xrow[u] * (uint32_t)K;
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void *)(uintptr_t)((src & pick) | (zeros & ~pick)),
                (__attribute__((address_space(3))) void *)(dst + kStageW + (64 * u + 8 * wave) * kBlk), 16, 0, 0);
        } else {
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(xsp + kb),
                                             (__attribute__((address_space(3))) void *)(dst + kStage + srow * 256), 4, 0, 0);
        }
    }

    // Step `st` after the turn of stage kb in buffer q: its share of the copies of stage
    // kb + NB into that buffer.  Before a stage's own turn, the steps are those after the
    // turn of the stage before it.
    __device__ __attribute__((always_inline)) inline void step(int st, int kb, int q) const
    {
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
            if (st % EVERY == 0 && i / EACH == st / EVERY)
                copy(i, min(kb + NB, KB - 1), q);
    }
    static constexpr int kPost = (POST + EVERY - 1) / EVERY * EACH < kCopies ? (POST + EVERY - 1) / EVERY * EACH : kCopies;

    // A scalar load: complete, with the LDS reads, at the next turn.
    __device__ inline float scale(int h, int kb) const
    {
        return *reinterpret_cast<const __attribute__((address_space(4))) float *>((uintptr_t)(ws[h] + kb));
    }

    // The first stages; of the last buffer's, what a turn would have sent.
    __device__ __attribute__((always_inline)) inline void begin() const
    {
#pragma unroll
        for (int q = 0; q < NB; ++q)
#pragma unroll
            for (int i = 0; i < (q + 1 < NB ? kCopies : kPost); ++i)
                copy(i, min(q, KB - 1), q);
        __builtin_amdgcn_s_waitcnt(wait_vm<(NB - 2) * kCopies + kPost>());
        asm volatile("s_barrier" ::: "memory");
    }

    // Every read of stage kb has been sent: waits for them and for the next stage (all but
    // the last NB - 2 stages' copies have landed).
    __device__ __attribute__((always_inline)) inline void turn(int kb)
    {
        const int k1 = min(kb + 1, KB - 1);
        swn[0] = scale(0, k1);
        swn[1] = scale(1, k1);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(wait_vm<(NB - 2) * kCopies>());
        asm volatile("s_barrier" ::: "memory");
    }

    // stage(buffer number as a constant, kb) for every block.
    template <typename F>
    __device__ __attribute__((always_inline)) inline void run(F &&stage)
    {
        int kb = 0;
        for (; kb + NB <= KB; kb += NB) {
            stage(std::integral_constant<int, 0>{}, kb);
            stage(std::integral_constant<int, 1>{}, kb + 1);
            if constexpr (NB > 2)
                stage(std::integral_constant<int, 2>{}, kb + 2);
        }
        if (kb < KB)
            stage(std::integral_constant<int, 0>{}, kb);
        if (NB > 2 && kb + 1 < KB)
            stage(std::integral_constant<int, 1>{}, kb + 1);
        __builtin_amdgcn_s_waitcnt(wait_vm<0>());  // no copy into LDS is left when it is used again
    }
};

// Rows of `bytes` bytes on their way out through LDS: a product's lane has 4 values of 16
// or 32 tokens, and stored from there a request would touch 16 or more lines (12 us a
// tile); from LDS it covers whole ones.
constexpr uint32_t kRowPad = 16;

__device__ __attribute__((always_inline)) inline void store_rows(const char *smem, uint32_t bytes, int rows, char *out,
                                                                size_t stride, int valid)
{
    const int per = (int)bytes / 16;
    for (int c = threadIdx.x; c < rows * per; c += kThreads) {
        const int r = c / per, b = c % per * 16;
        if (b < valid)
            *reinterpret_cast<u32x4 *>(out + (size_t)r * stride + b) =
                *reinterpret_cast<const u32x4 *>(smem + (uint32_t)r * (bytes + kRowPad) + b);
    }
}

// The product's tile of up to TOK tokens: put(f) calls f(half, token, row of the half, four
// values) for what the lane holds.  Rows of fp32 are too long for LDS with 256 tokens and
// leave half by half.
template <int TOK, typename F>
__device__ __attribute__((always_inline)) inline void store_product(const Fp8Params &P, const Tile &t, char *smem, F &&put)
{
    const int size = P.out_dtype == APMOE_F32 ? 4 : 2;
    const int n0 = t.nt * 2 * kHalf;
    if (P.N * size % 16 != 0) {  // rows that do not start on 16 bytes
        put([&](int h, int tok, int n, const float4v &v) {
            if (tok < t.M && n0 + h * kHalf + n < P.N)
                store4(P, (size_t)(t.r0 + t.m0 + tok), n0 + h * kHalf + n, v);
        });
        return;
    }
    static_assert(TOK * (2 * kHalf * 2 + kRowPad) <= kLds, "rows of 16-bit values fit");
    static_assert(TOK * ((TOK <= 128 ? 2 : 1) * kHalf * 4 + kRowPad) <= kLds, "rows of fp32, or their halves, fit");
    const int halves = TOK <= 128 || size == 2 ? 2 : 1;  // of a pass
    const uint32_t bytes = (uint32_t)(halves * kHalf * size);
    for (int h0 = 0; h0 < 2; h0 += halves) {
        __syncthreads();  // the last stage is read, or the rows of the pass before
        put([&](int h, int tok, int n, const float4v &v) {
            if (h < h0 || h >= h0 + halves)
                return;
            char *at = smem + (uint32_t)tok * (bytes + kRowPad) + (uint32_t)(((h - h0) * kHalf + n) * size);
            const u32x4 o = pack4(P.out_dtype, v);
            if (size == 4)
                *reinterpret_cast<u32x4 *>(at) = o;
            else
                *reinterpret_cast<u32x2 *>(at) = u32x2{o[0], o[1]};
        });
        __syncthreads();
        const int n = n0 + h0 * kHalf;
        store_rows(smem, bytes, t.M, static_cast<char *>(P.out) + ((size_t)(t.r0 + t.m0) * P.N + n) * size,
                   (size_t)P.N * size, min(P.N - n, 2 * kHalf) * size);
    }
}

// 4 weight tiles x TTN token tiles of 16 a wave, one e4m3 MFMA and four additions each
// for a block.  Lane l has token l % 16 and weight rows 4 (l / 16) .. + 3 of a product.
template <int TTN>
__device__ __attribute__((always_inline)) inline void tile_fast(const TileParams &T, const Tile &t, char *smem)
{
    static_assert(TTN % 2 == 0, "b's two register sets alternate across stages");
    const Fp8Params &P = T.p;
    typedef Stages<false, 32 * TTN, TTN == 2 ? 3 : 2, 1, 2> S;
    constexpr int NB = S::NB;
    S s(T, t, smem);
    const int lane = threadIdx.x % kWave, wr = s.wave & 3, wt = s.wave >> 2;
    const int j = lane & 15, g = lane >> 4;

    // LDS addresses in a buffer: chunks g and g + 4 of the wave's first weight and token
    // row, and the scale of its first token.  Everything else is a constant further; the
    // empty asm keeps the compiler from holding each sum in a register of its own.
    struct At {
        uint32_t a[2], b[2], s;
    };
    const uint32_t base = lds_addr(smem), swz = 16u * (uint32_t)(g ^ ((j / 2) % 8));
    auto at = [&](int buf) {
        const uint32_t sb = base + buf * S::kBuffer;
        const uint32_t arow = sb + (uint32_t)(32 * wr + j) * kBlk, brow = sb + kStageW + (uint32_t)(wt * 16 * TTN + j) * kBlk;
        At v = {{arow + swz, arow + (swz ^ 64u)}, {brow + swz, brow + (swz ^ 64u)},
                sb + S::kStage + 4u * (uint32_t)(wt * 16 * TTN + j)};
        asm volatile("" : "+v"(v.a[0]), "+v"(v.a[1]), "+v"(v.b[0]), "+v"(v.b[1]), "+v"(v.s));
        return v;
    };
    auto read_a = [&](const At &v, int r) {
        const uint32_t o = (r >> 1) * kHalf * kBlk + (r & 1) * 16 * kBlk;
        return Frag8{lds_b128(v.a[0] + o), lds_b128(v.a[1] + o)};
    };
    auto read_b = [&](const At &v, int c) {
        return Frag8{lds_b128(v.b[0] + c * 16 * kBlk), lds_b128(v.b[1] + c * 16 * kBlk)};
    };
    auto read_sx = [&](const At &v, int c) { return lds_f32(v.s + 64u * c); };

    float4v acc[4][TTN], p[4];
    float sx[2], f[2] = {0.f, 0.f};
    auto add = [&](int r, int c) {  // the product in p[r] is tile c's
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[r][c][i] = __builtin_fmaf(p[r][i], f[r >> 1], acc[r][c][i]);
    };
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        p[r] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < TTN; ++c)
            acc[r][c] = p[r];
    }
    s.begin();
    const At bufs[3] = {at(0), at(1), at(NB > 2 ? 2 : 0)};
    Frag8 a[NB][2], a2[2], b[2];  // weight tiles 0, 1 in a set for each buffer; 2, 3 in one
#pragma unroll
    for (int r = 0; r < 4; ++r)
        (r < 2 ? a[0][r] : a2[r - 2]) = read_a(bufs[0], r);
    b[0] = read_b(bufs[0], 0);
    sx[0] = read_sx(bufs[0], 0);
    // Step c multiplies token tile c by the four weight tiles.  Each MFMA is preceded by
    // the four additions of the product that its registers held; b is read a step ahead.
    s.run([&](auto q, int kb) {
        constexpr int Q = decltype(q)::value;
        const At &sb = bufs[Q], &sn = bufs[(Q + 1) % NB];
#pragma unroll
        for (int c = 0; c < TTN; ++c) {
            if (c + 1 < TTN) {  // (in step TTN - 2: before the turn)
                b[(c + 1) % 2] = read_b(sb, c + 1);
                sx[(c + 1) % 2] = read_sx(sb, c + 1);
            }
            if (c == TTN - 2)
                s.turn(kb);
            if (c + 1 == TTN) {
                b[0] = read_b(sn, 0);
                sx[0] = read_sx(sn, 0);
            }
            if (c >= TTN - 2)
                a[(Q + 1) % NB][c + 2 - TTN] = read_a(sn, c + 2 - TTN);
            if (c >= TTN - 2)
                s.step(c + 2 - TTN, kb, Q);
            else
                s.step(c + 2, kb - 1, (Q + NB - 1) % NB);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                add(r, c == 0 ? TTN - 1 : c - 1);
                p[r] = block_product(r < 2 ? a[Q][r] : a2[r - 2], b[c % 2]);
                __builtin_amdgcn_sched_barrier(0);
                if (r >= 2 && c == TTN - 1)
                    a2[r - 2] = read_a(sn, r);
            }
            f[0] = sx[c % 2] * s.sw[0];
            f[1] = sx[c % 2] * s.sw[1];
        }
        s.sw[0] = s.swn[0];
        s.sw[1] = s.swn[1];
    });
#pragma unroll
    for (int r = 0; r < 4; ++r)
        add(r, TTN - 1);

    store_product<32 * TTN>(P, t, smem, [&](auto &&put) {
#pragma unroll
        for (int c = 0; c < TTN; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                put(r >> 1, wt * 16 * TTN + 16 * c + j, 32 * wr + 16 * (r & 1) + 4 * g, acc[r][c]);
    });
}

// 2 weight tiles (one of each half) x TB token tiles of 32 a wave.  Lane l has token
// l % 32 and weight rows 8 (v / 4) + 4 (l / 32) + v % 4, v = 0 .. 15, of a product.
//
// Eighth q of a stage: the 16 columns of one fp16 MFMA for all 2 x TB products, whose sums
// over the stage stay in p.  Between the MFMAs, four conversions for each: the next token
// tile's eighth, and the next eighth of the weights.  A fragment's register is read again
// right after its last conversion, a pass of MFMAs before it is needed.
template <bool ACT, int TB>
__device__ __attribute__((always_inline)) inline void tile_exact(const TileParams &T, const Tile &t, char *smem)
{
    const Fp8Params &P = T.p;
    constexpr int TOK = 64 * TB;
    typedef Stages<ACT, TOK, 1, TB, 2 * TB> S;
    constexpr int NB = S::NB;
    S s(T, t, smem);
    const int lane = threadIdx.x % kWave, wr = s.wave & 3, wt = s.wave >> 2;
    const int i = lane & 31, g = lane >> 5;

    // Eighths 2h and 2h + 1 are the two halves of chunk 2h + g.
    struct At {
        uint32_t a[4], b[4], s;
    };
    const uint32_t base = lds_addr(smem);
    auto at = [&](int buf) {
        const uint32_t sb = base + buf * S::kBuffer;
        At v;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const uint32_t c = 16u * (uint32_t)((2 * h + g) ^ ((i / 2) % 8));
            v.a[h] = sb + (uint32_t)(32 * wr + i) * kBlk + c;
            v.b[h] = sb + kStageW + (uint32_t)(wt * 32 * TB + i) * kBlk + c;
            asm volatile("" : "+v"(v.a[h]), "+v"(v.b[h]));
        }
        v.s = sb + S::kStage + 4u * (uint32_t)(wt * 32 * TB + i);
        return v;
    };
    auto read_a = [&](const At &v, int r, int h) { return lds_b128(v.a[h] + r * kHalf * kBlk); };
    auto read_b = [&](const At &v, int c, int h) { return lds_b128(v.b[h] + c * 32 * kBlk); };

    float16v acc[2][TB], p[2][TB];
    float sx[TB], swp[2] = {0.f, 0.f};  // scales of the products in p
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < TB; ++c)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                acc[r][c][v] = 0.f;
                p[r][c][v] = 0.f;
            }
    auto add = [&](int r, int c) {
        const float f = sx[c] * swp[r];
#pragma unroll
        for (int v = 0; v < 16; ++v)
            acc[r][c][v] = __builtin_fmaf(p[r][c][v], f, acc[r][c][v]);
    };
    s.begin();
    const At bufs[3] = {at(0), at(1), at(2)};
    static_assert(NB == 3, "three buffers");
    u32x4 a[2][2], b[2], ra[2], rb[TB];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        ra[r] = read_a(bufs[0], r, 0);
#pragma unroll
        for (int w = 0; w < 4; ++w)
            a[0][r][w] = half2_of(ra[r], 0, w);
    }
#pragma unroll
    for (int c = 0; c < TB; ++c) {
        rb[c] = read_b(bufs[0], c, 0);
        sx[c] = 0.f;
    }
#pragma unroll
    for (int w = 0; w < 4; ++w)
        b[0][w] = half2_of(rb[0], 0, w);
    s.run([&](auto qq, int kb) {
        constexpr int Q = decltype(qq)::value;
        const At &sb = bufs[Q], &sn = bufs[(Q + 1) % NB];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            // chunk h is read when chunk h - 1 has been converted: the stage's last reads are
            // sent in eighth 5 (b: 2h + 1 = 5 reads chunk 3)
            if (q == 6)
                s.turn(kb);
#pragma unroll
            for (int c = 0; c < TB; ++c) {
                const int cur = (q * TB + c) % 2;
                const int nc = (c + 1) % TB, nq = c + 1 < TB ? q : q + 1;  // the next token fragment
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const half8 av = __builtin_bit_cast(half8, a[q % 2][r]), bv = __builtin_bit_cast(half8, b[cur]);
                    if (q == 0) {
                        add(r, c);
#pragma unroll
                        for (int v = 0; v < 16; ++v)
                            p[r][c][v] = 0.f;
                    }
                    p[r][c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(av, bv, p[r][c], 0, 0, 0);
#pragma unroll
                    for (int w = 0; w < 2; ++w)
                        b[1 - cur][2 * r + w] = half2_of(rb[nc], nq % 2, 2 * r + w);
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        if (TB == 1 || w / 2 == r)  // TB = 2: weight tile c beside token tile c
                            a[(q + 1) % 2][TB == 1 ? r : c][w] = half2_of(ra[TB == 1 ? r : c], (q + 1) % 2, w);
                    __builtin_amdgcn_sched_barrier(0);
                }
                // fragments whose two eighths are converted: the next chunk, of this stage or
                // of the next
                if (nq % 2 == 1)
                    rb[nc] = nq < 7 ? read_b(sb, nc, (nq + 1) / 2) : read_b(sn, nc, 0);
                if (q % 2 == 0) {
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (TB == 1 || r == c)
                            ra[r] = q < 6 ? read_a(sb, r, q / 2 + 1) : read_a(sn, r, 0);
                }
                if (q == 1)
                    sx[c] = lds_f32(sb.s + 128u * c);
                if (q >= 6)
                    s.step((q - 6) * TB + c, kb, Q);
                else
                    s.step((q + 2) * TB + c, kb - 1, (Q + NB - 1) % NB);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        swp[0] = s.sw[0];
        swp[1] = s.sw[1];
        s.sw[0] = s.swn[0];
        s.sw[1] = s.swn[1];
    });
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < TB; ++c)
            add(r, c);

    if constexpr (ACT) {
        const int fb = (P.F + kBlk - 1) / kBlk, f0 = t.nt * kHalf + 32 * wr + 4 * g;
        uint32_t *amax = reinterpret_cast<uint32_t *>(smem);  // [4 row groups][TOK], then the 8-bit rows
        char *out8 = smem + 4 * TOK * sizeof(uint32_t);
        static_assert(4 * TOK * sizeof(uint32_t) + TOK * (kHalf + kRowPad) <= kLds, "the 8-bit rows fit");
        __syncthreads();                                      // the last stage is read
#pragma unroll
        for (int c = 0; c < TB; ++c) {
            uint32_t mx = 0;
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                acc[0][c][v] = silu_mul32(acc[0][c][v], acc[1][c][v]);
                if (f0 + 8 * (v / 4) < P.F)  // F is a multiple of 16
                    mx = max(mx, mag(acc[0][c][v]));
            }
            mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32, kWave));
            if (g == 0)
                amax[wr * TOK + wt * 32 * TB + 32 * c + i] = mx;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < TB; ++c) {
            const int tok = wt * 32 * TB + 32 * c + i;
            uint32_t mx = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                mx = max(mx, amax[w * TOK + tok]);
            const float sc = scale_of(mx), inv = 1.0f / sc;
#pragma unroll
            for (int v = 0; v < 16; v += 4)
                *reinterpret_cast<uint32_t *>(out8 + (uint32_t)tok * (kHalf + kRowPad) + 32 * wr + 4 * g + 2 * v) =
                    to_e4m3x4(acc[0][c][v] * inv, acc[0][c][v + 1] * inv, acc[0][c][v + 2] * inv, acc[0][c][v + 3] * inv);
            if (tok < t.M && wr == 0 && g == 0)
                P.os[(size_t)(t.r0 + t.m0 + tok) * fb + t.nt] = sc;
        }
        __syncthreads();
        store_rows(out8, kHalf, t.M, static_cast<char *>(P.out) + (size_t)(t.r0 + t.m0) * P.F + t.nt * kHalf, P.F,
                   P.F - t.nt * kHalf);
    } else {
        store_product<TOK>(P, t, smem, [&](auto &&put) {
#pragma unroll
            for (int c = 0; c < TB; ++c)
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int v = 0; v < 16; v += 4)
                        put(r, wt * 32 * TB + 32 * c + i, 32 * wr + 4 * g + 2 * v,
                            float4v{acc[r][c][v], acc[r][c][v + 1], acc[r][c][v + 2], acc[r][c][v + 3]});
        });
    }
}

template <bool EXACT, bool ACT>
__global__ void __launch_bounds__(kThreads) fp8_tile_kernel(const TileParams T)
{
    __shared__ __attribute__((aligned(1024))) char smem[kLds];
    Tile t = {0, 0, 0, 0, 0};
    if (!resolve(T, fp8_tile_tokens(EXACT), t))
        return;
    if constexpr (EXACT) {
        if (t.M > 64)
            tile_exact<ACT, 2>(T, t, smem);
        else
            tile_exact<ACT, 1>(T, t, smem);
    } else {
        if (t.M > 128)
            tile_fast<8>(T, t, smem);
        else if (t.M > 64)
            tile_fast<4>(T, t, smem);
        else
            tile_fast<2>(T, t, smem);
    }
}

}  // namespace

static int weight_tiles(const Fp8Params &P, bool act)
{
    return act ? (P.F + kHalf - 1) / kHalf : (P.N + 2 * kHalf - 1) / (2 * kHalf);
}

long fp8_tiles(const Fp8Params &P, bool act, int tok)
{
    return fp8_token_tiles(P.E, P.R, tok) * weight_tiles(P, act);
}

hipError_t launch_fp8_tile(const Fp8Params &P, bool act, bool exact, hipStream_t s)
{
    const TileParams T{P, weight_tiles(P, act)};
    const long tiles = fp8_tiles(P, act, fp8_tile_tokens(exact)), round = kXcds * kXcdCus;
    const long blocks = (tiles + round - 1) / round * round;  // the last round whole: its tiles may be split
    const dim3 grid((unsigned)std::min(blocks, (long)kGridX), (unsigned)((blocks + kGridX - 1) / kGridX));
    if (act)
        hipLaunchKernelGGL((fp8_tile_kernel<true, true>), grid, dim3(kThreads), 0, s, T);
    else if (exact)
        hipLaunchKernelGGL((fp8_tile_kernel<true, false>), grid, dim3(kThreads), 0, s, T);
    else
        hipLaunchKernelGGL((fp8_tile_kernel<false, false>), grid, dim3(kThreads), 0, s, T);
    return hipGetLastError();
}

}  // namespace apmoe
