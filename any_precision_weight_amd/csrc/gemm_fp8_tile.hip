// gemm_fp8_tile.hip -- the e4m3 product of experts with many rows: LDS tiles of weights
// and tokens, matrix units fed from them.
//
// Tile: 256 weight rows in two halves of 128 (with the activation: 128 gate rows and the
// 128 matching up rows, so that one workgroup holds the group of 128 values behind a
// scale of a8) x up to 256 tokens, one workgroup of 8 waves.  Wave (wr, wt) multiplies
// rows 32 wr .. + 31 of both halves by token half wt: 4 x TTN products of 16 x 16, whose
// fp32 results are scaled and added once per block of 128 columns.
//
// A stage is one block: 256 + 256 rows of 128 bytes and the tokens' scales, copied
// global -> LDS without passing registers while the previous stage is multiplied; one
// barrier per stage.  A row's 16-byte chunk c is stored in slot c ^ ((row / 2) % 8), so
// 16 lanes reading one chunk of 16 consecutive rows hit distinct banks.
#include "gemm_fp8.h"

namespace apmoe {
namespace {

constexpr int kThreads = 512;
constexpr int kHalf = 128;             // weight rows of a half
constexpr int kGroup = 8;              // weight tiles that share their token tiles through an XCD's L2
constexpr uint32_t kStageW = 2 * kHalf * kBlk;
// LDS of tiles of 32 TTN tokens: NB buffers, each a stage and its tokens' scales.  A
// stage is multiplied in about 1 us, less than a copy may take: three buffers where they
// fit.
template <int TTN>
struct Lds {
    static constexpr uint32_t kStage = kStageW + 32 * TTN * kBlk;
    static constexpr uint32_t kBuffer = kStage + 32 * TTN * 4;
    static constexpr int NB = TTN <= 4 ? 3 : 2;
};
constexpr uint32_t kLds = 3 * Lds<4>::kBuffer;
static_assert(kLds >= 2 * Lds<8>::kBuffer && kLds <= 160 * 1024, "LDS of a workgroup");

__device__ const u32x4 kZeros = {0, 0, 0, 0};

struct TileParams {
    Fp8Params p;
    int NT;  // weight tiles of an expert
};

struct Tile {
    int e, r0, m0, M, nt;
};

// Workgroup -> tile; every thread computes the same answer.  Tiles in order: groups of
// kGroup weight tiles, in a group the token tiles of every served expert, then the
// group's weight tiles.  XCD x (workgroups b with b % 8 = x) takes the x-th eighth.
__device__ inline bool resolve(const TileParams &T, int tok, int *scan, Tile &t)
{
    const Fp8Params &P = T.p;
    const int tid = threadIdx.x;
    int n = 0;
    if (tid < P.E) {
        int r0, m;
        expert_rows(P, tid, r0, m);
        n = m > kStreamMax ? (m + tok - 1) / tok : 0;
    }
    scan[tid] = n;
    __syncthreads();
    for (int d = 1; d < APMOE_MAX_EXPERTS; d <<= 1) {
        const int v = tid >= d ? scan[tid - d] : 0;
        __syncthreads();
        scan[tid] += v;
        __syncthreads();
    }
    const int MT = scan[APMOE_MAX_EXPERTS - 1];
    const int total = MT * T.NT, per = (total + kXcds - 1) / kXcds;
    const int local = (int)blockIdx.x / kXcds, l = ((int)blockIdx.x % kXcds) * per + local;
    if (local >= per || l >= total)
        return false;
    const int k = l / (kGroup * MT);
    const int gs = min(kGroup, T.NT - kGroup * k);
    const int rem = l - k * kGroup * MT;
    const int u = rem / gs;
    int lo = 0, hi = P.E - 1;  // the first expert with scan > u
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (scan[mid] > u)
            hi = mid;
        else
            lo = mid + 1;
    }
    int r0, m;
    expert_rows(P, lo, r0, m);
    const int m0 = (u - (lo > 0 ? scan[lo - 1] : 0)) * tok;
    t = Tile{lo, r0, m0, min(tok, m - m0), k * kGroup + rem % gs};
    return true;
}

// A pointer that is the same in every lane, in scalar registers.
__device__ inline const uint8_t *scalar_ptr(const uint8_t *p)
{
    const uint64_t v = (uint64_t)(uintptr_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<const uint8_t *>((uintptr_t)((uint64_t)hi << 32 | lo));
}

// TTN: 16-token tiles of a wave.  EXACT: fp16 products (block_product).
template <bool EXACT, bool ACT, int TTN>
__device__ __attribute__((always_inline)) inline void tile(const TileParams &T, const Tile &t, char *smem)
{
    const Fp8Params &P = T.p;
    constexpr int kTok = 32 * TTN;  // tokens of the tile
    constexpr int kXi = kTok > 64 ? kTok / 64 : 1;
    constexpr int kCopies = 4 + kXi + 1;  // requests of a wave for a stage
    constexpr uint32_t kStage = Lds<TTN>::kStage, kBuffer = Lds<TTN>::kBuffer;
    constexpr int NB = Lds<TTN>::NB;
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wr = wave & 3, wt = wave >> 2;
    const int j = lane & 15, g = lane >> 4;
    const int K = P.K, KB = (K + kBlk - 1) / kBlk, nb = (P.N + kBlk - 1) / kBlk, fb = (P.F + kBlk - 1) / kBlk;
    const uint32_t base = lds_addr(smem);

    // first row of each half, and how many it has
    int row[2], rows[2];
    const float *ws[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int lim = ACT ? (h + 1) * P.F : P.N;
        row[h] = ACT ? h * P.F + t.nt * kHalf : t.nt * 2 * kHalf + h * kHalf;
        rows[h] = max(0, min(kHalf, lim - row[h]));
        const int blk = ACT ? t.nt : min(2 * t.nt + h, nb - 1);
        ws[h] = P.ws + (ACT ? (size_t)(2 * t.e + h) * fb + blk : (size_t)t.e * nb + blk) * KB;
    }
    // ---- copies: wave w, instruction i: rows 64 i + 8 w + lane / 8, slot lane % 8
    const uint8_t *wbase = P.w8 + (size_t)t.e * P.N * K;
    __amdgpu_buffer_rsrc_t rw[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)  // rows past the matrix read as zeros
        rw[h] = make_rsrc(scalar_ptr(wbase + (size_t)row[h] * K),
                          __builtin_amdgcn_readfirstlane((uint32_t)rows[h] * (uint32_t)K));
    const int crow = 8 * wave + lane / 8;
    const int chunk = (lane % 8) ^ ((crow / 2) % 8);
    uint32_t woff[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        woff[i] = (uint32_t)(64 * i + crow) * (uint32_t)K + 16u * chunk;
    uint32_t xrow[kXi];  // token rows
#pragma unroll
    for (int i = 0; i < kXi; ++i)
        xrow[i] = (uint32_t)src_row(P, t.r0 + t.m0 + min(64 * i + crow, t.M - 1));
    const uint8_t *x8 = scalar_ptr(P.x8);
    // every 64 tokens' scales are copied by one wave of kXi (and again by the others: no
    // branch in the pipeline)
    const int srow = kTok > 64 ? wave % kXi : 0;
    const float *xsp = P.xs + src_row(P, t.r0 + t.m0 + min(srow * 64 + lane, t.M - 1)) * KB;
    const uint64_t zeros = (uint64_t)(uintptr_t)&kZeros;
    auto copy = [&](int kb, uint32_t buf) {
        char *dst = smem + buf;
        // K's last block may be shorter: zeros there, for the weights by an offset out of
        // range, for the tokens from kZeros
        const bool in = kb * kBlk + 16 * chunk < K;
        const uint64_t pick = in ? ~0ull : 0ull;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rw[h], (__attribute__((address_space(3))) void *)(dst + h * kHalf * kBlk + (64 * i + 8 * wave) * kBlk), 16,
                    in ? woff[i] : 0x80000000u, (uint32_t)kb * kBlk, 0, 0);
#pragma unroll
        for (int i = 0; i < kXi; ++i) {
            const uint64_t src = (uint64_t)(uintptr_t)(x8 + (uint32_t)kb * kBlk + 16 * chunk) + (uint64_t)xrow[i] * (uint32_t)K;
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void *)(uintptr_t)((src & pick) | (zeros & ~pick)),
                (__attribute__((address_space(3))) void *)(dst + kStageW + (64 * i + 8 * wave) * kBlk), 16, 0, 0);
        }
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(xsp + kb),
                                         (__attribute__((address_space(3))) void *)(dst + kStage + srow * 256), 4, 0, 0);
    };

    const uint32_t swz = 16u * (uint32_t)(g ^ ((j / 2) % 8));  // chunk g of rows j, j + 16, ...; chunk g + 4 is at swz ^ 64
    const uint32_t arow = (uint32_t)(32 * wr + j) * kBlk, brow = kStageW + (uint32_t)(wt * 16 * TTN + j) * kBlk;
    float4v acc[4][TTN];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < TTN; ++c)
            acc[r][c] = float4v{0.f, 0.f, 0.f, 0.f};
    // LDS addresses of a buffer: chunks g and g + 4 of the wave's first weight and token
    // row, and the scale of its first token.  Everything else is a constant further; the
    // empty asm keeps the compiler from holding each sum in a register of its own.
    struct At {
        uint32_t a[2], b[2], s;
    };
    auto at = [&](uint32_t buf) {
        const uint32_t sb = base + buf;
        At v = {{sb + arow + swz, sb + arow + (swz ^ 64u)},
                {sb + brow + swz, sb + brow + (swz ^ 64u)},
                sb + kStage + 4u * (uint32_t)(wt * 16 * TTN + j)};
        asm volatile("" : "+v"(v.a[0]), "+v"(v.a[1]), "+v"(v.b[0]), "+v"(v.b[1]), "+v"(v.s));
        return v;
    };
    // half 0: chunk g, half 1: chunk g + 4
    auto read_a = [&](const At &v, int r, int half) {
        return lds_b128(v.a[half] + (r >> 1) * kHalf * kBlk + (r & 1) * 16 * kBlk);
    };
    auto read_b = [&](const At &v, int c, int half) { return lds_b128(v.b[half] + c * 16 * kBlk); };
    auto read_sx = [&](const At &v, int c) {
        return *reinterpret_cast<const __attribute__((address_space(3))) float *>((uintptr_t)(v.s + 64u * c));
    };

    // Both pipelines read their fragments ahead.  When every read of a stage has been
    // sent, one barrier (turn) says that the stage's buffer is free and that the next
    // stage has landed; the next stage's first fragments are read while the rest of this
    // one multiplies.  The products of a step are scaled and added before the MFMA that
    // writes their registers again.
    static_assert(TTN % 2 == 0, "b's two register sets alternate across stages");
#pragma unroll
    for (int i = 0; i < NB; ++i)
        copy(min(i, KB - 1), i * kBuffer);
    __builtin_amdgcn_s_waitcnt(wait_vm<(NB - 1) * kCopies>());
    asm volatile("s_barrier" ::: "memory");
    const At bufs[3] = {at(0), at(kBuffer), at(NB > 2 ? 2 * kBuffer : 0)};
    // the weights' scales: scalar loads, complete with the LDS reads at a turn
    auto scale = [&](int h, int kb) {
        return *reinterpret_cast<const __attribute__((address_space(4))) float *>((uintptr_t)(ws[h] + kb));
    };
    float sw[2] = {scale(0, 0), scale(1, 0)}, swn[2] = {0.f, 0.f};
    auto turn = [&](int kb, uint32_t buf) {  // the barrier of stage kb, whose buffer is buf
        const int k1 = min(kb + 1, KB - 1);
        swn[0] = scale(0, k1);
        swn[1] = scale(1, k1);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(wait_vm<(NB - 2) * kCopies>());  // stage kb + 1 has landed
        asm volatile("s_barrier" ::: "memory");
        copy(min(kb + NB, KB - 1), buf);
    };
    auto run = [&](auto &&stage) {
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
    };

    if constexpr (EXACT) {
        // Quarter q of a stage: the 32 columns of one fp16 MFMA for all 4 x TTN products,
        // whose sums over the four quarters stay in p.  Between the MFMAs, one conversion
        // for each: the next token tile's quarter, and the next quarter of the weights
        // (the vector unit would otherwise be idle in the 16 clocks of an MFMA, and a run
        // of conversions would leave the matrix unit idle).  A fragment's register is read
        // again right after its last conversion, 4 TTN MFMAs before it is needed.
        u32x4 a[2][4], b[2], ra[4], rb[TTN];
        float4v p[4][TTN];
        float sx[TTN], swp[2] = {0.f, 0.f};  // of the products in p
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            ra[r] = read_a(bufs[0], r, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a[0][r][i] = half2_of(ra[r], 0, i);
        }
#pragma unroll
        for (int c = 0; c < TTN; ++c) {
            rb[c] = read_b(bufs[0], c, 0);
            sx[c] = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                p[r][c] = float4v{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            b[0][i] = half2_of(rb[0], 0, i);
        auto add = [&](int r, int c) {
            const float f = sx[c] * swp[r >> 1];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[r][c][i] = __builtin_fmaf(p[r][c][i], f, acc[r][c][i]);
        };
        auto stage = [&](auto par, int kb) {
            constexpr int Q = decltype(par)::value;  // buffer of this stage
            const At &sb = bufs[Q], &sn = bufs[(Q + 1) % NB];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (q == 2)
                    turn(kb, Q * kBuffer);
#pragma unroll
                for (int c = 0; c < TTN; ++c) {
                    const int cur = (q * TTN + c) % 2;
                    const int nc = (c + 1) % TTN, nq = c + 1 < TTN ? q : q + 1;  // the next token fragment
                    constexpr int kA = 4 / TTN > 1 ? 4 / TTN : 1;                 // weight tiles converted beside c
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const half8 av = __builtin_bit_cast(half8, a[q % 2][r]), bv = __builtin_bit_cast(half8, b[cur]);
                        if (q == 0) {
                            add(r, c);
                            p[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, bv, float4v{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
                        } else {
                            p[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, bv, p[r][c], 0, 0, 0);
                        }
                        b[1 - cur][r] = half2_of(rb[nc], nq % 2, r);
#pragma unroll
                        for (int w = 0; w < kA; ++w)
                            if (kA * c + w < 4)
                                a[(q + 1) % 2][kA * c + w][r] = half2_of(ra[kA * c + w], (q + 1) % 2, r);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    // fragments whose two quarters are converted: the next half, of this
                    // stage or the next
                    if (nq % 2 == 1)
                        rb[nc] = nq == 1 ? read_b(sb, nc, 1) : read_b(sn, nc, 0);
                    if (q % 2 == 0) {
#pragma unroll
                        for (int w = 0; w < kA; ++w)
                            if (kA * c + w < 4)
                                ra[kA * c + w] = q == 0 ? read_a(sb, kA * c + w, 1) : read_a(sn, kA * c + w, 0);
                    }
                    if (q == 1)
                        sx[c] = read_sx(sb, c);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            swp[0] = sw[0];
            swp[1] = sw[1];
            sw[0] = swn[0];
            sw[1] = swn[1];
        };
        run(stage);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < TTN; ++c)
                add(r, c);
    } else {
        // Step c multiplies token tile c by the four weight tiles.  Each MFMA is preceded
        // by the four additions of the product that its registers held; b is read a step
        // ahead.
        Frag8 a[NB][2], a2[2], b[2];  // weight tiles 0, 1 in a set for each buffer; 2, 3 in one
        float4v p[4];
        float sx[2], f[2] = {0.f, 0.f};
        auto frag_a = [&](const At &v, int r) { return Frag8{read_a(v, r, 0), read_a(v, r, 1)}; };
        auto frag_b = [&](const At &v, int c) { return Frag8{read_b(v, c, 0), read_b(v, c, 1)}; };
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            (r < 2 ? a[0][r] : a2[r - 2]) = frag_a(bufs[0], r);
            p[r] = float4v{0.f, 0.f, 0.f, 0.f};
        }
        b[0] = frag_b(bufs[0], 0);
        sx[0] = read_sx(bufs[0], 0);
        auto add = [&](int r, int c) {  // the product in p[r] is tile c's
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[r][c][i] = __builtin_fmaf(p[r][i], f[r >> 1], acc[r][c][i]);
        };
        auto stage = [&](auto par, int kb) {
            constexpr int Q = decltype(par)::value;  // buffer of this stage
            const At &sb = bufs[Q], &sn = bufs[(Q + 1) % NB];
#pragma unroll
            for (int c = 0; c < TTN; ++c) {
                if (c + 1 < TTN) {  // (in step TTN - 2: before the turn)
                    b[(c + 1) % 2] = frag_b(sb, c + 1);
                    sx[(c + 1) % 2] = read_sx(sb, c + 1);
                }
                if (c == TTN - 2)
                    turn(kb, Q * kBuffer);
                if (c + 1 == TTN) {
                    b[0] = frag_b(sn, 0);
                    sx[0] = read_sx(sn, 0);
                }
                if (c >= TTN - 2)
                    a[(Q + 1) % NB][c + 2 - TTN] = frag_a(sn, c + 2 - TTN);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    add(r, c == 0 ? TTN - 1 : c - 1);
                    p[r] = block_product(r < 2 ? a[Q][r] : a2[r - 2], b[c % 2]);
                    __builtin_amdgcn_sched_barrier(0);
                    if (r >= 2 && c == TTN - 1)
                        a2[r - 2] = frag_a(sn, r);
                }
                f[0] = sx[c % 2] * sw[0];
                f[1] = sx[c % 2] * sw[1];
            }
            sw[0] = swn[0];
            sw[1] = swn[1];
        };
        run(stage);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            add(r, TTN - 1);
    }

    // ---- epilogue
    const bool active = wt * 16 * TTN < t.M;  // this half of the tile has tokens
    if constexpr (ACT) {
        uint32_t *amax = reinterpret_cast<uint32_t *>(smem);  // [4 row groups][kTok]
        __syncthreads();                                      // the last stage is read
        float a[2][TTN][4];
        const int f0 = t.nt * kHalf + 32 * wr + 4 * g;
        if (active) {
#pragma unroll
            for (int c = 0; c < TTN; ++c) {
                uint32_t mx = 0;
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a[r][c][i] = silu_mul32(acc[r][c][i], acc[2 + r][c][i]);
                        if (f0 + 16 * r + i < P.F)
                            mx = max(mx, mag(a[r][c][i]));
                    }
                mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16, kWave));
                mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32, kWave));
                if (g == 0)
                    amax[wr * kTok + wt * 16 * TTN + 16 * c + j] = mx;
            }
        }
        __syncthreads();
        if (active) {
#pragma unroll
            for (int c = 0; c < TTN; ++c) {
                const int tok = wt * 16 * TTN + 16 * c + j;
                uint32_t mx = 0;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    mx = max(mx, amax[w * kTok + tok]);
                const float s = scale_of(mx), inv = 1.0f / s;
                if (tok < t.M) {
                    const size_t orow = (size_t)(t.r0 + t.m0 + tok);
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (f0 + 16 * r < P.F)  // F is a multiple of 16
                            *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(P.out) + orow * P.F + f0 + 16 * r) =
                                to_e4m3x4(a[r][c][0] * inv, a[r][c][1] * inv, a[r][c][2] * inv, a[r][c][3] * inv);
                    if (wr == 0 && g == 0)
                        P.os[orow * fb + t.nt] = s;
                }
            }
        }
    } else if (active) {
#pragma unroll
        for (int c = 0; c < TTN; ++c) {
            const int tok = wt * 16 * TTN + 16 * c + j;
            if (tok >= t.M)
                continue;
            const size_t orow = (size_t)(t.r0 + t.m0 + tok);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int n = row[r >> 1] + 32 * wr + 16 * (r & 1) + 4 * g;
                if (n < P.N)
                    store4(P, orow, n, acc[r][c]);
            }
        }
    }
}

// Tokens of a tile.  fp16 fragments take twice the registers: 128 tokens (EXTOK).
template <bool EXACT>
constexpr int kTileTok = EXACT ? 128 : 256;

template <bool EXACT, bool ACT>
__global__ void __launch_bounds__(kThreads) fp8_tile_kernel(const TileParams T)
{
    __shared__ __attribute__((aligned(1024))) char smem[kLds];
    Tile t = {0, 0, 0, 0, 0};
    if (!resolve(T, kTileTok<EXACT>, reinterpret_cast<int *>(smem), t))
        return;
    __syncthreads();  // the scan is read
    // the same in every lane: into scalar registers (here, behind the branch that the
    // compiler takes to depend on the lane)
    t.e = __builtin_amdgcn_readfirstlane(t.e);
    t.r0 = __builtin_amdgcn_readfirstlane(t.r0);
    t.m0 = __builtin_amdgcn_readfirstlane(t.m0);
    t.M = __builtin_amdgcn_readfirstlane(t.M);
    t.nt = __builtin_amdgcn_readfirstlane(t.nt);
    if (!EXACT && t.M > 128)
        tile<EXACT, ACT, EXACT ? 2 : 8>(T, t, smem);
    else if (t.M > 64)
        tile<EXACT, ACT, 4>(T, t, smem);
    else
        tile<EXACT, ACT, 2>(T, t, smem);
}

}  // namespace

hipError_t launch_fp8_tile(const Fp8Params &P, int most, bool act, bool exact, hipStream_t s)
{
    if (most <= kStreamMax)
        return hipSuccess;
    // token tiles: at most one for each `tok` rows, and one more for each served expert
    const int tok = exact ? kTileTok<true> : kTileTok<false>;
    const int served = P.E < P.R / (kStreamMax + 1) ? P.E : P.R / (kStreamMax + 1);
    if (served == 0)
        return hipSuccess;
    const long MT = (long)(P.R / tok) + served;
    const TileParams T{P, act ? (P.F + kHalf - 1) / kHalf : (P.N + 2 * kHalf - 1) / (2 * kHalf)};
    const long grid = (MT * T.NT + kXcds - 1) / kXcds * kXcds;
    if (grid > 0x7FFFFFFFl)
        return hipErrorInvalidValue;
    if (act)
        hipLaunchKernelGGL((fp8_tile_kernel<true, true>), dim3((unsigned)grid), dim3(kThreads), 0, s, T);
    else if (exact)
        hipLaunchKernelGGL((fp8_tile_kernel<true, false>), dim3((unsigned)grid), dim3(kThreads), 0, s, T);
    else
        hipLaunchKernelGGL((fp8_tile_kernel<false, false>), dim3((unsigned)grid), dim3(kThreads), 0, s, T);
    return hipGetLastError();
}

}  // namespace apmoe
