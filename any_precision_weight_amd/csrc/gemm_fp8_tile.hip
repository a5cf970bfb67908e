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
constexpr int kMaxTok = 256;           // tokens of a tile
constexpr int kGroup = 8;              // weight tiles that share their token tiles through an XCD's L2
constexpr uint32_t kStageW = 2 * kHalf * kBlk;
constexpr uint32_t kStage = kStageW + kMaxTok * kBlk;
constexpr uint32_t kScales = kMaxTok * 4;
constexpr uint32_t kLds = 2 * (kStage + kScales);

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
__device__ inline bool resolve(const TileParams &T, int *scan, Tile &t)
{
    const Fp8Params &P = T.p;
    const int tid = threadIdx.x;
    int n = 0;
    if (tid < P.E) {
        int r0, m;
        expert_rows(P, tid, r0, m);
        n = m > kStreamMax ? (m + kMaxTok - 1) / kMaxTok : 0;
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
    const int m0 = (u - (lo > 0 ? scan[lo - 1] : 0)) * kMaxTok;
    t.e = __builtin_amdgcn_readfirstlane(lo);
    t.r0 = __builtin_amdgcn_readfirstlane(r0);
    t.m0 = __builtin_amdgcn_readfirstlane(m0);
    t.M = __builtin_amdgcn_readfirstlane(min(kMaxTok, m - m0));
    t.nt = __builtin_amdgcn_readfirstlane(k * kGroup + rem % gs);
    return true;
}

template <bool EXACT>
struct Operand;
template <>
struct Operand<true> {
    typedef Frag16 type;
    static __device__ inline Frag16 of(const Frag8 &f) { return to_frag16(f); }
};
template <>
struct Operand<false> {
    typedef Frag8 type;
    static __device__ inline Frag8 of(const Frag8 &f) { return f; }
};

// TTN: 16-token tiles of a wave.  EXACT: fp16 products (block_product).
template <bool EXACT, bool ACT, int TTN>
__device__ __attribute__((always_inline)) inline void tile(const TileParams &T, const Tile &t, char *smem)
{
    const Fp8Params &P = T.p;
    typedef Operand<EXACT> Op;
    constexpr int kTok = 32 * TTN;  // tokens of the tile
    constexpr int kXi = kTok > 64 ? kTok / 64 : 1;
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
        rw[h] = make_rsrc(wbase + (size_t)row[h] * K, (uint32_t)rows[h] * (uint32_t)K);
    const int crow = 8 * wave + lane / 8;
    const int chunk = (lane % 8) ^ ((crow / 2) % 8);
    uint32_t woff[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        woff[i] = (uint32_t)(64 * i + crow) * (uint32_t)K + 16u * chunk;
    const uint8_t *xp[kXi];
#pragma unroll
    for (int i = 0; i < kXi; ++i)
        xp[i] = P.x8 + src_row(P, t.r0 + t.m0 + min(64 * i + crow, t.M - 1)) * K + 16 * chunk;
    const bool scaler = wave * 64 < kTok;  // waves that copy the tokens' scales
    const float *xsp = P.xs;
    if (scaler)
        xsp += src_row(P, t.r0 + t.m0 + min(wave * 64 + lane, t.M - 1)) * KB;
    auto copy = [&](int kb, uint32_t buf) {
        char *dst = smem + buf;
        // K's last block may be shorter: zeros there, for the weights by an offset out of range
        const bool in = kb * kBlk + 16 * chunk < K;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rw[h], (__attribute__((address_space(3))) void *)(dst + h * kHalf * kBlk + (64 * i + 8 * wave) * kBlk), 16,
                    in ? woff[i] : 0x80000000u, (uint32_t)kb * kBlk, 0, 0);
#pragma unroll
        for (int i = 0; i < kXi; ++i) {
            const void *src = in ? (const void *)(xp[i] + (size_t)kb * kBlk) : (const void *)&kZeros;
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                             (__attribute__((address_space(3))) void *)(dst + kStageW + (64 * i + 8 * wave) * kBlk),
                                             16, 0, 0);
        }
        if (scaler)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(xsp + kb),
                                             (__attribute__((address_space(3))) void *)(dst + kStage + wave * 256), 4, 0, 0);
    };

    const uint32_t swz = 16u * (uint32_t)(g ^ ((j / 2) % 8));  // chunk g of rows j, j + 16, ...; chunk g + 4 is at swz ^ 64
    const uint32_t arow = (uint32_t)(32 * wr + j) * kBlk, brow = kStageW + (uint32_t)(wt * 16 * TTN + j) * kBlk;
    float4v acc[4][TTN];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < TTN; ++c)
            acc[r][c] = float4v{0.f, 0.f, 0.f, 0.f};
    const bool active = wt * 16 * TTN < t.M;

    copy(0, 0);
    uint32_t buf = 0;
    for (int kb = 0; kb < KB; ++kb) {
        // this stage has landed for every wave, and every wave is done with the other buffer
        __builtin_amdgcn_s_waitcnt(wait_vm<0>());
        asm volatile("s_barrier" ::: "memory");
        const uint32_t next = buf ^ (kStage + kScales);
        if (kb + 1 < KB)
            copy(kb + 1, next);
        if (active) {
            const uint32_t sb = base + buf;
            const float sw0 = ws[0][kb], sw1 = ws[1][kb];
            typename Op::type a[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t ad = sb + (r >> 1) * kHalf * kBlk + arow + (r & 1) * 16 * kBlk;
                a[r] = Op::of(Frag8{lds_b128(ad + swz), lds_b128(ad + (swz ^ 64u))});
            }
#pragma unroll
            for (int c = 0; c < TTN; ++c) {
                const uint32_t bd = sb + brow + c * 16 * kBlk;
                const typename Op::type b = Op::of(Frag8{lds_b128(bd + swz), lds_b128(bd + (swz ^ 64u))});
                const float sx = *reinterpret_cast<const __attribute__((address_space(3))) float *>(
                    (uintptr_t)(sb + kStage + 4u * (wt * 16 * TTN + 16 * c + j)));
                const float f0 = sx * sw0, f1 = sx * sw1;
                float4v p[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    p[r] = block_product(a[r], b);
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[r][c][i] = __builtin_fmaf(p[r][i], r < 2 ? f0 : f1, acc[r][c][i]);
            }
        }
        buf = next;
    }

    // ---- epilogue
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

template <bool EXACT, bool ACT>
__global__ void __launch_bounds__(kThreads) fp8_tile_kernel(const TileParams T)
{
    __shared__ __attribute__((aligned(1024))) char smem[kLds];
    Tile t;
    const bool mine = resolve(T, reinterpret_cast<int *>(smem), t);
    __syncthreads();  // the scan is read
    if (!mine)
        return;
    if (t.M > 128)
        tile<EXACT, ACT, 8>(T, t, smem);
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
    // token tiles: at most one per started kMaxTok rows of an expert with more than kStreamMax
    const int served = P.E < P.R / (kStreamMax + 1) ? P.E : P.R / (kStreamMax + 1);
    if (served == 0)
        return hipSuccess;
    const long MT = (long)(P.R / kMaxTok) + served;
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
