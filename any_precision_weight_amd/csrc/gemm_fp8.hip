// gemm_fp8.hip -- the experts' products on e4m3 weights with fp32 scales:
//
//   out[r][n] = sum_b xs[src(r)][b] * ws[e][n / 128][b] * sum_{c in block b} x8[src(r)][c] * w8[e][n][c]
//
// for the rows r of expert e, and the gate_up product with SiLU(gate) * up written in
// 8 bits.  A block's inner sum comes from the matrix units, started from zero
// (block_product); its fp32 result is scaled by xs * ws and added to fp32 accumulators.
//
// Stream product: weights go from HBM to the matrix units through registers, each
// weight byte read once per 32 rows; a wave holds two 16-row weight tiles, kDepth
// blocks ahead.  Bound by the weights' bytes (gate_up of 16 tokens, 8 experts of 2 x 14336 x
// 4096: 157 us, 6.0 TB/s), where they are few by the latency of a wave's blocks (6144 x 4096
// for 8 tokens 11 us, 2.3 TB/s).
#include <algorithm>

#include "gemm_fp8.h"
#include "launch_fp8.h"
#include "stream_fp8.h"

namespace apmoe {
namespace {

constexpr int kDepth = 2;  // column blocks requested ahead
constexpr int kStreamWaves = 8;
constexpr int kStreamRows = 32;  // weight rows of a wave
constexpr int kCus = 256;

// blockIdx.x: weight rows, blockIdx.y: expert, blockIdx.z: 16 TT of its rows.  KS waves
// share a wave's 32 weight rows, a KS-th of the columns each; their sums meet in LDS in the
// order of the parts.
template <int KS, int TT>
__device__ __attribute__((always_inline)) inline void stream_tokens(const Fp8Params &P, int e, int r0, int m,
                                                                   float *red)
{
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int j = lane & 15, g = lane >> 4;
    const uint32_t woff = 16u * line_chunk(j, g);
    const int kp = wave % KS;
    const int n0 = ((int)blockIdx.x * (kStreamWaves / KS) + wave / KS) * kStreamRows;
    const int KB = (P.K + kBlk - 1) / kBlk;
    // weight rows past the last repeat it; nothing of them is stored
    const int nl = P.N - 1;
    const int nb = (P.N + kBlk - 1) / kBlk;
    const float *sc = P.ws + (size_t)e * nb * KB;
    const uint8_t *wbase[2], *xr[TT];
    uint32_t wo[2][2];
    const float *wsc[2], *xsc[TT];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int nr = min(n0 + 16 * r, nl);
        wbase[r] = P.w8 + ((size_t)e * P.N + nr) * P.K;
        wo[r][0] = (uint32_t)min(j % 8, nl - nr) * (uint32_t)P.K + woff;
        wo[r][1] = (uint32_t)min(8 + j % 8, nl - nr) * (uint32_t)P.K + woff;
        wsc[r] = sc + (size_t)(nr / kBlk) * KB;
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const size_t row = src_row(P, r0 + min(16 * t + j, m - 1));
        xr[t] = P.x8 + row * P.K + 16 * g;
        xsc[t] = P.xs + row * KB;
    }
    float4v acc[2][TT];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
            acc[r][t] = float4v{0.f, 0.f, 0.f, 0.f};
    const int per = (KB + KS - 1) / KS;
    stream_product<2, TT, kDepth>(wbase, wo, wsc, xr, xsc, kp * per, min(KB, (kp + 1) * per), P.K, 16 * g, (int)woff, 4 * wave + (int)blockIdx.x, acc);
    if constexpr (KS > 1) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t)
                *reinterpret_cast<float4v *>(red + ((wave * 2 + r) * TT + t) * 256 + lane * 4) = acc[r][t];
        __syncthreads();
        if (kp != 0)
            return;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int p = 1; p < KS; ++p)
                    acc[r][t] += *reinterpret_cast<const float4v *>(red + (((wave + p) * 2 + r) * TT + t) * 256 + lane * 4);
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int tok = 16 * t + j;
        if (tok >= m)
            continue;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int n = n0 + 16 * r + 4 * g;
            if (n < P.N)
                store4(P, (size_t)(r0 + tok), n, acc[r][t]);
        }
    }
}

template <int KS, int TT>
__global__ void __launch_bounds__(kStreamWaves *kWave, TT == 1 ? 4 : 2) stream_kernel(const Fp8Params P)
{
    __shared__ __attribute__((aligned(16))) float red[KS > 1 ? kStreamWaves * 2 * TT * 256 : 4];
    const int e = blockIdx.y;
    int r0, m;
    expert_rows(P, e, r0, m);
    constexpr int kRows = 16 * TT;
    for (int c = kRows * (int)blockIdx.z; c < m; c += kRows * (int)gridDim.z) {
        const int n = min(m - c, kRows);
        if (TT == 2 && n > 16)
            stream_tokens<KS, 2>(P, e, r0 + c, n, red);
        else
            stream_tokens<KS, 1>(P, e, r0 + c, n, red);
        if (KS > 1)
            __syncthreads();  // red is read
    }
}

// gate_up: a wave holds NP pairs of a tile of 16 gate rows and the tile of the matching up
// rows, the workgroup the 128 + 128 rows behind one group of 128 values of a8, whose scale
// needs all of them.
template <int TT, int NP>
__device__ __attribute__((always_inline)) inline void stream_act_tokens(const Fp8Params &P, int e, int r0, int m,
                                                                       uint32_t *amax)
{
    constexpr int kWaves = kStreamWaves / NP;
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int j = lane & 15, g = lane >> 4;
    const uint32_t woff = 16u * line_chunk(j, g);
    const int fw = (int)blockIdx.x * kBlk + 16 * NP * wave;
    const int KB = (P.K + kBlk - 1) / kBlk, fb = (P.F + kBlk - 1) / kBlk;
    const uint8_t *wbase[2 * NP], *xr[TT];
    uint32_t wo[2 * NP][2];
    const float *wsc[2 * NP], *xsc[TT];
#pragma unroll
    for (int r = 0; r < 2 * NP; ++r) {
        const int h = r % 2, fc = min(fw + 16 * (r / 2), P.F - 16);  // F is a multiple of 16
        wbase[r] = P.w8 + ((size_t)e * P.N + (size_t)h * P.F + fc) * P.K;
        wo[r][0] = (uint32_t)(j % 8) * (uint32_t)P.K + woff;
        wo[r][1] = (uint32_t)(8 + j % 8) * (uint32_t)P.K + woff;
        wsc[r] = P.ws + ((size_t)(2 * e + h) * fb + blockIdx.x) * KB;
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const size_t row = src_row(P, r0 + min(16 * t + j, m - 1));
        xr[t] = P.x8 + row * P.K + 16 * g;
        xsc[t] = P.xs + row * KB;
    }
    float4v acc[2 * NP][TT];
#pragma unroll
    for (int r = 0; r < 2 * NP; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t)
            acc[r][t] = float4v{0.f, 0.f, 0.f, 0.f};
    stream_product<2 * NP, TT, kDepth>(wbase, wo, wsc, xr, xsc, 0, KB, P.K, 16 * g, (int)woff, 4 * wave + (int)blockIdx.x,
                                       acc);
    float4v a[NP][TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        uint32_t mx = 0;
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[p][t][i] = silu_mul32(acc[2 * p][t][i], acc[2 * p + 1][t][i]);
                mx = max(mx, fw + 16 * p < P.F ? mag(a[p][t][i]) : 0u);
            }
        mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16, kWave));
        mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32, kWave));
        if (g == 0)
            amax[(wave * TT + t) * 16 + j] = mx;
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        uint32_t mx = 0;
#pragma unroll
        for (int v = 0; v < kWaves; ++v)
            mx = max(mx, amax[(v * TT + t) * 16 + j]);
        const float s = scale_of(mx), inv = 1.0f / s;
        const int tok = 16 * t + j;
        if (tok < m) {
            const size_t row = (size_t)(r0 + tok);
#pragma unroll
            for (int p = 0; p < NP; ++p)
                if (fw + 16 * p < P.F)
                    *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(P.out) + row * P.F + fw + 16 * p + 4 * g) =
                        to_e4m3x4(a[p][t][0] * inv, a[p][t][1] * inv, a[p][t][2] * inv, a[p][t][3] * inv);
            if (wave == 0 && g == 0)
                P.os[row * fb + blockIdx.x] = s;
        }
    }
}

template <int TT, int NP>
__global__ void __launch_bounds__(kStreamWaves / NP *kWave, NP == 2 ? 3 : TT == 1 ? 4 : 2)
    stream_act_kernel(const Fp8Params P)
{
    __shared__ uint32_t amax[kStreamWaves / NP * TT * 16];
    const int e = blockIdx.y;
    int r0, m;
    expert_rows(P, e, r0, m);
    constexpr int kRows = 16 * TT;
    for (int c = 0; c < m; c += kRows) {
        const int n = min(m - c, kRows);
        if (TT == 2 && n > 16)
            stream_act_tokens<2, NP>(P, e, r0 + c, n, amax);
        else
            stream_act_tokens<1, NP>(P, e, r0 + c, n, amax);
        __syncthreads();  // amax is read
    }
}

// Whether a call takes the tile product or the stream product.
//
// The product.  Few tiles leave most of the device idle, and the stream product, split over
// K and over chunks of 32 rows, fills it although each chunk reads the weights again.  Up to
// 64 chunks of 256 weight rows it is ahead (weights from HBM, to bf16 as chunks and as tiles,
// us; to fp32 the tiles are up to 5 slower): 64 rows of 6144 x 4096 (48 chunks) 26 and 38, 128
// of 4096 x 14336 (64) 70 and 116, 512 of 1024 x 8192 (64) 44 and 58, 64 tokens of 2 of 8
// experts of 1024 x 2048 (44) 10 and 17; 256 rows of 2048 x 2048 (64) 17 and 15.3, to fp32 17
// and 20.  With more and above 32 tokens tiles: 128 rows of 6144 x 4096 (96 chunks) 43 and 37,
// 192 of 4096 x 14336 (96) 131 and 113, 8 experts of 4096 x 7168, 128 tokens of 2, 127 and 61.
// Experts with a few rows each stream a little faster if the routing is even (60 of 2048 x
// 1408, 64 tokens of 4, 35 us against 40), and much slower if it is not, when few experts'
// waves are left (the same with most of the experts idle 40 against 16; 64 of 1024 x 2048, 64
// tokens of 2, 44 against 20).
//
// gate_up, whose stream product is not split over K.  More than 32 rows take tiles (E = 1,
// 48 rows of 2 x 2048 x 4096: 77 us streamed, 33 as tiles), and more than 16 where every CU
// has one at most (24 rows of that one expert 69 and 31; 8 experts of 2 x 2048 x 7168, 32
// tokens of 2, 128 tiles, 82 and 56; of 2 x 4096 x 4096, 256 tiles, 53 and 67).
bool takes_tiles(const Fp8Params &P, int most, bool act)
{
    if (act)
        return most > kStreamMax || (most > 16 && fp8_tiles(P, act, fp8_tile_tokens(true)) < kCus);
    return most > kStreamMax && fp8_tiles(P, act, kStreamMax) > 64;
}

}  // namespace

hipError_t launch_gemm_fp8(const uint8_t *x8, const float *xs, const uint8_t *w8, const float *ws, int E, int N, int K,
                           int gather, const int32_t *perm, const int32_t *offsets, int topk, int R, void *out,
                           int out_dtype, bool exact, hipStream_t s)
{
    const Fp8Params P{x8, xs, w8, ws, perm, offsets, out, nullptr, E, N, K, topk, gather, out_dtype, R, 0};
    const int most = most_rows(P);
    if (takes_tiles(P, most, false))
        return launch_fp8_tile(P, false, exact, s);
    const unsigned chunks = (unsigned)(most + kStreamMax - 1) / kStreamMax;
    // KS: enough waves to fill the device, 8 on a CU (KS = 1, 2, 4, 8: 6144 x 4096, 192 waves,
    // 47, 26, 16, 10.9 us; 28672 x 4096, 896 waves, 47, 29, 32, 36; 8 experts of 4096 x 2048,
    // 1024 waves, 23, 14.8, 17, 21; 60 of 2048 x 1408, 3840 waves, 31, 31, 30, 40).
    const int active = E < R ? E : R;
    const long parts = std::min((long)active * chunks, (long)(R - active) / kStreamMax + active);  // that have rows
    const long waves = parts * ((N + kStreamRows - 1) / kStreamRows);
    const int KB = (K + kBlk - 1) / kBlk;
    auto go = [&](auto ks) {
        constexpr int KS = decltype(ks)::value;
        const int rows = kStreamWaves / KS * kStreamRows;
        const dim3 grid((N + rows - 1) / rows, E, chunks), block(kStreamWaves * kWave);
        if (most > 16)
            hipLaunchKernelGGL((stream_kernel<KS, 2>), grid, block, 0, s, P);
        else
            hipLaunchKernelGGL((stream_kernel<KS, 1>), grid, block, 0, s, P);
    };
    if (waves >= 2048 || KB < 4)
        go(std::integral_constant<int, 1>{});
    else if (waves >= 768 || KB < 8)
        go(std::integral_constant<int, 2>{});
    else if (waves >= 384 || KB < 16)
        go(std::integral_constant<int, 4>{});
    else
        go(std::integral_constant<int, 8>{});
    return hipGetLastError();
}

hipError_t launch_gemm_act_fp8(const uint8_t *x8, const float *xs, const uint8_t *w8, const float *ws, int E, int F,
                               int K, int gather, const int32_t *perm, const int32_t *offsets, int topk, int R,
                               uint8_t *a8, float *as, hipStream_t s)
{
    const Fp8Params P{x8, xs, w8, ws, perm, offsets, a8, as, E, 2 * F, K, topk, gather, 0, R, F};
    const dim3 grid((F + kBlk - 1) / kBlk, E);
    const int most = most_rows(P);
    if (takes_tiles(P, most, true))
        return launch_fp8_tile(P, true, true, s);
    // Up to 16 rows four waves with two pairs of tiles each, three workgroups on a CU (16 tokens,
    // 8 experts of 2 x 14336 x 4096: 172 us, eight waves with one pair 176); more rows have no
    // registers for that.
    if (most > 16)
        hipLaunchKernelGGL((stream_act_kernel<2, 1>), grid, dim3(kStreamWaves * kWave), 0, s, P);
    else
        hipLaunchKernelGGL((stream_act_kernel<1, 2>), grid, dim3(kStreamWaves / 2 * kWave), 0, s, P);
    return hipGetLastError();
}

}  // namespace apmoe
