// norm.hip -- root-mean-square norm in front of the MoE layer: the residual's addition,
// the norm, and the row in 8 bits with its scales, in one pass over the data.
//
//   h = x + residual (fp32, stored in the residual's type), or x without one;
//   y = h * gamma / sqrt(mean(h^2) + eps);  y8, s = y in e4m3 with a scale per 128 columns.
//
// Bound by memory for many rows (8192 x 6144 bf16 with an fp32 residual: 114 us, 5.3 TB/s),
// by the latency of one load, sum and store for few (1 x 4096: 5 us, 2 to 3 of them the launch).
#include "fp8.h"
#include "launch_fp8.h"

namespace apmoe {
namespace {

struct NormParams {
    const void *x;
    const void *residual;
    void *h;
    const void *gamma;
    void *y;
    uint8_t *y8;
    float *ys;
    float eps;
    int T, H;
};

template <int DT>
__device__ inline void load8(const void *p, size_t at, float (&v)[8])
{
    if constexpr (DT == APMOE_F32) {
        const float4v a = *reinterpret_cast<const float4v *>(static_cast<const float *>(p) + at);
        const float4v b = *reinterpret_cast<const float4v *>(static_cast<const float *>(p) + at + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
        const u32x4 r = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p) + at);
        if constexpr (DT == APMOE_F16) {
            const half8 h = __builtin_bit_cast(half8, r);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = (float)h[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = __builtin_bit_cast(float, (i & 1) ? r[i / 2] & 0xFFFF0000u : r[i / 2] << 16);
        }
    }
}

// Stores 8 values in type DT and returns them as stored.
template <int DT>
__device__ inline void store8(void *p, size_t at, float (&v)[8])
{
    if constexpr (DT == APMOE_F32) {
        float4v a, b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = v[i];
            b[i] = v[4 + i];
        }
        *reinterpret_cast<float4v *>(static_cast<float *>(p) + at) = a;
        *reinterpret_cast<float4v *>(static_cast<float *>(p) + at + 4) = b;
    } else if constexpr (DT == APMOE_F16) {
        half8 h;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[i] = (_Float16)v[i];
            v[i] = (float)h[i];
        }
        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p) + at) = __builtin_bit_cast(u32x4, h);
    } else {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = to_bf16(v[2 * i]), hi = to_bf16(v[2 * i + 1]);
            r[i] = lo | hi << 16;
            v[2 * i] = __builtin_bit_cast(float, lo << 16);
            v[2 * i + 1] = __builtin_bit_cast(float, hi << 16);
        }
        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p) + at) = r;
    }
}

constexpr int kNoRes = -1;
constexpr int kNormThreads = 256;
constexpr uint32_t kNormGrid = 1u << 20;  // workgroups in x; a dimension has fewer than 2^32 threads

// TPR threads hold a row, VPT chunks of 8 columns each (chunk t + v * TPR); a workgroup
// of max(TPR, 256) threads holds max(1, 256 / TPR) rows.  The row stays in registers
// between the sum and the output, so x and the residual are read once.  The sum of
// squares and y are fp64: squares of fp32 / bf16 values leave fp32's range, and a value
// next to a border of e4m3 then rounds as its quotient in fp32 does.  fp64 runs at the rate of
// unpacked fp32 here and the kernel is bound by memory.
template <int XT, int RT, int TPR, int VPT>
__global__ void __launch_bounds__(TPR > kNormThreads ? TPR : kNormThreads) norm_kernel(const NormParams P)
{
    constexpr int NT = TPR > kNormThreads ? TPR : kNormThreads;
    constexpr int kRows = NT / TPR;
    constexpr int kWavesPerRow = TPR / kWave;
    const int tid = threadIdx.x, t = tid % TPR;
    const uint32_t row = (blockIdx.y * kNormGrid + blockIdx.x) * kRows + tid / TPR;
    const int chunks = P.H / 8;
    const bool live = row < (uint32_t)P.T;  // the threads of a row past the last one only meet the barrier
    const size_t base = (size_t)(live ? row : 0) * P.H;
    float h[VPT][8];
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = t + v * TPR;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h[v][i] = 0.f;
        if (live && c < chunks)
            load8<XT>(P.x, base + 8 * c, h[v]);
    }
    if constexpr (RT != kNoRes) {
        float r[VPT][8];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = t + v * TPR;
            if (live && c < chunks)
                load8<RT>(P.residual, base + 8 * c, r[v]);
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int c = t + v * TPR;
            if (live && c < chunks) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    h[v][i] += r[v][i];
                store8<RT>(P.h, base + 8 * c, h[v]);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum = __builtin_fma((double)h[v][i], (double)h[v][i], sum);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        sum += __shfl_xor(sum, d, kWave);
    if constexpr (kWavesPerRow > 1) {
        __shared__ double part[NT / kWave];
        if (tid % kWave == 0)
            part[tid / kWave] = sum;
        __syncthreads();
        sum = 0.0;
#pragma unroll
        for (int w = 0; w < kWavesPerRow; ++w)
            sum += part[tid / TPR * kWavesPerRow + w];
    }
    if (!live)
        return;
    const double rstd = 1.0 / sqrt(sum / (double)P.H + (double)P.eps);
    const int groups = (P.H + kBlk - 1) / kBlk;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const int c = t + v * TPR;
        const bool in = c < chunks;
        double y[8];
        float g[8];
        if (in)
            load8<XT>(P.gamma, 8 * (size_t)c, g);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = in ? (double)h[v][i] * rstd * (double)g[i] : 0.0;
        if (P.y8) {
            // 16 lanes hold a group; magnitudes as integers (mag)
            uint64_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint64_t b = __builtin_bit_cast(uint64_t, y[i]) & 0x7FFFFFFFFFFFFFFFull;
                m = b > m ? b : m;
            }
#pragma unroll
            for (int d = 8; d >= 1; d >>= 1) {
                const uint64_t o = (uint64_t)__shfl_xor((unsigned long long)m, d, kWave);
                m = o > m ? o : m;
            }
            float s = (float)(__builtin_bit_cast(double, m) / (double)kE4m3Max);
            s = s < kScaleMin ? kScaleMin : s;
            if (in) {
                const double inv = 1.0 / (double)s;
                float q[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    q[i] = (float)(y[i] * inv);
                u32x2 o;
                o[0] = to_e4m3x4(q[0], q[1], q[2], q[3]);
                o[1] = to_e4m3x4(q[4], q[5], q[6], q[7]);
                *reinterpret_cast<u32x2 *>(P.y8 + base + 8 * c) = o;
                if (c % 16 == 0)
                    P.ys[(size_t)row * groups + c / 16] = s;
            }
        }
        if (P.y && in) {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i] = (float)y[i];
            store8<XT>(P.y, base + 8 * c, o);
        }
    }
}

template <int XT, int RT, int TPR, int VPT>
hipError_t norm_launch(const NormParams &P, hipStream_t s)
{
    constexpr int NT = TPR > kNormThreads ? TPR : kNormThreads;
    constexpr int kRows = NT / TPR;
    const uint32_t blocks = ((uint32_t)P.T + kRows - 1) / kRows;
    hipLaunchKernelGGL((norm_kernel<XT, RT, TPR, VPT>),
                       dim3(blocks < kNormGrid ? blocks : kNormGrid, (blocks + kNormGrid - 1) / kNormGrid), dim3(NT), 0,
                       s, P);
    return hipGetLastError();
}

template <int XT, int RT>
hipError_t norm_shape(const NormParams &P, hipStream_t s)
{
    const int chunks = P.H / 8;
    // Few rows are a matter of latency: more threads a row (bf16 with an fp32 residual, both
    // outputs, 128 rows of 1024 3.4 us against 4.7, of 8192 6.1 against 8.5; 512 rows 4.4 and
    // 5.1, 14.0 and 15.4).  Many take the threads that are all in use and have more loads in
    // flight each (2048 rows of 4096 22 us against 28, 8192 rows of 4096 87 and 126, 5.3 TB/s).
    const bool few = P.T <= 512;
    if (chunks <= 64)
        return norm_launch<XT, RT, 64, 1>(P, s);
    if (chunks <= 128 && !few)
        return norm_launch<XT, RT, 64, 2>(P, s);
    if (chunks <= 256)
        return norm_launch<XT, RT, 256, 1>(P, s);
    if (chunks <= 512 && !few)
        return norm_launch<XT, RT, 256, 2>(P, s);
    if (chunks <= 1024 && !few)
        return norm_launch<XT, RT, 256, 4>(P, s);
    if (chunks <= 1024)
        return norm_launch<XT, RT, 1024, 1>(P, s);
    if (chunks <= 2048)
        return norm_launch<XT, RT, 1024, 2>(P, s);
    if (chunks <= 4096)
        return norm_launch<XT, RT, 1024, 4>(P, s);
    return norm_launch<XT, RT, 1024, 8>(P, s);
}

template <int XT>
hipError_t norm_res(const NormParams &P, int rt, hipStream_t s)
{
    if (!P.residual)
        return norm_shape<XT, kNoRes>(P, s);
    if (rt == APMOE_F16)
        return norm_shape<XT, APMOE_F16>(P, s);
    if (rt == APMOE_BF16)
        return norm_shape<XT, APMOE_BF16>(P, s);
    return norm_shape<XT, APMOE_F32>(P, s);
}

}  // namespace

hipError_t launch_norm(const void *x, int x_dtype, const void *residual, void *h, int res_dtype, const void *gamma,
                       float eps, int T, int H, void *y, uint8_t *y8, float *ys, hipStream_t s)
{
    const NormParams P{x, residual, h, gamma, y, y8, ys, eps, T, H};
    if (x_dtype == APMOE_F16)
        return norm_res<APMOE_F16>(P, res_dtype, s);
    if (x_dtype == APMOE_BF16)
        return norm_res<APMOE_BF16>(P, res_dtype, s);
    return norm_res<APMOE_F32>(P, res_dtype, s);
}

}  // namespace apmoe
