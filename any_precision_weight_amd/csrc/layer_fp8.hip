// layer_fp8.hip -- the whole layer on e4m3 experts for a few tokens (at most 16).
//
// A few tokens read every chosen expert's weights for a handful of rows: the layer is
// bound by those bytes and, on small experts, by the time its launches take to begin
// and end.  Three launches do it:
//
//   few_logits      one wave for each (token, expert): the fp64 logit.  (Every workgroup of
//                   few_gate_up computing them saves the launch and costs more even with 8
//                   experts: one token of 2048 x 2048 22.4 us against 20.7, two 31.5 and 25.8.)
//   few_gate_up     every workgroup selects the experts itself from the logits, finds the
//                   expert of its slot and multiplies that expert's gate and up rows by
//                   all T tokens at once -- the 16 columns of a matrix product hold
//                   them, chosen or not -- and stores the rows of the tokens that chose
//                   it.  One more workgroup writes the choices and routing weights.
//   few_down        a workgroup owns 16 columns of the output and walks every active
//                   expert and column block, its 8 waves a part each: the routing
//                   weight is folded into the scales, so the sum over a token's experts
//                   is the accumulator itself and no partial result leaves the
//                   workgroup.
//
// Nothing is counted or waited for between workgroups.  Measured: one token, 8 of 60 + 4
// experts of 1408 x 2048, 29.8 us (2 + 15 + 11 in the kernels at best, 2.3 TB/s: latency);
// four tokens, 8 experts of 14336 x 4096, 173 to 199 us by the experts they reach (5.7 TB/s).
// few_layer_fits has both sides of the choice against the steps' own launches.
#include "gemm_fp8.h"
#include "layer_fp8.h"
#include "stream_fp8.h"

namespace apmoe {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;

// The logit of (token t, expert e): fp64 sums of exact products, every expert in the
// same order.  All lanes of the wave return it.
__device__ inline double logit(const FewParams &P, int t, int e, int lane)
{
    const uint16_t *x = P.x + (size_t)t * P.H, *w = P.wr + (size_t)e * P.H;
    double s = 0.0;
    for (int u = lane; u < P.H / 8; u += kWave) {
        const half8 a = *reinterpret_cast<const half8 *>(x + 8 * u), b = *reinterpret_cast<const half8 *>(w + 8 * u);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s = __builtin_fma((double)a[i], (double)b[i], s);
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        s += __shfl_xor(s, d, kWave);
    return s + (P.bias ? (double)P.bias[e] : 0.0);
}

__global__ void __launch_bounds__(256) few_logits(const FewParams P)
{
    const int pair = (int)blockIdx.x * 4 + (int)threadIdx.x / kWave, lane = threadIdx.x % kWave;
    if (pair >= P.T * P.Er)
        return;
    const double z = logit(P, pair / P.Er, pair % P.Er, lane);
    if (lane == 0)
        P.z[pair] = z;
}

// A logit's place in the order: NaN below every number.
__device__ inline double order(double z) { return z == z ? z : -INFINITY; }

// The choices of all tokens: ids[t][0 .. kt).  Expert e of token t is chosen when fewer
// than topk experts come before it (larger logit, or the same and a lower index), and
// their number is its place.  zs: T x Er logits in LDS; the whole workgroup calls.
__device__ inline void choose(const FewParams &P, const double *zs, int *ids, int threads)
{
    for (int i = threadIdx.x; i < P.T * P.Er; i += threads) {
        const int t = i / P.Er, e = i % P.Er;
        const double z = order(zs[i]);
        int before = 0;
        for (int o = 0; o < P.Er; ++o) {
            const double y = order(zs[t * P.Er + o]);
            before += (y > z || (y == z && o < e)) ? 1 : 0;
        }
        if (before < P.topk)
            ids[t * P.kt + before] = e;
    }
    for (int i = threadIdx.x; i < P.T * (P.kt - P.topk); i += threads) {
        const int t = i / (P.kt - P.topk), s = i % (P.kt - P.topk);
        ids[t * P.kt + P.topk + s] = P.Er + s;
    }
}

// Which experts have a token, as bits; every wave computes the same from ids in LDS.
struct Active {
    uint64_t m[APMOE_MAX_EXPERTS / 64];
};

__device__ inline Active active_experts(const int *flags, int lane)
{
    Active a;
#pragma unroll
    for (int c = 0; c < APMOE_MAX_EXPERTS / 64; ++c)
        a.m[c] = __ballot(flags[64 * c + lane] != 0);
    return a;
}

// The slot-th active expert, -1 past the last.
__device__ inline int nth_expert(const Active &a, int slot)
{
#pragma unroll
    for (int c = 0; c < APMOE_MAX_EXPERTS / 64; ++c) {
        const int n = __builtin_popcountll(a.m[c]);
        if (slot < n) {
            uint64_t m = a.m[c];
            for (; slot > 0; --slot)
                m &= m - 1;
            return 64 * c + __builtin_ctzll(m);
        }
        slot -= n;
    }
    return -1;
}

// Choices and routing weights for few_down: a wave for each token.
__device__ inline void write_choices(const FewParams &P, const double *zs, const int *ids, int waves)
{
    const int lane = threadIdx.x % kWave;
    for (int t = threadIdx.x / kWave; t < P.T; t += waves) {
        const double *z = zs + t * P.Er;
        const double zmax = z[ids[t * P.kt]];
        const double ex = lane < P.topk ? exp(z[ids[t * P.kt + lane]] - zmax) : 0.0;
        double den = ex;
        if (!P.renorm) {
            den = 0.0;
            for (int e = lane; e < P.Er; e += kWave)
                den += exp(z[e] - zmax);
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1)
            den += __shfl_xor(den, d, kWave);
        if (lane < P.kt) {
            P.ids[t * P.kt + lane] = ids[t * P.kt + lane];
            P.w[t * P.kt + lane] = lane < P.topk ? (float)(ex / den) : 1.0f;
        }
    }
}

// blockIdx.x: part of F, blockIdx.y: slot of the active experts; one more y for the
// choices.  A wave holds NP pairs of a gate and an up tile of 16 rows.  NW = 4 waves with
// two pairs hold a group of 128 values and quantise it (a8, as): three such workgroups
// fit a CU, so 4 tokens' 5 or 6 active experts of the Mixtral shape (560 to 672
// workgroups) run at once, where 8 waves with one pair took another round for a part of
// them (190 -> 184 us a layer).  With NW = 2 and one pair the workgroups are four times
// as many, each with 32 values, stored in fp32 (a32) and quantised by few_down.  (Also
// measured: four waves sharing a pair's columns, quantised by the last workgroup of a
// group: slower, each workgroup pays for its selection, 133 -> 147 us.)
template <int NW, int NP>
__global__ void __launch_bounds__(NW *kWave, NP == 2 ? 3 : 4) few_gate_up(const FewParams P)
{
    extern __shared__ __attribute__((aligned(16))) char smem[];
    double *zs = reinterpret_cast<double *>(smem);
    __shared__ int ids[kFewTokens * APMOE_MAX_ASSIGN];
    __shared__ int flags[APMOE_MAX_EXPERTS];
    __shared__ uint32_t amax[NW * 16];
    constexpr int kFw = 16 * NP;  // values of F of a wave
    constexpr int NT = NW * kWave;
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const bool writer = (int)blockIdx.y == P.slots;
    if (writer && blockIdx.x != 0)
        return;
    for (int i = tid; i < APMOE_MAX_EXPERTS; i += NT)
        flags[i] = 0;
    for (int i = tid; i < P.T * P.kt; i += NT)
        ids[i] = 0;
    for (int i = tid; i < P.T * P.Er; i += NT)
        zs[i] = P.z[i];
    __syncthreads();
    choose(P, zs, ids, NT);
    __syncthreads();
    if (writer) {
        write_choices(P, zs, ids, NW);
        return;
    }
    for (int i = tid; i < P.T * P.kt; i += NT)
        flags[ids[i]] = 1;
    __syncthreads();
    const int e = __builtin_amdgcn_readfirstlane(nth_expert(active_experts(flags, lane), blockIdx.y));
    if (e < 0)
        return;

    const int j = lane & 15, g = lane >> 4;
    const uint32_t woff = 16u * line_chunk(j, g);
    const int F = P.F, K = P.H, KB = (K + kBlk - 1) / kBlk, fb = (F + kBlk - 1) / kBlk;
    const int fw = ((int)blockIdx.x * NW + wave) * kFw;
    const uint8_t *wbase[2 * NP], *xr[1];
    uint32_t wo[2 * NP][2];
    const float *wsc[2 * NP], *xsc[1];
#pragma unroll
    for (int r = 0; r < 2 * NP; ++r) {  // gate and up tile of each 16 values
        const int h = r % 2, fc = min(fw + 16 * (r / 2), F - 16);  // F is a multiple of 16
        wbase[r] = P.gate_up + ((size_t)e * 2 * F + (size_t)h * F + fc) * K;
        wo[r][0] = (uint32_t)(j % 8) * (uint32_t)K + woff;
        wo[r][1] = (uint32_t)(8 + j % 8) * (uint32_t)K + woff;
        wsc[r] = P.gate_up_s + ((size_t)(2 * e + h) * fb + fc / kBlk) * KB;
    }
    const int t = min(j, P.T - 1);
    xr[0] = P.x8 + (size_t)t * K + 16 * g;
    xsc[0] = P.xs + (size_t)t * KB;
    float4v acc[2 * NP][1];
#pragma unroll
    for (int r = 0; r < 2 * NP; ++r)
        acc[r][0] = float4v{0.f, 0.f, 0.f, 0.f};
    stream_product<2 * NP, 1, kFewDepth>(wbase, wo, wsc, xr, xsc, 0, KB, K, 16 * g, (int)woff,
                                         4 * wave + (int)blockIdx.x, acc);

    int row = -1;  // this lane's token's assignment to e
    if (j < P.T)
        for (int s = 0; s < P.kt; ++s)
            if (ids[j * P.kt + s] == e)
                row = j * P.kt + s;
    float4v a[NP];
    uint32_t mx = 0;
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[p][i] = silu_mul32(acc[2 * p][0][i], acc[2 * p + 1][0][i]);
            mx = max(mx, fw + 16 * p < F ? mag(a[p][i]) : 0u);
        }
    if constexpr (NW * kFw == kBlk) {
        mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16, kWave));
        mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32, kWave));
        if (g == 0)
            amax[wave * 16 + j] = mx;
        __syncthreads();
        if (row < 0)
            return;
        mx = 0;
#pragma unroll
        for (int v = 0; v < NW; ++v)
            mx = max(mx, amax[v * 16 + j]);
        const float s = scale_of(mx), inv = 1.0f / s;
#pragma unroll
        for (int p = 0; p < NP; ++p)
            if (fw + 16 * p < F)
                *reinterpret_cast<uint32_t *>(P.a8 + (size_t)row * F + fw + 16 * p + 4 * g) =
                    to_e4m3x4(a[p][0] * inv, a[p][1] * inv, a[p][2] * inv, a[p][3] * inv);
        if (wave == 0 && g == 0)
            P.as[(size_t)row * fb + blockIdx.x] = s;
    } else if (row >= 0) {
#pragma unroll
        for (int p = 0; p < NP; ++p)
            if (fw + 16 * p < F)
                *reinterpret_cast<float4v *>(P.a32 + (size_t)row * F + fw + 16 * p + 4 * g) = a[p];
    }
}

// One (expert, column block) of few_down: 16 rows of weights, 16 tokens.
struct DownStage {
    Frag8 a, b;
    float sw, f;
    bool chosen, lo, hi;  // whether the token chose the expert; whether b.lo / b.hi are columns below F
};

// blockIdx.x: 16 columns of the output.  QUANT: a32 is quantised into LDS first.
template <bool QUANT>
__global__ void __launch_bounds__(kThreads) few_down(const FewParams P)
{
    extern __shared__ __attribute__((aligned(16))) char smem[];
    __shared__ int flags[APMOE_MAX_EXPERTS];
    __shared__ int list[APMOE_MAX_EXPERTS];             // the active experts
    __shared__ int16_t rows[kFewTokens * APMOE_MAX_ASSIGN][kFewTokens];  // [active expert][token]: its assignment, -1
    __shared__ float wt[kFewTokens * APMOE_MAX_ASSIGN];
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int R = P.T * P.kt, F = P.F, FB = (F + kBlk - 1) / kBlk;
    for (int i = tid; i < APMOE_MAX_EXPERTS; i += kThreads)
        flags[i] = 0;
    for (int i = tid; i < R * kFewTokens; i += kThreads)
        rows[i / kFewTokens][i % kFewTokens] = -1;
    __syncthreads();
    for (int i = tid; i < R; i += kThreads) {
        flags[P.ids[i]] = 1;
        wt[i] = P.w[i];
    }
    __syncthreads();
    const Active act = active_experts(flags, lane);
    int A = 0;
#pragma unroll
    for (int c = 0; c < APMOE_MAX_EXPERTS / 64; ++c)
        A += __builtin_popcountll(act.m[c]);
    A = __builtin_amdgcn_readfirstlane(A);
    // place of an expert among the active ones
    auto place = [&](int e) {
        int p = 0;
#pragma unroll
        for (int c = 0; c < APMOE_MAX_EXPERTS / 64; ++c)
            p += __builtin_popcountll(e >= 64 * (c + 1) ? act.m[c] : e >= 64 * c ? act.m[c] & ((1ull << (e - 64 * c)) - 1) : 0);
        return p;
    };
    if (tid < APMOE_MAX_EXPERTS && flags[tid])
        list[place(tid)] = tid;
    for (int i = tid; i < R; i += kThreads)
        rows[place(P.ids[i])][i / P.kt] = (int16_t)i;
    // the activation's scales [R][FB]; with QUANT after the rows themselves
    float *qs = reinterpret_cast<float *>(smem + (QUANT ? R * F : 0));
    if constexpr (!QUANT) {
        for (int i = tid; i < R * FB; i += kThreads)
            qs[i] = P.as[i];
    } else {
        // 16 lanes take a group of 128 values, 8 each
        char *q8 = smem;
        for (int i = tid; i < R * FB * 16; i += kThreads) {
            const int grp = i / 16, r = grp / FB, kb = grp % FB, c = kb * kBlk + 8 * (i % 16);
            float v[8];
            uint32_t mx = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] = 0.f;
            if (c < F) {
                const float4v lo = *reinterpret_cast<const float4v *>(P.a32 + (size_t)r * F + c);
                const float4v hi = *reinterpret_cast<const float4v *>(P.a32 + (size_t)r * F + c + 4);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    v[q] = lo[q];
                    v[4 + q] = hi[q];
                }
            }
#pragma unroll
            for (int q = 0; q < 8; ++q)
                mx = max(mx, mag(v[q]));
#pragma unroll
            for (int d = 8; d >= 1; d >>= 1)
                mx = max(mx, (uint32_t)__shfl_xor((int)mx, d, kWave));
            const float s = scale_of(mx), inv = 1.0f / s;
            if (c < F) {
                u32x2 o;
                o[0] = to_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
                o[1] = to_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
                *reinterpret_cast<u32x2 *>(q8 + (size_t)r * F + c) = o;
            }
            if (i % 16 == 0)
                qs[grp] = s;
        }
    }
    __syncthreads();

    const int j = lane & 15, g = lane >> 4;
    const int wc = 16 * line_chunk(j, g);
    const int n0 = (int)blockIdx.x * 16;
    const int S = A * FB, lo = S * wave / kWaves, n = S * (wave + 1) / kWaves - lo;
    const int nbk = (P.H + kBlk - 1) / kBlk;
    const int rot = n > 0 ? (5 * (int)blockIdx.x) % n : 0;
    float4v acc = {0.f, 0.f, 0.f, 0.f};
    auto load = [&](DownStage &s, int i) {
        const int st = lo + (i + rot < n ? i + rot : i + rot - n);
        const int ai = st / FB, kb = st % FB;
        const int e = __builtin_amdgcn_readfirstlane(list[ai]);
        const uint8_t *wb = P.down + ((size_t)e * P.H + n0) * F;
        // past a short last block: any column of the row, multiplied by b's zeros
        const uint32_t col = kb * kBlk + wc < F ? (uint32_t)(kb * kBlk + wc) : 0u;
        s.a.lo = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wb + (uint32_t)(j % 8) * (uint32_t)F + col));
        s.a.hi = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wb + (uint32_t)(8 + j % 8) * (uint32_t)F + col));
        s.sw = P.down_s[((size_t)e * nbk + n0 / kBlk) * FB + kb];
        // what is loaded for a token that did not choose the expert is another row's (no
        // request is skipped: stream_product)
        const int r = rows[ai][j], rc = max(r, 0), c = kb * kBlk + 16 * g;
        s.chosen = r >= 0;
        s.lo = c < F;
        s.hi = c + 64 < F;
        const char *q8 = QUANT ? smem + rc * F : reinterpret_cast<const char *>(P.a8) + (size_t)rc * F;
        s.b.lo = *reinterpret_cast<const u32x4 *>(q8 + (c < F ? c : 0));
        s.b.hi = *reinterpret_cast<const u32x4 *>(q8 + (c + 64 < F ? c + 64 : 0));
        s.f = qs[rc * FB + kb] * wt[rc];
    };
    auto mul = [&](const DownStage &s) {
        Frag8 b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b.lo[i] = s.lo ? s.b.lo[i] : 0u;
            b.hi[i] = s.hi ? s.b.hi[i] : 0u;
        }
        const float4v p = block_product(to_frag16(whole_rows(s.a)), to_frag16(b));
        const float f = s.f * s.sw;
        // selected, not multiplied by zero: a NaN weight or scale of an expert is not for the
        // tokens that did not choose it
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc[i] = s.chosen ? __builtin_fmaf(p[i], f, acc[i]) : acc[i];
    };
    if (n > 0) {
        constexpr int D = kDownDepth;
        DownStage st[D];
#pragma unroll
        for (int s = 0; s < D; ++s)
            load(st[s], min(s, n - 1));
        int i = 0;
        for (; i + D <= n; i += D) {
#pragma unroll
            for (int s = 0; s < D; ++s) {
                mul(st[s]);
                load(st[s], min(i + s + D, n - 1));
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int s = 0; s < D - 1; ++s)
            if (i + s < n)
                mul(st[s]);
    }
    // ---- the waves' sums, in the order of their parts
    __syncthreads();  // smem (q8) is read
    float *red = reinterpret_cast<float *>(smem);
    *reinterpret_cast<float4v *>(red + wave * 256 + j * 16 + 4 * g) = acc;
    __syncthreads();
    if (tid < P.T * 16) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            v += red[w * 256 + tid];
        reinterpret_cast<_Float16 *>(P.out)[(size_t)(tid / 16) * P.H + n0 + tid % 16] = (_Float16)v;
    }
}

}  // namespace

hipError_t launch_few_layer(FewParams P, hipStream_t s)
{
    const size_t zbytes = (size_t)P.T * P.Er * sizeof(double);
    const bool quant = few_quantises_late(P.T, P.topk, P.kt, P.Er, P.F);
    P.slots = few_slots(P.T, P.topk, P.kt, P.Er);
    hipLaunchKernelGGL(few_logits, dim3((P.T * P.Er + 3) / 4), dim3(256), 0, s, P);
    const int per = quant ? 32 : kBlk;
    const dim3 grid((P.F + per - 1) / per, P.slots + 1), block((quant ? 2 : 4) * kWave);
    if (quant)
        hipLaunchKernelGGL((few_gate_up<2, 1>), grid, block, zbytes, s, P);
    else
        hipLaunchKernelGGL((few_gate_up<4, 2>), grid, block, zbytes, s, P);
    const size_t red = kWaves * 256 * sizeof(float);
    const size_t q = (size_t)P.T * P.kt * ((quant ? P.F : 0) + 4 * ((P.F + kBlk - 1) / kBlk));
    const size_t lds = q > red ? q : red;
    if (quant)
        hipLaunchKernelGGL((few_down<true>), dim3(P.H / 16), dim3(kThreads), lds, s, P);
    else
        hipLaunchKernelGGL((few_down<false>), dim3(P.H / 16), dim3(kThreads), lds, s, P);
    return hipGetLastError();
}

}  // namespace apmoe
