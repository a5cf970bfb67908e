// gemm_fp8.h -- what the e4m3 stream and tile products share (not installed).
#pragma once

#include "fp8.h"
#include "launch_fp8.h"

namespace apmoe {

struct Fp8Params {
    const uint8_t *x8;
    const float *xs;
    const uint8_t *w8;
    const float *ws;
    const int32_t *perm;
    const int32_t *offsets;  // NULL: one expert with all R rows
    void *out;               // product; a8 with the activation
    float *os;               // scales of a8
    int E, N, K, topk, gather, out_dtype, R;
    int F;  // with the activation: N = 2 F
};

// Rows of an expert up to which the stream product reads its weights once; with more the
// tile product is a choice (takes_tiles).
constexpr int kStreamMax = 32;

__device__ inline void expert_rows(const Fp8Params &P, int e, int &r0, int &m)
{
    r0 = P.offsets ? P.offsets[e] : 0;
    m = (P.offsets ? P.offsets[e + 1] : P.R) - r0;
}

__device__ inline size_t src_row(const Fp8Params &P, int r)
{
    return (size_t)(P.gather ? P.perm[r] / P.topk : r);
}

// SiLU(g) * u in fp32 (the hardware reciprocal, 1 ulp).
__device__ inline float silu_mul32(float g, float u)
{
    return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Four outputs in the product's type: 16 bytes, or the lower 8 of them.
__device__ inline u32x4 pack4(int dtype, const float4v &v)
{
    if (dtype == APMOE_F32)
        return __builtin_bit_cast(u32x4, v);
    u32x4 o = {0, 0, 0, 0};
    if (dtype == APMOE_F16) {
        const half4 h = {(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
        const u32x2 b = __builtin_bit_cast(u32x2, h);
        o[0] = b[0];
        o[1] = b[1];
    } else {
        o[0] = to_bf16(v[0]) | (uint32_t)to_bf16(v[1]) << 16;
        o[1] = to_bf16(v[2]) | (uint32_t)to_bf16(v[3]) << 16;
    }
    return o;
}

// Four consecutive outputs of a row, those below N.
__device__ inline void store4(const Fp8Params &P, size_t row, int n, const float4v &v)
{
    const size_t at = row * (size_t)P.N + n;
    const u32x4 o = pack4(P.out_dtype, v);
    if (n + 4 <= P.N && P.N % 4 == 0) {
        if (P.out_dtype == APMOE_F32)
            *reinterpret_cast<u32x4 *>(static_cast<float *>(P.out) + at) = o;
        else
            *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(P.out) + at) = u32x2{o[0], o[1]};
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (n + i >= P.N)
            break;
        if (P.out_dtype == APMOE_F32)
            static_cast<uint32_t *>(P.out)[at + i] = o[i];
        else
            static_cast<uint16_t *>(P.out)[at + i] = (uint16_t)(o[i / 2] >> (16 * (i % 2)));
    }
}

// Rows that an expert has at most, as a choice of kernels: a token's experts are distinct as
// the routing gives them, so one for each token (rows beyond that are computed, slower);
// a single expert has every row.
inline int most_rows(const Fp8Params &P) { return P.E == 1 ? P.R : P.R / P.topk; }

// Tokens of a tile: 128 where the products of a stage stay in registers.
constexpr int fp8_tile_tokens(bool exact) { return exact ? kMinTileTokens : 256; }

// Upper bound of the tiles of `tok` rows: of the rows times of the weights.
long fp8_tiles(const Fp8Params &P, bool act, int tok);

// exact: fp32 sums inside a block (block_product), which fp32 results keep.
hipError_t launch_fp8_tile(const Fp8Params &P, bool act, bool exact, hipStream_t s);

}  // namespace apmoe
