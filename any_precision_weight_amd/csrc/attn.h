// attn.h -- attention over a paged key-value cache: what its kernels share (not installed).
//
// A page holds `page` tokens of every key-value head; inside a page each head has page * D
// elements of K and of V, in the order of the matrix instructions' operands:
//
//   K  16-token tiles [D / c][16][c], c = 16 bytes of elements: 64 lanes that read 16 bytes
//      each, one after the other, get the operand of 32 columns (2-byte elements) or 64
//      (e4m3) of a 16-row product, 1 KB in whole lines, without LDS or a lane exchange;
//   V  32-token tiles [4][D][8]: entry (g, d) holds tokens 4g .. 4g+3 and 16+4g .. 16+4g+3 of
//      column d.  Those are the tokens whose scores lane group g of two 16 x 16 products
//      holds, so probabilities go into the second product from the registers they are in.
//
// Both products are computed transposed (keys x queries, then values x queries), so that a
// lane keeps one query column through both: its running maximum and sum need no lane but
// those with the same column.
#pragma once

#include "fp8.h"
#include "launch_attn.h"

namespace apmoe {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float2v __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 32;  // tokens of a V tile

__device__ inline float4v mfma16(int dt, const u32x4 &a, const u32x4 &b, const float4v &c)
{
    if (dt == APMOE_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0,
                                                      0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

__device__ inline float16v mfma32(int dt, const u32x4 &a, const u32x4 &b, const float16v &c)
{
    if (dt == APMOE_F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0,
                                                      0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// Two fp32 values as two 16-bit ones, to nearest even, lo in the low half.
template <int DT>
__device__ inline uint32_t pack2(float lo, float hi)
{
    const float2v v = {lo, hi};
    if constexpr (DT == APMOE_F16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, half2v));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

template <int DT>
__device__ inline float low16(uint32_t w)
{
    if constexpr (DT == APMOE_F16)
        return (float)__builtin_bit_cast(half2v, w)[0];
    else
        return __builtin_bit_cast(float, w << 16);
}

template <int DT>
__device__ inline float high16(uint32_t w)
{
    if constexpr (DT == APMOE_F16)
        return (float)__builtin_bit_cast(half2v, w)[1];
    else
        return __builtin_bit_cast(float, w & 0xFFFF0000u);
}

// Eight e4m3 bytes as eight 16-bit values (exact: both types hold e4m3's).
template <int DT>
__device__ inline u32x4 from_e4m3x8(uint32_t lo, uint32_t hi)
{
    if constexpr (DT == APMOE_F16)
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true))};
    else
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true))};
}

// A value that all lanes have, in a scalar register.
__device__ inline float uniform(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
}

// exp2's argument is (s - m) c: c > 0 for scores s of queries whose signs are turned where the
// scale is negative, so the maximum m is that of the scores as the products give them.  The
// largest one's argument is 0 exactly, and no product of a score and c has to be a number.
// A scale of 0 (or next to it) takes fp32's smallest number: arguments below 2^-20 for any
// scores, and -infinity stays what it is.
__device__ inline float score_factor(float scale) { return uniform(fmaxf(__builtin_fabsf(scale) * kLog2e, 0x1p-149f)); }

__device__ inline uint32_t query_sign(float scale) { return scale < 0.0f ? 0x80008000u : 0u; }

// Probabilities and their sum are 2^kTop times what they are by the formula.  fp16 has numbers up
// to 2^15 and none below 2^-25, so the largest probability goes there.  bf16 has fp32's range, and
// its values too: with 2^-30 the sum over 2^30 tokens is at most 1, and no sum of probabilities
// times values is larger than the largest value.
template <int DT>
constexpr float kTop = DT == APMOE_F16 ? 15.0f : -30.0f;

// Factor of a part with maximum m and sum l where the largest maximum is M.  m = -infinity with
// l = 0 is a part that saw nothing (or scores of -infinity only): 0.  The maximum passes a NaN
// by, the sum does not: m = -infinity with any other l is a part whose scores were NaN, and
// the factor is that NaN.
__device__ inline float part_factor(float m, float l, float M, float c)
{
    return m == -INFINITY ? l : __builtin_amdgcn_exp2f((m - M) * c);
}

// Tokens of a sequence of `len` tokens that the cache can hold at all.
__device__ inline int cached_tokens(const AttnBatch &S, int len) { return max(0, min(len, S.room)); }

// Sum over the lanes up to and with this one: within rows of 16 lanes, then rows 0 and 2 into
// the next one, then lane 31 into the upper half (lane exchanges without LDS).
__device__ inline int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);  // from 1, 2, 4, 8 lanes below
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row's last lane to the next row
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // lane 31 to the upper half
    return v;
}

__device__ inline int wave_sum(int v) { return __builtin_amdgcn_readlane(wave_scan(v), kWave - 1); }

// Items of the sequences one after the other, count(b) of sequence b: the sequence b and the
// index `local` in it of item w, and the sequence's number of items n; false when there are
// no more than w items.  Every wave computes the same answer; 64 sequences a step.
template <class Count>
__device__ inline bool find_item(int B, int w, const Count &count, int &b, int &local, int &n)
{
    const int lane = threadIdx.x % kWave;
    int base = 0;
    for (int b0 = 0; b0 < B; b0 += kWave) {
        const int mine = b0 + lane < B ? count(b0 + lane) : 0;
        const int incl = wave_scan(mine);
        const int total = __builtin_amdgcn_readlane(incl, kWave - 1);
        if (w - base < total) {
            const int at = (int)__builtin_ctzll(__ballot(incl > w - base));
            b = b0 + at;
            n = __builtin_amdgcn_readlane(mine, at);
            local = w - base - (__builtin_amdgcn_readlane(incl, at) - n);
            return true;
        }
        base += total;
    }
    return false;
}

}  // namespace apmoe
