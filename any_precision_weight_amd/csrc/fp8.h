// fp8.h -- device helpers of the 8-bit path (not installed): e4m3 rows with a scale for
// each group of 128 columns, and the matrix product of two e4m3 fragments.
//
// A row in 8 bits: group g holds columns 128g .. 128g+127 (the last group may be
// shorter), s[g] = max(max |v| / 448, 2^-126) in fp32 and q[c] = e4m3(v[c] / s[g]),
// round to nearest even; it stands for q * s.  448 is e4m3's largest value, so no
// quotient overflows; the lower bound keeps s and 1 / s normal numbers for a group of
// zeros.  A group with an infinity or a NaN has that as its scale, so all of it stands
// for NaN.
#pragma once

#include "device.h"

namespace apmoe {

constexpr int kBlk = 128;  // columns that share a scale; also the columns of one MFMA
constexpr float kE4m3Max = 448.0f;
constexpr float kScaleMin = 0x1p-126f;

typedef int int8v __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));

// 32 bytes of an e4m3 row, a lane's part of one 128-column block.
struct Frag8 {
    u32x4 lo, hi;
};

// 16 rows x 128 columns are read as two requests of 8 whole rows (128-byte lines): a CU
// takes 46 GB/s that way against 25 with 16 half rows a request, and the device 5.8
// against 5.4 TB/s.  Lane l (j = l % 16, g = l / 16) asks for chunk g + 4 (j / 8) of rows
// j % 8 (lo) and 8 + j % 8 (hi); line_chunk is that chunk.  whole_rows exchanges the
// quarters that belong to the other half of the 16 lanes: row j's chunks g and g + 4.
__device__ inline int line_chunk(int j, int g) { return g + 4 * (j >> 3); }

__device__ inline Frag8 whole_rows(const Frag8 &f)
{
    constexpr int kRor8 = 0x128;  // within 16 lanes, from lane j ^ 8
    Frag8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.lo[i] = (uint32_t)__builtin_amdgcn_update_dpp((int)f.lo[i], (int)f.hi[i], kRor8, 0xF, 0xC, false);
        r.hi[i] = (uint32_t)__builtin_amdgcn_update_dpp((int)f.hi[i], (int)f.lo[i], kRor8, 0xF, 0x3, false);
    }
    return r;
}

// A Frag8 in fp16 (e4m3's values are fp16 values: exact), as four operands of the
// 32-column fp16 MFMA.
struct Frag16 {
    half8 k[4];
};

// Word i (two values) of the fp16 operand made of half h of 16 bytes.
__device__ inline uint32_t half2_of(const u32x4 &v, int h, int i)
{
    const uint32_t w = v[2 * h + (i >> 1)];
    return __builtin_bit_cast(uint32_t, (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true)
                                                : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
}

// Operand i of Frag16.
__device__ inline half8 quarter(const Frag8 &f, int i)
{
    const u32x4 &v = i < 2 ? f.lo : f.hi;
    const u32x4 q = {half2_of(v, i & 1, 0), half2_of(v, i & 1, 1), half2_of(v, i & 1, 2), half2_of(v, i & 1, 3)};
    return __builtin_bit_cast(half8, q);
}

__device__ inline Frag16 to_frag16(const Frag8 &f)
{
    return Frag16{{quarter(f, 0), quarter(f, 1), quarter(f, 2), quarter(f, 3)}};
}

// The product of one block, C[16][16] (fp32) = A[16][128] * B[128][16].  Lane l gives 32
// bytes of A's row l % 16 and of B's column l % 16; which of the 128 columns they are
// follows from l / 16 in the same way for A and B, and a sum over columns does not ask
// for their order, so any assignment that A and B share is right.  Lane l receives
// column l % 16, rows 4 (l / 16) .. + 3.
//
// There are two forms.  In fp16 the products are exact and the sum is an fp32 one
// (2^-22 of the terms' magnitudes, measured).  The e4m3 instruction takes half the
// time (32 clocks against 4 x 16), but in each group of 8 columns it cuts the products
// off below 2^-13 of the largest one's power of two (measured with pairs of products;
// the same for its 32-column form): normally distributed operands give a relative error
// of 1.5e-5 in norm.  So it serves only where the result is rounded to 16 bits at once
// (2^-12 for fp16 on average, 16 times that); sums that are kept in fp32 or quantised
// again take fp16.
__device__ inline float4v block_product(const Frag16 &a, const Frag16 &b)
{
    float4v c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.k[i], b.k[i], c, 0, 0, 0);
    return c;
}

__device__ inline float4v block_product(const Frag8 &a, const Frag8 &b)
{
    auto v = [](const Frag8 &f) {
        return int8v{(int)f.lo[0], (int)f.lo[1], (int)f.lo[2], (int)f.lo[3],
                     (int)f.hi[0], (int)f.hi[1], (int)f.hi[2], (int)f.hi[3]};
    };
    // the instruction's own power-of-two block scales are left out (operands 0)
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v(a), v(b), float4v{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

__device__ inline float lds_f32(uint32_t addr)
{
    return *reinterpret_cast<const __attribute__((address_space(3))) float *>((uintptr_t)addr);
}

// Magnitude as an unsigned integer: ordered as the magnitudes are, an infinity above
// every number and a NaN above that, so an integer maximum passes both on (the float
// maximum drops a NaN).
__device__ inline uint32_t mag(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }

// Scale of a group from the largest magnitude of its values.
__device__ inline float scale_of(uint32_t amax)
{
    const float s = __builtin_bit_cast(float, amax) / kE4m3Max;
    return s < kScaleMin ? kScaleMin : s;  // a NaN stays
}

// Four values -> four e4m3 bytes, v[0] lowest.
__device__ inline uint32_t to_e4m3x4(float v0, float v1, float v2, float v3)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(v0, v1, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(v2, v3, r, true);
    return (uint32_t)r;
}

// fp32 -> bf16, round to nearest even; a NaN stays one.
__device__ inline uint16_t to_bf16(float v)
{
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}

}  // namespace apmoe
