// launch_fp8.h -- launches of the 8-bit path, definitions in apmoe.h (not installed).
#pragma once

#include "internal.h"

namespace apmoe {

// Tiles of the product: workgroups count them in 32 bits.
constexpr long kMaxTiles8 = 1l << 30;
constexpr int kMinTileTokens = 128;

// Upper bound of the tiles of `tok` rows of R rows and E experts: for each expert that may
// have rows the last one started (ceil(m / tok) = (m - 1) / tok + 1).
inline long fp8_token_tiles(int E, int R, int tok)
{
    const int served = E < R ? E : R;
    return (long)(R - served) / tok + served;
}

// Whether the tiles of R rows and N weight rows an expert can be counted.
inline bool fp8_tiles_fit(int E, long N, int R)
{
    return fp8_token_tiles(E, R, kMinTileTokens) * ((N + 255) / 256) <= kMaxTiles8;
}

hipError_t launch_norm(const void *x, int x_dtype, const void *residual, void *h, int res_dtype, const void *gamma,
                       float eps, int T, int H, void *y, uint8_t *y8, float *ys, hipStream_t s);
// exact: the sums inside a block of 128 columns in fp32 even where the outputs have 16 bits.
hipError_t launch_gemm_fp8(const uint8_t *x8, const float *xs, const uint8_t *w8, const float *ws, int E, int N, int K,
                           int gather, const int32_t *perm, const int32_t *offsets, int topk, int R, void *out,
                           int out_dtype, bool exact, hipStream_t s);
hipError_t launch_gemm_act_fp8(const uint8_t *x8, const float *xs, const uint8_t *w8, const float *ws, int E, int F,
                               int K, int gather, const int32_t *perm, const int32_t *offsets, int topk, int R,
                               uint8_t *a8, float *as, hipStream_t s);

}  // namespace apmoe
