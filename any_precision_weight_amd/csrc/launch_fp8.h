// launch_fp8.h -- launches of the 8-bit path, definitions in apmoe.h (not installed).
#pragma once

#include "internal.h"

namespace apmoe {

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
