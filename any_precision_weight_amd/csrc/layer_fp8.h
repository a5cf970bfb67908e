// layer_fp8.h -- the few-token layer's arguments and the rules that choose it (not
// installed).
#pragma once

#include "launch_fp8.h"

namespace apmoe {

constexpr int kFewTokens = 16;  // columns of one matrix product
constexpr int kFewDepth = 2;    // column blocks requested ahead by few_gate_up
constexpr int kDownDepth = 4;   // by few_down

struct FewParams {
    const uint16_t *x;
    const uint8_t *x8;
    const float *xs;
    const uint16_t *wr;
    const float *bias;
    const uint8_t *gate_up;
    const float *gate_up_s;
    const uint8_t *down;
    const float *down_s;
    int T, topk, kt, Er, H, F, renorm;
    double *z;     // [T][Er] logits
    int32_t *ids;  // [T][kt]
    float *w;      // [T][kt]
    uint8_t *a8;   // [T * kt][F]
    float *as;
    float *a32;    // [T * kt][F], where few_down quantises
    uint16_t *out;
    int slots;
};

// Active experts at most: workgroup rows of few_gate_up.
inline int few_slots(int T, int topk, int kt, int Er) { return (T * topk < Er ? T * topk : Er) + (kt - topk); }

// Bytes of LDS for the activation in 8 bits, beside few_down's tables (12 KB).
constexpr long kFewRows8 = 48 * 1024;

// gate_up in workgroups of 32 values of F instead of 128, which leaves the quantisation
// to few_down: where 128 would give the device fewer workgroups than it has CUs by a
// quarter, and the rows fit few_down's LDS.  One token: 60 + 4 experts of 1408 x 2048 (88
// workgroups) 31 us against 38, 8 of 2048 x 2048 (32) 22 against 31; of 14336 x 4096 (224)
// 77 against 70.
inline bool few_quantises_late(int T, int topk, int kt, int Er, int F)
{
    const long rows8 = (long)T * kt * (F + 4 * ((F + 127) / 128));
    return (long)few_slots(T, topk, kt, Er) * ((F + 127) / 128) < 192 && rows8 <= kFewRows8;
}

// The selection compares every expert of a token with every other: at most this many
// comparisons (512 threads share them).  few_down holds the activation's scales in LDS.
inline bool few_layer_fits(int T, int kt, int Er, int F)
{
    return T <= kFewTokens && (long)T * Er * Er <= 256 * 1024 && (long)T * kt * 4 * ((F + 127) / 128) <= kFewRows8;
}

hipError_t launch_few_layer(FewParams P, hipStream_t s);

}  // namespace apmoe
