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

// Comparisons of a selection: every expert of a token with every other.  Each workgroup of
// few_gate_up makes one for itself, with 256 threads, or 128 where few_down quantises.
inline long few_compares(int T, int Er) { return (long)T * Er * Er; }

// gate_up in workgroups of 32 values of F instead of 128, which leaves the quantisation
// to few_down: where 128 would give the device fewer workgroups than it has CUs by a
// quarter, the rows fit few_down's LDS and the selection is short enough for 128 threads.
// One token: 60 + 4 experts of 1408 x 2048 (88 workgroups) 31 us against 38, 8 of 2048 x 2048
// (32) 22 against 31; of 14336 x 4096 (224) 77 against 70.  Of 128 experts of 768 x 2048 12
// tokens of 2 (196608 comparisons, 144 workgroups) 100 against 70.
inline bool few_quantises_late(int T, int topk, int kt, int Er, int F)
{
    const long rows8 = (long)T * kt * (F + 4 * ((F + 127) / 128));
    return (long)few_slots(T, topk, kt, Er) * ((F + 127) / 128) < 192 && rows8 <= kFewRows8 &&
           few_compares(T, Er) <= 128 * 1024;
}

// Whether a layer takes the few-token launches; few_down holds the activation's scales in
// LDS.  Against the route, products and combine in launches of their own (us):
//   one token, 8 experts of 14336 x 4096 68 and 116, 60 + 4 of 1408 x 2048 32 and 63, 128 of
//   768 x 2048 (8 a token) 27 and 64; 4 tokens of the first 183 and 197, of the second 53 and
//   109; 16 of the second 108 and 119.
// They lose to them where
//   - a selection is long: up to 393216 comparisons (256 experts of 768 x 2048, 2 a token: 4
//     tokens 68 and 93, 6, 393216, 88 and 96, 8 108 and 99; 160 of 1536 x 5120, 1 a token, 12
//     tokens 137 and 246);
//   - the selections add up: up to 192 million comparisons in all workgroups (128 experts of
//     768 x 2048, 8 a token: 14 tokens 124 and 129, 16 tokens, 201 million, 151 and 132; 160
//     experts of 1536 x 5120, 6 a token, 10 tokens, 184 million, 310 and 331);
//   - many tokens meet many bytes of down weights, which the stream product reads with two
//     weight tiles for a tile of tokens: from 12 tokens and 2^28 active weights on (8 experts
//     of 14336 x 4096, 2 a token: 8 tokens 236 and 240, 12 252 and 245, 16 263 and 247; of
//     16384 x 6144, 16 tokens 475 and 432; 16 experts of 4096 x 4096, 2^28, 137 and 137).
inline bool few_layer_fits(int T, int topk, int kt, int Er, int H, int F)
{
    const long slots = few_slots(T, topk, kt, Er), compares = few_compares(T, Er);
    return T <= kFewTokens && (long)T * kt * 4 * ((F + 127) / 128) <= kFewRows8 && compares <= 384 * 1024 &&
           slots * ((F + 127) / 128) * compares <= 192 * 1000 * 1000 && (T < 12 || slots * H * F < 1l << 28);
}

hipError_t launch_few_layer(FewParams P, hipStream_t s);

}  // namespace apmoe
