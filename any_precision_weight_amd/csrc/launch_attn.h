// launch_attn.h -- launches of the paged cache's calls, definitions in apmoe.h (not installed).
#pragma once

#include "internal.h"

namespace apmoe {

struct KvView {
    void *k;
    void *v;
    float *ks;  // e4m3: [n_pages][Hkv][page]
    float *vs;
    int n_pages, page_shift, Hkv, D;
    int c8;
};

struct AttnBatch {
    const int32_t *pages;  // [B][max_pages]
    const int32_t *lens;
    const int32_t *q_offsets;  // [B + 1] or NULL: row b is sequence b's only one
    int B, T, max_pages;
    int room;  // tokens of a sequence that are looked at: at most max_pages * page, at most 2^30
};

struct AppendParams {
    KvView kv;
    AttnBatch s;
    const uint16_t *q;
    const uint16_t *k;
    const uint16_t *v;
    int64_t q_stride, k_stride, v_stride;
    int dtype, Hq;
    const float *rope;
    int n_pos, rot, interleaved;
    uint16_t *q_out;
};

struct AttnParams {
    KvView kv;
    AttnBatch s;
    const uint16_t *q;
    int64_t q_stride;
    int dtype, Hq;
    float scale;
    int window, sinks;  // window 0: none
    uint16_t *out;      // NULL or out8 is
    uint8_t *out8;
    float *out_scale;
    // The parts of what is split: D sums a row, and a maximum and a sum.  decode: [slots][Hq];
    // prefill: [tiles][parts][Hkv][kPartRows]
    float *part_o;
    float *part_ml;
    int slots, part_tiles, few;
    int tiles, parts;
};

constexpr int kPartRows = 128;    // rows of a tile of prefill
constexpr int kPartBlocks = 512;  // prefill splits no call into more workgroups than this

// How a decode call is split: slots of parts (as many as sequences: not at all), the shortest
// part in tiles of 32 tokens, and whether it has few workgroups.
struct DecodePlan {
    int slots, part_tiles, few;
};
DecodePlan decode_plan(int B, int Hkv, int Hq, bool c8, int64_t seen);
int decode_slots_most(int B, int Hkv, int Hq);  // for B sequences or fewer

// Row tiles of a prefill call with groups of G heads, an upper bound, and the parts that each
// is split into.
int prefill_tiles(int B, int T, int G);
int prefill_parts(int tiles, int Hkv, int room);

hipError_t launch_kv_append(const AppendParams &P, hipStream_t s);
hipError_t launch_attn_decode(const AttnParams &P, hipStream_t s);
hipError_t launch_attn_prefill(const AttnParams &P, hipStream_t s);

}  // namespace apmoe
