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
    // decode: the parts of sequences that are split, [slots][Hq] of D sums, and of a maximum
    // and a sum
    float *part_o;
    float *part_ml;
    int slots;
};

// Slots of the parts of a decode call: one a sequence and as many again as fill the device.
int decode_slots(int B, int Hkv, int Hq);

hipError_t launch_kv_append(const AppendParams &P, hipStream_t s);
hipError_t launch_attn_decode(const AttnParams &P, hipStream_t s);
hipError_t launch_attn_prefill(const AttnParams &P, hipStream_t s);

}  // namespace apmoe
