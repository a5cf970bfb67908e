// stream_fp8.h -- the register-fed e4m3 product shared by the stream product and the
// few-token layer (not installed).
#pragma once

#include "fp8.h"

namespace apmoe {

constexpr int kDepth = 4;  // column blocks requested ahead

template <int NR, int TT>
struct StreamStage {
    Frag8 a[NR], b[TT];
    float sw[NR], sx[TT];
};

// acc[r][t] += the product of weight tile r (16 rows) and token tile t (16 rows) over
// column blocks kb0 .. kb1-1.  wr / xr: this lane's row of each tile at column `off` =
// 16 (lane / 16); a block's fragment is the 16 bytes there and the 16 bytes 64 further.
// wsc / xsc: the rows' scales by block.  The blocks run kDepth ahead of the products in
// registers; K's last block may be shorter than 128, a multiple of 16: the lanes past it
// give zeros.
template <int NR, int TT>
__device__ __attribute__((always_inline)) inline void stream_product(const uint8_t *const (&wr)[NR],
                                                                    const float *const (&wsc)[NR],
                                                                    const uint8_t *const (&xr)[TT],
                                                                    const float *const (&xsc)[TT], int kb0, int kb1,
                                                                    int K, int off, float4v (&acc)[NR][TT])
{
    if (kb0 >= kb1)
        return;
    const int full = K / kBlk;  // whole blocks
    const int kf = min(kb1, full), n = kf - kb0;
    StreamStage<NR, TT> S[kDepth];
    auto load = [&](StreamStage<NR, TT> &s, int b) {
        const size_t o = (size_t)b * kBlk;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            s.a[r].lo = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wr[r] + o));
            s.a[r].hi = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wr[r] + o + 64));
            s.sw[r] = wsc[r][b];
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            s.b[t].lo = *reinterpret_cast<const u32x4 *>(xr[t] + o);
            s.b[t].hi = *reinterpret_cast<const u32x4 *>(xr[t] + o + 64);
            s.sx[t] = xsc[t][b];
        }
    };
    auto mul = [&](const StreamStage<NR, TT> &s) {
        Frag16 b[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t)
            b[t] = to_frag16(s.b[t]);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const Frag16 a = to_frag16(s.a[r]);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const float4v p = block_product(a, b[t]);
                const float f = s.sw[r] * s.sx[t];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[r][t][i] = __builtin_fmaf(p[i], f, acc[r][t][i]);
            }
        }
    };
    if (n > 0) {
#pragma unroll
        for (int s = 0; s < kDepth; ++s)
            if (s < n)
                load(S[s], kb0 + s);
        int i = 0;
        for (; i + 2 * kDepth <= n; i += kDepth) {
#pragma unroll
            for (int s = 0; s < kDepth; ++s) {
                mul(S[s]);
                load(S[s], kb0 + i + s + kDepth);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // up to 2 kDepth - 1 blocks are left, the first kDepth of them requested
#pragma unroll
        for (int s = 0; s < kDepth; ++s)
            if (i + s < n) {
                mul(S[s]);
                if (i + s + kDepth < n)
                    load(S[s], kb0 + i + s + kDepth);
            }
#pragma unroll
        for (int s = 0; s < kDepth; ++s)
            if (i + kDepth + s < n)
                mul(S[s]);
    }
    if (kb1 > full) {  // K's last, shorter block
        const int c0 = full * kBlk + off;
        const u32x4 z = {0, 0, 0, 0};
        StreamStage<NR, TT> s;
        const size_t o = (size_t)full * kBlk;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            s.a[r].lo = c0 < K ? *reinterpret_cast<const u32x4 *>(wr[r] + o) : z;
            s.a[r].hi = c0 + 64 < K ? *reinterpret_cast<const u32x4 *>(wr[r] + o + 64) : z;
            s.sw[r] = wsc[r][full];
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            s.b[t].lo = c0 < K ? *reinterpret_cast<const u32x4 *>(xr[t] + o) : z;
            s.b[t].hi = c0 + 64 < K ? *reinterpret_cast<const u32x4 *>(xr[t] + o + 64) : z;
            s.sx[t] = xsc[t][full];
        }
        mul(s);
    }
}

}  // namespace apmoe
