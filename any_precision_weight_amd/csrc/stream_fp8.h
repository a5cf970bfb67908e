// stream_fp8.h -- the register-fed e4m3 product shared by the stream product and the
// few-token layer (not installed).
#pragma once

#include "fp8.h"

namespace apmoe {

template <int NR, int TT>
struct StreamStage {
    Frag8 a[NR], b[TT];
    float sw[NR], sx[TT];
};

// acc[r][t] += the product of weight tile r (16 rows) and token tile t (16 rows) over
// column blocks kb0 .. kb1-1.  Weights: lane offsets wo from wbase (the same in every
// lane), at column woff = 16 line_chunk, of the rows that the lane asks for
// (whole_rows).  xr: the lane's token row at column off = 16 (lane / 16); a block's
// fragment is the 16 bytes there and the 16 bytes 64 further.  wsc / xsc: the rows'
// scales by block.  The blocks are requested D ahead of their products, into registers,
// starting with block rot of the range: workgroups that start at different columns do
// not ask the same memory channels all at once (rows are a multiple of a large power of
// two apart; 4.2 -> 4.5 TB/s where it was first measured).  K's last block may be shorter than 128, a multiple of
// 16: the lanes past it give zeros.
template <int NR, int TT, int D>
__device__ __attribute__((always_inline)) inline void stream_product(const uint8_t *const (&wbase)[NR], const uint32_t (&wo)[NR][2],
                                                                    const float *const (&wsc)[NR],
                                                                    const uint8_t *const (&xr)[TT],
                                                                    const float *const (&xsc)[TT], int kb0, int kb1,
                                                                    int K, int off, int woff, int rot, float4v (&acc)[NR][TT])
{
    if (kb0 >= kb1)
        return;
    const int full = K / kBlk;  // whole blocks
    const int kf = min(kb1, full), n = kf - kb0;
    StreamStage<NR, TT> S[D];
    rot = n > 0 ? rot % n : 0;
    auto load = [&](StreamStage<NR, TT> &s, int i) {
        const int b = kb0 + (i + rot < n ? i + rot : i + rot - n);
        const size_t o = (size_t)b * kBlk;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            s.a[r].lo = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wbase[r] + o + wo[r][0]));
            s.a[r].hi = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wbase[r] + o + wo[r][1]));
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
            const Frag16 a = to_frag16(whole_rows(s.a[r]));
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
        // Requests are never skipped (past the last block they ask for it again, from the
        // caches): the number in flight is then known at every wait, and the compiler
        // waits for the oldest block only.
#pragma unroll
        for (int s = 0; s < D; ++s)
            load(S[s], min(s, n - 1));
        int i = 0;
        for (; i + D <= n; i += D) {
#pragma unroll
            for (int s = 0; s < D; ++s) {
                mul(S[s]);
                load(S[s], min(i + s + D, n - 1));
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int s = 0; s < D - 1; ++s)
            if (i + s < n)
                mul(S[s]);
    }
    if (kb1 > full) {  // K's last, shorter block
        const int c0 = full * kBlk + off, w0 = full * kBlk + woff;
        const u32x4 z = {0, 0, 0, 0};
        StreamStage<NR, TT> s;
        const size_t o = (size_t)full * kBlk;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            s.a[r].lo = w0 < K ? *reinterpret_cast<const u32x4 *>(wbase[r] + o + wo[r][0]) : z;
            s.a[r].hi = w0 < K ? *reinterpret_cast<const u32x4 *>(wbase[r] + o + wo[r][1]) : z;
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
