// kv_append.hip -- new tokens into the paged cache: the position rotation of queries and
// keys, the keys and values in the cache's order (attn.h), in 16 bits or as e4m3 rows.
//
// A rotated pair is (x c - y s, x s + y c), in fp64: the products are exact there and a
// value is rounded once, to the type it is stored in.  An e4m3 row is s = max(max |v| / 448,
// 2^-126) in fp32 and v / s, in fp64 too: 16-bit rows have many quotients on or next to a
// border between two e4m3 values.
#include "attn.h"

namespace apmoe {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kGridX = 1u << 22;

// A token of the call: its position, and its place in the cache (page < 0: none).
struct Place {
    int pos, page, at;
};

__device__ inline Place place_of(const AppendParams &P, int b, int pos)
{
    Place r{pos, -1, pos & ((1 << P.kv.page_shift) - 1)};
    if (pos >= 0 && pos < P.s.room && !(P.rope && pos >= P.n_pos)) {
        const int p = P.s.pages[(size_t)b * P.s.max_pages + (pos >> P.kv.page_shift)];
        r.page = p >= 0 && p < P.kv.n_pages ? p : -1;
    }
    return r;
}

__device__ inline void load8(int dt, const uint16_t *p, double (&v)[8])
{
    const u32x4 r = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = r[i / 2];
        if (dt == APMOE_F16)
            v[i] = (double)((i & 1) ? high16<APMOE_F16>(w) : low16<APMOE_F16>(w));
        else
            v[i] = (double)((i & 1) ? high16<APMOE_BF16>(w) : low16<APMOE_BF16>(w));
    }
}

// fp64 -> fp32 for a second rounding to few bits: the last bit is set where the value is
// not exact (round to odd), so the second rounding sees on which side of a border it is.
__device__ inline float to_odd(double v)
{
    float f = (float)v;
    const double d = (double)f;
    if (d != v) {
        uint32_t b = __builtin_bit_cast(uint32_t, f);
        if (__builtin_fabs(d) > __builtin_fabs(v))
            b -= 1;  // toward zero
        f = __builtin_bit_cast(float, b | 1u);
    }
    return f;
}

__device__ inline u32x4 to16(int dt, const double (&v)[8])
{
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = to_odd(v[2 * i]), hi = to_odd(v[2 * i + 1]);
        r[i] = dt == APMOE_F16 ? pack2<APMOE_F16>(lo, hi) : pack2<APMOE_BF16>(lo, hi);
    }
    return r;
}

// Columns 8c .. 8c+7 of a row at x, rotated for position pos.
__device__ inline void rotated(const AppendParams &P, const uint16_t *x, int c, int pos, double (&v)[8])
{
    load8(P.dtype, x + 8 * c, v);
    if (8 * c >= P.rot)
        return;
    const int half = P.rot / 2;
    const float *row = P.rope + (size_t)pos * P.rot;
    if (P.interleaved) {
        const float4v co = *reinterpret_cast<const float4v *>(row + 4 * c);
        const float4v si = *reinterpret_cast<const float4v *>(row + half + 4 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double a = v[2 * i], b = v[2 * i + 1], cd = (double)co[i], sd = (double)si[i];
            v[2 * i] = a * cd - b * sd;
            v[2 * i + 1] = a * sd + b * cd;
        }
        return;
    }
    const bool first = 8 * c < half;
    const int at = first ? 8 * c : 8 * c - half;
    double o[8];
    load8(P.dtype, x + (first ? 8 * c + half : at), o);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float4v co = *reinterpret_cast<const float4v *>(row + at + 4 * h);
        const float4v si = *reinterpret_cast<const float4v *>(row + half + at + 4 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double sd = first ? -(double)si[i] : (double)si[i];
            v[4 * h + i] = v[4 * h + i] * (double)co[i] + o[4 * h + i] * sd;
        }
    }
}

// Scale of a row whose columns lie with `lanes` neighbouring lanes, 8 each.
__device__ inline float row_scale(const double (&v)[8], int lanes)
{
    uint64_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v[i]) & 0x7FFFFFFFFFFFFFFFull;
        m = b > m ? b : m;
    }
    for (int d = lanes / 2; d >= 1; d >>= 1) {
        const uint64_t o = (uint64_t)__shfl_xor((unsigned long long)m, d, kWave);
        m = o > m ? o : m;
    }
    const float s = (float)(__builtin_bit_cast(double, m) / (double)kE4m3Max);
    return s < kScaleMin ? kScaleMin : s;  // a NaN stays
}

__device__ inline u32x2 to8(const double (&v)[8], float scale)
{
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        q[i] = to_odd(v[i] / (double)scale);
    return u32x2{to_e4m3x4(q[0], q[1], q[2], q[3]), to_e4m3x4(q[4], q[5], q[6], q[7])};
}

// Where head h of a page starts, in elements of K or V.
__device__ inline size_t head_base(const KvView &kv, int page, int h)
{
    return ((size_t)page * kv.Hkv + h) * ((size_t)kv.D << kv.page_shift);
}

__device__ inline size_t scale_at(const KvView &kv, int page, int h, int at)
{
    return (((size_t)page * kv.Hkv + h) << kv.page_shift) + at;
}

__device__ inline void store_k(const KvView &kv, int dt, const Place &pl, int h, int c, const double (&v)[8])
{
    const size_t tile = head_base(kv, pl.page, h) + (size_t)(pl.at / 16) * 16 * kv.D;
    if (kv.c8) {
        const float s = row_scale(v, kv.D / 8);
        *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(kv.k) + tile + (c / 2 * 16 + pl.at % 16) * 16 + c % 2 * 8) =
            to8(v, s);
        if (c == 0)
            kv.ks[scale_at(kv, pl.page, h, pl.at)] = s;
    } else {
        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(kv.k) + tile + (c * 16 + pl.at % 16) * 8) = to16(dt, v);
    }
}

// One token's columns of V, element by element: a granule of V holds 8 tokens.
__device__ inline void store_v(const KvView &kv, const Place &pl, int h, int c, const u32x4 &x, const double (&v)[8])
{
    const int u = pl.at % kTile;
    const size_t at = head_base(kv, pl.page, h) + (size_t)(pl.at / kTile) * kTile * kv.D +
                      ((size_t)(u % 16 / 4) * kv.D + 8 * c) * 8 + u / 16 * 4 + u % 4;
    if (kv.c8) {
        const float s = row_scale(v, kv.D / 8);
        const u32x2 q = to8(v, s);
        uint8_t *p = static_cast<uint8_t *>(kv.v) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            p[8 * i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
        if (c == 0)
            kv.vs[scale_at(kv, pl.page, h, pl.at)] = s;
    } else {
        uint16_t *p = static_cast<uint16_t *>(kv.v) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            p[8 * i] = (uint16_t)(x[i / 2] >> (16 * (i % 2)));
    }
}

// A thread has 8 columns of one head of one token: queries, then keys, then values.
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams P)
{
    const KvView &kv = P.kv;
    const int chunks = kv.D / 8, heads = P.Hq + 2 * kv.Hkv;
    const uint32_t t = blockIdx.y * kGridX + blockIdx.x;
    if (t >= (uint32_t)P.s.T)
        return;
    int b = (int)t, pos;
    if (P.s.q_offsets) {
        int local, n;
        const int32_t *off = P.s.q_offsets;
        if ((int)t < off[0] ||
            !find_item(P.s.B, (int)t - off[0], [&](int i) { return max(0, off[i + 1] - off[i]); }, b, local, n))
            return;
        pos = P.s.lens[b] - n + local;
    } else {
        pos = P.s.lens[b] - 1;
    }
    const Place pl = place_of(P, b, pos);
    if (pl.page < 0)
        return;
    // lanes of a row are neighbours and their number divides a wave's, so a row's lanes
    // are in here together
    for (int i = threadIdx.x; i < heads * chunks; i += kThreads) {
        const int h = i / chunks, c = i % chunks;
        double v[8];
        if (h < P.Hq) {
            rotated(P, P.q + (size_t)t * P.q_stride + (size_t)h * kv.D, c, pos, v);
            *reinterpret_cast<u32x4 *>(P.q_out + ((size_t)t * P.Hq + h) * kv.D + 8 * c) = to16(P.dtype, v);
        } else if (h < P.Hq + kv.Hkv) {
            rotated(P, P.k + (size_t)t * P.k_stride + (size_t)(h - P.Hq) * kv.D, c, pos, v);
            store_k(kv, P.dtype, pl, h - P.Hq, c, v);
        } else {
            const int g = h - P.Hq - kv.Hkv;
            const uint16_t *x = P.v + (size_t)t * P.v_stride + (size_t)g * kv.D + 8 * c;
            load8(P.dtype, x, v);
            store_v(kv, pl, g, c, *reinterpret_cast<const u32x4 *>(x), v);
        }
    }
}

}  // namespace

hipError_t launch_kv_append(const AppendParams &P, hipStream_t s)
{
    const uint32_t T = (uint32_t)P.s.T;
    hipLaunchKernelGGL(append_kernel, dim3(T < kGridX ? T : kGridX, (T + kGridX - 1) / kGridX), dim3(kThreads), 0, s, P);
    return hipGetLastError();
}

}  // namespace apmoe
