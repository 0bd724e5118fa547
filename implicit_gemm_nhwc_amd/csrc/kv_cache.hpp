// The paged cache of keys and values in 8 bits: writing and reading back.
//
// Pages hold [kv heads][page tokens][D rounded up to 16] integers and
// [kv heads][page tokens] scales: the rows that one head's attention walks lie
// side by side.  Both kernels are bound by HBM.  LPR lanes of 8 values take a
// row; a lane group takes the same token of up to four heads, neighbouring
// groups neighbouring tokens, so that a wave reads whole heads of a token and
// writes runs of a page.
#pragma once

#include "cache_plan.hpp"
#include "rows_i8.hpp"

namespace igc {

struct CacheArgs {
    int8_t* pool[2];       // keys, values
    float* scale[2];
    uint8_t* t[2];         // the 16-bit tensors [B, T, H, D]
    int64_t t_b[2], t_t[2], t_h[2];   // bytes
    const int32_t* table;
    const int32_t* start;
    const int32_t* lens;   // tokens of each sequence, or null (T)
    int64_t table_stride;
    int B, T, H, D, Dp;
    int hc;                // lane groups a token: ceil(H / kCacheHeads)
    int64_t items;         // B * hc * T
    int entries, pages, shift;
};

constexpr int kCacheHeads = 4, kCacheThreads = 256;

// What a lane group works on: heads h0 .. h0 + nh - 1 of token t of sequence b,
// at position p of page `id` (-1: none).  `given` is false for tokens past the
// sequence's length.
struct CacheItem {
    int b, t, h0, nh, id;
    int64_t p;
    bool given;
};
__device__ __forceinline__ CacheItem cache_item(const CacheArgs& a, int64_t item) {
    CacheItem x;
    const bool live = item < a.items;
    const int64_t at = live ? item : 0, bh = at / a.T;
    x.t = (int)(at - bh * a.T);
    x.b = (int)(bh / a.hc);
    x.h0 = (int)(bh - (int64_t)x.b * a.hc) * kCacheHeads;
    x.nh = live ? min(kCacheHeads, a.H - x.h0) : 0;
    x.given = x.t < (a.lens ? a.lens[x.b] : a.T);
    x.p = (int64_t)a.start[x.b] + x.t;
    x.id = x.given ? cache_page(a.table + x.b * a.table_stride, x.p, a.shift, a.entries, a.pages)
                   : -1;
    return x;
}

template <int DT, int LPR>
__global__ __launch_bounds__(kCacheThreads) void kv_cache_write_kernel(CacheArgs a) {
    const int which = blockIdx.y, c = (int)(threadIdx.x % LPR) * 8;
    const CacheItem x = cache_item(
        a, (int64_t)blockIdx.x * (kCacheThreads / LPR) + threadIdx.x / LPR);
    // the rows of a wave are summed up together: no lane leaves before that
    const int nh = x.id >= 0 && c < a.D ? x.nh : 0;
    const uint8_t* src = a.t[which] + x.b * a.t_b[which] + x.t * a.t_t[which] +
                         x.h0 * a.t_h[which] + 2 * c;
    u32x4 raw[kCacheHeads];
#pragma unroll
    for (int i = 0; i < kCacheHeads; ++i)
        raw[i] = i < nh ? *reinterpret_cast<const u32x4*>(src + i * a.t_h[which])
                        : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kCacheHeads; ++i) {
        float v[8];
        unpack8<DT>(raw[i], v);
        const RowScale rs = row_scale(row_top<LPR>(top_bits(v, 0), nullptr));
        if (i < nh) {
            const int64_t row = cache_row(x.id, a.H, x.h0 + i, x.p, a.shift);
            *reinterpret_cast<u32x2*>(a.pool[which] + row * a.Dp + c) = row_bytes(v, rs);
            if (c == 0) a.scale[which][row] = rs.scale;
        }
    }
}

// Every token of the output is written: zeros past a sequence's length, NaN
// where its position or page does not exist.
template <int DT, int LPR>
__global__ __launch_bounds__(kCacheThreads) void kv_cache_read_kernel(CacheArgs a) {
    const int which = blockIdx.y, c = (int)(threadIdx.x % LPR) * 8;
    const CacheItem x = cache_item(
        a, (int64_t)blockIdx.x * (kCacheThreads / LPR) + threadIdx.x / LPR);
    if (c >= a.D) return;
    u32x2 raw[kCacheHeads];
    float scale[kCacheHeads];
#pragma unroll
    for (int i = 0; i < kCacheHeads; ++i) {
        raw[i] = u32x2{0, 0};
        scale[i] = x.given ? __builtin_nanf("") : 0.0f;
        if (x.id >= 0 && i < x.nh) {
            const int64_t row = cache_row(x.id, a.H, x.h0 + i, x.p, a.shift);
            raw[i] = *reinterpret_cast<const u32x2*>(a.pool[which] + row * a.Dp + c);
            scale[i] = a.scale[which][row];
        }
    }
    uint8_t* dst = a.t[which] + x.b * a.t_b[which] + x.t * a.t_t[which] + x.h0 * a.t_h[which] +
                   2 * c;
#pragma unroll
    for (int i = 0; i < kCacheHeads; ++i) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = (float)(int8_t)(raw[i][j / 4] >> (8 * (j & 3))) * scale[i];
        if (i < x.nh) *reinterpret_cast<u32x4*>(dst + i * a.t_h[which]) = pack8<DT>(v);
    }
}

}  // namespace igc
