// The paged cache of keys and values in 8 bits: writing and reading back.
//
// Pages hold [kv heads][page tokens][D rounded up to 16] integers and
// [kv heads][page tokens] scales: the rows that one head's attention walks lie
// side by side.  Both kernels are bound by HBM.  LPR lanes of 8 values take a
// row; a lane group takes a token of up to four heads, a workgroup a run of
// tokens of them.  Workgroups that follow one another take the other heads of
// the same tokens, and then their values: together they go through whole rows
// of the 16-bit tensors (16 x 4096 tokens written and read, 8 heads of 128: 151
// us; keys first, and heads by fours, 162).  With the rows asked for together
// and the maxima over lanes by permutations the two take 64 to 82 and 58 to 63 us
// of kernels (5.0 to 3.9 and 6.2 to 5.7 TB/s, vector units 72 and 43 % busy; ragged
// lengths, of which the whole output is written back).
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
    int hc;                // workgroups a run of tokens: ceil(H / kCacheHeads)
    int runs;              // runs of tokens a sequence
    int entries, pages, shift;
};

constexpr int kCacheHeads = 4, kCacheThreads = 256;

// Tokens a workgroup (of lpr lanes a row).
constexpr int cache_run(int lpr) { return kCacheThreads / lpr; }

// What a lane group works on: heads h0 .. h0 + nh - 1 of the keys (0) or values
// of token t of sequence b, at position p of page `id` (-1: none).  `given` is
// false for tokens past the sequence's length.
struct CacheItem {
    int which, b, t, h0, nh, id;
    int64_t p;
    bool given;
};
template <int LPR>
__device__ __forceinline__ CacheItem cache_item(const CacheArgs& a) {
    CacheItem x;
    const int kv = blockIdx.x / a.hc, run = kv >> 1;
    x.which = kv & 1;
    x.h0 = (int)(blockIdx.x - kv * a.hc) * kCacheHeads;
    x.b = run / a.runs;
    x.t = (run - x.b * a.runs) * cache_run(LPR) + threadIdx.x / LPR;
    const bool live = x.t < a.T;
    if (!live) x.t = 0;
    x.nh = live ? min(kCacheHeads, a.H - x.h0) : 0;
    x.given = x.t < (a.lens ? a.lens[x.b] : a.T);
    x.p = (int64_t)a.start[x.b] + x.t;
    x.id = x.given ? cache_page(a.table + x.b * a.table_stride, x.p, a.shift, a.entries, a.pages)
                   : -1;
    return x;
}

template <int DT, int LPR>
__global__ __launch_bounds__(kCacheThreads) void kv_cache_write_kernel(CacheArgs a) {
    const int c = (int)(threadIdx.x % LPR) * 8;
    const CacheItem x = cache_item<LPR>(a);
    const int which = x.which;
    // The rows are asked for before the page is known, all at once: where there
    // is none to take, the group's first, which exists.
    const int nr = x.given && c < a.D ? x.nh : 0;
    if (!__any(nr > 0)) return;   // whole waves: the maxima are theirs
    const uint8_t* src = a.t[which] + x.b * a.t_b[which] + x.t * a.t_t[which] +
                         x.h0 * a.t_h[which] + (c < a.D ? 2 * c : 0);
    u32x4 raw[kCacheHeads];
#pragma unroll
    for (int i = 0; i < kCacheHeads; ++i)
        raw[i] = *reinterpret_cast<const u32x4*>(src + (i < nr ? i : 0) * a.t_h[which]);
    const int nh = x.id >= 0 ? nr : 0;
#pragma unroll
    for (int i = 0; i < kCacheHeads; ++i) {
        if (i >= nr) raw[i] = u32x4{0, 0, 0, 0};
        const RowScale rs = row_scale<DT>(row_top<LPR>(top_pairs(raw[i], 0), nullptr));
        if (i < nh) {
            float v[8];
            unpack8<DT>(raw[i], v);
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
    const int c = (int)(threadIdx.x % LPR) * 8;
    const CacheItem x = cache_item<LPR>(a);
    const int which = x.which;
    if (c >= a.D) return;
    u32x2 raw[kCacheHeads];
    float scale[kCacheHeads];
    if (a.pages > 0) {   // a page 0 exists
#pragma unroll
        for (int i = 0; i < kCacheHeads; ++i) {
            const int64_t row = x.id >= 0 && i < x.nh
                                    ? cache_row(x.id, a.H, x.h0 + i, x.p, a.shift) : 0;
            raw[i] = *reinterpret_cast<const u32x2*>(a.pool[which] + row * a.Dp + c);
            scale[i] = a.scale[which][row];
        }
    }
#pragma unroll
    for (int i = 0; i < kCacheHeads; ++i)
        if (x.id < 0) {
            raw[i] = u32x2{0, 0};
            scale[i] = x.given ? __builtin_nanf("") : 0.0f;
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
