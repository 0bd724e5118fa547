// Host-side checks shared by the attention operators and those around them:
// views of tensors, overlaps, launch sizes.
#pragma once

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "igemm_attn.h"

namespace igc {

constexpr int64_t kLim31 = (int64_t)1 << 31;
constexpr int64_t kStrideLim = (int64_t)1 << 23;        // strides within a tile, elements
constexpr int64_t kBatchStrideLim = (int64_t)1 << 40;   // strides between 64-bit bases, elements
constexpr double kExtentLim = 0x1p56;                   // no address space holds more

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Whether a launch of so many workgroups holds fewer than 2^32 threads; HIP
// takes the count modulo 2^32 (2^24 - 16 workgroups of 512 threads ran half of
// themselves and reported success).
inline bool launchable(int64_t groups, int64_t threads) {
    return groups <= (((int64_t)1 << 32) - 1) / threads;
}

inline bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

inline bool meet(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + nb && b0 < a0 + na;
}

// A tensor [batch, token, head, d] behind a view: its byte range, with the
// strides of axes of one entry (which say nothing) taken as 0.
struct Tensor {
    const void* p;
    int64_t b, t, h;   // strides, bytes
    size_t bytes;      // first to last element
};

// Gate of one view; `write` for outputs.  Empty tensors may be NULL.
inline int32_t check_view(const igc_attn_view& v, int64_t nb, int64_t nt, int64_t nh, int64_t d,
                   bool write, int64_t head_lim, Tensor* out) {
    Tensor x{v.data, 0, 0, 0, 0};
    const int64_t n[3] = {nb, nt, nh};
    int64_t s[3] = {v.batch, v.token, v.head};
    if (nb == 0 || nt == 0 || nh == 0) {
        *out = x;
        return IGC_OK;
    }
    if (!v.data) return IGC_DECLINE_NULL_POINTER;
    if (!aligned(v.data, 16)) return IGC_DECLINE_ALIGNMENT;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) s[i] = 0;
        if (s[i] < 0) return IGC_DECLINE_STRIDE;
        if (s[i] % 8) return IGC_DECLINE_ALIGNMENT;
        if (s[i] >= (i == 0 ? kBatchStrideLim : i == 1 ? kStrideLim : head_lim))
            return IGC_DECLINE_SIZE_LIMIT;
    }
    if ((double)nb * (double)s[0] + (double)nt * (double)s[1] + (double)nh * (double)s[2] >
        kExtentLim)
        return IGC_DECLINE_SIZE_LIMIT;
    if (write) {
        // axes from the smallest stride up: each has to step over all before
        int ord[3] = {0, 1, 2};
        for (int i = 0; i < 3; ++i)
            for (int j = i + 1; j < 3; ++j)
                if (s[ord[j]] < s[ord[i]]) { const int t = ord[i]; ord[i] = ord[j]; ord[j] = t; }
        int64_t ext = d;
        for (int i = 0; i < 3; ++i) {
            const int k = ord[i];
            if (n[k] == 1) continue;
            if (s[k] < ext) return IGC_DECLINE_OVERLAP;
            ext += (n[k] - 1) * s[k];
        }
    }
    x.b = s[0] * 2;
    x.t = s[1] * 2;
    x.h = s[2] * 2;
    x.bytes = (size_t)((n[0] - 1) * x.b + (n[1] - 1) * x.t + (n[2] - 1) * x.h + d * 2);
    *out = x;
    return IGC_OK;
}

}  // namespace igc
