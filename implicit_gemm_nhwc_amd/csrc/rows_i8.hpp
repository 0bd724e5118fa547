// Rows held in 8 bits: integers and one fp32 scale a row.
//
//   m = max |x|,  s = m / 127,  q_i = round(127 x_i / m), ties to even.
//
// The quotient is formed so that its rounding to an integer is the exact
// one.  a = 127 x is exact in fp32 (11 and 7 bits).  t = a r, r the hardware's
// reciprocal of m, is within a few units in the last place; t + (a - t m) r has
// the quotient's error squared before its own rounding.  Where 127 x / m is a
// half-integer it is a short binary number, so that the result is exactly it;
// elsewhere it differs from every half-integer by more than 2^-19 of itself
// (the quotient of integers below 2^18 and 2^11), and fp32 cannot cross that.
#pragma once

#include "layer_norm.hpp"

namespace igc {

struct RowScale {
    float scale;   // what a step of the integers stands for
    float mul;     // a = x mul: 127 times the power of two that keeps m in range
    float m, r;    // m times that power, and its reciprocal
    uint32_t keep; // 0 for rows of zeros, infinities or NaNs
};

// Largest |x| of 8 values of a 16-bit type as its bits, in pairs: an infinity or
// a NaN compares above every number.
__device__ __forceinline__ uint32_t top_pairs(const u32x4& raw, uint32_t top) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int k = 0; k < 4; ++k)
        top = __builtin_bit_cast(
            uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, top),
                                                __builtin_bit_cast(u16x2, raw[k] & 0x7fff7fffu)));
    return top;
}

// From the row's largest |x| as the type's bits.
template <int DT>
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
    const float m = DT == DT_FP16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)top)
                                  : __builtin_bit_cast(float, top << 16);
    const bool bad = top >= (DT == DT_FP16 ? 0x7c00u : 0x7f80u), none = m < 0x1p-110f;
    const float f = m > 0x1p96f ? 0x1p-64f : m < 0x1p-60f ? 0x1p64f : 1.0f;
    RowScale s;
    s.keep = bad || none ? 0u : ~0u;
    s.mul = 127.0f * f;
    s.m = bad || none ? 1.0f : m * f;
    s.r = __builtin_amdgcn_rcpf(s.m);
    s.scale = bad ? __builtin_nanf("") : none ? 0.0f : m / 127.0f;
    return s;
}

// 8 values as 8 bytes.
__device__ __forceinline__ u32x2 row_bytes(const float* v, const RowScale& s) {
    uint32_t b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float a = v[j] * s.mul;
        float t = a * s.r;
        t = __builtin_fmaf(__builtin_fmaf(-t, s.m, a), s.r, t);
        // 1.5 2^23 + t rounds t to the nearest integer, ties to even, and has
        // it in its low bits
        b[j] = __builtin_bit_cast(uint32_t, t + 0x1.8p23f);
    }
    u32x2 o;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        o[k] = __builtin_amdgcn_perm(
                   __builtin_amdgcn_perm(b[4 * k + 3], b[4 * k + 2], 0x0c0c0400u),
                   __builtin_amdgcn_perm(b[4 * k + 1], b[4 * k], 0x0c0c0400u), 0x05040100u) &
               s.keep;
    return o;
}

// Maximum of the pairs over the lanes of a row (RowSum's way).
template <int LPR>
__device__ __forceinline__ uint32_t row_top(uint32_t top, uint32_t* lds) {
    top = max(top & 0xffffu, top >> 16);
    top = over_lanes<(LPR < 64 ? LPR : 64)>(top,
                                            [](uint32_t a, uint32_t b) { return max(a, b); });
    if constexpr (LPR > 64) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = top;
        __syncthreads();
        top = lds[0];
#pragma unroll
        for (int w = 1; w < LPR / 64; ++w) top = max(top, lds[w]);
    }
    return top;
}

struct QuantArgs {
    const uint8_t* x;
    uint8_t* q;
    float* scale;          // [rows]
    int64_t x_s[3], q_s[3];   // bytes
    int n1, n2, flat;
    int rows, C;
};

// Bound by HBM: a row stays in its lanes' registers between the maximum and
// the rounding (LONG, past 16384 values: all but its last piece is read twice).
// 16384 rows of 4096 out of HBM: 36 to 43 us, 39 on average (201 MB, 5.1 TB/s;
// vector units 78 % busy); in rows of 1023 33 us, of 4096 32 out of the Infinity
// Cache.
template <int DT, int LPR, int NC, int NT, bool LONG>
__global__ __launch_bounds__(NT) void quantize_rows_kernel(QuantArgs a) {
    constexpr int W = LPR * NC * 8;
    __shared__ __attribute__((aligned(16))) uint32_t red[LPR > 64 ? LPR / 64 : 4];
    lds_poison<NT>(reinterpret_cast<uint8_t*>(red), sizeof(red));
    const int c0 = (int)(threadIdx.x % LPR) * 8;
    const int row = (int)(blockIdx.x * (NT / LPR) + threadIdx.x / LPR);
    const bool live = row < a.rows;   // rows of more than a wave always are
    const int at = live ? row : 0;
    const int i01 = a.flat ? 0 : at / a.n2, i0 = a.flat ? 0 : i01 / a.n1;
    const int i1 = i01 - i0 * a.n1, i2 = at - i01 * a.n2;
    const uint8_t* x = a.x + i0 * a.x_s[0] + i1 * a.x_s[1] + i2 * a.x_s[2];
    u32x4 raw[NC];
    uint32_t top = 0;
    const int segs = LONG ? (a.C + W - 1) / W : 1;
    for (int s = 0; s < segs; ++s) {
        ln_load(x + 2 * (s * W + c0), a.C - (s * W + c0), LPR * 8, a.C, live, raw);
#pragma unroll
        for (int i = 0; i < NC; ++i) top = top_pairs(raw[i], top);
    }
    const RowScale rs = row_scale<DT>(row_top<LPR>(top, red));
    if (!live) return;
    uint8_t* q = a.q + i0 * a.q_s[0] + i1 * a.q_s[1] + i2 * a.q_s[2];
    for (int s = segs - 1; s >= 0; --s) {   // the last piece is still here
        if (s < segs - 1)
            ln_load(x + 2 * (s * W + c0), a.C - (s * W + c0), LPR * 8, a.C, true, raw);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = s * W + c0 + i * LPR * 8, left = a.C - c;
            float v[8];
            unpack8<DT>(raw[i], v);
            const u32x2 o = row_bytes(v, rs);
            if (left >= 8) {
                *reinterpret_cast<u32x2*>(q + c) = o;
            } else if (left > 0) {
                uint32_t w = o[0];
                uint8_t* to = q + c;
                if (left & 4) {
                    *reinterpret_cast<uint32_t*>(to) = w;
                    to += 4;
                    w = o[1];
                }
                if (left & 2) {
                    *reinterpret_cast<uint16_t*>(to) = (uint16_t)w;
                    to += 2;
                    w >>= 16;
                }
                if (left & 1) *to = (uint8_t)w;
            }
        }
    }
    if (c0 == 0) a.scale[row] = rs.scale;
}

}  // namespace igc
