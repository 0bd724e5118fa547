// Layer norm over the channels, and its gradient.
//
// A row is the C channels of one pixel or token.  mean = sum x / C,
// r = (sum (x - mean)^2 / C + eps)^-1/2, xh = (x - mean) r, y = xh w + b.  The
// gradient, with u = dy w:  dx = r (u - mean(u) - xh mean(u xh)),
// dw = sum over rows of dy xh,  db = sum dy.
//
// Both are bound by HBM: a row stays in the registers of its LPR lanes (NC
// chunks of 8 values a lane), so that the variance is taken about the mean
// (no cancellation), the gradient needs no statistics of the forward pass, and
// each value is read and written once.  100352 rows of 768 in bf16: 55 us forward
// (308 MB, 5.6 TB/s), 93 backward (462 MB, 5.0) and 5.9 for the sum of the
// workgroups' weight gradients, which has to follow in a launch of its own to
// keep its order; 65536 rows of 512 in fp16: 21 us (134 MB, 6.4 TB/s out of the
// Infinity Cache).  A few rows are a launch and a round trip: 2.5 us.
#pragma once

#include "attn_common.hpp"

namespace igc {

struct LnArgs {
    const uint8_t* x;
    const uint8_t* dy;
    uint8_t* out;          // y forward, dx backward
    const float *w, *b;    // [C] or null
    float *dw, *db;        // [C] or null
    float* partial;        // backward: [blocks][2][C]
    int64_t x_s[3], g_s[3], o_s[3];   // row strides of the three leading axes, bytes
    int n1, n2;            // the inner two leading axes
    int flat;              // one stride (index 2) reaches every row
    int rows, C;
    int blocks;            // backward
    float eps, inv_c;
};

typedef uint32_t u32x4h __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4w __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ int64_t ln_row(const LnArgs& a, const int64_t* s, int row) {
    if (a.flat) return row * s[2];
    const int i01 = row / a.n2, i0 = i01 / a.n1;
    return i0 * s[0] + (i01 - i0 * a.n1) * s[1] + (row - i01 * a.n2) * s[2];
}

// 8 values of a row of at least 8 from p (2-byte aligned) on, of which `left` are
// in the row: where those are fewer, the row's last 8, which ln_trim shifts.
__device__ __forceinline__ u32x4 ln_fetch(const uint8_t* p, int left) {
    return u32x4(*reinterpret_cast<const u32x4h*>(p + 2 * (int64_t)min(left - 8, 0)));
}
__device__ __forceinline__ u32x4 ln_trim(u32x4 r, int left) {
    const int s = 8 - left;
    if (s > 0) {
        if (s & 4) r = u32x4{r[2], r[3], 0, 0};
        if (s & 2) r = u32x4{r[1], r[2], r[3], 0};
        if (s & 1)
            r = u32x4{r[0] >> 16 | r[1] << 16, r[1] >> 16 | r[2] << 16,
                      r[2] >> 16 | r[3] << 16, r[3] >> 16};
        if (s >= 8) r = u32x4{0, 0, 0, 0};
    }
    return r;
}
// N chunks of 8 values of a row of C, `step` values apart from p (2-byte
// aligned) on, `left` of them in the row; zeros past it, and only zeros unless
// `live`.  One load a chunk for every lane (154 MB in rows of 1023: 81 us forward
// and 97 backward; value by value 102 and 205), all of them asked for before the
// first is looked at.
template <int N>
__device__ __forceinline__ void ln_load(const uint8_t* p, int left, int step, int C, bool live,
                                        u32x4 (&to)[N]) {
    if (C < 8) {   // one chunk
#pragma unroll
        for (int i = 0; i < N; ++i) to[i] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (live && j < left)
                to[0][j / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + 2 * j)
                                << (16 * (j & 1));
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) to[i] = ln_fetch(p + 2 * i * step, left - i * step);
#pragma unroll
    for (int i = 0; i < N; ++i) to[i] = ln_trim(to[i], live ? left - i * step : 0);
}
template <int DT>
__device__ __forceinline__ void ln_store(uint8_t* p, int left, const float* v) {
    typedef uint32_t u32x2h __attribute__((ext_vector_type(2), aligned(2)));
    typedef uint32_t u32h __attribute__((aligned(2)));
    u32x4 r = pack8<DT>(v);
    if (left >= 8) {
        *reinterpret_cast<u32x4h*>(p) = r;
        return;
    }
    if (left <= 0) return;
    if (left & 4) {
        *reinterpret_cast<u32x2h*>(p) = u32x2{r[0], r[1]};
        p += 8;
        r[0] = r[2];
        r[1] = r[3];
    }
    if (left & 2) {
        *reinterpret_cast<u32h*>(p) = r[0];
        p += 4;
        r[0] = r[1];
    }
    if (left & 1) *reinterpret_cast<uint16_t*>(p) = (uint16_t)r[0];
}
// 8 of the C values of w from c on (`none` without w and past the end).
__device__ __forceinline__ void ln_weights(const float* w, int c, int C, float none, float* v) {
    if (w && c + 8 <= C) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const f32x4w x = *reinterpret_cast<const f32x4w*>(w + c + 4 * k);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * k + j] = x[j];
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = w && c + j < C ? w[c + j] : none;
}

// f(x, y) with y the value of a partner lane whose group of O lanes differs in
// bit log2(O) from this one's, for values that all lanes of a group share (so
// that any lane of the other group will do): lane permutations of the vector
// unit, without a trip through LDS.
template <int O, typename F>
__device__ __forceinline__ uint32_t with_group(uint32_t x, F f) {
    static_assert(O <= 32, "within a wave");
    if constexpr (O == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        const uint32_t a = r[0], b = r[1];
        return f(a, b);
    } else if constexpr (O == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        const uint32_t a = r[0], b = r[1];
        return f(a, b);
    } else {
        // quad_perm 1 0 3 2, 2 3 0 1; half rows and rows mirrored
        constexpr int ctrl = O == 1 ? 0xb1 : O == 2 ? 0x4e : O == 4 ? 0x141 : 0x140;
        return f(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, ctrl, 0xf, 0xf, true));
    }
}
// f over the N lanes of a group, for every lane.
template <int N, int O = 1, typename F>
__device__ __forceinline__ uint32_t over_lanes(uint32_t x, F f) {
    if constexpr (O < N) return over_lanes<N, 2 * O>(with_group<O>(x, f), f);
    return x;
}
template <int N>
__device__ __forceinline__ float sum_lanes(float x) {
    return __builtin_bit_cast(
        float, over_lanes<N>(__builtin_bit_cast(uint32_t, x), [](uint32_t a, uint32_t b) {
            return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) +
                                                    __builtin_bit_cast(float, b));
        }));
}

// Sums over the lanes of a row.  Rows of more than a wave add the waves' sums
// in order through LDS; consecutive sums use the two slots in turn, so that
// one barrier each is enough.
template <int LPR>
struct RowSum {
    static constexpr int NW = LPR > 64 ? LPR / 64 : 1;
    float* lds;   // [2][2][NW]
    int slot = 0;
    __device__ __forceinline__ void add(float& x) {
        float y = 0.0f;
        add<1>(x, y);
    }
    template <int N = 2>
    __device__ __forceinline__ void add(float& x, float& y) {
        x = sum_lanes<(LPR < 64 ? LPR : 64)>(x);
        if constexpr (N > 1) y = sum_lanes<(LPR < 64 ? LPR : 64)>(y);
        if constexpr (LPR > 64) {
            float* s = lds + slot * 2 * NW;
            slot ^= 1;
            const int wave = threadIdx.x >> 6;
            if ((threadIdx.x & 63) == 0) {
                s[wave] = x;
                if constexpr (N > 1) s[NW + wave] = y;
            }
            __syncthreads();
            x = s[0];
#pragma unroll
            for (int w = 1; w < NW; ++w) x += s[w];
            if constexpr (N > 1) {
                y = s[NW];
#pragma unroll
                for (int w = 1; w < NW; ++w) y += s[NW + w];
            }
        }
    }
};

// v -> v - mean (zeros past the row); returns r.
template <int LPR, int NC>
__device__ __forceinline__ float ln_stats(RowSum<LPR>& sum, float (&v)[NC][8], int c0, int C,
                                          float inv_c, float eps) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        float t = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) t += v[i][j];
        s += t;
    }
    sum.add(s);
    // divided, not times the rounded 1 / C: a constant row gives zeros
    const float mean = s / (float)C;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int left = C - (c0 + i * LPR * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[i][j] = j < left ? v[i][j] - mean : 0.0f;
            q = __builtin_fmaf(v[i][j], v[i][j], q);
        }
    }
    sum.add(q);
    return 1.0f / sqrtf(__builtin_fmaf(q, inv_c, eps));
}

template <int DT, int LPR, int NC, int NT>
__global__ __launch_bounds__(NT) void layer_norm_fwd_kernel(LnArgs a) {
    __shared__ __attribute__((aligned(16))) float red[4 * RowSum<LPR>::NW];
    lds_poison<NT>(reinterpret_cast<uint8_t*>(red), sizeof(red));
    RowSum<LPR> sum{red};
    const int c0 = (int)(threadIdx.x % LPR) * 8;
    const int row = (int)(blockIdx.x * (NT / LPR) + threadIdx.x / LPR);
    const bool live = row < a.rows;   // rows of more than a wave always are
    const uint8_t* x = a.x + (live ? ln_row(a, a.x_s, row) : 0);
    u32x4 raw[NC];
    ln_load(x + 2 * c0, a.C - c0, LPR * 8, a.C, live, raw);
    float v[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) unpack8<DT>(raw[i], v[i]);
    // Weights asked for before the sums save their round trip, and cost waves
    // by their registers (154 MB: 64 channels 59 us, after the sums 65; 16384 65
    // and 70; but 333 99 and 89, 4096 72 and 65).
    constexpr bool EARLY = LPR > 64 ? NC >= 3 : NC <= 2;
    float w[NC][8], b[NC][8];
    auto weights = [&](int i) {
        ln_weights(a.w, c0 + i * LPR * 8, a.C, 1.0f, w[i]);
        ln_weights(a.b, c0 + i * LPR * 8, a.C, 0.0f, b[i]);
    };
    if constexpr (EARLY) {
#pragma unroll
        for (int i = 0; i < NC; ++i) weights(i);
    }
    const float r = ln_stats<LPR, NC>(sum, v, c0, a.C, a.inv_c, a.eps);
    if (!live) return;
    uint8_t* y = a.out + ln_row(a, a.o_s, row);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = c0 + i * LPR * 8;
        if constexpr (!EARLY) weights(i);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = __builtin_fmaf(v[i][j] * r, w[i][j], b[i][j]);
        ln_store<DT>(y + 2 * c, a.C - c, v[i]);
    }
}

// Workgroups walk the rows, so that the partial gradients of the weights stay
// few; every lane of a workgroup runs the same number of rounds.
template <int DT, int LPR, int NC, int NT>
__global__ __launch_bounds__(NT) void layer_norm_bwd_kernel(LnArgs a) {
    constexpr int PER = NT / LPR;
    constexpr int W = LPR * NC * 8;   // channels of a row, rounded up
    __shared__ __attribute__((aligned(16))) float red[PER > 1 ? PER * W : 4 * RowSum<LPR>::NW];
    lds_poison<NT>(reinterpret_cast<uint8_t*>(red), sizeof(red));
    RowSum<LPR> sum{red};
    const int c0 = (int)(threadIdx.x % LPR) * 8;
    float w[NC][8], dw[NC][8], db[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        ln_weights(a.w, c0 + i * LPR * 8, a.C, 1.0f, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.0f;
    }
    const int rounds = (int)(((int64_t)a.rows + (int64_t)a.blocks * PER - 1) /
                             ((int64_t)a.blocks * PER));
    // A workgroup that takes one row at a time asks for the next one's values
    // before it sums up this one's; where waves have rows of their own, the
    // other waves' requests fill the gap.
    constexpr bool AHEAD = LPR > 64;
    auto row_of = [&](int k) { return ((int64_t)k * a.blocks + blockIdx.x) * PER + threadIdx.x / LPR; };
    auto load = [&](const uint8_t* p, const int64_t* s, int64_t at, u32x4 (&to)[NC]) {
        const bool live = at < a.rows;
        const uint8_t* x = p + ln_row(a, s, live ? (int)at : 0);
        // a chunk at a time: together they take two registers too many for a
        // third workgroup a CU (333 channels: 96 us, 127)
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = c0 + i * LPR * 8;
            if constexpr (AHEAD) {   // trimmed in its turn (8191: 113 us, at once 166)
                to[i] = ln_fetch(x + 2 * c, a.C - c);
            } else {
                u32x4 one[1];
                ln_load(x + 2 * c, a.C - c, 0, a.C, live, one);
                to[i] = one[0];
            }
        }
    };
    u32x4 rx[NC], rg[NC], ng[NC];
    if constexpr (AHEAD) {
        load(a.x, a.x_s, row_of(0), rx);
        load(a.dy, a.g_s, row_of(0), ng);
    }
    for (int k = 0; k < rounds; ++k) {
        const int64_t at = row_of(k);
        const bool live = at < a.rows;
        const int row = live ? (int)at : 0;
        if constexpr (!AHEAD) {
            load(a.x, a.x_s, at, rx);
            load(a.dy, a.g_s, at, rg);
        }
        float v[NC][8];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if constexpr (AHEAD) {
                const int left = live ? a.C - (c0 + i * LPR * 8) : 0;
                rx[i] = ln_trim(rx[i], left);
                rg[i] = ln_trim(ng[i], left);
            }
            unpack8<DT>(rx[i], v[i]);
        }
        if constexpr (AHEAD) {
            if (k + 1 < rounds) {
                load(a.x, a.x_s, row_of(k + 1), rx);
                load(a.dy, a.g_s, row_of(k + 1), ng);
            }
        }
        float r = ln_stats<LPR, NC>(sum, v, c0, a.C, a.inv_c, a.eps);
        if (!live) r = 0.0f;   // eps = 0 gives infinity there
        float s = 0.0f, q = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float u[8];
            unpack8<DT>(rg[i], u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] *= r;   // xh
                // rows past the last hold zeros in u
                dw[i][j] = __builtin_fmaf(u[j], v[i][j], dw[i][j]);
                db[i][j] += u[j];
                const float t = u[j] * w[i][j];
                s += t;
                q = __builtin_fmaf(t, v[i][j], q);
            }
        }
        sum.add(s, q);
        s *= a.inv_c;
        q *= a.inv_c;
        if (live) {
            uint8_t* dx = a.out + ln_row(a, a.o_s, row);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = c0 + i * LPR * 8;
                float u[8];
                unpack8<DT>(rg[i], u);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    u[j] = r * (__builtin_fmaf(u[j], w[i][j], -s) - v[i][j] * q);
                ln_store<DT>(dx + 2 * c, a.C - c, u);
            }
        }
    }
    if (!a.partial) return;
    // the workgroup's sums, row groups in order
    float* dst = a.partial + (int64_t)blockIdx.x * 2 * a.C;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        if constexpr (PER > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    red[(threadIdx.x / LPR) * W + c0 + i * LPR * 8 + j] = p ? db[i][j] : dw[i][j];
            __syncthreads();
            for (int c = threadIdx.x; c < a.C; c += NT) {
                float s = 0.0f;
#pragma unroll
                for (int g = 0; g < PER; ++g) s += red[g * W + c];
                dst[p * a.C + c] = s;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = c0 + i * LPR * 8 + j;
                    if (c < a.C) dst[p * a.C + c] = p ? db[i][j] : dw[i][j];
                }
        }
    }
}

// Sum of the workgroups' partial gradients of weight and bias in a fixed
// order: a workgroup takes 16 of the 2 C values, 64 groups of 16 lanes every
// 64th partial, and the groups' sums are added as a tree.
template <int DT>
__global__ __launch_bounds__(1024) void layer_norm_dw_kernel(LnArgs a) {
    __shared__ __attribute__((aligned(16))) float sum[64][17];
    lds_poison<1024>(reinterpret_cast<uint8_t*>(sum), sizeof(sum));
    const int x = threadIdx.x & 15, g = threadIdx.x >> 4;
    const int c = (int)blockIdx.x * 16 + x, n = 2 * a.C;
    float s = 0.0f;
    if (c < n) {
#pragma unroll 8
        for (int i = g; i < a.blocks; i += 64) s += a.partial[(int64_t)i * n + c];
    }
    sum[g][x] = s;
    for (int k = 32; k; k >>= 1) {
        __syncthreads();
        if (g < k) sum[g][x] += sum[g + k][x];
    }
    if (g == 0 && c < n) {
        float* dst = c < a.C ? a.dw : a.db;
        if (dst) dst[c < a.C ? c : c - a.C] = sum[0][x];
    }
}

}  // namespace igc
