// Norm of queries and keys per head with the position rotation in the same
// pass, and its gradient.
//
// A row is the D values of one head of one token.  r = (mean x^2 + eps)^-1/2,
// n_d = x_d r w_d, then the first R values turn in pairs (a, b) by the angle
// of the token's table row: y_a = n_a cos - n_b sin, y_b = n_b cos + n_a sin.
// The gradient turns dy back (g = R^T dy), takes dw_d += g_d x_d r and, with
// u = g w and xh = x r, dx = r (u - xh mean(u xh)).
//
// Both are bound by HBM: each value is read and written once.  A row lies
// across LPR lanes of 8 values (16-byte accesses), so its sums take log2(LPR)
// lane exchanges and nothing goes through memory twice.  One lane group takes
// up to four heads of a token: the token's cosines and sines, four bytes for
// each two of a value, are loaded once for them, and four rows are in flight.
// 16 x 4096 tokens of 16 heads and 1024 of 8, 128 values: 117 us forward (5.1
// TB/s); 32 x 3136 and 333 tokens, 8 heads of 64: 40 us forward (5.6 TB/s), 70
// backward (4.9).  One token is a launch and a round trip, 5 us.
#pragma once

#include "attn_common.hpp"

namespace igc {

struct QkPart {
    const uint8_t* x;
    const uint8_t* dy;
    uint8_t* out;          // y forward, dx backward
    const float* w;
    const float* table;    // [table_rows][R]: cosines, then sines
    const int32_t* pos;    // [B][T] rows of the table, or null (the token's number)
    float* dw;
    int64_t pos_b;
    int64_t x_b, x_t, x_h, dy_b, dy_t, dy_h, o_b, o_t, o_h;   // bytes
    int B, T, H;
    int table_rows;
    int hc;                // lane groups a token: ceil(H / kQkHeads)
    int64_t items;         // B * T * hc
    int blocks;            // workgroups
};

struct QkArgs {
    QkPart part[2];        // queries, keys
    float* partial;        // backward: [blocks of q + of k][LPR * 8]
    int D, R;
    float eps, inv_d;
};

enum { ROT_HALVES = 0, ROT_HALVES_ANY = 1, ROT_PAIRS = 2 };
constexpr int kQkHeads = 4;
constexpr int kQkThreads = 256;

template <int LPR>
__device__ __forceinline__ float sum_row(float v) {
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// The token's cosines and sines for the 8 values of chunk c.  Values at or
// past R keep cosine 1, sine 0.  A position outside the table gives NaN.
template <int MODE>
struct Turn {
    float cs[8], sn[8];
    __device__ __forceinline__ void load(const float* table, int64_t row, bool ok, int R, int c) {
        const float* t = table + row * R;
        const int h = R >> 1;
        // a chunk that turns as a whole: 16-byte loads (4-byte aligned)
        typedef float f32x4a __attribute__((ext_vector_type(4), aligned(4)));
        if constexpr (MODE != ROT_HALVES_ANY) {
            if (ok && 8 * c + 8 <= R) {
                if constexpr (MODE == ROT_PAIRS) {
                    const f32x4a x = *reinterpret_cast<const f32x4a*>(t + 4 * c);
                    const f32x4a y = *reinterpret_cast<const f32x4a*>(t + h + 4 * c);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        cs[j] = x[j >> 1];
                        sn[j] = y[j >> 1];
                    }
                } else {
                    const int i = 8 * c < h ? 8 * c : 8 * c - h;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const f32x4a x = *reinterpret_cast<const f32x4a*>(t + i + 4 * k);
                        const f32x4a y = *reinterpret_cast<const f32x4a*>(t + h + i + 4 * k);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            cs[4 * k + j] = x[j];
                            sn[4 * k + j] = y[j];
                        }
                    }
                }
                return;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = 8 * c + j;
            cs[j] = 1.0f;
            sn[j] = 0.0f;
            if (e < R) {
                if (!ok) cs[j] = sn[j] = __builtin_nanf("");
                else {
                    const int i = MODE == ROT_PAIRS ? e >> 1 : (e < h ? e : e - h);
                    cs[j] = t[i];
                    sn[j] = t[h + i];
                }
            }
        }
    }
    // v turned forwards (dir = 1) or back (dir = -1) in place; pad: this
    // wave's 64 * 8 floats of LDS (ROT_HALVES_ANY)
    template <int LPR>
    __device__ __forceinline__ void apply(float* v, float dir, int R, int c, int lane,
                                          float* pad) const {
        float o[8];
        const int h = R >> 1;
        if constexpr (MODE == ROT_PAIRS) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                o[j] = -v[j + 1];
                o[j + 1] = v[j];
            }
        } else if constexpr (MODE == ROT_HALVES) {
            // R / 2 is a multiple of 8: the partners of a chunk are a chunk
            const int hc = h >> 3;
            const int pc = c < hc ? c + hc : c < 2 * hc ? c - hc : c;
            const int from = (lane & ~(LPR - 1)) + pc;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float p = __shfl(v[j], from, 64);
                o[j] = c < hc ? -p : p;
            }
        } else {
            float* row = pad + (lane & ~(LPR - 1)) * 8;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int j = 0; j < 8; ++j) row[8 * c + j] = v[j];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = 8 * c + j;
                const float p = row[e < h ? e + h : e < R ? e - h : e];
                o[j] = e < h ? -p : p;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (8 * c + j < R) v[j] = __builtin_fmaf(o[j], dir * sn[j], v[j] * cs[j]);
    }
};

// Item -> (batch, token, first head).
__device__ __forceinline__ void qk_item(const QkPart& p, int64_t item, int* b, int* t, int* h0) {
    const int64_t bt = item / p.hc;
    *h0 = (int)(item - bt * p.hc) * kQkHeads;
    *b = (int)(bt / p.T);
    *t = (int)(bt - (int64_t)*b * p.T);
}

template <int MODE>
__device__ __forceinline__ void qk_turn(const QkPart& p, int R, int b, int t, int c,
                                        Turn<MODE>* turn) {
    int64_t at = t;
    if (p.pos) at = p.pos[(int64_t)b * p.pos_b + t];
    const bool ok = at >= 0 && at < p.table_rows;
    turn->load(p.table, ok ? at : 0, ok, p.table ? R : 0, c);
}

template <int DT, int LPR, int MODE>
__global__ __launch_bounds__(kQkThreads) void qk_norm_fwd_kernel(QkArgs a) {
    __shared__ __attribute__((aligned(16))) float
        pad[MODE == ROT_HALVES_ANY ? kQkThreads * 8 : 4];
    lds_poison<kQkThreads>(reinterpret_cast<uint8_t*>(pad), sizeof(pad));
    const bool second = (int)blockIdx.x >= a.part[0].blocks;
    const QkPart& p = a.part[second];
    const int lane = threadIdx.x & 63, c = lane % LPR;
    const int64_t item = (int64_t)((int)blockIdx.x - (second ? a.part[0].blocks : 0)) *
                             (kQkThreads / LPR) + threadIdx.x / LPR;
    const bool live = item < p.items;
    int b, t, h0;
    qk_item(p, live ? item : 0, &b, &t, &h0);
    const bool mine = live && c * 8 < a.D;
    const int nh = min(kQkHeads, p.H - h0);

    u32x4 raw[kQkHeads];
    const uint8_t* x = p.x + b * p.x_b + t * p.x_t + h0 * p.x_h + c * 16;
#pragma unroll
    for (int i = 0; i < kQkHeads; ++i)
        raw[i] = mine && i < nh ? *reinterpret_cast<const u32x4*>(x + i * p.x_h)
                                : u32x4{0, 0, 0, 0};
    Turn<MODE> turn;
    qk_turn(p, a.R, b, t, c, &turn);
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = p.w && c * 8 < a.D ? p.w[c * 8 + j] : 1.0f;
    uint8_t* y = p.out + b * p.o_b + t * p.o_t + h0 * p.o_h + c * 16;
#pragma unroll
    for (int i = 0; i < kQkHeads; ++i) {
        float v[8], s = 0.0f;
        unpack8<DT>(raw[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = __builtin_fmaf(v[j], v[j], s);
        s = sum_row<LPR>(s);
        const float r = 1.0f / sqrtf(__builtin_fmaf(s, a.inv_d, a.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] * r * w[j];
        turn.template apply<LPR>(v, 1.0f, a.R, c, lane,
                                 pad + (MODE == ROT_HALVES_ANY ? (threadIdx.x & ~63) * 8 : 0));
        if (mine && i < nh) *reinterpret_cast<u32x4*>(y + i * p.o_h) = pack8<DT>(v);
    }
}

template <int DT, int LPR, int MODE>
__global__ __launch_bounds__(kQkThreads) void qk_norm_bwd_kernel(QkArgs a) {
    __shared__ __attribute__((aligned(16))) float pad[kQkThreads * 8];
    lds_poison<kQkThreads>(reinterpret_cast<uint8_t*>(pad), sizeof(pad));
    const bool second = (int)blockIdx.x >= a.part[0].blocks;
    const QkPart& p = a.part[second];
    const int lane = threadIdx.x & 63, c = lane % LPR;
    const int blk = (int)blockIdx.x - (second ? a.part[0].blocks : 0);
    constexpr int PER = kQkThreads / LPR;
    float w[8], dw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        w[j] = p.w && c * 8 < a.D ? p.w[c * 8 + j] : 1.0f;
        dw[j] = 0.0f;
    }
    // every lane of the workgroup runs the same number of rounds
    const int64_t rounds = (p.items + (int64_t)p.blocks * PER - 1) / ((int64_t)p.blocks * PER);
    for (int64_t k = 0; k < rounds; ++k) {
        const int64_t item = (k * p.blocks + blk) * PER + threadIdx.x / LPR;
        const bool live = item < p.items;
        int b, t, h0;
        qk_item(p, live ? item : 0, &b, &t, &h0);
        const bool mine = live && c * 8 < a.D;
        const int nh = min(kQkHeads, p.H - h0);
        u32x4 rx[kQkHeads], rg[kQkHeads];
        const uint8_t* x = p.x + b * p.x_b + t * p.x_t + h0 * p.x_h + c * 16;
        const uint8_t* g = p.dy + b * p.dy_b + t * p.dy_t + h0 * p.dy_h + c * 16;
#pragma unroll
        for (int i = 0; i < kQkHeads; ++i) {
            const bool on = mine && i < nh;
            rx[i] = on ? *reinterpret_cast<const u32x4*>(x + i * p.x_h) : u32x4{0, 0, 0, 0};
            rg[i] = on ? *reinterpret_cast<const u32x4*>(g + i * p.dy_h) : u32x4{0, 0, 0, 0};
        }
        Turn<MODE> turn;
        qk_turn(p, a.R, b, t, c, &turn);
        uint8_t* dx = p.out + b * p.o_b + t * p.o_t + h0 * p.o_h + c * 16;
#pragma unroll
        for (int i = 0; i < kQkHeads; ++i) {
            float v[8], u[8], s = 0.0f, q = 0.0f;
            unpack8<DT>(rx[i], v);
            unpack8<DT>(rg[i], u);
            turn.template apply<LPR>(u, -1.0f, a.R, c, lane, pad + (threadIdx.x & ~63) * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) s = __builtin_fmaf(v[j], v[j], s);
            s = sum_row<LPR>(s);
            const float r = 1.0f / sqrtf(__builtin_fmaf(s, a.inv_d, a.eps));
            const bool on = mine && i < nh;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] *= r;                                   // xh
                if (on) dw[j] = __builtin_fmaf(u[j], v[j], dw[j]);
                u[j] *= w[j];
                q = __builtin_fmaf(u[j], v[j], q);
            }
            q = sum_row<LPR>(q) * a.inv_d;
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = r * (u[j] - v[j] * q);
            if (on) *reinterpret_cast<u32x4*>(dx + i * p.o_h) = pack8<DT>(u);
        }
    }
    if (!p.dw) return;
    // the workgroup's sum: lane groups in order
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) pad[threadIdx.x * 8 + j] = dw[j];
    __syncthreads();
    if (threadIdx.x < LPR * 8) {
        float s = 0.0f;
        for (int g = 0; g < PER; ++g) s += pad[g * LPR * 8 + threadIdx.x];
        a.partial[(int64_t)blockIdx.x * (LPR * 8) + threadIdx.x] = s;
    }
}

// Sum of the workgroups' partial weight gradients in a fixed order: a
// workgroup takes 16 values of one part, 64 groups of 16 lanes every 64th
// partial, and the groups' sums are added as a tree (4 to 5 us; over 16 groups
// 18 us).
template <int DT>
__global__ __launch_bounds__(1024) void qk_norm_dw_kernel(QkArgs a, int width) {
    __shared__ __attribute__((aligned(16))) float sum[64][17];
    lds_poison<1024>(reinterpret_cast<uint8_t*>(sum), sizeof(sum));
    const int part = blockIdx.y;
    const QkPart& p = a.part[part];
    if (!p.dw) return;
    const int x = threadIdx.x & 15, g = threadIdx.x >> 4, d = blockIdx.x * 16 + x;
    const float* src = a.partial + (int64_t)(part ? a.part[0].blocks : 0) * width;
    float s = 0.0f;
    if (d < width) {
#pragma unroll 8
        for (int i = g; i < p.blocks; i += 64) s += src[(int64_t)i * width + d];
    }
    sum[g][x] = s;
    for (int n = 32; n; n >>= 1) {
        __syncthreads();
        if (g < n) sum[g][x] += sum[g + n][x];
    }
    if (g == 0 && d < a.D) p.dw[d] = sum[0][x];
}

}  // namespace igc
