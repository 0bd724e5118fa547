// Product of two matrices of 8-bit integers with a scale a row of each:
//   y[m][n] = (sum_k x[m][k] w[n][k]) xs[m] ws[n] + bias[n]
//
// Both operands have k adjacent, as the matrix instructions take them (16 k a
// lane).  w is the A operand and x the B operand, so that a lane of the result
// owns one row of y and neighbouring columns.  The integer sums are exact; they
// are scaled in fp32 and rounded once.
//
// The tile kernel stages 128 k of its rows and columns in LDS by direct loads,
// double buffered; the few-rows kernel, which the weights' bytes bound, takes
// 16 columns a workgroup, gives each wave a part of k and reads both operands
// straight into registers.
#pragma once

#include "layer_norm.hpp"

namespace igc {

typedef int i32x16 __attribute__((ext_vector_type(16)));

struct LinArgs {
    const uint8_t *x, *w;
    const float *xs, *ws, *bias;
    uint8_t* y;
    int64_t x_p, w_p, y_p;   // row pitches, bytes
    int M, N, K, K16;        // K16: K rounded up to whole 16-byte chunks
    int tiles_m, tiles_n;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t lin_rsrc(const uint8_t* base, unsigned bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), (short)0, (int)bytes,
                                             0x00020000);
}
// Bytes from the first of `rows` rows of 16-byte chunks to the end of the last.
__device__ __forceinline__ unsigned lin_bytes(int rows, int64_t pitch, int K16) {
    return rows > 0 ? (unsigned)((rows - 1) * pitch) + (unsigned)K16 : 0u;
}

// Chunk of 16 bytes with those from `left` on cleared.
__device__ __forceinline__ i32x4 lin_clear(i32x4 v, int left) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = left - 4 * i;   // bytes kept of this word
        v[i] = n >= 4 ? v[i] : n <= 0 ? 0 : v[i] & (int)((1u << (8 * n)) - 1);
    }
    return v;
}

// Columns n .. n + 3 of row m.
template <int DT>
__device__ __forceinline__ void lin_store4(const LinArgs& a, int m, int n, const int* acc) {
    typedef uint32_t u32x2h __attribute__((ext_vector_type(2), aligned(2)));
    const float xs = a.xs[m];
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = min(n + i, a.N - 1);
        v[i] = (float)acc[i] * xs * a.ws[c] + (a.bias ? a.bias[c] : 0.0f);
    }
    const u32x2 o = {pack_out2(v[0], v[1], DT), pack_out2(v[2], v[3], DT)};
    uint8_t* y = a.y + (int64_t)m * a.y_p + 2 * (int64_t)n;
    if (n + 4 <= a.N) {
        *reinterpret_cast<u32x2h*>(y) = o;
        return;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (n + i < a.N)
            *reinterpret_cast<uint16_t*>(y + 2 * i) = (uint16_t)(o[i / 2] >> (16 * (i & 1)));
}

// ---------------------------------------------------------------------------
// At most 16 MT rows.
constexpr int kFewWaves = 8;
template <int DT, int MT>
__global__ __launch_bounds__(kFewWaves * 64) void linear_i8_few_kernel(LinArgs a) {
    __shared__ __attribute__((aligned(16))) int part[kFewWaves][MT][64][4];
    lds_poison<kFewWaves * 64>(reinterpret_cast<uint8_t*>(part), sizeof(part));
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int n0 = (int)blockIdx.x * 16;
    const __amdgpu_buffer_rsrc_t wr = lin_rsrc(
        a.w + n0 * a.w_p, lin_bytes(min(16, a.N - n0), a.w_p, a.K16));
    const __amdgpu_buffer_rsrc_t xr = lin_rsrc(a.x, lin_bytes(a.M, a.x_p, a.K16));
    // lane l: row l % 16, 16 k from 16 (l / 16) on; a wave takes 128 k of each
    // row (a line) and then the waves' next 128
    const unsigned woff = (unsigned)((lane & 15) * a.w_p) + 16 * (lane >> 4);
    const unsigned xoff = (unsigned)((lane & 15) * a.x_p) + 16 * (lane >> 4);
    const unsigned xrow = (unsigned)(16 * a.x_p);
    i32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = i32x4{0, 0, 0, 0};
    constexpr int STEP = kFewWaves * 128;
    auto at = [&](int k) { return k + 16 * (lane >> 4); };   // first k of the lane's chunk
    i32x4 w[2], nw[2];
    const int k0 = wave * 128;
    auto load_w = [&](int k, i32x4* to) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
            to[s] = __builtin_bit_cast(i32x4, load16(wr, at(k + 64 * s) < a.K
                                                             ? woff + k + 64 * s : kOut));
    };
    load_w(k0, w);
    for (int k = k0; k < a.K; k += STEP) {
        load_w(k + STEP, nw);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int c = at(k + 64 * s);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                i32x4 x = __builtin_bit_cast(
                    i32x4, load16(xr, c < a.K ? xoff + t * xrow + k + 64 * s : kOut));
                if (c + 16 > a.K) x = lin_clear(x, a.K - c);
                acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[s], x, acc[t], 0, 0, 0);
            }
        }
        w[0] = nw[0];
        w[1] = nw[1];
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) *reinterpret_cast<i32x4*>(part[wave][t][lane]) = acc[t];
    __syncthreads();
    // result: lane l has row l % 16 of x, columns 4 (l / 16) .. + 3
    for (int e = threadIdx.x; e < MT * 64; e += kFewWaves * 64) {
        const int t = e >> 6, l = e & 63, m = 16 * t + (l & 15), n = n0 + 4 * (l >> 4);
        i32x4 s = *reinterpret_cast<const i32x4*>(part[0][t][l]);
#pragma unroll
        for (int v = 1; v < kFewWaves; ++v)
            s += *reinterpret_cast<const i32x4*>(part[v][t][l]);
        if (m < a.M && n < a.N) {
            const int v[4] = {s[0], s[1], s[2], s[3]};
            lin_store4<DT>(a, m, n, v);
        }
    }
}

// ---------------------------------------------------------------------------
// Tiles of BM rows of x and BN of w, WM x WN waves.
constexpr int kLinKT = 128;   // k a tile, bytes
template <int DT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void linear_i8_tile_kernel(LinArgs a) {
    constexpr int NW = WM * WN, MB = BM / WM / 32, NB = BN / WN / 32;
    constexpr int XT = BM * kLinKT, WT = BN * kLinKT;
    constexpr int XP = XT / 1024 / NW, WP = WT / 1024 / NW;   // loads a wave
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];   // 2 x {x, w}
    lds_poison<NW * 64>(lds, 2 * (XT + WT));
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wm = wave / WN, wn = wave % WN, half = lane >> 5;

    // an XCD's run of tiles goes through bands of 8 tiles of x, column by
    // column: the workgroups that run at once share both operands in its L2
    const int tile = xcd_remap(blockIdx.x, gridDim.x);
    const int band = tile / (8 * a.tiles_n), rows = min(8, a.tiles_m - 8 * band);
    const int in = tile - band * 8 * a.tiles_n;
    const int m0 = (8 * band + in % rows) * BM, n0 = in / rows * BN;

    const __amdgpu_buffer_rsrc_t xr = lin_rsrc(
        a.x + m0 * a.x_p, lin_bytes(min(BM, a.M - m0), a.x_p, a.K16));
    const __amdgpu_buffer_rsrc_t wr = lin_rsrc(
        a.w + n0 * a.w_p, lin_bytes(min(BN, a.N - n0), a.w_p, a.K16));
    // a piece is 8 rows; the 16-byte chunk c of row r lies at c ^ (r % 8)
    const int chunk = (lane & 7) ^ (lane >> 3);
    const unsigned xo = (unsigned)((lane >> 3) * a.x_p) + 16 * chunk;
    const unsigned wo = (unsigned)((lane >> 3) * a.w_p) + 16 * chunk;
    auto issue = [&](int k, uint8_t* to) {
        typedef __attribute__((address_space(3))) void* lp;
        const bool in_k = k + 16 * chunk < a.K;   // w's bytes past K meet zeros of x
#pragma unroll
        for (int i = 0; i < XP; ++i) {
            const int p = wave * XP + i;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                xr, (lp)(to + p * 1024), 16, in_k ? xo + (unsigned)(8 * p * a.x_p) + k : kOut, 0,
                0, 0);
        }
#pragma unroll
        for (int i = 0; i < WP; ++i) {
            const int p = wave * WP + i;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                wr, (lp)(to + XT + p * 1024), 16, wo + (unsigned)(8 * p * a.w_p) + k, 0, 0, 0);
        }
    };
    i32x16 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
    if (a.K > 0) issue(0, lds);
    int buf = 0;
    for (int k = 0; k < a.K; k += kLinKT) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        uint8_t* xl = lds + buf * (XT + WT);
        const uint8_t* wl = xl + XT;
        if (k + kLinKT < a.K) {
            issue(k + kLinKT, lds + (buf ^ 1) * (XT + WT));
        } else if (a.K != a.K16) {
            // x's bytes past K in its last chunk become zeros
            for (int r = threadIdx.x; r < BM; r += NW * 64) {
                i32x4* c = reinterpret_cast<i32x4*>(
                    xl + r * kLinKT + ((((a.K - k) >> 4) ^ (r & 7)) << 4));
                *c = lin_clear(*c, (a.K - k) & 15);
            }
            __syncthreads();
        }
#pragma unroll
        for (int s = 0; s < kLinKT / 32; ++s) {
            i32x4 xf[MB], wf[NB];
            const int c = 2 * s + half;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int r = (wn * NB + j) * 32 + (lane & 31);
                wf[j] = *reinterpret_cast<const i32x4*>(wl + r * kLinKT + ((c ^ (r & 7)) << 4));
            }
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                const int r = (wm * MB + i) * 32 + (lane & 31);
                xf[i] = *reinterpret_cast<const i32x4*>(xl + r * kLinKT + ((c ^ (r & 7)) << 4));
            }
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[j], xf[i], acc[i][j], 0,
                                                                      0, 0);
        }
        buf ^= 1;
    }
    // register 4 g + r of half h is column 8 g + 4 h + r of the block
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int m = m0 + (wm * MB + i) * 32 + (lane & 31);
        if (m < a.M) {
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int n = n0 + (wn * NB + j) * 32 + 8 * g + 4 * half;
                    const int v[4] = {acc[i][j][4 * g], acc[i][j][4 * g + 1],
                                      acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
                    if (n < a.N) lin_store4<DT>(a, m, n, v);
                }
        }
    }
}

}  // namespace igc
