// Product of two matrices of 8-bit integers with a scale a row of each:
//   y[m][n] = (sum_k x[m][k] w[n][k]) xs[m] ws[n] + bias[n]
//
// Both operands have k adjacent, as the matrix instructions take them (16 k a
// lane).  w is the A operand and x the B operand, so that a lane of the result
// owns one row of y and neighbouring columns.  The integer sums are exact; they
// are scaled in fp32 and rounded once.
//
// The tile kernel stages its rows and columns in LDS by direct loads: 16384 x
// 4096 x 4096 in 259 to 265 us for a few calls (2.1 PFLOP/s) and in 284 to 350 once
// the clock has been held down, 8192 x 8192 x 8192 in 483 (2.28).  The power limit
// bounds it: the matrix cores are busy 59 % at about 2.0 GHz, and on such data they
// hold 1.65 GHz when they do nothing else.  The few-rows kernel, which the weights'
// bytes bound, takes 16
// columns a workgroup, gives each wave a part of k and reads both operands
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

// Scales and bias of columns n .. n + 3 of row m (past N the last column's, past
// M the last row's; such results are not stored).
struct LinScales {
    float xs;
    f32x4 ws, bs;
    __device__ __forceinline__ void load(const LinArgs& a, int m, int n) {
        xs = a.xs[min(m, a.M - 1)];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = min(n + i, a.N - 1);
            ws[i] = a.ws[c];
            bs[i] = a.bias ? a.bias[c] : 0.0f;
        }
    }
};
template <int DT>
__device__ __forceinline__ void lin_store4(const LinArgs& a, int m, int n, const i32x4& acc,
                                           const LinScales& sc) {
    typedef uint32_t u32x2h __attribute__((ext_vector_type(2), aligned(2)));
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf((float)acc[i] * sc.xs, sc.ws[i], sc.bs[i]);
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
// At most 16 MT rows.  The waves take a line of 128 k of each row in turn, U = 2
// at once: the weights of 8192 x 2048 arrive in 5.6 us, of 28672 x 4096 in 27.3
// with the launch (4.3 TB/s; eight waves, or four lines at once, within 4 %).
constexpr int kFewWaves = 4;
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
    constexpr int U = 2, STEP = kFewWaves * 128 * U;
    auto at = [&](int k) { return k + 16 * (lane >> 4); };   // first k of the lane's chunk
    // what the results need is asked for before the sums begin: result lane l
    // has row l % 16 of x, columns 4 (l / 16) .. + 3
    static_assert(MT <= kFewWaves, "a thread a result");
    const int rt = threadIdx.x >> 6, m = 16 * rt + (lane & 15), n = n0 + 4 * (lane >> 4);
    LinScales sc;
    if (rt < MT) sc.load(a, m, n);
    for (int k0 = wave * 128; k0 < a.K; k0 += STEP) {
        i32x4 w[U][2], x[U][2][MT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = k0 + u * kFewWaves * 128 + 64 * s;
                const bool in = at(k) < a.K;
                w[u][s] = __builtin_bit_cast(i32x4, load16(wr, in ? woff + k : kOut));
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    x[u][s][t] = __builtin_bit_cast(i32x4,
                                                    load16(xr, in ? xoff + t * xrow + k : kOut));
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int c = at(k0 + u * kFewWaves * 128 + 64 * s);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    if (c + 16 > a.K) x[u][s][t] = lin_clear(x[u][s][t], a.K - c);
                    acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][s], x[u][s][t], acc[t], 0,
                                                                   0, 0);
                }
            }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) *reinterpret_cast<i32x4*>(part[wave][t][lane]) = acc[t];
    __syncthreads();
    if (rt >= MT) return;
    i32x4 s = *reinterpret_cast<const i32x4*>(part[0][rt][lane]);
#pragma unroll
    for (int v = 1; v < kFewWaves; ++v) s += *reinterpret_cast<const i32x4*>(part[v][rt][lane]);
    if (m < a.M && n < a.N) lin_store4<DT>(a, m, n, s, sc);
}

// ---------------------------------------------------------------------------
// Square tiles of B rows of x and B of w, four waves of a quarter each.  A
// stage is KT k of all rows; NS of them are under way or being read.  A step is
// 32 k: the fragments of the next one are read while its products run, and a
// stage's last step reads the next stage's first, so that the matrix cores see
// no seam.  One barrier a stage: behind it the next stage is whole, and the one
// just read may be overwritten.  A barrier costs as much as several products of
// a small tile, which therefore takes long stages (64 rows x 4096 x 4096 in
// tiles of 64: 12.2 us in stages of 64 k, 10.6 of 128, 8.7 of 256; in tiles of
// 128, 1024 rows: 23.6 of 64 and 22.5 of 128).  Where tiles of 64 are more
// than the CUs, two stages let two workgroups share one (512 rows: 15.5 us,
// three stages 17.4; 64 rows 10.3 and 8.7).
template <int B, int NS>
struct LinTile {
    static constexpr int KT = B == 256 ? 64 : B == 128 ? 128 : 256;
    static constexpr int T = B * KT;   // bytes of one operand's stage
    static constexpr int LDS = NS * 2 * T;
};

template <int DT, int B, int NS>
__global__ __launch_bounds__(256, B == 256 ? 1 : 2) void linear_i8_tile_kernel(LinArgs a) {
    constexpr int NW = 4, MB = B / 64;   // blocks of 32 a wave, each way
    constexpr int KT = LinTile<B, NS>::KT, T = LinTile<B, NS>::T;
    constexpr int STEPS = KT / 32, CH = KT / 16;   // 16-byte chunks of a row
    constexpr int P = T / 1024 / NW, PR = 1024 / KT;   // loads a wave of one operand; their rows
    static_assert(2 * P == STEPS * MB && STEPS % 2 == 0, "MB loads a step");
    static_assert(P * PR % 16 == 0, "a wave's rows start at a multiple of 16");
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];   // NS x {x, w}
    lds_poison<NW * 64>(lds, LinTile<B, NS>::LDS);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wm = wave >> 1, wn = wave & 1, half = lane >> 5;

    // an XCD's run of tiles goes through bands of 8 tiles of x, column by
    // column: the workgroups that run at once share both operands in its L2
    const int tile = xcd_remap(blockIdx.x, gridDim.x);
    const int band = tile / (8 * a.tiles_n), rows = min(8, a.tiles_m - 8 * band);
    const int in = tile - band * 8 * a.tiles_n;
    const int m0 = (8 * band + in % rows) * B, n0 = in / rows * B;
    const __amdgpu_buffer_rsrc_t xr = lin_rsrc(
        a.x + m0 * a.x_p, lin_bytes(min(B, a.M - m0), a.x_p, a.K16));
    const __amdgpu_buffer_rsrc_t wr = lin_rsrc(
        a.w + n0 * a.w_p, lin_bytes(min(B, a.N - n0), a.w_p, a.K16));

    // Chunk c of row r lies at c ^ turn(r), which spreads a chunk of 16 rows over
    // all banks.
    auto turn = [](int r) { return r / (256 / KT) & (CH - 1); };
    const int lrow = lane / CH;   // the lane's row in a load
    const unsigned xo = (unsigned)((wave * P * PR + lrow) * a.x_p);
    const unsigned wo = (unsigned)((wave * P * PR + lrow) * a.w_p);
    const unsigned xr1 = (unsigned)(PR * a.x_p), wr1 = (unsigned)(PR * a.w_p);
    typedef __attribute__((address_space(3))) void* lp;
    // load l of the 2 P of the stage at k
    auto issue = [&](int k, uint8_t* to, int l) {
        const int i = l < P ? l : l - P;
        const int at = k + 16 * ((lane % CH) ^ turn(i * PR + lrow));
        if (l < P)   // zeros past K
            __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (lp)(to + (wave * P + i) * 1024), 16,
                                                     at < a.K ? xo + i * xr1 + at : kOut, 0, 0, 0);
        else         // past K anything: it meets zeros
            __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, (lp)(to + T + (wave * P + i) * 1024), 16,
                                                     wo + i * wr1 + at, 0, 0, 0);
    };
    // This wave's part of the stage at k is here: all of it, for all waves, is.
    // (A bare barrier: __syncthreads would wait for the later stages too.)
    auto barrier = [&] {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    auto arrived = [&](int k, uint8_t* at) {
        barrier();
        if (a.K - k < KT && a.K > k && a.K != a.K16) {
            // x's bytes past K in its last chunk become zeros
            for (int r = threadIdx.x; r < B; r += NW * 64) {
                i32x4* c = reinterpret_cast<i32x4*>(
                    at + r * KT + ((((a.K - k) >> 4) ^ turn(r)) << 4));
                *c = lin_clear(*c, (a.K - k) & 15);
            }
            barrier();
        }
    };
    // What the results need: a thread's column, a lane's rows.  The large tile
    // has no registers for it before its sums are done.
    float my_ws, my_bs, xs[MB];
    auto scales = [&] {
        const int c = min(n0 + (int)threadIdx.x % B, a.N - 1);
        my_ws = a.ws[c];
        my_bs = a.bias ? a.bias[c] : 0.0f;
#pragma unroll
        for (int i = 0; i < MB; ++i)
            xs[i] = a.xs[min(m0 + (wm * MB + i) * 32 + (lane & 31), a.M - 1)];
    };
    if constexpr (B < 256) scales();
    i32x4 xf[2][MB], wf[2][MB];
    // rows of a block start at multiples of 32
    const uint8_t* xl = lds + (wm * MB * 32 + (lane & 31)) * KT;
    const uint8_t* wl = lds + T + (wn * MB * 32 + (lane & 31)) * KT;
    auto read = [&](int buf, int s, int set, int i) {   // buf: the stage's place
        const int c = buf * 2 * T + (((2 * s + half) ^ turn(lane & 31)) << 4);
        wf[set][i] = *reinterpret_cast<const i32x4*>(wl + c + i * 32 * KT);
        xf[set][i] = *reinterpret_cast<const i32x4*>(xl + c + i * 32 * KT);
    };
    i32x16 acc[MB][MB];
    // Products of one step, and between them the reads of the next one and a
    // few loads: in a burst the loads would hold up the products behind them.
    auto step = [&](int set, int next_buf, int next_s, int k, uint8_t* to, int first) {
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            read(next_buf, next_s, set ^ 1, i);
            issue(k, to, first + i);
#pragma unroll
            for (int j = 0; j < MB; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[set][j], xf[set][i],
                                                                  acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    int buf = 0, old = NS - 1;   // the stage being read, and the one before it
    if (a.K > 0) {   // stages past K are loaded too (zeros), and not read
#pragma unroll
        for (int n = 0; n < NS - 1; ++n)
#pragma unroll
            for (int l = 0; l < 2 * P; ++l) issue(n * KT, lds + n * 2 * T, l);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 2) * 2 * P) : "memory");
        arrived(0, lds);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            issue((NS - 1) * KT, lds + (NS - 1) * 2 * T, i);
            read(0, 0, 0, i);
        }
    }
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
    for (int k = 0; k < a.K; k += KT) {
        uint8_t* to = lds + old * 2 * T;
#pragma unroll
        for (int s = 0; s < STEPS - 1; ++s)
            step(s & 1, buf, s + 1, k + (NS - 1) * KT, to, (s + 1) * MB);
        // the last step's fragments and the next stage
        asm volatile("s_waitcnt lgkmcnt(0) vmcnt(%0)" ::"n"((NS - 2) * 2 * P) : "memory");
        old = buf;
        buf = buf + 1 < NS ? buf + 1 : 0;
        arrived(k + KT, lds + buf * 2 * T);
        step(1, buf, 0, k + NS * KT, lds + old * 2 * T, 0);
    }
    // nothing may be under way to LDS when the workgroup ends
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    // Scales and bias of the columns go through LDS, and the results too, 32
    // rows of a wave at a time, so that whole lines are stored.
    barrier();
    float* col = reinterpret_cast<float*>(lds);   // [2][B]
    static_assert(B <= NW * 64, "a column a thread");
    if constexpr (B == 256) scales();
    if ((int)threadIdx.x < B) {
        col[threadIdx.x] = my_ws;
        col[B + threadIdx.x] = my_bs;
    }
    __syncthreads();
    constexpr int OC = MB * 4, RL = 64 / OC;   // 16-byte chunks of a row; rows a store
    uint8_t* out = lds + 2 * B * 4 + wave * (32 * OC * 16);
    const bool inner = m0 + B <= a.M && n0 + B <= a.N;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int mb = m0 + (wm * MB + i) * 32, nb = n0 + wn * MB * 32;
        const int r = lane & 31;
        // register 4 g + e of half h is column 8 g + 4 h + e of a block; the
        // halves exchange groups, so that each lane holds 8 neighbouring
        // columns: half h the groups h and 2 + h
#pragma unroll
        for (int j = 0; j < MB; ++j)
#pragma unroll
            for (int gg = 0; gg < 2; ++gg) {
                const float* c = col + (wn * MB + j) * 32 + 16 * gg + 4 * half;
                uint32_t v[4];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const f32x4 ws = *reinterpret_cast<const f32x4*>(c + 8 * g);
                    const f32x4 bs = *reinterpret_cast<const f32x4*>(c + B + 8 * g);
                    float f[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        f[e] = __builtin_fmaf((float)acc[i][j][8 * gg + 4 * g + e] * xs[i], ws[e],
                                              bs[e]);
                    v[2 * g] = pack_out2(f[0], f[1], DT);
                    v[2 * g + 1] = pack_out2(f[2], f[3], DT);
                }
                const auto p = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
                const auto q = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
                const int ch = 4 * j + 2 * gg + half;
                *reinterpret_cast<u32x4*>(out + (r * OC + (ch ^ (r & (OC - 1)))) * 16) =
                    u32x4{p[0], q[0], p[1], q[1]};
                __builtin_amdgcn_sched_barrier(0);   // a block's sums at a time: no spills
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the wave's own rows
#pragma unroll
        for (int t = 0; t < 32 / RL; ++t) {
            const int row = t * RL + lane / OC, ch = lane % OC;
            const u32x4 o = *reinterpret_cast<const u32x4*>(
                out + (row * OC + (ch ^ (row & (OC - 1)))) * 16);
            const int m = mb + row, n = nb + 8 * ch;
            uint8_t* y = a.y + (int64_t)m * a.y_p + 2 * (int64_t)n;
            if (inner) {
                *reinterpret_cast<u32x4h*>(y) = o;
            } else if (m < a.M) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (n + e < a.N)
                        *reinterpret_cast<uint16_t*>(y + 2 * e) =
                            (uint16_t)(o[e / 2] >> (16 * (e & 1)));
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

}  // namespace igc
