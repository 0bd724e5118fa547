// Cross attention to at most 128 keys (a text prompt's states): forward, and
// the pass of the backward that owns rows.
//
// All keys and values of a head fit LDS, and all scores of 32 rows a wave's
// registers.  A workgroup stages the keys once, and its waves then walk
// blocks of 32 rows on their own, without barriers, the next block's rows in
// flight.  The softmax needs no running maximum, and blocks of 32 keys
// without a valid one are left out.  What is left is bound by the rows' bytes
// (q and out; q, do and dq): 8 x 4096 rows, 77 keys, 4 heads of 64 take 10 us
// (3.3 TB/s), the small map's 64 rows 5.0 us, which is the launch and two
// memory round trips.  Against the kernels that walk tiles of keys: 32 x 784
// rows, 77 keys, 8 heads of 64 16 us forward and 46 backward, by tiles 18.5
// and 69; 2 x 4096 rows, 128 keys, 16 heads of 128 19 and 69, by tiles 23 and
// 87.
#pragma once

#include "attn_bwd.hpp"

namespace igc {

// LDS: two tiles of 64 keys, two of values, and for each key 0 or, where it
// is not valid, -inf, with which the score products start.
template <int DP>
constexpr int short_lds() { return 2 * kShortKeys * DP * 2 + kShortKeys * 4; }

// Keys and values of one head in LDS, and the words of valid keys of the four
// blocks of 32.
template <int DP, int NW>
__device__ __forceinline__ void stage_short(const AttnArgs& a, int b, int hk, int wave, int lane,
                                            uint8_t* lds, uint32_t (&word)[4]) {
    constexpr int TILE = 64 * DP * 2;
    const int len = a.lens ? max(0, min(a.lens[b], a.Tk)) : a.Tk;
    const uint8_t* kbase = a.k + (int64_t)b * a.k_b + (int64_t)hk * a.k_h;
    const uint8_t* vbase = a.v + (int64_t)b * a.v_b + (int64_t)hk * a.v_h;
    const uint8_t* mrow = a.mask ? a.mask + (int64_t)b * a.mask_b : nullptr;
    TileStage<DP, 64, NW> ks, vs;
    ks.init(wave, lane, a.D, (unsigned)a.k_t);
    vs.init(wave, lane, a.D, (unsigned)a.v_t);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const uint64_t w = mask_word(mask_byte(mrow, 64 * t, len, lane), len - 64 * t);
        word[2 * t] = (uint32_t)w;
        word[2 * t + 1] = (uint32_t)(w >> 32);
        if (w == 0) continue;
        ks.issue(kbase + (int64_t)(64 * t) * a.k_t, w, lds + t * TILE, wave);
        vs.issue(vbase + (int64_t)(64 * t) * a.v_t, w, lds + (2 + t) * TILE, wave);
    }
    if (wave == 0) {
        float* bias = reinterpret_cast<float*>(lds + 4 * TILE);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t w = lane < 32 ? word[2 * t] : word[2 * t + 1];
            bias[64 * t + lane] = (w >> (lane & 31)) & 1 ? 0.0f : -__builtin_inff();
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

// Products of the 32 keys of block kb in a staged tile with 32 rows, added to
// s.
template <int DT, int DP>
__device__ __forceinline__ f32x16 short_scores(const uint8_t* tile, int kb, int lane,
                                               const i32x4 (&f)[DP / 16], f32x16 s) {
#pragma unroll
    for (int x = 0; x < DP / 16; ++x) {
        const i32x4 kf =
            frag_row<DP>(tile, 32 * kb + (lane & 31), 2 * x + (lane >> 5));
        s = mfma32<DT>(&kf, &f[x], s);
    }
    return s;
}

// -inf for the block's keys that are not valid, 0 for the others, in result
// order.
__device__ __forceinline__ f32x16 short_bias(const uint8_t* bias, int kb, int half) {
    f32x16 s;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const f32x4 x =
            *reinterpret_cast<const f32x4*>(bias + (32 * kb + 8 * g + 4 * half) * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[4 * g + i] = x[i];
    }
    return s;
}

template <int DT, int DP, int NW>
__global__ __launch_bounds__(NW * 64, DP > 64 ? 2 : 3) void attn_short_fwd_kernel(AttnArgs a) {
    constexpr int DB = DP / 32, KS = DP / 16, TILE = 64 * DP * 2;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    lds_poison<NW * 64>(lds, short_lds<DP>());
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int half = lane >> 5;
    int idx = launch_place(a);
    const int first = idx % a.row_tiles * NW + wave;
    idx /= a.row_tiles;
    const int hk = idx % a.Hk, b = idx / a.Hk;
    const int step = a.row_tiles * NW;   // blocks of 32 rows between a wave's
    const int blocks = (a.rows + 31) >> 5;

    const uint8_t* qbase = a.q + (int64_t)b * a.q_b + (int64_t)hk * a.G * a.q_h;
    auto load = [&](int row0, i32x4(&f)[KS]) {
        const int t0 = div_g(a, row0);
        load_rows<DP>(attn_rsrc(qbase + (int64_t)t0 * a.q_t),
                      packed_off(a, row0 + (lane & 31), t0, a.q_t, a.q_h), a.D, half, f);
    };
    i32x4 qf[KS], qn[KS];
    load(first * 32, qf);
    uint32_t word[4];
    stage_short<DP, NW>(a, b, hk, wave, lane, lds, word);

    for (int blk = first; blk < blocks; blk += step) {
        if (blk + step < blocks) load((blk + step) * 32, qn);
        f32x16 s[4], acc[DB];
        float m = -__builtin_inff();
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
            if (word[kb]) {
                s[kb] = short_scores<DT, DP>(lds + (kb >> 1) * TILE, kb & 1, lane, qf,
                                             short_bias(lds + 4 * TILE, kb, half));
#pragma unroll
                for (int i = 0; i < 16; i += 2) m = fmaxf(fmaxf(s[kb][i], s[kb][i + 1]), m);
            }
        m = max_halves(m) * a.c;
        const float ms = (m == -__builtin_inff() ? 0.0f : m) - p_shift<DT>();
        float sum[4] = {0, 0, 0, 0};
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
            if (word[kb]) {
                float p[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][i], a.c, -ms));
                    sum[i & 3] += p[i];
                }
                i32x4 pf[2];
                pack_frag<DT>(p, pf);
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        const i32x4 vf =
                            frag_col<DP>(lds + (4 + kb) * (TILE / 2), 16 * g, d, lane);
                        acc[d] = mfma32<DT>(&vf, &pf[g], acc[d]);
                    }
            }
        fwd_finish<DT, DB>(a, b, hk, 0, blk * 32, lane, acc, m,
                           (sum[0] + sum[1]) + (sum[2] + sum[3]));
#pragma unroll
        for (int x = 0; x < KS; ++x) qf[x] = qn[x];
    }
}

// Rows of the backward: dq, Delta and lse in powers of two.  Delta is the sum
// of p dp over the keys themselves: with few keys out is as large as the
// values, and Delta from the rounded out would cost dq and dk as much again
// as all other roundings together (fp16, 25 keys: error 1.57 times the
// rounding of the result alone, here 1.4).  In fp16 the scale of ds comes
// from each row's own largest |dp - Delta|; the largest of the wave's rows
// goes to `bound` for the dk dv pass.  Bound by q, do and dq in HBM and the
// waves that registers leave (32 x 784 rows, 77 keys, 8 heads of 64: 22 us).
template <int DT, int DP, int NW>
__global__ __launch_bounds__(NW * 64, DP > 64 ? 1 : 2) void attn_short_rows_kernel(AttnArgs a) {
    constexpr int DB = DP / 32, KS = DP / 16, TILE = 64 * DP * 2;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    lds_poison<NW * 64>(lds, short_lds<DP>());
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int half = lane >> 5;
    int idx = launch_place(a);
    const int first = idx % a.row_tiles * NW + wave;
    const int bh = idx / a.row_tiles;
    const int hk = bh % a.Hk, b = bh / a.Hk;
    const int step = a.row_tiles * NW;
    const int blocks = a.rows_pad >> 5;   // padding rows get their statistics too

    const uint8_t* qbase = a.q + (int64_t)b * a.q_b + (int64_t)hk * a.G * a.q_h;
    const uint8_t* gbase = a.dout + (int64_t)b * a.do_b + (int64_t)hk * a.G * a.do_h;
    const __amdgpu_buffer_rsrc_t lrs = lse_base(a, b, hk);
    i32x4 qf[KS], gf[KS], qn[KS], gn[KS];
    float ln = 0.0f;   // lse, as loaded: of the next block while one is worked on
    auto load = [&](int row0, i32x4(&fq)[KS], i32x4(&fg)[KS]) {
        const int t0 = div_g(a, row0), row = row0 + (lane & 31);
        load_rows<DP>(attn_rsrc(qbase + (int64_t)t0 * a.q_t),
                      packed_off(a, row, t0, a.q_t, a.q_h), a.D, half, fq);
        load_rows<DP>(attn_rsrc(gbase + (int64_t)t0 * a.do_t),
                      packed_off(a, row, t0, a.do_t, a.do_h), a.D, half, fg);
        ln = load4(lrs, lse_off(a, row));
    };
    load(first * 32, qf, gf);
    uint32_t word[4];
    stage_short<DP, NW>(a, b, hk, wave, lane, lds, word);
    float* lse2 = a.stat + (int64_t)bh * a.rows_pad;
    float* delta = a.stat + ((int64_t)a.B * a.Hk + bh) * a.rows_pad;
    float top = 0.0f;

    for (int blk = first; blk < blocks; blk += step) {
        const int row = blk * 32 + (lane & 31);
        // -inf: no valid key (or a padding row); +inf makes every p 0
        const float L =
            ln == -__builtin_inff() || row >= a.rows ? __builtin_inff() : ln * kLog2e;
        if (blk + step < blocks) load((blk + step) * 32, qn, gn);
        f32x16 s[4], dp[4];
        float De = 0.0f;
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
            if (word[kb]) {
                f32x16 zero;
#pragma unroll
                for (int i = 0; i < 16; ++i) zero[i] = 0.0f;
                s[kb] = short_scores<DT, DP>(lds + (kb >> 1) * TILE, kb & 1, lane, qf,
                                             short_bias(lds + 4 * TILE, kb, half));
                dp[kb] = short_scores<DT, DP>(lds + (2 + (kb >> 1)) * TILE, kb & 1, lane, gf, zero);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[kb][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][i], a.c, -L));
                float t[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    t[i & 1] = __builtin_fmaf(s[kb][i], dp[kb][i], t[i & 1]);
                De += t[0] + t[1];
            }
        De = sum_halves(De);
        float f = 1.0f;
        if constexpr (DT == DT_FP16) {
            float x = 0.0f;
#pragma unroll
            for (int kb = 0; kb < 4; ++kb)
                if (word[kb])
#pragma unroll
                    for (int i = 0; i < 16; ++i) x = fmaxf(x, fabsf(dp[kb][i] - De));
            x = max_halves(x);
            f = range_scale(x);
            if (L != __builtin_inff()) top = fmaxf(top, x);
        }
        const unsigned soff = half == 0 ? (unsigned)lane * 4 : kOut;
        store4(attn_rsrc(lse2 + blk * 32), soff, L);
        store4(attn_rsrc(delta + blk * 32), soff, L != __builtin_inff() ? -De : 0.0f);
        if (a.dq) {
            f32x16 dq[DB];
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) dq[d][i] = 0.0f;
#pragma unroll
            for (int kb = 0; kb < 4; ++kb)
                if (word[kb]) {
                    float ds[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) ds[i] = s[kb][i] * ((dp[kb][i] - De) * f);
                    i32x4 df[2];
                    pack_frag<DT>(ds, df);
#pragma unroll
                    for (int g = 0; g < 2; ++g)
#pragma unroll
                        for (int d = 0; d < DB; ++d) {
                            const i32x4 kt = frag_col<DP>(lds + kb * (TILE / 2), 16 * g, d, lane);
                            dq[d] = mfma32<DT>(&kt, &df[g], dq[d]);
                        }
                }
            const int t0 = div_g(a, blk * 32);
            const __amdgpu_buffer_rsrc_t rs =
                attn_rsrc(a.dq + (int64_t)b * a.dq_b + (int64_t)hk * a.G * a.dq_h +
                          (int64_t)t0 * a.dq_t);
            const unsigned off = packed_off(a, row, t0, a.dq_t, a.dq_h);
#pragma unroll
            for (int d = 0; d < DB; ++d)
                store_block<DT>(rs, off, dq[d], a.scale / f, 32 * d, a.D, half);
        }
#pragma unroll
        for (int x = 0; x < KS; ++x) {
            qf[x] = qn[x];
            gf[x] = gn[x];
        }
    }
    if constexpr (DT == DT_FP16) {
        // ds_scale's form of a bound: 2 sqrt(x) sqrt(y)
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
        store4(attn_rsrc(a.bound + ((int64_t)bh * a.bound_n + first) * 2),
               lane < 2 ? (unsigned)lane * 4 : kOut, lane ? 0.25f : top * top);
    }
}

}  // namespace igc
