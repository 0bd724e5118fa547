// Cross attention, backward.
//
// With p = exp(s - lse), Delta = do . o and dp = do . v of a (row, key) pair:
//   ds = p (dp - Delta),  dq = scale sum_keys ds k,
//   dk = scale sum_rows ds q,  dv = sum_rows p do
// where a key head's rows are all queries of its group, so shared heads'
// gradients sum in the same products.  Three kernels, without atomics, so
// that results do not change from run to run:
//   rows   one pass over o and do: Delta, and lse in powers of two
//   dk dv  workgroups own keys and walk the rows
//   dq     workgroups own rows and walk the keys
// Scores are formed again in both (7 products in all instead of 5), which
// costs less than writing ds or adding dq through memory.
#pragma once

#include "attn_fwd.hpp"
#include "attn_host.hpp"

namespace igc {

// Rows of the statistics are padded to whole row tiles (kRowTile); padding
// rows, and rows without a valid key, hold lse = +inf, which makes every p 0.

// fp16 has 5 exponent bits, while p ~ 1 / keys and ds scales with the
// incoming gradient: both are multiplied by a power of two before they are
// rounded and the sums divided by it.  p <= 1 takes 2^14.  |ds| is at most
// |do| (|v| + |o|) <= 2 max|do| max|v| (o is a mean of v rows), so with the
// head's maxima the largest power that keeps it under 2^15 is known before
// the first product.  bf16 has fp32's exponent range and takes 1.
__device__ __forceinline__ float range_scale(float s) {
    if (!(s > 0.0f) || !(s < 3e38f)) return 1.0f;
    int e;
    frexpf(s, &e);   // s < 2^e
    return ldexpf(1.0f, min(max(14 - e, -100), 100));
}

template <int DT>
__device__ __forceinline__ float ds_scale(const AttnArgs& a, int64_t bh, int lane) {
    if constexpr (DT != DT_FP16) return 1.0f;
    const float* p = reinterpret_cast<const float*>(a.bound) + bh * a.bound_n * 2;
    float g = 0.0f, v = 0.0f;
    for (int i = 0; i < a.bound_n; i += 64) {
        const int x = min(i + lane, a.bound_n - 1);
        g = fmaxf(g, p[2 * x]);
        v = fmaxf(v, p[2 * x + 1]);
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        g = fmaxf(g, __shfl_xor(g, o, 64));
        v = fmaxf(v, __shfl_xor(v, o, 64));
    }
    return range_scale(2.0f * sqrtf(g) * sqrtf(v));
}

// -Delta and lse of the packed rows [bh][rows_pad], and for fp16 the squared
// maxima of do and v of this workgroup's share of a head.  16 lanes a row;
// bound by the bytes of o and do (2 x 4096 rows, 16 heads of 128: 14 us).
// Delta takes the rounded out: over more than 128 keys out is small against
// the values, and so is what its rounding adds to ds (few keys: Delta from the
// probabilities, attn_short.hpp).
template <int DT>
__global__ __launch_bounds__(256) void attn_bwd_rows_kernel(AttnArgs a) {
    const int bh = blockIdx.x / a.bound_n, ch = blockIdx.x - bh * a.bound_n;
    const int b = bh / a.Hk, hk = bh - b * a.Hk;
    const int sub = threadIdx.x >> 4, c = threadIdx.x & 15;
    const bool on = c * 8 < a.D;
    const uint8_t* ob = a.o + (int64_t)b * a.o_b + (int64_t)hk * a.G * a.o_h + c * 16;
    const uint8_t* gb = a.dout + (int64_t)b * a.do_b + (int64_t)hk * a.G * a.do_h + c * 16;
    float* lse2 = a.stat + (int64_t)bh * a.rows_pad;
    float* delta = a.stat + ((int64_t)a.B * a.Hk + bh) * a.rows_pad;
    float gmax = 0.0f, vmax = 0.0f;
    for (int64_t r64 = (int64_t)ch * 16 + sub; r64 < a.rows_pad; r64 += (int64_t)a.bound_n * 16) {
        const int r = (int)r64;
        const bool live = r < a.rows;
        float s = 0.0f, n = 0.0f;
        if (live && on) {
            float x[8], g[8];
            const int tok = div_g(a, r), h = r - tok * a.G;
            unpack8<DT>(*reinterpret_cast<const u32x4*>(ob + tok * a.o_t + h * a.o_h), x);
            unpack8<DT>(*reinterpret_cast<const u32x4*>(gb + tok * a.do_t + h * a.do_h), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s = __builtin_fmaf(x[j], g[j], s);
                n = __builtin_fmaf(g[j], g[j], n);
            }
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) s += __shfl_xor(s, o, 64);
        if constexpr (DT == DT_FP16) {
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) n += __shfl_xor(n, o, 64);
            gmax = fmaxf(gmax, n);
        }
        if (c == 0) {
            float l = __builtin_inff();
            if (live) {
                const int tok = div_g(a, r);
                l = a.lse[((int64_t)b * a.Hq + hk * a.G + (r - tok * a.G)) * a.Tq + tok] * kLog2e;
                if (l == -__builtin_inff()) l = __builtin_inff();
            }
            lse2[r] = l;
            delta[r] = live && l != __builtin_inff() ? -s : 0.0f;
        }
    }
    if constexpr (DT == DT_FP16) {
        const int len = a.lens ? max(0, min(a.lens[b], a.Tk)) : a.Tk;
        const uint8_t* vb = a.v + (int64_t)b * a.v_b + (int64_t)hk * a.v_h + c * 16;
        const uint8_t* mrow = a.mask ? a.mask + (int64_t)b * a.mask_b : nullptr;
        for (int64_t j = (int64_t)ch * 16 + sub; j < len; j += (int64_t)a.bound_n * 16) {
            float n = 0.0f;
            if (on && (!mrow || mrow[j])) {
                float x[8];
                unpack8<DT>(*reinterpret_cast<const u32x4*>(vb + j * a.v_t), x);
#pragma unroll
                for (int i = 0; i < 8; ++i) n = __builtin_fmaf(x[i], x[i], n);
            }
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) n += __shfl_xor(n, o, 64);
            vmax = fmaxf(vmax, n);
        }
        __shared__ __attribute__((aligned(16))) float red[2][16];
        lds_poison<256>(reinterpret_cast<uint8_t*>(red), sizeof(red));
        if (c == 0) {
            red[0][sub] = gmax;
            red[1][sub] = vmax;
        }
        __syncthreads();
        if (threadIdx.x < 2) {
            float m = 0.0f;
            for (int i = 0; i < 16; ++i) m = fmaxf(m, red[threadIdx.x][i]);
            a.bound[((int64_t)bh * a.bound_n + ch) * 2 + threadIdx.x] =
                __builtin_bit_cast(uint32_t, m);
        }
    }
}

// Direct loads of packed rows r0 .. r0 + ROWS - 1 (see TileStage).  Where the
// group's heads divide the tile every tile starts a token, and its rows lie at
// the offsets formed once (st.init_packed); other groups' offsets are formed
// for each tile.
template <int DP, int ROWS, int NW>
__device__ __forceinline__ void issue_packed(const TileStage<DP, ROWS, NW>& st, const AttnArgs& a,
                                             bool fixed, const uint8_t* base, int64_t pt,
                                             int64_t ph, int r0, uint8_t* lds, int wave, int lane) {
    const int t0 = div_g(a, r0);
    if (fixed) {
        st.issue_first(base + (int64_t)t0 * pt, a.rows - r0, lds, wave);
        return;
    }
    const __amdgpu_buffer_rsrc_t rs = attn_rsrc(base + (int64_t)t0 * pt);
#pragma unroll
    for (int i = 0; i < TileStage<DP, ROWS, NW>::PER; ++i) {
        TileStage<DP, ROWS, NW> s;
        const unsigned c = s.place(i, wave, lane, a.D);
        const unsigned at = packed_off(a, r0 + s.row[i], t0, pt, ph) + c;
        st.load(rs, i, c == kOut ? kOut : at, lds, wave);
    }
}

// ---------------------------------------------------------------------------
// dk and dv: each wave owns 32 keys and walks the rows in tiles of QT (q and
// do in LDS).  S = Q K^T has rows down the registers and a key a lane, so p
// and ds go into dv^T += do^T p and dk^T += q^T ds as B operands without
// leaving their lane; do^T and q^T come by transposing reads of the same
// tiles.  The keys' own operands (k and v) stay in registers, or in LDS
// (KV_LDS) where the registers of two waves a SIMD do not hold them.  RG = 2:
// two waves a key block take alternate blocks of 32 rows, and their sums are
// added through LDS at the end.  Long walks keep the matrix cores busy for
// half of the time (2 x 4096 rows x 2048 keys ragged, 16 heads on 8 of 128:
// 255 to 280 us); short ones are bound by their rows' round trips (32 x 784
// rows, 77 keys, 8 heads of 64: 21 us, of which the loads alone take 14).
template <int DP, int NWK, int RG, int QT, bool KV_LDS>
struct KvShape {
    static constexpr int NW = NWK * RG;
    static constexpr int TILE = QT * DP * 2;
    static constexpr int STAGE = (2 * TILE + 2 * QT * 4 + 1023) / 1024 * 1024;  // q, do, lse, Delta
    static constexpr int KEYS = KV_LDS ? 2 * NWK * 32 * DP * 2 : 0;             // k, v
    static constexpr int SUM = RG / 2 * NWK * 64 * DP * 2;                      // over all of it
    static constexpr int LDS = KEYS + 2 * STAGE > SUM ? KEYS + 2 * STAGE : SUM;
};

template <int DT, int DP, int NWK, int RG, int QT, bool KV_LDS, int OCC>
__global__ __launch_bounds__(NWK * RG * 64, OCC) void attn_bwd_kv_kernel(AttnArgs a) {
    typedef KvShape<DP, NWK, RG, QT, KV_LDS> Sh;
    constexpr int NW = Sh::NW, TILE = Sh::TILE, STAGE = Sh::STAGE;
    constexpr int DB = DP / 32, KS = DP / 16;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds_all[];
    lds_poison<NW * 64>(lds_all, Sh::LDS);
    uint8_t* lds = lds_all + Sh::KEYS;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int half = lane >> 5;
    const int wk = RG > 1 ? wave % NWK : wave, rg = RG > 1 ? wave / NWK : 0;

    int idx = launch_place(a);
    const int kt = idx % a.key_tiles;
    idx /= a.key_tiles;
    const int sp = idx % a.nsplit;
    const int bh = idx / a.nsplit;
    const int hk = bh % a.Hk, b = bh / a.Hk;
    const int len = a.lens ? max(0, min(a.lens[b], a.Tk)) : a.Tk;
    const int key0 = (kt * NWK + wk) * 32, kr = lane & 31;
    const uint8_t* mrow = a.mask ? a.mask + (int64_t)b * a.mask_b : nullptr;
    const bool valid = mask_byte(mrow, key0, len, kr) != 0 && key0 + kr < len;
    // the whole workgroup's keys may be out of range: nothing to sum then
    const int r_begin = sp * a.split;
    const int r_end = kt * NWK * 32 < len ? split_end(r_begin, a.split, a.rows) : r_begin;
    const bool idle = !__any(valid);   // this wave then only stages

    i32x4 kf[KS], vf[KS];
    f32x16 dk[DB], dv[DB];
    const uint8_t* kp = a.k + (int64_t)b * a.k_b + (int64_t)hk * a.k_h;
    const uint8_t* vp = a.v + (int64_t)b * a.v_b + (int64_t)hk * a.v_h;
    if constexpr (KV_LDS) {
        TileStage<DP, 32, NW> ks, vs;
        ks.init(wave, lane, a.D, (unsigned)a.k_t);
        vs.init(wave, lane, a.D, (unsigned)a.v_t);
#pragma unroll
        for (int w = 0; w < NWK; ++w) {
            const int k0 = (kt * NWK + w) * 32;
            const uint32_t word = (uint32_t)mask_word(mask_byte(mrow, k0, len, lane), len - k0);
            ks.issue(kp + (int64_t)k0 * a.k_t, word, lds_all + w * 64 * DP, wave);
            vs.issue(vp + (int64_t)k0 * a.v_t, word, lds_all + (NWK + w) * 64 * DP, wave);
        }
    } else {
        load_rows<DP>(attn_rsrc(kp + (int64_t)key0 * a.k_t),
                      valid ? (unsigned)kr * (unsigned)a.k_t : kOut, a.D, half, kf);
        load_rows<DP>(attn_rsrc(vp + (int64_t)key0 * a.v_t),
                      valid ? (unsigned)kr * (unsigned)a.v_t : kOut, a.D, half, vf);
    }
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[d][i] = dv[d][i] = 0.0f;
    const float f = ds_scale<DT>(a, bh, lane);
    constexpr float PS = DT == DT_FP16 ? 14.0f : 0.0f;   // p carries 2^PS
    const float fp = DT == DT_FP16 ? f * 0.00006103515625f : f;

    const uint8_t* qbase = a.q + (int64_t)b * a.q_b + (int64_t)hk * a.G * a.q_h;
    const uint8_t* gbase = a.dout + (int64_t)b * a.do_b + (int64_t)hk * a.G * a.do_h;
    const float* lse2 = a.stat + (int64_t)bh * a.rows_pad;
    const float* delta = a.stat + ((int64_t)a.B * a.Hk + bh) * a.rows_pad;
    TileStage<DP, QT, NW> qs, gs;
    const bool fixed = QT % a.G == 0;
    qs.init_packed(a, wave, lane, a.q_t, a.q_h);
    gs.init_packed(a, wave, lane, a.do_t, a.do_h);
    auto issue = [&](int r0, uint8_t* to) {
        issue_packed(qs, a, fixed, qbase, a.q_t, a.q_h, r0, to, wave, lane);
        issue_packed(gs, a, fixed, gbase, a.do_t, a.do_h, r0, to + TILE, wave, lane);
#pragma unroll
        for (int x = 0; x < QT / 32; ++x)   // QT floats each: lse, then Delta
            if (wave == x % NW)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    attn_rsrc((x < QT / 64 ? lse2 : delta - QT) + r0 + x * 64),
                    (__attribute__((address_space(3))) void*)(to + 2 * TILE + x * 256), 4,
                    lane * 4, 0, 0, 0);
    };
    const uint8_t* kl = lds_all + wk * 64 * DP;
    const uint8_t* vl = kl + NWK * 64 * DP;
    if (r_begin < r_end) {
        issue(r_begin, lds);
        int buf = 0;
        for (int r0 = r_begin; r0 < r_end; r0 += QT) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            const uint8_t* ql = lds + buf * STAGE;
            const uint8_t* gl = ql + TILE;
            const float* ls = reinterpret_cast<const float*>(ql + 2 * TILE);
            if (r0 + QT < r_end) issue(r0 + QT, lds + (buf ^ 1) * STAGE);
            if (!idle)
#pragma unroll
            for (int rx = 0; rx < QT / 32 / RG; ++rx) {
                const int rb = rx * RG + rg;
                // columns (keys) do not mix: those of keys that are not valid
                // sum anything and are left out at the end
                f32x16 s, dp;
#pragma unroll
                for (int i = 0; i < 16; ++i) s[i] = 0.0f;
#pragma unroll
                for (int x = 0; x < KS; ++x) {
                    const i32x4 qf = frag_row<DP>(ql, 32 * rb + (lane & 31), 2 * x + half);
                    const i32x4 kx = KV_LDS ? frag_row<DP>(kl, lane & 31, 2 * x + half) : kf[x];
                    s = mfma32<DT>(&qf, &kx, s);
                }
                float p[16], ds[16];
                i32x4 pf[2], df[2];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4 L =
                        *reinterpret_cast<const f32x4*>(ls + 32 * rb + 8 * g + 4 * half);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        p[4 * g + i] = __builtin_amdgcn_exp2f(
                            __builtin_fmaf(s[4 * g + i], a.c, PS - L[i]));
                }
                pack_frag<DT>(p, pf);
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        const i32x4 gt = frag_col<DP>(gl, 32 * rb + 16 * g, d, lane);
                        dv[d] = mfma32<DT>(&gt, &pf[g], dv[d]);
                    }
                // dp starts from -Delta
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x4 De =
                        *reinterpret_cast<const f32x4*>(ls + QT + 32 * rb + 8 * g + 4 * half);
#pragma unroll
                    for (int i = 0; i < 4; ++i) dp[4 * g + i] = De[i];
                }
#pragma unroll
                for (int x = 0; x < KS; ++x) {
                    const i32x4 gf = frag_row<DP>(gl, 32 * rb + (lane & 31), 2 * x + half);
                    const i32x4 vx = KV_LDS ? frag_row<DP>(vl, lane & 31, 2 * x + half) : vf[x];
                    dp = mfma32<DT>(&gf, &vx, dp);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    ds[e] = p[e] * dp[e];
                    if constexpr (DT == DT_FP16) ds[e] *= fp;
                }
                pack_frag<DT>(ds, df);
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        const i32x4 qt = frag_col<DP>(ql, 32 * rb + 16 * g, d, lane);
                        dk[d] = mfma32<DT>(&qt, &df[g], dk[d]);
                    }
            }
            buf ^= 1;
        }
    } else if constexpr (KV_LDS) {
        // without rows nothing above has waited for the keys' direct loads,
        // and the sums below take their place in LDS
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    if constexpr (RG > 1) {
        // the row groups' sums through LDS, dk then dv, lane by lane: the upper
        // half of the groups adds to the lower, until one is left
        constexpr int N = NWK * 64;   // f32x4 between a lane's
#pragma unroll
        for (int n = RG / 2; n; n /= 2)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                f32x16(&acc)[DB] = t ? dv : dk;
                f32x4* x = reinterpret_cast<f32x4*>(lds_all) + (rg % n) * (N * DP / 8) +
                           (wk * 64 + lane);
                __syncthreads();
                if (rg >= n && rg < 2 * n) {
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            x[(4 * d + g) * N] = f32x4{acc[d][4 * g], acc[d][4 * g + 1],
                                                       acc[d][4 * g + 2], acc[d][4 * g + 3]};
                }
                __syncthreads();
                if (rg < n) {
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const f32x4 y = x[(4 * d + g) * N];
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[d][4 * g + i] += y[i];
                        }
                }
            }
        if (rg >= 1) return;
    }
    const float fk = a.scale / f, fv = DT == DT_FP16 ? 0.00006103515625f : 1.0f;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            dk[d][i] = valid ? dk[d][i] : 0.0f;
            dv[d][i] = valid ? dv[d][i] : 0.0f;
        }
    const bool live = key0 + kr < a.Tk;
    if (a.nsplit > 1) {
        const int64_t n = (int64_t)a.B * a.Hk * a.Tk * a.D;
        float* o = a.part + sp * n + ((int64_t)bh * a.Tk + key0) * a.D;
        const __amdgpu_buffer_rsrc_t k1 = attn_rsrc(o), v1 = attn_rsrc(o + a.nsplit * n);
        const unsigned off = live ? (unsigned)(kr * a.D) * 4 : kOut;
#pragma unroll
        for (int d = 0; d < DB; ++d) {
            store_part(k1, off, dk[d], fk, 32 * d, a.D, half);
            store_part(v1, off, dv[d], fv, 32 * d, a.D, half);
        }
        return;
    }
    const __amdgpu_buffer_rsrc_t ko = attn_rsrc(a.dk + (int64_t)b * a.dk_b +
                                                (int64_t)hk * a.dk_h + (int64_t)key0 * a.dk_t);
    const __amdgpu_buffer_rsrc_t vo = attn_rsrc(a.dv + (int64_t)b * a.dv_b +
                                                (int64_t)hk * a.dv_h + (int64_t)key0 * a.dv_t);
    const unsigned koff = live ? (unsigned)kr * (unsigned)a.dk_t : kOut;
    const unsigned voff = live ? (unsigned)kr * (unsigned)a.dv_t : kOut;
#pragma unroll
    for (int d = 0; d < DB; ++d) {
        store_block<DT>(ko, koff, dk[d], fk, 32 * d, a.D, half);
        store_block<DT>(vo, voff, dv[d], fv, 32 * d, a.D, half);
    }
}

// ---------------------------------------------------------------------------
// dq: the forward kernel's walk (32 rows a wave, keys in tiles of 64) with
// both score products, S^T = K Q^T and dP^T = V dO^T, and dq^T += K^T ds^T.
// Bound as that kernel (2 x 4096 rows x 2048 keys ragged, 16 heads on 8 of
// 128: 158 to 175 us, matrix cores busy for half of it).
template <int DT, int DP, int NW>
__global__ __launch_bounds__(NW * 64, 2) void attn_bwd_q_kernel(AttnArgs a) {
    constexpr int KT = 64, DB = DP / 32, KS = DP / 16;
    constexpr int TILE = KT * DP * 2;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    lds_poison<NW * 64>(lds, 4 * TILE);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int half = lane >> 5;

    int idx = launch_place(a);
    const int rt = idx % a.row_tiles;
    idx /= a.row_tiles;
    const int sp = idx % a.nsplit;
    const int bh = idx / a.nsplit;
    const int hk = bh % a.Hk, b = bh / a.Hk;
    const int len = a.lens ? max(0, min(a.lens[b], a.Tk)) : a.Tk;
    const int j_begin = sp * a.split, j_end = split_end(j_begin, a.split, len);

    const int row0 = (rt * NW + wave) * 32, row = row0 + (lane & 31), t0 = div_g(a, row0);
    i32x4 qf[KS], gf[KS];
    load_rows<DP>(attn_rsrc(a.q + (int64_t)b * a.q_b + (int64_t)hk * a.G * a.q_h +
                            (int64_t)t0 * a.q_t),
                  packed_off(a, row, t0, a.q_t, a.q_h), a.D, half, qf);
    load_rows<DP>(attn_rsrc(a.dout + (int64_t)b * a.do_b + (int64_t)hk * a.G * a.do_h +
                            (int64_t)t0 * a.do_t),
                  packed_off(a, row, t0, a.do_t, a.do_h), a.D, half, gf);
    const bool live = row < a.rows;
    // padding rows have statistics, rows past the padding read as 0: their
    // results are not stored
    const unsigned soff = row < a.rows_pad ? (unsigned)(lane & 31) * 4 : kOut;
    const float L = load4(attn_rsrc(a.stat + (int64_t)bh * a.rows_pad + row0), soff);
    const float De =
        load4(attn_rsrc(a.stat + ((int64_t)a.B * a.Hk + bh) * a.rows_pad + row0), soff);
    const float f = ds_scale<DT>(a, bh, lane);
    f32x16 dq[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[d][i] = 0.0f;

    const uint8_t* kbase = a.k + (int64_t)b * a.k_b + (int64_t)hk * a.k_h;
    const uint8_t* vbase = a.v + (int64_t)b * a.v_b + (int64_t)hk * a.v_h;
    const uint8_t* mrow = a.mask ? a.mask + (int64_t)b * a.mask_b : nullptr;
    TileStage<DP, KT, NW> ks, vs;
    ks.init(wave, lane, a.D, (unsigned)a.k_t);
    vs.init(wave, lane, a.D, (unsigned)a.v_t);
    if (j_begin < j_end) {
        uint64_t word = mask_word(mask_byte(mrow, j_begin, j_end, lane), j_end - j_begin);
        ks.issue(kbase + (int64_t)j_begin * a.k_t, word, lds, wave);
        vs.issue(vbase + (int64_t)j_begin * a.v_t, word, lds + TILE, wave);
        uint32_t mb = mask_byte(mrow, j_begin + KT, j_end, lane);
        int buf = 0;
        for (int j = j_begin; j < j_end; j += KT) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            const uint8_t* kl = lds + buf * 2 * TILE;
            const uint8_t* vl = kl + TILE;
            const uint64_t next = mask_word(mb, j_end - (j + KT));
            if (j + KT < j_end) {
                uint8_t* nl = lds + (buf ^ 1) * 2 * TILE;
                ks.issue(kbase + (int64_t)(j + KT) * a.k_t, next, nl, wave);
                vs.issue(vbase + (int64_t)(j + KT) * a.v_t, next, nl + TILE, wave);
                mb = mask_byte(mrow, j + 2 * KT, j_end, lane);
            }
            if (word != 0) {
#pragma unroll
                for (int kb = 0; kb < KT / 32; ++kb) {
                    f32x16 s, dp;
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.0f;
#pragma unroll
                    for (int x = 0; x < KS; ++x) {
                        const i32x4 kf = frag_row<DP>(kl, 32 * kb + (lane & 31), 2 * x + half);
                        s = mfma32<DT>(&kf, &qf[x], s);
                    }
#pragma unroll
                    for (int x = 0; x < KS; ++x) {
                        const i32x4 vf = frag_row<DP>(vl, 32 * kb + (lane & 31), 2 * x + half);
                        dp = mfma32<DT>(&vf, &gf[x], dp);
                    }
                    const uint32_t w = (uint32_t)(word >> (32 * kb)) >> (4 * half);
                    float ds[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], a.c, -L));
                        ds[i] = p * (dp[i] + De) * f;
                    }
                    if (word != ~0ull) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (!((w >> (8 * (i / 4) + i % 4)) & 1)) ds[i] = 0.0f;
                    }
                    i32x4 df[2];
                    pack_frag<DT>(ds, df);
#pragma unroll
                    for (int g = 0; g < 2; ++g)
#pragma unroll
                        for (int d = 0; d < DB; ++d) {
                            const i32x4 kt = frag_col<DP>(kl, 32 * kb + 16 * g, d, lane);
                            dq[d] = mfma32<DT>(&kt, &df[g], dq[d]);
                        }
                }
            }
            word = next;
            buf ^= 1;
        }
    }
    const float fq = a.scale / f;
    if (a.nsplit > 1) {
        const int64_t n = (int64_t)a.B * a.Hk * a.rows * a.D;
        const __amdgpu_buffer_rsrc_t rs =
            attn_rsrc(a.part + sp * n + ((int64_t)bh * a.rows + row0) * a.D);
        const unsigned off = live ? (unsigned)((lane & 31) * a.D) * 4 : kOut;
#pragma unroll
        for (int d = 0; d < DB; ++d) store_part(rs, off, dq[d], fq, 32 * d, a.D, half);
        return;
    }
    const __amdgpu_buffer_rsrc_t rs = attn_rsrc(a.dq + (int64_t)b * a.dq_b +
                                                (int64_t)hk * a.G * a.dq_h + (int64_t)t0 * a.dq_t);
    const unsigned off = packed_off(a, row, t0, a.dq_t, a.dq_h);
#pragma unroll
    for (int d = 0; d < DB; ++d) store_block<DT>(rs, off, dq[d], fq, 32 * d, a.D, half);
}

// ---------------------------------------------------------------------------
// Sums of split launches, splits in order: 4 values a thread.  keys: dk
// (blockIdx.y = 0) and dv (1) of a dk dv launch; otherwise dq.
template <int DT>
__global__ __launch_bounds__(256) void attn_bwd_join_kernel(AttnArgs a, int keys) {
    const int per = a.D / 4;
    const int count = keys ? a.Tk : a.rows;
    const int64_t n = (int64_t)a.B * a.Hk * count;
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= n * per) return;
    const int64_t at = e / per;
    const int d = (int)(e - at * per) * 4;
    const float* src = a.part + (blockIdx.y ? a.nsplit * n * a.D : 0) + at * a.D + d;
    f32x4 o = {0, 0, 0, 0};
#pragma unroll 4
    for (int s = 0; s < a.nsplit; ++s) o += *reinterpret_cast<const f32x4*>(src + s * n * a.D);
    const int64_t bh = at / count;
    const int r = (int)(at - bh * count);
    const int b = (int)(bh / a.Hk), hk = (int)(bh - (int64_t)b * a.Hk);
    uint8_t* dst;
    const int tok = div_g(a, r);
    if (!keys)
        dst = a.dq + (int64_t)b * a.dq_b + (int64_t)hk * a.G * a.dq_h + (int64_t)tok * a.dq_t +
              packed_off(a, r, tok, a.dq_t, a.dq_h);
    else if (blockIdx.y == 0)
        dst = a.dk + (int64_t)b * a.dk_b + (int64_t)hk * a.dk_h + (int64_t)r * a.dk_t;
    else
        dst = a.dv + (int64_t)b * a.dv_b + (int64_t)hk * a.dv_h + (int64_t)r * a.dv_t;
    *reinterpret_cast<u32x2*>(dst + d * 2) =
        u32x2{pack_out2(o[0], o[1], DT), pack_out2(o[2], o[3], DT)};
}

}  // namespace igc
