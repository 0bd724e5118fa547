// Cross attention, forward.
//
// Rows are the Tq * G queries that share one key head (G query heads a key
// head), so grouped heads read their keys once.  Each wave keeps a block of
// 32 rows: scores come as S^T = K Q^T (keys down the registers, one row a
// lane), which makes the softmax statistics of a row a sum over one lane's
// registers plus one exchange between the wave's halves, and lets P^T go into
// O^T += V^T P^T as the B operand without leaving its lane.
#pragma once

#include "attn_common.hpp"

namespace igc {

// fp16 holds probabilities down to 2^-14 with full precision: they are
// scaled by 2^7 (the sum l with them, so the factor leaves in O / l).  With
// the statistics' slack of 2^8 below they stay under 2^15.  bf16 has fp32's
// range and needs none.
template <int DT>
__device__ __forceinline__ constexpr float p_shift() {
    return DT == DT_FP16 ? 7.0f : 0.0f;
}
// The running maximum follows the true one only when a row exceeds it by
// 2^kSlack: O and l are then rescaled, which most tiles so skip.  The
// maximum only guards the range, so the result does not depend on it beyond
// rounding.
constexpr float kSlack = 8.0f;

// Softmax step of one block of 32 rows over KB blocks of 32 keys: scores s
// become probabilities, m (scaled by c, in powers of two) and l follow, and
// acc is rescaled where a maximum moved.  `word` has a bit per key.
template <int DT, int KB, int DB>
__device__ __forceinline__ void softmax_step(f32x16 (&s)[KB], uint64_t word, bool full, float c,
                                             float& m, float& l, f32x16 (&acc)[DB], int half) {
    if (!full) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const uint32_t w = (uint32_t)(word >> (32 * kb)) >> (4 * half);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (!((w >> (8 * (i / 4) + i % 4)) & 1)) s[kb][i] = -__builtin_inff();
        }
    }
    float t = -__builtin_inff();
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; i += 2) t = fmaxf(fmaxf(s[kb][i], s[kb][i + 1]), t);
    t = max_halves(t) * c;
    if (__any(t > m + kSlack)) {   // also the first tile with a valid key: m = -inf
        const float mn = fmaxf(m, t);
        // rows still without a valid key: 2^(-inf - 0) keeps everything 0
        const float f = mn == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= f;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[d][i] *= f;
    }
    const float ms = (m == -__builtin_inff() ? 0.0f : m) - p_shift<DT>();
    float sum[4] = {0, 0, 0, 0};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][i], c, -ms));
            s[kb][i] = p;
            sum[i & 3] += p;
        }
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

// Results of a block of 32 rows from row0 (this lane's: row0 + lane % 32):
// the final output, or the partial result of one split.
template <int DT, int DB>
__device__ __forceinline__ void fwd_finish(const AttnArgs& a, int b, int hk, int sp, int row0,
                                           int lane, f32x16 (&acc)[DB], float m, float l) {
    const int half = lane >> 5, r = lane & 31, row = row0 + r;
    l = sum_halves(l);
    const bool live = row < a.rows;
    if (a.nsplit > 1) {
        const int64_t bh = (int64_t)b * a.Hk + hk;
        const int64_t at = ((int64_t)sp * a.B * a.Hk + bh) * a.rows + row0;
        const __amdgpu_buffer_rsrc_t rs = attn_rsrc(a.part + at * a.D);
        const unsigned off = live ? (unsigned)(r * a.D) * 4 : kOut;
#pragma unroll
        for (int db = 0; db < DB; ++db) store_part(rs, off, acc[db], 1.0f, 32 * db, a.D, half);
        store4(attn_rsrc(a.stat + at * 2), live ? (unsigned)(r * 2 + half) * 4 : kOut,
               half ? l : m);
        return;
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);   // NaN stays NaN
    const int t0 = div_g(a, row0);
    const __amdgpu_buffer_rsrc_t rs = attn_rsrc(a.out + (int64_t)b * a.o_b +
                                                (int64_t)hk * a.G * a.o_h + (int64_t)t0 * a.o_t);
    const unsigned off = packed_off(a, row, t0, a.o_t, a.o_h);
#pragma unroll
    for (int db = 0; db < DB; ++db) store_block<DT>(rs, off, acc[db], inv, 32 * db, a.D, half);
    if (a.lse)   // l carries 2^p_shift
        store4(lse_base(a, b, hk), half == 0 ? lse_off(a, row) : kOut,
               l == 0.0f ? -__builtin_inff()
                         : (m + __builtin_amdgcn_logf(l) - p_shift<DT>()) * kLn2);
}

// ---------------------------------------------------------------------------
// Many rows: NW waves of 32 rows walk the keys in tiles of 64, double buffered
// in LDS through direct loads, one barrier a tile.  At 128 values a head the
// matrix cores and the vector units are both busy for half of the time and the
// power limit sets the clock (2 x 16384 rows x 4096 keys, 16 heads: 1.04 ms,
// 1.05 PFLOP/s; with two blocks of rows a wave, which leaves one wave a SIMD,
// 2.7 ms).  At 64 the softmax's vector instructions bound it (4 x 3136 x 1333
// ragged, 16 heads: 67 to 75 us).
// Waves a SIMD that the registers of the kernel below are cut to (and its LDS
// allows): one register more than 512 / waves costs a wave.
constexpr int fwd_waves(int dp) { return dp <= 64 ? 4 : dp <= 96 ? 3 : 2; }

// MASK: a key mask is given, so that any tile may have keys that are not
// valid; their score products then start from -inf (LDS), which costs eight
// LDS reads a tile instead of three instructions a score.
template <int DT, int DP, int NW, bool MASK>
__global__ __launch_bounds__(NW * 64, fwd_waves(DP)) void attn_fwd_kernel(AttnArgs a) {
    constexpr int KT = 64, KB = 2, DB = DP / 32, KS = DP / 16;
    constexpr int TILE = KT * DP * 2;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    lds_poison<NW * 64>(lds, 4 * TILE + 2 * KT * 4);
    float* bias = reinterpret_cast<float*>(lds + 4 * TILE);   // [2][KT], MASK
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int half = lane >> 5;

    int idx = launch_place(a);
    const int rt = idx % a.row_tiles;
    idx /= a.row_tiles;
    const int sp = idx % a.nsplit;
    idx /= a.nsplit;
    const int hk = idx % a.Hk, b = idx / a.Hk;

    const int len = a.lens ? max(0, min(a.lens[b], a.Tk)) : a.Tk;
    const int j_begin = sp * a.split, j_end = split_end(j_begin, a.split, len);

    i32x4 qf[KS];
    f32x16 acc[DB];
    float m = -__builtin_inff(), l = 0.0f;
    const int row0 = (rt * NW + wave) * 32, t0 = div_g(a, row0);
    const __amdgpu_buffer_rsrc_t qrs = attn_rsrc(
        a.q + (int64_t)b * a.q_b + (int64_t)hk * a.G * a.q_h + (int64_t)t0 * a.q_t);
    load_rows<DP>(qrs, packed_off(a, row0 + (lane & 31), t0, a.q_t, a.q_h), a.D, half, qf);
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;

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
        if (MASK && wave == 0) bias[lane] = (word >> lane) & 1 ? 0.0f : -__builtin_inff();
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
                if (MASK && wave == 0)
                    bias[(buf ^ 1) * KT + lane] = (next >> lane) & 1 ? 0.0f : -__builtin_inff();
            }
            if (word != 0) {
                f32x16 s[KB];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        f32x4 x = {0, 0, 0, 0};
                        if constexpr (MASK)
                            x = *reinterpret_cast<const f32x4*>(bias + buf * KT + 32 * kb + 8 * g +
                                                                4 * half);
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[kb][4 * g + i] = x[i];
                    }
#pragma unroll
                    for (int x = 0; x < KS; ++x) {
                        const i32x4 kf = frag_row<DP>(kl, 32 * kb + (lane & 31), 2 * x + half);
                        s[kb] = mfma32<DT>(&kf, &qf[x], s[kb]);
                    }
                }
                softmax_step<DT, KB, DB>(s, word, MASK || word == ~0ull, a.c, m, l, acc, half);
                i32x4 pf[KB][2];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    float p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) p[i] = s[kb][i];
                    pack_frag<DT>(p, pf[kb]);
                }
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int g = 0; g < 2; ++g)
#pragma unroll
                        for (int d = 0; d < DB; ++d) {
                            const i32x4 vf = frag_col<DP>(vl, 32 * kb + 16 * g, d, lane);
                            acc[d] = mfma32<DT>(&vf, &pf[kb][g], acc[d]);
                        }
            }
            word = next;
            buf ^= 1;
        }
    }
    fwd_finish<DT, DB>(a, b, hk, sp, row0, lane, acc, m, l);
}

// ---------------------------------------------------------------------------
// At most 32 rows (single tokens): the waves of a workgroup take blocks of 32
// keys in turn, each through LDS of its own without barriers.  A wave asks
// for its next block's keys as soon as the score products have read the
// present ones, and for the next values after the second product, so that its
// memory requests never pause; the waves' results are joined through LDS at
// the end.  Long caches are bound by HBM (4 sequences of up to 65537 keys, 8
// key heads of 128: 149 us, 5.4 TB/s), short ones by latency, one a round of
// all waves: eight waves in half the LDS each (8 x 784 keys: 8.5 us, the long
// ones 144 to 149) beat four with whole double buffers (11.0 and 158).
template <int DT, int DP, int NW>
__global__ __launch_bounds__(NW * 64, 2) void attn_token_kernel(AttnArgs a) {
    constexpr int KT = 32, DB = DP / 32, KS = DP / 16;
    constexpr int TILE = KT * DP * 2;
    constexpr int STAGE = 2 * TILE;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    lds_poison<NW * 64>(lds, NW * STAGE + NW * 64 * 4);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int half = lane >> 5;
    uint8_t* mine = lds + wave * STAGE;   // keys, values
    float* st_m = reinterpret_cast<float*>(lds + NW * STAGE);   // [NW][32] m, then l
    float* st_l = st_m + NW * 32;

    int idx = launch_place(a);
    const int sp = idx % a.nsplit;
    idx /= a.nsplit;
    const int hk = idx % a.Hk, b = idx / a.Hk;
    const int len = a.lens ? max(0, min(a.lens[b], a.Tk)) : a.Tk;
    const int j_begin = sp * a.split + wave * KT, j_end = split_end(sp * a.split, a.split, len);

    const int row = lane & 31;
    i32x4 qf[KS];
    load_rows<DP>(attn_rsrc(a.q + (int64_t)b * a.q_b + (int64_t)hk * a.G * a.q_h),
                  packed_off(a, row, 0, a.q_t, a.q_h), a.D, half, qf);
    f32x16 acc[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f;

    const uint8_t* kbase = a.k + (int64_t)b * a.k_b + (int64_t)hk * a.k_h;
    const uint8_t* vbase = a.v + (int64_t)b * a.v_b + (int64_t)hk * a.v_h;
    const uint8_t* mrow = a.mask ? a.mask + (int64_t)b * a.mask_b : nullptr;
    TileStage<DP, KT, 1> ks, vs;
    ks.init(0, lane, a.D, (unsigned)a.k_t);
    vs.init(0, lane, a.D, (unsigned)a.v_t);
    constexpr int LOADS = TileStage<DP, KT, 1>::PIECES;   // requests a block of keys, or of values
    constexpr int STEP = NW * KT;

    auto word_at = [&](uint32_t mb, int j) -> uint32_t {
        return (uint32_t)(mask_word(mb, j_end - j) & 0xffffffffu);
    };
    if (j_begin < j_end) {
        uint32_t w0 = word_at(mask_byte(mrow, j_begin, j_end, lane), j_begin), w1 = 0;
        uint32_t mb = mask_byte(mrow, j_begin + STEP, j_end, lane);
        ks.issue(kbase + (int64_t)j_begin * a.k_t, w0, mine, 0);
        vs.issue(vbase + (int64_t)j_begin * a.v_t, w0, mine + TILE, 0);
        for (int j = j_begin; j < j_end; j += STEP) {
            const bool more = j + STEP < j_end;
            // the keys: all but the values requested after them
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS) : "memory");
            f32x16 s[1];
#pragma unroll
            for (int i = 0; i < 16; ++i) s[0][i] = 0.0f;
#pragma unroll
            for (int x = 0; x < KS; ++x) {
                const i32x4 kf = frag_row<DP>(mine, lane & 31, 2 * x + half);
                s[0] = mfma32<DT>(&kf, &qf[x], s[0]);
            }
            // their LDS is read: the next block's may arrive
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (more) {
                w1 = word_at(mb, j + STEP);
                mb = mask_byte(mrow, j + 2 * STEP, j_end, lane);
                ks.issue(kbase + (int64_t)(j + STEP) * a.k_t, w1, mine, 0);
            }
            softmax_step<DT, 1, DB>(s, w0, w0 == ~0u, a.c, m, l, acc, half);
            i32x4 pf[2];
            float p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) p[i] = s[0][i];
            pack_frag<DT>(p, pf);
            // the values: all but the next keys (the mask byte is older)
            if (more) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS) : "memory");
            else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    const i32x4 vf = frag_col<DP>(mine + TILE, 16 * g, d, lane);
                    acc[d] = mfma32<DT>(&vf, &pf[g], acc[d]);
                }
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (more) vs.issue(vbase + (int64_t)(j + STEP) * a.v_t, w1, mine + TILE, 0);
            w0 = w1;
        }
    }
    // join: wave w's rows as floats [rows][DP] over its own LDS.  The one lane
    // branch around accumulators: they end in it, so that nothing is copied at
    // its join (all 32 rows stored without it: 8 x 784 keys 9.5 -> 11.9 us)
    l = sum_halves(l);
    float* po = reinterpret_cast<float*>(mine);
    if (row < a.rows) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<f32x4*>(po + row * DP + 32 * d + 8 * g + 4 * half) =
                    f32x4{acc[d][4 * g], acc[d][4 * g + 1], acc[d][4 * g + 2], acc[d][4 * g + 3]};
        if (half == 0) {
            st_m[wave * 32 + row] = m;
            st_l[wave * 32 + row] = l;
        }
    }
    __syncthreads();
    // four values a thread
    const int per = a.D / 4;
    for (int e = threadIdx.x; e < a.rows * per; e += NW * 64) {
        const int r = e / per, d = (e - r * per) * 4;
        float mm = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < NW; ++w) mm = fmaxf(mm, st_m[w * 32 + r]);
        const float ms = mm == -__builtin_inff() ? 0.0f : mm;
        float ll = 0.0f;
        f32x4 o = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = __builtin_amdgcn_exp2f(st_m[w * 32 + r] - ms);
            ll = __builtin_fmaf(st_l[w * 32 + r], f, ll);
            const f32x4 x = *reinterpret_cast<const f32x4*>(
                reinterpret_cast<const float*>(lds + w * STAGE) + r * DP + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(x[i], f, o[i]);
        }
        const int64_t bh = (int64_t)b * a.Hk + hk;
        if (a.nsplit > 1) {
            const int64_t at = ((int64_t)sp * a.B * a.Hk + bh) * a.rows + r;
            *reinterpret_cast<f32x4*>(a.part + at * a.D + d) = o;
            if (d == 0) {
                a.stat[at * 2] = mm;
                a.stat[at * 2 + 1] = ll;
            }
            continue;
        }
        const float inv = ll > 0.0f ? 1.0f / ll : (ll == 0.0f ? 0.0f : ll);
        uint8_t* dst = a.out + (int64_t)b * a.o_b + (int64_t)hk * a.G * a.o_h +
                       packed_off(a, r, 0, a.o_t, a.o_h) + d * 2;
        *reinterpret_cast<u32x2*>(dst) =
            u32x2{pack_out2(o[0] * inv, o[1] * inv, DT), pack_out2(o[2] * inv, o[3] * inv, DT)};
        const int tok = div_g(a, r);
        if (a.lse && d == 0)
            a.lse[((int64_t)b * a.Hq + hk * a.G + (r - tok * a.G)) * a.Tq + tok] =
                ll == 0.0f ? -__builtin_inff()
                           : (mm + __builtin_amdgcn_logf(ll) - p_shift<DT>()) * kLn2;
    }
}

// ---------------------------------------------------------------------------
// Join of split launches.  32 lanes take a packed row, 4 values a lane.  Few
// rows of many splits: a workgroup a row, its GR = 8 groups of lanes sum
// every 8th split, and the 8 sums are added in order through LDS.  Few splits
// (GR = 1): 8 rows a workgroup, each group sums its row's splits in order
// (2 splits of 19800 rows: 20.6 us with a workgroup a row).
constexpr int kJoinLanes = 32, kJoinFew = 8;
template <int DT, int GR>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
    __shared__ f32x4 part[GR][kJoinLanes];
    __shared__ __attribute__((aligned(16))) float sum[GR > 4 ? GR : 4];
    if constexpr (GR > 1) {
        lds_poison<256>(reinterpret_cast<uint8_t*>(part), sizeof(part));
        lds_poison<256>(reinterpret_cast<uint8_t*>(sum), sizeof(sum));
    }
    const int64_t n = (int64_t)a.B * a.Hk * a.rows;
    const int lane = threadIdx.x % kJoinLanes, group = threadIdx.x / kJoinLanes;
    const int64_t at = GR > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 8 + group;
    const int g = GR > 1 ? group : 0, d = lane * 4;
    if (at >= n) return;   // GR = 1 only, which has no barrier below
    // the maximum over the splits, by every group of 32 lanes
    float mm = -__builtin_inff();
    for (int s = lane; s < a.nsplit; s += kJoinLanes)
        mm = fmaxf(mm, a.stat[(s * n + at) * 2]);
#pragma unroll
    for (int o = 1; o < kJoinLanes; o <<= 1) mm = fmaxf(mm, __shfl_xor(mm, o, 64));
    const float ms = mm == -__builtin_inff() ? 0.0f : mm;
    float ll = 0.0f;
    f32x4 o = {0, 0, 0, 0};
    for (int s = g; s < a.nsplit; s += GR) {
        const float f = __builtin_amdgcn_exp2f(a.stat[(s * n + at) * 2] - ms);
        ll = __builtin_fmaf(a.stat[(s * n + at) * 2 + 1], f, ll);
        if (d < a.D) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(a.part + (s * n + at) * a.D + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(x[i], f, o[i]);
        }
    }
    if constexpr (GR > 1) {
        part[g][lane] = o;
        if (d == 0) sum[g] = ll;
        __syncthreads();
        if (g != 0) return;
        ll = sum[0];
        for (int i = 1; i < GR; ++i) {
            ll += sum[i];
            o += part[i][lane];
        }
    }
    if (d >= a.D) return;
    const float inv = ll > 0.0f ? 1.0f / ll : (ll == 0.0f ? 0.0f : ll);
    const int64_t bh = at / a.rows;
    const int r = (int)(at - bh * a.rows);
    const int b = (int)(bh / a.Hk), hk = (int)(bh - (int64_t)b * a.Hk);
    const int tok = div_g(a, r);
    uint8_t* dst = a.out + (int64_t)b * a.o_b + (int64_t)hk * a.G * a.o_h +
                   (int64_t)tok * a.o_t + packed_off(a, r, tok, a.o_t, a.o_h) + d * 2;
    *reinterpret_cast<u32x2*>(dst) =
        u32x2{pack_out2(o[0] * inv, o[1] * inv, DT), pack_out2(o[2] * inv, o[3] * inv, DT)};
    if (a.lse && d == 0)
        a.lse[((int64_t)b * a.Hq + hk * a.G + (r - tok * a.G)) * a.Tq + tok] =
            ll == 0.0f ? -__builtin_inff()
                       : (mm + __builtin_amdgcn_logf(ll) - p_shift<DT>()) * kLn2;
}

}  // namespace igc
