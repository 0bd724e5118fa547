// Attention of a few new tokens over the paged cache in 8 bits.
//
// Rows are the Tq * G queries that share one key head, 16 RB a workgroup; its
// eight waves take blocks of 32 keys in turn.  With k_j = ks_j K_j and v_j = vs_j V_j
// (integers K, V):
//   s_j = (q . K_j) ks_j scale,  p_j = 2^(s_j log2 e - m),
//   out = sum (p_j vs_j) V_j / sum p_j
// so that the integers enter the matrix products as they are: 8 bits are exact
// in both 16-bit types, and the scales go to the scores and probabilities.
//
// All products are v_mfma_f32_16x16x32: lane l supplies row (A) or column (B)
// l % 16 with 8 k at slots 8 (l / 16), and the result has column l % 16 and, in
// register i, row 4 (l / 16) + i.  Scores come as S^T = K Q^T, two products of
// 16 keys (t = 0, 1); row r of product t is given key 8 (r / 4) + 4 t + r % 4,
// so that a lane's 8 scores are 8 neighbouring keys and become a B operand of
// O^T += V^T P^T without leaving it; the other operand is one transposing 8-bit
// read of the values.
//
// p vs is held as the sum of two bf16 numbers (16 bits of its own), which
// doubles the second products but leaves the outputs as accurate as fp32
// probabilities, for both types; the matrix cores are busy 11 %.
//
// Long caches are bound by HBM: 4 sequences of 22000 to 65537 tokens, 8 key heads
// of 128, in 76 to 82 us (369 MB, 4.5 to 4.9 TB/s), then 5.0 us for the join.  Short
// ones by vector instructions, of which a block of 32 keys takes about 340, half
// of them for turning 8-bit values into 16-bit ones (0.8 us a block and SIMD), and
// by round trips: entry of the table, keys, values.  16 sequences of 4099 with 5
// drafts, 8 heads of 80: 17 to 19 us, vector units 61 % busy.
#pragma once

#include "attn_common.hpp"
#include "cache_plan.hpp"

namespace igc {

struct CacheAttnArgs {
    AttnArgs a;            // q, out, lse, sizes; part, stat
    const int8_t* pool[2];
    const float* scales[2];
    const int32_t* table;
    const int32_t* lens;
    int64_t table_stride;
    int64_t capacity;      // tokens a row of the table reaches
    int64_t slots;         // of cache_plan.hpp
    int entries, pages, shift, Dp;
    int causal;
    int tile;              // rows a workgroup: 16 or 32
    int split;             // whether workgroups share a sequence (then a join follows)
    int fixed;             // slots of each sequence, or 0: divided by their lengths
};

constexpr int kCacheWaves = 8;   // a workgroup
// The running maximum follows the true one only when a row exceeds it by
// 2^kCacheSlack: it only guards the range.
constexpr float kCacheSlack = 8.0f;

// One transposing read of 8-bit values: 16 lanes address 8 rows of 16 bytes,
// lane i bytes 8 (i % 2) of row i / 2, and lane i gets the 8 rows of column i.
// Restrict for the same reason as read_tr.
__device__ __forceinline__ u32x2 read_tr8(const uint8_t* __restrict__ p) {
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    typedef __attribute__((address_space(3))) i32x2* lp;
    typedef __attribute__((address_space(3))) const uint8_t* bp;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lp)(bp)p));
}

// Four values of a packed row's result, and the row's lse; given: the
// sequence's length as given, not negative.  l is 0 without a key, and where all
// scores are -inf, which is NaN: the largest finite score would add 1 or more.
template <int DT>
__device__ __forceinline__ void cache_attn_out(const CacheAttnArgs& x, int b, int hk, int row,
                                               int d, int given, const f32x4& o, float m,
                                               float l) {
    const AttnArgs& a = x.a;
    const int tok = div_g(a, row), g = row - tok * a.G;
    const int seen = given - (x.causal ? a.Tq - 1 - tok : 0);
    if (l == 0.0f && seen > 0 && x.capacity > 0) l = __builtin_nanf("");
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);   // NaN stays NaN
    uint8_t* dst = a.out + (int64_t)b * a.o_b + (int64_t)tok * a.o_t +
                   ((int64_t)hk * a.G + g) * a.o_h + d * 2;
    *reinterpret_cast<u32x2*>(dst) =
        u32x2{pack_out2(o[0] * inv, o[1] * inv, DT), pack_out2(o[2] * inv, o[3] * inv, DT)};
    if (a.lse && d == 0)
        a.lse[((int64_t)b * a.Hq + (int64_t)hk * a.G + g) * a.Tq + tok] =
            l == 0.0f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

// A workgroup's place: sequence, (key head, row tile), part of the sequence's
// parts, and the first of its keys and the end.
struct CachePlace {
    int b, hr, part, parts;
    int64_t begin, end;
    int len;
    int slot0;             // slot of part 0 of the sequence's first (key head, row tile)
};

// The same for sequences with slots of their own, x.fixed a (key head, row
// tile): no sums over the lengths (8 x 784: 10.2 -> 9.7 us).
__device__ __forceinline__ void cache_fixed_place(const CacheAttnArgs& x, int b, int hr_n,
                                                  CachePlace* o) {
    typedef __attribute__((address_space(4))) const int32_t* sp;
    o->b = b;
    o->len = cache_len(((sp)x.lens)[b], x.capacity);
    o->parts = (int)cache_parts(o->len, kCacheLeast);
    o->slot0 = b * hr_n * x.fixed;
}

// Sum of x over the lanes up to this one.
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
    // within rows of 16 lanes, then the rows before
#define IGC_STEP(ctrl, rows) \
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, ctrl, rows, 0xf, false)
    IGC_STEP(0x111, 0xf);   // row_shr:1
    IGC_STEP(0x112, 0xf);
    IGC_STEP(0x114, 0xf);
    IGC_STEP(0x118, 0xf);
    IGC_STEP(0x142, 0xa);   // row_bcast:15 to rows 1 and 3
    IGC_STEP(0x143, 0xc);   // row_bcast:31 to rows 2 and 3
#undef IGC_STEP
    return x;
}
__device__ __forceinline__ uint32_t lane_value(uint32_t x, int lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)x, lane);
}

// Division of the work, by whole waves: every wave forms it.
struct CacheDivision {
    uint32_t chunk;
    int first;             // the lane's length, of the first 64 sequences
    __device__ __forceinline__ int len(const CacheAttnArgs& x, int b) const {
        return b < x.a.B ? cache_len(x.lens[b], x.capacity) : 0;
    }
    __device__ __forceinline__ void init(const CacheAttnArgs& x, int lane) {
        first = len(x, lane);
        uint32_t total = lane_value(wave_scan(cache_units(first)), 63);
        for (int base = 64; base < x.a.B; base += 64)
            total += lane_value(wave_scan(cache_units(len(x, base + lane))), 63);
        chunk = cache_chunk(total, (uint32_t)(x.slots - x.a.B));
        uint32_t low = cache_chunk(total, (uint32_t)x.slots);   // chunk fits; below low nothing does
        for (int i = 0; i < kCacheBisect && low < chunk; ++i) {
            const uint32_t mid = low + (chunk - low) / 2;
            if (parts(x, lane, mid) <= (uint32_t)x.slots) chunk = mid;
            else low = mid + 1;
        }
    }
    __device__ __forceinline__ uint32_t parts(const CacheAttnArgs& x, int lane,
                                              uint32_t c) const {
        uint32_t n = 0;
        for (int base = 0; base < x.a.B; base += 64)
            n += lane_value(wave_scan(base + lane < x.a.B
                                          ? cache_parts(base ? len(x, base + lane) : first, c) : 0),
                            63);
        return n;
    }
    // The sequence that workgroup w works on (b < 0), or sequence b: its
    // parts, length and first slot.  False for workgroups past the last part.
    __device__ __forceinline__ bool find(const CacheAttnArgs& x, int lane, uint32_t w, int hr_n,
                                         int b, CachePlace* o) const {
        uint32_t before = 0;
        for (int base = 0; base < x.a.B; base += 64) {
            const int n = base ? len(x, base + lane) : first;
            const uint32_t k = base + lane < x.a.B ? cache_parts(n, chunk) : 0;
            const uint32_t sum = wave_scan(k);
            const uint64_t here = b >= 0 ? (b < base + 64 ? 1ull << (b - base) : 0)
                                         : __ballot(w < (before + sum) * hr_n && k > 0);
            if (here) {
                const int f = __builtin_ctzll(here);
                o->b = base + f;
                o->parts = (int)lane_value(k, f);
                o->len = (int)lane_value((uint32_t)n, f);
                o->slot0 = (int)((before + lane_value(sum, f) - o->parts) * hr_n);
                return true;
            }
            before += lane_value(sum, 63);
        }
        return false;
    }
};

// 8 bytes as 8 values of the 16-bit type.
template <int DT>
__device__ __forceinline__ i32x4 bytes_frag(uint32_t lo, uint32_t hi) {
    i32x4 f;
    if constexpr (DT == DT_FP16) {
        // 0x6400 | u is 1024 + u; less 1152 it is u - 128
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        const h2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
        lo ^= 0x80808080u;
        hi ^= 0x80808080u;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t u = __builtin_amdgcn_perm(0x64646464u, k < 2 ? lo : hi,
                                                     k & 1 ? 0x04030402u : 0x04010400u);
            f[k] = __builtin_bit_cast(int, __builtin_bit_cast(h2, u) - off);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int w = (int)(k < 2 ? lo : hi) << (k & 1 ? 0 : 16);
            f[k] = (int)pack_out2((float)(int8_t)(w >> 16), (float)(w >> 24), DT_BF16);
        }
    }
    return f;
}

// Tiles hold 32 rows of DP bytes.  Chunk c (16 bytes) of row r lies at a place
// turned by r, so that the 16 rows that a product's lanes read (8 a + 4 t + 0 ..
// 3) and the 8 of a transposing read lie in different banks (96 bytes: nearly).
template <int DP>
__device__ __forceinline__ int tile8_turn(int r) {
    if constexpr (DP == 128)
        return ((r >> 1) & 1) | ((r >> 2) & 2) | ((((r >> 4) ^ (r >> 2)) & 1) << 2);
    if constexpr (DP == 64) return ((r >> 3) ^ ((r >> 2) & 1)) & 3;
    return r >> 3;
}
template <int DP>
__device__ __forceinline__ int tile8_off(int r, int c) {
    const int t = tile8_turn<DP>(r);
    if constexpr (DP == 96) return r * DP + ((c + t) % 6) * 16;
    if constexpr (DP == 32) return r * DP + ((c ^ (t & 1)) << 4);
    return r * DP + ((c ^ t) << 4);
}

// Direct loads of 32 rows of a pool's integers and of their scales; a lane's
// place in LDS fixes its row and chunk.  Chunks past the row read its first
// one: the queries' zeros, or columns that are not stored, meet them.
template <int DP>
struct CacheStage {
    static constexpr int TILE = 32 * DP, PIECES = TILE / 1024;
    static constexpr int BYTES = TILE + 256;   // integers, scales (twice)
    static constexpr int LOADS = PIECES + 1;
    int off[PIECES];
    bool high[PIECES];   // rows 16 .. 31

    __device__ __forceinline__ void init(int lane, int Dp) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int at = i * 1024 + lane * 16, r = at / DP, p = (at % DP) >> 4;
            const int t = tile8_turn<DP>(r);
            const int c = DP == 96 ? (p + 6 - t) % 6 : p ^ (DP == 32 ? t & 1 : t);
            high[i] = r >= 16;
            off[i] = (r & 15) * Dp + (c * 16 < Dp ? c * 16 : 0);
        }
    }
    // rows r0 (the first 16 keys) and r1 of a pool
    __device__ __forceinline__ void issue(const int8_t* pool, const float* scale, int Dp,
                                          int64_t r0, int64_t r1, int lane, uint8_t* lds) const {
        typedef __attribute__((address_space(1))) void* gp;
        typedef __attribute__((address_space(3))) void* lp;
        const int8_t* b0 = pool + r0 * Dp;
        const int8_t* b1 = pool + r1 * Dp;
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
            __builtin_amdgcn_global_load_lds((gp)((high[i] ? b1 : b0) + off[i]),
                                             (lp)(lds + i * 1024), 16, 0, 0);
        const float* s = scale + ((lane & 16) ? r1 : r0) + (lane & 15);
        __builtin_amdgcn_global_load_lds((gp)s, (lp)(lds + TILE), 4, 0, 0);
    }
};

template <int DT>
__device__ __forceinline__ f32x4 mfma16(const i32x4& a, const i32x4& b, f32x4 c) {
    if constexpr (DT == DT_FP16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// x over a lane and those 16, 32 and 48 away.
__device__ __forceinline__ void both_rows(float x, float* lo, float* hi) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t r0 = r[0], r1 = r[1];
    *lo = __builtin_bit_cast(float, r0);
    *hi = __builtin_bit_cast(float, r1);
}
__device__ __forceinline__ float max_quarters(float x) {
    float a, b;
    both_rows(x, &a, &b);
    return max_halves(fmaxf(a, b));
}
__device__ __forceinline__ float sum_quarters(float x) {
    float a, b;
    both_rows(x, &a, &b);
    return sum_halves(a + b);
}

template <int DT, int DP, int RB>
__global__ __launch_bounds__(kCacheWaves * 64, RB == 1 ? 4 : 2) void cache_attn_kernel(CacheAttnArgs x) {
    const AttnArgs& a = x.a;
    constexpr int NW = kCacheWaves, DB = DP / 16, KS = DP / 32, ROWS = 16 * RB;
    using Stage = CacheStage<DP>;
    constexpr int OWN = 2 * Stage::BYTES;   // a wave's keys and values, then 16 rows of results
    static_assert(OWN >= 16 * DP * 4, "a wave's results fit its stages");
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    lds_poison<NW * 64>(lds, NW * OWN + NW * 32 * 4);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int quarter = lane >> 4, r16 = lane & 15;
    uint8_t* kl = lds + wave * OWN;
    uint8_t* vl = kl + Stage::BYTES;
    float* st_m = reinterpret_cast<float*>(lds + NW * OWN);   // [NW][16] m, then l
    float* st_l = st_m + NW * 16;

    const int hr_n = a.Hk * a.row_tiles;
    CachePlace at;
    if (x.split) {
        uint32_t chunk = kCacheLeast;
        if (x.fixed) {
            at.hr = (int)(blockIdx.x / (uint32_t)x.fixed);
            at.part = (int)blockIdx.x - at.hr * x.fixed;
            const int b = at.hr / hr_n;
            at.hr -= b * hr_n;
            cache_fixed_place(x, b, hr_n, &at);
            if (at.part >= at.parts) return;   // all waves
        } else {
            CacheDivision div;
            div.init(x, lane);
            if (!div.find(x, lane, blockIdx.x, hr_n, -1, &at)) return;   // all waves
            const int r = (int)blockIdx.x - at.slot0;
            at.hr = r / at.parts;
            at.part = r - at.hr * at.parts;
            chunk = div.chunk;
        }
        at.begin = (int64_t)at.part * chunk * kCacheUnit;
        at.end = at.begin + (int64_t)chunk * kCacheUnit;
        if (at.end > at.len) at.end = at.len;
    } else {
        at.b = blockIdx.x / hr_n;
        at.hr = blockIdx.x - at.b * hr_n;
        at.len = cache_len(x.lens[at.b], x.capacity);
        at.parts = 1;
        at.begin = 0;
        at.end = at.len;
    }
    const int b = __builtin_amdgcn_readfirstlane(at.b), hr = __builtin_amdgcn_readfirstlane(at.hr);
    const int parts = __builtin_amdgcn_readfirstlane(at.parts);
    const int begin = __builtin_amdgcn_readfirstlane((int)at.begin);
    int end = __builtin_amdgcn_readfirstlane((int)at.end);
    // the length as given places the new tokens, also past the table
    typedef __attribute__((address_space(4))) const int32_t* sp;
    const int given = max(((sp)x.lens)[b], 0);
    const int hk = hr / a.row_tiles, row0 = (hr - hk * a.row_tiles) * ROWS;
    const int t0 = div_g(a, row0);
    // keys past what the last of these rows sees are not read (a prompt of 2048
    // tokens, 16 heads of 128 over 4 key heads: 130 -> 102 us, 97 now)
    if (x.causal) end = min(end, given - (a.Tq - 1 - div_g(a, min(row0 + ROWS, a.rows) - 1)));
    const bool empty = x.pages == 0;   // a pool without pages: nothing to read
    const int stop = empty ? 0 : end;

    Stage stage;
    stage.init(lane, x.Dp);
    // scalar loads: a vector load's wait would be one for the stages in flight
    const sp table = (sp)(x.table + b * x.table_stride);
    constexpr int STEP = NW * 32;
    // Entries of the two halves of the block at j, and the pages they name: the
    // loads are asked for long before their values are looked at.
    auto entries = [&](int j, int* e0, int* e1) {
        *e0 = table[min(j >> x.shift, x.entries - 1)];
        *e1 = table[min((j + 16) >> x.shift, x.entries - 1)];
    };
    auto page = [&](int e, int j) {
        return j >> x.shift < x.entries && e >= 0 && e < x.pages ? e : -1;
    };
    auto issue = [&](int which, int j, int id0, int id1) {
        stage.issue(x.pool[which], x.scales[which], x.Dp,
                    cache_row(id0 < 0 ? 0 : id0, a.Hk, hk, j, x.shift),
                    cache_row(id1 < 0 ? 0 : id1, a.Hk, hk, j + 16, x.shift), lane,
                    which ? vl : kl);
    };

    // queries: a lane reads whole 16-byte chunks of the keys, which are two k
    // steps: steps 2 y + z of quarter f hold values 64 y + 16 f + 8 z .. + 7; a
    // last single step 8 f .. + 7 of its 32
    i32x4 qf[RB][KS];
    int last[RB];   // this lane's row sees the keys before `last`
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const int row = row0 + 16 * i + r16;
        const __amdgpu_buffer_rsrc_t rs = attn_rsrc(
            a.q + (int64_t)b * a.q_b + (int64_t)hk * a.G * a.q_h + (int64_t)t0 * a.q_t);
        const unsigned off = packed_off(a, row, t0, a.q_t, a.q_h);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = (KS & 1) && s == KS - 1 ? 32 * s + 8 * quarter
                                                  : 64 * (s >> 1) + 16 * quarter + 8 * (s & 1);
            qf[i][s] = __builtin_bit_cast(i32x4, load16(rs, d < a.D ? off + 2 * d : kOut));
        }
        last[i] = x.causal ? given - (a.Tq - 1 - div_g(a, min(row, a.rows - 1))) : given;
    }
    f32x4 acc[RB][DB];
    float m[RB], l[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
#pragma unroll
        for (int d = 0; d < DB; ++d) acc[i][d] = f32x4{0, 0, 0, 0};
        m[i] = -__builtin_inff();
        l[i] = 0.0f;
    }

    if (empty) {   // rows with a key are NaN
#pragma unroll
        for (int i = 0; i < RB; ++i)
            if (min(last[i], end) > begin) l[i] = __builtin_nanf("");
    }
    const int j0 = begin + wave * 32;
    int id0 = 0, id1 = 0, nx0 = 0, nx1 = 0;
    // Without a split the first block is asked for before the length is here;
    // whatever the table says past it, the places exist.
    if (j0 < (x.split || empty ? stop : (int)x.capacity)) {
        entries(j0, &nx0, &nx1);
        id0 = page(nx0, j0);
        id1 = page(nx1, j0 + 16);
        issue(0, j0, id0, id1);
        issue(1, j0, id0, id1);
    }
    for (int j = j0; j < stop; j += STEP) {
        const bool more = j + STEP < stop;
        if (more) entries(j + STEP, &nx0, &nx1);
        // the keys: all but the values asked for after them
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(Stage::LOADS) : "memory");
        f32x4 s[RB][2];
#pragma unroll
        for (int i = 0; i < RB; ++i) s[i][0] = s[i][1] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int key = 8 * (r16 >> 2) + 4 * t + (r16 & 3);
#pragma unroll
            for (int y = 0; y < KS / 2; ++y) {
                const u32x4 kb = *reinterpret_cast<const u32x4*>(
                    kl + tile8_off<DP>(key, 4 * y + quarter));
                const i32x4 k0 = bytes_frag<DT>(kb[0], kb[1]), k1 = bytes_frag<DT>(kb[2], kb[3]);
#pragma unroll
                for (int i = 0; i < RB; ++i) {
                    s[i][t] = mfma16<DT>(k0, qf[i][2 * y], s[i][t]);
                    s[i][t] = mfma16<DT>(k1, qf[i][2 * y + 1], s[i][t]);
                }
            }
            if constexpr (KS & 1) {
                const u32x2 kb = *reinterpret_cast<const u32x2*>(
                    kl + tile8_off<DP>(key, 2 * (KS - 1) + (quarter >> 1)) + 8 * (quarter & 1));
                const i32x4 k0 = bytes_frag<DT>(kb[0], kb[1]);
#pragma unroll
                for (int i = 0; i < RB; ++i) s[i][t] = mfma16<DT>(k0, qf[i][KS - 1], s[i][t]);
            }
        }
        // the lane's keys are 8 quarter .. + 7: score k is register k % 4 of
        // product k / 4
        float ks[8];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const f32x4 u = *reinterpret_cast<const f32x4*>(kl + Stage::TILE + 32 * quarter +
                                                            16 * g);
#pragma unroll
            for (int k = 0; k < 4; ++k) ks[4 * g + k] = u[k] * a.c;
        }
        // they are read: the next block's may arrive
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (more) {
            nx0 = page(nx0, j + STEP);
            nx1 = page(nx1, j + STEP + 16);
            issue(0, j + STEP, nx0, nx1);
        }
        const bool bad = (quarter < 2 ? id0 : id1) < 0;   // no such page
        if (id0 < 0 || id1 < 0) {   // its keys, as far as they count, are NaN
#pragma unroll
            for (int k = 0; k < 8; ++k) ks[k] = bad ? __builtin_nanf("") : ks[k];
        }
        float p[RB][8];
        bool full = true;
        int left[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            left[i] = min(last[i], end) - j - 8 * quarter;   // the lane's keys that count
            full = full && left[i] >= 8;
#pragma unroll
            for (int k = 0; k < 8; ++k) p[i][k] = s[i][k >> 2][k & 3] * ks[k];
        }
        full = __all(full);
        if (!full) {
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k >= left[i]) p[i][k] = -__builtin_inff();
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            float t = fmaxf(p[i][0], p[i][1]);
#pragma unroll
            for (int k = 2; k < 8; k += 2) t = fmaxf(fmaxf(p[i][k], p[i][k + 1]), t);
            t = max_quarters(t);
            if (__any(t > m[i] + kCacheSlack)) {
                const float mn = fmaxf(m[i], t);
                // rows still without a key: 2^(-inf - 0) keeps everything 0
                const float f =
                    mn == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m[i] - mn);
                m[i] = mn;
                l[i] *= f;
#pragma unroll
                for (int d = 0; d < DB; ++d) acc[i][d] *= f;
            }
            const float ms = m[i] == -__builtin_inff() ? 0.0f : m[i];
            float sum[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                p[i][k] = __builtin_amdgcn_exp2f(p[i][k] - ms);
                sum[k & 1] += p[i][k];
            }
            l[i] += sum[0] + sum[1];
        }
        // the values: all but the next keys
        if (more) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(Stage::LOADS) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        float vs[8];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const f32x4 u = *reinterpret_cast<const f32x4*>(vl + Stage::TILE + 32 * quarter +
                                                            16 * g);
#pragma unroll
            for (int k = 0; k < 4; ++k) vs[4 * g + k] = u[k];
        }
        if (id0 < 0 || id1 < 0) {
#pragma unroll
            for (int k = 0; k < 8; ++k) vs[k] = bad ? __builtin_nanf("") : vs[k];
        }
        i32x4 hi[RB], lo[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                p[i][k] *= vs[k];
                // keys that do not count may hold anything
                if (!full && k >= left[i]) p[i][k] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                const uint32_t h = pack_out2(p[i][k], p[i][k + 1], DT_BF16);
                hi[i][k / 2] = (int)h;
                lo[i][k / 2] = (int)pack_out2(p[i][k] - __builtin_bit_cast(float, h << 16),
                                              p[i][k + 1] -
                                                  __builtin_bit_cast(float, h & 0xffff0000u),
                                              DT_BF16);
            }
        }
        // values: lane i of 16 reads 8 bytes of row i / 2 of the quarter's 8 and
        // gets its 8 rows of column i
#pragma unroll
        for (int d = 0; d < DB; ++d) {
            const u32x2 vb = read_tr8(vl + tile8_off<DP>(8 * quarter + (r16 >> 1), d) +
                                      8 * (lane & 1));
            const i32x4 vf = bytes_frag<DT_BF16>(vb[0], vb[1]);
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                acc[i][d] = mfma16<DT_BF16>(vf, hi[i], acc[i][d]);
                acc[i][d] = mfma16<DT_BF16>(vf, lo[i], acc[i][d]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (more) issue(1, j + STEP, nx0, nx1);
        id0 = nx0;
        id1 = nx1;
    }
    // join of the waves, 16 rows at a time: each wave's as floats [16][DP] over
    // its stages, once nothing is under way to them
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    float* po = reinterpret_cast<float*>(kl);
    const int per = a.D / 4;
#pragma unroll
    for (int i = 0; i < RB; ++i) {
        const int n = min(16, a.rows - row0 - 16 * i);
        if (i > 0) __syncthreads();
        const float ls = sum_quarters(l[i]);
        if (r16 < n) {
#pragma unroll
            for (int d = 0; d < DB; ++d)
                *reinterpret_cast<f32x4*>(po + r16 * DP + 16 * d + 4 * quarter) = acc[i][d];
            if (quarter == 0) {
                st_m[wave * 16 + r16] = m[i];
                st_l[wave * 16 + r16] = ls;
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < n * per; e += NW * 64) {
            const int r = e / per, d = (e - r * per) * 4;
            float mm = -__builtin_inff();
#pragma unroll
            for (int w = 0; w < NW; ++w) mm = fmaxf(mm, st_m[w * 16 + r]);
            const float ms = mm == -__builtin_inff() ? 0.0f : mm;
            float ll = 0.0f;
            f32x4 o = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = __builtin_amdgcn_exp2f(st_m[w * 16 + r] - ms);
                ll = __builtin_fmaf(st_l[w * 16 + r], f, ll);
                const f32x4 v = *reinterpret_cast<const f32x4*>(
                    reinterpret_cast<const float*>(lds + w * OWN) + r * DP + d);
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] = __builtin_fmaf(v[k], f, o[k]);
            }
            const int row = row0 + 16 * i + r;
            if (parts > 1) {
                const int64_t to = (int64_t)blockIdx.x * min(a.rows, ROWS) + 16 * i + r;
                *reinterpret_cast<f32x4*>(a.part + to * a.D + d) = o;
                if (d == 0) {
                    a.stat[to * 2] = mm;
                    a.stat[to * 2 + 1] = ll;
                }
            } else {
                cache_attn_out<DT>(x, b, hk, row, d, given, o, mm, ll);
            }
        }
    }
}

// Join of the parts of a sequence that several workgroups read: a workgroup a
// row, its eight groups of 32 lanes (4 values a lane) take every eighth part,
// and the eight results are added in order through LDS.  A part's statistics
// and values are asked for together: the groups follow a running maximum of
// their own.
template <int DT>
__global__ __launch_bounds__(256) void cache_attn_join_kernel(CacheAttnArgs x) {
    __shared__ __attribute__((aligned(16))) f32x4 part[8][32];
    __shared__ __attribute__((aligned(16))) float st[2][8];
    lds_poison<256>(reinterpret_cast<uint8_t*>(part), sizeof(part));
    lds_poison<256>(reinterpret_cast<uint8_t*>(st), sizeof(st));
    const AttnArgs& a = x.a;
    const int lane = threadIdx.x & 63, g = threadIdx.x >> 5, d = (threadIdx.x & 31) * 4;
    const int rows_tile = min(a.rows, x.tile), hr_n = a.Hk * a.row_tiles;
    const int br = (int)(blockIdx.x / rows_tile), r = (int)blockIdx.x - br * rows_tile;
    const int b = br / hr_n, hr = br - b * hr_n;
    const int hk = hr / a.row_tiles, row = (hr - hk * a.row_tiles) * x.tile + r;
    if (row >= a.rows) return;
    CachePlace at;
    if (x.fixed) {
        cache_fixed_place(x, b, hr_n, &at);
    } else {
        CacheDivision div;
        div.init(x, lane);
        div.find(x, lane, 0, hr_n, b, &at);
    }
    if (at.parts <= 1) return;   // written where it was read
    const int64_t slot = at.slot0 + hr * (x.fixed ? x.fixed : at.parts);
    const float* stat = a.stat + (slot * rows_tile + r) * 2;
    const float* from = a.part + (slot * rows_tile + r) * a.D + (d < a.D ? d : 0);
    const int64_t pitch = (int64_t)rows_tile * a.D;
    float mm = -__builtin_inff(), ll = 0.0f;
    f32x4 o = {0, 0, 0, 0};
    auto scale = [](float from, float to) {   // 2^(from - to), parts without a key left out
        return from == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(from - to);
    };
    constexpr int U = 4;   // parts asked for at once
    for (int s0 = g; s0 < at.parts; s0 += 8 * U) {
        float m[U], l[U];
        f32x4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + 8 * u;
            const int64_t i = s < at.parts ? s : s0;
            m[u] = stat[i * rows_tile * 2];
            l[u] = stat[i * rows_tile * 2 + 1];
            v[u] = *reinterpret_cast<const f32x4*>(from + i * pitch);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + 8 * u >= at.parts) break;
            const float n = fmaxf(mm, m[u]), f = scale(mm, n), k = scale(m[u], n);
            mm = n;
            ll = __builtin_fmaf(l[u], k, ll * f);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(v[u][i], k, o[i] * f);
        }
    }
    part[g][threadIdx.x & 31] = o;
    if (d == 0) {
        st[0][g] = mm;
        st[1][g] = ll;
    }
    __syncthreads();
    if (g != 0 || d >= a.D) return;
    mm = st[0][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) mm = fmaxf(mm, st[0][i]);
    ll = 0.0f;
    o = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float k = scale(st[0][i], mm);
        ll = __builtin_fmaf(st[1][i], k, ll);
        const f32x4 v = part[i][threadIdx.x];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(v[e], k, o[e]);
    }
    cache_attn_out<DT>(x, b, hk, row, d, max(x.lens[b], 0), o, mm, ll);
}

}  // namespace igc
