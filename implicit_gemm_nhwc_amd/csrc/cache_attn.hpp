// Attention of a few new tokens over the paged cache in 8 bits.
//
// Rows are the Tq * G queries that share one key head, 32 a workgroup; its
// waves take blocks of 32 keys in turn.  With k_j = ks_j K_j and v_j = vs_j V_j
// (integers K, V):
//   s_j = (q . K_j) ks_j scale,  p_j = 2^(s_j log2 e - m),
//   out = sum (p_j vs_j) V_j / sum p_j
// so that the integers enter the matrix products as they are: 8 bits are exact
// in both 16-bit types, and the scales go to the scores and probabilities.
//
// Scores come as S^T = K Q^T (keys down the registers, one row a lane).  The
// result's register i of half h is row 8 (i / 4) + 4 h + i % 4; it is given key
// 16 (i / 8) + 8 h + i % 8 by reading the keys in that order, so that the 8
// probabilities of a product's k slots are 8 neighbouring keys: one transposing
// 8-bit read of the values and two reads of the scales.
//
// p vs is held as the sum of two bf16 numbers (16 bits of its own), which
// doubles the second products but leaves the outputs as accurate as fp32
// probabilities, for both types; the cache's bytes bound the kernel, not the
// matrix cores.
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
    int split;             // whether workgroups share a sequence (then a join follows)
};

constexpr int kCacheWaves = 8;
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

// Four values of a packed row's result, and the row's lse.
template <int DT>
__device__ __forceinline__ void cache_attn_out(const AttnArgs& a, int b, int hk, int row, int d,
                                               const f32x4& o, float m, float l) {
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);   // NaN stays NaN
    const int tok = div_g(a, row), g = row - tok * a.G;
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
    int64_t slot0;         // slot of part 0
};

// Division of the work, by whole waves: every wave forms it.
struct CacheDivision {
    int64_t chunk;
    __device__ __forceinline__ int len(const CacheAttnArgs& x, int b) const {
        return cache_len(x.lens[b], x.capacity);
    }
    __device__ __forceinline__ void init(const CacheAttnArgs& x, int lane) {
        int64_t total = 0;
        for (int b = lane; b < x.a.B; b += 64) total += cache_units(len(x, b));
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) total += __shfl_xor(total, o, 64);
        chunk = cache_chunk(total, x.slots, x.a.B);
    }
    // parts of sequence `b` and of those before it; returns the first
    // sequence whose parts reach past `slot` (in parts, not workgroups) when
    // b < 0
    __device__ __forceinline__ bool find(const CacheAttnArgs& x, int lane, int64_t w, int hr_n,
                                         int b, CachePlace* o) const {
        int64_t before = 0;
        for (int base = 0; base < x.a.B; base += 64) {
            const int mine = base + lane;
            const int n = mine < x.a.B ? len(x, mine) : 0;
            int64_t k = mine < x.a.B ? cache_parts(n, chunk) : 0, sum = k;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int64_t up = __shfl_up(sum, d, 64);
                if (lane >= d) sum += up;
            }
            const uint64_t here = b >= 0 ? (b >= base && b < base + 64 ? 1ull << (b - base) : 0)
                                         : __ballot(w < (before + sum) * hr_n && k > 0);
            if (here) {
                const int f = __builtin_ctzll(here);
                o->b = base + f;
                o->parts = (int)__shfl(k, f, 64);
                o->len = __shfl(n, f, 64);
                before += __shfl(sum, f, 64) - o->parts;
                o->slot0 = before * hr_n;
                return true;
            }
            before += __shfl(sum, 63, 64);
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

// Chunk c of row r of a tile of 8-bit rows at its place: 16-byte chunks turned
// by the row so that 8 rows of one chunk lie in different banks.
template <int DP>
__device__ __forceinline__ int tile8_off(int r, int c) {
    const int turn = DP == 128 ? r & 7 : DP == 64 ? (r >> 1) & 3 : 0;
    return r * DP + ((c ^ turn) << 4);
}

// Direct loads of 32 rows of both pools' integers and of the scales; a lane's
// place in LDS fixes its row and chunk.  Chunks past the row read its first
// one: the queries' zeros, or columns that are not stored, meet them.
template <int DP>
struct CacheStage {
    static constexpr int TILE = 32 * DP, PIECES = TILE / 1024;
    static constexpr int BYTES = 2 * TILE + 256;   // keys, values, their scales
    static constexpr int LOADS = 2 * PIECES + 1;
    int off[PIECES];
    bool high[PIECES];   // rows 16 .. 31

    __device__ __forceinline__ void init(int lane, int Dp) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int at = i * 1024 + lane * 16, r = at / DP;
            const int turn = DP == 128 ? r & 7 : DP == 64 ? (r >> 1) & 3 : 0;
            const int c = ((at % DP) >> 4) ^ turn;
            high[i] = r >= 16;
            off[i] = (r & 15) * Dp + (c * 16 < Dp ? c * 16 : 0);
        }
    }
    // rows r0 (the first 16 keys) and r1 of the pools
    __device__ __forceinline__ void issue(const CacheAttnArgs& x, int64_t r0, int64_t r1,
                                          int lane, uint8_t* lds) const {
        typedef __attribute__((address_space(1))) void* gp;
        typedef __attribute__((address_space(3))) void* lp;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int8_t* b0 = x.pool[t] + r0 * x.Dp;
            const int8_t* b1 = x.pool[t] + r1 * x.Dp;
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
                __builtin_amdgcn_global_load_lds((gp)((high[i] ? b1 : b0) + off[i]),
                                                 (lp)(lds + t * TILE + i * 1024), 16, 0, 0);
        }
        // lanes 0 .. 31 the keys' scales, the others the values'
        const float* s = (lane < 32 ? x.scales[0] : x.scales[1]) + ((lane & 16) ? r1 : r0);
        __builtin_amdgcn_global_load_lds((gp)(s + (lane & 15)), (lp)(lds + 2 * TILE), 4, 0, 0);
    }
};

template <int DT, int DP, int NW>
__global__ __launch_bounds__(NW * 64, 2) void cache_attn_kernel(CacheAttnArgs x) {
    const AttnArgs& a = x.a;
    constexpr int DB = DP / 32, KS = DP / 16;
    using Stage = CacheStage<DP>;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int half = lane >> 5;
    const int rows_tile = min(a.rows, 32);
    // a wave's two stages, which its results reuse
    constexpr int own = 2 * Stage::BYTES;
    static_assert(own >= 32 * DP * 4, "a wave's results fit its stages");
    lds_poison<NW * 64>(lds, NW * own + NW * 64 * 4);
    uint8_t* mine = lds + wave * own;
    float* st_m = reinterpret_cast<float*>(lds + NW * own);   // [NW][32] m, then l
    float* st_l = st_m + NW * 32;

    const int hr_n = a.Hk * a.row_tiles;
    CachePlace at;
    if (x.split) {
        CacheDivision div;
        div.init(x, lane);
        if (!div.find(x, lane, blockIdx.x, hr_n, -1, &at)) return;   // all waves
        const int r = (int)((int64_t)blockIdx.x - at.slot0);
        at.hr = r / at.parts;
        at.part = r - at.hr * at.parts;
        at.begin = at.part * div.chunk * kCacheUnit;
        at.end = at.begin + div.chunk * kCacheUnit;
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
    const int end = __builtin_amdgcn_readfirstlane((int)at.end);
    const int len = __builtin_amdgcn_readfirstlane(at.len);
    const int hk = hr / a.row_tiles, row0 = (hr - hk * a.row_tiles) * 32;
    const int row = row0 + (lane & 31), t0 = div_g(a, row0);

    // queries: k step 2 y + z, half h holds values 32 y + 16 h + 8 z .. + 7, as
    // the keys' 16-byte chunks do
    i32x4 qf[KS];
    {
        const __amdgpu_buffer_rsrc_t rs = attn_rsrc(
            a.q + (int64_t)b * a.q_b + (int64_t)hk * a.G * a.q_h + (int64_t)t0 * a.q_t);
        const unsigned off = packed_off(a, row, t0, a.q_t, a.q_h);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = 32 * (s >> 1) + 16 * half + 8 * (s & 1);
            qf[s] = __builtin_bit_cast(i32x4, load16(rs, d < a.D ? off + 2 * d : kOut));
        }
    }
    // this lane's row sees the keys before `last`
    int last = len;
    if (x.causal) last = len - (a.Tq - 1 - div_g(a, min(row, a.rows - 1)));
    f32x16 acc[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f;

    Stage stage;
    stage.init(lane, x.Dp);
    // scalar loads: a vector load's wait would be one for the stages in flight
    typedef __attribute__((address_space(4))) const int32_t* sp;
    const sp table = (sp)(x.table + b * x.table_stride);
    constexpr int STEP = NW * 32;
    // pages of the two halves of the block at j; keys at or past the end need none
    auto pages = [&](int j, int* id0, int* id1) {
        *id0 = j < end ? cache_page(table, j, x.shift, x.entries, x.pages) : 0;
        *id1 = j + 16 < end ? cache_page(table, j + 16, x.shift, x.entries, x.pages) : 0;
    };
    auto issue = [&](int j, int id0, int id1, uint8_t* to) {
        stage.issue(x, cache_row(id0 < 0 ? 0 : id0, a.Hk, hk, j, x.shift),
                    cache_row(id1 < 0 ? 0 : id1, a.Hk, hk, j + 16, x.shift), lane, to);
    };
    const int j0 = begin + wave * 32;
    int id0 = 0, id1 = 0, nx0 = 0, nx1 = 0;   // the block's pages, and the next one's
    if (j0 < end) {
        pages(j0, &id0, &id1);
        issue(j0, id0, id1, mine);
        if (j0 + STEP < end) {
            pages(j0 + STEP, &nx0, &nx1);
            issue(j0 + STEP, nx0, nx1, mine + Stage::BYTES);
        }
    }
    int buf = 0;
    for (int j = j0; j < end; j += STEP) {
        // this block: all but the next one's loads
        if (j + STEP < end) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(Stage::LOADS) : "memory");
        else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const uint8_t* kl = mine + buf * Stage::BYTES;
        const uint8_t* vl = kl + Stage::TILE;
        const float* sl = reinterpret_cast<const float*>(vl + Stage::TILE);
        f32x16 s;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 0.0f;
        // row l % 32 of the product is key 16 (l / 16) + 8 bit 2 + 4 bit 3 + l % 4
        const int key = (lane & 0x13) | ((lane & 4) << 1) | ((lane & 8) >> 1);
#pragma unroll
        for (int y = 0; y < DP / 32; ++y) {
            const u32x4 kb = *reinterpret_cast<const u32x4*>(kl + tile8_off<DP>(key, 2 * y + half));
            const i32x4 k0 = bytes_frag<DT>(kb[0], kb[1]), k1 = bytes_frag<DT>(kb[2], kb[3]);
            s = mfma32<DT>(&k0, &qf[2 * y], s);
            s = mfma32<DT>(&k1, &qf[2 * y + 1], s);
        }
        float ks[16], vs[16];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int at4 = 16 * (g >> 1) + 8 * half + 4 * (g & 1);
            const f32x4 u = *reinterpret_cast<const f32x4*>(sl + at4);
            const f32x4 w = *reinterpret_cast<const f32x4*>(sl + 32 + at4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ks[4 * g + i] = u[i];
                vs[4 * g + i] = w[i];
            }
        }
        if (id0 < 0 || id1 < 0) {   // no such page: its keys are NaN
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if ((i < 8 ? id0 : id1) < 0) ks[i] = vs[i] = __builtin_nanf("");
        }
        const int left = min(last, end) - j;
        const bool full = __all(left >= 32);
        float t = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] *= ks[i] * a.c;
        if (!full) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (16 * (i >> 3) + 8 * half + (i & 7) >= left) {
                    s[i] = -__builtin_inff();
                    vs[i] = 0.0f;   // may be anything there
                }
        }
#pragma unroll
        for (int i = 0; i < 16; i += 2) t = fmaxf(fmaxf(s[i], s[i + 1]), t);
        t = max_halves(t);
        if (__any(t > m + kCacheSlack)) {
            const float mn = fmaxf(m, t);
            // rows still without a key: 2^(-inf - 0) keeps everything 0
            const float f = mn == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[d][i] *= f;
        }
        const float ms = m == -__builtin_inff() ? 0.0f : m;
        float sum[4] = {0, 0, 0, 0};
        i32x4 hi[2], lo[2];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            float p[2], q[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                p[k] = __builtin_amdgcn_exp2f(s[i + k] - ms);
                sum[(i + k) & 3] += p[k];
                p[k] *= vs[i + k];
            }
            const uint32_t h = pack_out2(p[0], p[1], DT_BF16);
            q[0] = p[0] - __builtin_bit_cast(float, h << 16);
            q[1] = p[1] - __builtin_bit_cast(float, h & 0xffff0000u);
            hi[i >> 3][(i >> 1) & 3] = (int)h;
            lo[i >> 3][(i >> 1) & 3] = (int)pack_out2(q[0], q[1], DT_BF16);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        // values: lane i of 16 reads 8 bytes of row i / 2 and gets 8 rows of
        // column i
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                const int r = 16 * g + 8 * half + ((lane & 15) >> 1);
                const u32x2 vb = read_tr8(vl + tile8_off<DP>(r, 2 * d + ((lane >> 4) & 1)) +
                                          8 * (lane & 1));
                const i32x4 vf = bytes_frag<DT_BF16>(vb[0], vb[1]);
                acc[d] = mfma32<DT_BF16>(&vf, &hi[g], acc[d]);
                acc[d] = mfma32<DT_BF16>(&vf, &lo[g], acc[d]);
            }
        // the stage is read: the block after the next may arrive
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        id0 = nx0;
        id1 = nx1;
        if (j + 2 * STEP < end) {
            pages(j + 2 * STEP, &nx0, &nx1);
            issue(j + 2 * STEP, nx0, nx1, mine + buf * Stage::BYTES);
        }
        buf ^= 1;
    }
    // join of the waves: each wave's rows as floats [rows][DP] over its stages
    l = sum_halves(l);
    float* po = reinterpret_cast<float*>(mine);
    const int r32 = lane & 31;
    if (r32 < rows_tile) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<f32x4*>(po + r32 * DP + 32 * d + 8 * g + 4 * half) =
                    f32x4{acc[d][4 * g], acc[d][4 * g + 1], acc[d][4 * g + 2], acc[d][4 * g + 3]};
        if (half == 0) {
            st_m[wave * 32 + r32] = m;
            st_l[wave * 32 + r32] = l;
        }
    }
    __syncthreads();
    const int per = a.D / 4, n = min(32, a.rows - row0);
    for (int e = threadIdx.x; e < n * per; e += NW * 64) {
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
            const f32x4 v = *reinterpret_cast<const f32x4*>(
                reinterpret_cast<const float*>(lds + w * own) + r * DP + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(v[i], f, o[i]);
        }
        if (parts > 1) {
            const int64_t to = (int64_t)blockIdx.x * rows_tile + r;
            *reinterpret_cast<f32x4*>(a.part + to * a.D + d) = o;
            if (d == 0) {
                a.stat[to * 2] = mm;
                a.stat[to * 2 + 1] = ll;
            }
            continue;
        }
        cache_attn_out<DT>(a, b, hk, row0 + r, d, o, mm, ll);
    }
}

// Join of the parts of a sequence that several workgroups read: a workgroup a
// (sequence, key head, row tile), 32 lanes a row, 4 values a lane, parts in
// order.
template <int DT>
__global__ __launch_bounds__(256) void cache_attn_join_kernel(CacheAttnArgs x) {
    const AttnArgs& a = x.a;
    const int lane = threadIdx.x & 63;
    const int hr_n = a.Hk * a.row_tiles, b = blockIdx.x / hr_n, hr = blockIdx.x - b * hr_n;
    CacheDivision div;
    div.init(x, lane);
    CachePlace at;
    div.find(x, lane, 0, hr_n, b, &at);
    if (at.parts <= 1) return;   // written where it was read
    const int hk = hr / a.row_tiles, row0 = (hr - hk * a.row_tiles) * 32;
    const int rows_tile = min(a.rows, 32), n = min(32, a.rows - row0);
    const int64_t slot = at.slot0 + (int64_t)hr * at.parts;
    const int d = (threadIdx.x & 31) * 4;
    for (int r = threadIdx.x >> 5; r < n; r += 8) {
        float mm = -__builtin_inff();
        for (int s = threadIdx.x & 31; s < at.parts; s += 32)
            mm = fmaxf(mm, a.stat[((slot + s) * rows_tile + r) * 2]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) mm = fmaxf(mm, __shfl_xor(mm, o, 64));
        const float ms = mm == -__builtin_inff() ? 0.0f : mm;
        float ll = 0.0f;
        f32x4 o = {0, 0, 0, 0};
        for (int s = 0; s < at.parts; ++s) {
            const int64_t from = (slot + s) * rows_tile + r;
            const float f = __builtin_amdgcn_exp2f(a.stat[from * 2] - ms);
            ll = __builtin_fmaf(a.stat[from * 2 + 1], f, ll);
            if (d < a.D) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(a.part + from * a.D + d);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(v[i], f, o[i]);
            }
        }
        if (d < a.D) cache_attn_out<DT>(a, b, hk, row0 + r, d, o, mm, ll);
    }
}

}  // namespace igc
