// Pieces shared by the attention kernels: argument block, tile staging, the
// MFMA operand layouts and the mask words.
//
// All of them work on blocks of 32 rows x 32 keys through
// v_mfma_f32_32x32x16 (bf16 / fp16): lane l supplies row (A) or column (B)
// l % 32 with 8 consecutive k at 8 * (l / 32); the result has column l % 32
// and, in register i, row 8 * (i / 4) + 4 * (l / 32) + i % 4.  A result
// therefore becomes the B operand of a following product without leaving its
// lane when that product numbers its k axis by the result's rows: k slot
// (half h, j) of a step of 16 is row 8 * (j / 4) + 4 * h + j % 4.  The other
// operand follows that numbering through transposing LDS reads
// (ds_read_b64_tr_b16: each lane gets 4 consecutive rows of one column).
#pragma once

#include "attn_split.hpp"
#include "igemm_kernels.hpp"

namespace igc {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

struct AttnArgs {
    const uint8_t *q, *k, *v, *o, *dout;
    uint8_t *out, *dq, *dk, *dv;
    float* lse;            // [B][Hq][Tq]
    const int32_t* lens;
    const uint8_t* mask;
    float* part;           // partial results of split launches
    float* stat;           // their (m, l); backward: [2][B][Hk][rows_pad], lse in powers of two
                           // and -Delta
    uint32_t* bound;       // backward, fp16: [B][Hk][bound_n] squared maxima of do and v, as
                           // float bits
    // strides in bytes
    int64_t q_b, q_t, q_h, k_b, k_t, k_h, v_b, v_t, v_h, o_b, o_t, o_h;
    int64_t do_b, do_t, do_h, dq_b, dq_t, dq_h, dk_b, dk_t, dk_h, dv_b, dv_t, dv_h;
    int64_t mask_b;
    int B, Tq, Tk, Hq, Hk, G, D;
    int rows;       // Tq * G: the queries that share one key head
    int rows_pad;   // backward: rows rounded up to whole row tiles
    int bound_n;    // backward: workgroups a (batch, key head) of the row pass
    int row_tiles;  // workgroups along the rows
    int key_tiles;  // backward: workgroups along the keys
    int nsplit;     // workgroups that share a tile's keys (backward dk / dv: its rows)
    int split;      // keys (rows) per split, a multiple of the key (row) tile
    float c;        // scale * log2(e): p = 2^(c s - c m)
    float scale;
    uint32_t g_mul; // row / G = mulhi(row, g_mul) >> g_shift, g_mul = 0 for G = 1
    int g_shift;
};

// row / G by the host's multiplier (exact for row < 2^31).
__device__ __forceinline__ int div_g(const AttnArgs& a, int row) {
    const int q = (int)(__umulhi((uint32_t)row, a.g_mul) >> a.g_shift);
    return a.g_mul ? q : row;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t attn_rsrc(const void* base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, 0x7fffffff,
                                             0x00020000);
}
// A buffer offset past the range: loads return zero, stores are dropped.
// Every masked access of the kernels with matrix products goes this way while
// their accumulators are needed further, by selecting the offset, and none by
// a branch on the lane: they fill the register file, and where a value is
// moved to an accumulation register at the join of such a branch the compiler
// was seen to put the copy before the execution mask is restored, which loses
// the other lanes' values.  (The single-token kernel's accumulators end in the
// branch that stores them; the joins of split launches and the row pass of the
// backward hold none; the compiler makes small lane branches of its own, such
// as around a division.  tests/test_attn_assembly.py reads the built code for
// such copies.)
constexpr unsigned kOut = 0x80000000u;

__device__ __forceinline__ u32x4 load16(const __amdgpu_buffer_rsrc_t& rs, unsigned off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
}
__device__ __forceinline__ float load4(const __amdgpu_buffer_rsrc_t& rs, unsigned off) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0));
}
__device__ __forceinline__ void store16(const __amdgpu_buffer_rsrc_t& rs, unsigned off, u32x4 v) {
    typedef decltype(__builtin_amdgcn_raw_buffer_load_b128(rs, 0, 0, 0)) V;
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(V, v), rs, off, 0, 0);
}
__device__ __forceinline__ void store4(const __amdgpu_buffer_rsrc_t& rs, unsigned off, float v) {
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), rs, off, 0, 0);
}

// Row `row` of the packed queries: byte offset of its (token, head) from
// token t0 and the first head of the group; rows past the last get kOut.
__device__ __forceinline__ unsigned packed_off(const AttnArgs& a, int row, int t0, int64_t st,
                                               int64_t sh) {
    const int tok = div_g(a, row);
    const unsigned off = (unsigned)(tok - t0) * (unsigned)st +
                         (unsigned)(row - tok * a.G) * (unsigned)sh;
    return row < a.rows ? off : kOut;
}

// This workgroup's place in the launch order.  Workgroups that share a key
// head follow one another there, and where all heads cost the same each XCD
// takes one run of them, so that its L2 holds few heads' keys (16384 rows x
// 4096 keys of 128, 32 heads).  With ragged lengths a run of long heads would
// leave the other XCDs idle: the hardware's round-robin order then deals
// every head's workgroups to all of them (4 x 3136 x 1333 ragged: 115 -> 73 us, the
// masked tiles' cheaper start included).
__device__ __forceinline__ int launch_place(const AttnArgs& a) {
    return a.lens || a.mask ? (int)blockIdx.x : xcd_remap(blockIdx.x, gridDim.x);
}

// lse entry of a packed row of key head hk, from lse_base.
__device__ __forceinline__ unsigned lse_off(const AttnArgs& a, int row) {
    const int tok = div_g(a, row);
    return row < a.rows ? (unsigned)((row - tok * a.G) * a.Tq + tok) * 4 : kOut;
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t lse_base(const AttnArgs& a, int b, int hk) {
    return attn_rsrc(a.lse + ((int64_t)b * a.Hq + hk * a.G) * a.Tq);
}

// LDS tiles hold rows of DP elements (DP = D rounded up to 32), the 16-byte
// chunk c of row r at c ^ lds_swz(r).  Two patterns read them: whole chunks
// of 16 consecutive rows (ds_read_b128), and 64 adjacent bytes of 4
// consecutive rows (the transposing read).  The low two chunk bits turn with
// r / 4, and the bits above with what of r % 4 the row pitch does not spread
// over the 256 bytes of banks by itself, so that both patterns reach
// different banks.
template <int DP>
__device__ __forceinline__ int lds_swz(int r) {
    const int lo = (r >> 2) & 3;
    if constexpr (DP == 128) return ((r & 3) << 2) | lo;
    if constexpr (DP == 64) return (((r >> 1) & 1) << 2) | lo;
    return lo;   // 32: pitch 64; 96: pitch 192
}

// Byte offset of chunk c of row r.
template <int DP>
__device__ __forceinline__ int tile_off(int r, int c) {
    return r * (DP * 2) + ((c ^ lds_swz<DP>(r)) << 4);
}

// Operand of 8 consecutive k of one row (chunk c of row r): plain read.
template <int DP>
__device__ __forceinline__ i32x4 frag_row(const uint8_t* lds, int r, int c) {
    return *reinterpret_cast<const i32x4*>(lds + tile_off<DP>(r, c));
}

// One transposing read.  The pointer is restrict only for its side effect:
// inlining then leaves alias metadata on the read, without which the compiler
// makes it wait for every direct load to LDS in flight, the next tile's among
// them.  The kernels order those loads by their own waits and barriers.
__device__ __forceinline__ u32x2 read_tr(const uint8_t* __restrict__ p) {
    typedef __attribute__((address_space(3))) s16x4* lp;
    typedef __attribute__((address_space(3))) const uint8_t* bp;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(bp)p));
}

// Operand whose row / column is column 32 * db + l % 32 of the tile and whose
// k slots are the tile's rows r0 + 8 * (j / 4) + 4 * h + j % 4, by transposing
// reads: their 16 lanes address 4 rows x 32 bytes, lane i row i / 4, bytes
// 8 * (i % 4).
template <int DP>
__device__ __forceinline__ i32x4 frag_col(const uint8_t* lds, int r0, int db, int lane) {
    const int r = r0 + 4 * (lane >> 5) + ((lane & 15) >> 2);
    const int c = 4 * db + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const int b = (lane & 1) * 8;
    const u32x2 x = read_tr(lds + tile_off<DP>(r, c) + b);
    const u32x2 y = read_tr(lds + tile_off<DP>(r + 8, c) + b);
    return i32x4{(int)x[0], (int)x[1], (int)y[0], (int)y[1]};
}

// Bit j of the result: key j0 + j is valid.  mb is the mask byte of key
// j0 + lane (any nonzero value without a mask); keys at or past `end` are not.
__device__ __forceinline__ uint64_t mask_word(uint32_t mb, int left) {
    const uint64_t w = __ballot(mb != 0);
    return left >= 64 ? w : left <= 0 ? 0 : w & (~0ull >> (64 - left));
}

// Mask byte of key j0 + lane for mask_word; reads only keys before `end`.
__device__ __forceinline__ uint32_t mask_byte(const uint8_t* row, int j0, int end, int lane) {
    if (!row) return 1;
    return __builtin_amdgcn_raw_buffer_load_b8(attn_rsrc(row + j0),
                                               lane < end - j0 ? (unsigned)lane : kOut, 0, 0);
}

// Direct loads of a tile of ROWS rows into LDS by NW waves: each wave writes
// 1 KB pieces (64 lanes x 16 bytes in LDS order), so a lane's LDS place fixes
// its row and, through the swizzle, the chunk it has to fetch.  Lanes whose
// chunk is past D or whose row is not to be read get an offset out of range,
// which stores zeros.  The offsets are the same for every tile, formed once.
template <int DP, int ROWS, int NW>
struct TileStage {
    static constexpr int PIECES = ROWS * DP * 2 / 1024;
    static constexpr int PER = (PIECES + NW - 1) / NW;
    static constexpr bool EVEN = PIECES % NW == 0;
    int row[PER];
    unsigned off[PER];

    // first byte of the lane's chunk in its row, kOut for a chunk past D
    __device__ __forceinline__ unsigned place(int i, int wave, int lane, int D) {
        const int p = ((i * NW + wave) * 1024 + lane * 16);
        row[i] = p / (DP * 2);
        const int c = ((p % (DP * 2)) >> 4) ^ lds_swz<DP>(row[i]);
        return c * 8 < D ? (unsigned)c * 16 : kOut;
    }
    // rows of `pitch` bytes
    __device__ __forceinline__ void init(int wave, int lane, int D, unsigned pitch) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const unsigned c = place(i, wave, lane, D);
            off[i] = c == kOut ? kOut : c + (unsigned)row[i] * pitch;
        }
    }
    // packed rows of a tile that starts with a group's first head
    __device__ __forceinline__ void init_packed(const AttnArgs& a, int wave, int lane, int64_t pt,
                                                int64_t ph) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const unsigned c = place(i, wave, lane, a.D);
            const int tok = div_g(a, row[i]);
            const unsigned at = (unsigned)tok * (unsigned)pt +
                                (unsigned)(row[i] - tok * a.G) * (unsigned)ph + c;
            off[i] = c == kOut ? kOut : at;
        }
    }
    __device__ __forceinline__ void load(const __amdgpu_buffer_rsrc_t& rs, int i, unsigned at,
                                         uint8_t* lds, int wave) const {
        if (!EVEN && i * NW + wave >= PIECES) return;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (__attribute__((address_space(3))) void*)(lds + (i * NW + wave) * 1024), 16, at, 0,
            0, 0);
    }
    // bit r of `valid` says row r is read
    __device__ __forceinline__ void issue(const uint8_t* base, uint64_t valid, uint8_t* lds,
                                          int wave) const {
        const __amdgpu_buffer_rsrc_t rs = attn_rsrc(base);
        constexpr uint64_t all = ~0ull >> (64 - ROWS);
        if (valid == all) {
#pragma unroll
            for (int i = 0; i < PER; ++i) load(rs, i, off[i], lds, wave);
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                load(rs, i, (valid >> row[i]) & 1 ? off[i] : kOut, lds, wave);
        }
    }
    // the first n rows
    __device__ __forceinline__ void issue_first(const uint8_t* base, int n, uint8_t* lds,
                                                int wave) const {
        const __amdgpu_buffer_rsrc_t rs = attn_rsrc(base);
#pragma unroll
        for (int i = 0; i < PER; ++i) load(rs, i, row[i] < n ? off[i] : kOut, lds, wave);
    }
};

// P (or ds) of 16 result registers as the two B operands of 16 rows each.  This
// is where they are rounded to 16 bits, which the matrix cores' operands have
// (products of fp32 operands run at a sixteenth of the rate).  Statistics and
// sums were taken in fp32 before, so a result moves by at most half a step of
// the type times the sum of the magnitudes behind it, no more than its own
// rounding; the error against 64 bits grows by 26 to 43 % over fp32
// probabilities (bf16 0.0017 to 0.0021 .. 0.0024 relative, fp16 0.00021 to
// 0.00027 .. 0.00029).
template <int DT>
__device__ __forceinline__ void pack_frag(const float* p, i32x4* f) {
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            f[g][j] = (int)pack_out2(p[8 * g + 2 * j], p[8 * g + 2 * j + 1], DT);
}

// 8 stored values as floats and back (one rounding).
template <int DT>
__device__ __forceinline__ void unpack8(const u32x4& u, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = out_to_f32((uint16_t)(u[i] & 0xffff), DT);
        f[2 * i + 1] = out_to_f32((uint16_t)(u[i] >> 16), DT);
    }
}
template <int DT>
__device__ __forceinline__ u32x4 pack8(const float* f) {
    return u32x4{pack_out2(f[0], f[1], DT), pack_out2(f[2], f[3], DT), pack_out2(f[4], f[5], DT),
                 pack_out2(f[6], f[7], DT)};
}

// Maximum and sum over a lane and the one 32 away.
__device__ __forceinline__ void both_halves(float x, float* lo, float* hi) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t r0 = r[0], r1 = r[1];   // a bit cast of r[1] itself would read r[0]
    *lo = __builtin_bit_cast(float, r0);
    *hi = __builtin_bit_cast(float, r1);
}
__device__ __forceinline__ float max_halves(float x) {
    float a, b;
    both_halves(x, &a, &b);
    return fmaxf(a, b);
}
__device__ __forceinline__ float sum_halves(float x) {
    float a, b;
    both_halves(x, &a, &b);
    return a + b;
}

// Store of a result block whose columns are tensor rows and whose rows are
// 32 values of the head axis: register 4 g + i of half h is value
// 8 g + 4 h + i.  After exchanging halves each lane holds 8 adjacent values:
// half h takes the groups g = h and 2 + h.  off is the lane's row (kOut: no
// store), d0 the block's first value, values at or past D are not stored.
template <int DT>
__device__ __forceinline__ void store_block(const __amdgpu_buffer_rsrc_t& rs, unsigned off,
                                            const f32x16& v, float f, int d0, int D, int half) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_out2(v[2 * i] * f, v[2 * i + 1] * f, DT);
#pragma unroll
    for (int gg = 0; gg < 2; ++gg) {
        // groups 2 gg (words 4 gg, 4 gg + 1) and 2 gg + 1 (words 4 gg + 2, + 3)
        const auto a = __builtin_amdgcn_permlane32_swap(w[4 * gg], w[4 * gg + 2], false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(w[4 * gg + 1], w[4 * gg + 3], false, false);
        const int d = d0 + 16 * gg + 8 * half;
        store16(rs, d < D ? off + 2 * d : kOut, u32x4{a[0], b[0], a[1], b[1]});
    }
}

// The same block as fp32 values (partial sums of split launches).
__device__ __forceinline__ void store_part(const __amdgpu_buffer_rsrc_t& rs, unsigned off,
                                           const f32x16& v, float f, int d0, int D, int half) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int d = d0 + 8 * g + 4 * half;
        store16(rs, d < D ? off + 4 * d : kOut,
                __builtin_bit_cast(u32x4, f32x4{v[4 * g] * f, v[4 * g + 1] * f, v[4 * g + 2] * f,
                                                v[4 * g + 3] * f}));
    }
}

// A block of 32 rows as operands, one row a lane: `off` the lane's row (kOut:
// zeros); values past D are zero.
template <int DP>
__device__ __forceinline__ void load_rows(const __amdgpu_buffer_rsrc_t& rs, unsigned off, int D,
                                          int half, i32x4 (&f)[DP / 16]) {
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
        const int d = 16 * s + 8 * half;
        f[s] = __builtin_bit_cast(i32x4, load16(rs, d < D ? off + 2 * d : kOut));
    }
}

}  // namespace igc
