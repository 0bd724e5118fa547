// Host-side pieces of the decoder block's operators shared by their
// translation units: per-type launchers and the rules that pick a kernel form.
#pragma once

#include "attn_host.hpp"
#include "cache_attn.hpp"
#include "igemm_host.hpp"
#include "kv_cache.hpp"
#include "layer_norm.hpp"
#include "linear_i8.hpp"
#include "rows_i8.hpp"

namespace igc {

constexpr int kLnMaxChannels = 16384;

// Form of the layer norm kernels for C channels: lanes a row, chunks of 8
// values a lane, threads a workgroup.  Two or three chunks a lane leave the
// fewest lanes without work (154 MB: 54 to 58 us forward and 92 to 96 backward
// wherever the row fills them; 768 channels on 32 lanes x 3 58 and 95, on 64 x 2
// 73 and 103; 512 on 32 x 2 54 and 94, on 64 x 1 62 and 109, on 16 x 4 58 and
// 104).  Past 2048 channels a workgroup takes a row (4096: 65 and 100; 8192: 65
// and 100, on 256 x 4 76 and 111; 16384: 71 and 116).
struct LnForm {
    int lanes, chunks, threads;
};
constexpr LnForm ln_form(int c) {
    if (c <= 64) return {8, 1, 256};
    if (c <= 2048) {
        int lanes = 8;
        while (lanes * 16 < c) lanes *= 2;   // two chunks a lane
        if (lanes > 8 && lanes * 12 >= c) return {lanes / 2, 3, 256};
        return lanes > 64 ? LnForm{64, 4, 256} : LnForm{lanes, 2, 256};
    }
    if (c <= 4096) return {256, 2, 256};
    if (c <= 6144) return {256, 3, 256};
    if (c <= 8192) return {512, 2, 512};
    return c <= 12288 ? LnForm{512, 3, 512} : LnForm{512, 4, 512};
}
// What ln_form returns.
#define IGC_LN_FORMS(F) \
    F(8, 1, 256) F(8, 2, 256) F(8, 3, 256) F(16, 2, 256) \
    F(16, 3, 256) F(32, 2, 256) F(32, 3, 256) F(64, 2, 256) \
    F(64, 3, 256) F(64, 4, 256) F(256, 2, 256) \
    F(256, 3, 256) F(512, 2, 512) F(512, 3, 512) F(512, 4, 512)

// Workgroups a CU of the backward pass, as the registers allow: with four
// chunks (three on many lanes) two (2048 channels: 96 us, three 109; 1536: 92
// and 97; 320 on 16 x 3 101 and 95), with a row a workgroup two of 256 threads
// (4096: 100, three 108) or one of 512 (8192: 100, two 117).
constexpr int ln_bwd_fill(const LnForm& f) {
    if (f.lanes > 64) return f.lanes == 256 ? 2 : 1;
    return f.chunks == 4 || (f.chunks == 3 && f.lanes >= 32) ? 2 : 3;
}

template <int DT>
hipError_t launch_layer_norm(const LnArgs& a, bool backward, hipStream_t stream);

constexpr int kQuantMaxChannels = 131071;

// Rows in 8 bits take the norm's forms; longer rows go through the last one in
// pieces.
template <int DT>
hipError_t launch_quantize_rows(const QuantArgs& a, hipStream_t stream);

// Form of the product: at most kFewRows rows of x, or square tiles.
constexpr int kFewRows = 32;
struct LinForm {
    int tile;         // 0: few rows
    int64_t tiles_m, tiles_n;
    int threads;
};

template <int DT>
hipError_t launch_linear_i8(const LinArgs& a, int tile, hipStream_t stream);

template <int DT>
hipError_t launch_kv_cache(const CacheArgs& a, bool write, hipStream_t stream);

static_assert(2 * kNumCUs <= kCacheMostSlots, "unit sums of split sequences fit 32 bits");

// groups: workgroups of the launch.
template <int DT>
hipError_t launch_cache_attn(const CacheAttnArgs& a, unsigned groups, hipStream_t stream);

}  // namespace igc
