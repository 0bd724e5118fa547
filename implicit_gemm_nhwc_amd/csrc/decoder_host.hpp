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
// values a lane, threads a workgroup.
struct LnForm {
    int lanes, chunks, threads;
};
constexpr LnForm ln_form(int c) {
    if (c <= 64) return {8, 1, 256};
    if (c <= 128) return {16, 1, 256};
    if (c <= 256) return {32, 1, 256};
    if (c <= 512) return {64, 1, 256};
    if (c <= 1024) return {64, 2, 256};
    if (c <= 2048) return {64, 4, 256};
    if (c <= 4096) return {256, 2, 256};
    if (c <= 8192) return {256, 4, 256};
    return {512, 4, 512};
}

template <int DT>
hipError_t launch_layer_norm(const LnArgs& a, bool backward, hipStream_t stream);

constexpr int kQuantMaxChannels = 131071;

// Rows in 8 bits take the norm's forms; longer rows go through the last one in
// pieces.
template <int DT>
hipError_t launch_quantize_rows(const QuantArgs& a, hipStream_t stream);

// Form of the product: at most kFewRows rows of x, or square tiles.
constexpr int kFewRows = 64;
struct LinForm {
    int tile;         // 0: few rows
    int64_t tiles_m, tiles_n;
    int threads;
};

template <int DT>
hipError_t launch_linear_i8(const LinArgs& a, int tile, hipStream_t stream);

template <int DT>
hipError_t launch_kv_cache(const CacheArgs& a, bool write, hipStream_t stream);

// Workgroups of the attention over the cache that split launches aim at, a CU.
constexpr int kCacheFill = 2;
static_assert(kCacheFill * kNumCUs <= kCacheMostSlots, "unit sums fit 32 bits");

// groups: workgroups of the launch.
template <int DT>
hipError_t launch_cache_attn(const CacheAttnArgs& a, unsigned groups, hipStream_t stream);

}  // namespace igc
