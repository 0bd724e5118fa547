// Host-side pieces of the attention operators shared by their translation
// units: launch plans and per-type launchers.
#pragma once

#include "attn_common.hpp"
#include "igemm_host.hpp"
#include "qk_norm.hpp"

namespace igc {

// Plan of one forward launch (fwd_plan in igemm_attn.hip).
struct AttnPlan {
    bool token;       // at most 32 rows a key head: attn_token_kernel
    bool few_keys;    // at most kShortKeys keys: attn_short_fwd_kernel
    int row_tiles, nsplit, split;
    int64_t part_floats, stat_floats;   // workspace of split launches
};

// Plan of a backward pass (bwd_plan in igemm_attn.hip).
struct AttnGradPlan {
    bool few_keys;        // at most kShortKeys keys: attn_short_rows_kernel instead of
                          // the row pass and the dq kernel
    int rows_pad, bound_n;
    int kv_waves;         // dk dv: key blocks (32 keys) a workgroup,
    int kv_groups;        // and waves a block, which take alternate row blocks
    int key_tiles, kv_nsplit, kv_split;   // dk dv: key tiles, splits of the rows
    int row_tiles, q_nsplit, q_split;     // dq: row tiles, splits of the keys
    int64_t stat_floats, bound_words, part_floats;   // workspace
};

constexpr int kAttnWaves = 4;     // waves a workgroup
constexpr int kShortKeys = 128;   // keys that the few-keys kernels hold in LDS
constexpr int kRowTile = 64;      // rows a tile of the dk dv kernel; padding of row statistics
constexpr int kKeyTile = 64;      // keys a tile of the forward kernel
constexpr int kTokenWaves = 8;    // waves a workgroup of the single-token kernel
constexpr int kTokenStep = 32 * kTokenWaves;   // keys a round of its waves

// D rounded up to the tile widths the kernels are built for.
inline int padded_dim(int d) { return d <= 32 ? 32 : d <= 64 ? 64 : d <= 96 ? 96 : 128; }

template <int DT>
hipError_t launch_attn_fwd(const AttnArgs& a, const AttnPlan& p, hipStream_t stream);
template <int DT>
hipError_t launch_attn_bwd(const AttnArgs& a, const AttnGradPlan& p, hipStream_t stream);

// Lanes a row of the norm kernels: chunks of 8 values, rounded up to a power
// of two, at least 4.
inline int qk_lanes(int d) { return d <= 32 ? 4 : d <= 64 ? 8 : 16; }

template <int DT>
hipError_t launch_qk_norm(const QkArgs& a, int mode, bool backward, hipStream_t stream);

}  // namespace igc
