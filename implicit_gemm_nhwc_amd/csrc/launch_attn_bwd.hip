// Launchers of the cross-attention backward kernels, one element type per
// translation unit (IGC_DT).
#include "attn_host.hpp"
#include "attn_short.hpp"

#ifndef IGC_DT
#error "IGC_DT must name the element type of this translation unit"
#endif

namespace igc {
namespace {

template <int DT, int DP, int NWK, int RG, int QT, bool KV_LDS, int OCC>
hipError_t launch_kv(AttnArgs a, const AttnGradPlan& p, hipStream_t stream) {
    auto kern = attn_bwd_kv_kernel<DT, DP, NWK, RG, QT, KV_LDS, OCC>;
    constexpr size_t lds = KvShape<DP, NWK, RG, QT, KV_LDS>::LDS;
    constexpr int NW = NWK * RG;
    static LdsAttr attr;
    hipError_t e = ensure_lds(attr, (const void*)kern, lds);
    if (e != hipSuccess) return e;
    a.key_tiles = p.key_tiles;
    a.nsplit = p.kv_nsplit;
    a.split = p.kv_split;
    const int64_t bh = (int64_t)a.B * a.Hk;
    hipLaunchKernelGGL(kern, dim3((unsigned)(bh * a.nsplit * a.key_tiles)), dim3(NW * 64), lds,
                       stream, a);
    e = hipGetLastError();
    if (e != hipSuccess || a.nsplit <= 1) return e;
    hipLaunchKernelGGL(attn_bwd_join_kernel<DT>,
                       dim3((unsigned)((bh * a.Tk * (a.D / 4) + 255) / 256), 2), dim3(256), 0,
                       stream, a, 1);
    return hipGetLastError();
}

// Two waves a SIMD.  Up to 96 values a head the keys' operands stay in
// registers (32 x 77 keys of 64, 784 rows: 21.5 us, from LDS 24.2); 128 do not
// fit two waves that way and are read from LDS (2 x 2048 keys, 8192 rows:
// 275 us; in registers with one wave a SIMD 375, spilling 467).
template <int DT, int DP, int NWK>
hipError_t launch_kv_dp(const AttnArgs& a, const AttnGradPlan& p, hipStream_t stream) {
    if constexpr (DP <= 96) {
        if (p.kv_groups == 1) return launch_kv<DT, DP, NWK, 1, kRowTile, false, 2>(a, p, stream);
        return launch_kv<DT, DP, NWK, 2, kRowTile, false, 2>(a, p, stream);
    } else {
        return launch_kv<DT, DP, NWK, 2, kRowTile, true, 2>(a, p, stream);
    }
}

template <int DT, int DP>
hipError_t launch_q(AttnArgs a, const AttnGradPlan& p, hipStream_t stream) {
    auto kern = attn_bwd_q_kernel<DT, DP, kAttnWaves>;
    constexpr size_t lds = 4 * (size_t)kKeyTile * DP * 2;
    static LdsAttr attr;
    hipError_t e = ensure_lds(attr, (const void*)kern, lds);
    if (e != hipSuccess) return e;
    a.row_tiles = p.row_tiles;
    a.nsplit = p.q_nsplit;
    a.split = p.q_split;
    const int64_t bh = (int64_t)a.B * a.Hk;
    hipLaunchKernelGGL(kern, dim3((unsigned)(bh * a.nsplit * a.row_tiles)), dim3(kAttnWaves * 64),
                       lds, stream, a);
    e = hipGetLastError();
    if (e != hipSuccess || a.nsplit <= 1) return e;
    hipLaunchKernelGGL(attn_bwd_join_kernel<DT>,
                       dim3((unsigned)((bh * a.rows * (a.D / 4) + 255) / 256), 1), dim3(256), 0,
                       stream, a, 0);
    return hipGetLastError();
}

template <int DT, int DP>
hipError_t launch_short(AttnArgs a, const AttnGradPlan& p, hipStream_t stream) {
    auto kern = attn_short_rows_kernel<DT, DP, kAttnWaves>;
    constexpr size_t lds = short_lds<DP>();
    static LdsAttr attr;
    const hipError_t e = ensure_lds(attr, (const void*)kern, lds);
    if (e != hipSuccess) return e;
    a.row_tiles = p.row_tiles;
    hipLaunchKernelGGL(kern, dim3((unsigned)((int64_t)a.B * a.Hk * a.row_tiles)),
                       dim3(kAttnWaves * 64), lds, stream, a);
    return hipGetLastError();
}

template <int DT, int DP>
hipError_t launch_dp(const AttnArgs& a, const AttnGradPlan& p, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a.rows > 0) {
        if (p.few_keys) {
            e = launch_short<DT, DP>(a, p, stream);
        } else {
            hipLaunchKernelGGL(attn_bwd_rows_kernel<DT>,
                               dim3((unsigned)((int64_t)a.B * a.Hk * a.bound_n)), dim3(256), 0,
                               stream, a);
            e = hipGetLastError();
        }
    }
    if (e == hipSuccess && a.Tk > 0 && a.dk) {
        switch (p.kv_waves) {
            case 1: e = launch_kv_dp<DT, DP, 1>(a, p, stream); break;
            case 2: e = launch_kv_dp<DT, DP, 2>(a, p, stream); break;
            case 3: e = launch_kv_dp<DT, DP, 3>(a, p, stream); break;
            default: e = launch_kv_dp<DT, DP, 4>(a, p, stream); break;
        }
    }
    if (e == hipSuccess && a.rows > 0 && a.dq && !p.few_keys) e = launch_q<DT, DP>(a, p, stream);
    return e;
}

}  // namespace

template <int DT>
hipError_t launch_attn_bwd(const AttnArgs& a, const AttnGradPlan& p, hipStream_t stream) {
    switch (padded_dim(a.D)) {
        case 32: return launch_dp<DT, 32>(a, p, stream);
        case 64: return launch_dp<DT, 64>(a, p, stream);
        case 96: return launch_dp<DT, 96>(a, p, stream);
        default: return launch_dp<DT, 128>(a, p, stream);
    }
}

template hipError_t launch_attn_bwd<IGC_DT>(const AttnArgs&, const AttnGradPlan&, hipStream_t);

}  // namespace igc
