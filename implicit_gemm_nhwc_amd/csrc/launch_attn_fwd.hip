// Launchers of the cross-attention forward kernels, one element type per
// translation unit (IGC_DT).
#include "attn_host.hpp"
#include "attn_short.hpp"

#ifndef IGC_DT
#error "IGC_DT must name the element type of this translation unit"
#endif

namespace igc {
namespace {

template <int DT, int DP, bool MASK>
hipError_t launch_rows(const AttnArgs& a, hipStream_t stream) {
    auto kern = attn_fwd_kernel<DT, DP, kAttnWaves, MASK>;
    constexpr size_t lds = 4 * (size_t)kKeyTile * DP * 2 + 2 * kKeyTile * 4;
    static LdsAttr attr;
    const hipError_t e = ensure_lds(attr, (const void*)kern, lds);
    if (e != hipSuccess) return e;
    const unsigned grid = (unsigned)((int64_t)a.B * a.Hk * a.nsplit * a.row_tiles);
    hipLaunchKernelGGL(kern, dim3(grid), dim3(kAttnWaves * 64), lds, stream, a);
    return hipGetLastError();
}

template <int DT, int DP>
hipError_t launch_short(const AttnArgs& a, hipStream_t stream) {
    auto kern = attn_short_fwd_kernel<DT, DP, kAttnWaves>;
    constexpr size_t lds = short_lds<DP>();
    static LdsAttr attr;
    const hipError_t e = ensure_lds(attr, (const void*)kern, lds);
    if (e != hipSuccess) return e;
    const unsigned grid = (unsigned)((int64_t)a.B * a.Hk * a.row_tiles);
    hipLaunchKernelGGL(kern, dim3(grid), dim3(kAttnWaves * 64), lds, stream, a);
    return hipGetLastError();
}

template <int DT, int DP>
hipError_t launch_token(const AttnArgs& a, hipStream_t stream) {
    auto kern = attn_token_kernel<DT, DP, kTokenWaves>;
    constexpr size_t lds = (size_t)kTokenWaves * (2 * 32 * DP * 2 + 64 * 4);
    static LdsAttr attr;
    const hipError_t e = ensure_lds(attr, (const void*)kern, lds);
    if (e != hipSuccess) return e;
    const unsigned grid = (unsigned)((int64_t)a.B * a.Hk * a.nsplit);
    hipLaunchKernelGGL(kern, dim3(grid), dim3(kTokenWaves * 64), lds, stream, a);
    return hipGetLastError();
}

template <int DT, int DP>
hipError_t launch_dp(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
    hipError_t e;
    if (p.token) e = launch_token<DT, DP>(a, stream);
    else if (p.few_keys) e = launch_short<DT, DP>(a, stream);
    else if (a.mask) e = launch_rows<DT, DP, true>(a, stream);
    else e = launch_rows<DT, DP, false>(a, stream);
    if (e != hipSuccess || a.nsplit <= 1) return e;
    const int64_t n = (int64_t)a.B * a.Hk * a.rows;
    if (a.nsplit <= kJoinFew)
        hipLaunchKernelGGL((attn_join_kernel<DT, 1>), dim3((unsigned)((n + 7) / 8)), dim3(256), 0,
                           stream, a);
    else
        hipLaunchKernelGGL((attn_join_kernel<DT, 8>), dim3((unsigned)n), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

template <int DT>
hipError_t launch_attn_fwd(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
    switch (padded_dim(a.D)) {
        case 32: return launch_dp<DT, 32>(a, p, stream);
        case 64: return launch_dp<DT, 64>(a, p, stream);
        case 96: return launch_dp<DT, 96>(a, p, stream);
        default: return launch_dp<DT, 128>(a, p, stream);
    }
}

template hipError_t launch_attn_fwd<IGC_DT>(const AttnArgs&, const AttnPlan&, hipStream_t);

}  // namespace igc
