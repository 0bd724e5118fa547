// Launchers of the per-head norm and rotation kernels, one element type per
// translation unit (IGC_DT).
#include "attn_host.hpp"
#include "qk_norm.hpp"

#ifndef IGC_DT
#error "IGC_DT must name the element type of this translation unit"
#endif

namespace igc {
namespace {

template <int DT, int LPR, int MODE>
hipError_t launch(const QkArgs& a, bool backward, hipStream_t stream) {
    const unsigned grid = (unsigned)(a.part[0].blocks + a.part[1].blocks);
    if (grid == 0) return hipSuccess;
    if (!backward) {
        hipLaunchKernelGGL((qk_norm_fwd_kernel<DT, LPR, MODE>), dim3(grid), dim3(kQkThreads), 0,
                           stream, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((qk_norm_bwd_kernel<DT, LPR, MODE>), dim3(grid), dim3(kQkThreads), 0,
                       stream, a);
    return hipGetLastError();
}

template <int DT, int LPR>
hipError_t launch_mode(const QkArgs& a, int mode, bool backward, hipStream_t stream) {
    if (mode == ROT_HALVES) return launch<DT, LPR, ROT_HALVES>(a, backward, stream);
    if (mode == ROT_PAIRS) return launch<DT, LPR, ROT_PAIRS>(a, backward, stream);
    return launch<DT, LPR, ROT_HALVES_ANY>(a, backward, stream);
}

}  // namespace

template <int DT>
hipError_t launch_qk_norm(const QkArgs& a, int mode, bool backward, hipStream_t stream) {
    const int lanes = qk_lanes(a.D);
    hipError_t e;
    if (lanes == 4) e = launch_mode<DT, 4>(a, mode, backward, stream);
    else if (lanes == 8) e = launch_mode<DT, 8>(a, mode, backward, stream);
    else e = launch_mode<DT, 16>(a, mode, backward, stream);
    if (e != hipSuccess || !backward || !(a.part[0].dw || a.part[1].dw)) return e;
    hipLaunchKernelGGL(qk_norm_dw_kernel<DT>, dim3((unsigned)((a.D + 15) / 16), 2), dim3(1024), 0,
                       stream, a, lanes * 8);
    return hipGetLastError();
}

template hipError_t launch_qk_norm<IGC_DT>(const QkArgs&, int, bool, hipStream_t);

}  // namespace igc
