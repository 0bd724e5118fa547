// Launchers of the layer norm kernels, one element type per translation unit
// (IGC_DT).
#include "decoder_host.hpp"

#ifndef IGC_DT
#error "IGC_DT must name the element type of this translation unit"
#endif

namespace igc {
namespace {

template <int DT, int LPR, int NC, int NT>
hipError_t launch(const LnArgs& a, bool backward, hipStream_t stream) {
    if (backward) {
        hipLaunchKernelGGL((layer_norm_bwd_kernel<DT, LPR, NC, NT>), dim3((unsigned)a.blocks),
                           dim3(NT), 0, stream, a);
    } else {
        constexpr int PER = NT / LPR;
        hipLaunchKernelGGL((layer_norm_fwd_kernel<DT, LPR, NC, NT>),
                           dim3((unsigned)(((int64_t)a.rows + PER - 1) / PER)), dim3(NT), 0,
                           stream, a);
    }
    return hipGetLastError();
}

}  // namespace

template <int DT>
hipError_t launch_layer_norm(const LnArgs& a, bool backward, hipStream_t stream) {
    if (a.rows > 0) {
        const LnForm f = ln_form(a.C);
        hipError_t e;
        if (f.lanes == 8) e = launch<DT, 8, 1, 256>(a, backward, stream);
        else if (f.lanes == 16) e = launch<DT, 16, 1, 256>(a, backward, stream);
        else if (f.lanes == 32) e = launch<DT, 32, 1, 256>(a, backward, stream);
        else if (f.lanes == 64 && f.chunks == 1) e = launch<DT, 64, 1, 256>(a, backward, stream);
        else if (f.lanes == 64 && f.chunks == 2) e = launch<DT, 64, 2, 256>(a, backward, stream);
        else if (f.lanes == 64) e = launch<DT, 64, 4, 256>(a, backward, stream);
        else if (f.lanes == 256 && f.chunks == 2) e = launch<DT, 256, 2, 256>(a, backward, stream);
        else if (f.lanes == 256) e = launch<DT, 256, 4, 256>(a, backward, stream);
        else e = launch<DT, 512, 4, 512>(a, backward, stream);
        if (e != hipSuccess) return e;
    }
    if (!backward || !(a.dw || a.db)) return hipSuccess;
    hipLaunchKernelGGL(layer_norm_dw_kernel<DT>, dim3((unsigned)((2 * a.C + 15) / 16)), dim3(1024),
                       0, stream, a);
    return hipGetLastError();
}

template hipError_t launch_layer_norm<IGC_DT>(const LnArgs&, bool, hipStream_t);

}  // namespace igc
