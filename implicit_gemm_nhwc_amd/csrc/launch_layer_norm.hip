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
        hipError_t e = hipErrorInvalidValue;
#define IGC_FORM(LANES, CHUNKS, THREADS)           \
    if (f.lanes == LANES && f.chunks == CHUNKS)    \
        e = launch<DT, LANES, CHUNKS, THREADS>(a, backward, stream);
        IGC_LN_FORMS(IGC_FORM)
#undef IGC_FORM
        if (e != hipSuccess) return e;
    }
    if (!backward || !(a.dw || a.db)) return hipSuccess;
    hipLaunchKernelGGL(layer_norm_dw_kernel<DT>, dim3((unsigned)((2 * a.C + 15) / 16)), dim3(1024),
                       0, stream, a);
    return hipGetLastError();
}

template hipError_t launch_layer_norm<IGC_DT>(const LnArgs&, bool, hipStream_t);

}  // namespace igc
