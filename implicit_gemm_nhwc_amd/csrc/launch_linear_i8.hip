// Launchers of the product in 8-bit integers, one element type of the output
// per translation unit (IGC_DT).
#include "decoder_host.hpp"

#ifndef IGC_DT
#error "IGC_DT must name the element type of this translation unit"
#endif

namespace igc {
namespace {

template <int DT, int MT>
hipError_t launch_few(const LinArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((linear_i8_few_kernel<DT, MT>), dim3((unsigned)a.tiles_n),
                       dim3(kFewWaves * 64), 0, stream, a);
    return hipGetLastError();
}

template <int DT, int B, int NS>
hipError_t launch_tile(const LinArgs& a, hipStream_t stream) {
    auto kern = linear_i8_tile_kernel<DT, B, NS>;
    constexpr size_t lds = LinTile<B, NS>::LDS;
    static LdsAttr attr;
    const hipError_t e = ensure_lds(attr, (const void*)kern, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)((int64_t)a.tiles_m * a.tiles_n)), dim3(256), lds,
                       stream, a);
    return hipGetLastError();
}

}  // namespace

template <int DT>
hipError_t launch_linear_i8(const LinArgs& a, int tile, hipStream_t stream) {
    if (tile == 256) return launch_tile<DT, 256, 3>(a, stream);
    if (tile == 128) return launch_tile<DT, 128, 3>(a, stream);
    if (tile == 64)
        return (int64_t)a.tiles_m * a.tiles_n > kNumCUs ? launch_tile<DT, 64, 2>(a, stream)
                                                        : launch_tile<DT, 64, 3>(a, stream);
    return a.M <= 16 ? launch_few<DT, 1>(a, stream) : launch_few<DT, 2>(a, stream);
}

template hipError_t launch_linear_i8<IGC_DT>(const LinArgs&, int, hipStream_t);

}  // namespace igc
