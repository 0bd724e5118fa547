// Launchers of the rows in 8 bits, the cache and the attention over it, one
// element type per translation unit (IGC_DT).
#include "decoder_host.hpp"

#ifndef IGC_DT
#error "IGC_DT must name the element type of this translation unit"
#endif

namespace igc {
namespace {

template <int DT, int LPR, int NC, int NT, bool LONG = false>
hipError_t launch_quant(const QuantArgs& a, hipStream_t stream) {
    constexpr int PER = NT / LPR;
    hipLaunchKernelGGL((quantize_rows_kernel<DT, LPR, NC, NT, LONG>),
                       dim3((unsigned)(((int64_t)a.rows + PER - 1) / PER)), dim3(NT), 0, stream,
                       a);
    return hipGetLastError();
}

template <int DT, int LPR>
hipError_t launch_io(const CacheArgs& a, bool write, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.B * a.runs * 2 * a.hc));
    if (write)
        hipLaunchKernelGGL((kv_cache_write_kernel<DT, LPR>), grid, dim3(kCacheThreads), 0, stream,
                           a);
    else
        hipLaunchKernelGGL((kv_cache_read_kernel<DT, LPR>), grid, dim3(kCacheThreads), 0, stream,
                           a);
    return hipGetLastError();
}

template <int DT, int DP, int RB>
hipError_t launch_attn(const CacheAttnArgs& x, unsigned groups, hipStream_t stream) {
    auto kern = cache_attn_kernel<DT, DP, RB>;
    constexpr size_t lds = (size_t)kCacheWaves * (2 * CacheStage<DP>::BYTES + 32 * 4);
    static LdsAttr attr;
    const hipError_t e = ensure_lds(attr, (const void*)kern, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3(groups), dim3(kCacheWaves * 64), lds, stream, x);
    return hipGetLastError();
}

template <int DT, int DP>
hipError_t launch_attn(const CacheAttnArgs& x, unsigned groups, hipStream_t stream) {
    return x.tile == 16 ? launch_attn<DT, DP, 1>(x, groups, stream)
                        : launch_attn<DT, DP, 2>(x, groups, stream);
}

}  // namespace

template <int DT>
hipError_t launch_quantize_rows(const QuantArgs& a, hipStream_t stream) {
    if (a.C > kLnMaxChannels) return launch_quant<DT, 512, 4, 512, true>(a, stream);
    const LnForm f = ln_form(a.C);
    hipError_t e = hipErrorInvalidValue;
#define IGC_FORM(LANES, CHUNKS, THREADS)        \
    if (f.lanes == LANES && f.chunks == CHUNKS) \
        e = launch_quant<DT, LANES, CHUNKS, THREADS>(a, stream);
    IGC_LN_FORMS(IGC_FORM)
#undef IGC_FORM
    return e;
}

template <int DT>
hipError_t launch_kv_cache(const CacheArgs& a, bool write, hipStream_t stream) {
    const int lanes = qk_lanes(a.D);
    if (lanes == 4) return launch_io<DT, 4>(a, write, stream);
    if (lanes == 8) return launch_io<DT, 8>(a, write, stream);
    return launch_io<DT, 16>(a, write, stream);
}

template <int DT>
hipError_t launch_cache_attn(const CacheAttnArgs& x, unsigned groups, hipStream_t stream) {
    const int dp = padded_dim(x.a.D);
    hipError_t e;
    if (dp == 32) e = launch_attn<DT, 32>(x, groups, stream);
    else if (dp == 64) e = launch_attn<DT, 64>(x, groups, stream);
    else if (dp == 96) e = launch_attn<DT, 96>(x, groups, stream);
    else e = launch_attn<DT, 128>(x, groups, stream);
    if (e != hipSuccess || !x.split) return e;
    hipLaunchKernelGGL(cache_attn_join_kernel<DT>,
                       dim3((unsigned)((int64_t)x.a.B * x.a.Hk * x.a.row_tiles *
                                       (x.a.rows < x.tile ? x.a.rows : x.tile))),
                       dim3(256), 0, stream, x);
    return hipGetLastError();
}

template hipError_t launch_quantize_rows<IGC_DT>(const QuantArgs&, hipStream_t);
template hipError_t launch_kv_cache<IGC_DT>(const CacheArgs&, bool, hipStream_t);
template hipError_t launch_cache_attn<IGC_DT>(const CacheAttnArgs&, unsigned, hipStream_t);

}  // namespace igc
