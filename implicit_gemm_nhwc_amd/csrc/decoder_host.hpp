// Host-side pieces of the decoder block's operators shared by their
// translation units: per-type launchers and the rules that pick a kernel form.
#pragma once

#include "igemm_host.hpp"
#include "layer_norm.hpp"

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

}  // namespace igc
