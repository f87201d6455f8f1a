// Backward gated scan of f32 tensors with log gates.
#include "gated_bwd.cuh"

namespace ssd {

template <> cudaError_t launch_gated_scan_bwd_as<float, false>(const GatedArgs& a, cudaStream_t st) {
    return gated::dispatch_bwd<float, false>(a, st);
}

}  // namespace ssd
