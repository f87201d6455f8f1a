// Backward gated scan of f32 tensors with logit gates.
#include "gated_bwd.cuh"

namespace ssd {

template <> cudaError_t launch_gated_scan_bwd_as<float, true>(const GatedArgs& a, cudaStream_t st) {
    return gated::dispatch_bwd<float, true>(a, st);
}

}  // namespace ssd
