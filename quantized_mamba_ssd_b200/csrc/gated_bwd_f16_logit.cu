// Backward gated scan of f16 tensors with logit gates.
#include "gated_bwd.cuh"

namespace ssd {

template <> cudaError_t launch_gated_scan_bwd_as<__half, true>(const GatedArgs& a, cudaStream_t st) {
    return gated::dispatch_bwd<__half, true>(a, st);
}

}  // namespace ssd
