// Forward gated scan of f32 tensors.
#include "gated_fwd.cuh"

namespace ssd {

template <> cudaError_t launch_gated_scan_as<float>(const GatedArgs& a, cudaStream_t st) {
    return gated::dispatch_fwd<float>(a, st);
}

}  // namespace ssd
