// Forward gated scan of f16 tensors.
#include "gated_fwd.cuh"

namespace ssd {

template <> cudaError_t launch_gated_scan_as<__half>(const GatedArgs& a, cudaStream_t st) {
    return gated::dispatch_fwd<__half>(a, st);
}

}  // namespace ssd
