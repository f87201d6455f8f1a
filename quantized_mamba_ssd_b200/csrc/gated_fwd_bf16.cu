// Forward gated scan of bf16 tensors.
#include "gated_fwd.cuh"

namespace ssd {

template <> cudaError_t launch_gated_scan_as<__nv_bfloat16>(const GatedArgs& a, cudaStream_t st) {
    return gated::dispatch_fwd<__nv_bfloat16>(a, st);
}

}  // namespace ssd
