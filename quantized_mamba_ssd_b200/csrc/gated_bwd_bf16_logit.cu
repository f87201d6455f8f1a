// Backward gated scan of bf16 tensors with logit gates.
#include "gated_bwd.cuh"

namespace ssd {

template <> cudaError_t launch_gated_scan_bwd_as<__nv_bfloat16, true>(const GatedArgs& a, cudaStream_t st) {
    return gated::dispatch_bwd<__nv_bfloat16, true>(a, st);
}

}  // namespace ssd
