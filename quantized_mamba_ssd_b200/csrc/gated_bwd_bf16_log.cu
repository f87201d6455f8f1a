// Backward gated scan of bf16 tensors with log gates.
#include "gated_bwd.cuh"

namespace ssd {

template <> cudaError_t launch_gated_scan_bwd_as<__nv_bfloat16, false>(const GatedArgs& a, cudaStream_t st) {
    return gated::dispatch_bwd<__nv_bfloat16, false>(a, st);
}

}  // namespace ssd
