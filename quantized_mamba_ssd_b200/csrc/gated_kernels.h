// Internal launcher interface of the gated recurrence and the 8-bit checkpoints (abi_gated.cu to
// the kernels).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace ssd {

// Rows of `channels` contiguous elements, one per (batch, token); strides in elements.
struct GatedRows {
    const void* ptr;
    long long batch_stride, token_stride;
};

struct GatedArgs {
    GatedRows x, gate;  // forward, and backward from the inputs
    GatedRows dy;       // backward
    GatedRows y;        // forward output
    GatedRows dx, dgate;  // backward outputs
    // 8-bit checkpoints, contiguous: codes [batch, seqlen, channels], exponents
    // [batch, ceil(seqlen / 16), channels]; null when not used
    int8_t* x_q;
    uint8_t* x_e;
    int8_t* gate_q;
    uint8_t* gate_e;
    const int32_t* cu;  // device [nseq + 1], or null: `batch` sequences of seqlen tokens
    int nseq;
    int batch, seqlen, channels;
    int logit, complement;  // gate and input form
    int io_dtype;           // SSD_IO_*
    const float* init_state;
    float* final_state;
    float* span_states;  // [batch, ceil(seqlen / 64), channels]
    const float* dfinal_state;
    float* dinit_state;
    void* workspace;  // gated_workspace_bytes
};

struct GatedStepArgs {
    float* state;
    const void* x;
    const void* gate;
    void* y;
    long long count;  // batch * channels
    int logit, complement, io_dtype;
};

// Workspace of the scans (the larger of the forward's and the backwards').
size_t gated_workspace_bytes(int batch, int seqlen, int channels, int io_dtype);
cudaError_t launch_gated_scan(const GatedArgs& a, cudaStream_t stream);
cudaError_t launch_gated_scan_bwd(const GatedArgs& a, cudaStream_t stream);
cudaError_t launch_gated_step(const GatedStepArgs& a, cudaStream_t stream);
// rows [batch, seqlen, channels] of io_dtype to codes and exponents, and back
cudaError_t launch_ckpt_pack(const GatedRows& x, int batch, int seqlen, int channels, int io_dtype,
                             int8_t* q, uint8_t* e, cudaStream_t stream);
cudaError_t launch_ckpt_unpack(const int8_t* q, const uint8_t* e, int batch, int seqlen,
                               int channels, int io_dtype, void* x, cudaStream_t stream);

}  // namespace ssd
