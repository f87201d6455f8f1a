// 8-bit activation checkpoints: blocks of 16 tokens of one channel as int8 codes with one
// power-of-two scale, and back.
#include "gated.cuh"
#include "gated_kernels.h"

namespace ssd {

namespace {

using namespace gated;

constexpr int kThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kThreads)
pack_kernel(GatedRows x, int seqlen, int d, int8_t* __restrict__ q, uint8_t* __restrict__ e) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= d) return;
    const int blocks = (seqlen + kBlock - 1) / kBlock;
    const int b = blockIdx.y / blocks, t0 = blockIdx.y % blocks * kBlock;
    const int n = min(kBlock, seqlen - t0);
    const T* src = static_cast<const T*>(x.ptr) + b * x.batch_stride + t0 * x.token_stride + c;
    uint32_t top = 0;
    for (int j = 0; j < n; ++j)
        top = max(top, __float_as_uint(fabsf(static_cast<float>(src[j * x.token_stride]))));
    const uint32_t ex = scale_exp(top);
    const float inv = inv_scale_of(ex);
    int8_t* dst = q + ((size_t)b * seqlen + t0) * d + c;
    for (int j = 0; j < n; ++j)
        dst[(size_t)j * d] = static_cast<int8_t>(code_of(static_cast<float>(src[j * x.token_stride]), inv));
    e[(size_t)blockIdx.y * d + c] = static_cast<uint8_t>(ex);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
unpack_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ e, int seqlen, int d,
              T* __restrict__ x) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= d) return;
    const int blocks = (seqlen + kBlock - 1) / kBlock;
    const int b = blockIdx.y / blocks, t0 = blockIdx.y % blocks * kBlock;
    const int n = min(kBlock, seqlen - t0);
    const float scale = scale_of(e[(size_t)blockIdx.y * d + c]);
    const size_t at = ((size_t)b * seqlen + t0) * d + c;
    for (int j = 0; j < n; ++j) x[at + (size_t)j * d] = static_cast<T>(scale * q[at + (size_t)j * d]);
}

}  // namespace

cudaError_t launch_ckpt_pack(const GatedRows& x, int batch, int seqlen, int d, int io_dtype,
                             int8_t* q, uint8_t* e, cudaStream_t st) {
    const dim3 grid((d + kThreads - 1) / kThreads, batch * ((seqlen + kBlock - 1) / kBlock));
    if (io_dtype == SSD_IO_F32) pack_kernel<float><<<grid, kThreads, 0, st>>>(x, seqlen, d, q, e);
    else if (io_dtype == SSD_IO_F16) pack_kernel<__half><<<grid, kThreads, 0, st>>>(x, seqlen, d, q, e);
    else pack_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(x, seqlen, d, q, e);
    return cudaGetLastError();
}

cudaError_t launch_ckpt_unpack(const int8_t* q, const uint8_t* e, int batch, int seqlen, int d,
                               int io_dtype, void* x, cudaStream_t st) {
    const dim3 grid((d + kThreads - 1) / kThreads, batch * ((seqlen + kBlock - 1) / kBlock));
    if (io_dtype == SSD_IO_F32)
        unpack_kernel<<<grid, kThreads, 0, st>>>(q, e, seqlen, d, static_cast<float*>(x));
    else if (io_dtype == SSD_IO_F16)
        unpack_kernel<<<grid, kThreads, 0, st>>>(q, e, seqlen, d, static_cast<__half*>(x));
    else
        unpack_kernel<<<grid, kThreads, 0, st>>>(q, e, seqlen, d, static_cast<__nv_bfloat16*>(x));
    return cudaGetLastError();
}

}  // namespace ssd
