// Arithmetic shared by the gated-recurrence and checkpoint kernels.
//
//   h_t = a_t h_{t-1} + w_t x_t        a = exp(gate) or 1 / (1 + exp(-gate)), w = 1 or 1 - a
//
// A recurrence with a long memory is sensitive to its decays: an error e in every a of a steady
// gate changes the state by e / (1 - a).  fp32 tensors therefore carry each decay as a sum of two
// floats, a = hi + lo with lo from 1 - a computed without cancellation, so that the error is a
// rounding of the state per step instead of one of the decay.  16-bit tensors carry one float
// from the fast exponential: its 2^-22 only reaches half a bf16 step (2^-9 of the state) at a
// memory of 1 / (1 - a) = 8192 tokens of one and the same gate.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/ssd_i8.h"

namespace ssd {
namespace gated {

constexpr int kSpan = SSD_GATED_SPAN;   // tokens between saved states
constexpr int kBlock = SSD_CKPT_BLOCK;  // tokens of one channel that share a checkpoint scale

// ---------------------------------------------------------------------------------------
// element types
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// ---------------------------------------------------------------------------------------
// decays
// ---------------------------------------------------------------------------------------
// Two-float decays for fp32 tensors (see the top of this file).
template <typename T> constexpr bool kTwo = sizeof(T) == 4;

struct Decay {
    float a;   // decay, rounded to one float
    float lo;  // a + lo is the decay to about 2^-24 of 1 - a (fp32 tensors; else 0)
    float u;   // 1 - a without cancellation
};

template <typename T, bool LOGIT>
__device__ __forceinline__ Decay decay_of(float g) {
    Decay d;
    if constexpr (LOGIT) {
        if constexpr (kTwo<T>) {
            const float t = expf(-fabsf(g));
            const float r = __frcp_rn(1.f + t), tr = __fdiv_rn(t, 1.f + t);
            d.a = g >= 0.f ? r : tr;
            d.u = g >= 0.f ? tr : r;
            if (!(g == g)) d.a = d.u = g;
        } else {
            // exp(-gate) = inf gives a = 0, 1 - a = 1; the product t a would be inf * 0 there
            const float t = __expf(-g);
            d.a = __fdividef(1.f, 1.f + t);
            d.u = d.a < 0.5f ? 1.f - d.a : t * d.a;
        }
    } else {
        d.a = kTwo<T> ? expf(g) : __expf(g);
        if constexpr (kTwo<T>) {
            d.u = -expm1f(g);
        } else {
            // 1 - exp(g) = -g (1 + g/2 + g^2/6 + ..): the three terms are 2^-16 accurate
            // below 1/16, above it the difference is
            const float s = -g * fmaf(g, fmaf(g, 1.f / 6.f, 0.5f), 1.f);
            d.u = fabsf(g) < 0.0625f ? s : 1.f - d.a;
        }
    }
    d.lo = kTwo<T> && d.a >= 0.5f ? (1.f - d.a) - d.u : 0.f;
    return d;
}

// a h + b
template <bool TWO>
__device__ __forceinline__ float step(const Decay& d, float h, float b) {
    return fmaf(d.a, h, TWO ? fmaf(d.lo, h, b) : b);
}

// ---------------------------------------------------------------------------------------
// packed sequences
// ---------------------------------------------------------------------------------------
// The sequence that holds token t: the last s in [0, nseq) with cu[s] <= t, if t < cu[s + 1];
// -1 otherwise.  Whatever cu holds, the result lies in [-1, nseq) and only cu[0 .. nseq] is read.
__device__ __forceinline__ int sequence_of(const int32_t* __restrict__ cu, int nseq, int t) {
    int lo = 0, hi = nseq;  // cu[s] <= t for s < lo, cu[s] > t for s >= hi (over 0 .. nseq - 1)
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid) <= t) lo = mid + 1;
        else hi = mid;
    }
    return lo > 0 && t < __ldg(cu + lo) ? lo - 1 : -1;
}

// ---------------------------------------------------------------------------------------
// 8-bit checkpoints: int8 codes of kBlock tokens of one channel with one scale 2^(e - 127)
// ---------------------------------------------------------------------------------------
constexpr uint32_t kExpNaN = 255;  // the block holds a value that is not finite

// Scale exponent for a block whose largest magnitude has the bit pattern `top`: top = m 2^E with
// 1 <= m < 2 gets the scale 2^(E - 6), so that its codes use 64 to 127; scales stop at 2^-126.
__device__ __forceinline__ uint32_t scale_exp(uint32_t top) {
    if (top >= 0x7f800000u) return kExpNaN;
    const int e = static_cast<int>(top >> 23) - 6;
    return e < 1 ? 1u : static_cast<uint32_t>(e);
}

// 2^(127 - e), the factor of the codes; 0 for a block that is not finite (its codes are 0)
__device__ __forceinline__ float inv_scale_of(uint32_t e) {
    return e == kExpNaN ? 0.f : __uint_as_float((254u - e) << 23);
}

// 2^(e - 127); NaN for a block that is not finite
__device__ __forceinline__ float scale_of(uint32_t e) {
    return __uint_as_float(e == kExpNaN ? 0x7fc00000u : e << 23);
}

// The product is exact (a power of two; what underflows rounds to 0 either way), so the code
// does not depend on the precision it is computed in.  Above 127.5 scales it stays at 127, not
// 128: twice the scale would cost every code of the block a bit, and the value 64 * 2^(E - 5)
// overflows where the largest magnitude is its type's largest number.
__device__ __forceinline__ int code_of(float v, float inv) {
    const int q = __float2int_rn(v * inv);  // NaN converts to 0
    return max(-127, min(127, q));
}

// What a checkpoint keeps of a gate: below -16 the decay (for logits, above 16 its complement)
// is within 1.2e-7 of its limit, and masks of the lowest value must not set the block's scale.
template <bool LOGIT>
__device__ __forceinline__ float held_gate(float g) {
    if (g < -16.f) g = -16.f;
    if (LOGIT && g > 16.f) g = 16.f;
    return g;
}

}  // namespace gated
}  // namespace ssd
