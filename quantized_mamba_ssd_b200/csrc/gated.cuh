// Arithmetic shared by the gated-recurrence and checkpoint kernels.
//
//   h_t = a_t h_{t-1} + w_t x_t        a = exp(gate) or 1 / (1 + exp(-gate)), w = 1 or 1 - a
//
// A recurrence with a long memory is sensitive to its decays: an error e in every a of a steady
// gate changes the state by e / (1 - a).  fp32 tensors therefore carry each decay as a sum of two
// floats, a = hi + lo with lo from 1 - a computed without cancellation, so that the error is a
// rounding of the state per step instead of one of the decay.  16-bit tensors carry one float
// from the fast exponential: over all their gates it is off by at most 1.9 x 2^-24 (for decays of
// 1/2 and more; one rounding of a float is 0.5), which reaches half a step of the output at a memory
// 1 / (1 - a) of 4400 (fp16) or 34000 (bf16) tokens of one and the same gate.  (Its results below
// 2^-126 are 0.)
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
// the channels of one lane: one fp32, or two 16-bit ones whose fp32 values share the two-wide
// instructions of sm_100 (half the instructions per element)
// ---------------------------------------------------------------------------------------
template <typename T> constexpr int kChannels = 4 / sizeof(T);

template <int V> struct Vec;
template <> struct Vec<1> {
    float x;
    __device__ __forceinline__ float operator[](int) const { return x; }
    __device__ __forceinline__ void set(int, float v) { x = v; }
};
template <> struct Vec<2> {
    float2 x;
    __device__ __forceinline__ float operator[](int i) const { return i ? x.y : x.x; }
    __device__ __forceinline__ void set(int i, float v) { (i ? x.y : x.x) = v; }
};

template <int V> __device__ __forceinline__ Vec<V> splat(float v) {
    Vec<V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.set(i, v);
    return r;
}

__device__ __forceinline__ unsigned long long as_pair(Vec<2> v) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x.x), "f"(v.x.y));
    return r;
}
__device__ __forceinline__ Vec<2> from_pair(unsigned long long r) {
    Vec<2> v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x.x), "=f"(v.x.y) : "l"(r));
    return v;
}

__device__ __forceinline__ Vec<1> fma(Vec<1> a, Vec<1> b, Vec<1> c) { return {fmaf(a.x, b.x, c.x)}; }
__device__ __forceinline__ Vec<1> mul(Vec<1> a, Vec<1> b) { return {a.x * b.x}; }
__device__ __forceinline__ Vec<1> add(Vec<1> a, Vec<1> b) { return {a.x + b.x}; }
__device__ __forceinline__ Vec<1> sub(Vec<1> a, Vec<1> b) { return {a.x - b.x}; }
__device__ __forceinline__ Vec<2> fma(Vec<2> a, Vec<2> b, Vec<2> c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(as_pair(a)), "l"(as_pair(b)), "l"(as_pair(c)));
    return from_pair(r);
}
__device__ __forceinline__ Vec<2> mul(Vec<2> a, Vec<2> b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_pair(a)), "l"(as_pair(b)));
    return from_pair(r);
}
__device__ __forceinline__ Vec<2> add(Vec<2> a, Vec<2> b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_pair(a)), "l"(as_pair(b)));
    return from_pair(r);
}
__device__ __forceinline__ Vec<2> sub(Vec<2> a, Vec<2> b) { return fma(b, splat<2>(-1.f), a); }

// ---------------------------------------------------------------------------------------
// decays
// ---------------------------------------------------------------------------------------
template <int V> struct Decay {
    Vec<V> a;   // decay, rounded to one float
    Vec<V> lo;  // V == 1 (fp32 tensors): a + lo is the decay to about 2^-24 of 1 - a
    Vec<V> u;   // 1 - a without cancellation
};

__device__ __forceinline__ float fast_exp2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float fast_rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

template <bool LOGIT>
__device__ __forceinline__ Decay<1> decay_of(Vec<1> gate) {
    const float g = gate.x;
    Decay<1> d;
    if constexpr (LOGIT) {
        // the larger of a and 1 - a is 1 / (1 + t) with t = exp(-|gate|) <= 1, the other t times it
        const float t = expf(-fabsf(g));
        const float r = fast_rcp(1.f + t), tr = t * r;
        d.a.x = g >= 0.f ? r : tr;
        d.u.x = g >= 0.f ? tr : r;
    } else {
        d.a.x = expf(g);
        d.u.x = -expm1f(g);
    }
    d.lo.x = d.a.x >= 0.5f ? (1.f - d.a.x) - d.u.x : 0.f;
    return d;
}

template <bool LOGIT>
__device__ __forceinline__ Decay<2> decay_of(Vec<2> g) {
    constexpr float kLog2e = 1.4426950408889634f;
    Decay<2> d;
    d.lo = splat<2>(0.f);
    const Vec<2> one = splat<2>(1.f);
    const Vec<2> e = mul(g, splat<2>(LOGIT ? -kLog2e : kLog2e));
    Vec<2> t;
    t.x = make_float2(fast_exp2(e.x.x), fast_exp2(e.x.y));
    if constexpr (LOGIT) {
        // t = inf gives a = 0 and 1 - a = 1; the product t a would be inf * 0 there
        const Vec<2> s = add(one, t);
        d.a.x = make_float2(fast_rcp(s.x.x), fast_rcp(s.x.y));
        const Vec<2> near = mul(t, d.a), far = sub(one, d.a);
        d.u.x = make_float2(d.a.x.x < 0.5f ? far.x.x : near.x.x, d.a.x.y < 0.5f ? far.x.y : near.x.y);
    } else {
        d.a = t;
        // 1 - exp(g) = g (-1 - g/2 - g^2/6 - g^3/24 - ..): below 1/16 the next term is 2^-22.9, and the
        // four are 2^-21 accurate with their roundings; above, the difference is 2^-18 (half a step of
        // either 16-bit type is far more, but the fp32 states show it: with three terms, 2^-16 too large)
        const Vec<2> p = fma(g, fma(g, fma(g, splat<2>(-1.f / 24.f), splat<2>(-1.f / 6.f)), splat<2>(-0.5f)),
                             splat<2>(-1.f));
        const Vec<2> near = mul(g, p), far = sub(one, d.a);
        d.u.x = make_float2(fabsf(g.x.x) < 0.0625f ? near.x.x : far.x.x,
                            fabsf(g.x.y) < 0.0625f ? near.x.y : far.x.y);
    }
    return d;
}

// a h + b
__device__ __forceinline__ Vec<1> step(Vec<1> a, Vec<1> lo, Vec<1> h, Vec<1> b) {
    return fma(a, h, fma(lo, h, b));
}
__device__ __forceinline__ Vec<2> step(Vec<2> a, Vec<2>, Vec<2> h, Vec<2> b) { return fma(a, h, b); }

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
constexpr uint32_t kCodeNaN = 0x80;  // the code -128, which no value has: one that is not finite

// Scale exponent for a block whose largest magnitude has the bit pattern `top`: top = m 2^E with
// 1 <= m < 2 gets the scale 2^(E - 6), so that its codes use 64 to 127; scales stop at 2^-126.
__device__ __forceinline__ uint32_t scale_exp(uint32_t top) {
    if (top >= 0x7f800000u) return kExpNaN;
    const int e = static_cast<int>(top >> 23) - 6;
    return e < 1 ? 1u : static_cast<uint32_t>(e);
}

// 2^(e - 127); NaN for a block that is not finite
__device__ __forceinline__ float scale_of(uint32_t e) {
    return __uint_as_float(e == kExpNaN ? 0x7fc00000u : e << 23);
}

// Codes of a block.  1.5 * 2^23 plus v / scale, a product that is exact (a power of two; what
// underflows rounds to 0 either way), is rounded once, to an integer, by the addition, and has the
// code in its low byte; conversion instructions run at an eighth of the rate.  The code does not
// depend on the precision it is computed in.  Above 127.5 scales it stays at 127, not 128: twice
// the scale would cost every code of the block a bit, and the value 64 * 2^(E - 5) overflows where
// the largest magnitude is its type's largest number.  Blocks that are not finite get codes 0.
constexpr float kCodeMagic = 12582912.f;
struct Coder {
    float inv, most;  // 2^(127 - e), and 127; both 0 for a block that is not finite
    __device__ __forceinline__ explicit Coder(uint32_t e) {
        inv = e == kExpNaN ? 0.f : __uint_as_float((254u - e) << 23);
        most = e == kExpNaN ? 0.f : 127.f;
    }
    __device__ __forceinline__ uint32_t code(float v) const {
        const float r = fmaf(v, inv, kCodeMagic);
        return __float_as_uint(fminf(fmaxf(r, kCodeMagic - most), kCodeMagic + most)) & 0xffu;
    }
};

// What a checkpoint keeps of a gate: below -16 the decay (for logits, above 16 its complement) is
// within 1.2e-7 of its limit, so a mask of the lowest value need not take all of the scale.  It takes
// what -16 takes: its block's scale is 2^-2, in which gates above -1/8 become 0.
constexpr float kHeldGate = 16.f;

}  // namespace gated
}  // namespace ssd
