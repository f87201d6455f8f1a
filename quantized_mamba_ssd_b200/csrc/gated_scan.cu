// Gated linear recurrence: the choice of the scan kernels by type, and the decode step.
#include <algorithm>

#include "gated_launch.cuh"

namespace ssd {

namespace {

using namespace gated;

constexpr int kThreads = 128;

// One token, in place: x, gate and the state are read, y and the state written.  A thread takes four
// elements, 16 bytes of the state; the end that does not fill four, and tensors that do not start
// at a multiple of theirs, go element by element.  The launch bounds it: 1.0 us for 1 x 4096 bf16, 2.2
// for 128 x 8192 (in a graph, the state in L2; 2.3 us is the floor from HBM).
template <typename T, bool LOGIT, bool WIDE>
__global__ void __launch_bounds__(kThreads) step_kernel(const GatedStepArgs a) {
    constexpr int V = kChannels<T>, N = WIDE ? 4 : V;
    const long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) * N;
    if (i >= a.count) return;
    const T* x = static_cast<const T*>(a.x) + i;
    const T* gate = static_cast<const T*>(a.gate) + i;
    T* y = static_cast<T*>(a.y) + i;
    float* state = a.state + i;
    auto next = [&](Vec<V> h, Vec<V> in, Vec<V> g) {
        const Decay<V> r = decay_of<LOGIT>(g);
        if (a.complement) in = mul(r.u, in);
        return step(r.a, r.lo, h, in);
    };
    if (WIDE && a.count - i >= 4) {
        struct alignas(4 * sizeof(T)) Four { uint32_t w[4 / V]; };
        const Four fx = *reinterpret_cast<const Four*>(x), fg = *reinterpret_cast<const Four*>(gate);
        float4 h = *reinterpret_cast<const float4*>(state);
        Four out;
        if constexpr (V == 1) {
            float* p = &h.x;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                p[k] = next({p[k]}, Pack<T>::get(fx.w[k]), Pack<T>::get(fg.w[k])).x;
                out.w[k] = __float_as_uint(p[k]);
            }
        } else {
            Vec<V> lo, hi;
            lo.x = make_float2(h.x, h.y);
            hi.x = make_float2(h.z, h.w);
            lo = next(lo, Pack<T>::get(fx.w[0]), Pack<T>::get(fg.w[0]));
            hi = next(hi, Pack<T>::get(fx.w[1]), Pack<T>::get(fg.w[1]));
            out.w[0] = Pack<T>::put(lo);
            out.w[1] = Pack<T>::put(hi);
            h = make_float4(lo[0], lo[1], hi[0], hi[1]);
        }
        *reinterpret_cast<float4*>(state) = h;
        *reinterpret_cast<Four*>(y) = out;
        return;
    }
    for (long long k = 0; k < N && k < a.count - i; k += V) {
        const int n = static_cast<int>(a.count - i - k < V ? a.count - i - k : V);
        Vec<V> g = splat<V>(0.f), in = g, h = g;
        for (int v = 0; v < n; ++v) {
            g.set(v, static_cast<float>(gate[k + v]));
            in.set(v, static_cast<float>(x[k + v]));
            h.set(v, state[k + v]);
        }
        h = next(h, in, g);
        for (int v = 0; v < n; ++v) {
            state[k + v] = h[v];
            y[k + v] = static_cast<T>(h[v]);
        }
    }
}

template <typename F>
cudaError_t by_type(int io_dtype, F f) {
    switch (io_dtype) {
        case SSD_IO_F32: return f(float{});
        case SSD_IO_F16: return f(__half{});
        case SSD_IO_BF16: return f(__nv_bfloat16{});
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

size_t gated_workspace_bytes(int batch, int seqlen, int channels, int io_dtype) {
    const int lanes = io_dtype == SSD_IO_F32 ? 32 : 64;  // channels of a strip
    const long long units = (long long)((channels + lanes - 1) / lanes) * batch;
    const int segments = (seqlen + kSub - 1) / kSub;
    const int sms = sm_count();
    int n = 1;
    for (bool aligned : {false, true})  // the alignment of the rows is not known here
        n = std::max({n, chunks_of(Work::kPlain, units, segments, kFwdWarps, kFwdBlocks, sms, aligned).count,
                      chunks_of(Work::kToCodes, units, segments, kFwdWarps, kFwdBlocks, sms, aligned).count,
                      chunks_of(Work::kPlain, units, segments, kBwdWarps<false>, kBwdBlocks<false>, sms, aligned).count,
                      chunks_of(Work::kFromCodes, units, segments, kBwdWarps<true>, kBwdBlocks<true>, sms, aligned).count});
    return n > 1 ? (size_t)units * n * MapSlots<1>::kFloats * sizeof(float) : 0;
}

cudaError_t launch_gated_scan(const GatedArgs& a, cudaStream_t st) {
    return by_type(a.io_dtype, [&](auto zero) { return launch_gated_scan_as<decltype(zero)>(a, st); });
}

cudaError_t launch_gated_scan_bwd(const GatedArgs& a, cudaStream_t st) {
    return by_type(a.io_dtype, [&](auto zero) {
        using T = decltype(zero);
        return a.logit ? launch_gated_scan_bwd_as<T, true>(a, st)
                       : launch_gated_scan_bwd_as<T, false>(a, st);
    });
}

cudaError_t launch_gated_step(const GatedStepArgs& a, cudaStream_t st) {
    return by_type(a.io_dtype, [&](auto zero) {
        using T = decltype(zero);
        const uintptr_t halves = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.gate) |
                                 reinterpret_cast<uintptr_t>(a.y);
        const bool wide = halves % (4 * sizeof(T)) == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0;
        const int per = kThreads * (wide ? 4 : kChannels<T>);
        const unsigned grid = static_cast<unsigned>((a.count + per - 1) / per);
        if (wide)
            (a.logit ? step_kernel<T, true, true> : step_kernel<T, false, true>)<<<grid, kThreads, 0, st>>>(a);
        else
            (a.logit ? step_kernel<T, true, false> : step_kernel<T, false, false>)<<<grid, kThreads, 0, st>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace ssd
