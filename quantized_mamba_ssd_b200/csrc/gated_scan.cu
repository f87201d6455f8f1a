// Gated linear recurrence: the choice of the scan kernels by type, and the decode step.
#include "gated_launch.cuh"

namespace ssd {

namespace {

using namespace gated;

constexpr int kThreads = 128;

template <typename T, bool LOGIT>
__global__ void __launch_bounds__(kThreads) step_kernel(const GatedStepArgs a) {
    constexpr int V = kChannels<T>;
    const long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) * V;
    if (i >= a.count) return;
    const int n = static_cast<int>(a.count - i < V ? a.count - i : V);
    Vec<V> g = splat<V>(0.f), x = g, h = g;
    for (int v = 0; v < n; ++v) {
        g.set(v, static_cast<float>(static_cast<const T*>(a.gate)[i + v]));
        x.set(v, static_cast<float>(static_cast<const T*>(a.x)[i + v]));
        h.set(v, a.state[i + v]);
    }
    const Decay<V> r = decay_of<LOGIT>(g);
    if (a.complement) x = mul(r.u, x);
    h = step(r.a, r.lo, h, x);
    for (int v = 0; v < n; ++v) {
        a.state[i + v] = h[v];
        static_cast<T*>(a.y)[i + v] = static_cast<T>(h[v]);
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
        constexpr int per = kThreads * kChannels<T>;
        const long long grid = (a.count + per - 1) / per;
        (a.logit ? step_kernel<T, true> : step_kernel<T, false>)<<<(unsigned)grid, kThreads, 0, st>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace ssd
