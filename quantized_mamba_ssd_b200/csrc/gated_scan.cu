// Gated linear recurrence over sequences, forward and backward: one thread per channel walks the
// tokens.
#include "gated_launch.cuh"

namespace ssd {

namespace {

using namespace gated;

constexpr int kThreads = 128;

template <typename T>
__device__ __forceinline__ float load(const GatedRows& r, int b, int t, int c) {
    return to_f32(static_cast<const T*>(r.ptr)[b * r.batch_stride + t * r.token_stride + c]);
}

template <typename T>
__device__ __forceinline__ void store(const GatedRows& r, int b, int t, int c, float v) {
    T* p = static_cast<T*>(const_cast<void*>(r.ptr));
    p[b * r.batch_stride + t * r.token_stride + c] = from_f32<T>(v);
}

template <typename T, bool LOGIT>
__global__ void __launch_bounds__(kThreads) scan_bwd_kernel(const GatedArgs a) {
    const int c = blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y;
    if (c >= a.channels) return;
    const int d = a.channels, spans = (a.seqlen + kSpan - 1) / kSpan;
    const int blocks = (a.seqlen + kBlock - 1) / kBlock;
    if (a.cu && a.dinit_state)
        for (int s = 0; s < a.nseq; ++s)
            if (a.cu[s + 1] <= a.cu[s])
                a.dinit_state[(size_t)s * d + c] = a.dfinal_state ? a.dfinal_state[(size_t)s * d + c] : 0.f;
    float back = !a.cu && a.dfinal_state ? a.dfinal_state[(size_t)b * d + c] : 0.f;
    float before[kSpan], xs[kSpan], gs[kSpan];
    for (int sp = spans - 1; sp >= 0; --sp) {
        const int t0 = sp * kSpan, n = min(kSpan, a.seqlen - t0);
        float h = a.span_states[((size_t)b * spans + sp) * d + c];
        for (int j = 0; j < n; ++j) {
            const int t = t0 + j;
            if (a.cu) {
                const int s = sequence_of(a.cu, a.nseq, t);
                if (s < 0) continue;
                if (a.cu[s] == t) h = a.init_state ? a.init_state[(size_t)s * d + c] : 0.f;
            }
            if (a.x_q) {
                const size_t at = ((size_t)b * a.seqlen + t) * d + c;
                const size_t ae = ((size_t)b * blocks + t / kBlock) * d + c;
                xs[j] = scale_of(a.x_e[ae]) * a.x_q[at];
                gs[j] = scale_of(a.gate_e[ae]) * a.gate_q[at];
            } else {
                xs[j] = load<T>(a.x, b, t, c);
                gs[j] = load<T>(a.gate, b, t, c);
            }
            const Decay k = decay_of<T, LOGIT>(gs[j]);
            before[j] = h;
            h = step<kTwo<T>>(k, h, a.complement ? k.u * xs[j] : xs[j]);
        }
        for (int j = n - 1; j >= 0; --j) {
            const int t = t0 + j;
            int s = b, first = 0, last = a.seqlen - 1;
            if (a.cu) {
                s = sequence_of(a.cu, a.nseq, t);
                if (s < 0) continue;
                first = a.cu[s];
                last = a.cu[s + 1] - 1;
                if (t == last) back = a.dfinal_state ? a.dfinal_state[(size_t)s * d + c] : 0.f;
            }
            const Decay k = decay_of<T, LOGIT>(gs[j]);
            const float dh = load<T>(a.dy, b, t, c) + back;
            back = step<kTwo<T>>(k, dh, 0.f);
            float dg = back * (a.complement ? before[j] - xs[j] : before[j]);
            if (LOGIT) dg *= k.u;
            store<T>(a.dx, b, t, c, a.complement ? k.u * dh : dh);
            store<T>(a.dgate, b, t, c, dg);
            if (a.dinit_state && t == first) a.dinit_state[(size_t)s * d + c] = back;
        }
    }
}

template <typename T, bool LOGIT>
__global__ void __launch_bounds__(kThreads) step_kernel(const GatedStepArgs a) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= a.count) return;
    const Decay k = decay_of<T, LOGIT>(to_f32(static_cast<const T*>(a.gate)[i]));
    const float x = to_f32(static_cast<const T*>(a.x)[i]);
    const float h = step<kTwo<T>>(k, a.state[i], a.complement ? k.u * x : x);
    a.state[i] = h;
    static_cast<T*>(a.y)[i] = from_f32<T>(h);
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
        const dim3 grid((a.channels + kThreads - 1) / kThreads, a.batch);
        (a.logit ? scan_bwd_kernel<T, true> : scan_bwd_kernel<T, false>)<<<grid, kThreads, 0, st>>>(a);
        return cudaGetLastError();
    });
}

cudaError_t launch_gated_step(const GatedStepArgs& a, cudaStream_t st) {
    return by_type(a.io_dtype, [&](auto zero) {
        using T = decltype(zero);
        const long long grid = (a.count + kThreads - 1) / kThreads;
        (a.logit ? step_kernel<T, true> : step_kernel<T, false>)<<<(unsigned)grid, kThreads, 0, st>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace ssd
