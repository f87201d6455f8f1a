// Launches of the scan kernels: alignments, and how many warps share a strip.
#pragma once

#include <cmath>

#include "gated_tile.cuh"

namespace ssd {
namespace gated {

struct TileArgs {
    int cluster;  // CTAs per strip
    int strips;   // strips per row
    int blocks;   // checkpoint blocks per row
    int spans;    // spans per row
    // what the start of every row is a multiple of (bytes): 16, 4 or less
    int align_x, align_gate, align_dy;
    int whole_out, whole_codes;  // outputs can be written as whole words (codes: pairs of bytes)
};

inline int alignment(const GatedRows& r, int elem) {
    const unsigned long long all = reinterpret_cast<uintptr_t>(r.ptr) |
                                   (unsigned long long)r.batch_stride * elem |
                                   (unsigned long long)r.token_stride * elem;
    return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : elem;
}

inline bool word_rows(const GatedRows& r, int elem) { return !r.ptr || alignment(r, elem) >= 4; }

template <typename T>
TileArgs tile_args(const GatedArgs& a) {
    constexpr int elem = sizeof(T), V = kChannels<T>;
    TileArgs t{};
    t.strips = (a.channels + 32 * V - 1) / (32 * V);
    t.spans = (a.seqlen + kSpan - 1) / kSpan;
    t.blocks = (a.seqlen + kBlock - 1) / kBlock;
    t.align_x = alignment(a.x, elem);
    t.align_gate = alignment(a.gate, elem);
    t.align_dy = alignment(a.dy, elem);
    t.whole_out = word_rows(a.y, elem) && word_rows(a.dx, elem) && word_rows(a.dgate, elem);
    auto all = [](auto... p) { return (reinterpret_cast<uintptr_t>(p) | ...); };
    if (a.x_q && !a.x.ptr) {  // backward from codes, rows of one byte per channel
        t.align_x = alignment({a.x_q, 0, a.channels}, 1);
        t.align_gate = alignment({a.gate_q, 0, a.channels}, 1);
    }
    t.whole_codes = (all(a.x_q, a.gate_q, a.x_e, a.gate_e) | a.channels) % 2 == 0;
    return t;
}

inline int sm_count() {
    static const int sms = [] {
        int dev = 0, n = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
            n = 148;
        return n;
    }();
    return sms;
}

// CTAs per strip, the R with the least waves(R) * steps(R) * (1 + the meeting's share of a step).
// Every CTA of a strip stays for as long as the strip takes, so waves of CTAs count whole.  A
// cluster's meeting adds 0.2 + 0.08 R of a step (measured on strips of 20011 and 65521 tokens: a
// step of 1.5 us alone grows to 1.9 with 2 CTAs, 2.7 with 8, 4.5 with 16), so with strips for all
// SMs R = 1 is best (256 strips of 2048 bf16 tokens: 38 us with 1, 46 with 2, 54 with 3), with
// fewer a larger one (80 strips: 239, 237, 177 us, and 251 with 4, whose CTAs need two waves; 16
// strips: 1373 us with 1, 296 with 8, 214 with 12, 244 with 16).
inline int cluster_size(long long strips, int segments, int warps, int per_sm) {
    const double room = (double)sm_count() * per_sm;
    const int tiles = (segments + warps - 1) / warps;
    const int most = warps == 8 ? 12 : kMaxCluster;  // (clusters of 96 warps or fewer find their place)
    int best = 1;
    double least = 0;
    for (int r = 1; r <= most && r <= tiles; ++r) {
        const double cost = std::ceil(strips * r / room) * ((tiles + r - 1) / r) *
                            (r > 1 ? 1.2 + 0.08 * r : 1.0);
        if (r == 1 || cost < 0.97 * least) {
            least = cost;
            best = r;
        }
    }
    return best;
}

// One launch of `warps` warps per CTA and t.cluster CTAs per strip.
template <typename K>
cudaError_t launch_strips(K kernel, const GatedArgs& a, const TileArgs& t, int warps, int smem,
                          cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (t.cluster > 8) {  // beyond the portable size
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((long long)t.strips * a.batch * t.cluster));
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = t.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a, t);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gated

// one translation unit per element type (backward: and gate form)
template <typename T> cudaError_t launch_gated_scan_as(const GatedArgs& a, cudaStream_t stream);
template <typename T, bool LOGIT>
cudaError_t launch_gated_scan_bwd_as(const GatedArgs& a, cudaStream_t stream);

}  // namespace ssd
