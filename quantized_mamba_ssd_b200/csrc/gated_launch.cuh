// Launches of the tile kernels: two channels per lane or one, and how many CTAs share a strip.
#pragma once

#include "gated_tile.cuh"

namespace ssd {
namespace gated {

constexpr int kFwdBlocks = 4;  // resident CTAs per SM the kernels are compiled for
constexpr int kBwdBlocks = 3;

struct Launch {
    int cluster;
    int strips;
    int tiles;
};

// CTAs per strip.  Every CTA of a strip runs for as long as the strip does, so what counts is how
// full the last wave of CTAs is; among equals the smallest cluster wins (fewest barriers' waits).
inline int cluster_size(long long units, int tiles, int blocks_per_sm) {
    static const int sms = [] {
        int dev = 0, n = 148;
        cudaGetDevice(&dev);
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        return n;
    }();
    const double room = (double)sms * blocks_per_sm;
    int best = 1;
    double most = 0;
    for (int r = 1; r <= kMaxCluster && (r == 1 || r <= tiles); r *= 2) {
        const double waves = units * r / room;
        const double full = waves / (waves <= 1 ? 1.0 : (double)(long long)(waves + 0.999999));
        if (full > most * 1.02) {
            most = full;
            best = r;
        }
    }
    return best;
}

template <typename K>
cudaError_t launch_tiles(K kernel, const GatedArgs& a, int V, int blocks_per_sm, cudaStream_t st) {
    const long long strips = (a.channels + 32LL * V - 1) / (32 * V), units = strips * a.batch;
    const int tiles = (a.seqlen + kTile - 1) / kTile;
    const int R = cluster_size(units, tiles, blocks_per_sm);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(units * R));
    cfg.blockDim = dim3(kTileThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = R;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, R);
    return e != cudaSuccess ? e : cudaGetLastError();
}

inline bool pairable(const GatedRows& r) {
    return !r.ptr || (reinterpret_cast<uintptr_t>(r.ptr) % 4 == 0 && r.batch_stride % 2 == 0 &&
                      r.token_stride % 2 == 0);
}

// Two 16-bit channels per lane wherever every row allows it (their codes then start at even
// elements, too).
inline bool two_channels(const GatedArgs& a) {
    auto even = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 2 == 0; };
    return a.io_dtype != SSD_IO_F32 && a.channels % 2 == 0 && pairable(a.x) && pairable(a.gate) &&
           pairable(a.y) && pairable(a.dy) && pairable(a.dx) && pairable(a.dgate) && even(a.x_q) &&
           even(a.x_e) && even(a.gate_q) && even(a.gate_e);
}

}  // namespace gated

// one translation unit per element type
template <typename T> cudaError_t launch_gated_scan_as(const GatedArgs& a, cudaStream_t stream);
template <typename T> cudaError_t launch_gated_scan_bwd_as(const GatedArgs& a, cudaStream_t stream);

}  // namespace ssd
