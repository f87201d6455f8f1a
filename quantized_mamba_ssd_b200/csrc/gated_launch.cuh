// Launches of the tile kernels: alignments, and how many CTAs share a strip.
#pragma once

#include <cmath>

#include "gated_tile.cuh"

namespace ssd {
namespace gated {

constexpr int kFwdBlocks = 4;  // resident CTAs per SM the kernels are compiled for
constexpr int kBwdBlocks = 3;
constexpr int kFwdStages = 2;  // segments in shared memory per warp: the current one and the next
constexpr int kBwdStages = 2;

struct TileArgs {
    int cluster;  // CTAs per strip
    int strips;   // strips of 32 lanes per row
    int blocks;   // checkpoint blocks per row
    // what the start of every row is a multiple of (bytes): 16, 4, 2 or 1
    int align_x, align_gate, align_dy, align_codes;
    int pair_out, pair_codes;  // outputs can be written as whole words (codes: pairs of bytes)
};

inline int alignment(const GatedRows& r, int elem) {
    const unsigned long long all = reinterpret_cast<uintptr_t>(r.ptr) |
                                   (unsigned long long)r.batch_stride * elem |
                                   (unsigned long long)r.token_stride * elem;
    return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : elem;
}

inline bool word_rows(const GatedRows& r, int elem) { return !r.ptr || alignment(r, elem) >= 4; }

// CTAs per strip.  Every CTA of a strip runs for as long as the strip does, so what counts is how
// full the last wave of CTAs is; among equals the smallest cluster wins (fewest to wait for).
inline int cluster_size(long long units, int tiles, int blocks_per_sm) {
    static const int sms = [] {
        int dev = 0, n = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
            n = 148;
        return n;
    }();
    const double room = (double)sms * blocks_per_sm;
    int best = 1;
    double most = 0;
    for (int r = 1; r <= kMaxCluster && (r == 1 || r <= tiles); ++r) {
        const double waves = units * r / room;
        const double full = waves <= 1 ? waves : waves / std::ceil(waves);
        if (full > most * 1.02) {
            most = full;
            best = r;
        }
    }
    return best;
}

template <typename T, typename K>
cudaError_t launch_tiles(K kernel, const GatedArgs& a, int blocks_per_sm, int smem, cudaStream_t st) {
    constexpr int elem = sizeof(T), V = kChannels<T>;
    const int tiles = (a.seqlen + kTile - 1) / kTile;
    TileArgs t{};
    t.strips = (a.channels + 32 * V - 1) / (32 * V);
    t.blocks = (a.seqlen + kBlock - 1) / kBlock;
    const long long units = (long long)t.strips * a.batch;
    t.cluster = cluster_size(units, tiles, blocks_per_sm);
    t.align_x = alignment(a.x, elem);
    t.align_gate = alignment(a.gate, elem);
    t.align_dy = alignment(a.dy, elem);
    t.pair_out = word_rows(a.y, elem) && word_rows(a.dx, elem) && word_rows(a.dgate, elem);
    const uintptr_t codes = reinterpret_cast<uintptr_t>(a.x_q) | reinterpret_cast<uintptr_t>(a.gate_q) |
                            a.channels;
    t.align_codes = codes % 16 == 0 ? 16 : codes % 4 == 0 ? 4 : codes % 2 == 0 ? 2 : 1;
    t.pair_codes = (codes | reinterpret_cast<uintptr_t>(a.x_e) | reinterpret_cast<uintptr_t>(a.gate_e)) % 2 == 0;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(units * t.cluster));
    cfg.blockDim = dim3(kTileThreads);
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
