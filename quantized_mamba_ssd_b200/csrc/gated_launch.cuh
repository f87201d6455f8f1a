// Launches of the scan kernels: alignments, and into how many chunks a strip is cut.
#pragma once

#include <algorithm>
#include <atomic>

#include "gated_tile.cuh"
#include "per_device.h"

namespace ssd {
namespace gated {

// Warps of a CTA and CTAs per SM.  Forward, 8 warps and 128 registers: with 4 warps twice as many
// steps, each with a barrier (256 strips of 2048 bf16 tokens: 38 us, with 4 warps 48).  Backward,
// 168 registers: 4 warps fit three times, 8 only once (63 us, 81); segments from codes are smaller,
// 8 warps of them fit twice, with 128 registers (66 us, with 4 warps 89).
constexpr int kFwdWarps = 8, kFwdBlocks = 2;
template <bool CKPT> constexpr int kBwdWarps = CKPT ? 8 : 4;
template <bool CKPT> constexpr int kBwdBlocks = CKPT ? 2 : 3;
constexpr int kMapWarps = 8;  // of the kernel that leaves the chunks' maps
constexpr int kMaxChunks = 64;

struct TileArgs {
    int strips;       // strips per row
    int blocks;       // segments (checkpoint blocks) per row
    int spans;        // spans per row
    int chunks;       // CTAs per strip
    int chunk_tiles;  // tiles of a chunk (the last one's may be fewer)
    float* maps;      // workspace: [strip of all rows][chunk][map of 32 lanes]
    bool aligned;     // every input's rows start at multiples of 16 bytes
    // outputs are written as whole words (codes: pairs of bytes): aligned, and no lane has a part
    bool whole_out, whole_codes;
};

// What the start of every row is a multiple of.
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
    // (16 for an input that the call does not have)
    int least = std::min({alignment(a.x, elem), alignment(a.gate, elem), alignment(a.dy, elem)});
    t.whole_out = a.channels % V == 0 && word_rows(a.y, elem) && word_rows(a.dx, elem) &&
                  word_rows(a.dgate, elem);
    auto all = [](auto... p) { return (reinterpret_cast<uintptr_t>(p) | ...); };
    if (a.x_q && !a.x.ptr)  // backward from codes, rows of one byte per channel
        least = std::min({least, alignment({a.x_q, 0, a.channels}, 1), alignment({a.gate_q, 0, a.channels}, 1)});
    t.aligned = least == 16;
    t.whole_codes = (all(a.x_q, a.gate_q, a.x_e, a.gate_e) | a.channels) % 2 == 0;
    return t;
}

// SMs of the current device (148 where none can be asked: the size of a workspace without a GPU).
inline int sm_count() {
    static PerDevice sms;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
    return sms.get(dev, 148, [](int d) {
        int n = 0;
        return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d) == cudaSuccess ? n : 0;
    });
}

struct Chunks {
    int count, tiles;  // chunks per strip, tiles per chunk
};

// Chunks per strip: the count with the least time by a model in steps of the scan (1.4 to 2 us, from
// and to codes 2 to 4).  A scan of S chunks takes ceil(tiles / S) steps and one to begin, times its
// CTAs per place (and about 0.4 of the last wave's gaps), and its steps are 1.4 times as long with
// the SMs full as with them empty; with S > 1 the maps before it take 0.85 of that again, and the
// second launch and its start about 4 steps (2 of the longer ones of rows that are not aligned).
// Beside the longer steps of a scan from or to codes both are less.  Only the counts that fill one
// to four waves are looked at.
// Measured, whole and in S chunks: forward 16 strips of 512 fp16 tiles 726 us, 133 (S = 18); 40 of
// 64 tiles 85, 41 (7); 80 of 157 bf16 tiles 200, 186 (3), 182 (8); 128 of 32 tiles 44, 53 (2), rows of
// 4090 channels 65, 80 (2); 75 of 10 fp32 tiles 19.0, 19.4 (4).  Forward with codes, 48 bf16 strips
// of 4 tiles 11.6, 8.7 (4); 128 of 32 tiles 77, 82 (2).  Backward from codes 13.2, 9.3 and 102, 97;
// 75 of 10 fp32 tiles 37, 32 (4).
// Shapes that the constants were not set on (11 strips of 24 tiles, 50 of 79, 60 of 235, 105 of 7, 210 of
// 47, 4 of 938, 270 of 20, 119 of 4, fp32 40 of 40 and 10 of 12; forward and backward, with codes and
// without), against the best of 19 counts each: within 3 % for 35 of the 40, the others 5, 6, 9, 10
// (backward of 105 strips of 7 tiles, left whole) and 12 % (backward from codes of 60 strips).
enum class Work { kPlain, kToCodes, kFromCodes };
inline Chunks chunks_of(Work work, long long strips, int segments, int warps, int per_sm, int sms,
                        bool aligned) {
    const long long room = (long long)sms * per_sm;
    const int tiles = (segments + warps - 1) / warps;
    const double maps = work == Work::kPlain ? 1.85 : work == Work::kToCodes ? 1.6 : 1.4;
    const double second = work == Work::kPlain ? (aligned ? 4 : 2) : work == Work::kToCodes && !aligned ? 0 : 1;
    auto time = [&](int s, int each) {
        const double full = (double)(strips * s) / room;
        const double scan = (full <= 1 ? 1 : full + 0.4) * (each + 1) * (1 + 0.4 * (full < 1 ? full : 1));
        return s == 1 ? scan : scan * maps + second;
    };
    Chunks best{1, tiles};
    double least = time(1, tiles);
    for (int waves = 1; waves <= 4; ++waves) {
        const long long most = std::min<long long>({waves * room / strips, kMaxChunks, tiles});
        if (most < 2) continue;
        const int each = (tiles + (int)most - 1) / (int)most;
        const int s = (tiles + each - 1) / each;  // no chunk is empty
        const double cost = time(s, each);
        if (s > 1 && cost < 0.97 * least) {
            least = cost;
            best = {s, each};
        }
    }
    return best;
}

// Launches `kernel` with all of an SM's shared memory allowed (asked for once per device; nothing
// here allocates or throws).  `follows`: the launch may begin while the one before it on the stream
// ends (the kernel waits for it where it needs its results).
template <auto kernel, typename... A>
cudaError_t launch_ctas(long long ctas, int warps, int smem, bool follows, cudaStream_t st, A... args) {
    constexpr int kMost = 227 << 10, kDevices = 64;
    static std::atomic<uint64_t> allowed{0};  // bit: device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < kDevices ? 1ull << dev : 0;
    if (!(allowed.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (e != cudaSuccess) return e;
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = follows ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gated

// one translation unit per element type (backward: and gate form)
template <typename T> cudaError_t launch_gated_scan_as(const GatedArgs& a, cudaStream_t stream);
template <typename T, bool LOGIT>
cudaError_t launch_gated_scan_bwd_as(const GatedArgs& a, cudaStream_t stream);

}  // namespace ssd
