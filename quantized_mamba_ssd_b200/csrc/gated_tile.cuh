// What the forward and the backward scan share: the tile, the joins of its parts, the loads.
//
// A cluster of R CTAs takes one strip of 32 * V channels of one row and walks its tokens in steps
// of R tiles, one tile of 64 tokens per CTA, one segment of 16 tokens per warp, V channels per
// lane.  A thread reduces its segment to the affine map carry -> A carry + B; the maps of a tile
// meet in shared memory, those of a step are sent to every CTA of the cluster (distributed shared
// memory), and each thread then computes the carry into its own segment and, redundantly, the
// carry into the next step.  So a step costs one cluster barrier, every input is read once, no
// CTA waits on memory flags, and the order of all sums is fixed.
#pragma once

#include "gated.cuh"
#include "gated_kernels.h"

namespace ssd {
namespace gated {

constexpr int kWarps = 4;
constexpr int kSeg = kBlock;               // tokens per warp: a checkpoint block stays in a thread
constexpr int kTile = kWarps * kSeg;       // tokens per CTA and step
constexpr int kTileThreads = 32 * kWarps;
constexpr int kRowBytes = 128;             // a token's channels of one warp
constexpr int kMaxCluster = 8;
static_assert(kTile == kSpan, "the backward starts every tile from a saved state");

// ---------------------------------------------------------------------------------------
// the channels of one token and lane: one 32-bit word, so that a warp's row is 128 bytes
// ---------------------------------------------------------------------------------------
template <typename T> constexpr int kChannels = 4 / sizeof(T);

template <typename T> struct Pack;
template <> struct Pack<float> {
    static __device__ __forceinline__ void get(uint32_t r, float (&f)[1]) { f[0] = __uint_as_float(r); }
    static __device__ __forceinline__ uint32_t put(const float (&f)[1]) { return __float_as_uint(f[0]); }
};
template <> struct Pack<__half> {
    static __device__ __forceinline__ void get(uint32_t r, float (&f)[2]) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&r));
        f[0] = v.x;
        f[1] = v.y;
    }
    static __device__ __forceinline__ uint32_t put(const float (&f)[2]) {
        const __half2 v = __floats2half2_rn(f[0], f[1]);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
};
template <> struct Pack<__nv_bfloat16> {
    static __device__ __forceinline__ void get(uint32_t r, float (&f)[2]) {
        f[0] = __uint_as_float(r << 16);
        f[1] = __uint_as_float(r & 0xffff0000u);
    }
    static __device__ __forceinline__ uint32_t put(const float (&f)[2]) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[0], f[1]);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
};

// Row pointers may be aligned to less than that word: `pair` says that every output row of the
// call is, and `count` is how many of the lane's channels exist (0 behind the last one).
template <typename T>
__device__ __forceinline__ void store_row(T* p, const float (&f)[kChannels<T>], bool pair, int count) {
    const uint32_t r = Pack<T>::put(f);
    if (pair && count == kChannels<T>) {
        *reinterpret_cast<uint32_t*>(p) = r;
    } else {
        uint16_t* h = reinterpret_cast<uint16_t*>(p);
        if (sizeof(T) == 2 && count > 0) h[0] = static_cast<uint16_t>(r);
        if (sizeof(T) == 2 && count > 1) h[1] = static_cast<uint16_t>(r >> 16);
    }
}

template <int V>
__device__ __forceinline__ void store_bytes(uint8_t* p, const int (&q)[V], bool pair, int count) {
    if (V == 2 && pair && count == 2) {
        *reinterpret_cast<uint16_t*>(p) =
            static_cast<uint16_t>((q[0] & 0xff) | (q[V - 1] & 0xff) << 8);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < count) p[v] = static_cast<uint8_t>(q[v]);
    }
}

template <int V>
__device__ __forceinline__ void load_floats(const float* p, float (&f)[V], int count) {
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = p && v < count ? p[v] : 0.f;
}

template <int V>
__device__ __forceinline__ void store_floats(float* p, const float (&f)[V], int count) {
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (v < count) p[v] = f[v];
}

// ---------------------------------------------------------------------------------------
// asynchronous copies of a warp's segment, kSeg rows of W bytes, into its own shared memory
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows at src + j * pitch (bytes); rows from `rows` on and bytes from `width` on become 0 and are
// not read.  `align` is what base and pitch are multiples of: 16, 4, or less.
template <int W>
__device__ __forceinline__ void stage_rows(void* dst, const char* src, long long pitch, int rows,
                                           int width, int align) {
    const int lane = threadIdx.x & 31;
    char* to = static_cast<char*>(dst);
    if (align == 16) {
        constexpr int kPer = W / 16;  // pieces per row
#pragma unroll
        for (int i = 0; i < kSeg * kPer / 32; ++i) {
            const int row = (lane + 32 * i) / kPer, at = (lane + 32 * i) % kPer * 16;
            const int bytes = row < rows ? max(0, min(16, width - at)) : 0;
            copy_async16(static_cast<uint32_t>(__cvta_generic_to_shared(to + row * W + at)),
                         bytes ? src + row * pitch + at : src, bytes);
        }
    } else if (align == 4) {
        constexpr int kPer = W / 4;
#pragma unroll
        for (int i = 0; i < kSeg * kPer / 32; ++i) {
            const int row = (lane + 32 * i) / kPer, at = (lane + 32 * i) % kPer * 4;
            const int bytes = row < rows ? max(0, min(4, width - at)) : 0;
            copy_async4(static_cast<uint32_t>(__cvta_generic_to_shared(to + row * W + at)),
                        bytes ? src + row * pitch + at : src, bytes);
        }
    } else if (align == 2) {
        constexpr int kPer = W / 2;
#pragma unroll 16
        for (int i = 0; i < kSeg * kPer / 32; ++i) {
            const int row = (lane + 32 * i) / kPer, at = (lane + 32 * i) % kPer * 2;
            const bool in = row < rows && at < width;
            *reinterpret_cast<uint16_t*>(to + row * W + at) =
                in ? __ldg(reinterpret_cast<const uint16_t*>(src + row * pitch + at)) : uint16_t(0);
        }
    } else {
#pragma unroll 16
        for (int i = 0; i < kSeg * W / 32; ++i) {
            const int row = (lane + 32 * i) / W, at = (lane + 32 * i) % W;
            const bool in = row < rows && at < width;
            to[row * W + at] = in ? __ldg(src + row * pitch + at) : char(0);
        }
    }
}

// ---------------------------------------------------------------------------------------
// the affine map of a run of tokens, carry -> (A + L) carry + B
// ---------------------------------------------------------------------------------------
// In packed rows A < 0 marks a run in which a sequence begins (or, backward, ends): the carry is
// dropped by a selection, not by a factor 0, so that what another sequence left in it (infinities
// and NaN included) cannot come through.
template <bool TWO> struct Map;
template <> struct Map<false> {
    float A, B;
};
template <> struct Map<true> {
    float A, B, L;
};

template <bool TWO>
__device__ __forceinline__ Map<TWO> identity_map() {
    Map<TWO> m;
    m.A = 1.f;
    m.B = 0.f;
    if constexpr (TWO) m.L = 0.f;
    return m;
}

template <bool TWO, bool PACKED>
__device__ __forceinline__ float through(const Map<TWO>& m, float carry) {
    float b = m.B;
    if constexpr (TWO) b = fmaf(m.L, carry, b);
    const float r = fmaf(m.A, carry, b);
    return PACKED && m.A < 0.f ? m.B : r;
}

// The decay product of a run followed by one more decay (B is the caller's).
template <bool TWO>
__device__ __forceinline__ void extend(Map<TWO>& m, const Decay& d) {
    const float p = m.A * d.a;
    if constexpr (TWO) m.L = fmaf(m.A, d.lo, fmaf(m.L, d.a, fmaf(m.A, d.a, -p)));
    m.A = p;
}

// first, then second
template <bool TWO, bool PACKED>
__device__ __forceinline__ Map<TWO> join(const Map<TWO>& first, const Map<TWO>& second) {
    Map<TWO> r;
    r.B = through<TWO, PACKED>(second, first.B);
    const float p = first.A * second.A;
    r.A = p;
    if constexpr (TWO)
        r.L = fmaf(first.A, second.L, fmaf(first.L, second.A, fmaf(first.A, second.A, -p)));
    if (PACKED && (first.A < 0.f || second.A < 0.f)) r.A = -1.f;
    return r;
}

// ---------------------------------------------------------------------------------------
// clusters
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
}

// Address of this CTA's shared-memory word `p` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote_smem(const void* p, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(r) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    return r;
}

__device__ __forceinline__ void store_remote(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Maps of `n` runs, [n][floats of a map][32 * V]: lanes read and write consecutive words.
template <int V, bool TWO>
struct MapSlots {
    static constexpr int kWords = TWO ? 3 : 2;
    static constexpr int kFloats = kWords * 32 * V;  // per run

    static __device__ __forceinline__ void write(float* s, int run, int lane, const Map<TWO> (&m)[V]) {
        float* p = s + run * kFloats + lane;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            p[(v * kWords + 0) * 32] = m[v].A;
            p[(v * kWords + 1) * 32] = m[v].B;
            if constexpr (TWO) p[(v * kWords + 2) * 32] = m[v].L;
        }
    }
    static __device__ __forceinline__ void read(const float* s, int run, int lane, Map<TWO> (&m)[V]) {
        const float* p = s + run * kFloats + lane;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            m[v].A = p[(v * kWords + 0) * 32];
            m[v].B = p[(v * kWords + 1) * 32];
            if constexpr (TWO) m[v].L = p[(v * kWords + 2) * 32];
        }
    }
    static __device__ __forceinline__ void send(const float* s, int run, int lane, int rank,
                                                const Map<TWO> (&m)[V]) {
        const uint32_t p = remote_smem(s + run * kFloats + lane, rank);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            store_remote(p + (v * kWords + 0) * 128, m[v].A);
            store_remote(p + (v * kWords + 1) * 128, m[v].B);
            if constexpr (TWO) store_remote(p + (v * kWords + 2) * 128, m[v].L);
        }
    }
    // The map of a whole tile: its warps' runs, written in the order of the recurrence.
    template <bool PACKED>
    static __device__ __forceinline__ void join_runs(const float* s, int lane, Map<TWO> (&all)[V]) {
        read(s, 0, lane, all);
#pragma unroll
        for (int i = 1; i < kWarps; ++i) {
            Map<TWO> m[V];
            read(s, i, lane, m);
#pragma unroll
            for (int v = 0; v < V; ++v) all[v] = join<TWO, PACKED>(all[v], m[v]);
        }
    }
    // `carry` through runs 0 .. n - 1; `mine` is what run `which` receives.
    template <bool PACKED>
    static __device__ __forceinline__ void carry_through(const float* s, int n, int which, int lane,
                                                         float (&carry)[V], float (&mine)[V]) {
        for (int i = 0; i < n; ++i) {
            Map<TWO> m[V];
            read(s, i, lane, m);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (i == which) mine[v] = carry[v];
                carry[v] = through<TWO, PACKED>(m[v], carry[v]);
            }
        }
    }
    // h through the runs before `to`
    template <bool PACKED>
    static __device__ __forceinline__ void carry_into(const float* s, int to, int lane,
                                                      float (&h)[V]) {
        for (int i = 0; i < to; ++i) {
            Map<TWO> m[V];
            read(s, i, lane, m);
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = through<TWO, PACKED>(m[v], h[v]);
        }
    }
};

// ---------------------------------------------------------------------------------------
// where the tokens of a segment stand in packed rows
// ---------------------------------------------------------------------------------------
// Bit j is token t0 + j.  `held` keeps the bounds of the last sequence met: a segment inside it
// needs no search.
struct Marks {
    uint32_t valid, begin, end;  // in a sequence; its first token; its last token
    int seq;                     // lane j < kSeg: the sequence of token t0 + j
};

struct Held {
    int seq = -1, from = 0, to = 0;
};

__device__ __forceinline__ Marks marks_of(const int32_t* __restrict__ cu, int nseq, int t0, int n,
                                          Held& held) {
    Marks m;
    const int lane = threadIdx.x & 31;
    if (n == kSeg && t0 > held.from && t0 + kSeg < held.to) {
        m.valid = (1u << kSeg) - 1;
        m.begin = m.end = 0;
        m.seq = held.seq;
        return m;
    }
    const int t = t0 + lane;
    int s = -1, from = 0, to = 0;
    if (lane < n) {
        s = sequence_of(cu, nseq, t);
        if (s >= 0) {
            from = __ldg(cu + s);
            to = __ldg(cu + s + 1);
        }
    }
    m.valid = __ballot_sync(0xffffffffu, s >= 0);
    m.begin = __ballot_sync(0xffffffffu, s >= 0 && t == from);
    m.end = __ballot_sync(0xffffffffu, s >= 0 && t + 1 == to);
    m.seq = s;
    // the sequence of the segment's middle token is as good a guess as any for the next segment
    const int src = kSeg / 2;
    held.seq = __shfl_sync(0xffffffffu, s, src);
    held.from = __shfl_sync(0xffffffffu, from, src);
    held.to = __shfl_sync(0xffffffffu, to, src);
    return m;
}

}  // namespace gated
}  // namespace ssd
