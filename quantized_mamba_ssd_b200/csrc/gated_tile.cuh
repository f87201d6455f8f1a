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
constexpr int kMaxCluster = 8;
static_assert(kTile == kSpan, "the backward starts every tile from a saved state");

// ---------------------------------------------------------------------------------------
// V channels of one token
// ---------------------------------------------------------------------------------------
template <typename T, int V> struct Pack;
template <> struct Pack<float, 1> {
    using Raw = uint32_t;
    static constexpr Raw kInf = 0x7f800000u;
    static __device__ __forceinline__ void get(Raw r, float (&f)[1]) { f[0] = __uint_as_float(r); }
    static __device__ __forceinline__ Raw put(const float (&f)[1]) { return __float_as_uint(f[0]); }
};
template <> struct Pack<__half, 1> {
    using Raw = uint16_t;
    static constexpr Raw kInf = 0x7c00u;
    static __device__ __forceinline__ void get(Raw r, float (&f)[1]) {
        f[0] = __half2float(__ushort_as_half(r));
    }
    static __device__ __forceinline__ Raw put(const float (&f)[1]) {
        return __half_as_ushort(__float2half_rn(f[0]));
    }
};
template <> struct Pack<__nv_bfloat16, 1> {
    using Raw = uint16_t;
    static constexpr Raw kInf = 0x7f80u;
    static __device__ __forceinline__ void get(Raw r, float (&f)[1]) {
        f[0] = __uint_as_float((uint32_t)r << 16);
    }
    static __device__ __forceinline__ Raw put(const float (&f)[1]) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    }
};
template <> struct Pack<__half, 2> {
    using Raw = uint32_t;
    static constexpr Raw kInf = 0x7c007c00u;
    static __device__ __forceinline__ void get(Raw r, float (&f)[2]) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&r));
        f[0] = v.x;
        f[1] = v.y;
    }
    static __device__ __forceinline__ Raw put(const float (&f)[2]) {
        const __half2 v = __floats2half2_rn(f[0], f[1]);
        return *reinterpret_cast<const Raw*>(&v);
    }
};
template <> struct Pack<__nv_bfloat16, 2> {
    using Raw = uint32_t;
    static constexpr Raw kInf = 0x7f807f80u;
    static __device__ __forceinline__ void get(Raw r, float (&f)[2]) {
        f[0] = __uint_as_float(r << 16);
        f[1] = __uint_as_float(r & 0xffff0000u);
    }
    static __device__ __forceinline__ Raw put(const float (&f)[2]) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[0], f[1]);
        return *reinterpret_cast<const Raw*>(&v);
    }
};

// int8 codes of V channels
template <int V> struct CodeRaw;
template <> struct CodeRaw<1> { using Raw = uint8_t; };
template <> struct CodeRaw<2> { using Raw = uint16_t; };

template <int V>
__device__ __forceinline__ typename CodeRaw<V>::Raw put_codes(const int (&q)[V]) {
    uint32_t r = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) r |= (static_cast<uint32_t>(q[v]) & 0xffu) << (8 * v);
    return static_cast<typename CodeRaw<V>::Raw>(r);
}

template <typename R>
__device__ __forceinline__ R load_once(const R* p) {
    return __ldg(p);
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
