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
constexpr uint32_t kAll = (1u << kSeg) - 1;  // every token of a segment
constexpr int kTile = kWarps * kSeg;       // tokens per CTA and step
constexpr int kTileThreads = 32 * kWarps;
constexpr int kRowBytes = 128;             // a token's channels of one warp
constexpr int kMaxCluster = 8;
static_assert(kTile == kSpan, "the backward starts every tile from a saved state");

// ---------------------------------------------------------------------------------------
// the channels of one token and lane: one 32-bit word, so that a warp's row is 128 bytes
// ---------------------------------------------------------------------------------------
template <typename T> struct Pack;
template <> struct Pack<float> {
    static constexpr uint32_t kInf = 0x7f800000u;
    static __device__ __forceinline__ Vec<1> get(uint32_t r) { return {__uint_as_float(r)}; }
    static __device__ __forceinline__ uint32_t put(Vec<1> f) { return __float_as_uint(f.x); }
};
template <> struct Pack<__half> {
    static constexpr uint32_t kInf = 0x7c007c00u;
    static __device__ __forceinline__ Vec<2> get(uint32_t r) {
        return {__half22float2(*reinterpret_cast<const __half2*>(&r))};
    }
    static __device__ __forceinline__ uint32_t put(Vec<2> f) {
        const __half2 v = __floats2half2_rn(f.x.x, f.x.y);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
};
template <> struct Pack<__nv_bfloat16> {
    static constexpr uint32_t kInf = 0x7f807f80u;
    static __device__ __forceinline__ Vec<2> get(uint32_t r) {
        return {make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u))};
    }
    static __device__ __forceinline__ uint32_t put(Vec<2> f) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f.x.x, f.x.y);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
};

// Row pointers may be aligned to less than that word, and the last strip may be narrower: `whole`
// (the same in all lanes) says that neither is so; `count` is how many of the lane's channels exist.
template <typename T>
__device__ __forceinline__ void store_row(char* p, Vec<kChannels<T>> f, bool whole, int count) {
    const uint32_t r = Pack<T>::put(f);
    if (whole) {
        *reinterpret_cast<uint32_t*>(p) = r;
    } else if (sizeof(T) == 2) {
        uint16_t* h = reinterpret_cast<uint16_t*>(p);
        if (count > 0) h[0] = static_cast<uint16_t>(r);
        if (count > 1) h[1] = static_cast<uint16_t>(r >> 16);
    } else if (count > 0) {
        *reinterpret_cast<uint32_t*>(p) = r;
    }
}

template <int V>
__device__ __forceinline__ void store_bytes(uint8_t* p, const int (&q)[V], bool whole, int count) {
    if (V == 2 && whole) {
        *reinterpret_cast<uint16_t*>(p) =
            static_cast<uint16_t>((q[0] & 0xff) | (q[V - 1] & 0xff) << 8);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < count) p[v] = static_cast<uint8_t>(q[v]);
    }
}

// Floats of the lane's channels; 0 from a null pointer and for channels that do not exist.
template <int V>
__device__ __forceinline__ Vec<V> load_floats(const float* p, int count) {
    Vec<V> f;
#pragma unroll
    for (int v = 0; v < V; ++v) f.set(v, p && v < count ? p[v] : 0.f);
    return f;
}

template <int V>
__device__ __forceinline__ void store_floats(float* p, Vec<V> f, int count) {
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
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
        constexpr int kPer = W / 16;   // pieces per row
        constexpr int kStep = 32 / kPer;  // rows per instruction
        const int row = lane / kPer, at = lane % kPer * 16;
        const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(to)) + row * W + at;
        const char* p = src + row * pitch + at;
        if (rows == kSeg && width >= W) {
#pragma unroll
            for (int i = 0; i < kSeg / kStep; ++i) {
                copy_async16(d + i * kStep * W, p);
                p += kStep * pitch;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kSeg / kStep; ++i) {
                const int bytes = row + i * kStep < rows ? max(0, min(16, width - at)) : 0;
                copy_async16(d + i * kStep * W, bytes ? p : src, bytes);
                p += kStep * pitch;
            }
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
template <int V> struct Map {
    Vec<V> A, B;
    Vec<V> L;  // V == 1 only: fp32 tensors carry decays as two floats
};

template <int V> __device__ __forceinline__ Map<V> identity_map() {
    return {splat<V>(1.f), splat<V>(0.f), splat<V>(0.f)};
}

template <bool PACKED, int V>
__device__ __forceinline__ Vec<V> through(const Map<V>& m, Vec<V> carry) {
    Vec<V> r = step(m.A, m.L, carry, m.B);
    if constexpr (PACKED) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (m.A[v] < 0.f) r.set(v, m.B[v]);
    }
    return r;
}

// The decay product of a run followed by one more decay (B is the caller's).
__device__ __forceinline__ void extend(Map<1>& m, const Decay<1>& d) {
    const Vec<1> p = mul(m.A, d.a);
    m.L = fma(m.A, d.lo, fma(m.L, d.a, fma(m.A, d.a, sub(splat<1>(0.f), p))));
    m.A = p;
}
__device__ __forceinline__ void extend(Map<2>& m, const Decay<2>& d) { m.A = mul(m.A, d.a); }

// first, then second
template <bool PACKED, int V>
__device__ __forceinline__ Map<V> join(const Map<V>& first, const Map<V>& second) {
    Map<V> r = first;
    r.B = through<PACKED>(second, first.B);
    extend(r, Decay<V>{second.A, second.L, second.A});
    if constexpr (PACKED) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (first.A[v] < 0.f || second.A[v] < 0.f) r.A.set(v, -1.f);
    }
    return r;
}

// ---------------------------------------------------------------------------------------
// clusters
// ---------------------------------------------------------------------------------------
// All threads of all CTAs of the cluster meet.  Only the threads that sent maps release: a release
// waits for every write the thread has in flight, its rows of the last step included.
__device__ __forceinline__ void cluster_barrier(bool sent) {
    if (sent) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    else asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Address of this CTA's shared-memory word `p` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote_smem(const void* p, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(r) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    return r;
}

__device__ __forceinline__ void store_remote(uint32_t addr, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y),
                 "f"(v.z), "f"(v.w)
                 : "memory");
}

// Maps of runs, [run][lane] as four floats each: A and B of two channels, or A, B and L of one.
template <int V>
struct MapSlots {
    static constexpr int kFloats = 4 * 32;  // per run

    static __device__ __forceinline__ float4 words(const Map<V>& m) {
        if constexpr (V == 1) return make_float4(m.A.x, m.B.x, m.L.x, 0.f);
        else return make_float4(m.A.x.x, m.A.x.y, m.B.x.x, m.B.x.y);
    }
    static __device__ __forceinline__ void write(float* s, int run, int lane, const Map<V>& m) {
        *reinterpret_cast<float4*>(s + run * kFloats + lane * 4) = words(m);
    }
    static __device__ __forceinline__ Map<V> read(const float* s, int run, int lane) {
        const float4 w = *reinterpret_cast<const float4*>(s + run * kFloats + lane * 4);
        Map<V> m;
        if constexpr (V == 1) {
            m.A.x = w.x;
            m.B.x = w.y;
            m.L.x = w.z;
        } else {
            m.A.x = make_float2(w.x, w.y);
            m.B.x = make_float2(w.z, w.w);
            m.L = splat<V>(0.f);
        }
        return m;
    }
    static __device__ __forceinline__ void send(const float* s, int run, int lane, int rank,
                                                const Map<V>& m) {
        store_remote(remote_smem(s + run * kFloats + lane * 4, rank), words(m));
    }
    // The map of a whole tile: its warps' runs, written in the order of the recurrence.
    template <bool PACKED>
    static __device__ __forceinline__ Map<V> join_runs(const float* s, int lane) {
        Map<V> all = read(s, 0, lane);
#pragma unroll
        for (int i = 1; i < kWarps; ++i) all = join<PACKED>(all, read(s, i, lane));
        return all;
    }
    // `carry` through runs 0 .. n - 1; returns what run `which` receives.
    template <bool PACKED>
    static __device__ __forceinline__ Vec<V> carry_through(const float* s, int n, int which,
                                                           int lane, Vec<V>& carry) {
        Vec<V> mine = carry;
        for (int i = 0; i < n; ++i) {
            if (i == which) mine = carry;
            carry = through<PACKED>(read(s, i, lane), carry);
        }
        return mine;
    }
    // h through the runs before `to`
    template <bool PACKED>
    static __device__ __forceinline__ Vec<V> carry_into(const float* s, int to, int lane, Vec<V> h) {
        for (int i = 0; i < to; ++i) h = through<PACKED>(read(s, i, lane), h);
        return h;
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
        m.valid = kAll;
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
