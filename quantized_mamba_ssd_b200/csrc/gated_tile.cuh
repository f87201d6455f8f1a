// What the forward and the backward scan share: the walk along a strip, the joins of its parts, the
// copies.
//
// A strip is the channels of 32 lanes (128 bytes of a token).  The W warps of a CTA share a strip
// and walk it in steps of W segments of 16 tokens: each warp reduces its segment to the affine map
// carry -> A carry + B, the maps meet in shared memory, and each warp then computes the carry into
// its own segment - and, redundantly, the carry into the next step.  Inputs are copied ahead
// asynchronously, each warp's own segments into its own shared memory, and are read once.
//
// With too few strips for the machine a strip is cut into chunks of tokens with a CTA each.  A
// kernel before the scan then walks all chunks but the last one of each strip (no meetings: a warp
// reduces a run of tokens to its map as it streams by) and leaves their maps in the workspace,
// where the scan composes the carry into its chunk.  That reads two of the inputs twice, often from
// the L2 cache; the alternatives cost more: in a cluster whose CTAs share a strip every step waits
// for a meeting of them all (a step of 1.5 us became 2.9 us with 3 CTAs and 4.8 us with 12).
// The order of all sums is fixed, and no CTA waits for another.
#pragma once

#include <type_traits>

#include "gated.cuh"
#include "gated_kernels.h"

namespace ssd {
namespace gated {

constexpr int kSub = kBlock;                 // tokens of a segment: one checkpoint block
constexpr uint32_t kAll = (1u << kSub) - 1;  // each of them
constexpr int kRowBytes = 128;  // a token's channels of one warp

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

// Row pointers may be aligned to less than that word, and a lane may have some of its channels only:
// `whole` (the same in all lanes) says that neither is so; `count` is how many of the lane's
// channels exist.
template <typename T>
__device__ __forceinline__ void store_row(char* p, Vec<kChannels<T>> f, bool whole, int count) {
    const uint32_t r = Pack<T>::put(f);
    if (whole) {
        if (count) *reinterpret_cast<uint32_t*>(p) = r;
    } else if (sizeof(T) == 2) {
        uint16_t* h = reinterpret_cast<uint16_t*>(p);
        if (count > 0) h[0] = static_cast<uint16_t>(r);
        if (count > 1) h[1] = static_cast<uint16_t>(r >> 16);
    } else if (count > 0) {
        *reinterpret_cast<uint32_t*>(p) = r;
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
// asynchronous copies of kSub rows of W bytes into a warp's own shared memory
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int AHEAD> __device__ __forceinline__ void copy_wait() {  // all but the last AHEAD commits
    asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD) : "memory");
}

// Rows whose starts are all multiples of 16 bytes (ANY false) are staged at a pitch of W bytes, from
// the start of their place.  Other rows (ANY) are copied as the aligned 16-byte pieces of memory
// that hold their bytes, so each stands at its address modulo 16.  With a pitch that is that of
// memory modulo 16 (and leaves the pieces of two rows apart), they still stand at even distances,
// and a lane's value of row j is at one offset plus j pitches (of 16-bit rows in two halves).
// Nothing but pieces that hold bytes of the rows is read.  Kernels of their own keep the others'
// loop small.  (2 x 4096 bf16 tokens of 4096, 4090 and 4095 channels: forward 40, 56 and 70 us,
// backward 73, 97 and 112; copied in 4-byte words 72 and 134, moved in shared memory to the start
// of their place 110 and 169.)
template <int W, bool ANY> constexpr int kSubBytes = kSub * (ANY ? W + 32 : W);  // room for kSub rows

template <int W, bool ANY> __device__ __forceinline__ int staged_pitch(long long pitch) {
    return ANY ? W + 16 + static_cast<int>(pitch & 15) : W;
}
template <bool ANY> __device__ __forceinline__ int staged_start(const char* src) {
    return ANY ? static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15) : 0;
}

// The rows' bytes from `width` on, and rows from `rows` on, stay undefined (kernels give no lane
// and no token a meaning that has none).  What most calls do not run is out of line: it would push
// the hot loop out of the instruction cache.
template <int W, bool ANY>
__device__ __noinline__ void stage_part(void* dst, const char* src, long long pitch, int rows, int width) {
    const int lane = threadIdx.x & 31;
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    const int q = staged_pitch<W, ANY>(pitch), start = staged_start<ANY>(src);
    constexpr int kPer = W / 16 + ANY;  // pieces of a row
    for (int i = lane; i < rows * kPer; i += 32) {
        const int row = i / kPer, at = i % kPer * 16;
        const int place = start + row * q, shift = place & 15;
        const int bytes = min(16, shift + width - at);
        if (bytes > 0) copy_async16(to + (place - shift) + at, src + row * pitch - shift + at, bytes);
    }
}

// kSub whole rows at src + j * pitch (bytes).
template <int W, bool ANY>
__device__ __forceinline__ void stage_rows(void* dst, const char* src, long long pitch, int width) {
    constexpr int kPer = W / 16, kStep = 32 / kPer;  // pieces per row, rows per instruction
    const int lane = threadIdx.x & 31, row = lane / kPer, at = lane % kPer * 16;
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if constexpr (!ANY) {
        const int bytes = max(0, min(16, width - at));
        const uint32_t d = to + row * W + at;
        const char* p = bytes ? src + row * pitch + at : src;
        const long long by = bytes ? kStep * pitch : 0;
#pragma unroll
        for (int i = 0; i < kSub / kStep; ++i) {
            copy_async16(d + i * kStep * W, p, bytes);
            p += by;
        }
    } else {
        const int q = staged_pitch<W, true>(pitch), start = staged_start<true>(src);
        int place = start + row * q;
        unsigned long long from = reinterpret_cast<unsigned long long>(src + row * pitch);
        auto piece = [&](int place, unsigned long long from, int at) {
            const int bytes = max(0, min(16, (place & 15) + width - at));
            copy_async16(to + (place & ~15) + at,
                         reinterpret_cast<const char*>(from & ~15ull) + (bytes ? at : 0), bytes);
        };
#pragma unroll
        for (int i = 0; i < kSub / kStep; ++i) {
            piece(place, from, at);
            place += kStep * q;
            from += kStep * pitch;
        }
        if (lane < kSub)  // the last piece of each row
            piece(start + lane * q, reinterpret_cast<unsigned long long>(src + lane * pitch), W);
    }
}

// The lane's word of a staged row.
template <typename T, bool ANY> __device__ __forceinline__ uint32_t row_word(const uint8_t* r) {
    if constexpr (ANY && sizeof(T) == 2) {
        const uint32_t low = *reinterpret_cast<const uint16_t*>(r);
        return low | static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(r + 2)) << 16;
    } else {
        return *reinterpret_cast<const uint32_t*>(r);
    }
}
template <typename T, bool ANY> __device__ __forceinline__ void set_row_word(uint8_t* r, uint32_t w) {
    if constexpr (ANY && sizeof(T) == 2) {
        *reinterpret_cast<uint16_t*>(r) = static_cast<uint16_t>(w);
        *reinterpret_cast<uint16_t*>(r + 2) = static_cast<uint16_t>(w >> 16);
    } else {
        *reinterpret_cast<uint32_t*>(r) = w;
    }
}

// ---------------------------------------------------------------------------------------
// 8-bit codes of one checkpoint block of every lane's channels, from the staged rows
// ---------------------------------------------------------------------------------------
// 16-bit values stay pairs: limits, magnitudes and their maximum are two-wide instructions on
// them (all exact: 16 and 127 scales are numbers of the type; 127 scales of a subnormal fp16 block
// round to within its numbers' distance, which no value of the block lies between).
template <typename T> __device__ __forceinline__ auto both(float a, float b) {
    if constexpr (std::is_same<T, __half>::value) return __floats2half2_rn(a, b);
    else return __floats2bfloat162_rn(a, b);
}

// Two channels' scale exponents, 127 scales as pairs of T, and the factors of their codes.
template <typename T, typename H2>
__device__ __forceinline__ void block_scales(H2 top, uint32_t& e0, uint32_t& e1, H2& most, Vec<2>& inv) {
    e0 = scale_exp(__float_as_uint(static_cast<float>(top.x)) & 0x7fffffffu);
    e1 = scale_exp(__float_as_uint(static_cast<float>(top.y)) & 0x7fffffffu);
    const Coder c0(e0), c1(e1);
    inv.x = make_float2(c0.inv, c1.inv);
    most = both<T>(e0 == kExpNaN ? 0.f : 127.f * scale_of(e0), e1 == kExpNaN ? 0.f : 127.f * scale_of(e1));
}

// The codes of two channels in the two low bytes of a word (the others are not theirs).
template <typename T, typename H2>
__device__ __forceinline__ uint32_t block_codes(H2 v, H2 most, Vec<2> inv) {
    v = __hmax2(__hmin2(v, most), __hneg2(most));
    const Vec<2> f = fma(Pack<T>::get(*reinterpret_cast<const uint32_t*>(&v)), inv, splat<2>(kCodeMagic));
    return __byte_perm(__float_as_uint(f.x.x), __float_as_uint(f.x.y), 0x0040);
}

// A gate's values are first held to >= -kHeldGate (FLOOR) and <= kHeldGate (CEIL; NaN stays).  Out
// of line: scans without checkpoints do without it in their loop.  Returns whether a value is not finite.
template <typename T, bool ANY, bool FLOOR, bool CEIL>
__device__ __noinline__ bool code_rows(const uint8_t* r, int pitch, uint32_t valid,
                                       int8_t* q, uint8_t* e, int d, bool whole, int count) {
    constexpr int V = kChannels<T>;
    uint8_t* out = reinterpret_cast<uint8_t*>(q);
    auto word = [&](int j) { return row_word<T, ANY>(r + j * (ANY ? pitch : kRowBytes)); };
    if constexpr (V == 1) {
        auto held = [&](int j) {
            float v = __uint_as_float(word(j));
            if (FLOOR && v < -kHeldGate) v = -kHeldGate;
            if (CEIL && v > kHeldGate) v = kHeldGate;
            return v;
        };
        uint32_t top = 0;  // bits of the magnitudes: their order, NaN on top
        if (valid == kAll) {
            float v[kSub];
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
                v[j] = held(j);
                top = max(top, __float_as_uint(fabsf(v[j])));
            }
            const Coder coder(scale_exp(top));
            if (count)
#pragma unroll
                for (int j = 0; j < kSub; ++j, out += d) *out = static_cast<uint8_t>(coder.code(v[j]));
        } else {
#pragma unroll 1
            for (int j = 0; j < kSub; ++j)
                if (valid >> j & 1) top = max(top, __float_as_uint(fabsf(held(j))));
            const Coder coder(scale_exp(top));
#pragma unroll 1
            for (int j = 0; j < kSub; ++j, out += d)
                if ((valid >> j & 1) && count) *out = static_cast<uint8_t>(coder.code(held(j)));
        }
        if (count) *e = static_cast<uint8_t>(scale_exp(top));
        return scale_exp(top) == kExpNaN;
    } else {
        using H2 = decltype(both<T>(0.f, 0.f));
        const H2 lowest = both<T>(-kHeldGate, -kHeldGate), highest = both<T>(kHeldGate, kHeldGate);
        auto held = [&](int j) {
            const uint32_t w = word(j);
            H2 v = *reinterpret_cast<const H2*>(&w);
            if constexpr (FLOOR) v = __hmax2_nan(v, lowest);
            if constexpr (CEIL) v = __hmin2_nan(v, highest);
            return v;
        };
        H2 top = both<T>(0.f, 0.f), most;
        uint32_t e0, e1;
        Vec<2> inv;
        if (valid == kAll && (ANY || whole)) {
            H2 v[kSub];
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
                v[j] = held(j);
                top = __hmax2_nan(top, __habs2(v[j]));
            }
            block_scales<T>(top, e0, e1, most, inv);
            if (whole && count) {
#pragma unroll
                for (int j = 0; j < kSub; ++j, out += d)
                    *reinterpret_cast<uint16_t*>(out) = static_cast<uint16_t>(block_codes<T>(v[j], most, inv));
            } else if (ANY) {
#pragma unroll
                for (int j = 0; j < kSub; ++j, out += d) {
                    const uint32_t w = block_codes<T>(v[j], most, inv);
                    if (count > 0) out[0] = static_cast<uint8_t>(w);
                    if (count > 1) out[1] = static_cast<uint8_t>(w >> 8);
                }
            }
        } else {
#pragma unroll 1
            for (int j = 0; j < kSub; ++j)
                if (valid >> j & 1) top = __hmax2_nan(top, __habs2(held(j)));
            block_scales<T>(top, e0, e1, most, inv);
#pragma unroll 1
            for (int j = 0; j < kSub; ++j, out += d) {
                if (!(valid >> j & 1)) continue;
                const uint32_t w = block_codes<T>(held(j), most, inv);
                if (count > 0) out[0] = static_cast<uint8_t>(w);
                if (count > 1) out[1] = static_cast<uint8_t>(w >> 8);
            }
        }
        if (count > 0) e[0] = static_cast<uint8_t>(e0);
        if (count > 1) e[1] = static_cast<uint8_t>(e1);
        return max(e0, e1) == kExpNaN;
    }
}

// A block that holds tokens of several sequences, where code_rows has met a value that is not finite: such
// values get the code kCodeNaN and no part in their channel's scale, so that the other sequences keep
// theirs.  (Only there: marks in every block of several sequences would make those wait, and their CTA with
// them; 20011 x 5120 packed bf16 rows in 22 sequences took 286 us instead of 264.)
template <typename T, bool ANY, bool FLOOR, bool CEIL>
__device__ __noinline__ void mark_rows(const uint8_t* r, int pitch, uint32_t valid, int8_t* q, uint8_t* e,
                                       int d, int count) {
    for (int v = 0; v < count; ++v) {
        auto held = [&](int j) {
            float f = Pack<T>::get(row_word<T, ANY>(r + j * (ANY ? pitch : kRowBytes)))[v];
            if (FLOOR && f < -kHeldGate) f = -kHeldGate;
            if (CEIL && f > kHeldGate) f = kHeldGate;
            return f;
        };
        uint32_t top = 0;  // of the finite values
        bool all = true;
#pragma unroll 4
        for (int j = 0; j < kSub; ++j) {
            const uint32_t m = __float_as_uint(fabsf(held(j)));
            if (!(valid >> j & 1)) continue;
            if (m < 0x7f800000u) top = max(top, m);
            else all = false;
        }
        if (all) continue;
        const Coder coder(scale_exp(top));
        for (int j = 0; j < kSub; ++j) {
            if (!(valid >> j & 1)) continue;
            const float f = held(j);
            q[(size_t)j * d + v] = static_cast<int8_t>(fabsf(f) < INFINITY ? coder.code(f) : kCodeNaN);
        }
        e[v] = static_cast<uint8_t>(scale_exp(top));
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
    // The map of runs `from` to `to` - 1 of N; the loads do not wait for the joins.
    template <bool PACKED, int N>
    static __device__ __forceinline__ Map<V> join_runs(const float* s, int from, int to, int lane) {
        Map<V> m[N];
#pragma unroll
        for (int i = 0; i < N; ++i) m[i] = read(s, i, lane);
        Map<V> all = identity_map<V>();
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i >= from && i < to) all = join<PACKED>(all, m[i]);
        return all;
    }
    // `carry` through runs 0 .. N - 1; returns what run `which` receives.
    template <bool PACKED, int N>
    static __device__ __forceinline__ Vec<V> carry_through(const float* s, int which, int lane,
                                                           Vec<V>& carry) {
        Map<V> m[N];
#pragma unroll
        for (int i = 0; i < N; ++i) m[i] = read(s, i, lane);
        Vec<V> mine = carry;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i == which) mine = carry;
            carry = through<PACKED>(m[i], carry);
        }
        return mine;
    }
};

// `carry` through the maps of `n` chunks in the workspace, from chunk `from` on, upward (by 1) or
// downward (by -1), eight loads at a time.
template <bool PACKED, int V>
__device__ __forceinline__ Vec<V> through_chunks(const float* maps, int from, int n, int by, int lane,
                                                 Vec<V> carry) {
    for (int i = 0; i < n; i += 8) {
        Map<V> m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = MapSlots<V>::read(maps, from + by * min(i + j, n - 1), lane);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j < n) carry = through<PACKED>(m[j], carry);
    }
    return carry;
}

// The scan may start while the kernel of its chunks' maps ends: that kernel allows it once a CTA is
// through its tokens, and the scan waits, its first copies on their way, before it reads the maps.
__device__ __forceinline__ void allow_next_kernel() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous_kernel() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// One step's meeting: every warp of the CTA gives the map of its segment and gets the carry into
// it; `carry` goes on to the next step.  `order`: the warp's place in the recurrence (0 first).
// The maps of two steps are kept in turn: a buffer is written again two steps later, when the
// barrier of the step between has seen every reader past it.
template <int V, int W> constexpr int kMeetingBytes = 2 * W * MapSlots<V>::kFloats * 4;

template <bool PACKED, int W, int V>
__device__ __forceinline__ Vec<V> meet(float* maps, int k, int order, const Map<V>& part, Vec<V>& carry) {
    const int lane = threadIdx.x & 31;
    float* m = maps + (k & 1) * W * MapSlots<V>::kFloats;
    MapSlots<V>::write(m, order, lane, part);
    __syncthreads();
    return MapSlots<V>::template carry_through<PACKED, W>(m, order, lane, carry);
}

// ---------------------------------------------------------------------------------------
// where the tokens of a segment stand in packed rows
// ---------------------------------------------------------------------------------------
// Bit j is token t0 + j.  `held` keeps the bounds of the last sequence met: tokens inside it
// need no search.
struct Marks {
    uint32_t valid, begin, end;  // in a sequence; its first token; its last token
    int seq;                     // lane j < kSub: the sequence of token t0 + j
};

// Whether tokens of several sequences share the segment: a beginning behind its first valid token.
__device__ __forceinline__ bool mixed_block(const Marks& m) {
    return (m.begin & ~(m.valid & (0u - m.valid))) != 0;
}

struct Held {
    int seq = -1, from = 0, to = 0;
};

__device__ __forceinline__ Marks marks_of(const int32_t* __restrict__ cu, int nseq, int t0, int n,
                                          Held& held) {
    Marks m;
    const int lane = threadIdx.x & 31;
    if (n == kSub && t0 > held.from && t0 + kSub < held.to) {
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
    // the sequence of the middle token is as good a guess as any for the next ones
    const int src = kSub / 2;
    held.seq = __shfl_sync(0xffffffffu, s, src);
    held.from = __shfl_sync(0xffffffffu, from, src);
    held.to = __shfl_sync(0xffffffffu, to, src);
    return m;
}

// f(s) for every sequence without a token; the strip's warps, `which` of `many`, share them, 32 looked
// at at a time (20000 tokens of 512 channels and 100000 sequences: forward 97 us, one by one 1385).
template <typename F>
__device__ __forceinline__ void for_empty_sequences(const int32_t* __restrict__ cu, int nseq, int which,
                                                    int many, F f) {
    for (long long s0 = 32ll * which; s0 < nseq; s0 += 32ll * many) {
        const long long s = s0 + (threadIdx.x & 31);
        uint32_t empty = __ballot_sync(0xffffffffu, s < nseq && __ldg(cu + s + 1) <= __ldg(cu + s));
        for (; empty; empty &= empty - 1) f(static_cast<int>(s0) + __ffs(empty) - 1);
    }
}

}  // namespace gated
}  // namespace ssd
