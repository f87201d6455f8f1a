// Forward gated scan (the walk along strips is described in gated_tile.cuh).
//
// Per element x and gate are read and y is written once.  A thread computes, over the 16 tokens of
// its segment and from a zero carry, the state B[j] and the product P[j] of the decays up to token
// j; the state behind token j is then P[j] carry + B[j], so that after the meeting no token waits
// for another.  (Going over the tokens again with the carry instead takes 2.7 more instructions per
// element for the loads and conversions, and 16 dependent steps.)
//
// What bounds it (one B200, of the measured copy bandwidth 6.47 TB/s): with enough strips HBM - 8 x
// 4096 x 5120 bf16 170 us, 92 %; 2 x 16384 x 8192 logits with 1 - a weights 290 us, 86 %; 4 x 2048 x
// 4096 bf16 36 us, 87 %, fp32 logits 72 us, 86 % - else the instructions: 18 per element (ncu), of which
// half are the segment's own (copies, maps, meeting), issued at about 2 per SM and cycle (58 % of the
// slots where a strip is cut into chunks), and for fp32 log gates, 93 us, 67 %, expf with expm1f.  With
// codes: 4 x 2048 x 4096 bf16 58 us, fp32 110 (logits) and 131.
#pragma once

#include <type_traits>

#include "gated_launch.cuh"

namespace ssd {
namespace gated {

// A warp's staged segment: x and gate.
template <bool ANY> constexpr int kFwdSegBytes = 2 * kSubBytes<kRowBytes, ANY>;
// Segments in shared memory per warp: the current one and those ahead, as many as leave room for a
// second CTA (128 strips of 4096 bf16 tokens: 42 us with two ahead, 47 with one).
template <bool ANY> constexpr int kFwdSlots = ANY ? 2 : 3;

template <typename T, bool LOGIT, bool COMP, bool PACKED, bool ANY>
__global__ void __launch_bounds__(32 * kFwdWarps, kFwdBlocks)
scan_kernel(const __grid_constant__ GatedArgs a, const __grid_constant__ TileArgs ta) {
    constexpr int V = kChannels<T>;
    using Pk = Pack<T>;
    using F = Vec<V>;
    extern __shared__ __align__(128) uint8_t staged[];

    // the shuffle tells the compiler that the warp's index, and with it every row's address, is
    // the same in all lanes
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    constexpr int W = kFwdWarps;
    const int chunk = blockIdx.x % ta.chunks, unit = blockIdx.x / ta.chunks;
    const int d = a.channels, b = unit / ta.strips, c0 = unit % ta.strips * 32 * V;
    const int c = c0 + lane * V, count = max(0, min(V, d - c));
    const bool whole = ta.whole_out, whole_codes = ta.whole_codes;
    const int first = chunk * ta.chunk_tiles * W;  // segment
    const int steps = (min(ta.blocks - first, ta.chunk_tiles * W) + W - 1) / W;
    const size_t row0 = (size_t)b * a.seqlen;

    const char* px = static_cast<const char*>(a.x.ptr) + (b * a.x.batch_stride + c0) * sizeof(T);
    const char* pg = static_cast<const char*>(a.gate.ptr) + (b * a.gate.batch_stride + c0) * sizeof(T);
    char* py = static_cast<char*>(const_cast<void*>(a.y.ptr)) + (b * a.y.batch_stride + c0) * sizeof(T);
    const long long sx = a.x.token_stride * sizeof(T), sg = a.gate.token_stride * sizeof(T);
    const long long sy = a.y.token_stride * sizeof(T);
    const int width = min(kRowBytes, (d - c0) * (int)sizeof(T));

    float* maps = reinterpret_cast<float*>(staged);
    constexpr int kSlots = kFwdSlots<ANY>, kSeg = kFwdSegBytes<ANY>, kGateAt = kSeg / 2;
    uint8_t* own = staged + kMeetingBytes<V, W> + warp * kSlots * kSeg;
    const int qx = staged_pitch<kRowBytes, ANY>(sx), qg = staged_pitch<kRowBytes, ANY>(sg);
    auto start = [&](int k) { return (first + k * W + warp) * kSub; };
    auto stage = [&](int k, int slot) {  // this warp's segment of step k
        const int t = start(k), n = max(0, min(kSub, a.seqlen - t));
        if (k < steps && n > 0) {
            uint8_t* to = own + slot * kSeg;
            if (n == kSub) [[likely]] {
                stage_rows<kRowBytes, ANY>(to, px + t * sx, sx, width);
                stage_rows<kRowBytes, ANY>(to + kGateAt, pg + t * sg, sg, width);
            } else {
                stage_part<kRowBytes, ANY>(to, px + t * sx, sx, n, width);
                stage_part<kRowBytes, ANY>(to + kGateAt, pg + t * sg, sg, n, width);
            }
        }
        copy_commit();
    };
    auto init_of = [&](int s) {
        return load_floats<V>(a.init_state ? a.init_state + (size_t)s * d + c : nullptr, count);
    };

    F carry = PACKED ? splat<V>(0.f) : init_of(b);
    if (PACKED && a.final_state)
        for_empty_sequences(a.cu, a.nseq, chunk * W + warp, ta.chunks * W, [&](int s) {
            store_floats<V>(a.final_state + (size_t)s * d + c, init_of(s), count);
        });
#pragma unroll 1
    for (int k = 0; k < kSlots - 1; ++k) stage(k, k);
    int slot = 0, free_slot = kSlots - 1;
    if (ta.chunks > 1) {
        wait_for_previous_kernel();
        const float* of_chunks = ta.maps + (size_t)unit * ta.chunks * MapSlots<V>::kFloats;
        carry = through_chunks<PACKED>(of_chunks, 0, chunk, 1, lane, carry);
    }
    Held held;
    for (int k = 0; k < steps; ++k) {
        const int t0 = start(k), n = max(0, min(kSub, a.seqlen - t0));
        Marks m;
        m.valid = (1u << n) - 1;
        m.begin = m.end = 0;
        if constexpr (PACKED) m = marks_of(a.cu, a.nseq, t0, n, held);
        copy_wait<kSlots - 2>();
        __syncwarp();  // the segment is here, and every lane is done with the slot filled next
        stage(k + kSlots - 1, free_slot);
        uint8_t* here = own + slot * kSeg;
        free_slot = slot;
        slot = slot + 1 == kSlots ? 0 : slot + 1;
        uint8_t* rx = here + staged_start<ANY>(px + t0 * sx) + lane * 4;
        uint8_t* rg = here + kGateAt + staged_start<ANY>(pg + t0 * sg) + lane * 4;
        if (m.valid != kAll) [[unlikely]] {
            // tokens of no sequence keep the state: x 0, decay 1 (each lane mends its own words)
            for (int j = 0; j < kSub; ++j)
                if (!(m.valid >> j & 1)) {
                    set_row_word<T, ANY>(rx + j * qx, 0u);
                    set_row_word<T, ANY>(rg + j * qg, LOGIT ? Pk::kInf : 0u);
                }
        }
        if (a.x_q && n > 0) {
            const size_t at = (row0 + t0) * d + c, be = ((size_t)b * ta.blocks + t0 / kBlock) * d + c;
            const bool odd_x = code_rows<T, ANY, false, false>(rx, qx, m.valid, a.x_q + at, a.x_e + be, d,
                                                               whole_codes, count);
            const bool odd_gate = code_rows<T, ANY, true, LOGIT>(rg, qg, m.valid, a.gate_q + at, a.gate_e + be, d,
                                                                 whole_codes, count);
            if (PACKED && (odd_x || odd_gate) && mixed_block(m)) [[unlikely]] {
                mark_rows<T, ANY, false, false>(rx, qx, m.valid, a.x_q + at, a.x_e + be, d, count);
                mark_rows<T, ANY, true, LOGIT>(rg, qg, m.valid, a.gate_q + at, a.gate_e + be, d, count);
            }
        }

        // The state behind token j is P[j] carry + B[j] (P with its low part Q in fp32): from the
        // carry on, the tokens do not depend on one another.
        F P[kSub], Q[V == 1 ? kSub : 1], B[kSub];
        Map<V> seg = identity_map<V>();
        // segments without a beginning, by far the most, go without the checks of every token
        auto map = [&](auto checks) {
            constexpr bool CHECK = decltype(checks)::value;
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
                F in = Pk::get(row_word<T, ANY>(rx + j * qx));
                const Decay<V> r = decay_of<LOGIT>(Pk::get(row_word<T, ANY>(rg + j * qg)));
                if (CHECK && (m.begin >> j & 1)) seg.B = init_of(__shfl_sync(0xffffffffu, m.seq, j));
                if constexpr (COMP) in = mul(r.u, in);
                seg.B = step(r.a, r.lo, seg.B, in);
                extend(seg, r);
                P[j] = seg.A;
                B[j] = seg.B;
                if constexpr (V == 1) Q[j] = seg.L;
            }
        };
        if (!PACKED || !m.begin) [[likely]] map(std::false_type{});
        else map(std::true_type{});
        if (PACKED && m.begin) seg.A = splat<V>(-1.f);
        F h = meet<PACKED, W>(maps, k, warp, seg, carry);
        if (a.span_states && n > 0 && t0 % kSpan == 0) {
            const bool none = PACKED && (!(m.valid & 1) || (m.begin & 1));
            store_floats<V>(a.span_states + ((size_t)b * ta.spans + t0 / kSpan) * d + c,
                            none ? splat<V>(0.f) : h, count);
        }
        if (PACKED && m.begin) [[unlikely]] {  // the carry only reaches the tokens before the first beginning
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
                if (!(m.begin & ((2u << j) - 1))) B[j] = step(P[j], Q[V == 1 ? j : 0], h, B[j]);
                P[j] = splat<V>(0.f);
                if constexpr (V == 1) Q[j] = P[j];
            }
            h = splat<V>(0.f);
        }
        if (PACKED && m.end && a.final_state) [[unlikely]] {
#pragma unroll
            for (int j = 0; j < kSub; ++j)
                if (m.end >> j & 1)
                    store_floats<V>(a.final_state + (size_t)__shfl_sync(0xffffffffu, m.seq, j) * d + c,
                                    step(P[j], Q[V == 1 ? j : 0], h, B[j]), count);
        }
        char* qy = py + t0 * sy + lane * 4;
        if (whole && m.valid == kAll) [[likely]] {
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
                store_row<T>(qy, step(P[j], Q[V == 1 ? j : 0], h, B[j]), true, count);
                qy += sy;
            }
        } else if (ANY && m.valid == kAll) {
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
                store_row<T>(qy, step(P[j], Q[V == 1 ? j : 0], h, B[j]), false, count);
                qy += sy;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
                if (m.valid >> j & 1)
                    store_row<T>(qy, step(P[j], Q[V == 1 ? j : 0], h, B[j]), whole, count);
                qy += sy;
            }
        }
    }
    // the carry behind the last tile is the final state, in every thread of its CTA
    if (!PACKED && a.final_state && chunk == ta.chunks - 1 && warp == 0)
        store_floats<V>(a.final_state + (size_t)b * d + c, carry, count);
}

// The maps of all chunks but the last of every strip: each warp reduces a run of whole segments.
template <bool ANY> constexpr int kMapSlots = ANY ? 2 : 3;
template <typename T, bool LOGIT, bool COMP, bool PACKED, bool ANY>
__global__ void __launch_bounds__(32 * kMapWarps)
chunk_map_kernel(const __grid_constant__ GatedArgs a, const __grid_constant__ TileArgs ta) {
    constexpr int V = kChannels<T>, W = kMapWarps;
    using Pk = Pack<T>;
    using F = Vec<V>;
    extern __shared__ __align__(128) uint8_t staged[];

    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int chunk = blockIdx.x % (ta.chunks - 1), unit = blockIdx.x / (ta.chunks - 1);
    const int d = a.channels, b = unit / ta.strips, c0 = unit % ta.strips * 32 * V;
    const int c = c0 + lane * V, count = max(0, min(V, d - c));
    const int run = ta.chunk_tiles * kFwdWarps / W;  // segments of a warp
    const int first = chunk * ta.chunk_tiles * kFwdWarps + warp * run;

    const char* px = static_cast<const char*>(a.x.ptr) + (b * a.x.batch_stride + c0) * sizeof(T);
    const char* pg = static_cast<const char*>(a.gate.ptr) + (b * a.gate.batch_stride + c0) * sizeof(T);
    const long long sx = a.x.token_stride * sizeof(T), sg = a.gate.token_stride * sizeof(T);
    const int width = min(kRowBytes, (d - c0) * (int)sizeof(T));
    float* maps = reinterpret_cast<float*>(staged);
    constexpr int kSlots = kMapSlots<ANY>, kSeg = kFwdSegBytes<ANY>, kGateAt = kSeg / 2;
    uint8_t* own = staged + kMeetingBytes<V, W> + warp * kSlots * kSeg;
    const int qx = staged_pitch<kRowBytes, ANY>(sx), qg = staged_pitch<kRowBytes, ANY>(sg);
    auto stage = [&](int k) {
        const int t = (first + k) * kSub, n = min(kSub, a.seqlen - t);
        if (k < run && n > 0) {
            uint8_t* to = own + k % kSlots * kSeg;
            if (n == kSub) [[likely]] {
                stage_rows<kRowBytes, ANY>(to, px + t * sx, sx, width);
                stage_rows<kRowBytes, ANY>(to + kGateAt, pg + t * sg, sg, width);
            } else {
                stage_part<kRowBytes, ANY>(to, px + t * sx, sx, n, width);
                stage_part<kRowBytes, ANY>(to + kGateAt, pg + t * sg, sg, n, width);
            }
        }
        copy_commit();
    };
    Map<V> all = identity_map<V>();
    bool begins = false;
    Held held;
#pragma unroll 1
    for (int k = 0; k < kSlots - 1; ++k) stage(k);
    for (int k = 0; k < run; ++k) {
        const int t0 = (first + k) * kSub, n = max(0, min(kSub, a.seqlen - t0));
        Marks m;
        m.valid = (1u << n) - 1;
        m.begin = m.end = 0;
        if constexpr (PACKED) m = marks_of(a.cu, a.nseq, t0, n, held);
        copy_wait<kSlots - 2>();
        __syncwarp();
        stage(k + kSlots - 1);
        uint8_t* here = own + k % kSlots * kSeg;
        const uint8_t* rx = here + staged_start<ANY>(px + t0 * sx) + lane * 4;
        const uint8_t* rg = here + kGateAt + staged_start<ANY>(pg + t0 * sg) + lane * 4;
        auto token = [&](int j) {
            F in = Pk::get(row_word<T, ANY>(rx + j * qx));
            const Decay<V> r = decay_of<LOGIT>(Pk::get(row_word<T, ANY>(rg + j * qg)));
            if constexpr (COMP) in = mul(r.u, in);
            all.B = step(r.a, r.lo, all.B, in);
            extend(all, r);
        };
        if (m.valid == kAll && !m.begin) [[likely]] {
#pragma unroll
            for (int j = 0; j < kSub; ++j) token(j);
        } else {
#pragma unroll 1
            for (int j = 0; j < kSub; ++j) {
                if (!(m.valid >> j & 1)) continue;
                if (PACKED && (m.begin >> j & 1)) {
                    const int s = __shfl_sync(0xffffffffu, m.seq, j);
                    all.B = load_floats<V>(a.init_state ? a.init_state + (size_t)s * d + c : nullptr, count);
                    begins = true;
                }
                token(j);
            }
        }
    }
    allow_next_kernel();
    if (begins) all.A = splat<V>(-1.f);
    MapSlots<V>::write(maps, warp, lane, all);
    __syncthreads();
    if (warp == 0)
        MapSlots<V>::write(ta.maps + (size_t)unit * ta.chunks * MapSlots<V>::kFloats, chunk, lane,
                           MapSlots<V>::template join_runs<PACKED, W>(maps, 0, W, lane));
}

template <typename T>
cudaError_t dispatch_fwd(const GatedArgs& a, cudaStream_t st) {
    using Y = std::true_type;
    using N = std::false_type;
    TileArgs t = tile_args<T>(a);
    const long long units = (long long)t.strips * a.batch;
    const Chunks ch = chunks_of(a.x_q ? Work::kToCodes : Work::kPlain, units, t.blocks, kFwdWarps, kFwdBlocks,
                                sm_count(), t.aligned);
    t.chunks = ch.count;
    t.chunk_tiles = ch.tiles;
    t.maps = static_cast<float*>(a.workspace);
    auto go = [&](auto logit, auto comp, auto packed, auto any) {
        constexpr bool L = decltype(logit)::value, C = decltype(comp)::value, K = decltype(packed)::value;
        constexpr bool A = decltype(any)::value;
        constexpr int V = kChannels<T>, kBytes = kFwdSegBytes<A>;
        if (t.chunks > 1) {
            constexpr int kSmem = kMeetingBytes<V, kMapWarps> + kMapWarps * kMapSlots<A> * kBytes;
            const cudaError_t e = launch_ctas<chunk_map_kernel<T, L, C, K, A>>(
                units * (t.chunks - 1), kMapWarps, kSmem, false, st, a, t);
            if (e != cudaSuccess) return e;
        }
        constexpr int kSmem = kMeetingBytes<V, kFwdWarps> + kFwdWarps * kFwdSlots<A> * kBytes;
        return launch_ctas<scan_kernel<T, L, C, K, A>>(units * t.chunks, kFwdWarps, kSmem, t.chunks > 1,
                                                       st, a, t);
    };
    auto rows = [&](auto logit, auto comp, auto packed) {
        return t.aligned ? go(logit, comp, packed, N{}) : go(logit, comp, packed, Y{});
    };
    auto packed = [&](auto logit, auto comp) { return a.cu ? rows(logit, comp, Y{}) : rows(logit, comp, N{}); };
    if (a.logit) return a.complement ? packed(Y{}, Y{}) : packed(Y{}, N{});
    return a.complement ? packed(N{}, Y{}) : packed(N{}, N{});
}

}  // namespace gated
}  // namespace ssd
