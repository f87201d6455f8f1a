// Forward gated scan (the tile scheme is described in gated_tile.cuh).
//
// Per element: x and gate are read and y is written once, one exponential (two fast operations for
// logits), about a dozen fp32 instructions.  Bound by HBM.
#pragma once

#include <type_traits>

#include "gated_launch.cuh"

namespace ssd {
namespace gated {

// Shared memory of the staged inputs: [stage][x, gate][warp][16 tokens][128 bytes].
constexpr int kFwdStage = 2 * kTile * kRowBytes;
constexpr int kFwdSmem = kFwdStages * kFwdStage;

template <typename T, bool LOGIT, bool COMP, bool PACKED>
__global__ void __launch_bounds__(kTileThreads, kFwdBlocks)
scan_kernel(const __grid_constant__ GatedArgs a, const TileArgs ta) {
    constexpr int V = kChannels<T>;
    using Pk = Pack<T>;
    using F = Vec<V>;
    using Slots = MapSlots<V>;
    extern __shared__ __align__(128) uint8_t staged[];
    __shared__ __align__(16) float seg_maps[2][kWarps * Slots::kFloats];
    __shared__ __align__(16) float cta_maps[2][kMaxCluster * Slots::kFloats];

    // the shuffle tells the compiler that the warp's index, and with it every row's address, is
    // the same in all lanes
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int R = ta.cluster, rank = blockIdx.x % R, unit = blockIdx.x / R;
    const int d = a.channels, b = unit / ta.strips, c0 = unit % ta.strips * 32 * V;
    const int c = c0 + lane * V, count = max(0, min(V, d - c));
    const bool full = d - c0 >= 32 * V, whole = full && ta.pair_out, whole_codes = full && ta.pair_codes;
    const int tiles = (a.seqlen + kTile - 1) / kTile, steps = (tiles + R - 1) / R;
    const size_t row0 = (size_t)b * a.seqlen;

    const char* px = static_cast<const char*>(a.x.ptr) + (b * a.x.batch_stride + c0) * sizeof(T);
    const char* pg = static_cast<const char*>(a.gate.ptr) + (b * a.gate.batch_stride + c0) * sizeof(T);
    char* py = static_cast<char*>(const_cast<void*>(a.y.ptr)) + (b * a.y.batch_stride + c0) * sizeof(T);
    const long long sx = a.x.token_stride * sizeof(T), sg = a.gate.token_stride * sizeof(T);
    const long long sy = a.y.token_stride * sizeof(T);
    const int width = min(kRowBytes, (d - c0) * (int)sizeof(T));

    auto slot = [&](int k, int tensor) {
        return staged + (k % kFwdStages) * kFwdStage + (tensor * kWarps + warp) * kSeg * kRowBytes;
    };
    auto stage = [&](int k) {  // this warp's segment of step k
        if (k < steps) {
            const int t0 = (k * R + rank) * kTile + warp * kSeg;
            const int n = max(0, min(kSeg, a.seqlen - t0));
            stage_rows<kRowBytes>(slot(k, 0), n ? px + t0 * sx : px, sx, n, width, ta.align_x);
            stage_rows<kRowBytes>(slot(k, 1), n ? pg + t0 * sg : pg, sg, n, width, ta.align_gate);
        }
        copy_commit();
    };
    auto init_of = [&](int s) {
        return load_floats<V>(a.init_state ? a.init_state + (size_t)s * d + c : nullptr, count);
    };

    F carry = PACKED ? splat<V>(0.f) : init_of(b);
    if (PACKED && a.final_state && rank == 0)  // sequences without a token
        for (int s = warp; s < a.nseq; s += kWarps)
            if (__ldg(a.cu + s + 1) <= __ldg(a.cu + s))
                store_floats<V>(a.final_state + (size_t)s * d + c, init_of(s), count);
    Held held;
#pragma unroll
    for (int k = 0; k < kFwdStages - 1; ++k) stage(k);
    for (int k = 0; k < steps; ++k) {
        const int tile = k * R + rank, t0 = tile * kTile + warp * kSeg;
        const int n = max(0, min(kSeg, a.seqlen - t0));
        Marks m;
        m.valid = (1u << n) - 1;
        m.begin = m.end = 0;
        if constexpr (PACKED) m = marks_of(a.cu, a.nseq, t0, n, held);
        copy_wait<kFwdStages - 2>();
        __syncwarp();  // the segment is here, and every lane is done with the slot filled next
        stage(k + kFwdStages - 1);
        uint32_t* rx = reinterpret_cast<uint32_t*>(slot(k, 0)) + lane;
        uint32_t* rg = reinterpret_cast<uint32_t*>(slot(k, 1)) + lane;
        if (m.valid != kAll) {
            // tokens of no sequence keep the state: x 0, decay 1 (each lane mends its own words)
            for (int j = 0; j < kSeg; ++j)
                if (!(m.valid >> j & 1)) {
                    rx[j * 32] = 0;
                    rg[j * 32] = LOGIT ? Pk::kInf : 0u;
                }
        }

        if (a.x_q && n > 0) {  // the segment is one checkpoint block per channel
            uint32_t top_x[V], top_g[V];  // bits of the magnitudes: their order, NaN on top
#pragma unroll
            for (int v = 0; v < V; ++v) top_x[v] = top_g[v] = 0;
#pragma unroll
            for (int j = 0; j < kSeg; ++j) {
                const F x = Pk::get(rx[j * 32]), g = Pk::get(rg[j * 32]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    top_x[v] = max(top_x[v], __float_as_uint(fabsf(x[v])));
                    if (!LOGIT || (m.valid >> j & 1))
                        top_g[v] = max(top_g[v], __float_as_uint(fabsf(held_gate<LOGIT>(g[v]))));
                }
            }
            float inv_x[V], inv_g[V];
            int ex[V], eg[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                ex[v] = scale_exp(top_x[v]);
                eg[v] = scale_exp(top_g[v]);
                inv_x[v] = inv_scale_of(ex[v]);
                inv_g[v] = inv_scale_of(eg[v]);
            }
            const size_t at = (row0 + t0) * d + c;
            uint8_t* qx = reinterpret_cast<uint8_t*>(a.x_q) + at;
            uint8_t* qg = reinterpret_cast<uint8_t*>(a.gate_q) + at;
#pragma unroll
            for (int j = 0; j < kSeg; ++j) {
                if (!(m.valid >> j & 1)) continue;
                const F x = Pk::get(rx[j * 32]), g = Pk::get(rg[j * 32]);
                int code[V];
#pragma unroll
                for (int v = 0; v < V; ++v) code[v] = code_of(x[v], inv_x[v]);
                store_bytes<V>(qx + (size_t)j * d, code, whole_codes, count);
#pragma unroll
                for (int v = 0; v < V; ++v) code[v] = code_of(held_gate<LOGIT>(g[v]), inv_g[v]);
                store_bytes<V>(qg + (size_t)j * d, code, whole_codes, count);
            }
            const size_t be = ((size_t)b * ta.blocks + t0 / kBlock) * d + c;
            store_bytes<V>(a.x_e + be, ex, whole_codes, count);
            store_bytes<V>(a.gate_e + be, eg, whole_codes, count);
        }

        // The state behind token j is P[j] carry + B[j] (P with its low part Q in fp32): from the
        // carry on, the tokens do not depend on one another.
        F P[kSeg], Q[V == 1 ? kSeg : 1], B[kSeg];
        Map<V> seg = identity_map<V>();
#pragma unroll
        for (int j = 0; j < kSeg; ++j) {
            F in = Pk::get(rx[j * 32]);
            const Decay<V> r = decay_of<LOGIT>(Pk::get(rg[j * 32]));
            if (PACKED && (m.begin >> j & 1)) seg.B = init_of(__shfl_sync(0xffffffffu, m.seq, j));
            if constexpr (COMP) in = mul(r.u, in);
            seg.B = step(r.a, r.lo, seg.B, in);
            extend(seg, r);
            P[j] = seg.A;
            B[j] = seg.B;
            if constexpr (V == 1) Q[j] = seg.L;
        }
        if (PACKED && m.begin) seg.A = splat<V>(-1.f);

        // the carry into this segment, and into the next step
        float* segs = seg_maps[k & 1];
        F h;
        Slots::write(segs, warp, lane, seg);
        __syncthreads();
        if (R > 1) {
            float* ctas = cta_maps[k & 1];
            if (warp == kWarps - 1) {
                const Map<V> all = Slots::template join_runs<PACKED>(segs, lane);
                for (int r = 0; r < R; ++r) Slots::send(ctas, rank, lane, r, all);
            }
            cluster_barrier(warp == kWarps - 1);
            h = Slots::template carry_through<PACKED>(ctas, R, rank, lane, carry);
            h = Slots::template carry_into<PACKED>(segs, warp, lane, h);
        } else {
            h = Slots::template carry_through<PACKED>(segs, kWarps, warp, lane, carry);
        }

        if (a.span_states && warp == 0 && n > 0) {
            const bool none = PACKED && (!(m.valid & 1) || (m.begin & 1));
            store_floats<V>(a.span_states + ((size_t)b * tiles + tile) * d + c,
                            none ? splat<V>(0.f) : h, count);
        }
        if (PACKED && m.begin) {  // the carry only reaches the tokens before the first beginning
#pragma unroll
            for (int j = 0; j < kSeg; ++j) {
                if (!(m.begin & ((2u << j) - 1))) B[j] = step(P[j], Q[V == 1 ? j : 0], h, B[j]);
                P[j] = splat<V>(0.f);
                if constexpr (V == 1) Q[j] = P[j];
            }
            h = splat<V>(0.f);
        }
        if (PACKED && m.end && a.final_state) {
#pragma unroll
            for (int j = 0; j < kSeg; ++j)
                if (m.end >> j & 1)
                    store_floats<V>(a.final_state + (size_t)__shfl_sync(0xffffffffu, m.seq, j) * d + c,
                                    step(P[j], Q[V == 1 ? j : 0], h, B[j]), count);
        }
        char* qy = py + t0 * sy + lane * 4;
        if (whole && m.valid == kAll) {
#pragma unroll
            for (int j = 0; j < kSeg; ++j) {
                *reinterpret_cast<uint32_t*>(qy) = Pk::put(step(P[j], Q[V == 1 ? j : 0], h, B[j]));
                qy += sy;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kSeg; ++j) {
                if (m.valid >> j & 1)
                    store_row<T>(qy, step(P[j], Q[V == 1 ? j : 0], h, B[j]), whole, count);
                qy += sy;
            }
        }
    }
    // the carry behind the last tile is the final state, in every thread of the cluster
    if (!PACKED && a.final_state && rank == 0 && warp == 0)
        store_floats<V>(a.final_state + (size_t)b * d + c, carry, count);
}

template <typename T>
cudaError_t dispatch_fwd(const GatedArgs& a, cudaStream_t st) {
    auto go = [&](auto logit, auto comp) {
        constexpr bool L = decltype(logit)::value, C = decltype(comp)::value;
        return a.cu ? launch_tiles<T>(scan_kernel<T, L, C, true>, a, kFwdBlocks, kFwdSmem, st)
                    : launch_tiles<T>(scan_kernel<T, L, C, false>, a, kFwdBlocks, kFwdSmem, st);
    };
    using Y = std::true_type;
    using N = std::false_type;
    if (a.logit) return a.complement ? go(Y{}, Y{}) : go(Y{}, N{});
    return a.complement ? go(N{}, Y{}) : go(N{}, N{});
}

}  // namespace gated
}  // namespace ssd
