// Forward gated scan (the tile scheme is described in gated_tile.cuh).
//
// Per element: x and gate are read and y is written once, one exponential (two fast operations for
// logits), about a dozen fp32 instructions.  Bound by HBM.
#pragma once

#include <type_traits>

#include "gated_launch.cuh"

namespace ssd {
namespace gated {

template <typename T, int V, bool LOGIT, bool COMP, bool PACKED>
__global__ void __launch_bounds__(kTileThreads, kFwdBlocks)
scan_kernel(const __grid_constant__ GatedArgs a, const int R) {
    constexpr bool TWO = kTwo<T>;
    using P = Pack<T, V>;
    using Raw = typename P::Raw;
    using Slots = MapSlots<V, TWO>;
    __shared__ float seg_maps[2][kWarps * Slots::kFloats];
    __shared__ float cta_maps[2][kMaxCluster * Slots::kFloats];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = blockIdx.x % R, unit = blockIdx.x / R;
    const int d = a.channels, strips = (d + 32 * V - 1) / (32 * V);
    const int b = unit / strips, c = (unit % strips) * 32 * V + lane * V;
    const bool active = c < d;
    const int tiles = (a.seqlen + kTile - 1) / kTile, steps = (tiles + R - 1) / R;

    const Raw* px = reinterpret_cast<const Raw*>(static_cast<const T*>(a.x.ptr) + b * a.x.batch_stride + c);
    const Raw* pg = reinterpret_cast<const Raw*>(static_cast<const T*>(a.gate.ptr) + b * a.gate.batch_stride + c);
    Raw* py = reinterpret_cast<Raw*>(static_cast<T*>(const_cast<void*>(a.y.ptr)) + b * a.y.batch_stride + c);
    const long long sx = a.x.token_stride / V, sg = a.gate.token_stride / V, sy = a.y.token_stride / V;
    const Raw gate_one = LOGIT ? P::kInf : Raw(0);  // the gate of a decay of 1

    // x and gate of the segment that this warp takes in step k; tokens behind the end keep the
    // state (x 0, decay 1)
    Raw rx[kSeg], rg[kSeg];
    auto load = [&](int k) {
        const int t0 = (k * R + rank) * kTile + warp * kSeg;
        const Raw* qx = px + t0 * sx;
        const Raw* qg = pg + t0 * sg;
#pragma unroll
        for (int j = 0; j < kSeg; ++j) {
            const bool in = active && t0 + j < a.seqlen;
            rx[j] = in ? load_once(qx + j * sx) : Raw(0);
            rg[j] = in ? load_once(qg + j * sg) : gate_one;
        }
    };

    float carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        carry[v] = !PACKED && active && a.init_state ? a.init_state[(size_t)b * d + c + v] : 0.f;
    if (PACKED && a.final_state && rank == 0 && active) {  // sequences without a token
        for (int s = warp; s < a.nseq; s += kWarps)
            if (__ldg(a.cu + s + 1) <= __ldg(a.cu + s))
                for (int v = 0; v < V; ++v)
                    a.final_state[(size_t)s * d + c + v] =
                        a.init_state ? a.init_state[(size_t)s * d + c + v] : 0.f;
    }
    Held held;
    load(0);
    for (int k = 0; k < steps; ++k) {
        const int tile = k * R + rank, t0 = tile * kTile + warp * kSeg;
        const int n = max(0, min(kSeg, a.seqlen - t0));
        Marks m;
        m.valid = (1u << n) - 1;
        m.begin = m.end = 0;
        if constexpr (PACKED) {
            m = marks_of(a.cu, a.nseq, t0, n, held);
            if (m.valid != (1u << kSeg) - 1) {
#pragma unroll
                for (int j = 0; j < kSeg; ++j)
                    if (!(m.valid >> j & 1)) {
                        rx[j] = 0;
                        rg[j] = gate_one;
                    }
            }
        }

        if (a.x_q && n > 0 && active) {  // the segment is one checkpoint block per channel
            float top_x[V], top_g[V];
#pragma unroll
            for (int v = 0; v < V; ++v) top_x[v] = top_g[v] = 0.f;
            bool nan_x[V] = {}, nan_g[V] = {};
#pragma unroll
            for (int j = 0; j < kSeg; ++j) {
                float x[V], g[V];
                P::get(rx[j], x);
                P::get(rg[j], g);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    // fmaxf drops a NaN: kept aside
                    top_x[v] = fmaxf(top_x[v], fabsf(x[v]));
                    nan_x[v] |= x[v] != x[v];
                    const float hg = m.valid >> j & 1 ? held_gate<LOGIT>(g[v]) : 0.f;
                    top_g[v] = fmaxf(top_g[v], fabsf(hg));
                    nan_g[v] |= hg != hg;
                }
            }
            float inv_x[V], inv_g[V];
            int ex[V], eg[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                ex[v] = scale_exp(nan_x[v] ? 0x7fc00000u : __float_as_uint(top_x[v]));
                eg[v] = scale_exp(nan_g[v] ? 0x7fc00000u : __float_as_uint(top_g[v]));
                inv_x[v] = inv_scale_of(ex[v]);
                inv_g[v] = inv_scale_of(eg[v]);
            }
            using Codes = typename CodeRaw<V>::Raw;
            const size_t at = ((size_t)b * a.seqlen + t0) * d + c;
#pragma unroll
            for (int j = 0; j < kSeg; ++j) {
                if (!(m.valid >> j & 1)) continue;
                float x[V], g[V];
                int qx[V], qg[V];
                P::get(rx[j], x);
                P::get(rg[j], g);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    qx[v] = code_of(x[v], inv_x[v]);
                    qg[v] = code_of(held_gate<LOGIT>(g[v]), inv_g[v]);
                }
                *reinterpret_cast<Codes*>(a.x_q + at + (size_t)j * d) = put_codes<V>(qx);
                *reinterpret_cast<Codes*>(a.gate_q + at + (size_t)j * d) = put_codes<V>(qg);
            }
            const int blocks = (a.seqlen + kBlock - 1) / kBlock;
            const size_t be = ((size_t)b * blocks + t0 / kBlock) * d + c;
            *reinterpret_cast<Codes*>(a.x_e + be) = put_codes<V>(ex);
            *reinterpret_cast<Codes*>(a.gate_e + be) = put_codes<V>(eg);
        }

        // decays and inputs of the segment, and its map
        float da[kSeg][V], lo[TWO ? kSeg : 1][V], in[kSeg][V], init[V];
        Map<TWO> seg[V];
#pragma unroll
        for (int v = 0; v < V; ++v) seg[v] = identity_map<TWO>();
#pragma unroll
        for (int j = 0; j < kSeg; ++j) {
            float x[V], g[V];
            P::get(rx[j], x);
            P::get(rg[j], g);
            const bool begins = PACKED && (m.begin >> j & 1);
            if (begins) {
                const int s = __shfl_sync(0xffffffffu, m.seq, j);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    init[v] = active && a.init_state ? a.init_state[(size_t)s * d + c + v] : 0.f;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Decay k = decay_of<T, LOGIT>(g[v]);
                da[j][v] = k.a;
                if constexpr (TWO) lo[j][v] = k.lo;
                in[j][v] = COMP ? k.u * x[v] : x[v];
                seg[v].B = step<TWO>(k, begins ? init[v] : seg[v].B, in[j][v]);
                extend<TWO>(seg[v], k);
            }
        }
        if (PACKED && m.begin) {
#pragma unroll
            for (int v = 0; v < V; ++v) seg[v].A = -1.f;
        }
        if (k + 1 < steps) load(k + 1);

        // the carry into this segment, and into the next step
        float* segs = seg_maps[k & 1];
        float* ctas = cta_maps[k & 1];
        Slots::write(segs, warp, lane, seg);
        __syncthreads();
        float h[V];
        Map<TWO> q[V];
        if (R > 1) {
            if (warp == kWarps - 1) {
                Map<TWO> all[V];
                Slots::read(segs, 0, lane, all);
                for (int i = 1; i < kWarps; ++i) {
                    Slots::read(segs, i, lane, q);
#pragma unroll
                    for (int v = 0; v < V; ++v) all[v] = join<TWO, PACKED>(all[v], q[v]);
                }
                for (int r = 0; r < R; ++r) Slots::send(ctas, rank, lane, r, all);
            }
            cluster_barrier();
            for (int r = 0; r < R; ++r) {
                Slots::read(ctas, r, lane, q);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (r == rank) h[v] = carry[v];
                    carry[v] = through<TWO, PACKED>(q[v], carry[v]);
                }
            }
            for (int i = 0; i < warp; ++i) {
                Slots::read(segs, i, lane, q);
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = through<TWO, PACKED>(q[v], h[v]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                Slots::read(segs, i, lane, q);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (i == warp) h[v] = carry[v];
                    carry[v] = through<TWO, PACKED>(q[v], carry[v]);
                }
            }
        }

        if (a.span_states && warp == 0 && n > 0 && active) {
            const size_t at = ((size_t)b * tiles + tile) * d + c;
            const bool none = PACKED && (!(m.valid & 1) || (m.begin & 1));
#pragma unroll
            for (int v = 0; v < V; ++v) a.span_states[at + v] = none ? 0.f : h[v];
        }
        Raw* qy = py + t0 * sy;
#pragma unroll
        for (int j = 0; j < kSeg; ++j) {
            if (PACKED && (m.begin >> j & 1)) {
                const int s = __shfl_sync(0xffffffffu, m.seq, j);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    h[v] = active && a.init_state ? a.init_state[(size_t)s * d + c + v] : 0.f;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float low = TWO ? fmaf(lo[TWO ? j : 0][v], h[v], in[j][v]) : in[j][v];
                h[v] = fmaf(da[j][v], h[v], low);
            }
            if ((m.valid >> j & 1) && active) qy[j * sy] = P::put(h);
            if (PACKED && (m.end >> j & 1)) {
                const int s = __shfl_sync(0xffffffffu, m.seq, j);
                if (a.final_state && active)
#pragma unroll
                    for (int v = 0; v < V; ++v) a.final_state[(size_t)s * d + c + v] = h[v];
            }
        }
    }
    // the carry behind the last tile is the final state, in every thread of the cluster
    if (!PACKED && a.final_state && rank == 0 && warp == 0 && active)
#pragma unroll
        for (int v = 0; v < V; ++v) a.final_state[(size_t)b * d + c + v] = carry[v];
}

template <typename T, int V>
cudaError_t dispatch_fwd_as(const GatedArgs& a, cudaStream_t st) {
    auto go = [&](auto logit, auto comp) {
        constexpr bool L = decltype(logit)::value, C = decltype(comp)::value;
        return a.cu ? launch_tiles(scan_kernel<T, V, L, C, true>, a, V, kFwdBlocks, st)
                    : launch_tiles(scan_kernel<T, V, L, C, false>, a, V, kFwdBlocks, st);
    };
    using Y = std::true_type;
    using N = std::false_type;
    if (a.logit) return a.complement ? go(Y{}, Y{}) : go(Y{}, N{});
    return a.complement ? go(N{}, Y{}) : go(N{}, N{});
}

template <typename T>
cudaError_t dispatch_fwd(const GatedArgs& a, cudaStream_t st) {
    if constexpr (sizeof(T) == 2)
        if (two_channels(a)) return dispatch_fwd_as<T, 2>(a, st);
    return dispatch_fwd_as<T, 1>(a, st);
}

}  // namespace gated
}  // namespace ssd
