// Backward gated scan (the tile scheme is described in gated_tile.cuh).
//
// The gradient E_t that a sequence's tokens from t on send to h_{t-1} obeys E_t = a_t (E_{t+1} +
// dy_t), a recurrence of the same kind in the other direction: the cluster walks the tiles from the
// last one down.  The states h_{t-1} that dgate needs are rebuilt inside each tile from the state
// that the forward pass saved before it, so x, gate and dy are read once and dx and dgate written
// once, and nothing depends on the rounding of y.
#pragma once

#include <type_traits>

#include "gated_launch.cuh"

namespace ssd {
namespace gated {

// Staged inputs: x, gate and dy as rows of 128 bytes, or codes as rows of one byte per channel.
template <typename T, bool CKPT>
constexpr int kInRow = CKPT ? 32 * kChannels<T> : kRowBytes;
template <typename T, bool CKPT>
constexpr int kBwdStage = kTile * (2 * kInRow<T, CKPT> + kRowBytes);
template <typename T, bool CKPT>
constexpr int kBwdSmem = kBwdStages * kBwdStage<T, CKPT>;

template <typename T, bool LOGIT, bool COMP, bool PACKED, bool CKPT>
__global__ void __launch_bounds__(kTileThreads, kBwdBlocks)
scan_bwd_kernel(const __grid_constant__ GatedArgs a, const TileArgs ta) {
    constexpr int V = kChannels<T>;
    constexpr bool TWO = kTwo<T>;
    constexpr int kRow = kInRow<T, CKPT>;
    using P = Pack<T>;
    using Slots = MapSlots<V, TWO>;
    extern __shared__ __align__(128) uint8_t staged[];
    __shared__ float fwd_maps[2][kWarps * Slots::kFloats];
    __shared__ float seg_maps[2][kWarps * Slots::kFloats];
    __shared__ float cta_maps[2][kMaxCluster * Slots::kFloats];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, R = ta.cluster;
    const int rank = blockIdx.x % R, unit = blockIdx.x / R;
    const int d = a.channels, b = unit / ta.strips, c0 = unit % ta.strips * 32 * V;
    const int c = c0 + lane * V, count = max(0, min(V, d - c));
    const int tiles = (a.seqlen + kTile - 1) / kTile, steps = (tiles + R - 1) / R;
    const size_t row0 = (size_t)b * a.seqlen;
    const float gate_one = LOGIT ? INFINITY : 0.f;  // the gate of a decay of 1

    const int width = min(kRowBytes, (d - c0) * (int)sizeof(T));
    const char *px, *pg;
    long long sx, sg;
    if constexpr (CKPT) {
        px = reinterpret_cast<const char*>(a.x_q) + row0 * d + c0;
        pg = reinterpret_cast<const char*>(a.gate_q) + row0 * d + c0;
        sx = sg = d;
    } else {
        px = static_cast<const char*>(a.x.ptr) + (b * a.x.batch_stride + c0) * sizeof(T);
        pg = static_cast<const char*>(a.gate.ptr) + (b * a.gate.batch_stride + c0) * sizeof(T);
        sx = a.x.token_stride * sizeof(T);
        sg = a.gate.token_stride * sizeof(T);
    }
    const char* pdy = static_cast<const char*>(a.dy.ptr) + (b * a.dy.batch_stride + c0) * sizeof(T);
    const long long sdy = a.dy.token_stride * sizeof(T);
    T* pdx = static_cast<T*>(const_cast<void*>(a.dx.ptr)) + b * a.dx.batch_stride + c;
    T* pdg = static_cast<T*>(const_cast<void*>(a.dgate.ptr)) + b * a.dgate.batch_stride + c;

    // rows of step k: x, gate (or their codes), dy
    auto slot = [&](int k, int tensor) {
        return staged + (k % kBwdStages) * kBwdStage<T, CKPT> +
               (tensor < 2 ? (tensor * kWarps + warp) * kSeg * kRow
                           : 2 * kTile * kRow + warp * kSeg * kRowBytes);
    };
    auto stage = [&](int k) {
        const int t0 = (tiles - 1 - (k * R + rank)) * kTile + warp * kSeg;
        if (k < steps && t0 >= 0) {
            const int n = max(0, min(kSeg, a.seqlen - t0));
            const int in_width = CKPT ? min(kRow, d - c0) : width;
            stage_rows<kRow>(slot(k, 0), n ? px + t0 * sx : px, sx, n, in_width,
                             CKPT ? ta.align_codes : ta.align_x);
            stage_rows<kRow>(slot(k, 1), n ? pg + t0 * sg : pg, sg, n, in_width,
                             CKPT ? ta.align_codes : ta.align_gate);
            stage_rows<kRowBytes>(slot(k, 2), n ? pdy + t0 * sdy : pdy, sdy, n, width, ta.align_dy);
        }
        copy_commit();
    };

    float carry[V];
    load_floats<V>(!PACKED && a.dfinal_state ? a.dfinal_state + (size_t)b * d + c : nullptr, carry, count);
    if (PACKED && a.dinit_state && rank == 0) {  // sequences without a token
        for (int s = warp; s < a.nseq; s += kWarps) {
            if (__ldg(a.cu + s + 1) > __ldg(a.cu + s)) continue;
            float h[V];
            load_floats<V>(a.dfinal_state ? a.dfinal_state + (size_t)s * d + c : nullptr, h, count);
            store_floats<V>(a.dinit_state + (size_t)s * d + c, h, count);
        }
    }
    Held held;
#pragma unroll
    for (int k = 0; k < kBwdStages - 1; ++k) stage(k);
    for (int k = 0; k < steps; ++k) {
        const int tile = tiles - 1 - (k * R + rank);  // below 0: nothing left for this CTA
        const int t0 = tile * kTile + warp * kSeg;
        const int n = tile < 0 ? 0 : max(0, min(kSeg, a.seqlen - t0));
        Marks m;
        m.valid = (1u << n) - 1;
        m.begin = m.end = 0;
        if constexpr (PACKED) m = marks_of(a.cu, a.nseq, t0, n, held);
        float before[V];  // the state before the tile, then before this warp's segment
        load_floats<V>(tile >= 0 ? a.span_states + ((size_t)b * tiles + tile) * d + c : nullptr,
                       before, count);
        float scale_x[V], scale_g[V];
        if constexpr (CKPT) {
            const size_t be = ((size_t)b * ta.blocks + t0 / kBlock) * d + c;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                scale_x[v] = n > 0 && v < count ? scale_of(__ldg(a.x_e + be + v)) : 1.f;
                scale_g[v] = n > 0 && v < count ? scale_of(__ldg(a.gate_e + be + v)) : 1.f;
            }
        }
        copy_wait<kBwdStages - 2>();
        __syncwarp();  // the segment is here, and every lane is done with the slot filled next
        stage(k + kBwdStages - 1);
        const uint8_t* rx = slot(k, 0) + lane * (kRow / 32);
        const uint8_t* rg = slot(k, 1) + lane * (kRow / 32);
        const uint32_t* rdy = reinterpret_cast<const uint32_t*>(slot(k, 2)) + lane;
        auto get = [&](const uint8_t* r, const float (&scale)[V], int j, float (&f)[V], float none) {
            if constexpr (CKPT) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    f[v] = scale[v] * static_cast<float>(reinterpret_cast<const int8_t*>(r)[j * kRow + v]);
            } else {
                P::get(*reinterpret_cast<const uint32_t*>(r + j * kRow), f);
            }
            if (!(m.valid >> j & 1))
#pragma unroll
                for (int v = 0; v < V; ++v) f[v] = none;
        };
        auto get_dy = [&](int j, float (&f)[V]) {
            P::get(rdy[j * 32], f);
            if (!(m.valid >> j & 1))
#pragma unroll
                for (int v = 0; v < V; ++v) f[v] = 0.f;
        };
        auto init_of = [&](int j, float (&h)[V]) {
            const int s = __shfl_sync(0xffffffffu, m.seq, j);
            load_floats<V>(a.init_state ? a.init_state + (size_t)s * d + c : nullptr, h, count);
        };
        auto dfinal_of = [&](int j, float (&h)[V]) {
            const int s = __shfl_sync(0xffffffffu, m.seq, j);
            load_floats<V>(a.dfinal_state ? a.dfinal_state + (size_t)s * d + c : nullptr, h, count);
        };

        // The segment's maps, both in one pass: of the state (forward), and of the gradient, which
        // from behind the segment reaches its first token through the product of the decays and
        // from token j through the product up to j.
        float da[kSeg][V], lo[TWO ? kSeg : 1][V];
        Map<TWO> fwd[V], back[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            fwd[v] = identity_map<TWO>();
            back[v].B = 0.f;
        }
#pragma unroll
        for (int j = 0; j < kSeg; ++j) {
            float x[V], g[V], dy[V];
            get(rx, scale_x, j, x, 0.f);
            get(rg, scale_g, j, g, gate_one);
            get_dy(j, dy);
            if (PACKED && (m.begin >> j & 1)) {
                float h[V];
                init_of(j, h);
#pragma unroll
                for (int v = 0; v < V; ++v) fwd[v].B = h[v];
            }
            if (PACKED && (m.end >> j & 1)) {
                float e[V];
                dfinal_of(j, e);
#pragma unroll
                for (int v = 0; v < V; ++v) dy[v] += e[v];
            }
            // behind the first end nothing reaches the segment's first token
            const bool open = !PACKED || !(m.end & ((1u << j) - 1));
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Decay r = decay_of<T, LOGIT>(g[v]);
                da[j][v] = r.a;
                if constexpr (TWO) lo[j][v] = r.lo;
                fwd[v].B = step<TWO>(r, fwd[v].B, COMP ? r.u * x[v] : x[v]);
                extend<TWO>(fwd[v], r);
                if (open) {
                    if constexpr (TWO) back[v].B = fmaf(fwd[v].L, dy[v], back[v].B);
                    back[v].B = fmaf(fwd[v].A, dy[v], back[v].B);
                }
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            back[v].A = PACKED && m.end ? -1.f : fwd[v].A;
            if constexpr (TWO) back[v].L = fwd[v].L;
            if (PACKED && m.begin) fwd[v].A = -1.f;
        }

        float* segs = seg_maps[k & 1];
        float* fwds = fwd_maps[k & 1];
        float e[V];  // the gradient from behind this segment
        Slots::write(segs, kWarps - 1 - warp, lane, back);
        Slots::write(fwds, warp, lane, fwd);
        __syncthreads();
        const int order = kWarps - 1 - warp;  // place of this warp's run
        if (R > 1) {
            float* ctas = cta_maps[k & 1];
            if (warp == 0) {
                Map<TWO> all[V];
                Slots::template join_runs<PACKED>(segs, lane, all);
                for (int r = 0; r < R; ++r) Slots::send(ctas, rank, lane, r, all);
            }
            cluster_barrier();
            Slots::template carry_through<PACKED>(ctas, R, rank, lane, carry, e);
            Slots::template carry_into<PACKED>(segs, order, lane, e);
        } else {
            Slots::template carry_through<PACKED>(segs, kWarps, order, lane, carry, e);
        }
        Slots::template carry_into<PACKED>(fwds, warp, lane, before);

        // the state before every token
        float h[kSeg][V];
#pragma unroll
        for (int j = 0; j < kSeg; ++j) {
            float x[V], g[V];
            get(rx, scale_x, j, x, 0.f);
            if constexpr (COMP) get(rg, scale_g, j, g, gate_one);
            if (PACKED && (m.begin >> j & 1)) init_of(j, before);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                h[j][v] = before[v];
                const float in = COMP ? decay_of<T, LOGIT>(g[v]).u * x[v] : x[v];
                before[v] = fmaf(da[j][v], before[v],
                                 TWO ? fmaf(lo[TWO ? j : 0][v], before[v], in) : in);
            }
        }
        T* qdx = pdx + t0 * a.dx.token_stride;
        T* qdg = pdg + t0 * a.dgate.token_stride;
#pragma unroll
        for (int j = kSeg - 1; j >= 0; --j) {
            float x[V], g[V], dy[V], dx[V], dg[V];
            if constexpr (COMP) get(rx, scale_x, j, x, 0.f);
            if constexpr (COMP || LOGIT) get(rg, scale_g, j, g, gate_one);
            get_dy(j, dy);
            if (PACKED && (m.end >> j & 1)) dfinal_of(j, e);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float dh = dy[v] + e[v];
                e[v] = da[j][v] * dh;
                if constexpr (TWO) e[v] = fmaf(da[j][v], dh, lo[TWO ? j : 0][v] * dh);
                const float u = COMP || LOGIT ? decay_of<T, LOGIT>(g[v]).u : 1.f;
                dx[v] = COMP ? u * dh : dh;
                dg[v] = e[v] * (COMP ? h[j][v] - x[v] : h[j][v]);
                if constexpr (LOGIT) dg[v] *= u;
            }
            if (m.valid >> j & 1) {
                store_row<T>(qdx + j * a.dx.token_stride, dx, ta.pair_out, count);
                store_row<T>(qdg + j * a.dgate.token_stride, dg, ta.pair_out, count);
            }
            if (PACKED && (m.begin >> j & 1)) {
                const int s = __shfl_sync(0xffffffffu, m.seq, j);
                if (a.dinit_state) store_floats<V>(a.dinit_state + (size_t)s * d + c, e, count);
            }
        }
    }
    // the carry behind the first tile is the initial state's gradient, in every thread
    if (!PACKED && a.dinit_state && rank == 0 && warp == 0)
        store_floats<V>(a.dinit_state + (size_t)b * d + c, carry, count);
}

template <typename T, bool LOGIT>
cudaError_t dispatch_bwd(const GatedArgs& a, cudaStream_t st) {
    auto go = [&](auto comp, auto packed, auto ckpt) {
        constexpr bool C = decltype(comp)::value, K = decltype(packed)::value, Q = decltype(ckpt)::value;
        return launch_tiles<T>(scan_bwd_kernel<T, LOGIT, C, K, Q>, a, kBwdBlocks, kBwdSmem<T, Q>, st);
    };
    using Y = std::true_type;
    using N = std::false_type;
    auto packed = [&](auto comp, auto ckpt) { return a.cu ? go(comp, Y{}, ckpt) : go(comp, N{}, ckpt); };
    auto input = [&](auto ckpt) { return a.complement ? packed(Y{}, ckpt) : packed(N{}, ckpt); };
    return a.x_q ? input(Y{}) : input(N{});
}

}  // namespace gated
}  // namespace ssd
