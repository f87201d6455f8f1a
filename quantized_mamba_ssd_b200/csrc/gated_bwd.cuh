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
    constexpr int kRow = kInRow<T, CKPT>;
    using Pk = Pack<T>;
    constexpr bool kUsesU = COMP || LOGIT;      // the gradients need 1 - a
    constexpr bool kHold = V == 1 || !kUsesU;  // decays stay in registers; else they are computed again
    using F = Vec<V>;
    using Slots = MapSlots<V>;
    extern __shared__ __align__(128) uint8_t staged[];
    __shared__ __align__(16) float fwd_maps[2][kWarps * Slots::kFloats];
    __shared__ __align__(16) float seg_maps[2][kWarps * Slots::kFloats];
    __shared__ __align__(16) float cta_maps[2][kMaxCluster * Slots::kFloats];

    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int R = ta.cluster, rank = blockIdx.x % R, unit = blockIdx.x / R;
    const int d = a.channels, b = unit / ta.strips, c0 = unit % ta.strips * 32 * V;
    const int c = c0 + lane * V, count = max(0, min(V, d - c));
    const bool whole = d - c0 >= 32 * V && ta.pair_out;
    const int tiles = (a.seqlen + kTile - 1) / kTile, steps = (tiles + R - 1) / R;
    const size_t row0 = (size_t)b * a.seqlen;

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
    char* pdx = static_cast<char*>(const_cast<void*>(a.dx.ptr)) + (b * a.dx.batch_stride + c0) * sizeof(T);
    char* pdg = static_cast<char*>(const_cast<void*>(a.dgate.ptr)) + (b * a.dgate.batch_stride + c0) * sizeof(T);
    const long long sdy = a.dy.token_stride * sizeof(T), sdx = a.dx.token_stride * sizeof(T);
    const long long sdg = a.dgate.token_stride * sizeof(T);

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
    auto state_of = [&](const float* states, int s) {
        return load_floats<V>(states ? states + (size_t)s * d + c : nullptr, count);
    };

    F carry = PACKED ? splat<V>(0.f) : state_of(a.dfinal_state, b);
    if (PACKED && a.dinit_state && rank == 0)  // sequences without a token
        for (int s = warp; s < a.nseq; s += kWarps)
            if (__ldg(a.cu + s + 1) <= __ldg(a.cu + s))
                store_floats<V>(a.dinit_state + (size_t)s * d + c, state_of(a.dfinal_state, s), count);
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
        // the state before the tile, then before this warp's segment
        F before = load_floats<V>(
            tile >= 0 ? a.span_states + ((size_t)b * tiles + tile) * d + c : nullptr, count);
        F scale_x, scale_g;
        if constexpr (CKPT) {
            const size_t be = ((size_t)b * ta.blocks + t0 / kBlock) * d + c;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                scale_x.set(v, n > 0 && v < count ? scale_of(__ldg(a.x_e + be + v)) : 0.f);
                scale_g.set(v, n > 0 && v < count ? scale_of(__ldg(a.gate_e + be + v)) : 0.f);
            }
        }
        copy_wait<kBwdStages - 2>();
        __syncwarp();  // the segment is here, and every lane is done with the slot filled next
        stage(k + kBwdStages - 1);
        uint8_t* rx = slot(k, 0) + lane * (kRow / 32);
        uint8_t* rg = slot(k, 1) + lane * (kRow / 32);
        uint32_t* rdy = reinterpret_cast<uint32_t*>(slot(k, 2)) + lane;
        if (m.valid != kAll) {
            // tokens of no sequence pass state and gradient on: x and dy 0, decay 1 (each lane
            // mends its own words)
            for (int j = 0; j < kSeg; ++j)
                if (!(m.valid >> j & 1)) {
                    rdy[j * 32] = 0;
                    if constexpr (CKPT) {
#pragma unroll
                        for (int v = 0; v < V; ++v) rx[j * kRow + v] = rg[j * kRow + v] = 0;
                    } else {
                        *reinterpret_cast<uint32_t*>(rx + j * kRow) = 0;
                        *reinterpret_cast<uint32_t*>(rg + j * kRow) = LOGIT ? Pk::kInf : 0u;
                    }
                }
        }
        auto decoded = [&](const uint8_t* r, F scale, int j) {
            if constexpr (CKPT) {
                F f;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    f.set(v, static_cast<float>(reinterpret_cast<const int8_t*>(r)[j * kRow + v]));
                return mul(f, scale);
            } else {
                return Pk::get(*reinterpret_cast<const uint32_t*>(r + j * kRow));
            }
        };
        auto x_of = [&](int j) { return decoded(rx, scale_x, j); };
        auto gate_of = [&](int j) {
            F g = decoded(rg, scale_g, j);
            // no code stands for the logit of a decay of 1
            if (CKPT && LOGIT && !(m.valid >> j & 1)) g = splat<V>(INFINITY);
            return g;
        };

        // The segment's maps, both in one pass: of the state, which behind token j is P[j] carry +
        // B[j] (P with its low part Q in fp32), and of the gradient, which from behind the segment
        // reaches its first token through the product of the decays and from token j through P[j].
        F P[kSeg], Q[V == 1 ? kSeg : 1], B[kSeg];
        F da[kHold ? kSeg : 1], lo[V == 1 ? kSeg : 1], u[V == 1 && kUsesU ? kSeg : 1];
        Map<V> fwd = identity_map<V>(), back = identity_map<V>();
#pragma unroll
        for (int j = 0; j < kSeg; ++j) {
            F in = x_of(j), dy = Pk::get(rdy[j * 32]);
            const Decay<V> r = decay_of<LOGIT>(gate_of(j));
            if (PACKED && (m.begin >> j & 1))
                fwd.B = state_of(a.init_state, __shfl_sync(0xffffffffu, m.seq, j));
            if (PACKED && (m.end >> j & 1))
                dy = add(dy, state_of(a.dfinal_state, __shfl_sync(0xffffffffu, m.seq, j)));
            if constexpr (kHold) da[j] = r.a;
            if constexpr (V == 1) lo[j] = r.lo;
            if constexpr (V == 1 && kUsesU) u[j] = r.u;
            if constexpr (COMP) in = mul(r.u, in);
            fwd.B = step(r.a, r.lo, fwd.B, in);
            extend(fwd, r);
            P[j] = fwd.A;
            B[j] = fwd.B;
            if constexpr (V == 1) Q[j] = fwd.L;
            // behind the first end nothing reaches the segment's first token
            if (!PACKED || !(m.end & ((1u << j) - 1))) back.B = step(fwd.A, fwd.L, dy, back.B);
        }
        back.A = PACKED && m.end ? splat<V>(-1.f) : fwd.A;
        back.L = fwd.L;
        if (PACKED && m.begin) fwd.A = splat<V>(-1.f);

        float* segs = seg_maps[k & 1];
        float* fwds = fwd_maps[k & 1];
        const int order = kWarps - 1 - warp;  // place of this warp's run
        F e;                                  // the gradient from behind this segment
        Slots::write(segs, order, lane, back);
        Slots::write(fwds, warp, lane, fwd);
        __syncthreads();
        if (R > 1) {
            float* ctas = cta_maps[k & 1];
            if (warp == 0) {
                const Map<V> all = Slots::template join_runs<PACKED>(segs, lane);
                for (int r = 0; r < R; ++r) Slots::send(ctas, rank, lane, r, all);
            }
            cluster_barrier(warp == 0);
            e = Slots::template carry_through<PACKED>(ctas, R, rank, lane, carry);
            e = Slots::template carry_into<PACKED>(segs, order, lane, e);
        } else {
            e = Slots::template carry_through<PACKED>(segs, kWarps, order, lane, carry);
        }
        before = Slots::template carry_into<PACKED>(fwds, warp, lane, before);

        F past0 = before;  // the state before the segment
        if (PACKED && m.begin) {  // it only reaches the tokens before the first beginning
#pragma unroll
            for (int j = 0; j < kSeg; ++j) {
                if (!(m.begin & ((2u << j) - 1))) B[j] = step(P[j], Q[V == 1 ? j : 0], before, B[j]);
                P[j] = splat<V>(0.f);
                if constexpr (V == 1) Q[j] = P[j];
            }
            before = splat<V>(0.f);
        }
        // token j's gradients, from the last token to the first
        auto gradients = [&](int j, F& dx, F& dg) {
            if (PACKED && (m.end >> j & 1))
                e = state_of(a.dfinal_state, __shfl_sync(0xffffffffu, m.seq, j));
            F past = j ? step(P[j ? j - 1 : 0], Q[V == 1 && j ? j - 1 : 0], before, B[j ? j - 1 : 0]) : past0;
            if (PACKED && (m.begin >> j & 1))
                past = state_of(a.init_state, __shfl_sync(0xffffffffu, m.seq, j));
            Decay<V> r;
            if constexpr (kHold) {
                r.a = da[j];
                r.lo = lo[V == 1 ? j : 0];
                r.u = u[V == 1 && kUsesU ? j : 0];
            } else {
                r = decay_of<LOGIT>(gate_of(j));
            }
            const F dh = add(Pk::get(rdy[j * 32]), e);
            e = step(r.a, r.lo, dh, splat<V>(0.f));
            dx = COMP ? mul(r.u, dh) : dh;
            if constexpr (COMP) past = sub(past, x_of(j));
            dg = mul(e, past);
            if constexpr (LOGIT) dg = mul(dg, r.u);
            if (PACKED && (m.begin >> j & 1)) {
                const int s = __shfl_sync(0xffffffffu, m.seq, j);
                if (a.dinit_state) store_floats<V>(a.dinit_state + (size_t)s * d + c, e, count);
            }
        };
        char* qdx = pdx + (t0 + kSeg - 1) * sdx + lane * 4;
        char* qdg = pdg + (t0 + kSeg - 1) * sdg + lane * 4;
        const bool plain = whole && m.valid == kAll;
#pragma unroll
        for (int j = kSeg - 1; j >= 0; --j) {
            F dx, dg;
            gradients(j, dx, dg);
            if (plain) {
                *reinterpret_cast<uint32_t*>(qdx) = Pk::put(dx);
                *reinterpret_cast<uint32_t*>(qdg) = Pk::put(dg);
            } else if (m.valid >> j & 1) {
                store_row<T>(qdx, dx, whole, count);
                store_row<T>(qdg, dg, whole, count);
            }
            qdx -= sdx;
            qdg -= sdg;
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
