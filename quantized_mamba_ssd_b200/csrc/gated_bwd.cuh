// Backward gated scan (the walk along strips is described in gated_tile.cuh).
//
// The gradient E_t that a sequence's tokens from t on send to h_{t-1} obeys E_t = a_t (E_{t+1} +
// dy_t), a recurrence of the same kind in the other direction: strips are walked from the last tile
// down.  The states h_{t-1} that dgate needs are rebuilt in each segment from the state that the
// forward pass saved before its span, so x, gate and dy are read once and dx and dgate written once,
// and nothing depends on the rounding of y.
//
// What bounds it (one B200, of the measured copy bandwidth 6.47 TB/s): with enough strips HBM - 8 x
// 4096 x 5120 bf16 287 us, 90 %; 2 x 16384 x 8192 logits with 1 - a weights 484 us, 86 %; 4 x 2048 x
// 4096 bf16 62 us, 84 %, fp32 133 to 140 us, 78 to 74 % - else the instructions.  From codes, where 65 us
// are 65 % (with 1 - a 79, logits 82, fp32 132 to 172), neither: half of the issue slots are free and DRAM
// gives 3.6 TB/s.  The main stall is the wait for global memory: a segment's scales and span state are
// loaded in the step that uses them.  31 of the 48 kernels from codes also spill, 12 to 124 bytes a thread
// (4 warps with registers enough took 89 us).
// The hot loop has to stay small and contiguous: with the tokens' checks of sequence borders and of
// odd rows inside it instead of in loops of their own, the second took 760 us.
#pragma once

#include <type_traits>

#include "gated_launch.cuh"

namespace ssd {
namespace gated {

// A warp's staged segment: x and gate (rows of 128 bytes, or codes, one byte per channel) and dy.
template <typename T, bool CKPT> constexpr int kInRow = CKPT ? 32 * kChannels<T> : kRowBytes;
template <typename T, bool CKPT, bool ANY>
constexpr int kBwdSegBytes = 2 * kSubBytes<kInRow<T, CKPT>, ANY> + kSubBytes<kRowBytes, ANY>;
constexpr int kSpanSegs = kSpan / kSub;
constexpr int kBwdSlots = 2;
template <int V, int W> constexpr int kFwdMapBytes = 2 * W * MapSlots<V>::kFloats * 4;

// The lane's channels of one staged row: values, or codes times their scales.  MARKS: the code kCodeNaN
// is NaN (it only stands in segments with a sequence border, and those have loops of their own).
template <typename T, bool CKPT, bool ANY, bool MARKS>
__device__ __forceinline__ Vec<kChannels<T>> row_value(const uint8_t* r, Vec<kChannels<T>> scale) {
    constexpr int V = kChannels<T>;
    if constexpr (CKPT && V == 2) {
        // code + 128 in the low byte of 2^23 is that number as a float, less 2^23 + 128 the code (in
        // one instruction with the scale, 2^23 of the largest ones would not be a number)
        const uint32_t q = (ANY ? r[0] | r[1] << 8 : *reinterpret_cast<const uint16_t*>(r)) ^ 0x8080u;
        Vec<2> f;
        f.x = make_float2(__uint_as_float(__byte_perm(q, 0x4b000000u, 0x7440)),
                          __uint_as_float(__byte_perm(q, 0x4b000000u, 0x7441)));
        f = mul(add(f, splat<V>(-8388736.f)), scale);
        if constexpr (MARKS) {
            if (!(q & 0x00ffu)) f.x.x = NAN;
            if (!(q & 0xff00u)) f.x.y = NAN;
        }
        return f;
    } else if constexpr (CKPT) {
        if (MARKS && *r == kCodeNaN) return {NAN};
        return mul(Vec<1>{static_cast<float>(*reinterpret_cast<const int8_t*>(r))}, scale);
    } else {
        return Pack<T>::get(row_word<T, ANY>(r));
    }
}

template <typename T, bool LOGIT, bool COMP, bool PACKED, bool CKPT, bool ANY>
__global__ void __launch_bounds__(32 * kBwdWarps<CKPT>, kBwdBlocks<CKPT>)
scan_bwd_kernel(const __grid_constant__ GatedArgs a, const __grid_constant__ TileArgs ta) {
    constexpr int V = kChannels<T>, kRow = kInRow<T, CKPT>;
    constexpr bool kUsesU = COMP || LOGIT;  // the gradients need 1 - a
    constexpr bool kStates = !kUsesU;       // the states stay in registers as maps of the carry
    using Pk = Pack<T>;
    using F = Vec<V>;
    extern __shared__ __align__(128) uint8_t staged[];

    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    constexpr int W = kBwdWarps<CKPT>;
    const int chunk = blockIdx.x % ta.chunks, unit = blockIdx.x / ta.chunks;
    const int d = a.channels, b = unit / ta.strips, c0 = unit % ta.strips * 32 * V;
    const int c = c0 + lane * V, count = max(0, min(V, d - c));
    const bool whole = ta.whole_out;
    const int tiles = (ta.blocks + W - 1) / W, low = chunk * ta.chunk_tiles;  // the chunk's first tile
    const int steps = min(tiles - low, ta.chunk_tiles);
    const size_t row0 = (size_t)b * a.seqlen;

    const int width = min(kRowBytes, (d - c0) * (int)sizeof(T));
    const int in_width = CKPT ? min(kRow, d - c0) : width;
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
    char* pdx = static_cast<char*>(const_cast<void*>(a.dx.ptr)) +
                (b * a.dx.batch_stride + c0) * sizeof(T);
    char* pdg = static_cast<char*>(const_cast<void*>(a.dgate.ptr)) +
                (b * a.dgate.batch_stride + c0) * sizeof(T);
    const long long sdy = a.dy.token_stride * sizeof(T), sdx = a.dx.token_stride * sizeof(T);
    const long long sdg = a.dgate.token_stride * sizeof(T);

    // the gradient's maps meet; the state's only serve the warps of the same tile
    float* maps = reinterpret_cast<float*>(staged);
    float* fwds = reinterpret_cast<float*>(staged + kMeetingBytes<V, W>);
    constexpr int kSeg = kBwdSegBytes<T, CKPT, ANY>, kIn = kSubBytes<kRow, ANY>;
    uint8_t* own = staged + kMeetingBytes<V, W> + kFwdMapBytes<V, W> + warp * kBwdSlots * kSeg;
    const int qx = staged_pitch<kRow, ANY>(sx), qg = staged_pitch<kRow, ANY>(sg);
    const int qdy = staged_pitch<kRowBytes, ANY>(sdy);
    // tiles of W segments, from the chunk's last one down
    auto start = [&](int k) { return ((low + steps - 1 - k) * W + warp) * kSub; };
    auto stage = [&](int k) {
        const int t = start(k), n = max(0, min(kSub, a.seqlen - t));
        if (k < steps && n > 0) {
            uint8_t* to = own + k % kBwdSlots * kSeg;
            if (n == kSub) [[likely]] {
                stage_rows<kRow, ANY>(to, px + t * sx, sx, in_width);
                stage_rows<kRow, ANY>(to + kIn, pg + t * sg, sg, in_width);
                stage_rows<kRowBytes, ANY>(to + 2 * kIn, pdy + t * sdy, sdy, width);
            } else {
                stage_part<kRow, ANY>(to, px + t * sx, sx, n, in_width);
                stage_part<kRow, ANY>(to + kIn, pg + t * sg, sg, n, in_width);
                stage_part<kRowBytes, ANY>(to + 2 * kIn, pdy + t * sdy, sdy, n, width);
            }
        }
        copy_commit();
    };
    auto state_of = [&](const float* states, int s) {
        return load_floats<V>(states ? states + (size_t)s * d + c : nullptr, count);
    };

    F carry = PACKED ? splat<V>(0.f) : state_of(a.dfinal_state, b);
    if (PACKED && a.dinit_state)
        for_empty_sequences(a.cu, a.nseq, chunk * W + warp, ta.chunks * W, [&](int s) {
            store_floats<V>(a.dinit_state + (size_t)s * d + c, state_of(a.dfinal_state, s), count);
        });
#pragma unroll 1
    for (int k = 0; k < kBwdSlots - 1; ++k) stage(k);
    if (ta.chunks > 1) {
        wait_for_previous_kernel();
        const float* of_chunks = ta.maps + (size_t)unit * ta.chunks * MapSlots<V>::kFloats;
        carry = through_chunks<PACKED>(of_chunks, ta.chunks - 1, ta.chunks - 1 - chunk, -1, lane, carry);
    }
    Held held;
    for (int k = 0; k < steps; ++k) {
        const int t0 = start(k), n = max(0, min(kSub, a.seqlen - t0));
        Marks m;
        m.valid = (1u << n) - 1;
        m.begin = m.end = 0;
        if constexpr (PACKED) m = marks_of(a.cu, a.nseq, t0, n, held);
        // the state before the segment's span, then before the segment
        F before = load_floats<V>(
            n > 0 ? a.span_states + ((size_t)b * ta.spans + t0 / kSpan) * d + c : nullptr, count);
        F scale_x, scale_g;
        if constexpr (CKPT) {
            const size_t be = ((size_t)b * ta.blocks + t0 / kBlock) * d + c;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                scale_x.set(v, n > 0 && v < count ? scale_of(__ldg(a.x_e + be + v)) : 0.f);
                scale_g.set(v, n > 0 && v < count ? scale_of(__ldg(a.gate_e + be + v)) : 0.f);
            }
        }
        copy_wait<kBwdSlots - 2>();
        __syncwarp();  // the segment is here, and every lane is done with the slot filled next
        stage(k + kBwdSlots - 1);
        uint8_t* here = own + k % kBwdSlots * kSeg;
        uint8_t* rx = here + staged_start<ANY>(px + t0 * sx) + lane * (kRow / 32);
        uint8_t* rg = here + kIn + staged_start<ANY>(pg + t0 * sg) + lane * (kRow / 32);
        uint8_t* rdy = here + 2 * kIn + staged_start<ANY>(pdy + t0 * sdy) + lane * 4;
        if (m.valid != kAll) [[unlikely]] {
            // tokens of no sequence pass state and gradient on: x and dy 0, decay 1 (each lane
            // mends its own words)
            for (int j = 0; j < kSub; ++j)
                if (!(m.valid >> j & 1)) {
                    set_row_word<T, ANY>(rdy + j * qdy, 0u);
                    if constexpr (CKPT) {
#pragma unroll
                        for (int v = 0; v < V; ++v) rx[j * qx + v] = rg[j * qg + v] = 0;
                    } else {
                        set_row_word<T, ANY>(rx + j * qx, 0u);
                        set_row_word<T, ANY>(rg + j * qg, LOGIT ? Pk::kInf : 0u);
                    }
                }
        }
        auto dy_of = [&](int j) { return Pk::get(row_word<T, ANY>(rdy + j * qdy)); };
        auto x_of = [&](auto checks, int j) {
            return row_value<T, CKPT, ANY, PACKED && decltype(checks)::value>(rx + j * qx, scale_x);
        };
        auto gate_of = [&](auto checks, int j) {
            F g = row_value<T, CKPT, ANY, PACKED && decltype(checks)::value>(rg + j * qg, scale_g);
            // no code stands for the logit of a decay of 1
            if (CKPT && LOGIT && !(m.valid >> j & 1)) g = splat<V>(INFINITY);
            return g;
        };

        // The segment's maps, both in one pass: of the state, and of the gradient, which from behind
        // the segment reaches its first token through the product of the decays and from token j
        // through the product up to j.  Where registers allow it (kStates), the state behind token j
        // is kept as the product P[j] and the rest B[j], which together with the carry give it at
        // once; else the states are computed again from the decays, which are kept in either case.
        F P[kStates ? kSub : 1], Q[kStates && V == 1 ? kSub : 1], B[kStates ? kSub : 1];
        F da[kSub], lo[V == 1 ? kSub : 1], u[kUsesU ? kSub : 1];
        Map<V> fwd = identity_map<V>(), back = identity_map<V>();
        // segments inside one sequence, by far the most, go without the checks of every token
        const bool inside = !PACKED || !(m.begin | m.end);
        auto reduce = [&](auto checks) {
            constexpr bool CHECK = decltype(checks)::value;
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
                F in = x_of(checks, j), dy = dy_of(j);
                const Decay<V> r = decay_of<LOGIT>(gate_of(checks, j));
                if (CHECK && (m.begin >> j & 1))
                    fwd.B = state_of(a.init_state, __shfl_sync(0xffffffffu, m.seq, j));
                if (CHECK && (m.end >> j & 1))
                    dy = add(dy, state_of(a.dfinal_state, __shfl_sync(0xffffffffu, m.seq, j)));
                da[j] = r.a;
                if constexpr (V == 1) lo[j] = r.lo;
                if constexpr (kUsesU) u[j] = r.u;
                if constexpr (COMP) in = mul(r.u, in);
                fwd.B = step(r.a, r.lo, fwd.B, in);
                extend(fwd, r);
                if constexpr (kStates) {
                    P[j] = fwd.A;
                    B[j] = fwd.B;
                    if constexpr (V == 1) Q[j] = fwd.L;
                }
                // behind the first end nothing reaches the segment's first token
                if (!CHECK || !(m.end & ((1u << j) - 1))) back.B = step(fwd.A, fwd.L, dy, back.B);
            }
        };
        if (inside) [[likely]] reduce(std::false_type{});
        else reduce(std::true_type{});
        back.A = PACKED && m.end ? splat<V>(-1.f) : fwd.A;
        back.L = fwd.L;
        if (PACKED && m.begin) fwd.A = splat<V>(-1.f);

        float* states = fwds + (k & 1) * W * MapSlots<V>::kFloats;
        MapSlots<V>::write(states, warp, lane, fwd);
        // the gradient from behind the segment
        F e = meet<PACKED, W>(maps, k, W - 1 - warp, back, carry);
        // (the spans of a tile begin at multiples of kSpanSegs warps)
        const Map<V> into = MapSlots<V>::template join_runs<PACKED, W>(
            states, warp - warp % kSpanSegs, warp, lane);
        before = through<PACKED>(into, before);

        char* qdx = pdx + (t0 + kSub - 1) * sdx + lane * 4;
        char* qdg = pdg + (t0 + kSub - 1) * sdg + lane * 4;
        auto gradients = [&](auto checks, auto wholes) {
            constexpr bool CHECK = decltype(checks)::value, WHOLE = decltype(wholes)::value;
            // what the gradient of token j's decay multiplies: h_{j-1}, or h_{j-1} - x_j
            F past[kSub];
#pragma unroll
            for (int j = 0; j < kSub; ++j) {
                const bool begins = CHECK && (m.begin >> j & 1);
                if constexpr (!kStates) {
                    F in = x_of(checks, j);
                    if (begins) before = state_of(a.init_state, __shfl_sync(0xffffffffu, m.seq, j));
                    past[j] = COMP ? sub(before, in) : before;
                    if constexpr (COMP) in = mul(u[kUsesU ? j : 0], in);
                    before = step(da[j], lo[V == 1 ? j : 0], before, in);
                } else {
                    constexpr int none = 0;
                    const int i = j ? j - 1 : none;
                    if (begins) past[j] = state_of(a.init_state, __shfl_sync(0xffffffffu, m.seq, j));
                    else if (!j) past[j] = before;
                    else if (CHECK && (m.begin & ((1u << j) - 1))) past[j] = B[i];  // the carry ends there
                    else past[j] = step(P[i], Q[V == 1 ? i : 0], before, B[i]);
                }
            }
#pragma unroll
            for (int j = kSub - 1; j >= 0; --j) {
                if (CHECK && (m.end >> j & 1))
                    e = state_of(a.dfinal_state, __shfl_sync(0xffffffffu, m.seq, j));
                const F dh = add(dy_of(j), e);
                e = step(da[j], lo[V == 1 ? j : 0], dh, splat<V>(0.f));
                const F dx = COMP ? mul(u[kUsesU ? j : 0], dh) : dh;
                F dg = mul(e, past[j]);
                if constexpr (LOGIT) dg = mul(dg, u[kUsesU ? j : 0]);
                if (CHECK && (m.begin >> j & 1)) {
                    const int s = __shfl_sync(0xffffffffu, m.seq, j);
                    if (a.dinit_state) store_floats<V>(a.dinit_state + (size_t)s * d + c, e, count);
                }
                if (!CHECK || (m.valid >> j & 1)) {
                    store_row<T>(qdx, dx, WHOLE || (CHECK && whole), count);
                    store_row<T>(qdg, dg, WHOLE || (CHECK && whole), count);
                }
                qdx -= sdx;
                qdg -= sdg;
            }
        };
        const bool plain = inside && m.valid == kAll;
        if (plain && whole) [[likely]] gradients(std::false_type{}, std::true_type{});
        else if (ANY && plain) gradients(std::false_type{}, std::false_type{});
        else gradients(std::true_type{}, std::false_type{});
    }
    // the carry behind the first tile is the initial state's gradient, in every thread of its CTA
    if (!PACKED && a.dinit_state && chunk == 0 && warp == 0)
        store_floats<V>(a.dinit_state + (size_t)b * d + c, carry, count);
}

// The gradient's maps of all chunks but the first of every strip: each warp reduces a run of whole
// segments of gate (or its codes) and dy, in the order of the tokens (see the scan's own map).
template <bool ANY> constexpr int kBackSlots = ANY ? 2 : 3;
template <typename T, bool CKPT, bool ANY>
constexpr int kBackSegBytes = kSubBytes<kInRow<T, CKPT>, ANY> + kSubBytes<kRowBytes, ANY>;

template <typename T, bool LOGIT, bool PACKED, bool CKPT, bool ANY>
__global__ void __launch_bounds__(32 * kMapWarps)
chunk_back_kernel(const __grid_constant__ GatedArgs a, const __grid_constant__ TileArgs ta) {
    constexpr int V = kChannels<T>, W = kMapWarps, kRow = kInRow<T, CKPT>;
    using Pk = Pack<T>;
    using F = Vec<V>;
    extern __shared__ __align__(128) uint8_t staged[];

    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int chunk = 1 + blockIdx.x % (ta.chunks - 1), unit = blockIdx.x / (ta.chunks - 1);
    const int d = a.channels, b = unit / ta.strips, c0 = unit % ta.strips * 32 * V;
    const int c = c0 + lane * V, count = max(0, min(V, d - c));
    // segments of the chunk, and of a warp (of full rows a tile has fewer than this CTA warps)
    const int all_of_them = ta.chunk_tiles * kBwdWarps<CKPT>, each = (all_of_them + W - 1) / W;
    const int first = chunk * all_of_them + warp * each, run = max(0, min(each, all_of_them - warp * each));

    const int width = min(kRowBytes, (d - c0) * (int)sizeof(T));
    const char* pg = CKPT ? reinterpret_cast<const char*>(a.gate_q) + (size_t)b * a.seqlen * d + c0
                          : static_cast<const char*>(a.gate.ptr) + (b * a.gate.batch_stride + c0) * sizeof(T);
    const long long sg = CKPT ? d : a.gate.token_stride * sizeof(T);
    const char* pdy = static_cast<const char*>(a.dy.ptr) + (b * a.dy.batch_stride + c0) * sizeof(T);
    const long long sdy = a.dy.token_stride * sizeof(T);
    float* maps = reinterpret_cast<float*>(staged);
    constexpr int kSlots = kBackSlots<ANY>, kSeg = kBackSegBytes<T, CKPT, ANY>, kIn = kSubBytes<kRow, ANY>;
    uint8_t* own = staged + kMeetingBytes<V, W> + warp * kSlots * kSeg;
    const int qg = staged_pitch<kRow, ANY>(sg), qdy = staged_pitch<kRowBytes, ANY>(sdy);
    auto stage = [&](int k) {
        const int t = (first + k) * kSub, n = min(kSub, a.seqlen - t);
        if (k < run && n > 0) {
            uint8_t* to = own + k % kSlots * kSeg;
            if (n == kSub) [[likely]] {
                stage_rows<kRow, ANY>(to, pg + t * sg, sg, CKPT ? min(kRow, d - c0) : width);
                stage_rows<kRowBytes, ANY>(to + kIn, pdy + t * sdy, sdy, width);
            } else {
                stage_part<kRow, ANY>(to, pg + t * sg, sg, n, CKPT ? min(kRow, d - c0) : width);
                stage_part<kRowBytes, ANY>(to + kIn, pdy + t * sdy, sdy, n, width);
            }
        }
        copy_commit();
    };
    const size_t blk0 = (size_t)b * ta.blocks;
    Map<V> all = identity_map<V>();
    bool closed = false;  // behind the first end nothing reaches the run's first token
    Held held;
#pragma unroll 1
    for (int k = 0; k < kSlots - 1; ++k) stage(k);
    for (int k = 0; k < run; ++k) {
        const int t0 = (first + k) * kSub, n = max(0, min(kSub, a.seqlen - t0));
        Marks m;
        m.valid = (1u << n) - 1;
        m.begin = m.end = 0;
        if constexpr (PACKED) m = marks_of(a.cu, a.nseq, t0, n, held);
        F scale;
        if constexpr (CKPT)
#pragma unroll
            for (int v = 0; v < V; ++v)
                scale.set(v, n > 0 && v < count
                                 ? scale_of(__ldg(a.gate_e + (blk0 + first + k) * d + c + v))
                                 : 0.f);
        copy_wait<kSlots - 2>();
        __syncwarp();
        stage(k + kSlots - 1);
        uint8_t* here = own + k % kSlots * kSeg;
        const uint8_t* rg = here + staged_start<ANY>(pg + t0 * sg) + lane * (kRow / 32);
        const uint8_t* rdy = here + kIn + staged_start<ANY>(pdy + t0 * sdy) + lane * 4;
        auto dy_of = [&](int j) { return Pk::get(row_word<T, ANY>(rdy + j * qdy)); };
        auto token = [&](auto checks, int j, F dy) {
            constexpr bool MARKS = PACKED && decltype(checks)::value;
            extend(all, decay_of<LOGIT>(row_value<T, CKPT, ANY, MARKS>(rg + j * qg, scale)));
            if (!PACKED || !closed) all.B = step(all.A, all.L, dy, all.B);
        };
        if (m.valid == kAll && !m.end) [[likely]] {
#pragma unroll
            for (int j = 0; j < kSub; ++j) token(std::false_type{}, j, dy_of(j));
        } else {
#pragma unroll 1
            for (int j = 0; j < kSub; ++j) {
                if (!(m.valid >> j & 1)) continue;
                F dy = dy_of(j);
                const bool ends = PACKED && (m.end >> j & 1);
                if (ends) {
                    const int s = __shfl_sync(0xffffffffu, m.seq, j);
                    dy = add(dy, load_floats<V>(
                                     a.dfinal_state ? a.dfinal_state + (size_t)s * d + c : nullptr, count));
                }
                token(std::true_type{}, j, dy);
                closed |= ends;
            }
        }
    }
    allow_next_kernel();
    if (closed) all.A = splat<V>(-1.f);
    MapSlots<V>::write(maps, W - 1 - warp, lane, all);
    __syncthreads();
    if (warp == 0)
        MapSlots<V>::write(ta.maps + (size_t)unit * ta.chunks * MapSlots<V>::kFloats, chunk, lane,
                           MapSlots<V>::template join_runs<PACKED, W>(maps, 0, W, lane));
}

template <typename T, bool LOGIT>
cudaError_t dispatch_bwd(const GatedArgs& a, cudaStream_t st) {
    using Y = std::true_type;
    using N = std::false_type;
    TileArgs t = tile_args<T>(a);
    auto go = [&](auto comp, auto packed, auto ckpt, auto any) {
        constexpr bool C = decltype(comp)::value, K = decltype(packed)::value, Q = decltype(ckpt)::value;
        constexpr bool A = decltype(any)::value;
        constexpr int W = kBwdWarps<Q>, V = kChannels<T>;
        const long long units = (long long)t.strips * a.batch;
        const Chunks ch = chunks_of(Q ? Work::kFromCodes : Work::kPlain, units, t.blocks, W, kBwdBlocks<Q>,
                                    sm_count(), t.aligned);
        t.chunks = ch.count;
        t.chunk_tiles = ch.tiles;
        t.maps = static_cast<float*>(a.workspace);
        if (t.chunks > 1) {
            constexpr int kSmem = kMeetingBytes<V, kMapWarps> + kMapWarps * kBackSlots<A> * kBackSegBytes<T, Q, A>;
            const cudaError_t e = launch_ctas<chunk_back_kernel<T, LOGIT, K, Q, A>>(
                units * (t.chunks - 1), kMapWarps, kSmem, false, st, a, t);
            if (e != cudaSuccess) return e;
        }
        constexpr int kSmem = kMeetingBytes<V, W> + kFwdMapBytes<V, W> + W * kBwdSlots * kBwdSegBytes<T, Q, A>;
        return launch_ctas<scan_bwd_kernel<T, LOGIT, C, K, Q, A>>(units * t.chunks, W, kSmem, t.chunks > 1,
                                                                  st, a, t);
    };
    auto rows = [&](auto comp, auto packed, auto ckpt) {
        return t.aligned ? go(comp, packed, ckpt, N{}) : go(comp, packed, ckpt, Y{});
    };
    auto packed = [&](auto comp, auto ckpt) { return a.cu ? rows(comp, Y{}, ckpt) : rows(comp, N{}, ckpt); };
    auto input = [&](auto ckpt) { return a.complement ? packed(Y{}, ckpt) : packed(N{}, ckpt); };
    return a.x_q ? input(Y{}) : input(N{});
}

}  // namespace gated
}  // namespace ssd
