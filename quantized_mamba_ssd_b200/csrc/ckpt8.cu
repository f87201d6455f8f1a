// 8-bit activation checkpoints: blocks of 16 tokens of one channel as int8 codes with one
// power-of-two scale, and back.
//
// Pure streaming.  A thread takes the 16 tokens of a few neighbouring channels, so that a block
// never leaves it: 16 independent loads in flight, the largest magnitude and the codes in
// registers, 16 stores.  As many channels as make 8 bytes of a row, or two 16-bit ones, where the
// rows' starts and the codes' allow words of them.
//
// What bounds it (one B200, of the measured copy bandwidth 6.47 TB/s): HBM where the words are whole -
// 4 x 4096 x 4096 bf16 34 us to pack, 95 %, and 36 us to unpack, 89 %; fp32 52 and 55 us, 102 and 95 %.
// 4090 bf16 channels, in pairs, take 38 and 47 us, 4095 52 and 59 (one channel a thread packs either
// in 76): stores across the 128-byte lines.
#include "gated_tile.cuh"

namespace ssd {

namespace {

using namespace gated;

constexpr int kThreads = 128;

template <int N> struct Word;
template <> struct Word<1> { using U = uint8_t; };
template <> struct Word<2> { using U = uint16_t; };
template <> struct Word<4> { using U = uint32_t; };
template <> struct Word<8> { using U = uint2; };

// N values of type T as one load or store
template <typename T, int N> union Values {
    typename Word<N * sizeof(T)>::U word;
    T v[N];
    __device__ Values() {}
};

// Two neighbouring 16-bit channels of a block: w(j) holds those of token j.
template <typename T> struct Pair {
    using H2 = decltype(both<T>(0.f, 0.f));
    uint32_t e0, e1;
    H2 most;
    Vec<2> inv;
    static __device__ __forceinline__ H2 as(uint32_t w) { return *reinterpret_cast<const H2*>(&w); }
    template <typename F> __device__ __forceinline__ explicit Pair(F w) {
        H2 top = both<T>(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kBlock; ++j) top = __hmax2_nan(top, __habs2(as(w(j))));
        block_scales<T>(top, e0, e1, most, inv);
    }
    __device__ __forceinline__ uint32_t codes(uint32_t w) const { return block_codes<T>(as(w), most, inv); }
};

// N channels a thread.  SPLIT: two 16-bit channels in accesses of one (their arithmetic stays
// two-wide), the last of which may not exist.
template <typename T, int N, bool SPLIT = false>
__global__ void __launch_bounds__(kThreads)
pack_kernel(GatedRows x, int batch, int seqlen, int d, int8_t* __restrict__ q,
            uint8_t* __restrict__ e) {
    const int groups = (d + N - 1) / N, chunks = (groups + kThreads - 1) / kThreads;
    const int blocks = (seqlen + kBlock - 1) / kBlock;
    const long long work = (long long)batch * blocks * chunks;
    for (long long w = blockIdx.x; w < work; w += gridDim.x) {
        const long long row = w / chunks;  // one block of one batch row
        const int g = static_cast<int>(w % chunks) * kThreads + threadIdx.x;
        if (g >= groups) continue;
        const int b = static_cast<int>(row / blocks), t0 = static_cast<int>(row % blocks) * kBlock;
        const int n = min(kBlock, seqlen - t0), c = g * N;
        const bool both_exist = !SPLIT || c + 1 < d;
        const T* src = static_cast<const T*>(x.ptr) + b * x.batch_stride + t0 * x.token_stride + c;
        Values<T, N> in[kBlock];
#pragma unroll
        for (int j = 0; j < kBlock; ++j) {
            const T* p = src + j * x.token_stride;
            if constexpr (SPLIT) {
#pragma unroll
                for (int i = 0; i < 2; ++i) in[j].v[i] = j < n && (!i || both_exist) ? p[i] : static_cast<T>(0.f);
            } else if (j < n) {
                in[j].word = *reinterpret_cast<const decltype(in[j].word)*>(p);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) in[j].v[i] = static_cast<T>(0.f);
            }
        }
        Values<uint8_t, N> ex;
        int8_t* dst = q + ((size_t)b * seqlen + t0) * d + c;
        uint8_t* ex_to = e + (size_t)row * d + c;
        if constexpr (sizeof(T) == 2 && N == 4) {  // pairs stay pairs
            const Pair<T> lo([&](int j) { return in[j].word.x; }), hi([&](int j) { return in[j].word.y; });
            ex.v[0] = lo.e0;
            ex.v[1] = lo.e1;
            ex.v[2] = hi.e0;
            ex.v[3] = hi.e1;
#pragma unroll
            for (int j = 0; j < kBlock; ++j) {
                if (j >= n) break;
                *reinterpret_cast<uint32_t*>(dst + (size_t)j * d) =
                    __byte_perm(lo.codes(in[j].word.x), hi.codes(in[j].word.y), 0x5410);
            }
        } else if constexpr (sizeof(T) == 2 && N == 2) {
            const Pair<T> pair([&](int j) { return in[j].word; });
            ex.v[0] = pair.e0;
            ex.v[1] = pair.e1;
#pragma unroll
            for (int j = 0; j < kBlock; ++j) {
                if (j >= n) break;
                const uint32_t codes = pair.codes(in[j].word);
                int8_t* to = dst + (size_t)j * d;
                if constexpr (SPLIT) {
                    to[0] = static_cast<int8_t>(codes);
                    if (both_exist) to[1] = static_cast<int8_t>(codes >> 8);
                } else {
                    *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(codes);
                }
            }
        } else {
            Values<int8_t, N> out[kBlock];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                uint32_t top = 0;  // bits of the magnitudes: their order, NaN on top
#pragma unroll
                for (int j = 0; j < kBlock; ++j)
                    top = max(top, __float_as_uint(fabsf(static_cast<float>(in[j].v[i]))));
                const uint32_t s = scale_exp(top);
                ex.v[i] = static_cast<uint8_t>(s);
                const Coder coder(s);
#pragma unroll
                for (int j = 0; j < kBlock; ++j)
                    out[j].v[i] = static_cast<int8_t>(coder.code(static_cast<float>(in[j].v[i])));
            }
#pragma unroll
            for (int j = 0; j < kBlock; ++j) {
                if (j >= n) break;
                *reinterpret_cast<decltype(out[j].word)*>(dst + (size_t)j * d) = out[j].word;
            }
        }
        if constexpr (SPLIT) {
            ex_to[0] = ex.v[0];
            if (both_exist) ex_to[1] = ex.v[1];
        } else {
            *reinterpret_cast<decltype(ex.word)*>(ex_to) = ex.word;
        }
    }
}

template <typename T, int N>
__global__ void __launch_bounds__(kThreads)
unpack_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ e, int batch, int seqlen,
              int d, T* __restrict__ x) {
    const int groups = d / N, chunks = (groups + kThreads - 1) / kThreads;
    const int blocks = (seqlen + kBlock - 1) / kBlock;
    const long long work = (long long)batch * blocks * chunks;
    for (long long w = blockIdx.x; w < work; w += gridDim.x) {
        const long long row = w / chunks;
        const int g = static_cast<int>(w % chunks) * kThreads + threadIdx.x;
        if (g >= groups) continue;
        const int b = static_cast<int>(row / blocks), t0 = static_cast<int>(row % blocks) * kBlock;
        const int n = min(kBlock, seqlen - t0), c = g * N;
        const size_t at = ((size_t)b * seqlen + t0) * d + c;
        Values<int8_t, N> in[kBlock];
        Values<uint8_t, N> ex;
        ex.word = *reinterpret_cast<const decltype(ex.word)*>(e + (size_t)row * d + c);
#pragma unroll
        for (int j = 0; j < kBlock; ++j)
            if (j < n) in[j].word = *reinterpret_cast<const decltype(in[j].word)*>(q + at + (size_t)j * d);
        float scale[N];
#pragma unroll
        for (int i = 0; i < N; ++i) scale[i] = scale_of(ex.v[i]);
        // Whether a code is kCodeNaN (rare: see mark_rows) is asked of words of codes, w: a zero byte of it.
        // w - 0x01010101 borrows at the lowest zero byte, and only there is a byte's top bit set in that and
        // not in w.  Single codes are asked one by one as they leave (4095 bf16 channels 59 us; all of them
        // before the first store 68, without the question 55).
        uint32_t zeros = 0;
        if constexpr (N > 1) {
#pragma unroll
            for (int j = 0; j < kBlock; ++j) {
                if (j >= n) break;
                const uint32_t w = (N == 2 ? in[j].word | 0xffff0000u : in[j].word) ^ 0x01010101u * kCodeNaN;
                zeros |= (w - 0x01010101u) & ~w;
            }
        }
        auto store = [&](auto marks) {
#pragma unroll
            for (int j = 0; j < kBlock; ++j) {
                if (j >= n) break;
                Values<T, N> out;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float v = scale[i] * in[j].v[i];
                    if (decltype(marks)::value && static_cast<uint8_t>(in[j].v[i]) == kCodeNaN) v = NAN;
                    out.v[i] = static_cast<T>(v);
                }
                *reinterpret_cast<decltype(out.word)*>(x + at + (size_t)j * d) = out.word;
            }
        };
        if (N > 1 && !(zeros & 0x80808080u)) [[likely]] store(std::false_type{});
        else store(std::true_type{});
    }
}

unsigned grid_of(int batch, int seqlen, int groups) {
    const long long blocks = (seqlen + kBlock - 1) / kBlock;
    const long long work = batch * blocks * ((groups + kThreads - 1) / kThreads);
    return static_cast<unsigned>(work < (1 << 30) ? work : 1 << 30);
}

bool multiple(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <typename T>
cudaError_t pack_as(const GatedRows& x, int batch, int seqlen, int d, int8_t* q, uint8_t* e,
                    cudaStream_t st) {
    auto words = [&](int n) {  // of n channels
        return d % n == 0 && multiple(x.ptr, n * sizeof(T)) && x.batch_stride % n == 0 &&
               x.token_stride % n == 0 && multiple(q, n) && multiple(e, n);
    };
    auto go = [&](auto kernel, int n) {
        kernel<<<grid_of(batch, seqlen, (d + n - 1) / n), kThreads, 0, st>>>(x, batch, seqlen, d, q, e);
    };
    constexpr int N = 8 / sizeof(T);
    if (words(N)) go(pack_kernel<T, N>, N);
    else if constexpr (sizeof(T) == 2) {
        if (words(2)) go(pack_kernel<T, 2>, 2);
        else go(pack_kernel<T, 2, true>, 2);
    } else {
        go(pack_kernel<T, 1>, 1);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t unpack_as(const int8_t* q, const uint8_t* e, int batch, int seqlen, int d, void* x,
                      cudaStream_t st) {
    auto words = [&](int n) {
        return d % n == 0 && multiple(x, n * sizeof(T)) && multiple(q, n) && multiple(e, n);
    };
    auto go = [&](auto kernel, int n) {
        kernel<<<grid_of(batch, seqlen, d / n), kThreads, 0, st>>>(q, e, batch, seqlen, d, static_cast<T*>(x));
    };
    constexpr int N = 8 / sizeof(T);
    if (words(N)) go(unpack_kernel<T, N>, N);
    else if (sizeof(T) == 2 && words(2)) go(unpack_kernel<T, 2>, 2);
    else go(unpack_kernel<T, 1>, 1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ckpt_pack(const GatedRows& x, int batch, int seqlen, int d, int io_dtype,
                             int8_t* q, uint8_t* e, cudaStream_t st) {
    switch (io_dtype) {
        case SSD_IO_F32: return pack_as<float>(x, batch, seqlen, d, q, e, st);
        case SSD_IO_F16: return pack_as<__half>(x, batch, seqlen, d, q, e, st);
        case SSD_IO_BF16: return pack_as<__nv_bfloat16>(x, batch, seqlen, d, q, e, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_ckpt_unpack(const int8_t* q, const uint8_t* e, int batch, int seqlen, int d,
                               int io_dtype, void* x, cudaStream_t st) {
    switch (io_dtype) {
        case SSD_IO_F32: return unpack_as<float>(q, e, batch, seqlen, d, x, st);
        case SSD_IO_F16: return unpack_as<__half>(q, e, batch, seqlen, d, x, st);
        case SSD_IO_BF16: return unpack_as<__nv_bfloat16>(q, e, batch, seqlen, d, x, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace ssd
