// extern "C" entry points of the gated recurrence and the 8-bit checkpoints: argument checks,
// then one launch on the caller's stream.  Declarations and their documentation live in
// include/ssd_i8.h.
#include <cstddef>
#include <cstdint>

#include "../../include/ssd_i8.h"
#include "gated_kernels.h"

namespace {

// token indices are 32-bit, with room for the tiles behind the last token
constexpr int kMaxSeqlen = 0x7fffffff - 65535;

size_t io_size(int io_dtype) {
    switch (io_dtype) {
        case SSD_IO_F32: return 4;
        case SSD_IO_F16:
        case SSD_IO_BF16: return 2;
        default: return 0;
    }
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// The memory of one argument: `rows` of `width` bytes at batch and token strides (bytes).
struct Region {
    uintptr_t at;
    unsigned long long bs, ts;
    unsigned long long batch, tokens, width;
    bool out;
    unsigned long long extent() const {
        return (batch - 1) * bs + (tokens - 1) * ts + width;
    }
};

using Wide = __int128;  // addresses and strides of any size, their products and differences

Wide floor_div(Wide a, Wide b) { return a / b - (a % b < 0); }  // b > 0

// One dimension of a pair of regions: the stride they have in common and the last index of either.
// False where their strides differ.  (An index that no stride follows counts once.)
struct Dim {
    Wide stride = 1, last_a = 0, last_b = 0;
    bool set(unsigned long long stride_a, unsigned long long count_a, unsigned long long stride_b,
             unsigned long long count_b) {
        if (count_a > 1 && stride_a) last_a = count_a - 1;
        if (count_b > 1 && stride_b) last_b = count_b - 1;
        if (last_a) stride = stride_a;
        else if (last_b) stride = stride_b;
        return !last_a || !last_b || stride_a == stride_b;
    }
};

// Whether two regions share a byte; also said of regions whose extents interleave at different strides.
// A row of b stands delta + i outer + j inner behind a row of a, with i and j from -last_a to last_b; the
// two share a byte where that lies between -b.width and a.width.
bool overlap(const Region& a, const Region& b) {
    if (!a.at || !b.at || !a.batch || !b.batch || !a.tokens || !b.tokens) return false;
    if (a.at + a.extent() <= b.at || b.at + b.extent() <= a.at) return false;
    Dim outer, inner;
    if (!outer.set(a.bs, a.batch, b.bs, b.batch) || !inner.set(a.ts, a.tokens, b.ts, b.tokens)) return true;
    if (outer.stride < inner.stride) {
        const Dim d = outer;
        outer = inner;
        inner = d;
    }
    const Wide delta = (Wide)b.at - (Wide)a.at, wa = a.width, wb = b.width;
    // the integers k with low < k stride < high, between -last_a and last_b
    auto from = [](Wide low, const Dim& d) {
        const Wide k = floor_div(low, d.stride) + 1;
        return k < -d.last_a ? -d.last_a : k;
    };
    auto to = [](Wide high, const Dim& d) {
        const Wide k = -floor_div(-high, d.stride) - 1;
        return k > d.last_b ? d.last_b : k;
    };
    const Wide i0 = from(-wb - inner.last_b * inner.stride - delta, outer);
    const Wide i1 = to(wa + inner.last_a * inner.stride - delta, outer);
    if (i1 - i0 > 7) return true;  // rows wider than their own pitch; two at most of any others
    for (Wide i = i0; i <= i1; ++i) {
        const Wide at = delta + i * outer.stride;
        if (from(-wb - at, inner) <= to(wa - at, inner)) return true;
    }
    return false;
}

// Collects the arguments' memory and refuses an output that shares bytes with another argument.
class Regions {
  public:
    void rows(const ssd::GatedRows& r, int batch, int tokens, int channels, size_t elem, bool out) {
        add(r.ptr, r.batch_stride * elem, r.token_stride * elem, batch, tokens, channels * elem, out);
    }
    void flat(const void* p, size_t bytes, bool out) { add(p, 0, 0, 1, 1, bytes, out); }
    bool clash() const {
        for (int i = 0; i < n_; ++i)
            for (int j = 0; j < i; ++j)
                if ((r_[i].out || r_[j].out) && overlap(r_[i], r_[j])) return true;
        return false;
    }

  private:
    void add(const void* p, unsigned long long bs, unsigned long long ts, unsigned long long batch,
             unsigned long long tokens, unsigned long long width, bool out) {
        if (p && width) r_[n_++] = {reinterpret_cast<uintptr_t>(p), bs, ts, batch, tokens, width, out};
    }
    Region r_[16];
    int n_ = 0;
};

// Strides of readable rows, and of rows that are written (distinct ones).
bool in_rows(const ssd::GatedRows& r, size_t elem) {
    return r.ptr && aligned(r.ptr, elem) && r.batch_stride >= 0 && r.token_stride >= 0;
}

bool out_rows(const ssd::GatedRows& r, int batch, int tokens, int channels, size_t elem) {
    if (!in_rows(r, elem)) return false;
    const bool tok = tokens <= 1 || r.token_stride >= channels;
    const bool bat = batch <= 1 || r.batch_stride >= channels;
    if (!tok || !bat) return false;
    if (tokens <= 1 || batch <= 1) return true;
    // compared by division: the products could pass 64 bits for absurd strides
    return (r.batch_stride - channels) / (tokens - 1) >= r.token_stride ||
           (r.token_stride - channels) / (batch - 1) >= r.batch_stride;
}

bool form_ok(int form) { return (form & ~(SSD_GATE_LOGIT | SSD_INPUT_COMPLEMENT)) == 0; }

// Checks shared by the scan's three entry points, before the pointers of the rows.
ssd_status shape_status(int batch, int seqlen, int channels, const int32_t* cu, int nseq, int form,
                        int io_dtype) {
    if (batch < 0 || seqlen < 0 || channels <= 0 || nseq < 0 || !form_ok(form) || !io_size(io_dtype))
        return SSD_ERR_INVALID_ARG;
    if (cu ? batch != 1 || !aligned(cu, 4) : nseq != 0) return SSD_ERR_INVALID_ARG;
    if (seqlen > kMaxSeqlen || (long long)batch * ((channels + 31LL) / 32) * 64 > 0x7fffffffLL)
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

bool workspace_ok(const void* p, size_t bytes, size_t need) {
    return need == 0 || (p && bytes >= need && aligned(p, 256));
}

// No token at all: the states pass through.
ssd_status pass_states(const float* from, float* to, size_t count, cudaStream_t st) {
    if (!to || !count) return SSD_OK;
    const size_t bytes = count * sizeof(float);
    const cudaError_t e = from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, st)
                               : cudaMemsetAsync(to, 0, bytes, st);
    return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status run_bwd(ssd::GatedArgs& a, size_t elem, size_t workspace_bytes, cudaStream_t st) {
    const size_t seqs = a.cu ? a.nseq : a.batch, d = a.channels;
    if (!aligned(a.init_state, 4) || !aligned(a.span_states, 4) || !aligned(a.dfinal_state, 4) ||
        !aligned(a.dinit_state, 4))
        return SSD_ERR_INVALID_ARG;
    const size_t state_bytes = seqs * d * 4;
    Regions r;
    r.flat(a.dfinal_state, state_bytes, false);
    r.flat(a.dinit_state, state_bytes, true);
    if (a.batch == 0 || (a.cu && a.nseq == 0)) return SSD_OK;
    if (a.seqlen == 0) {
        if (r.clash()) return SSD_ERR_INVALID_ARG;
        return pass_states(a.dfinal_state, a.dinit_state, seqs * d, st);
    }
    if (!a.span_states || !in_rows(a.dy, elem) ||
        !out_rows(a.dx, a.batch, a.seqlen, a.channels, elem) ||
        !out_rows(a.dgate, a.batch, a.seqlen, a.channels, elem))
        return SSD_ERR_INVALID_ARG;
    const size_t n = (size_t)a.batch * a.seqlen * d;
    const size_t spans = ((size_t)a.seqlen + SSD_GATED_SPAN - 1) / SSD_GATED_SPAN;
    if (a.x_q) {
        const size_t ne = (size_t)a.batch * (((size_t)a.seqlen + SSD_CKPT_BLOCK - 1) / SSD_CKPT_BLOCK) * d;
        r.flat(a.x_q, n, false);
        r.flat(a.gate_q, n, false);
        r.flat(a.x_e, ne, false);
        r.flat(a.gate_e, ne, false);
    } else {
        if (!in_rows(a.x, elem) || !in_rows(a.gate, elem)) return SSD_ERR_INVALID_ARG;
        r.rows(a.x, a.batch, a.seqlen, a.channels, elem, false);
        r.rows(a.gate, a.batch, a.seqlen, a.channels, elem, false);
    }
    r.rows(a.dy, a.batch, a.seqlen, a.channels, elem, false);
    r.rows(a.dx, a.batch, a.seqlen, a.channels, elem, true);
    r.rows(a.dgate, a.batch, a.seqlen, a.channels, elem, true);
    r.flat(a.span_states, (size_t)a.batch * spans * d * 4, false);
    r.flat(a.init_state, state_bytes, false);
    if (a.cu) r.flat(a.cu, ((size_t)a.nseq + 1) * 4, false);
    const size_t need = ssd_i8_gated_scan_workspace_size(a.batch, a.seqlen, a.channels, a.io_dtype);
    if (!workspace_ok(a.workspace, workspace_bytes, need)) return SSD_ERR_WORKSPACE;
    r.flat(a.workspace, need, true);
    if (r.clash()) return SSD_ERR_INVALID_ARG;
    return ssd::launch_gated_scan_bwd(a, st) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t ssd_i8_gated_scan_workspace_size(int batch, int seqlen, int channels, int io_dtype) {
    if (batch <= 0 || seqlen <= 0 ||
        shape_status(batch, seqlen, channels, nullptr, 0, 0, io_dtype) != SSD_OK)
        return 0;
    return ssd::gated_workspace_bytes(batch, seqlen, channels, io_dtype);
}

ssd_status ssd_i8_gated_scan(const void* x, long long x_batch_stride, long long x_token_stride,
                             const void* gate, long long gate_batch_stride,
                             long long gate_token_stride, void* y, long long y_batch_stride,
                             long long y_token_stride, int batch, int seqlen, int channels,
                             const int32_t* cu_seqlens, int nseq, int form, int io_dtype,
                             const float* init_state, float* final_state, float* span_states,
                             int8_t* ckpt_x, uint8_t* ckpt_x_exp, int8_t* ckpt_gate,
                             uint8_t* ckpt_gate_exp, void* workspace, size_t workspace_bytes,
                             void* stream) {
    const ssd_status s = shape_status(batch, seqlen, channels, cu_seqlens, nseq, form, io_dtype);
    if (s != SSD_OK) return s;
    const bool ckpt = ckpt_x || ckpt_x_exp || ckpt_gate || ckpt_gate_exp;
    if (ckpt && !(ckpt_x && ckpt_x_exp && ckpt_gate && ckpt_gate_exp) && seqlen > 0)
        return SSD_ERR_INVALID_ARG;
    if (!aligned(init_state, 4) || !aligned(final_state, 4) || !aligned(span_states, 4))
        return SSD_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t elem = io_size(io_dtype), d = channels, seqs = cu_seqlens ? nseq : batch;
    Regions r;
    r.flat(init_state, seqs * d * 4, false);
    r.flat(final_state, seqs * d * 4, true);
    // (without a sequence there still are span states and checkpoint scales, those of no token)
    if (batch == 0 || (cu_seqlens && nseq == 0 && !span_states && !ckpt)) return SSD_OK;
    if (seqlen == 0) {
        if (r.clash()) return SSD_ERR_INVALID_ARG;
        return pass_states(init_state, final_state, seqs * d, st);
    }
    ssd::GatedArgs a{};
    a.x = {x, x_batch_stride, x_token_stride};
    a.gate = {gate, gate_batch_stride, gate_token_stride};
    a.y = {y, y_batch_stride, y_token_stride};
    if (!in_rows(a.x, elem) || !in_rows(a.gate, elem) || !out_rows(a.y, batch, seqlen, channels, elem))
        return SSD_ERR_INVALID_ARG;
    r.rows(a.x, batch, seqlen, channels, elem, false);
    r.rows(a.gate, batch, seqlen, channels, elem, false);
    r.rows(a.y, batch, seqlen, channels, elem, true);
    const size_t n = (size_t)batch * seqlen * d;
    const size_t spans = ((size_t)seqlen + SSD_GATED_SPAN - 1) / SSD_GATED_SPAN;
    const size_t ne = (size_t)batch * (((size_t)seqlen + SSD_CKPT_BLOCK - 1) / SSD_CKPT_BLOCK) * d;
    r.flat(span_states, (size_t)batch * spans * d * 4, true);
    r.flat(ckpt_x, n, true);
    r.flat(ckpt_gate, n, true);
    r.flat(ckpt_x_exp, ne, true);
    r.flat(ckpt_gate_exp, ne, true);
    if (cu_seqlens) r.flat(cu_seqlens, ((size_t)nseq + 1) * 4, false);
    const size_t need = ssd_i8_gated_scan_workspace_size(batch, seqlen, channels, io_dtype);
    if (!workspace_ok(workspace, workspace_bytes, need)) return SSD_ERR_WORKSPACE;
    r.flat(workspace, need, true);
    if (r.clash()) return SSD_ERR_INVALID_ARG;
    a.workspace = workspace;
    a.x_q = ckpt_x;
    a.x_e = ckpt_x_exp;
    a.gate_q = ckpt_gate;
    a.gate_e = ckpt_gate_exp;
    a.cu = cu_seqlens;
    a.nseq = nseq;
    a.batch = batch;
    a.seqlen = seqlen;
    a.channels = channels;
    a.logit = (form & SSD_GATE_LOGIT) != 0;
    a.complement = (form & SSD_INPUT_COMPLEMENT) != 0;
    a.io_dtype = io_dtype;
    a.init_state = init_state;
    a.final_state = final_state;
    a.span_states = span_states;
    return ssd::launch_gated_scan(a, st) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_i8_gated_scan_bwd(const void* dy, long long dy_batch_stride,
                                 long long dy_token_stride, const void* x,
                                 long long x_batch_stride, long long x_token_stride,
                                 const void* gate, long long gate_batch_stride,
                                 long long gate_token_stride, void* dx, long long dx_batch_stride,
                                 long long dx_token_stride, void* dgate,
                                 long long dgate_batch_stride, long long dgate_token_stride,
                                 int batch, int seqlen, int channels, const int32_t* cu_seqlens,
                                 int nseq, int form, int io_dtype, const float* init_state,
                                 const float* span_states, const float* dfinal_state,
                                 float* dinit_state, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    const ssd_status s = shape_status(batch, seqlen, channels, cu_seqlens, nseq, form, io_dtype);
    if (s != SSD_OK) return s;
    ssd::GatedArgs a{};
    a.dy = {dy, dy_batch_stride, dy_token_stride};
    a.x = {x, x_batch_stride, x_token_stride};
    a.gate = {gate, gate_batch_stride, gate_token_stride};
    a.dx = {dx, dx_batch_stride, dx_token_stride};
    a.dgate = {dgate, dgate_batch_stride, dgate_token_stride};
    a.cu = cu_seqlens;
    a.nseq = nseq;
    a.batch = batch;
    a.seqlen = seqlen;
    a.channels = channels;
    a.logit = (form & SSD_GATE_LOGIT) != 0;
    a.complement = (form & SSD_INPUT_COMPLEMENT) != 0;
    a.io_dtype = io_dtype;
    a.init_state = init_state;
    a.span_states = const_cast<float*>(span_states);  // read by the backward kernels
    a.dfinal_state = dfinal_state;
    a.dinit_state = dinit_state;
    a.workspace = workspace;
    return run_bwd(a, io_size(io_dtype), workspace_bytes, static_cast<cudaStream_t>(stream));
}

ssd_status ssd_i8_gated_scan_bwd_ckpt(const void* dy, long long dy_batch_stride,
                                      long long dy_token_stride, const int8_t* ckpt_x,
                                      const uint8_t* ckpt_x_exp, const int8_t* ckpt_gate,
                                      const uint8_t* ckpt_gate_exp, void* dx,
                                      long long dx_batch_stride, long long dx_token_stride,
                                      void* dgate, long long dgate_batch_stride,
                                      long long dgate_token_stride, int batch, int seqlen,
                                      int channels, const int32_t* cu_seqlens, int nseq, int form,
                                      int io_dtype, const float* init_state,
                                      const float* span_states, const float* dfinal_state,
                                      float* dinit_state, void* workspace, size_t workspace_bytes,
                                      void* stream) {
    const ssd_status s = shape_status(batch, seqlen, channels, cu_seqlens, nseq, form, io_dtype);
    if (s != SSD_OK) return s;
    if (batch > 0 && seqlen > 0 && (!ckpt_x || !ckpt_x_exp || !ckpt_gate || !ckpt_gate_exp))
        return SSD_ERR_INVALID_ARG;
    ssd::GatedArgs a{};
    a.dy = {dy, dy_batch_stride, dy_token_stride};
    a.dx = {dx, dx_batch_stride, dx_token_stride};
    a.dgate = {dgate, dgate_batch_stride, dgate_token_stride};
    a.x_q = const_cast<int8_t*>(ckpt_x);  // read by the backward kernels
    a.x_e = const_cast<uint8_t*>(ckpt_x_exp);
    a.gate_q = const_cast<int8_t*>(ckpt_gate);
    a.gate_e = const_cast<uint8_t*>(ckpt_gate_exp);
    a.cu = cu_seqlens;
    a.nseq = nseq;
    a.batch = batch;
    a.seqlen = seqlen;
    a.channels = channels;
    a.logit = (form & SSD_GATE_LOGIT) != 0;
    a.complement = (form & SSD_INPUT_COMPLEMENT) != 0;
    a.io_dtype = io_dtype;
    a.init_state = init_state;
    a.span_states = const_cast<float*>(span_states);
    a.dfinal_state = dfinal_state;
    a.dinit_state = dinit_state;
    a.workspace = workspace;
    return run_bwd(a, io_size(io_dtype), workspace_bytes, static_cast<cudaStream_t>(stream));
}

ssd_status ssd_i8_gated_step(float* state, const void* x, const void* gate, void* y, int batch,
                             int channels, int form, int io_dtype, void* stream) {
    const size_t elem = io_size(io_dtype);
    if (batch < 0 || channels <= 0 || !form_ok(form) || !elem) return SSD_ERR_INVALID_ARG;
    const long long count = (long long)batch * channels;
    if (count > 0x7fffffffLL * 128) return SSD_ERR_UNSUPPORTED;
    if (batch == 0) return SSD_OK;
    if (!state || !x || !gate || !y || !aligned(state, 4) || !aligned(x, elem) ||
        !aligned(gate, elem) || !aligned(y, elem))
        return SSD_ERR_INVALID_ARG;
    Regions r;
    r.flat(state, count * 4, true);
    r.flat(x, count * elem, false);
    r.flat(gate, count * elem, false);
    r.flat(y, count * elem, true);
    if (r.clash()) return SSD_ERR_INVALID_ARG;
    const ssd::GatedStepArgs a{state, x, gate, y, count, (form & SSD_GATE_LOGIT) != 0,
                               (form & SSD_INPUT_COMPLEMENT) != 0, io_dtype};
    return ssd::launch_gated_step(a, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SSD_OK
               : SSD_ERR_CUDA;
}

ssd_status ssd_i8_ckpt_pack(const void* x, long long x_batch_stride, long long x_token_stride,
                            int batch, int seqlen, int channels, int io_dtype, int8_t* q,
                            uint8_t* e, void* stream) {
    const ssd_status s = shape_status(batch, seqlen, channels, nullptr, 0, 0, io_dtype);
    if (s != SSD_OK) return s;
    if (batch == 0 || seqlen == 0) return SSD_OK;
    const size_t elem = io_size(io_dtype), d = channels;
    const ssd::GatedRows rows{x, x_batch_stride, x_token_stride};
    if (!in_rows(rows, elem) || !q || !e) return SSD_ERR_INVALID_ARG;
    Regions r;
    r.rows(rows, batch, seqlen, channels, elem, false);
    r.flat(q, (size_t)batch * seqlen * d, true);
    r.flat(e, (size_t)batch * (((size_t)seqlen + SSD_CKPT_BLOCK - 1) / SSD_CKPT_BLOCK) * d, true);
    if (r.clash()) return SSD_ERR_INVALID_ARG;
    return ssd::launch_ckpt_pack(rows, batch, seqlen, channels, io_dtype, q, e,
                                 static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SSD_OK
               : SSD_ERR_CUDA;
}

ssd_status ssd_i8_ckpt_unpack(const int8_t* q, const uint8_t* e, int batch, int seqlen,
                              int channels, int io_dtype, void* x, void* stream) {
    const ssd_status s = shape_status(batch, seqlen, channels, nullptr, 0, 0, io_dtype);
    if (s != SSD_OK) return s;
    if (batch == 0 || seqlen == 0) return SSD_OK;
    const size_t elem = io_size(io_dtype), d = channels, n = (size_t)batch * seqlen * d;
    if (!q || !e || !x || !aligned(x, elem)) return SSD_ERR_INVALID_ARG;
    Regions r;
    r.flat(q, n, false);
    r.flat(e, (size_t)batch * (((size_t)seqlen + SSD_CKPT_BLOCK - 1) / SSD_CKPT_BLOCK) * d, false);
    r.flat(x, n * elem, true);
    if (r.clash()) return SSD_ERR_INVALID_ARG;
    return ssd::launch_ckpt_unpack(q, e, batch, seqlen, channels, io_dtype, x,
                                   static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? SSD_OK
               : SSD_ERR_CUDA;
}

}  // extern "C"
