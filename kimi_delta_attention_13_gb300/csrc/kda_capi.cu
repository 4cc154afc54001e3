// kda_capi.cu -- the C ABI of libkda_gb300: host-side argument validation and kernel dispatch.
// Declarations, argument meaning, layouts and error behaviour: include/kda.h.
#include <cmath>
#include <cstdio>
#include <initializer_list>

#include <nvtx3/nvToolsExt.h>

#include "kda_internal.cuh"

using namespace kda;

namespace {

// An NVTX range over one C-ABI call, so that profiler captures can be scoped to a call.  Without
// a tool attached the push and pop do nothing.
struct CallRange {
    explicit CallRange(const char *name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange &) = delete;
    CallRange &operator=(const CallRange &) = delete;
};

bool bad_dtype(int32_t dtype) { return dtype != KDA_BF16 && dtype != KDA_F32; }

// Validation shared by both prefill entry points.  Returns KDA_OK when the call may launch.
int check_prefill(const void *q, const void *k, const void *v, const void *g, const void *beta,
                  const int32_t *cu_seqlens, int32_t n_seqs, int64_t total_tokens, int32_t n_heads,
                  int32_t d_k, int32_t d_v, int32_t dtype, int32_t out_dtype,
                  const float *init_state, const void *out, const float *final_state,
                  int32_t ckpt_stride, const float *ckpts)
{
    if (n_seqs < 0 || total_tokens < 0 || n_heads < 1 || d_k < 1 || d_v < 1 || bad_dtype(dtype) ||
        bad_dtype(out_dtype))
        return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!q || !k || !v || !g || !beta || !out)) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && n_seqs == 0) return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens && n_seqs > 1) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;  // cu_seqlens are int32
    // a checkpoint falls on a boundary of the tensor-core kernel's 32-token steps
    if (ckpt_stride < 0 || ckpt_stride % 32 != 0) return KDA_ERR_INVALID_ARG;
    if (ckpt_stride > 0 && !ckpts) return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, g, beta, init_state, out, final_state, ckpts};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return KDA_ERR_MISALIGNED;
    const int esz = dtype == KDA_BF16 ? 2 : 4, osz = out_dtype == KDA_BF16 ? 2 : 4;
    // every row of q/k/g/v/out must start 16-byte aligned for the vector and TMA paths
    if (((int64_t)d_k * esz) % 16 != 0 || ((int64_t)d_v * esz) % 16 != 0 ||
        ((int64_t)d_v * osz) % 16 != 0)
        return KDA_ERR_UNSUPPORTED_SHAPE;
    if (out && (out == q || out == k || out == v || out == g || out == beta))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// Validation shared by the two staged entry points (everything but the scratch).
int check_staged(const void *h_q, const void *h_k, const void *h_v, const void *h_g, const void *h_beta,
                 const int32_t *h_cu_seqlens, int32_t n_seqs, int64_t total_tokens, int32_t n_heads,
                 int32_t dtype, int32_t out_dtype, const float *init_state, void *d_q, void *d_k,
                 void *d_v, void *d_g, void *d_beta, void *d_out, void *h_out, float *final_state,
                 int64_t chunk_tokens)
{
    if (n_seqs < 0 || total_tokens < 0 || n_heads < 1 || chunk_tokens < 1 || bad_dtype(dtype) ||
        bad_dtype(out_dtype) || total_tokens > 0x7fffffffLL)
        return KDA_ERR_INVALID_ARG;
    if ((total_tokens > 0 && n_seqs == 0) || (n_seqs > 0 && !final_state) || (n_seqs > 1 && !h_cu_seqlens))
        return KDA_ERR_INVALID_ARG;
    const void *host_in[] = {h_q, h_k, h_v, h_g, h_beta, h_out};
    const void *dev_buf[] = {d_q, d_k, d_v, d_g, d_beta, d_out};
    for (int i = 0; i < 6; ++i)
        if (total_tokens > 0 && (!host_in[i] || !dev_buf[i])) return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {h_q, h_k, h_v, h_g, h_beta, h_out, d_q, d_k, d_v, d_g, d_beta, d_out,
                          init_state, final_state};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    // every chunk after the first starts at a multiple of chunk_tokens (or of 32 in the cut-up
    // last chunk), and its beta rows must start 16-byte aligned like every pointer of a prefill
    const int64_t esz = dtype == KDA_BF16 ? 2 : 4;
    if (total_tokens > chunk_tokens && (chunk_tokens * n_heads * esz) % 16 != 0) return KDA_ERR_INVALID_ARG;
    if (n_seqs > 1) {   // the host table is checked in full here
        if (h_cu_seqlens[0] != 0 || h_cu_seqlens[n_seqs] != total_tokens) return KDA_ERR_INVALID_ARG;
        for (int n = 0; n < n_seqs; ++n)
            if (h_cu_seqlens[n + 1] < h_cu_seqlens[n]) return KDA_ERR_INVALID_ARG;
    }
    return KDA_OK;
}

bool tc_supported(int32_t d_k, int32_t d_v, int32_t dtype)
{
    return dtype == KDA_BF16 && d_k == 128 && d_v == 128;
}

// Head sizes of the linear-attention calls: rows are whole 16-byte units in every type.
bool bad_linear_dims(int32_t d_k, int32_t d_v)
{
    return d_k < 8 || d_k > 256 || d_k % 8 != 0 || d_v < 8 || d_v > 256 || d_v % 8 != 0;
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether an output's address is one of those it must not share.
bool aliases(const void *out, std::initializer_list<const void *> others)
{
    if (out)
        for (const void *p : others)
            if (out == p) return true;
    return false;
}

// Whether two ranges of memory meet.
bool meet(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && a_bytes > 0 && b_bytes > 0 && x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

int64_t bytes_of(int32_t dtype) { return dtype == KDA_BF16 ? 2 : 4; }

// Whether what a kda_delta call writes meets the operands of its `rows` tokens.
bool delta_overlap(const void *to, int64_t bytes, const void *q, const void *k, const void *v, const float *g,
                   int32_t g_per_token, const float *beta, int64_t rows, int32_t n_heads, int32_t n_key_heads,
                   int32_t d_k, int32_t d_v, int32_t dtype)
{
    const int64_t keys = rows * n_key_heads * d_k * bytes_of(dtype);
    return meet(to, bytes, q, keys) || meet(to, bytes, k, keys) || meet(to, bytes, v, rows * n_heads * d_v * bytes_of(dtype)) ||
           meet(to, bytes, g, (g_per_token ? rows : 1) * n_heads * 4) || meet(to, bytes, beta, rows * n_heads * 4);
}

// Validation shared by kda_state_pack and kda_state_unpack: the pool (`held`, `scales`) and the states.
int check_pack(const void *held, const float *scales, int32_t format, const int64_t *held_idx, int64_t n_held,
               const float *full, const int64_t *full_idx, int64_t n_full, int64_t n, int32_t n_heads, int32_t d_k,
               int32_t d_v)
{
    if (n < 0 || n_held < 0 || n_full < 0 || n_heads < 1 || d_k < 1 || d_v < 1 ||
        (format != KDA_STATE_BF16 && format != KDA_STATE_INT8))
        return KDA_ERR_INVALID_ARG;
    if (d_k > 256 || d_v > 256 || d_v % 4 != 0) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (n > 0 && (!held || !full)) return KDA_ERR_INVALID_ARG;
    if (format == KDA_STATE_INT8 ? n > 0 && !scales : scales != nullptr) return KDA_ERR_INVALID_ARG;
    if ((!held_idx && n > n_held) || (!full_idx && n > n_full)) return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {held, scales, held_idx, full, full_idx};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    const int64_t rows = (int64_t)n_heads * d_k, held_bytes = n_held * rows * d_v * (format == KDA_STATE_INT8 ? 1 : 2);
    const int64_t full_bytes = n_full * rows * d_v * 4, scale_bytes = n_held * rows * 4;
    if (meet(held, held_bytes, full, full_bytes) || meet(scales, scale_bytes, full, full_bytes) ||
        meet(scales, scale_bytes, held, held_bytes))
        return KDA_ERR_INVALID_ARG;
    for (const int64_t *idx : {held_idx, full_idx})
        if (meet(idx, 8 * n, held, held_bytes) || meet(idx, 8 * n, full, full_bytes) || meet(idx, 8 * n, scales, scale_bytes))
            return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace

extern "C" {

int kda_abi_version(void) { return KDA_ABI_VERSION; }

const char *kda_status_string(int status)
{
    switch (status) {
    case KDA_OK: return "KDA_OK";
    case KDA_ERR_INVALID_ARG: return "KDA_ERR_INVALID_ARG: invalid argument";
    case KDA_ERR_UNSUPPORTED_SHAPE: return "KDA_ERR_UNSUPPORTED_SHAPE: head sizes not implemented";
    case KDA_ERR_MISALIGNED: return "KDA_ERR_MISALIGNED: pointer not 16-byte aligned";
    case KDA_ERR_CUDA: return "KDA_ERR_CUDA: CUDA runtime call or launch failed";
    case KDA_ERR_DEVICE_TIMEOUT: return "KDA_ERR_DEVICE_TIMEOUT: bounded device wait expired";
    case KDA_ERR_INDEX_RANGE: return "KDA_ERR_INDEX_RANGE: state index out of range";
    case KDA_ERR_DEVICE_BOUNDS: return "KDA_ERR_DEVICE_BOUNDS: device-side bounds check failed";
    default: return "KDA_ERR_UNKNOWN";
    }
}

int kda_prefill_path(int32_t d_k, int32_t d_v, int32_t dtype)
{
    if (d_k < 1 || d_v < 1 || bad_dtype(dtype)) return -KDA_ERR_INVALID_ARG;
    if (tc_supported(d_k, d_v, dtype)) return 1;
    if (d_k <= 128 && d_v % 32 == 0 && d_v <= 256) return 0;
    return -KDA_ERR_UNSUPPORTED_SHAPE;
}

int kda_prefill(const void *q, const void *k, const void *v, const void *g, const void *beta,
                const int32_t *cu_seqlens, int32_t n_seqs, int64_t total_tokens, int32_t n_heads,
                int32_t d_k, int32_t d_v, int32_t dtype, int32_t out_dtype, const float *init_state,
                void *out, float *final_state, int32_t ckpt_stride, float *ckpts, void *stream)
{
    const CallRange range("kda_prefill");
    int rc = check_prefill(q, k, v, g, beta, cu_seqlens, n_seqs, total_tokens, n_heads, d_k, d_v,
                           dtype, out_dtype, init_state, out, final_state, ckpt_stride, ckpts);
    if (rc != KDA_OK) return rc;
    if (tc_supported(d_k, d_v, dtype) && total_tokens > 0)
        return launch_prefill_tc(q, k, v, g, beta, cu_seqlens, n_seqs, total_tokens, n_heads,
                                 out_dtype, init_state, out, final_state, ckpt_stride, ckpts,
                                 (cudaStream_t)stream);
    return launch_prefill_recurrent(q, k, v, g, beta, cu_seqlens, n_seqs, total_tokens, n_heads,
                                    d_k, d_v, dtype, out_dtype, init_state, out, final_state,
                                    ckpt_stride, ckpts, (cudaStream_t)stream);
}

int kda_prefill_precise(const void *q, const void *k, const void *v, const void *g,
                        const void *beta, const int32_t *cu_seqlens, int32_t n_seqs,
                        int64_t total_tokens, int32_t n_heads, int32_t d_k, int32_t d_v,
                        int32_t dtype, int32_t out_dtype, const float *init_state, void *out,
                        float *final_state, int32_t ckpt_stride, float *ckpts, void *stream)
{
    const CallRange range("kda_prefill_precise");
    int rc = check_prefill(q, k, v, g, beta, cu_seqlens, n_seqs, total_tokens, n_heads, d_k, d_v,
                           dtype, out_dtype, init_state, out, final_state, ckpt_stride, ckpts);
    if (rc != KDA_OK) return rc;
    if (tc_supported(d_k, d_v, dtype) && total_tokens > 0)
        return launch_prefill_tc_precise(q, k, v, g, beta, cu_seqlens, n_seqs, total_tokens,
                                         n_heads, out_dtype, init_state, out, final_state,
                                         ckpt_stride, ckpts, (cudaStream_t)stream);
    return launch_prefill_recurrent(q, k, v, g, beta, cu_seqlens, n_seqs, total_tokens, n_heads,
                                    d_k, d_v, dtype, out_dtype, init_state, out, final_state,
                                    ckpt_stride, ckpts, (cudaStream_t)stream);
}

int kda_prefill_recurrent(const void *q, const void *k, const void *v, const void *g,
                          const void *beta, const int32_t *cu_seqlens, int32_t n_seqs,
                          int64_t total_tokens, int32_t n_heads, int32_t d_k, int32_t d_v,
                          int32_t dtype, int32_t out_dtype, const float *init_state, void *out,
                          float *final_state, int32_t ckpt_stride, float *ckpts, void *stream)
{
    const CallRange range("kda_prefill_recurrent");
    int rc = check_prefill(q, k, v, g, beta, cu_seqlens, n_seqs, total_tokens, n_heads, d_k, d_v,
                           dtype, out_dtype, init_state, out, final_state, ckpt_stride, ckpts);
    if (rc != KDA_OK) return rc;
    return launch_prefill_recurrent(q, k, v, g, beta, cu_seqlens, n_seqs, total_tokens, n_heads,
                                    d_k, d_v, dtype, out_dtype, init_state, out, final_state,
                                    ckpt_stride, ckpts, (cudaStream_t)stream);
}

int kda_decode(const void *q, const void *k, const void *v, const void *g, const void *beta,
               float *state, void *out, int32_t n_seqs, int32_t n_heads, int32_t d_k, int32_t d_v,
               int32_t dtype, int32_t out_dtype, void *stream)
{
    const CallRange range("kda_decode");
    if (n_seqs < 0 || n_heads < 1 || d_k < 1 || d_v < 1 || bad_dtype(dtype) || bad_dtype(out_dtype))
        return KDA_ERR_INVALID_ARG;
    if (n_seqs > 0 && (!q || !k || !v || !g || !beta || !state || !out)) return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, g, beta, state, out};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    if (out && (out == q || out == k || out == v || out == g || out == beta || out == state))
        return KDA_ERR_INVALID_ARG;
    return launch_decode(q, k, v, g, beta, state, out, n_seqs, n_heads, d_k, d_v, dtype, out_dtype,
                         (cudaStream_t)stream);
}

int kda_state_copy(float *dst, const int64_t *dst_idx, int64_t n_dst_slots, const float *src,
                   const int64_t *src_idx, int64_t n_src_slots, int64_t n, int32_t n_heads,
                   int32_t d_k, int32_t d_v, void *stream)
{
    const CallRange range("kda_state_copy");
    if (n < 0 || n_dst_slots < 0 || n_src_slots < 0 || n_heads < 1 || d_k < 1 || d_v < 1)
        return KDA_ERR_INVALID_ARG;
    if (n > 0 && (!dst || !src)) return KDA_ERR_INVALID_ARG;
    if ((!dst_idx && n > n_dst_slots) || (!src_idx && n > n_src_slots)) return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {dst, dst_idx, src, src_idx};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    const int64_t unit = (int64_t)n_heads * d_k * d_v;
    return launch_state_copy(dst, dst_idx, n_dst_slots, src, src_idx, n_src_slots, n, unit,
                             (cudaStream_t)stream);
}

int kda_premix(const void *xq, const void *xk, const void *xv, const void *a, const void *b,
               const float *w, const void *hist, const int32_t *cu_seqlens, int32_t n_seqs,
               int64_t total_tokens, int32_t n_heads, int32_t d, float eps, int32_t dtype, void *q,
               void *k, void *v, void *g, void *beta, void *stream)
{
    const CallRange range("kda_premix");
    if (n_seqs < 0 || total_tokens < 0 || n_heads < 1 || d < 1 || bad_dtype(dtype) || !(eps > 0.f))
        return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && n_seqs == 0) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;   // cu_seqlens are int32
    if (!cu_seqlens && n_seqs > 1) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!xq || !xk || !xv || !a || !b || !w || !q || !k || !v || !g || !beta))
        return KDA_ERR_INVALID_ARG;
    if (d > 256 || (d & (d - 1)) != 0 || d < 8) return KDA_ERR_UNSUPPORTED_SHAPE;
    const void *ptrs[] = {xq, xk, xv, a, b, w, hist, q, k, v, g, beta};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return KDA_ERR_MISALIGNED;
    const void *ins[] = {xq, xk, xv, a, b, hist};
    const void *outs[] = {q, k, v, g, beta};
    for (const void *o : outs)
        for (const void *i : ins)
            if (o && o == i) return KDA_ERR_INVALID_ARG;
    return launch_premix(xq, xk, xv, a, b, w, hist, cu_seqlens, n_seqs, total_tokens, n_heads, d,
                         eps, dtype, q, k, v, g, beta, (cudaStream_t)stream);
}

int kda_output_gate(const void *o, int32_t o_dtype, const void *z, int32_t z_dtype, void *out,
                    int32_t out_dtype, int64_t n, void *stream)
{
    const CallRange range("kda_output_gate");
    if (n < 0 || bad_dtype(o_dtype) || bad_dtype(z_dtype) || bad_dtype(out_dtype))
        return KDA_ERR_INVALID_ARG;
    if (n > 0 && (!o || !z || !out)) return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {o, z, out};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    // in place over o is fine (same element type: each element is read before it is written)
    if (out && ((out == o && out_dtype != o_dtype) || out == z)) return KDA_ERR_INVALID_ARG;
    return launch_output_gate(o, o_dtype, z, z_dtype, out, out_dtype, n, (cudaStream_t)stream);
}

int kda_cp_combine(const float *s_loc, const float *m, const int32_t *seq_seg, int32_t n_seqs,
                   int32_t n_heads, int32_t d, float *s_start, float *final_state, void *stream)
{
    const CallRange range("kda_cp_combine");
    if (n_seqs < 0 || n_heads < 1 || d < 1) return KDA_ERR_INVALID_ARG;
    if (d != 128) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (n_seqs > 0 && (!s_loc || !m || !seq_seg || !s_start)) return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {s_loc, m, s_start, final_state};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(seq_seg) & 3u) != 0) return KDA_ERR_MISALIGNED;
    if (s_start && (s_start == s_loc || s_start == m)) return KDA_ERR_INVALID_ARG;
    if (final_state && (final_state == s_loc || final_state == m || final_state == s_start))
        return KDA_ERR_INVALID_ARG;
    return launch_cp_combine(s_loc, m, seq_seg, n_seqs, n_heads, s_start, final_state,
                             (cudaStream_t)stream);
}

int kda_cp_correct(const float *u, const float *s_start, const int32_t *cu_seg, int32_t n_seg,
                   const int32_t *skip_seg, int32_t n_skip, int64_t total_tokens, int32_t n_heads,
                   int32_t d, float *out, void *stream)
{
    const CallRange range("kda_cp_correct");
    if (n_seg < 0 || n_skip < 0 || total_tokens < 0 || n_heads < 1 || d < 1) return KDA_ERR_INVALID_ARG;
    if (d != 128) return KDA_ERR_UNSUPPORTED_SHAPE;
    if (n_seg > 0 && (!u || !s_start || !cu_seg || !out || (n_skip > 0 && !skip_seg)))
        return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {u, s_start, out};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(cu_seg) & 3u) != 0 || (reinterpret_cast<uintptr_t>(skip_seg) & 3u) != 0)
        return KDA_ERR_MISALIGNED;
    if (out && (out == u || reinterpret_cast<const void *>(out) == s_start)) return KDA_ERR_INVALID_ARG;
    return launch_cp_correct(u, s_start, cu_seg, n_seg, skip_seg, n_skip, n_heads, (long long)total_tokens,
                             out, (cudaStream_t)stream);
}

int64_t kda_linear_prefill_workspace(int32_t n_seqs, int64_t total_tokens, int32_t n_heads, int32_t d_k,
                                     int32_t d_v, int32_t dtype)
{
    if (n_seqs < 0 || total_tokens < 0 || total_tokens > 0x7fffffffLL || n_heads < 1 || bad_dtype(dtype) ||
        bad_linear_dims(d_k, d_v))
        return -1;
    return linear_workspace_bytes(n_seqs, total_tokens, n_heads, d_k, d_v, dtype);
}

int kda_linear_prefill(const void *q, const void *k, const void *v, const float *g, int32_t g_per_token,
                       const int32_t *cu_seqlens, int32_t n_seqs, int64_t total_tokens, int32_t n_heads,
                       int32_t n_kv_heads, int32_t d_k, int32_t d_v, float scale, int32_t dtype,
                       int32_t out_dtype, const float *init_state, void *out, float *final_state,
                       void *workspace, int64_t workspace_bytes, void *stream)
{
    const CallRange range("kda_linear_prefill");
    if (n_seqs < 0 || total_tokens < 0 || n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads != 0 ||
        d_k < 1 || d_v < 1 || bad_dtype(dtype) || bad_dtype(out_dtype) || !std::isfinite(scale))
        return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!q || !k || !v || !g || !out)) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && n_seqs == 0) return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens && n_seqs > 1) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;   // cu_seqlens are int32
    if (bad_linear_dims(d_k, d_v)) return KDA_ERR_UNSUPPORTED_SHAPE;
    const void *ptrs[] = {q, k, v, g, init_state, out, final_state, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return KDA_ERR_MISALIGNED;
    if (aliases(out, {q, k, v, g, cu_seqlens, init_state, final_state, workspace}) ||
        aliases(final_state, {q, k, v, g, cu_seqlens, workspace}) ||
        aliases(workspace, {q, k, v, g, cu_seqlens, init_state}))
        return KDA_ERR_INVALID_ARG;
    const int64_t need = linear_workspace_bytes(n_seqs, total_tokens, n_heads, d_k, d_v, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_INVALID_ARG;
    return launch_linear_prefill(q, k, v, g, g_per_token != 0, cu_seqlens, n_seqs, total_tokens, n_heads,
                                 n_kv_heads, d_k, d_v, scale, dtype, out_dtype, init_state, out, final_state,
                                 workspace, (cudaStream_t)stream);
}

int kda_linear_decode(const void *q, const void *k, const void *v, const float *g, int32_t g_per_token,
                      float *state, void *out, int32_t n_seqs, int32_t n_heads, int32_t n_kv_heads,
                      int32_t d_k, int32_t d_v, float scale, int32_t dtype, int32_t out_dtype, void *stream)
{
    const CallRange range("kda_linear_decode");
    if (n_seqs < 0 || n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads != 0 || d_k < 1 || d_v < 1 ||
        bad_dtype(dtype) || bad_dtype(out_dtype) || !std::isfinite(scale))
        return KDA_ERR_INVALID_ARG;
    if (n_seqs > 0 && (!q || !k || !v || !g || !state || !out)) return KDA_ERR_INVALID_ARG;
    if (bad_linear_dims(d_k, d_v)) return KDA_ERR_UNSUPPORTED_SHAPE;
    const void *ptrs[] = {q, k, v, g, state, out};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    if (aliases(out, {q, k, v, g, state}) || aliases(state, {q, k, v, g})) return KDA_ERR_INVALID_ARG;
    return launch_linear_decode(q, k, v, g, g_per_token != 0, state, out, n_seqs, n_heads, n_kv_heads, d_k,
                                d_v, scale, dtype, out_dtype, (cudaStream_t)stream);
}

int kda_delta_prefill(const void *q, const void *k, const void *v, const float *g, int32_t g_per_token,
                      const float *beta, const int32_t *cu_seqlens, int32_t n_seqs, int64_t total_tokens,
                      int32_t n_heads, int32_t n_key_heads, int32_t d_k, int32_t d_v, float scale, int32_t dtype,
                      int32_t out_dtype, const float *init_state, void *out, float *final_state, void *stream)
{
    const CallRange range("kda_delta_prefill");
    if (n_seqs < 0 || total_tokens < 0 || n_heads < 1 || n_key_heads < 1 || n_heads % n_key_heads != 0 ||
        d_k < 1 || d_v < 1 || bad_dtype(dtype) || bad_dtype(out_dtype) || !std::isfinite(scale))
        return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!q || !k || !v || !g || !beta || !out)) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && n_seqs == 0) return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens && n_seqs > 1) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0x7fffffffLL) return KDA_ERR_INVALID_ARG;   // cu_seqlens are int32
    if (bad_linear_dims(d_k, d_v)) return KDA_ERR_UNSUPPORTED_SHAPE;
    const void *ptrs[] = {q, k, v, init_state, out, final_state};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    if (!aligned4(g) || !aligned4(beta) || !aligned4(cu_seqlens)) return KDA_ERR_MISALIGNED;
    if ((int64_t)n_seqs * n_heads > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED_SHAPE;
    const int64_t states = (int64_t)n_seqs * n_heads * d_k * d_v * 4;
    if (delta_overlap(out, total_tokens * n_heads * d_v * bytes_of(out_dtype), q, k, v, g, g_per_token, beta,
                      total_tokens, n_heads, n_key_heads, d_k, d_v, dtype) ||
        delta_overlap(final_state, states, q, k, v, g, g_per_token, beta, total_tokens, n_heads, n_key_heads, d_k, d_v,
                      dtype) ||
        meet(out, total_tokens * n_heads * d_v * bytes_of(out_dtype), init_state, states) ||
        meet(out, total_tokens * n_heads * d_v * bytes_of(out_dtype), final_state, states) ||
        meet(out, total_tokens * n_heads * d_v * bytes_of(out_dtype), cu_seqlens, 4 * ((int64_t)n_seqs + 1)) ||
        meet(final_state, states, cu_seqlens, 4 * ((int64_t)n_seqs + 1)) ||
        (final_state != init_state && meet(final_state, states, init_state, states)))
        return KDA_ERR_INVALID_ARG;
    return launch_delta_prefill(q, k, v, g, g_per_token != 0, beta, cu_seqlens, n_seqs, total_tokens, n_heads,
                                n_key_heads, d_k, d_v, scale, dtype, out_dtype, init_state, out, final_state,
                                (cudaStream_t)stream);
}

int kda_delta_decode(const void *q, const void *k, const void *v, const float *g, int32_t g_per_token,
                     const float *beta, float *state, void *out, int32_t n_seqs, int32_t n_heads,
                     int32_t n_key_heads, int32_t d_k, int32_t d_v, float scale, int32_t dtype, int32_t out_dtype,
                     void *stream)
{
    const CallRange range("kda_delta_decode");
    if (n_seqs < 0 || n_heads < 1 || n_key_heads < 1 || n_heads % n_key_heads != 0 || d_k < 1 || d_v < 1 ||
        bad_dtype(dtype) || bad_dtype(out_dtype) || !std::isfinite(scale))
        return KDA_ERR_INVALID_ARG;
    if (n_seqs > 0 && (!q || !k || !v || !g || !beta || !state || !out)) return KDA_ERR_INVALID_ARG;
    if (bad_linear_dims(d_k, d_v)) return KDA_ERR_UNSUPPORTED_SHAPE;
    const void *ptrs[] = {q, k, v, state, out};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    if (!aligned4(g) || !aligned4(beta)) return KDA_ERR_MISALIGNED;
    if ((int64_t)n_seqs * n_heads > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED_SHAPE;
    const int64_t states = (int64_t)n_seqs * n_heads * d_k * d_v * 4;
    const int64_t outs = (int64_t)n_seqs * n_heads * d_v * bytes_of(out_dtype);
    if (delta_overlap(out, outs, q, k, v, g, g_per_token, beta, n_seqs, n_heads, n_key_heads, d_k, d_v, dtype) ||
        delta_overlap(state, states, q, k, v, g, g_per_token, beta, n_seqs, n_heads, n_key_heads, d_k, d_v, dtype) ||
        meet(out, outs, state, states))
        return KDA_ERR_INVALID_ARG;
    return launch_delta_decode(q, k, v, g, g_per_token != 0, beta, state, out, n_seqs, n_heads, n_key_heads, d_k,
                               d_v, scale, dtype, out_dtype, (cudaStream_t)stream);
}

int kda_state_pack(void *dst, float *dst_scales, int32_t format, const int64_t *dst_idx, int64_t n_dst_slots,
                   const float *src, const int64_t *src_idx, int64_t n_src_slots, int64_t n, int32_t n_heads,
                   int32_t d_k, int32_t d_v, void *stream)
{
    const CallRange range("kda_state_pack");
    const int rc = check_pack(dst, dst_scales, format, dst_idx, n_dst_slots, src, src_idx, n_src_slots, n, n_heads,
                              d_k, d_v);
    if (rc != KDA_OK) return rc;
    return launch_state_pack(dst, dst_scales, format, dst_idx, n_dst_slots, src, src_idx, n_src_slots, n,
                             (int64_t)n_heads * d_k, d_v, (cudaStream_t)stream);
}

int kda_state_unpack(float *dst, const int64_t *dst_idx, int64_t n_dst_slots, const void *src,
                     const float *src_scales, int32_t format, const int64_t *src_idx, int64_t n_src_slots, int64_t n,
                     int32_t n_heads, int32_t d_k, int32_t d_v, void *stream)
{
    const CallRange range("kda_state_unpack");
    const int rc = check_pack(src, src_scales, format, src_idx, n_src_slots, dst, dst_idx, n_dst_slots, n, n_heads,
                              d_k, d_v);
    if (rc != KDA_OK) return rc;
    return launch_state_unpack(dst, dst_idx, n_dst_slots, src, src_scales, format, src_idx, n_src_slots, n,
                               (int64_t)n_heads * d_k, d_v, (cudaStream_t)stream);
}

int kda_norm_gate(const void *o, int32_t o_dtype, const void *z, int32_t z_dtype, const float *w,
                  int32_t w_heads, void *out, int32_t out_dtype, int64_t tokens, int32_t n_heads, int32_t d,
                  float eps, void *stream)
{
    const CallRange range("kda_norm_gate");
    if (tokens < 0 || n_heads < 1 || d < 1 || (w_heads != 1 && w_heads != n_heads) || bad_dtype(o_dtype) ||
        bad_dtype(z_dtype) || bad_dtype(out_dtype) || !(eps > 0.f) || !std::isfinite(eps))
        return KDA_ERR_INVALID_ARG;
    if (tokens > 0 && (!o || !z || !w || !out)) return KDA_ERR_INVALID_ARG;
    if (d % 8 != 0 || d > 256) return KDA_ERR_UNSUPPORTED_SHAPE;
    const void *ptrs[] = {o, z, w, out};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    // in place over o or z is fine (same element type: each element is read before it is written)
    if (out && ((out == o && out_dtype != o_dtype) || (out == z && out_dtype != z_dtype) || out == w))
        return KDA_ERR_INVALID_ARG;
    return launch_norm_gate(o, o_dtype, z, z_dtype, w, w_heads, out, out_dtype, tokens, n_heads, d, eps,
                            (cudaStream_t)stream);
}

int kda_residual_norm(const void *x, int32_t res_dtype, const void *y, const void *z, int32_t dtype,
                      const float *w_post, const float *w, float scale, float eps, void *res, void *out,
                      int64_t tokens, int32_t width, void *stream)
{
    const CallRange range("kda_residual_norm");
    if (tokens < 0 || width < 1 || bad_dtype(res_dtype) || bad_dtype(dtype) || !std::isfinite(scale) ||
        !(eps > 0.f) || !std::isfinite(eps))
        return KDA_ERR_INVALID_ARG;
    if (tokens > 0 && (!x || !w || !out || (y && !res))) return KDA_ERR_INVALID_ARG;
    if (!y && (z || w_post || res)) return KDA_ERR_INVALID_ARG;   // parts of an add that is not there
    const void *ptrs[] = {x, y, z, w_post, w, res, out};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return KDA_ERR_MISALIGNED;
    // res may be x (in place), or y of the same element type; out may be y or z
    if (aliases(out, {x, res, w, w_post}) || aliases(res, {z, w, w_post})) return KDA_ERR_INVALID_ARG;
    if (res && res == y && res_dtype != dtype) return KDA_ERR_INVALID_ARG;
    return launch_residual_norm(x, res_dtype, y, z, dtype, w_post, w, scale, eps, res, out, tokens, width,
                                (cudaStream_t)stream);
}

int64_t kda_prefill_staged_scratch(const int32_t *h_cu_seqlens, int32_t n_seqs, int64_t total_tokens,
                                   int64_t chunk_tokens)
{
    if (n_seqs < 0 || total_tokens < 0 || chunk_tokens < 1 || (n_seqs > 1 && !h_cu_seqlens)) return -1;
    return staged_scratch_ints(h_cu_seqlens, n_seqs, total_tokens, chunk_tokens);
}

int kda_prefill_staged(const void *h_q, const void *h_k, const void *h_v, const void *h_g,
                       const void *h_beta, const int32_t *h_cu_seqlens, int32_t n_seqs,
                       int64_t total_tokens, int32_t n_heads, int32_t dtype, int32_t out_dtype,
                       const float *init_state, void *d_q, void *d_k, void *d_v, void *d_g,
                       void *d_beta, void *d_out, void *h_out, float *final_state,
                       int32_t *d_scratch, int64_t scratch_ints, int64_t chunk_tokens, void *stream)
{
    const CallRange range("kda_prefill_staged");
    int rc = check_staged(h_q, h_k, h_v, h_g, h_beta, h_cu_seqlens, n_seqs, total_tokens, n_heads,
                          dtype, out_dtype, init_state, d_q, d_k, d_v, d_g, d_beta, d_out, h_out,
                          final_state, chunk_tokens);
    if (rc != KDA_OK) return rc;
    if (d_scratch && !aligned16(d_scratch)) return KDA_ERR_MISALIGNED;
    const int64_t need = staged_scratch_ints(h_cu_seqlens, n_seqs, total_tokens, chunk_tokens);
    if (need > 0 && (!d_scratch || scratch_ints < need)) return KDA_ERR_INVALID_ARG;
    const void *h_in[5] = {h_q, h_k, h_v, h_g, h_beta};
    void *d_in[5] = {d_q, d_k, d_v, d_g, d_beta};
    return run_prefill_staged(h_in, h_cu_seqlens, n_seqs, total_tokens, n_heads, dtype, out_dtype,
                              init_state, d_in, d_out, h_out, final_state, d_scratch, chunk_tokens,
                              (cudaStream_t)stream);
}

int kda_prefill_staged_static(const void *h_q, const void *h_k, const void *h_v, const void *h_g,
                              const void *h_beta, const int32_t *h_cu_seqlens, int32_t n_seqs,
                              int64_t total_tokens, int32_t n_heads, int32_t dtype, int32_t out_dtype,
                              const float *init_state, void *d_q, void *d_k, void *d_v, void *d_g,
                              void *d_beta, void *d_out, void *h_out, float *final_state,
                              int64_t chunk_tokens, void *stream)
{
    const CallRange range("kda_prefill_staged_static");
    int rc = check_staged(h_q, h_k, h_v, h_g, h_beta, h_cu_seqlens, n_seqs, total_tokens, n_heads,
                          dtype, out_dtype, init_state, d_q, d_k, d_v, d_g, d_beta, d_out, h_out,
                          final_state, chunk_tokens);
    if (rc != KDA_OK) return rc;
    const void *h_in[5] = {h_q, h_k, h_v, h_g, h_beta};
    void *d_in[5] = {d_q, d_k, d_v, d_g, d_beta};
    return run_prefill_staged_static(h_in, h_cu_seqlens, n_seqs, total_tokens, n_heads, dtype,
                                     out_dtype, init_state, d_in, d_out, h_out, final_state,
                                     chunk_tokens, (cudaStream_t)stream);
}

int kda_diag_device_timeout(int64_t timeout_cycles, void *stream)
{
    if (timeout_cycles < 1 || timeout_cycles > 4000000000LL) return KDA_ERR_INVALID_ARG;
    return kda::launch_wait_timeout_probe((long long)timeout_cycles, (cudaStream_t)stream);
}

int kda_diag_linear_timeout(int64_t timeout_cycles, void *stream)
{
    if (timeout_cycles < 1 || timeout_cycles > 4000000000LL) return KDA_ERR_INVALID_ARG;
    return kda::launch_linear_timeout_probe((uint32_t)timeout_cycles, (cudaStream_t)stream);
}

int kda_diag_delta_timeout(int64_t timeout_cycles, void *stream)
{
    if (timeout_cycles < 1 || timeout_cycles > 4000000000LL) return KDA_ERR_INVALID_ARG;
    return kda::launch_delta_timeout_probe((uint32_t)timeout_cycles, (cudaStream_t)stream);
}

int kda_diag_staged_handles(int64_t *created)
{
    if (!created) return KDA_ERR_INVALID_ARG;
    *created = staged_handles_created();
    return KDA_OK;
}

int kda_diag_bounds_check(int32_t run_probe, int32_t *site, void *stream)
{
    if (!site) return KDA_ERR_INVALID_ARG;
    if (run_probe && kda::launch_bounds_check_probe((cudaStream_t)stream) != KDA_OK) return KDA_ERR_CUDA;
    int32_t a = 0, b = 0;   // the default and the precise build of the tensor-core prefill
    if (kda::read_and_clear_debug_site((cudaStream_t)stream, &a) != KDA_OK ||
        kda::read_and_clear_debug_site_precise((cudaStream_t)stream, &b) != KDA_OK)
        return KDA_ERR_CUDA;
    *site = a != 0 ? a : b;
    return KDA_OK;
}

int kda_device_status(int32_t *status, void *stream)
{
    if (!status) return KDA_ERR_INVALID_ARG;
    return read_and_clear_status((cudaStream_t)stream, status);
}

}  // extern "C"
