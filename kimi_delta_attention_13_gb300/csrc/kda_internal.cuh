// kda_internal.cuh -- helpers shared by the CUDA translation units of libkda_gb300.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {

// Element conversions for the two input/output dtypes.
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store_as(float *p, float x) { *p = x; }
__device__ __forceinline__ void store_as(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// Retention factor of one token for one key channel: exp of the log-decay clamped to the
// published range [-5, 0] ("Kimi K3 im Detail", section "Sequenz-Mixing", log-decay floor).
__device__ __forceinline__ float retention(float g) { return expf(fminf(fmaxf(g, -5.0f), 0.0f)); }

// 8 consecutive elements <-> 8 floats (16-byte bf16 vector, or two 16-byte fp32 vectors)
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8])
{
    const uint4 r = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8])
{
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

__host__ __device__ constexpr int ceil_div(int a, int b) { return (a + b - 1) / b; }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Per-translation-unit readers of the sticky device error words (see kda_device_status).
int read_and_clear_status_state_copy(cudaStream_t s, int32_t *status);
int read_and_clear_status_prefill_tc(cudaStream_t s, int32_t *status);
int read_and_clear_status_prefill_tc_precise(cudaStream_t s, int32_t *status);
int read_and_clear_status_decode(cudaStream_t s, int32_t *status);
int read_and_clear_status_cp(cudaStream_t s, int32_t *status);
int read_and_clear_status_linear(cudaStream_t s, int32_t *status);
// Launch the one-CTA probe whose bounded device wait expires after `cycles` SM cycles.
int launch_wait_timeout_probe(long long cycles, cudaStream_t stream);
// The same with the linear-attention prefill's wait.
int launch_linear_timeout_probe(uint32_t cycles, cudaStream_t stream);
// Launch the one-thread run of the shared-memory bounds check on an out-of-window offset; read
// (and clear) the site number of the first failed bounds check.
int launch_bounds_check_probe(cudaStream_t stream);
int read_and_clear_debug_site(cudaStream_t s, int32_t *site);
int read_and_clear_debug_site_precise(cudaStream_t s, int32_t *site);

// Kernel launchers (host side, no validation: the C ABI validates first).
int launch_decode(const void *q, const void *k, const void *v, const void *g, const void *beta,
                  float *state, void *out, int n_seqs, int n_heads, int d_k, int d_v, int dtype,
                  int out_dtype, cudaStream_t stream);
int launch_state_copy(float *dst, const int64_t *dst_idx, int64_t n_dst, const float *src,
                      const int64_t *src_idx, int64_t n_src, int64_t n, int64_t unit_floats,
                      cudaStream_t stream);
int launch_prefill_recurrent(const void *q, const void *k, const void *v, const void *g,
                             const void *beta, const int32_t *cu_seqlens, int n_seqs,
                             int64_t total_tokens, int n_heads, int d_k, int d_v, int dtype,
                             int out_dtype, const float *init_state, void *out, float *final_state,
                             int ckpt_stride, float *ckpts, cudaStream_t stream);
int launch_premix(const void *xq, const void *xk, const void *xv, const void *a, const void *b,
                  const float *w, const void *hist, const int32_t *cu_seqlens, int n_seqs,
                  long long total_tokens, int n_heads, int d, float eps, int dtype, void *q,
                  void *k, void *v, void *g, void *beta, cudaStream_t stream);
int launch_output_gate(const void *o, int o_dtype, const void *z, int z_dtype, void *out,
                       int out_dtype, long long n, cudaStream_t stream);
int64_t linear_workspace_bytes(int n_seqs, int64_t T, int H, int d_k, int d_v, int dtype);
int launch_linear_prefill(const void *q, const void *k, const void *v, const float *g, int g_per_token,
                          const int32_t *cu, int n_seqs, int64_t T, int H, int Hkv, int d_k, int d_v,
                          float scale, int dtype, int out_dtype, const float *init, void *out,
                          float *final_state, void *workspace, cudaStream_t stream);
int launch_linear_decode(const void *q, const void *k, const void *v, const float *g, int g_per_token,
                         float *state, void *out, int n_seqs, int H, int Hkv, int d_k, int d_v, float scale,
                         int dtype, int out_dtype, cudaStream_t stream);
int launch_norm_gate(const void *o, int o_dtype, const void *z, int z_dtype, const float *w, int w_heads,
                     void *out, int out_dtype, int64_t T, int H, int d, float eps, cudaStream_t stream);
int launch_residual_norm(const void *x, int res_dtype, const void *y, const void *z, int dtype,
                         const float *w_post, const float *w, float scale, float eps, void *res, void *out,
                         int64_t T, int D, cudaStream_t stream);
int launch_cp_correct(const float *u, const float *s_start, const int32_t *cu_seg, int n_seg,
                      const int32_t *skip_seg, int n_skip, int H, long long T, float *out,
                      cudaStream_t stream);
int launch_cp_combine(const float *s_loc, const float *m, const int32_t *seq_seg, int n_seqs, int H,
                      float *s_start, float *final_state, cudaStream_t stream);
int64_t staged_scratch_ints(const int32_t *h_cu, int n_seqs, long long T, long long chunk_tokens);
int run_prefill_staged(const void *const h_in[5], const int32_t *h_cu, int n_seqs, long long T,
                       int H, int dtype, int out_dtype, const float *init_state, void *const d_in[5],
                       void *d_out, void *h_out, float *final_state, int32_t *d_scratch,
                       long long chunk_tokens, cudaStream_t stream);
int run_prefill_staged_static(const void *const h_in[5], const int32_t *h_cu, int n_seqs, long long T,
                              int H, int dtype, int out_dtype, const float *init_state,
                              void *const d_in[5], void *d_out, void *h_out, float *final_state,
                              long long chunk_tokens, cudaStream_t stream);
// streams and events the staged calls have created so far in this process
long long staged_handles_created();
int launch_prefill_tc(const void *q, const void *k, const void *v, const void *g,
                      const void *beta, const int32_t *cu_seqlens, int n_seqs,
                      int64_t total_tokens, int n_heads, int out_dtype, const float *init_state,
                      void *out, float *final_state, int ckpt_stride, float *ckpts,
                      cudaStream_t stream);
// the same kernel in its precise mode (Aqk carried in two fp16 parts)
int launch_prefill_tc_precise(const void *q, const void *k, const void *v, const void *g,
                              const void *beta, const int32_t *cu_seqlens, int n_seqs,
                              int64_t total_tokens, int n_heads, int out_dtype,
                              const float *init_state, void *out, float *final_state,
                              int ckpt_stride, float *ckpts, cudaStream_t stream);

}  // namespace kda
