// kda_delta.cuh -- shared by the kernels of the gated delta rule with one decay per head.
//
//     S' = exp(g_t) S_(t-1),   S_t = S' + beta_t k_t (v_t - S'^T k_t)^T,   o_t = scale S_t^T q_t
//
// q and k have heads of their own, each shared by `group` value heads; every value head has a state.
#pragma once

#include "kda_internal.cuh"

namespace kda {
namespace delta {

struct Args {
    const void *q, *k, *v;       // [T, H / group, dk] twice, [T, H, dv]
    const float *g;              // [T, H] or [H]
    int g_per_token;
    const float *beta;           // [T, H]
    const int32_t *cu;           // [n_seqs + 1] or null (one sequence)
    int n_seqs;
    long long T;
    int H, group;                // value heads, value heads per query/key head
    int dk, dv;
    float scale;
    const float *init;           // [n_seqs, H, dk, dv] or null
    void *out;                   // [T, H, dv]
    float *final_state;          // [n_seqs, H, dk, dv] or null
};

// tokens [b, e) of sequence s; a bad table stays inside the tensors
__device__ __forceinline__ void bounds(const Args &p, int s, long long &b, long long &e)
{
    b = 0;
    e = p.T;
    if (p.cu) {
        b = min(max((long long)p.cu[s], 0ll), p.T);
        e = min(max((long long)p.cu[s + 1], b), p.T);
    }
}

// two products (and sums) an instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    unsigned long long r, x, y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)   // a b + c
{
    unsigned long long r, x, y, z;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}

// Values in three bf16 parts, x = hi - mid + lo, all 24 bits: what a rounding leaves is its result less the value,
// which takes a half of a packed pair as it is (unpacked, a part of a pair cost four instructions on the ALU,
// which was the chain's busiest pipe, in place of one).
__device__ __forceinline__ void rest(uint32_t h, float2 &x)   // x = h - x
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tsub.rn.f32.bf16 %0, a, %0;\n\tsub.rn.f32.bf16 %1, b, %1;\n\t}"
        : "+f"(x.x), "+f"(x.y) : "r"(h));
}

int run_token_path(const Args &p, int dtype, int out_dtype, cudaStream_t stream);
int run_tc_path(const Args &p, int out_dtype, cudaStream_t stream);   // bf16 operands, d <= 128

}  // namespace delta
}  // namespace kda
