// kda_linear.cuh -- shared by the kernels of linear attention with one decay per head: the call's
// parameters and the cut of packed sequences into segments.
//
//     S_t = exp(g_t) S_(t-1) + k_t v_t^T,     o_t = scale S_t^T q_t
//
// The recurrence is affine in the state with a scalar factor, so a sequence may be cut into
// segments that are worked on side by side: a segment's end state is (product of its decays) x
// (its start state) + (its end state from zero).
#pragma once

#include "kda_internal.cuh"

namespace kda {
namespace lin {

struct Args {
    const void *q, *k, *v;       // [T, H, dk], [T, Hkv, dk], [T, Hkv, dv]
    const float *g;              // [T, H] or [H]
    int g_per_token;
    const int32_t *cu;           // [n_seqs + 1] or null (one sequence)
    int n_seqs;
    long long T;
    int H, group;                // query heads, query heads per key/value head
    int dk, dv;
    float scale;
    const float *init;           // [n_seqs, H, dk, dv] or null
    void *out;                   // [T, H, dv]
    float *final_state;          // [n_seqs, H, dk, dv] or null
    int seg_len;                 // tokens of a segment, 0 = sequences are not cut
    int items;                   // segments of all sequences, at most
    float *starts;               // [items, H, dk, dv]: a segment's start state (seg_len > 0)
    float *decays;               // [items, H]: the product of a segment's decays
};

// Segment `item` of the packed sequences: every sequence has max(1, ceil(len / seg_len)) of them,
// so that an empty one has a place where its final state is written.
struct Item {
    int seq, seg, nseg;          // seq < 0: no such item
    long long t0, t1;            // its tokens
};

__device__ __forceinline__ void bounds(const int32_t *cu, long long T, int s, long long &b, long long &e)
{
    b = 0;
    e = T;
    if (cu) {   // a bad table stays inside the tensors
        b = min(max((long long)cu[s], 0ll), T);
        e = min(max((long long)cu[s + 1], b), T);
    }
}

__device__ __forceinline__ int segments(long long len, int seg_len)
{
    return seg_len == 0 ? 1 : max(1, (int)((len + seg_len - 1) / seg_len));
}

// Called by one whole warp; every lane gets the answer.
__device__ __forceinline__ Item find_item(const int32_t *cu, int n_seqs, long long T, int seg_len, int item)
{
    const int lane = threadIdx.x & 31;
    Item it;
    it.seq = -1;
    it.seg = 0;
    it.nseg = 1;
    it.t0 = it.t1 = 0;
    if (seg_len == 0 || !cu) {
        it.seq = seg_len == 0 ? item : 0;
        it.seg = seg_len == 0 ? 0 : item;
        if (it.seq >= n_seqs) it.seq = -1;
    } else {
        int base = 0;
        for (int s0 = 0; s0 < n_seqs; s0 += 32) {
            int cnt = 0;
            if (s0 + lane < n_seqs) {
                long long b, e;
                bounds(cu, T, s0 + lane, b, e);
                cnt = segments(e - b, seg_len);
            }
            int upto = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            const unsigned past = __ballot_sync(0xffffffffu, item - base < upto);
            if (past) {
                const int src = __ffs(past) - 1;
                it.seq = s0 + src;
                it.seg = item - base - __shfl_sync(0xffffffffu, upto - cnt, src);
                break;
            }
            base += __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    if (it.seq < 0) return it;
    long long b, e;
    bounds(cu, T, it.seq, b, e);
    it.nseg = segments(e - b, seg_len);
    if (it.seg >= it.nseg) {
        it.seq = -1;
        return it;
    }
    it.t0 = seg_len ? b + (long long)it.seg * seg_len : b;
    it.t1 = seg_len ? min(e, it.t0 + seg_len) : e;
    return it;
}

// join of the segments, after a state pass
void launch_join(const Args &p, cudaStream_t stream);
int run_tc_path(const Args &p, int out_dtype, cudaStream_t stream);   // bf16 operands
int run_token_path(const Args &p, int dtype, int out_dtype, cudaStream_t stream);
// whether the tensor-core kernel takes these operands
inline bool tc_path(int d_k, int d_v, int dtype) { return dtype == KDA_BF16 && d_k <= 128 && d_v <= 128; }
// tokens of a segment for these sizes, 0 where the sequences are not cut
int plan_segments(int n_seqs, int64_t T, int H, int d_k, int d_v, int dtype);

}  // namespace lin
}  // namespace kda
