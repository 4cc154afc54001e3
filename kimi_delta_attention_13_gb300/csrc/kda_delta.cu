// kda_delta.cu -- the gated delta rule with one decay per head, token by token on CUDA cores.
//
//     S' = exp(g_t) S_(t-1),   S_t = S' + beta_t k_t (v_t - S'^T k_t)^T,   o_t = scale S_t^T q_t
//
// The columns of a state (value channels) do not meet, so a warp keeps all key channels of NC columns in
// registers, R rows a lane, and needs no other warp: the sums over key channels stay inside it.  A sum of
// NC columns over 32 lanes is folded so that every step halves the columns a lane still carries, and a lane
// ends with one column's sum (NC = 8: 9 shuffles in place of 40).
#include "kda_delta.cuh"

namespace kda {
namespace delta {
namespace {

constexpr int kWarps = 4;      // warps of a block, each on its own columns
constexpr int kAhead = 4;      // tokens whose loads are in flight

template <int R>
__device__ __forceinline__ void load_row(const float *p, float (&x)[R])
{
#pragma unroll
    for (int i = 0; i < R; i += 2) {
        const float2 f = *reinterpret_cast<const float2 *>(p + i);
        x[i] = f.x;
        x[i + 1] = f.y;
    }
}
template <int R>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *p, float (&x)[R])
{
#pragma unroll
    for (int i = 0; i < R; i += 2) {
        const uint32_t u = *reinterpret_cast<const uint32_t *>(p + i);
        x[i] = __uint_as_float(u << 16);
        x[i + 1] = __uint_as_float(u & 0xffff0000u);
    }
}

// Sums s[c] over the lanes, for NC columns; lane l ends with that of column l / (32 / NC).
template <int NC>
__device__ __forceinline__ float fold(float (&s)[NC], int lane)
{
    int o = 16;
#pragma unroll
    for (int n = NC / 2; n >= 1; n /= 2, o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int c = 0; c < n; ++c) {
            const float send = up ? s[c] : s[c + n];
            const float keep = up ? s[c + n] : s[c];
            s[c] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    float x = s[0];
#pragma unroll
    for (; o >= 1; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename T, typename TO, int R, int NC>
__global__ void __launch_bounds__(32 * kWarps) delta_token_kernel(const Args p)
{
    constexpr int SUB = 32 / NC;   // lanes that end with the same column
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int seq = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / p.group, Hk = p.H / p.group;
    const int c0 = (blockIdx.y * kWarps + warp) * NC;
    if (c0 >= p.dv) return;
    long long b, e;
    bounds(p, seq, b, e);
    const int row = lane * R, col = c0 + lane / SUB;
    const bool row_ok = row < p.dk, col_ok = col < p.dv;   // (d_k is a multiple of 8, so of R)
    const long long own = (((long long)seq * p.H + h) * p.dk + row) * p.dv + c0;
    float2 st[R][NC / 2];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.init && row_ok && c0 + c < p.dv) s = *reinterpret_cast<const float4 *>(p.init + own + (long long)r * p.dv + c);
            st[r][c / 2] = make_float2(s.x, s.y);
            st[r][c / 2 + 1] = make_float2(s.z, s.w);
        }
    const T *q = static_cast<const T *>(p.q) + hk * p.dk + row, *k = static_cast<const T *>(p.k) + hk * p.dk + row;
    const T *v = static_cast<const T *>(p.v) + (long long)h * p.dv + col;
    const long long qk_step = (long long)Hk * p.dk, v_step = (long long)p.H * p.dv;
    float nk[kAhead][R], nq[kAhead][R], nv[kAhead], ng[kAhead], nb[kAhead];
    auto fetch = [&](long long t, int i) {
#pragma unroll
        for (int r = 0; r < R; ++r) nk[i][r] = nq[i][r] = 0.f;
        nv[i] = ng[i] = nb[i] = 0.f;
        if (t < e) {
            if (row_ok) {
                load_row<R>(k + t * qk_step, nk[i]);
                load_row<R>(q + t * qk_step, nq[i]);
            }
            if (col_ok) nv[i] = to_f32(v[t * v_step]);
            ng[i] = p.g[p.g_per_token ? t * p.H + h : h];
            nb[i] = p.beta[t * p.H + h];
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(b + i, i);
    for (long long t0 = b; t0 < e; t0 += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const long long t = t0 + i;
            if (t >= e) break;
            const float a = expf(ng[i]);
            float2 acc[NC / 2] = {};
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int c = 0; c < NC / 2; ++c) acc[c] = fma2(st[r][c], make_float2(nk[i][r], nk[i][r]), acc[c]);
            float s[NC];
#pragma unroll
            for (int c = 0; c < NC / 2; ++c) {
                s[2 * c] = acc[c].x;
                s[2 * c + 1] = acc[c].y;
            }
            const float u = nb[i] * fmaf(-a, fold<NC>(s, lane), nv[i]);
            float2 o[NC / 2] = {};
#pragma unroll
            for (int c = 0; c < NC / 2; ++c) {
                const float2 uc = make_float2(__shfl_sync(0xffffffffu, u, 2 * c * SUB), __shfl_sync(0xffffffffu, u, (2 * c + 1) * SUB));
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    st[r][c] = fma2(make_float2(nk[i][r], nk[i][r]), uc, mul2(st[r][c], make_float2(a, a)));
                    o[c] = fma2(st[r][c], make_float2(nq[i][r], nq[i][r]), o[c]);
                }
            }
#pragma unroll
            for (int c = 0; c < NC / 2; ++c) {
                s[2 * c] = o[c].x;
                s[2 * c + 1] = o[c].y;
            }
            const float sum = fold<NC>(s, lane);
            if (lane % SUB == 0 && col_ok)
                store_as(static_cast<TO *>(p.out) + (t * p.H + h) * p.dv + col, sum * p.scale);
            fetch(t + kAhead, i);
        }
    }
    if (p.final_state && row_ok) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < NC; c += 4)
                if (c0 + c < p.dv)
                    *reinterpret_cast<float4 *>(p.final_state + own + (long long)r * p.dv + c) =
                        make_float4(st[r][c / 2].x, st[r][c / 2].y, st[r][c / 2 + 1].x, st[r][c / 2 + 1].y);
    }
}

template <typename T, typename TO>
int launch(const Args &p, cudaStream_t stream)
{
    constexpr int NC = 8;
    const dim3 grid((unsigned)(p.n_seqs * p.H), (unsigned)ceil_div(p.dv, NC * kWarps));
    if (p.dk <= 64) delta_token_kernel<T, TO, 2, NC><<<grid, 32 * kWarps, 0, stream>>>(p);
    else if (p.dk <= 128) delta_token_kernel<T, TO, 4, NC><<<grid, 32 * kWarps, 0, stream>>>(p);
    else delta_token_kernel<T, TO, 8, NC><<<grid, 32 * kWarps, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

int run_token_path(const Args &p, int dtype, int out_dtype, cudaStream_t stream)
{
    if (dtype == KDA_BF16)
        return out_dtype == KDA_BF16 ? launch<__nv_bfloat16, __nv_bfloat16>(p, stream) : launch<__nv_bfloat16, float>(p, stream);
    return out_dtype == KDA_BF16 ? launch<float, __nv_bfloat16>(p, stream) : launch<float, float>(p, stream);
}

// Whether the tensor-core kernel takes these operands.
bool tc_path(int n_seqs, int64_t T, int d_k, int d_v, int dtype)
{
    return dtype == KDA_BF16 && d_k <= 128 && d_v <= 128 && T >= 8 * (int64_t)n_seqs;
}

}  // namespace delta

int launch_delta_prefill(const void *q, const void *k, const void *v, const float *g, int g_per_token,
                         const float *beta, const int32_t *cu, int n_seqs, int64_t T, int H, int Hk, int d_k,
                         int d_v, float scale, int dtype, int out_dtype, const float *init, void *out,
                         float *final_state, cudaStream_t stream)
{
    if (n_seqs == 0) return KDA_OK;
    if ((int64_t)n_seqs * H > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED_SHAPE;
    delta::Args p;
    p.q = q; p.k = k; p.v = v; p.g = g;
    p.g_per_token = g_per_token;
    p.beta = beta;
    p.cu = n_seqs == 1 ? nullptr : cu;
    p.n_seqs = n_seqs;
    p.T = T;
    p.H = H;
    p.group = H / Hk;
    p.dk = d_k; p.dv = d_v;
    p.scale = scale;
    p.init = init;
    p.out = out;
    p.final_state = final_state;
    if (delta::tc_path(n_seqs, T, d_k, d_v, dtype)) return delta::run_tc_path(p, out_dtype, stream);
    return delta::run_token_path(p, dtype, out_dtype, stream);
}

}  // namespace kda
