// kda_delta_decode.cu -- one token per sequence of the gated delta rule with one decay per head, state
// updated in place.
//
//     u = beta (v - a S^T k),   S <- a S + k u^T,   o = scale S^T q = scale (a S_old^T q + (k . q) u),   a = exp(g)
//
// A state is read and written once, all else is small (HBM-bound, 1.5 flops a byte).  u needs the sums over
// all key channels of the old state, so a block keeps its columns of the state in registers between the
// read and the write: LANES float4 columns of one (sequence, head), DEPTH rows a thread, all their loads in
// flight at once; both sums (with k and with q) are taken in one sweep and joined across the warps once.
#include <type_traits>

#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxDim = 256;

template <typename T, typename TO, int LANES, int DEPTH>
__global__ void __launch_bounds__(kThreads)
delta_decode_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                    const float *__restrict__ g, int g_per_token, const float *__restrict__ beta,
                    float *__restrict__ state, TO *__restrict__ out, int H, int group, int dk, int dv, float scale)
{
    constexpr int ROWS = kThreads / LANES;   // rows of the state side by side
    __shared__ float s_k[kMaxDim], s_q[kMaxDim];
    __shared__ __align__(16) float4 s_part[2][kWarps][LANES];
    __shared__ float s_kq[kWarps];
    const long long nh = blockIdx.x;
    const int h = (int)(nh % H), Hk = H / group;
    const long long nk = nh / H * Hk + h / group;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid % LANES, row = tid / LANES;
    const int col = (blockIdx.y * LANES + lane) * 4;
    const bool ok = col < dv;
    const int pitch = dv / 4;
    float4 *S = reinterpret_cast<float4 *>(state + nh * dk * dv + col);
    float4 st[DEPTH];
#pragma unroll
    for (int m = 0; m < DEPTH; ++m) {   // the state's loads go out before the small operands'
        const int i = row + m * ROWS;
        st[m] = ok && i < dk ? __ldcs(S + (long long)i * pitch) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float kq = 0.f;
    if (tid < kMaxDim) {
        const float ki = tid < dk ? to_f32(k[nk * dk + tid]) : 0.f, qi = tid < dk ? to_f32(q[nk * dk + tid]) : 0.f;
        s_k[tid] = ki;
        s_q[tid] = qi;
        kq = ki * qi;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, o);
    if ((tid & 31) == 0) s_kq[warp] = kq;
    const float a = expf(g[g_per_token ? nh : h]), b = beta[nh];
    float x[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = ok ? to_f32(v[nh * dv + col + c]) : 0.f;
    __syncthreads();
    float4 rk = make_float4(0.f, 0.f, 0.f, 0.f), rq = rk;
#pragma unroll
    for (int m = 0; m < DEPTH; ++m) {
        const float ki = s_k[row + m * ROWS], qi = s_q[row + m * ROWS];   // (0 past d_k)
        rk.x = fmaf(st[m].x, ki, rk.x); rk.y = fmaf(st[m].y, ki, rk.y);
        rk.z = fmaf(st[m].z, ki, rk.z); rk.w = fmaf(st[m].w, ki, rk.w);
        rq.x = fmaf(st[m].x, qi, rq.x); rq.y = fmaf(st[m].y, qi, rq.y);
        rq.z = fmaf(st[m].z, qi, rq.z); rq.w = fmaf(st[m].w, qi, rq.w);
    }
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) {   // rows within the warp
        rk.x += __shfl_xor_sync(0xffffffffu, rk.x, o); rk.y += __shfl_xor_sync(0xffffffffu, rk.y, o);
        rk.z += __shfl_xor_sync(0xffffffffu, rk.z, o); rk.w += __shfl_xor_sync(0xffffffffu, rk.w, o);
        rq.x += __shfl_xor_sync(0xffffffffu, rq.x, o); rq.y += __shfl_xor_sync(0xffffffffu, rq.y, o);
        rq.z += __shfl_xor_sync(0xffffffffu, rq.z, o); rq.w += __shfl_xor_sync(0xffffffffu, rq.w, o);
    }
    if ((tid & 31) < LANES) {
        s_part[0][warp][lane] = rk;
        s_part[1][warp][lane] = rq;
    }
    __syncthreads();
    rk = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float4 p = s_part[0][w][lane];
        rk.x += p.x; rk.y += p.y; rk.z += p.z; rk.w += p.w;
    }
    const float4 u = make_float4(b * fmaf(-a, rk.x, x[0]), b * fmaf(-a, rk.y, x[1]), b * fmaf(-a, rk.z, x[2]),
                                 b * fmaf(-a, rk.w, x[3]));
#pragma unroll
    for (int m = 0; m < DEPTH; ++m) {
        const int i = row + m * ROWS;
        if (ok && i < dk) {
            const float ki = s_k[i];
            float4 s = st[m];
            s.x = fmaf(s.x, a, ki * u.x); s.y = fmaf(s.y, a, ki * u.y);
            s.z = fmaf(s.z, a, ki * u.z); s.w = fmaf(s.w, a, ki * u.w);
            __stcs(S + (long long)i * pitch, s);
        }
    }
    if (row == 0 && ok) {
        float sum = 0.f;
        rq = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 p = s_part[1][w][lane];
            rq.x += p.x; rq.y += p.y; rq.z += p.z; rq.w += p.w;
            sum += s_kq[w];
        }
        TO *o = out + nh * dv + col;
        store_as(o, scale * fmaf(a, rq.x, sum * u.x));
        store_as(o + 1, scale * fmaf(a, rq.y, sum * u.y));
        store_as(o + 2, scale * fmaf(a, rq.z, sum * u.z));
        store_as(o + 3, scale * fmaf(a, rq.w, sum * u.w));
    }
}

}  // namespace

int launch_delta_decode(const void *q, const void *k, const void *v, const float *g, int g_per_token,
                        const float *beta, float *state, void *out, int n_seqs, int H, int Hk, int d_k, int d_v,
                        float scale, int dtype, int out_dtype, cudaStream_t stream)
{
    const int64_t blocks = (int64_t)n_seqs * H;
    if (blocks == 0) return KDA_OK;
    if (blocks > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED_SHAPE;
    auto go = [&](auto in_tag, auto out_tag, auto lanes, auto depth) {
        using T = decltype(in_tag);
        using TO = decltype(out_tag);
        constexpr int L = decltype(lanes)::value, D = decltype(depth)::value;
        const dim3 grid((unsigned)blocks, (unsigned)ceil_div(d_v, 4 * L));
        delta_decode_kernel<T, TO, L, D><<<grid, kThreads, 0, stream>>>(
            (const T *)q, (const T *)k, (const T *)v, g, g_per_token, beta, state, (TO *)out, H, H / Hk, d_k, d_v, scale);
    };
    auto sizes = [&](auto in_tag, auto out_tag) {
        using std::integral_constant;
        if (d_k > 128) go(in_tag, out_tag, integral_constant<int, 8>{}, integral_constant<int, 8>{});
        else if (d_k > 64) go(in_tag, out_tag, integral_constant<int, 8>{}, integral_constant<int, 4>{});
        else go(in_tag, out_tag, integral_constant<int, 8>{}, integral_constant<int, 2>{});
    };
    if (dtype == KDA_BF16) {
        if (out_dtype == KDA_BF16) sizes(__nv_bfloat16{}, __nv_bfloat16{}); else sizes(__nv_bfloat16{}, float{});
    } else {
        if (out_dtype == KDA_BF16) sizes(float{}, __nv_bfloat16{}); else sizes(float{}, float{});
    }
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace kda
