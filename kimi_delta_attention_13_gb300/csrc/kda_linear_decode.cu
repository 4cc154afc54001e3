// kda_linear_decode.cu -- one token per sequence of linear attention with one decay per head,
// state updated in place:
//
//     S <- exp(g) S + k v^T,     o = scale S^T q
//
// A state of d_k x d_v fp32 is read and written once, all else is small (HBM-bound, about half a
// flop per byte).  Unlike the delta rule nothing about the old state is needed before it is
// written back, so a row is updated, stored and added into the read as it arrives.  A block takes
// `LANES` float4 columns of one (sequence, head); its threads are rows x LANES and each keeps eight
// rows' loads in flight.  256 sequences of 96 heads (128 x 128): 0.466 ms, 1.03 of the measured copy
// rate, so the states move by plain wide loads and stores; a handful of states is bound by the
// launch (32 states 2.7 us on the device).
#include <type_traits>

#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDim = 256;

template <typename T, typename TO, int LANES>
__global__ void __launch_bounds__(kThreads)
linear_decode_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                     const float *__restrict__ g, int g_per_token, float *__restrict__ state,
                     TO *__restrict__ out, int H, int group, int dk, int dv, float scale)
{
    constexpr int ROWS = kThreads / LANES;   // rows of the state side by side
    constexpr int DEPTH = 8;
    __shared__ float s_k[kMaxDim], s_q[kMaxDim];
    __shared__ __align__(16) float4 s_part[ROWS][LANES];
    const long long nh = blockIdx.x;
    const int h = (int)(nh % H), Hkv = H / group;
    const long long nk = nh / H * Hkv + h / group;
    const int tid = threadIdx.x, lane = tid % LANES, row = tid / LANES;
    const int col = (blockIdx.y * LANES + lane) * 4;
    const bool ok = col < dv;
    float4 *S = reinterpret_cast<float4 *>(state + nh * dk * dv + col);
    const int pitch = dv / 4;
    float4 st[DEPTH];
    auto load = [&](int i0) {
#pragma unroll
        for (int m = 0; m < DEPTH; ++m) {
            const int i = i0 + row + m * ROWS;
            st[m] = ok && i < dk ? __ldcs(S + (long long)i * pitch) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    load(0);   // the state's loads go out before the small operands'
    for (int i = tid; i < dk; i += kThreads) {
        s_k[i] = to_f32(k[nk * dk + i]);
        s_q[i] = to_f32(q[nh * dk + i]);
    }
    const float a = expf(g[g_per_token ? nh : h]);
    float x[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = ok ? to_f32(v[nk * dv + col + c]) : 0.f;
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < dk; i0 += DEPTH * ROWS) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int m = 0; m < DEPTH; ++m) {
            const int i = i0 + row + m * ROWS;
            if (i < dk && ok) {
                const float ki = s_k[i], qi = s_q[i];
                float4 s = st[m];
                s.x = fmaf(s.x, a, ki * x[0]); s.y = fmaf(s.y, a, ki * x[1]);
                s.z = fmaf(s.z, a, ki * x[2]); s.w = fmaf(s.w, a, ki * x[3]);
                __stcs(S + (long long)i * pitch, s);
                acc.x = fmaf(s.x, qi, acc.x); acc.y = fmaf(s.y, qi, acc.y);
                acc.z = fmaf(s.z, qi, acc.z); acc.w = fmaf(s.w, qi, acc.w);
            }
        }
    }
    s_part[row][lane] = acc;
    __syncthreads();
    if (tid < 4 * LANES) {
        float sum = 0.f;
        for (int r = 0; r < ROWS; ++r) sum += reinterpret_cast<const float *>(&s_part[r][0])[tid];
        const int c = blockIdx.y * LANES * 4 + tid;
        if (c < dv) store_as(out + nh * dv + c, sum * scale);
    }
}

}  // namespace

int launch_linear_decode(const void *q, const void *k, const void *v, const float *g, int g_per_token,
                         float *state, void *out, int n_seqs, int H, int Hkv, int d_k, int d_v, float scale,
                         int dtype, int out_dtype, cudaStream_t stream)
{
    const int64_t blocks = (int64_t)n_seqs * H;
    if (blocks == 0) return KDA_OK;
    if (blocks > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED_SHAPE;
    auto go = [&](auto in_tag, auto out_tag, auto lanes) {
        using T = decltype(in_tag);
        using TO = decltype(out_tag);
        constexpr int L = decltype(lanes)::value;
        const dim3 grid((unsigned)blocks, (unsigned)ceil_div(d_v, 4 * L));
        linear_decode_kernel<T, TO, L><<<grid, kThreads, 0, stream>>>(
            (const T *)q, (const T *)k, (const T *)v, g, g_per_token, state, (TO *)out, H, H / Hkv, d_k, d_v,
            scale);
    };
    auto lanes = [&](auto in_tag, auto out_tag) {
        // Fewer states than SMs: slices of 32 columns (whole 128-byte lines), so that four times the SMs
        // take part (32 states 2.7 us against 3.6 us, 288 states 6.3 against 5.1).
        if (blocks < 152 || d_v <= 32) go(in_tag, out_tag, std::integral_constant<int, 8>{});
        else if (d_v <= 64) go(in_tag, out_tag, std::integral_constant<int, 16>{});
        else go(in_tag, out_tag, std::integral_constant<int, 32>{});
    };
    if (dtype == KDA_BF16) {
        if (out_dtype == KDA_BF16) lanes(__nv_bfloat16{}, __nv_bfloat16{}); else lanes(__nv_bfloat16{}, float{});
    } else {
        if (out_dtype == KDA_BF16) lanes(float{}, __nv_bfloat16{}); else lanes(float{}, float{});
    }
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace kda
