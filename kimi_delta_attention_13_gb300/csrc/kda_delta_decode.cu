// kda_delta_decode.cu -- one token per sequence of the gated delta rule with one decay per head, state
// updated in place.
//
//     u = beta (v - a S^T k),   S <- a S + k u^T,   o = scale S^T q = scale (a S_old^T q + (k . q) u),   a = exp(g)
//
// A state is read and written once, all else is small (HBM-bound, 1.5 flops a byte).  u needs the sums over
// all key channels of the old state, so a block keeps its columns of the state in registers between the
// read and the write: LANES float4 columns of one (sequence, head), DEPTH rows a thread, all their loads in
// flight at once; both sums (with k and with q) are taken in one sweep and joined across the warps once.  Many
// large states go through shared memory instead (delta_decode_bulk_kernel).  256 sequences of 96 heads (128 x 128):
// 0.463 ms, 1.03 of the measured copy rate; 32 states 2.9 us on the device, bound by the launch.
#include <type_traits>

#include "kda_internal.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxDim = 256;

// A token's decay.  It is 1 + expm1 where it is near 1: rounded to fp32 itself, a decay that stays the same would be
// off the same way token after token (over 256 tokens of memory 1e-6 of the state).
struct Decay {
    float a, m, one;   // the decay; and as m + one
    __device__ __forceinline__ explicit Decay(float g)
    {
        const bool near = g > -0.25f;
        m = near ? expm1f(g) : expf(g);
        a = near ? 1.f + m : m;
        one = near ? 1.f : 0.f;
    }
    __device__ __forceinline__ float4 step(float4 s, float k, float4 u) const   // a s + k u
    {
        return make_float4(fmaf(k, u.x, fmaf(s.x, m, s.x * one)), fmaf(k, u.y, fmaf(s.y, m, s.y * one)),
                           fmaf(k, u.z, fmaf(s.z, m, s.z * one)), fmaf(k, u.w, fmaf(s.w, m, s.w * one)));
    }
};

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
    const Decay d(g[g_per_token ? nh : h]);
    const float b = beta[nh];
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
    const float4 u = make_float4(b * fmaf(-d.a, rk.x, x[0]), b * fmaf(-d.a, rk.y, x[1]), b * fmaf(-d.a, rk.z, x[2]),
                                 b * fmaf(-d.a, rk.w, x[3]));
#pragma unroll
    for (int m = 0; m < DEPTH; ++m) {
        const int i = row + m * ROWS;
        if (ok && i < dk) {
            __stcs(S + (long long)i * pitch, d.step(st[m], s_k[i], u));
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
        store_as(o, scale * fmaf(d.a, rq.x, sum * u.x));
        store_as(o + 1, scale * fmaf(d.a, rq.y, sum * u.y));
        store_as(o + 2, scale * fmaf(d.a, rq.z, sum * u.z));
        store_as(o + 3, scale * fmaf(d.a, rq.w, sum * u.w));
    }
}

// A state of up to 64 KB, one contiguous block, by one bulk copy each way through shared memory: three such blocks
// share an SM, so that up to 192 KB are in flight whatever the registers hold.
constexpr uint32_t kMaxBulk = 65536;
constexpr long long kTimeout = 2000000000ll;   // SM cycles (~1 s): bounded waits

__device__ int g_delta_decode_error;   // sticky device error word of this translation unit

template <typename T, typename TO>
__global__ void __launch_bounds__(kThreads)
delta_decode_bulk_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                         const float *__restrict__ g, int g_per_token, const float *__restrict__ beta,
                         float *__restrict__ state, TO *__restrict__ out, int H, int group, int dk, int dv, float scale)
{
    using namespace ptx;
    extern __shared__ __align__(128) float4 sS[];
    __shared__ __align__(8) uint64_t bar;
    __shared__ float s_k[kMaxDim], s_q[kMaxDim];
    __shared__ __align__(16) float4 s_part[kThreads];
    __shared__ float s_kq[kWarps];
    __shared__ int s_zero;   // the abort flag of the waits: never set, they end by timeout only
    const long long nh = blockIdx.x;
    const int h = (int)(nh % H), Hk = H / group;
    const long long nk = nh / H * Hk + h / group;
    const int tid = threadIdx.x, warp = tid >> 5;
    const int lanes = dv / 4, rows = kThreads / lanes, lane = tid % lanes, row = tid / lanes;
    const bool ok = row < rows;
    const uint32_t bytes = (uint32_t)(dk * dv * 4);
    float *S = state + nh * dk * dv;
    if (tid == 0) {
        s_zero = 0;
        mbar_init(&bar, 1);
        fence_barrier_init();
        mbar_arrive_expect_tx(&bar, bytes);
        bulk_load_1d(sS, S, bytes, &bar);   // the state goes out first
    }
    const float ki = tid < dk ? to_f32(k[nk * dk + tid]) : 0.f, qi = tid < dk ? to_f32(q[nk * dk + tid]) : 0.f;
    s_k[tid] = ki;
    s_q[tid] = qi;
    float kq = ki * qi;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, o);
    if ((tid & 31) == 0) s_kq[warp] = kq;
    const Decay d(g[g_per_token ? nh : h]);
    const float b = beta[nh];
    float x[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = ok ? to_f32(v[nh * dv + 4 * lane + c]) : 0.f;
    __syncthreads();
    const bool landed = mbar_wait(&bar, 0, &s_zero, kTimeout);
    if (!__syncthreads_and(landed)) {
        if (tid == 0) {
            atomicExch(&g_delta_decode_error, KDA_ERR_DEVICE_TIMEOUT);
            mbar_wait(&bar, 0, &s_zero, kTimeout);   // no copy left in flight at exit
        }
        return;
    }
    float4 rk = make_float4(0.f, 0.f, 0.f, 0.f), rq = rk;
    if (ok) {
#pragma unroll 4
        for (int i = row; i < dk; i += rows) {
            const float4 s = sS[i * lanes + lane];
            const float kr = s_k[i], qr = s_q[i];
            rk.x = fmaf(s.x, kr, rk.x); rk.y = fmaf(s.y, kr, rk.y); rk.z = fmaf(s.z, kr, rk.z); rk.w = fmaf(s.w, kr, rk.w);
            rq.x = fmaf(s.x, qr, rq.x); rq.y = fmaf(s.y, qr, rq.y); rq.z = fmaf(s.z, qr, rq.z); rq.w = fmaf(s.w, qr, rq.w);
        }
    }
    auto joined = [&](float4 part) {   // the sum of all rows' parts (one buffer, so that three blocks share an SM)
        s_part[tid] = part;
        __syncthreads();
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ok)
            for (int r = 0; r < rows; ++r) {
                const float4 a = s_part[r * lanes + lane];
                sum.x += a.x; sum.y += a.y; sum.z += a.z; sum.w += a.w;
            }
        __syncthreads();
        return sum;
    };
    rk = joined(rk);
    const float4 u = make_float4(b * fmaf(-d.a, rk.x, x[0]), b * fmaf(-d.a, rk.y, x[1]), b * fmaf(-d.a, rk.z, x[2]),
                                 b * fmaf(-d.a, rk.w, x[3]));
    if (ok) {
#pragma unroll 4
        for (int i = row; i < dk; i += rows) sS[i * lanes + lane] = d.step(sS[i * lanes + lane], s_k[i], u);
    }
    fence_proxy_async_smem();
    rq = joined(rq);   // (and every thread's part of the state is written)
    if (tid == 0) {
        bulk_store_1d(S, sS, bytes);
        bulk_commit();
    }
    if (row == 0) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += s_kq[w];
        TO *o = out + nh * dv + 4 * lane;
        store_as(o, scale * fmaf(d.a, rq.x, sum * u.x));
        store_as(o + 1, scale * fmaf(d.a, rq.y, sum * u.y));
        store_as(o + 2, scale * fmaf(d.a, rq.z, sum * u.z));
        store_as(o + 3, scale * fmaf(d.a, rq.w, sum * u.w));
    }
    if (tid == 0) bulk_wait_read_all();   // the shared-memory source stays until the copy has read it
}

}  // namespace

int *status_word_delta_decode()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_delta_decode_error) == cudaSuccess ? static_cast<int *>(p) : nullptr;
}

int launch_delta_decode(const void *q, const void *k, const void *v, const float *g, int g_per_token,
                        const float *beta, float *state, void *out, int n_seqs, int H, int Hk, int d_k, int d_v,
                        float scale, int dtype, int out_dtype, cudaStream_t stream)
{
    const int64_t blocks = (int64_t)n_seqs * H;
    if (blocks == 0) return KDA_OK;
    if (blocks > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED_SHAPE;
    bool attr_ok = true;
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
        using T = decltype(in_tag);
        using TO = decltype(out_tag);
        const int bytes = d_k * d_v * 4;
        // Large states, and enough of them that an SM has three at a time, by bulk copies (128 x 128, us, by bulk
        // copies and by slices of 64 columns: 24,576 states 462, 544; 6144 122, 133; 512 14.0, 15.2; 128 6.0, 5.4;
        // 64 x 64 is better off in slices: 6144 states 44.7, 34.9).
        if (bytes > (int)kMaxBulk / 2 && bytes <= (int)kMaxBulk && blocks >= 512) {
            // a function attribute belongs to the current device: set it on every launch
            attr_ok = cudaFuncSetAttribute(delta_decode_bulk_kernel<T, TO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)kMaxBulk) == cudaSuccess;
            if (attr_ok)
                delta_decode_bulk_kernel<T, TO><<<(unsigned)blocks, kThreads, bytes, stream>>>(
                    (const T *)q, (const T *)k, (const T *)v, g, g_per_token, beta, state, (TO *)out, H, H / Hk, d_k, d_v, scale);
        } else if (d_k > 128) {
            go(in_tag, out_tag, integral_constant<int, 8>{}, integral_constant<int, 8>{});
        } else if (blocks < 152) {
            // Fewer states than SMs: slices of 32 columns (whole 128-byte lines), so that more SMs take part (32
            // states of 128 x 128 2.9 us against 3.3 in slices of 64; 592 of 64 x 64 7.4 against 5.6).
            if (d_k > 64) go(in_tag, out_tag, integral_constant<int, 8>{}, integral_constant<int, 4>{});
            else go(in_tag, out_tag, integral_constant<int, 8>{}, integral_constant<int, 2>{});
        } else {
            if (d_k > 64) go(in_tag, out_tag, integral_constant<int, 16>{}, integral_constant<int, 8>{});
            else go(in_tag, out_tag, integral_constant<int, 16>{}, integral_constant<int, 4>{});
        }
    };
    if (dtype == KDA_BF16) {
        if (out_dtype == KDA_BF16) sizes(__nv_bfloat16{}, __nv_bfloat16{}); else sizes(__nv_bfloat16{}, float{});
    } else {
        if (out_dtype == KDA_BF16) sizes(float{}, __nv_bfloat16{}); else sizes(float{}, float{});
    }
    return attr_ok && cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace kda
