// kda_norm.cu -- the norms around a mixer: the gated head norm on its output, and the residual add
// between two blocks with the norm after the first and the norm before the second.
//
//   norm_gate:      out = o rsqrt(mean(o^2) + eps) w sigmoid(z)            over a head's d channels
//   residual_norm:  u = y, or y rsqrt(mean(y^2) + eps) w_post;  u = u sigmoid(z) if z is given
//                   r = x + scale u;   out = r rsqrt(mean(r^2) + eps) w    over a row's D channels
//
// Both stream HBM once: a row stays in registers between its sum of squares and its use, in 32
// bits, and each output is rounded once (the norm of r is taken before r is rounded).  Measured, of
// the copy rate: norm_gate 8192 x 96 x 128 bf16 0.093 ms (0.96; one row a thread group at a time 0.109),
// residual_norm 8192 x 12288 bf16 with both norms and the gate 0.165 ms (0.90; inputs unpacked on
// arrival, which left one block an SM, 0.297).  In fp32 the registers leave room for fewer blocks: norm_gate
// 0.172 (1.03), residual_norm 0.401 (0.74), an fp32 stream with bf16 blocks 0.270 (0.77).
#include <type_traits>

#include "kda_internal.cuh"

namespace kda {
namespace {

// sigmoid(z) = (z < 0 ? e : 1) / (1 + e) with e = exp(-|z|), so that neither e nor the denominator, in
// [1, 2], leaves the range however far out z lies (1 / (1 + exp(-z)) is 0 from z = -88.8 on, where the
// value is 3e-39 and may meet a large factor).  The reciprocal is good to an ulp.  Where every result is
// rounded to bf16 (2^-8) the exponential is the hardware's, of half the argument and squared, which
// keeps a subnormal e: relative error (4 + |z|) 2^-23.  Where one is fp32 it is the full one.
template <bool FULL>
__device__ __forceinline__ float gate(float z)
{
    float e, r;
    if constexpr (FULL) {
        e = expf(-fabsf(z));
    } else {
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fabsf(z) * -0.72134752f));   // log2(e) / 2
        e *= e;
    }
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    if (z < 0.f) r *= e;
    return r;
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// 8 elements as loaded: packed until they are used, so that many loads stay in flight at few registers
template <typename T>
struct Raw8 {
    uint4 u[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p)   // read once: past the L1
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(u[i].x), "=r"(u[i].y), "=r"(u[i].z), "=r"(u[i].w) : "l"(p + i * 4));
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void unpack(float (&v)[8]) const
    {
        if constexpr (sizeof(T) == 2) {
            const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const uint4 a = u[0], b = u[1];
            v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z);
            v[3] = __uint_as_float(a.w); v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
            v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
        }
    }
};

// ---------------------------------------------------------------------------------------------
// norm_gate: GROUP lanes of a warp hold one (token, head) row, 8 channels each; a group takes DEPTH
// rows at a time, all of whose loads go out first

template <typename TX, typename TZ, typename TO, int GROUP, int DEPTH>
__global__ void __launch_bounds__(256) norm_gate_kernel(const TX *o, const TZ *z, const float *__restrict__ w,
                                                        TO *out, long long rows, int H, int w_heads, int d, float eps)
{
    constexpr int PER = 256 / GROUP;   // rows of a block side by side
    const int lane = threadIdx.x % GROUP;
    const bool ok = 8 * lane < d;
    const float inv_d = 1.f / (float)d;
    const long long r0 = (long long)blockIdx.x * PER * DEPTH + threadIdx.x / GROUP;
    Raw8<TX> x[DEPTH];
    Raw8<TZ> g[DEPTH];
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
        const long long r = r0 + i * PER;
        if (ok && r < rows) {
            x[i].load(o + r * d + 8 * lane);
            g[i].load(z + r * d + 8 * lane);
        } else {
            x[i].zero();
            g[i].zero();
        }
    }
    float wv[8] = {};
    if (ok && w_heads == 1) load8(w + 8 * lane, wv);
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) {
        const long long r = r0 + i * PER;
        float v[8], gv[8];
        x[i].unpack(v);
        g[i].unpack(gv);
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) ss = fmaf(v[c], v[c], ss);
#pragma unroll
        for (int m = GROUP / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float inv = rsqrtf(fmaf(ss, inv_d, eps));
        if (ok && r < rows) {
            if (w_heads > 1) load8(w + r % H * d + 8 * lane, wv);
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] *= inv * wv[c] * gate<sizeof(TO) == 4>(gv[c]);
            store8(out + r * d + 8 * lane, v);
        }
    }
}

// ---------------------------------------------------------------------------------------------
// residual_norm: one row per block of THREADS, VECS groups of 8 channels per thread

struct ResidualArgs {
    const void *x, *y, *z;       // [T, D]; y and z may be null
    const float *w_post, *w;     // w_post may be null
    void *res, *out;
    long long rows;
    int D;
    float scale, eps;
};

template <int THREADS>
__device__ __forceinline__ float block_sum(float x, float *buf)
{
    x = warp_sum(x);
    if constexpr (THREADS > 32) {
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) x += buf[i];
    }
    return x;
}

// The row's inputs are loaded at once and stay packed; where that leaves 64 registers a thread
// enough, 1024 threads of several blocks share an SM, one's loads beside another's sums.
template <typename TR, typename TB, int VECS>
constexpr bool fits64() { return 2 * VECS * (sizeof(TR) + 2 * sizeof(TB)) <= 36; }

template <typename TR, typename TB, int THREADS, int VECS>
__global__ void __launch_bounds__(THREADS, fits64<TR, TB, VECS>() ? 1024 / THREADS : 1) residual_norm_kernel(const ResidualArgs p)
{
    __shared__ float buf[2][32];
    const long long row = blockIdx.x, base = row * p.D;
    const TR *x = static_cast<const TR *>(p.x) + base;
    const TB *y = p.y ? static_cast<const TB *>(p.y) + base : nullptr;
    const TB *z = p.z ? static_cast<const TB *>(p.z) + base : nullptr;
    Raw8<TR> xr[VECS];
    Raw8<TB> yr[VECS], zr[VECS];
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int c = (i * THREADS + threadIdx.x) * 8;
        yr[i].zero();
        xr[i].zero();
        zr[i].zero();
        if (c < p.D) {
            if (y) yr[i].load(y + c);
            xr[i].load(x + c);
            if (z) zr[i].load(z + c);
        }
    }
    float inv_post = p.scale;
    if (y && p.w_post) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            float u[8];
            yr[i].unpack(u);
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(u[e], u[e], ss);
        }
        inv_post = p.scale * rsqrtf(block_sum<THREADS>(ss, buf[0]) / (float)p.D + p.eps);
    }
    float r[VECS][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int c = (i * THREADS + threadIdx.x) * 8;
        xr[i].unpack(r[i]);
        if (y && c < p.D) {
            float u[8];
            yr[i].unpack(u);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] *= inv_post;
            if (p.w_post) {
                float wp[8];
                load8(p.w_post + c, wp);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] *= wp[e];
            }
            if (z) {
                float g[8];
                zr[i].unpack(g);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] *= gate<(sizeof(TR) == 4 || sizeof(TB) == 4)>(g[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) r[i][e] += u[e];
            store8(static_cast<TR *>(p.res) + base + c, r[i]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(r[i][e], r[i][e], ss);
    }
    const float inv = rsqrtf(block_sum<THREADS>(ss, buf[1]) / (float)p.D + p.eps);
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int c = (i * THREADS + threadIdx.x) * 8;
        if (c >= p.D) continue;
        float wv[8];
        load8(p.w + c, wv);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] *= inv * wv[e];
        store8(static_cast<TB *>(p.out) + base + c, r[i]);
    }
}

// Any width: scalar accesses, r computed once for its sum and once for its use (8192 rows with both norms
// and the gate: 1001 channels 35.5 us, 0.34 of the copy rate; 12289 365 us, 0.41).
template <typename TR, typename TB>
__global__ void __launch_bounds__(256) residual_norm_any_kernel(const ResidualArgs p)
{
    __shared__ float buf[2][32];
    const long long base = (long long)blockIdx.x * p.D;
    const TR *x = static_cast<const TR *>(p.x) + base;
    const TB *y = p.y ? static_cast<const TB *>(p.y) + base : nullptr;
    const TB *z = p.z ? static_cast<const TB *>(p.z) + base : nullptr;
    float inv_post = p.scale;
    if (y && p.w_post) {
        float ss = 0.f;
        for (int c = threadIdx.x; c < p.D; c += 256) {
            const float t = to_f32(y[c]);
            ss = fmaf(t, t, ss);
        }
        inv_post = p.scale * rsqrtf(block_sum<256>(ss, buf[0]) / (float)p.D + p.eps);
    }
    auto value = [&](int c) {
        float r = to_f32(x[c]);
        if (y) {
            float t = to_f32(y[c]) * inv_post;
            if (p.w_post) t *= p.w_post[c];
            if (z) t *= gate<(sizeof(TR) == 4 || sizeof(TB) == 4)>(to_f32(z[c]));
            r += t;
        }
        return r;
    };
    float ss = 0.f;
    for (int c = threadIdx.x; c < p.D; c += 256) {
        const float r = value(c);
        ss = fmaf(r, r, ss);
    }
    const float inv = rsqrtf(block_sum<256>(ss, buf[1]) / (float)p.D + p.eps);
    for (int c = threadIdx.x; c < p.D; c += 256) {   // res may be x: a channel is read before it is written
        const float r = value(c);
        if (y) store_as(static_cast<TR *>(p.res) + base + c, r);
        store_as(static_cast<TB *>(p.out) + base + c, r * inv * p.w[c]);
    }
}

template <typename TR, typename TB>
void launch_residual(const ResidualArgs &p, cudaStream_t stream)
{
    const unsigned rows = (unsigned)p.rows;
    if (p.D % 8 != 0 || p.D > 16384) {
        residual_norm_any_kernel<TR, TB><<<rows, 256, 0, stream>>>(p);
        return;
    }
    const int vecs = p.D / 8;
    // Two or three groups of channels a thread rather than one: more rows share an SM, and their loads
    // cover one another's sums (8192 x 4096, norms and gate: 55.5 us with 192 threads, 65.8 with 512;
    // 8192 x 1024: 15.5 with 64, 16.3 with 128). At 12288 blocks of 768 were slower than 512.  Blocks of 512
    // from 4104 channels on leave threads idle (8192 rows, norms and gate: 4104 85.8 us, 0.58 of the copy
    // rate; 5120 92.1, 0.67; 6144 98.3, 0.75; 8192 116, 0.85).  Without an add the registers for y and z
    // stay reserved: 8192 x 4096 28.5 us, 0.69; 8192 x 12288 83.4, 0.71.
    if (vecs <= 128) residual_norm_kernel<TR, TB, 64, 2><<<rows, 64, 0, stream>>>(p);
    else if (vecs <= 256) residual_norm_kernel<TR, TB, 128, 2><<<rows, 128, 0, stream>>>(p);
    else if (vecs <= 512) residual_norm_kernel<TR, TB, 192, 3><<<rows, 192, 0, stream>>>(p);
    else if (vecs <= 1024) residual_norm_kernel<TR, TB, 512, 2><<<rows, 512, 0, stream>>>(p);
    else if (vecs <= 1536) residual_norm_kernel<TR, TB, 512, 3><<<rows, 512, 0, stream>>>(p);
    else residual_norm_kernel<TR, TB, 512, 4><<<rows, 512, 0, stream>>>(p);
}

}  // namespace

int launch_norm_gate(const void *o, int o_dtype, const void *z, int z_dtype, const float *w, int w_heads,
                     void *out, int out_dtype, int64_t T, int H, int d, float eps, cudaStream_t stream)
{
    const long long rows = T * H;
    if (rows == 0) return KDA_OK;
    auto go = [&](auto xt, auto zt, auto ot) {
        using X = decltype(xt);
        using Z = decltype(zt);
        using O = decltype(ot);
        auto launch = [&](auto group) {
            constexpr int G = decltype(group)::value, PER = 256 / G, DEPTH = 4;
            auto run = [&](auto depth) {
                constexpr int N = decltype(depth)::value;
                norm_gate_kernel<X, Z, O, G, N><<<(unsigned)((rows + PER * N - 1) / (PER * N)), 256, 0, stream>>>(
                    (const X *)o, (const Z *)z, w, (O *)out, rows, H, w_heads, d, eps);
            };
            // Few rows (less than 32 such blocks an SM): one at a time, so that more blocks take part
            // (d = 128: 160 rows 1.6 us against 2.0, 98304 rows 11.9 against 13.0, 786432 rows 95.6
            // against 91.0).
            if (rows >= 152ll * 32 * PER * DEPTH) run(std::integral_constant<int, DEPTH>{});
            else run(std::integral_constant<int, 1>{});
        };
        if (d <= 64) launch(std::integral_constant<int, 8>{});
        else if (d <= 128) launch(std::integral_constant<int, 16>{});
        else launch(std::integral_constant<int, 32>{});
    };
    auto with_z = [&](auto xt, auto zt) {
        if (out_dtype == KDA_BF16) go(xt, zt, __nv_bfloat16{}); else go(xt, zt, float{});
    };
    auto with_x = [&](auto xt) {
        if (z_dtype == KDA_BF16) with_z(xt, __nv_bfloat16{}); else with_z(xt, float{});
    };
    if (o_dtype == KDA_BF16) with_x(__nv_bfloat16{}); else with_x(float{});
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int launch_residual_norm(const void *x, int res_dtype, const void *y, const void *z, int dtype,
                         const float *w_post, const float *w, float scale, float eps, void *res, void *out,
                         int64_t T, int D, cudaStream_t stream)
{
    if (T == 0) return KDA_OK;
    if (T > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED_SHAPE;
    const ResidualArgs p = {x, y, z, w_post, w, res, out, T, D, scale, eps};
    if (res_dtype == KDA_BF16) {
        if (dtype == KDA_BF16) launch_residual<__nv_bfloat16, __nv_bfloat16>(p, stream);
        else launch_residual<__nv_bfloat16, float>(p, stream);
    } else {
        if (dtype == KDA_BF16) launch_residual<float, __nv_bfloat16>(p, stream);
        else launch_residual<float, float>(p, stream);
    }
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace kda
