// kda_state_pack.cu -- states kept in fewer bits: written into slots of a pool and read back.
//
//     bf16:  held = x rounded to bf16
//     int8:  s = max |row| / 127 in fp32,  held = x / s rounded to the nearest whole number, ties to even,
//            per row of a state (one key channel's value channels);   read back as held s
//
// A row has a scale of its own because a state's key channels differ in magnitude by what was written under
// them.  The code is that of the exact quotient: the remainder x - code s is exact in one fused
// multiply-add, and a code that it shows to be the wrong neighbour is moved by one.
// Bound by HBM: 4 bytes an element on one side, 1 (and 4 a row) or 2 on the other.  LANES lanes take a row in V
// pieces of four columns each, U rows in flight a thread.  64 slots of 96 heads of 128 x 128, warm, of the measured
// copy rate: int8 written 88 us (0.85), read back 80 us (0.93); bf16 written 103 us (0.87), read back 92 us (0.96).
// 64 x 64: 25 us (0.75) and 24 us (0.79).  72 columns, written: 66 us (0.64), one lane in four of the row idle.
#include <type_traits>

#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

__device__ int g_state_pack_error;    // sticky device error word of this translation unit

struct Move {
    void *held;                 // pool [n_held, rows, dv] of int8 or bf16
    float *scales;              // [n_held, rows] (int8)
    float *full;                // states [n_full, rows, dv] fp32
    const int64_t *held_idx, *full_idx;
    int64_t n_held, n_full, n;
    int64_t rows;               // of a state: H dk
    int dv;
};

// the slots of pair i; false (and the error word) where one is out of range
__device__ __forceinline__ bool slots(const Move &m, int64_t i, int64_t &held, int64_t &full)
{
    held = m.held_idx ? m.held_idx[i] : i;
    full = m.full_idx ? m.full_idx[i] : i;
    if (held >= 0 && held < m.n_held && full >= 0 && full < m.n_full) return true;
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicExch(&g_state_pack_error, KDA_ERR_INDEX_RANGE);
    return false;
}

constexpr float kMagic = 12582912.f;  // 1.5 x 2^23: a sum with it is rounded to a whole number, in its low bits

// The codes of four values, as bytes.  A code is that of the exact quotient x / s, ties to even: what x / s rounds
// to may be the wrong one of two neighbours, which the exact remainder x - code s shows.
__device__ __forceinline__ uint32_t codes(float4 f, float s, float inv)
{
    const float x[4] = {f.x, f.y, f.z, f.w};
    float m[4], far = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        m[e] = fmaf(x[e], inv, kMagic);
        far = fmaxf(far, fabsf(fmaf(kMagic - m[e], s, x[e])));
    }
    if (!(2.f * far < s) || inv == 0.f) {   // a remainder of half a step or more, or no reciprocal
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float r = inv > 0.f ? m[e] - kMagic : rintf(x[e] / s);
            const float left = fmaf(-r, s, x[e]), twice = 2.f * fabsf(left);
            if (twice > s || (twice == s && ((int)r & 1))) r += copysignf(1.f, left);
            m[e] = fminf(fmaxf(r, -127.f), 127.f) + kMagic;
        }
    }
    return __byte_perm(__byte_perm(__float_as_uint(m[0]), __float_as_uint(m[1]), 0x0040),
                       __byte_perm(__float_as_uint(m[2]), __float_as_uint(m[3]), 0x0040), 0x5410);
}

// max / 127 correctly rounded: a quotient by the rounded reciprocal, corrected once by its remainder (Markstein)
__device__ __forceinline__ float scale_of(float top)
{
    if (top < 1e-30f) return __fdiv_rn(top, 127.f);   // (its remainder would underflow)
    const float q = top * (1.f / 127.f);
    return fmaf(fmaf(-q, 127.f, top), 1.f / 127.f, q);
}

// LANES lanes a row of at most 4 LANES V columns, U rows in flight a thread
template <int LANES, int V, int U>
__global__ void __launch_bounds__(kThreads) state_pack8_kernel(const Move m)
{
    constexpr int SIDE = kThreads / LANES;           // rows of the block side by side
    const int lane = threadIdx.x % LANES, side = threadIdx.x / LANES;
    for (int64_t i = blockIdx.y; i < m.n; i += gridDim.y) {
        int64_t hs, fs;
        if (!slots(m, i, hs, fs)) continue;
        const float *from = m.full + fs * m.rows * m.dv;
        uint8_t *to = static_cast<uint8_t *>(m.held) + hs * m.rows * m.dv;
        float *scales = m.scales + hs * m.rows;
        for (int64_t r0 = (int64_t)blockIdx.x * SIDE * U; r0 < m.rows; r0 += (int64_t)gridDim.x * SIDE * U) {
            float4 x[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    const int64_t row = r0 + u * SIDE + side;
                    const int col = 4 * (lane + c * LANES);
                    x[u][c] = row < m.rows && col < m.dv ? __ldcs(reinterpret_cast<const float4 *>(from + row * m.dv + col))
                                                        : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            uint32_t top[U];                         // magnitudes as bits: infinities and NaN are the largest
#pragma unroll
            for (int u = 0; u < U; ++u) {
                top[u] = 0;
#pragma unroll
                for (int c = 0; c < V; ++c)
                    top[u] = max(top[u], max(max(__float_as_uint(x[u][c].x) & 0x7fffffffu, __float_as_uint(x[u][c].y) & 0x7fffffffu),
                                             max(__float_as_uint(x[u][c].z) & 0x7fffffffu, __float_as_uint(x[u][c].w) & 0x7fffffffu)));
            }
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
                for (int u = 0; u < U; ++u) top[u] = max(top[u], __shfl_xor_sync(0xffffffffu, top[u], o));
            float s[U], inv[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[u] = top[u] >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : scale_of(__uint_as_float(top[u]));
                // (the reciprocal of a scale that is all but 0 would overflow)
                inv[u] = s[u] >= 1e-30f ? __frcp_rn(s[u]) : 0.f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = r0 + u * SIDE + side;
                if (row >= m.rows) break;
                if (lane == 0) scales[row] = s[u];
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    const int col = 4 * (lane + c * LANES);
                    // a row of zeros, or one not finite, has codes 0
                    if (col < m.dv) *reinterpret_cast<uint32_t *>(to + row * m.dv + col) = s[u] > 0.f ? codes(x[u][c], s[u], inv[u]) : 0u;
                }
            }
        }
    }
}

template <int LANES, int V, int U>
__global__ void __launch_bounds__(kThreads) state_unpack8_kernel(const Move m)
{
    constexpr int SIDE = kThreads / LANES;
    const int lane = threadIdx.x % LANES, side = threadIdx.x / LANES;
    for (int64_t i = blockIdx.y; i < m.n; i += gridDim.y) {
        int64_t hs, fs;
        if (!slots(m, i, hs, fs)) continue;
        float *to = m.full + fs * m.rows * m.dv;
        const uint8_t *from = static_cast<const uint8_t *>(m.held) + hs * m.rows * m.dv;
        const float *scales = m.scales + hs * m.rows;
        for (int64_t r0 = (int64_t)blockIdx.x * SIDE * U; r0 < m.rows; r0 += (int64_t)gridDim.x * SIDE * U) {
            uint32_t w[U][V];
            float s[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = r0 + u * SIDE + side;
                s[u] = row < m.rows ? __ldg(scales + row) : 0.f;
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    const int col = 4 * (lane + c * LANES);
                    w[u][c] = row < m.rows && col < m.dv ? __ldcs(reinterpret_cast<const uint32_t *>(from + row * m.dv + col)) : 0u;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    const int64_t row = r0 + u * SIDE + side;
                    const int col = 4 * (lane + c * LANES);
                    if (row < m.rows && col < m.dv) {
                        const uint32_t x = w[u][c];
                        __stcs(reinterpret_cast<float4 *>(to + row * m.dv + col),
                               make_float4((float)(int8_t)(x & 0xffu) * s[u], (float)(int8_t)(x >> 8 & 0xffu) * s[u],
                                           (float)(int8_t)(x >> 16 & 0xffu) * s[u], (float)(int8_t)(x >> 24) * s[u]));
                    }
                }
        }
    }
}

template <bool PACK>
__global__ void __launch_bounds__(kThreads) state_bf16_kernel(const Move m)
{
    constexpr int U = 4;
    const int64_t vecs = m.rows * m.dv / 4, stride = (int64_t)gridDim.x * kThreads;
    for (int64_t i = blockIdx.y; i < m.n; i += gridDim.y) {
        int64_t hs, fs;
        if (!slots(m, i, hs, fs)) continue;
        float4 *full = reinterpret_cast<float4 *>(m.full) + fs * vecs;
        uint2 *held = static_cast<uint2 *>(m.held) + hs * vecs;
        for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < vecs; e += U * stride) {
            if constexpr (PACK) {
                float4 x[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (e + u * stride < vecs) x[u] = __ldcs(full + e + u * stride);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (e + u * stride < vecs) {
                        const __nv_bfloat162 a = __floats2bfloat162_rn(x[u].x, x[u].y), b = __floats2bfloat162_rn(x[u].z, x[u].w);
                        held[e + u * stride] = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
                    }
            } else {
                uint2 w[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (e + u * stride < vecs) w[u] = __ldcs(held + e + u * stride);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (e + u * stride < vecs)
                        __stcs(full + e + u * stride,
                               make_float4(__uint_as_float(w[u].x << 16), __uint_as_float(w[u].x & 0xffff0000u),
                                           __uint_as_float(w[u].y << 16), __uint_as_float(w[u].y & 0xffff0000u)));
            }
        }
    }
}

int run(const Move &m, int format, bool pack, cudaStream_t stream)
{
    if (m.n == 0) return KDA_OK;
    if (m.dv % 4 != 0 || m.dv > 256) return KDA_ERR_UNSUPPORTED_SHAPE;
    const unsigned ys = (unsigned)(m.n < 65535 ? m.n : 65535);
    auto blocks = [&](int64_t each) {   // of a state, `each` rows or vectors a block
        const int64_t rows = format == KDA_STATE_INT8 ? m.rows : m.rows * m.dv / 4;
        const int64_t b = (rows + each - 1) / each;
        return dim3((unsigned)(b < 65536 ? b : 65536), ys);
    };
    if (format == KDA_STATE_BF16) {
        if (pack) state_bf16_kernel<true><<<blocks(4 * kThreads), kThreads, 0, stream>>>(m);
        else state_bf16_kernel<false><<<blocks(4 * kThreads), kThreads, 0, stream>>>(m);
    } else {
        auto pack8 = [&](auto lanes, auto v, auto u) {
            constexpr int L = decltype(lanes)::value, V = decltype(v)::value, U = decltype(u)::value;
            state_pack8_kernel<L, V, U><<<blocks(kThreads / L * U), kThreads, 0, stream>>>(m);
        };
        auto unpack8 = [&](auto lanes, auto v, auto u) {
            constexpr int L = decltype(lanes)::value, V = decltype(v)::value, U = decltype(u)::value;
            state_unpack8_kernel<L, V, U><<<blocks(kThreads / L * U), kThreads, 0, stream>>>(m);
        };
        using std::integral_constant;
        using one = integral_constant<int, 1>;
        using two = integral_constant<int, 2>;
        using three = integral_constant<int, 3>;
        using four = integral_constant<int, 4>;
        using quarter = integral_constant<int, 4>;
        using eight = integral_constant<int, 8>;
        using half = integral_constant<int, 16>;
        using whole = integral_constant<int, 32>;
        // Packing wants few rows in flight and long pieces of them: a row's maximum crosses its lanes and is divided
        // by 127 in each, so eight lanes of sixteen values cost less than thirty-two of four.  64 x 96 states of
        // 128 x 128: 32 lanes and 4 rows 106 us, 8 rows 135; 16 lanes and 4, 2, 1 rows 117, 95, 116; 8 lanes and 1
        // row 88.  64 wide: 16 lanes 32, 8 lanes 27, 4 lanes 25.  72 wide: 32 lanes of which 14 idle 104, here 66.
        // 32 states of 32 heads of 256 x 256: 32 lanes and 2 rows 66, 16 lanes 60, 8 lanes 56.
        // Reading back has nothing across lanes and wants every load in flight that registers hold.
        if (pack) {
            if (m.dv <= 32) pack8(quarter{}, two{}, two{});
            else if (m.dv <= 64) pack8(quarter{}, four{}, one{});
            else if (m.dv <= 96) pack8(eight{}, three{}, one{});
            else if (m.dv <= 128) pack8(eight{}, four{}, one{});
            else pack8(eight{}, eight{}, one{});
        } else {
            if (m.dv <= 32) unpack8(eight{}, one{}, eight{});
            else if (m.dv <= 64) unpack8(half{}, one{}, eight{});
            else if (m.dv <= 96) unpack8(eight{}, three{}, four{});
            else if (m.dv <= 128) unpack8(whole{}, one{}, eight{});
            else unpack8(whole{}, two{}, four{});
        }
    }
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

int launch_state_pack(void *dst, float *scales, int format, const int64_t *dst_idx, int64_t n_dst, const float *src,
                      const int64_t *src_idx, int64_t n_src, int64_t n, int64_t rows, int dv, cudaStream_t stream)
{
    const Move m{dst, scales, const_cast<float *>(src), dst_idx, src_idx, n_dst, n_src, n, rows, dv};
    return run(m, format, true, stream);
}

int launch_state_unpack(float *dst, const int64_t *dst_idx, int64_t n_dst, const void *src, const float *scales,
                        int format, const int64_t *src_idx, int64_t n_src, int64_t n, int64_t rows, int dv,
                        cudaStream_t stream)
{
    const Move m{const_cast<void *>(src), const_cast<float *>(scales), dst, src_idx, dst_idx, n_src, n_dst, n, rows, dv};
    return run(m, format, false, stream);
}

int *status_word_state_pack()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_state_pack_error) == cudaSuccess ? static_cast<int *>(p) : nullptr;
}

}  // namespace kda
