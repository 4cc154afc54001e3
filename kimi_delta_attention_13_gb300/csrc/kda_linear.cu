// kda_linear.cu -- linear attention with one decay per head, token by token on CUDA cores, and
// the join of segments.
//
//     S_t = exp(g_t) S_(t-1) + k_t v_t^T,     o_t = scale S_t^T q_t
//
// This is the path for fp32 inputs and for head sizes the tensor-core kernel does not take.  A
// block owns 32 value columns of one (segment, head): lane = column, warp w = key channels
// [w ROWS, (w + 1) ROWS), the state in registers.  Per token and thread that is a multiply, a
// fused multiply-add into the state and one into the read for each of its rows; key and query rows
// come from shared memory as broadcasts, a block of tokens at a time.
//
// Long sequences are cut into segments worked on side by side: linear_token_kernel<.., false>
// leaves the end state of every segment but a sequence's last (from zeros; a first segment from
// the initial state), linear_join_kernel turns those into the segments' true start states, and
// linear_token_kernel<.., true> computes the outputs.
#include "kda_linear.cuh"

namespace kda {
namespace lin {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCols = 32;

template <typename T, typename TO, int ROWS, bool OUT>
__global__ void __launch_bounds__(kThreads) linear_token_kernel(const Args p)
{
    constexpr int DK = ROWS * kWarps;          // padded key channels
    constexpr int TB = ROWS <= 16 ? 16 : 8;    // tokens staged at a time
    __shared__ __align__(16) float sk[TB][DK];
    __shared__ __align__(16) float sq[OUT ? TB : 1][DK];
    __shared__ float sv[TB][kCols];
    __shared__ float sa[TB];
    __shared__ float part[OUT ? TB : 1][kWarps][kCols];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % p.H, item = blockIdx.x / p.H, hk = h / p.group;
    const int col = blockIdx.y * kCols + lane;
    const bool col_ok = col < p.dv;
    const Item it = find_item(p.cu, p.n_seqs, p.T, p.seg_len, item);
    if (it.seq < 0 || (!OUT && it.seg == it.nseg - 1)) return;

    const long long unit = (long long)p.dk * p.dv;
    const long long own = ((long long)it.seq * p.H + h) * unit, slot = ((long long)item * p.H + h) * unit;
    const float *from = nullptr;
    if (it.seg == 0) from = p.init ? p.init + own : nullptr;
    if (OUT && it.nseg > 1 && (it.seg > 0 || p.init)) from = p.starts + slot;
    float st[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int i = warp * ROWS + r;
        st[r] = from && col_ok && i < p.dk ? from[(long long)i * p.dv + col] : 0.f;
        // a first segment's start is kept: the last segment may overwrite it (final_state = init)
        if (!OUT && it.seg == 0 && p.init && col_ok && i < p.dk)
            p.starts[slot + (long long)i * p.dv + col] = st[r];
    }
    float whole = 1.f;
    const T *q = static_cast<const T *>(p.q), *k = static_cast<const T *>(p.k), *v = static_cast<const T *>(p.v);
    const int Hkv = p.H / p.group;
    for (long long tb = it.t0; tb < it.t1; tb += TB) {
        const int n = (int)min((long long)TB, it.t1 - tb);
        __syncthreads();
        for (int e = tid; e < TB * DK; e += kThreads) {
            const int t = e / DK, i = e % DK;
            const bool ok = t < n && i < p.dk;
            sk[t][i] = ok ? to_f32(k[((tb + t) * Hkv + hk) * p.dk + i]) : 0.f;
            if constexpr (OUT) sq[t][i] = ok ? to_f32(q[((tb + t) * p.H + h) * p.dk + i]) : 0.f;
        }
        for (int e = tid; e < TB * kCols; e += kThreads) {
            const int t = e / kCols, c = blockIdx.y * kCols + e % kCols;
            sv[t][e % kCols] = t < n && c < p.dv ? to_f32(v[((tb + t) * Hkv + hk) * p.dv + c]) : 0.f;
        }
        if (tid < TB) sa[tid] = tid < n ? expf(p.g_per_token ? p.g[(tb + tid) * p.H + h] : p.g[h]) : 1.f;
        __syncthreads();
        for (int t = 0; t < n; ++t) {
            const float a = sa[t], x = sv[t][lane];
            const float4 *k4 = reinterpret_cast<const float4 *>(&sk[t][warp * ROWS]);
            float acc = 0.f;
#pragma unroll
            for (int r = 0; r < ROWS / 4; ++r) {
                const float4 kr = k4[r];
                st[4 * r] = fmaf(st[4 * r], a, kr.x * x);
                st[4 * r + 1] = fmaf(st[4 * r + 1], a, kr.y * x);
                st[4 * r + 2] = fmaf(st[4 * r + 2], a, kr.z * x);
                st[4 * r + 3] = fmaf(st[4 * r + 3], a, kr.w * x);
                if constexpr (OUT) {
                    const float4 qr = reinterpret_cast<const float4 *>(&sq[t][warp * ROWS])[r];
                    acc += st[4 * r] * qr.x + st[4 * r + 1] * qr.y + st[4 * r + 2] * qr.z + st[4 * r + 3] * qr.w;
                }
            }
            if constexpr (OUT) part[t][warp][lane] = acc;
            if constexpr (!OUT) whole *= a;
        }
        if constexpr (OUT) {
            __syncthreads();
            for (int e = tid; e < n * kCols; e += kThreads) {
                const int t = e / kCols, c = e % kCols;
                float acc = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) acc += part[t][w][c];
                if (blockIdx.y * kCols + c < p.dv)
                    store_as(static_cast<TO *>(p.out) + ((tb + t) * p.H + h) * p.dv + blockIdx.y * kCols + c,
                             acc * p.scale);
            }
        }
    }
    // OUT: the last segment leaves the sequence's final state.  Otherwise the end state from zeros
    // goes to the next segment's place, and the segment's decay to its own.
    float *to = nullptr;
    if (OUT) to = it.seg == it.nseg - 1 && p.final_state ? p.final_state + own : nullptr;
    else to = p.starts + slot + (long long)p.H * unit;
    if (to && col_ok) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int i = warp * ROWS + r;
            if (i < p.dk) to[(long long)i * p.dv + col] = st[r];
        }
    }
    if (!OUT && tid == 0 && blockIdx.y == 0) p.decays[(long long)item * p.H + h] = whole;
}

// starts[j + 1] = decays[j] starts[j] + (end of segment j from zeros), for j = 1 .. nseg - 2 of every
// sequence; one float4 of a state per thread, the chain over segments in registers
__global__ void __launch_bounds__(256) linear_join_kernel(const Args p)
{
    const int seq = blockIdx.x / p.H, h = blockIdx.x % p.H, lane = threadIdx.x & 31;
    int first = 0;
    if (p.cu) {
        for (int s = lane; s < seq; s += 32) {
            long long b, e;
            bounds(p.cu, p.T, s, b, e);
            first += segments(e - b, p.seg_len);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) first += __shfl_xor_sync(0xffffffffu, first, o);
    }
    long long b, e;
    bounds(p.cu, p.T, seq, b, e);
    const int nseg = segments(e - b, p.seg_len);
    const long long unit4 = (long long)p.dk * p.dv / 4;
    const long long x = (long long)blockIdx.y * blockDim.x + threadIdx.x;
    if (nseg < 3 || first + nseg > p.items || x >= unit4) return;
    float4 *s = reinterpret_cast<float4 *>(p.starts) + ((long long)first * p.H + h) * unit4 + x;
    const float *a = p.decays + (long long)first * p.H + h;
    const long long step = (long long)p.H * unit4;
    float4 cur = s[step];
#pragma unroll 4
    for (int j = 1; j < nseg - 1; ++j) {
        const float f = a[(long long)j * p.H];
        const float4 d = s[(j + 1) * step];
        cur = make_float4(fmaf(f, cur.x, d.x), fmaf(f, cur.y, d.y), fmaf(f, cur.z, d.z), fmaf(f, cur.w, d.w));
        s[(j + 1) * step] = cur;
    }
}

template <typename T, typename TO, bool OUT>
void launch_tokens(const Args &p, cudaStream_t stream)
{
    const dim3 grid((unsigned)(p.items * p.H), (unsigned)ceil_div(p.dv, kCols));
    if (p.dk <= 64) linear_token_kernel<T, TO, 8, OUT><<<grid, kThreads, 0, stream>>>(p);
    else if (p.dk <= 128) linear_token_kernel<T, TO, 16, OUT><<<grid, kThreads, 0, stream>>>(p);
    else linear_token_kernel<T, TO, 32, OUT><<<grid, kThreads, 0, stream>>>(p);
}

template <typename T, typename TO>
int run_tokens(const Args &p, cudaStream_t stream)
{
    if (p.seg_len > 0) {
        launch_tokens<T, float, false>(p, stream);
        launch_join(p, stream);
    }
    launch_tokens<T, TO, true>(p, stream);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

void launch_join(const Args &p, cudaStream_t stream)
{
    const dim3 grid((unsigned)(p.n_seqs * p.H), (unsigned)ceil_div(p.dk * p.dv / 4, 256));
    linear_join_kernel<<<grid, 256, 0, stream>>>(p);
}

int run_token_path(const Args &p, int dtype, int out_dtype, cudaStream_t stream)
{
    if (dtype == KDA_BF16)
        return out_dtype == KDA_BF16 ? run_tokens<__nv_bfloat16, __nv_bfloat16>(p, stream)
                                     : run_tokens<__nv_bfloat16, float>(p, stream);
    return out_dtype == KDA_BF16 ? run_tokens<float, __nv_bfloat16>(p, stream)
                                 : run_tokens<float, float>(p, stream);
}

// Segments are cut when the uncut sequences give the machine too few blocks.
int plan_segments(int n_seqs, int64_t T, int H, int d_k, int d_v, int dtype)
{
    if (tc_path(d_k, d_v, dtype)) {
        const int64_t ctas = (int64_t)n_seqs * H;
        if (ctas >= 76) return 0;
        int64_t len = (T * H / 152 + 127) / 128 * 128;
        if (len < 512) len = 512;
        return T <= len ? 0 : (int)len;
    }
    const int64_t slices = ceil_div(d_v, kCols), blocks = (int64_t)n_seqs * H * slices;
    const int64_t want = 152 * 4;
    if (blocks >= want) return 0;
    int64_t len = (T * H * slices / want + 15) / 16 * 16;
    if (len < 64) len = 64;
    return T <= len ? 0 : (int)len;
}

}  // namespace lin

int64_t linear_workspace_bytes(int n_seqs, int64_t T, int H, int d_k, int d_v, int dtype)
{
    const int seg = lin::plan_segments(n_seqs, T, H, d_k, d_v, dtype);
    if (seg == 0) return 0;
    const int64_t items = T / seg + n_seqs;
    return items * H * d_k * d_v * 4 + (items * H * 4 + 15) / 16 * 16;
}

int launch_linear_prefill(const void *q, const void *k, const void *v, const float *g, int g_per_token,
                          const int32_t *cu, int n_seqs, int64_t T, int H, int Hkv, int d_k, int d_v,
                          float scale, int dtype, int out_dtype, const float *init, void *out,
                          float *final_state, void *workspace, cudaStream_t stream)
{
    if (n_seqs == 0) return KDA_OK;
    lin::Args p;
    p.q = q; p.k = k; p.v = v; p.g = g;
    p.g_per_token = g_per_token;
    p.cu = n_seqs == 1 ? nullptr : cu;
    p.n_seqs = n_seqs;
    p.T = T;
    p.H = H;
    p.group = H / Hkv;
    p.dk = d_k; p.dv = d_v;
    p.scale = scale;
    p.init = init;
    p.out = out;
    p.final_state = final_state;
    p.seg_len = lin::plan_segments(n_seqs, T, H, d_k, d_v, dtype);
    const int64_t items = p.seg_len ? T / p.seg_len + n_seqs : n_seqs;
    if (items * H > 0x7fffffffLL || (int64_t)n_seqs * H > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED_SHAPE;
    p.items = (int)items;
    p.starts = static_cast<float *>(workspace);
    p.decays = p.starts ? p.starts + items * H * d_k * d_v : nullptr;
    if (lin::tc_path(d_k, d_v, dtype) && T > 0) return lin::run_tc_path(p, out_dtype, stream);
    return lin::run_token_path(p, dtype, out_dtype, stream);
}

}  // namespace kda
