// kda_delta.cu -- the gated delta rule with one decay per head on CUDA cores: fp32 inputs and head sizes that the
// tensor-core kernel does not take.
//
//     S' = exp(g_t) S_(t-1),   S_t = S' + beta_t k_t (v_t - S'^T k_t)^T,   o_t = scale S_t^T q_t
//
// A block owns 64 value columns of one (sequence, head), or 32: a thread holds 8 key channels x 2 columns (or 1) of
// the state in registers, warp w the channels [8 w, 8 w + 8).  Eight tokens (i, j) are taken at a time (four where d_k is
// over 128).  With w_ij = exp(g_(j+1) + .. + g_i), G_i = g_1 + .. + g_i and S the state before them,
//     u_i = beta_i (v_i - e^(G_i) S^T k_i - sum_(j < i) w_ij (k_i . k_j) u_j)
//     o_i = scale (e^(G_i) S^T q_i + sum_(j <= i) w_ij (q_i . k_j) u_j)
//     S  <- e^(G_8) S + sum_j k_j (e^(G_8 - G_j) u_j)^T
// so that the sums over all key channels, which have to cross the warps, are taken for eight tokens at once, and
// what follows token after token is a small substitution.  Products of decays are exponentials of their own sums
// of log decays; the state's is taken as 1 + expm1 where it is near 1: rounded to fp32 itself, a decay that stays
// the same would be off the same way block after block (over 256 tokens of memory 1e-6 of the state).
// Bound by latency: a block of tokens is five steps with a barrier after each (staging, scores and the products with
// the state, sums, substitution, outputs and update), some 3700 cycles for 64 x 32 of a state and 130 of FMA a
// scheduler for the update.  2560 tokens in two sequences, 16 heads of 64 x 128: 0.50 ms (token by token, with
// the sums folded inside a warp, 0.88; 64 columns a block 0.55).
#include "kda_delta.cuh"

namespace kda {
namespace delta {
namespace {

constexpr int kRows = 8;     // key channels of a warp

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ uint2 load4(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint2 *>(p); }
__device__ __forceinline__ float4 widen(float4 x) { return x; }
__device__ __forceinline__ float4 widen(uint2 x)
{
    return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                       __uint_as_float(x.y & 0xffff0000u));
}

// tokens at a time
template <int WARPS>
constexpr int kTokens = WARPS <= 16 ? 8 : 4;

template <typename T, typename TO, int WARPS, int CPL>
__global__ void __launch_bounds__(32 * WARPS) delta_token_kernel(const Args p)
{
    constexpr int THREADS = 32 * WARPS, DK = kRows * WARPS, TB = kTokens<WARPS>, kCols = 32 * CPL;
    constexpr int KUNITS = TB * DK / 4, VUNITS = TB * kCols / 4;
    constexpr int KU = (KUNITS + THREADS - 1) / THREADS;
    constexpr int DP = DK + 4;                        // padded rows: the score threads walk several at once
    constexpr int SUB = THREADS / (TB * TB) < 32 ? THREADS / (TB * TB) : 32;   // threads of a score
    using Four = decltype(load4((const T *)nullptr));
    extern __shared__ __align__(16) float parts[];    // [2][TB][WARPS][kCols]: S^T k, S^T q of a warp's channels
    __shared__ __align__(16) float sk[TB][DP], sq[TB][DP];
    __shared__ __align__(16) float sv[TB][kCols], su[TB][kCols];
    struct Decays {
        float g[TB], beta[TB], pre[TB], suf[TB];      // log decays, beta, e^G, e^(G_last - G)
        float all, one;                               // the whole block's decay (see above)
    };
    __shared__ Decays sd[2];                          // this block's and the next one's
    __shared__ float sa[TB][TB + 1], sp[TB][TB + 1];  // beta w (k . k), w (q . k)
    constexpr int DEC = 2;                            // the warp that makes the decays, while others substitute
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int seq = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / p.group, Hk = p.H / p.group;
    const int cb = blockIdx.y * kCols, col = cb + lane;
    auto part = [&](int which, int t, int w) { return parts + ((which * TB + t) * WARPS + w) * kCols; };
    long long b, e;
    bounds(p, seq, b, e);
    const long long own = ((long long)seq * p.H + h) * p.dk * p.dv;
    float st[kRows][CPL];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            const int i = warp * kRows + r;
            st[r][c] = p.init && col + 32 * c < p.dv && i < p.dk ? p.init[own + (long long)i * p.dv + col + 32 * c] : 0.f;
        }
    const T *q = static_cast<const T *>(p.q), *k = static_cast<const T *>(p.k), *v = static_cast<const T *>(p.v);
    Four nk[KU], nq[KU], nv;
    float ng = 0.f, nb = 0.f;
    auto fetch = [&](long long tb) {
        const Four zero = {};
#pragma unroll
        for (int u = 0; u < KU; ++u) {
            const int x = tid + u * THREADS, t = x / (DK / 4), i = x % (DK / 4) * 4;
            const bool ok = x < KUNITS && tb + t < e && i < p.dk;
            nk[u] = ok ? load4(k + ((tb + t) * Hk + hk) * p.dk + i) : zero;
            nq[u] = ok ? load4(q + ((tb + t) * Hk + hk) * p.dk + i) : zero;
        }
        {
            const int t = tid / (kCols / 4), c = cb + tid % (kCols / 4) * 4;
            nv = tid < VUNITS && tb + t < e && c < p.dv ? load4(v + ((tb + t) * p.H + h) * p.dv + c) : zero;
        }
        if (warp == DEC && lane < TB) {   // (tokens past the end neither decay nor write)
            const bool ok = tb + lane < e;
            ng = ok ? p.g[p.g_per_token ? (tb + lane) * p.H + h : h] : 0.f;
            nb = ok ? p.beta[(tb + lane) * p.H + h] : 0.f;
        }
    };
    auto decays = [&](Decays &to) {   // (lanes from TB on hold 0, the sums that reach past the block stay in it)
        float after = ng, before = ng;
#pragma unroll
        for (int o = 1; o < TB; o <<= 1) {
            after += __shfl_down_sync(0xffffffffu, after, o);
            const float x = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += x;
        }
        const float rest = __shfl_down_sync(0xffffffffu, after, 1);
        if (lane < TB) {
            to.g[lane] = ng;
            to.beta[lane] = nb;
            to.pre[lane] = expf(before);
            to.suf[lane] = expf(rest);   // (of the last: of nothing)
        }
        if (lane == 0) {
            const bool near = after > -0.25f;
            to.all = near ? expm1f(after) : expf(after);
            to.one = near ? 1.f : 0.f;
        }
    };
    int cur = 0;
    if (b < e) {
        fetch(b);
        if (warp == DEC) decays(sd[0]);
    }
    for (long long tb = b; tb < e; tb += TB, cur ^= 1) {
        const int n = (int)min((long long)TB, e - tb);
#pragma unroll
        for (int u = 0; u < KU; ++u) {
            const int x = tid + u * THREADS;
            if (x < KUNITS) {
                *reinterpret_cast<float4 *>(&sk[x / (DK / 4)][x % (DK / 4) * 4]) = widen(nk[u]);
                *reinterpret_cast<float4 *>(&sq[x / (DK / 4)][x % (DK / 4) * 4]) = widen(nq[u]);
            }
        }
        if (tid < VUNITS) *reinterpret_cast<float4 *>(&sv[0][0] + 4 * tid) = widen(nv);
        const Decays &d = sd[cur];
        __syncthreads();
        if (tb + TB < e) fetch(tb + TB);
        if (tid < TB * TB * SUB) {   // scores
            const int i = tid / SUB / TB, j = tid / SUB % TB;
            float kk = 0.f, qk = 0.f;
#pragma unroll 4
            for (int x = tid % SUB * 4; x < DK; x += 4 * SUB) {
                const float4 a = *reinterpret_cast<const float4 *>(&sk[j][x]);
                const float4 c = *reinterpret_cast<const float4 *>(&sk[i][x]);
                const float4 f = *reinterpret_cast<const float4 *>(&sq[i][x]);
                kk += a.x * c.x + a.y * c.y + a.z * c.z + a.w * c.w;
                qk += a.x * f.x + a.y * f.y + a.z * f.z + a.w * f.w;
            }
#pragma unroll
            for (int o = SUB / 2; o > 0; o >>= 1) {
                kk += __shfl_xor_sync(0xffffffffu, kk, o);
                qk += __shfl_xor_sync(0xffffffffu, qk, o);
            }
            float w = 0.f;
#pragma unroll
            for (int l = 1; l < TB; ++l) w += l > j && l <= i ? d.g[l] : 0.f;
            w = expf(w);
            if (tid % SUB == 0) {
                sa[i][j] = d.beta[i] * w * kk;
                sp[i][j] = w * qk;
            }
        }
#pragma unroll 4
        for (int t = 0; t < TB; ++t) {   // S^T k, S^T q over the warp's channels
            float ak[CPL] = {}, aq[CPL] = {};
#pragma unroll
            for (int r = 0; r < kRows; r += 4) {
                const float4 kr = *reinterpret_cast<const float4 *>(&sk[t][warp * kRows + r]);
                const float4 qr = *reinterpret_cast<const float4 *>(&sq[t][warp * kRows + r]);
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    ak[c] = fmaf(st[r + 3][c], kr.w, fmaf(st[r + 2][c], kr.z, fmaf(st[r + 1][c], kr.y, fmaf(st[r][c], kr.x, ak[c]))));
                    aq[c] = fmaf(st[r + 3][c], qr.w, fmaf(st[r + 2][c], qr.z, fmaf(st[r + 1][c], qr.y, fmaf(st[r][c], qr.x, aq[c]))));
                }
            }
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                part(0, t, warp)[lane + 32 * c] = ak[c];
                part(1, t, warp)[lane + 32 * c] = aq[c];
            }
        }
        __syncthreads();
#pragma unroll
        for (int x0 = 0; x0 < 2 * TB * kCols; x0 += THREADS) {   // over all of them: R, and what outputs take from S
            const int x = x0 + tid, t = x / kCols % TB, c = x % kCols, which = x / (TB * kCols);
            if (x >= 2 * TB * kCols) break;
            float *from = part(which, t, 0) + c, sum = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) sum += from[w * kCols];
            from[0] = which ? d.pre[t] * sum : d.beta[t] * fmaf(-d.pre[t], sum, sv[t][c]);
        }
        __syncthreads();
        if (tid < kCols) {   // a column's substitution
            float u[TB];
#pragma unroll
            for (int i = 0; i < TB; ++i) u[i] = part(0, i, 0)[tid];
#pragma unroll
            for (int j = 0; j < TB; ++j)
#pragma unroll
                for (int i = j + 1; i < TB; ++i) u[i] = fmaf(-sa[i][j], u[j], u[i]);
#pragma unroll
            for (int i = 0; i < TB; ++i) su[i][tid] = u[i];
        }
        if (warp == DEC && tb + TB < e) decays(sd[cur ^ 1]);
        __syncthreads();
        for (int x = tid; x < n * kCols; x += THREADS) {
            const int i = x / kCols, c = x % kCols;
            float o = part(1, i, 0)[c];
#pragma unroll
            for (int j = 0; j < TB; ++j)
                if (j <= i) o = fmaf(sp[i][j], su[j][c], o);
            if (cb + c < p.dv) store_as(static_cast<TO *>(p.out) + ((tb + i) * p.H + h) * p.dv + cb + c, o * p.scale);
        }
        const float all = d.all, one = d.one;
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int c = 0; c < CPL; ++c) st[r][c] = fmaf(st[r][c], all, st[r][c] * one);
#pragma unroll 4
        for (int t = 0; t < TB; ++t) {
            const float f = d.suf[t];
            float u[CPL];
#pragma unroll
            for (int c = 0; c < CPL; ++c) u[c] = f * su[t][lane + 32 * c];
#pragma unroll
            for (int r = 0; r < kRows; r += 4) {
                const float4 kr = *reinterpret_cast<const float4 *>(&sk[t][warp * kRows + r]);
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    st[r][c] = fmaf(kr.x, u[c], st[r][c]);
                    st[r + 1][c] = fmaf(kr.y, u[c], st[r + 1][c]);
                    st[r + 2][c] = fmaf(kr.z, u[c], st[r + 2][c]);
                    st[r + 3][c] = fmaf(kr.w, u[c], st[r + 3][c]);
                }
            }
        }
        __syncthreads();
    }
    if (p.final_state) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                const int i = warp * kRows + r;
                if (i < p.dk && col + 32 * c < p.dv) p.final_state[own + (long long)i * p.dv + col + 32 * c] = st[r][c];
            }
    }
}

template <typename T, typename TO, int WARPS, int CPL>
int launch_cols(const Args &p, cudaStream_t stream)
{
    constexpr int bytes = 2 * kTokens<WARPS> * WARPS * 32 * CPL * 4;
    // a function attribute belongs to the current device: set it on every launch
    if (cudaFuncSetAttribute(delta_token_kernel<T, TO, WARPS, CPL>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
        cudaSuccess)
        return KDA_ERR_CUDA;
    const dim3 grid((unsigned)(p.n_seqs * p.H), (unsigned)ceil_div(p.dv, 32 * CPL));
    delta_token_kernel<T, TO, WARPS, CPL><<<grid, 32 * WARPS, bytes, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <typename T, typename TO, int WARPS>
int launch_warps(const Args &p, cudaStream_t stream)
{
    // 32 columns a block where 64 would leave SMs idle
    if ((long long)p.n_seqs * p.H * ceil_div(p.dv, 64) < 152) return launch_cols<T, TO, WARPS, 1>(p, stream);
    return launch_cols<T, TO, WARPS, 2>(p, stream);
}

template <typename T, typename TO>
int launch(const Args &p, cudaStream_t stream)
{
    if (p.dk <= 64) return launch_warps<T, TO, 8>(p, stream);
    if (p.dk <= 128) return launch_warps<T, TO, 16>(p, stream);
    return launch_warps<T, TO, 32>(p, stream);
}

}  // namespace

int run_token_path(const Args &p, int dtype, int out_dtype, cudaStream_t stream)
{
    if (dtype == KDA_BF16)
        return out_dtype == KDA_BF16 ? launch<__nv_bfloat16, __nv_bfloat16>(p, stream) : launch<__nv_bfloat16, float>(p, stream);
    return out_dtype == KDA_BF16 ? launch<float, __nv_bfloat16>(p, stream) : launch<float, float>(p, stream);
}

// Whether the tensor-core kernel takes these operands: from a mean length on at which it is the faster (us, here and
// there, with initial states: 32 heads of 128 x 128, one sequence of 16 tokens 7.6, 14.0, of 32 12.5, 13.6, of 64 22.6,
// 12.8; 16 sequences of 8 36, 55, of 16 59, 55; 16 heads of 64 x 64, one of 64 16.2, 10.7, 16 of 32 15.8, 23.0).
bool tc_path(int n_seqs, int64_t T, int d_k, int d_v, int dtype)
{
    return dtype == KDA_BF16 && d_k <= 128 && d_v <= 128 && T >= (d_k <= 64 ? 48 : 16) * (int64_t)n_seqs;
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
    p.cu = cu;
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
