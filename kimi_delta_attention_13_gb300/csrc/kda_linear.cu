// kda_linear.cu -- linear attention with one decay per head, token by token on CUDA cores, and
// the join of segments.
//
//     S_t = exp(g_t) S_(t-1) + k_t v_t^T,     o_t = scale S_t^T q_t
//
// This is the path for fp32 inputs and for head sizes the tensor-core kernel does not take.  A
// block owns 128 value columns of one (segment, head): a thread holds 16 key channels x 4 columns of
// the state in registers, warp w the channels [16 w, 16 w + 16), lane l the columns 4 l .. 4 l + 3.
// Eight tokens (i, j) are taken at a time.  With a_t = exp(g_t) and S the state before them,
//     o_i = scale ( (prod_(l <= i) a_l) S^T q_i + sum_(j <= i) (prod_(j < l <= i) a_l) (q_i . k_j) v_j )
//     S  <- (prod a) S + sum_j k_j (prod_(l > j) a_l v_j)^T
// Every product of decays is the exponential of its own sum of log decays: a product of rounded factors is
// off by their roundings, which for a constant decay are all alike (over a memory of 256 tokens 3e-6,
// against 5e-7).  An element of the state costs one fused multiply-add a token for the read and one for
// the update, two rows an instruction (decaying it token by token would cost a multiply more).  Key and
// query rows come from shared memory as broadcasts; the next tokens' loads are in flight meanwhile.
// Bound by the FMA pipe: 2 d_k d_v operations a token and head, 1 in the pass for states alone; the
// pipe is busy for half of the time (2560 tokens in two sequences, 16 heads of 64 x 128: 55 us the
// outputs, 26 us the states, 10 us the join; token by token with the decay 131 us in all).  A block has
// its 128 columns and a warp its 16 channels whatever the head's size: 64 x 64 takes 87 us, 64 x
// 128 88, 32 x 32 still 85.  bf16 heads over 128 come here too: 8192 tokens, 16 heads of 128 x 256 0.89 ms,
// 256 x 128 1.10, 256 x 256 2.8, where the tensor-core kernel takes 0.078 for 128 x 128.
//
// Long sequences are cut into segments worked on side by side: linear_token_kernel<.., false>
// leaves the end state of every segment but a sequence's last (from zeros; a first segment from
// the initial state), linear_join_kernel turns those into the segments' true start states, and
// linear_token_kernel<.., true> computes the outputs.
#include "kda_linear.cuh"

namespace kda {
namespace lin {
namespace {

constexpr int kCols = 128;   // value columns of a block
constexpr int kRows = 16;    // key channels of a warp

__device__ __forceinline__ float2 pair_fma(float2 a, float2 b, float2 c)
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
__device__ __forceinline__ float2 pair_mul(float2 a, float2 b)
{
    unsigned long long r, x, y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}

// 4 consecutive elements as fp32
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p)
{
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}

__device__ __forceinline__ void store4(float *p, const float (&f)[4])
{
    *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&f)[4])
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

template <typename T, typename TO, int WARPS, bool OUT>
__global__ void __launch_bounds__(32 * WARPS) linear_token_kernel(const Args p)
{
    constexpr int THREADS = 32 * WARPS, DK = kRows * WARPS;
    constexpr int TB = WARPS <= 8 ? 8 : 4;   // tokens staged at a time
    constexpr int KUNITS = TB * DK / 4, VUNITS = TB * kCols / 4;
    constexpr int KU = (KUNITS + THREADS - 1) / THREADS, VU = (VUNITS + THREADS - 1) / THREADS;
    constexpr int DP = DK + 4;               // padded rows: the score threads walk several at once
    constexpr int SUB = THREADS / (TB * TB); // threads of a score
    __shared__ __align__(16) float sk[TB][DP];
    __shared__ __align__(16) float sq[OUT ? TB : 1][DP];
    __shared__ __align__(16) float sv[TB][kCols];
    __shared__ float sg[TB];                 // log decays
    __shared__ float sa[TB + 1];             // the decays after a token in the block; then those of all
    __shared__ float sall;                   // the sum of the block's log decays
    __shared__ float sw[TB][TB + 1];         // a score's weight times the score; then the prefix of i
    __shared__ __align__(16) float part[OUT ? TB : 1][WARPS][kCols];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % p.H, item = blockIdx.x / p.H, hk = h / p.group, Hkv = p.H / p.group;
    const int cb = blockIdx.y * kCols, col = cb + 4 * lane;
    const bool col_ok = col < p.dv;
    const Item it = find_item(p.cu, p.n_seqs, p.T, p.seg_len, item);
    if (it.seq < 0 || (!OUT && (it.seg == it.nseg - 1 || item + 1 >= p.items))) return;   // (a bad table
    // could name more segments than there are places for)

    const long long unit = (long long)p.dk * p.dv;
    const long long own = ((long long)it.seq * p.H + h) * unit, slot = ((long long)item * p.H + h) * unit;
    const float *from = nullptr;
    if (it.seg == 0) from = p.init ? p.init + own : nullptr;
    if (OUT && it.nseg > 1 && (it.seg > 0 || p.init)) from = p.starts + slot;
    float2 st[kRows / 2][4];   // rows 2 r, 2 r + 1 of the warp's; column 4 lane + c
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int i = warp * kRows + r;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (from && col_ok && i < p.dk) s = *reinterpret_cast<const float4 *>(from + (long long)i * p.dv + col);
        // a first segment's start is kept: the last segment may overwrite it (final_state = init)
        if (!OUT && it.seg == 0 && p.init && col_ok && i < p.dk)
            *reinterpret_cast<float4 *>(p.starts + slot + (long long)i * p.dv + col) = s;
        const float e[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (r & 1) st[r / 2][c].y = e[c];
            else st[r / 2][c].x = e[c];
        }
    }
    const T *q = static_cast<const T *>(p.q), *k = static_cast<const T *>(p.k), *v = static_cast<const T *>(p.v);
    float4 nk[KU], nq[OUT ? KU : 1], nv[VU];
    float ng = 0.f;
    auto fetch = [&](long long tb) {
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < KU; ++u) {
            const int e = tid + u * THREADS, t = e / (DK / 4), i = e % (DK / 4) * 4;
            const bool ok = e < KUNITS && tb + t < it.t1 && i < p.dk;
            nk[u] = ok ? load4(k + ((tb + t) * Hkv + hk) * p.dk + i) : zero;
            if constexpr (OUT) nq[u] = ok ? load4(q + ((tb + t) * p.H + h) * p.dk + i) : zero;
        }
#pragma unroll
        for (int u = 0; u < VU; ++u) {
            const int e = tid + u * THREADS, t = e / (kCols / 4), c = cb + e % (kCols / 4) * 4;
            nv[u] = e < VUNITS && tb + t < it.t1 && c < p.dv ? load4(v + ((tb + t) * Hkv + hk) * p.dv + c) : zero;
        }
        if (tid < TB) ng = tb + tid < it.t1 ? (p.g_per_token ? p.g[(tb + tid) * p.H + h] : p.g[h]) : 0.f;
    };
    float whole = 0.f;                       // sum of the segment's log decays
    if (it.t0 < it.t1) fetch(it.t0);
    for (long long tb = it.t0; tb < it.t1; tb += TB) {
        const int n = (int)min((long long)TB, it.t1 - tb);
#pragma unroll
        for (int u = 0; u < KU; ++u) {
            const int e = tid + u * THREADS;
            if (e < KUNITS) {
                *reinterpret_cast<float4 *>(&sk[e / (DK / 4)][e % (DK / 4) * 4]) = nk[u];
                if constexpr (OUT) *reinterpret_cast<float4 *>(&sq[e / (DK / 4)][e % (DK / 4) * 4]) = nq[u];
            }
        }
#pragma unroll
        for (int u = 0; u < VU; ++u)
            if (tid + u * THREADS < VUNITS) *reinterpret_cast<float4 *>(&sv[0][0] + 4 * (tid + u * THREADS)) = nv[u];
        if (warp == 0) {   // (lanes from TB on hold 0, the sums that reach past the block stay in it)
            float after = ng;
#pragma unroll
            for (int o = 1; o < TB; o <<= 1) after += __shfl_down_sync(0xffffffffu, after, o);
            const float rest = __shfl_down_sync(0xffffffffu, after, 1);
            if (lane < TB) {
                sg[lane] = ng;
                sa[lane] = expf(rest);       // (lane TB - 1: of nothing)
            }
            if (lane == 0) {
                sa[TB] = expf(after);
                sall = after;
            }
        }
        __syncthreads();
        if (tb + TB < it.t1) fetch(tb + TB);
        if constexpr (OUT) {
            {   // scores within the block
                const int pair = tid / SUB, i = pair / TB, j = pair % TB;
                float sum = 0.f;
#pragma unroll 4
                for (int x = tid % SUB * 4; x < DK; x += 4 * SUB) {
                    const float4 kr = *reinterpret_cast<const float4 *>(&sk[j][x]);
                    const float4 qr = *reinterpret_cast<const float4 *>(&sq[i][x]);
                    sum += kr.x * qr.x + kr.y * qr.y + kr.z * qr.z + kr.w * qr.w;
                }
#pragma unroll
                for (int o = SUB / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                float w = 0.f;
                for (int l = i; l > j; --l) w += sg[l];
                if (tid % SUB == 0 && j <= i) {
                    sw[i][j] = sum * expf(w);
                    if (j == 0) sw[i][TB] = expf(w + sg[0]);
                }
            }
#pragma unroll 1
            for (int t = 0; t < n; ++t) {
                float2 acc[4] = {};
#pragma unroll
                for (int r = 0; r < kRows / 4; ++r) {
                    const float4 qr = *reinterpret_cast<const float4 *>(&sq[t][warp * kRows + 4 * r]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        acc[c] = pair_fma(st[2 * r][c], make_float2(qr.x, qr.y), acc[c]);
                        acc[c] = pair_fma(st[2 * r + 1][c], make_float2(qr.z, qr.w), acc[c]);
                    }
                }
                *reinterpret_cast<float4 *>(&part[t][warp][4 * lane]) =
                    make_float4(acc[0].x + acc[0].y, acc[1].x + acc[1].y, acc[2].x + acc[2].y, acc[3].x + acc[3].y);
            }
        }
        const float all = sa[TB];   // (tokens past the segment's end do not decay)
        if constexpr (!OUT) whole += sall;
#pragma unroll
        for (int r = 0; r < kRows / 2; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) st[r][c] = pair_mul(st[r][c], make_float2(all, all));
#pragma unroll 1
        for (int t = n - 1; t >= 0; --t) {
            const float4 x = *reinterpret_cast<const float4 *>(&sv[t][4 * lane]);
            const float suf = sa[t];
            const float xs[4] = {x.x * suf, x.y * suf, x.z * suf, x.w * suf};
#pragma unroll
            for (int r = 0; r < kRows / 4; ++r) {
                const float4 kr = *reinterpret_cast<const float4 *>(&sk[t][warp * kRows + 4 * r]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 xx = make_float2(xs[c], xs[c]);
                    st[2 * r][c] = pair_fma(make_float2(kr.x, kr.y), xx, st[2 * r][c]);
                    st[2 * r + 1][c] = pair_fma(make_float2(kr.z, kr.w), xx, st[2 * r + 1][c]);
                }
            }
        }
        __syncthreads();
        if constexpr (OUT) {
            for (int e = tid; e < n * (kCols / 4); e += THREADS) {
                const int t = e / (kCols / 4), c = e % (kCols / 4) * 4;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    const float4 x = *reinterpret_cast<const float4 *>(&part[t][w][c]);
                    acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
                }
                const float pre = sw[t][TB];
                acc.x *= pre; acc.y *= pre; acc.z *= pre; acc.w *= pre;
#pragma unroll
                for (int j = 0; j < TB; ++j) {
                    if (j > t) break;
                    const float4 x = *reinterpret_cast<const float4 *>(&sv[j][c]);
                    const float f = sw[t][j];
                    acc.x = fmaf(f, x.x, acc.x); acc.y = fmaf(f, x.y, acc.y);
                    acc.z = fmaf(f, x.z, acc.z); acc.w = fmaf(f, x.w, acc.w);
                }
                if (cb + c < p.dv) {
                    TO *o = static_cast<TO *>(p.out) + ((tb + t) * p.H + h) * p.dv + cb + c;
                    const float f[4] = {acc.x * p.scale, acc.y * p.scale, acc.z * p.scale, acc.w * p.scale};
                    store4(o, f);
                }
            }
            __syncthreads();
        }
    }
    // OUT: the last segment leaves the sequence's final state.  Otherwise the end state from zeros
    // goes to the next segment's place, and the segment's decay to its own.
    float *to = nullptr;
    if (OUT) to = it.seg == it.nseg - 1 && p.final_state ? p.final_state + own : nullptr;
    else to = p.starts + slot + (long long)p.H * unit;
    if (to && col_ok) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int i = warp * kRows + r;
            const float2 *s = st[r / 2];
            if (i < p.dk)
                *reinterpret_cast<float4 *>(to + (long long)i * p.dv + col) =
                    r & 1 ? make_float4(s[0].y, s[1].y, s[2].y, s[3].y) : make_float4(s[0].x, s[1].x, s[2].x, s[3].x);
        }
    }
    if (!OUT && tid == 0 && blockIdx.y == 0) p.decays[(long long)item * p.H + h] = expf(whole);
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
    constexpr int AHEAD = 8;   // segments whose loads are in flight
    for (int j0 = 1; j0 < nseg - 1; j0 += AHEAD) {
        float f[AHEAD];
        float4 d[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int j = min(j0 + i, nseg - 2);
            f[i] = a[(long long)j * p.H];
            d[i] = s[(j + 1) * step];
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (j0 + i >= nseg - 1) break;
            cur = make_float4(fmaf(f[i], cur.x, d[i].x), fmaf(f[i], cur.y, d[i].y), fmaf(f[i], cur.z, d[i].z),
                              fmaf(f[i], cur.w, d[i].w));
            s[(j0 + i + 1) * step] = cur;
        }
    }
}

template <typename T, typename TO, bool OUT>
void launch_tokens(const Args &p, cudaStream_t stream)
{
    const dim3 grid((unsigned)(p.items * p.H), (unsigned)ceil_div(p.dv, kCols));
    if (p.dk <= 64) linear_token_kernel<T, TO, 4, OUT><<<grid, 128, 0, stream>>>(p);
    else if (p.dk <= 128) linear_token_kernel<T, TO, 8, OUT><<<grid, 256, 0, stream>>>(p);
    else linear_token_kernel<T, TO, 16, OUT><<<grid, 512, 0, stream>>>(p);
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

// Tokens of a segment, 0 where the sequences are not cut.
//
// Tensor-core kernel: the cut sequences give at most one block an SM, and are taken where they are the
// faster for sequences of one length, by a fit to measured times (us): 8 + 3 a chunk of an uncut sequence,
// 17 + 5.5 a chunk of a segment (two passes and the join).  T x H cut, uncut, in a graph: 512 x 8 22.8, 19.4;
// 640 x 8 22.9, 22.5; 768 x 8 23.3, 25.6; 65536 x 8 169, 1512; 1400 x 32 33, 42; 8192 x 32 107, 201; 2048 x 64
// 65, 58; 4096 x 64 106, 108; four of 2048 x 8 45, 57; eight of 2048 x 8 80, 57.
// The lengths are on the device, so the mean stands for the longest: a long sequence among short ones stays
// whole (65,536 tokens with 8 short sequences, 8 heads: 1517 where it alone takes 181; 32,768 with one of
// 232, 32 heads: 784 where it alone takes 368).  Such prompts are faster in a call of their own.
// Token kernel: cut to 16 warps an SM where there are less (2560 tokens, 16 heads: 64 x 128 in blocks of
// four warps 85, 78, 91 us at 8, 16, 32 warps; 128 x 128 in blocks of eight 135 us at 16, 149 at 32).
int plan_segments(int n_seqs, int64_t T, int H, int d_k, int d_v, int dtype)
{
    if (tc_path(d_k, d_v, dtype)) {
        const int64_t ctas = (int64_t)n_seqs * H, sms = 152;
        if (ctas == 0 || ctas > sms / 2 || T == 0) return 0;
        const int64_t per = sms / H;   // segments of one sequence
        const int64_t len = ((n_seqs == 1 ? (T + per - 1) / per : T * H / (sms - ctas)) + 127) / 128 * 128;
        return 34 + 11 * (len / 128) < 16 + 6 * (T / n_seqs / 128) ? (int)len : 0;
    }
    const int64_t slices = ceil_div(d_v, kCols), blocks = (int64_t)n_seqs * H * slices;
    const int64_t want = d_k <= 64 ? 152 * 4 : d_k <= 128 ? 152 * 2 : 152;   // 16 warps an SM
    if (blocks >= want) return 0;
    int64_t len = (T * H * slices / want + 7) / 8 * 8;
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
