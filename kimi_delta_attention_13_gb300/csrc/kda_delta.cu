// kda_delta.cu -- the gated delta rule with one decay per head for fp32 inputs, head sizes that kda_delta_tc.cu does
// not take, and short sequences.
//
//     S' = exp(g_t) S_(t-1),   S_t = S' + beta_t k_t (v_t - S'^T k_t)^T,   o_t = scale S_t^T q_t
//
// Eight tokens (i, j) are taken at a time.  With w_ij = exp(g_(j+1) + .. + g_i), G_i = g_1 + .. + g_i, S the state before
// them, A_ij = beta_i w_ij (k_i . k_j) for j < i and M = (I + A)^-1 diag(beta),
//     U  = M R,   r_i = v_i - e^(G_i) S^T k_i
//     o_i = scale (e^(G_i) S^T q_i + sum_(j <= i) w_ij (q_i . k_j) u_j)
//     S  <- e^(G_8) S + sum_j k_j (e^(G_8 - G_j) u_j)^T
// Products of decays are exponentials of their own sums of log decays; the state's is taken as 1 + expm1 where it is near
// 1: rounded to fp32 itself, a decay that stays the same would be off the same way block after block (over 256 tokens of
// memory 1e-6 of the state).
//
// A block owns 64 value columns of one (sequence, head).  Four warps are the chain: a warp holds S^T for 16 columns in
// registers, as the accumulators of [16 columns x 8 channels] products of mma.sync, whose layout is also that of
// the operands which S^T k, S^T q, M R and the update take, so that nothing crosses lanes.  A factor is three bf16 parts
// (two side by side along k where that is only eight tokens long); of the nine products of two factors the three smallest,
// 2^-24 of the whole, are left out; a bf16 input is one part.  A warp's CUDA cores would take 768 cycles of FMA for
// eight tokens of 16 columns x 64 channels, and each of their operands from shared memory: the 78 products take 640.
// Four warps load four blocks ahead, make the parts and, three ahead, the scores, each for a quarter of the channels; a
// warp each makes the decays, the scores' sums and weights, and M, a thread a column, one block ahead.  A barrier of these
// eleven warps ends a block.  Registers are moved to the chain.  (tcgen05's 64-token chunks, kda_delta_tc.cu, would need k
// and q in three parts in shared memory as well.)
//
// Bound by the chain's latency, one warp a scheduler: some 1,400 cycles of the 1,650 that a block of tokens takes, the
// other warps' instructions between them.  2560 tokens in two sequences, 16 heads of 64 x 128, fp32: 215 us.  Before, on
// CUDA cores with a barrier between the steps: 454; sums over lanes in place of shared memory: 372, bound by shared
// memory's 128 bytes a cycle; all but the chain in four warps: 285; decays and M in one warp: 250; scores by fp32 FMA: 233;
// q's products behind the new values, outputs a block later or before the update, the state's decay earlier, a block
// an SM with more registers: no gain.  2048 tokens of 96 heads of 128 x 128 0.67 ms (1.58 before), of 16 heads of 256 x 256 in
// bf16 0.45 (1.20).  Above 128 channels the chain spills: 128 accumulators a thread and the parts of products leave 324 (bf16
// operands) to 360 bytes (fp32) of a thread's values in local memory.
#include "kda_delta.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace delta {
namespace {

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ uint2 load4(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint2 *>(p); }
__device__ __forceinline__ float4 widen(float4 x) { return x; }
__device__ __forceinline__ float4 widen(uint2 x)
{
    return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                       __uint_as_float(x.y & 0xffff0000u));
}

constexpr int TB = 8;        // tokens at a time
constexpr int kChain = 4;    // warps that hold the state, 16 value columns each
constexpr int kMakers = 4;   // warps that make what does not depend on it
constexpr int COLS = 16 * kChain;
constexpr int kThreads = 32 * (kChain + kMakers + 4);   // and a warpgroup of which three warps work

// Registers a thread: at launch, then of each warpgroup (their sum may not pass the block's)
template <int DK>
constexpr int kRegs[4] = {DK == 64 ? 80 : 168, DK == 64 ? 144 : 240, DK == 64 ? 56 : 160, DK == 64 ? 40 : 104};
static_assert(kRegs<64>[1] + kRegs<64>[2] + kRegs<64>[3] <= 3 * kRegs<64>[0] && kRegs<128>[1] + kRegs<128>[2] + kRegs<128>[3] <= 3 * kRegs<128>[0], "");
template <int LAUNCH, int N>
__device__ __forceinline__ void set_regs()
{
    if constexpr (N > LAUNCH) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// what a block of tokens is worked from: staged, scored, weighted, solved and used in five periods
template <int DK, int PARTS>
struct __align__(16) Stage {
    uint16_t k[PARTS][TB][DK + 8], q[PARTS][TB][DK + 8];   // bf16 parts (rows padded against bank conflicts)
    float v[TB][COLS + 4];
    float a[TB][12], m[TB][12], p[TB][12];     // beta w (k . k);  (I + a)^-1 diag(beta);  w (q . k)
    float w[TB][TB];                           // for j <= i
    float beta[TB], pre[TB], suf[TB];          // beta, e^G, e^(G_last - G)
    float all, near, unused[2];                // the whole block's decay, less 1 where it is near 1
};
constexpr int kStages = 5;
struct Scores {
    float sum[kMakers][2 * TB][TB];            // a maker's channels' part of k . k, then of q . k
};

// x, y as three packed pairs of bf16, which sum to them
__device__ __forceinline__ void split(float x, float y, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    float2 r = make_float2(x, y);
    hi = ptx::pack_bf16x2(r.x, r.y);
    rest(hi, r);
    mid = ptx::pack_bf16x2(r.x, r.y);
    rest(mid, r);
    mid ^= 0x80008000u;
    lo = ptx::pack_bf16x2(r.x, r.y);
}

// c [16 x 8] += a [16 x 16] b [16 x 8]; lane l = 4 x + y has of c the rows x, x + 8 and columns 2 y, 2 y + 1; of a the
// same rows at k = 2 y, + 1, then at k + 8; of b column x at k = 2 y, + 1, then at k + 8
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// four tiles of 8 tokens x 8 channels: element (token x, channels 2 y, + 1), or (tokens 2 y, + 1, channel x)
__device__ __forceinline__ void tiles(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void tiles_trans(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

// c += x y over 8 tokens, x [16 x 8] and y [8 x 8] in three parts: two parts of x side by side in k
__device__ __forceinline__ void mma_tokens(float (&c)[4], float (&small)[4], const uint32_t (&x)[3][2], const uint32_t (&y)[3])
{
    mma(c, x[0][0], x[0][1], x[1][0], x[1][1], y[0], y[0]);
    mma(small, x[0][0], x[0][1], x[1][0], x[1][1], y[1], y[1]);
    mma(small, x[0][0], x[0][1], x[2][0], x[2][1], y[2], y[0]);
}

template <typename T, typename TO, int DK>
__global__ void __launch_bounds__(kThreads, DK == 64 ? 2 : 1) delta_token_kernel(const Args p)
{
    constexpr int PARTS = sizeof(T) == 4 ? 3 : 1, MT = 32 * kMakers;
    constexpr int KU = TB * DK / 4 / MT, PITCH = (DK + 8) * 2;
    static_assert(TB * DK / 4 % MT == 0 && TB * COLS / 4 == MT && DK / 16 % kMakers == 0, "");
    using Four = decltype(load4((const T *)nullptr));
    extern __shared__ __align__(16) char raw[];
    Stage<DK, PARTS> *stages = reinterpret_cast<Stage<DK, PARTS> *>(raw);
    Scores *scores = reinterpret_cast<Scores *>(stages + kStages);          // [2]
    auto stage_of = [&](int m) -> Stage<DK, PARTS> & { return stages[(unsigned)m % kStages]; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int seq = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / p.group, Hk = p.H / p.group;
    const int cb = blockIdx.y * COLS;
    long long b, e;
    bounds(p, seq, b, e);
    const int len = (int)(e - b), nb = len / TB + (len % TB != 0), first = nb ? -4 : 0;
    auto meet = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 * (kChain + kMakers + 3)) : "memory"); };
    if (warp >= kChain && warp < kChain + kMakers) {
        set_regs<kRegs<DK>[0], kRegs<DK>[2]>();
        const int mid = tid - 32 * kChain;
        const T *q = static_cast<const T *>(p.q), *k = static_cast<const T *>(p.k), *v = static_cast<const T *>(p.v);
        Four nk[KU], nq[KU], nv;
        // a thread's places: units of four channels of k and q, STEP tokens apart, and one of v
        constexpr int STEP = MT / (DK / 4);
        const int kt = mid / (DK / 4), ki = mid % (DK / 4) * 4, vt = mid / (COLS / 4), vi = mid % (COLS / 4) * 4;
        const bool kin = ki < p.dk, vin = cb + vi < p.dv;
        const long long krow = (long long)Hk * p.dk, vrow = (long long)p.H * p.dv;
        long long ko = (b + kt) * krow + (long long)hk * p.dk + ki, vo = (b + vt) * vrow + (long long)h * p.dv + cb + vi;
        auto fetch = [&](int left) {   // the next block into registers; `left` tokens are
            const Four zero = {};
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                const bool ok = kin && kt + u * STEP < left;
                nk[u] = ok ? load4(k + ko + u * STEP * krow) : zero;
                nq[u] = ok ? load4(q + ko + u * STEP * krow) : zero;
            }
            nv = vin && vt < left ? load4(v + vo) : zero;
            ko += TB * krow;
            vo += TB * vrow;
        };
        auto put = [&](uint16_t (&to)[PARTS][TB][DK + 8], int t, int i, Four x) {
            if constexpr (PARTS == 3) {
                const float4 f = widen(x);
                uint2 hi, md, lo;
                split(f.x, f.y, hi.x, md.x, lo.x);
                split(f.z, f.w, hi.y, md.y, lo.y);
                *reinterpret_cast<uint2 *>(&to[0][t][i]) = hi;
                *reinterpret_cast<uint2 *>(&to[1][t][i]) = md;
                *reinterpret_cast<uint2 *>(&to[2][t][i]) = lo;
            } else {
                *reinterpret_cast<uint2 *>(&to[0][t][i]) = x;
            }
        };
        // scores, of DK / kMakers channels: rows k and then q of eight tokens by columns k; the four tiles of an operand
        const int who = warp - kChain, x = lane >> 2, y = lane & 3;
        const uint32_t tile = (lane & 7) * PITCH + (lane >> 4) * 16 + who * (DK / kMakers) * 2 + (lane >> 3 & 1) * (uint32_t)sizeof(Stage<DK, PARTS>::k);
        if (nb) fetch(len);
        for (int it = first; it < nb; ++it) {
            if (it + 3 >= 0 && it + 3 < nb) {   // score
                const uint32_t at = ptx::smem_u32(&stage_of(it + 3).k[0][0][0]) + tile;
                float c[3][4] = {};
#pragma unroll
                for (int n = 0; n < DK / 16 / kMakers; ++n) {
                    uint32_t f[PARTS][4];
#pragma unroll
                    for (int a = 0; a < PARTS; ++a) tiles(f[a], at + a * TB * PITCH + 32 * n);
                    auto one = [&](int to, int a, int z) { mma(c[to], f[a][0], f[a][1], f[a][2], f[a][3], f[z][0], f[z][2]); };
                    one(0, 0, 0);
                    if constexpr (PARTS == 3) {
                        one(1, 0, 1);
                        one(2, 1, 1);
                        one(1, 1, 0);
                        one(2, 0, 2);
                        one(2, 2, 0);
                    }
                }
                float (&to)[2 * TB][TB] = scores[it & 1].sum[who];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<float2 *>(&to[x + TB * i][2 * y]) =
                        make_float2(c[0][2 * i] + (c[1][2 * i] + c[2][2 * i]), c[0][2 * i + 1] + (c[1][2 * i + 1] + c[2][2 * i + 1]));
            }
            if (it + 4 < nb) {   // stage
                Stage<DK, PARTS> &s = stage_of(it + 4);
#pragma unroll
                for (int u = 0; u < KU; ++u) {
                    put(s.k, kt + u * STEP, ki, nk[u]);
                    put(s.q, kt + u * STEP, ki, nq[u]);
                }
                *reinterpret_cast<float4 *>(&s.v[vt][vi]) = widen(nv);
                if (it + 5 < nb) fetch(len - (it + 5) * TB);
            }
            meet();
        }
        return;
    }
    if (warp >= kChain) {                             // solves, decays, weights
        set_regs<kRegs<DK>[0], kRegs<DK>[3]>();
        if (warp > kChain + kMakers + 2) return;
        if (warp == kChain + kMakers + 2) {           // weights
            for (int it = first; it < nb; ++it) {
                if (it + 2 >= 0 && it + 2 < nb) {
                    Stage<DK, PARTS> &s = stage_of(it + 2);
                    const Scores &f = scores[(it + 1) & 1];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int i = (lane >> 3) + 4 * n, j = lane & 7;
                        float kk = 0.f, qk = 0.f;
#pragma unroll
                        for (int a = 0; a < kMakers; ++a) {
                            kk += f.sum[a][i][j];
                            qk += f.sum[a][TB + i][j];
                        }
                        const float w = s.w[i][j];
                        s.a[i][j] = s.beta[i] * w * kk;
                        s.p[i][j] = j <= i ? w * qk : 0.f;
                    }
                }
                meet();
            }
            return;
        }
        if (warp == kChain + kMakers) {
            for (int it = first; it < nb; ++it) {
                if (it + 1 >= 0 && it + 1 < nb && lane < TB) {   // solve: a thread a column
                    Stage<DK, PARTS> &s = stage_of(it + 1);
                    float x[TB];
#pragma unroll
                    for (int i = 0; i < TB; ++i) x[i] = i == lane ? 1.f : 0.f;
#pragma unroll
                    for (int j = 0; j < TB - 1; ++j)
#pragma unroll
                        for (int i = j + 1; i < TB; ++i) {
                            const float y = fmaf(-s.a[i][j], x[j], x[i]);
                            x[i] = j >= lane ? y : x[i];   // (a NaN stays behind its token)
                        }
                    const float beta = s.beta[lane];
#pragma unroll
                    for (int i = 0; i < TB; ++i) s.m[i][lane] = x[i] * beta;
                }
                meet();
            }
            return;
        }
        float ng = 0.f, nbeta = 0.f;                  // of tokens past the end: they neither decay nor write
        long long at = (b + lane) * p.H + h;
        int pi = 1, pj = lane;                        // a lane's pair of tokens, the later first
#pragma unroll
        for (int i = 1; i < TB; ++i)
            if (pj >= pi) {
                pj -= pi;
                ++pi;
            }
        auto fetch = [&](int left) {
            const bool ok = lane < TB && lane < left;
            ng = ok ? p.g[p.g_per_token ? at : h] : 0.f;
            nbeta = ok ? p.beta[at] : 0.f;
            at += (long long)TB * p.H;
        };
        if (nb) fetch(len);
        for (int it = first; it < nb; ++it) {
            if (it + 4 < nb) {   // (lanes from TB on hold 0, the sums that reach past the block stay in it)
                Stage<DK, PARTS> &s = stage_of(it + 4);
                float after = ng, before = ng;
#pragma unroll
                for (int o = 1; o < TB; o <<= 1) {
                    after += __shfl_down_sync(0xffffffffu, after, o);
                    const float x = __shfl_up_sync(0xffffffffu, before, o);
                    if (lane >= o) before += x;
                }
                const float left = __shfl_down_sync(0xffffffffu, after, 1);
                if (lane < TB) {
                    s.beta[lane] = nbeta;
                    s.pre[lane] = expf(before);
                    s.suf[lane] = expf(left);   // (of the last: of nothing)
                }
                if (lane < TB) s.w[lane][lane] = 1.f;
                float sum = 0.f;                      // of the log decays between a pair's tokens
#pragma unroll
                for (int l = 1; l < TB; ++l) {
                    const float gl = __shfl_sync(0xffffffffu, ng, l);
                    sum += l > pj && l <= pi ? gl : 0.f;
                }
                if (lane < TB * (TB - 1) / 2) s.w[pi][pj] = expf(sum);
                if (lane == 0) {
                    const bool near = after > -0.25f;
                    s.all = near ? expm1f(after) : expf(after);
                    s.near = near ? 1.f : 0.f;
                }
                if (it + 5 < nb) fetch(len - (it + 5) * TB);
            }
            meet();
        }
        return;
    }
    set_regs<kRegs<DK>[0], kRegs<DK>[1]>();
    // the chain: the state's transpose as the accumulators of [16 columns x 8 channels] products
    constexpr int NT = DK / 8;
    const int x = lane >> 2, y = lane & 3, t0 = 2 * y, wc = 16 * warp, col = cb + wc + x;
    const bool busy = cb + wc < p.dv;
    const long long own = ((long long)seq * p.H + h) * p.dk * p.dv;
    float st[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ch = 8 * n + t0 + (i & 1), c = col + 8 * (i >> 1);
            st[n][i] = p.init && ch < p.dk && c < p.dv ? p.init[own + (long long)ch * p.dv + c] : 0.f;
        }
    const long long orow = (long long)p.H * p.dv;
    long long oo = (b + t0) * orow + (long long)h * p.dv + col;
    // a lane's row of the four tiles that it addresses
    const uint32_t tile = (lane & 7) * PITCH + (lane >> 3) * 16;
    for (int it = first; it < nb; ++it) {
        if (it >= 0 && busy) {
            const Stage<DK, PARTS> &s = stage_of(it);
            const int left = len - it * TB;
            const uint32_t ak = ptx::smem_u32(&s.k[0][0][0]) + tile, aq = ptx::smem_u32(&s.q[0][0][0]) + tile;
            float xk[3][4] = {}, xq[3][4] = {};       // S^T k, S^T q: the large, the middle and the small products
#pragma unroll
            for (int c = 0; c < DK / 32; ++c) {
                uint32_t kb[PARTS][4], qb[PARTS][4];
#pragma unroll
                for (int a = 0; a < PARTS; ++a) {
                    tiles(kb[a], ak + a * TB * PITCH + 64 * c);
                    tiles(qb[a], aq + a * TB * PITCH + 64 * c);
                }
#pragma unroll
                for (int o = 0; o < 4; o += 2) {
                    uint32_t f[3][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int n = 4 * c + o + (i >> 1), r = 2 * (i & 1);
                        split(st[n][r], st[n][r + 1], f[0][i], f[1][i], f[2][i]);
                    }
                    // (k's and q's in turn, so that a sum's next product is six away)
                    auto both = [&](int to, int a, int z) {
                        mma(xk[to], f[a][0], f[a][1], f[a][2], f[a][3], kb[z][o], kb[z][o + 1]);
                        mma(xq[to], f[a][0], f[a][1], f[a][2], f[a][3], qb[z][o], qb[z][o + 1]);
                    };
                    both(0, 0, 0);
                    both(1, 1, 0);
                    both(2, 2, 0);
                    if constexpr (PARTS == 3) {
                        both(1, 0, 1);
                        both(2, 1, 1);
                        both(0, 0, 2);
                    }
                }
            }
            const float pre[2] = {s.pre[t0], s.pre[t0 + 1]}, suf[2] = {s.suf[t0], s.suf[t0 + 1]};
            float r[4], u[4] = {}, small[4] = {}, out[4], low[4] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r[i] = fmaf(-pre[i & 1], xk[0][i] + (xk[1][i] + xk[2][i]), s.v[t0 + (i & 1)][wc + x + 8 * (i >> 1)]);
                out[i] = pre[i & 1] * (xq[0][i] + (xq[1][i] + xq[2][i]));
            }
            uint32_t f[3][2], w[3];
            split(s.m[x][t0], s.m[x][t0 + 1], w[0], w[1], w[2]);
#pragma unroll
            for (int i = 0; i < 2; ++i) split(r[2 * i], r[2 * i + 1], f[0][i], f[1][i], f[2][i]);
            mma_tokens(u, small, f, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] += small[i];
            uint32_t d[3][2];                         // the new values as the state takes them
#pragma unroll
            for (int i = 0; i < 2; ++i) split(suf[0] * u[2 * i], suf[1] * u[2 * i + 1], d[0][i], d[1][i], d[2][i]);
            const float all = s.all;
            if (s.near != 0.f) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) st[n][i] = fmaf(st[n][i], all, st[n][i]);
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) st[n][i] *= all;
            }
#pragma unroll
            for (int c = 0; c < DK / 32; ++c) {
                uint32_t kb[PARTS][4];
#pragma unroll
                for (int a = 0; a < PARTS; ++a) tiles_trans(kb[a], ak + a * TB * PITCH + 64 * c);
#pragma unroll
                for (int n = 0; n < 4; ++n) mma(st[4 * c + n], d[0][0], d[0][1], d[1][0], d[1][1], kb[0][n], kb[0][n]);
                if constexpr (PARTS == 3) {
#pragma unroll
                    for (int n = 0; n < 4; ++n) mma(st[4 * c + n], d[0][0], d[0][1], d[1][0], d[1][1], kb[1][n], kb[1][n]);
#pragma unroll
                    for (int n = 0; n < 4; ++n) mma(st[4 * c + n], d[0][0], d[0][1], d[2][0], d[2][1], kb[2][n], kb[0][n]);
                } else {
#pragma unroll
                    for (int n = 0; n < 4; ++n) mma(st[4 * c + n], d[2][0], d[2][1], 0u, 0u, kb[0][n], 0u);
                }
            }
            split(s.p[x][t0], s.p[x][t0 + 1], w[0], w[1], w[2]);
#pragma unroll
            for (int i = 0; i < 2; ++i) split(u[2 * i], u[2 * i + 1], f[0][i], f[1][i], f[2][i]);
            mma_tokens(out, low, f, w);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t0 + (i & 1) < left && col + 8 * (i >> 1) < p.dv)
                    store_as(static_cast<TO *>(p.out) + oo + (i & 1) * orow + 8 * (i >> 1), (out[i] + low[i]) * p.scale);
            oo += TB * orow;
        }
        meet();
    }
    if (p.final_state) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int ch = 8 * n + t0 + (i & 1), c = col + 8 * (i >> 1);
                if (ch < p.dk && c < p.dv) p.final_state[own + (long long)ch * p.dv + c] = st[n][i];
            }
    }
}

template <typename T, typename TO, int DK>
int launch_size(const Args &p, cudaStream_t stream)
{
    constexpr int bytes = kStages * sizeof(Stage<DK, sizeof(T) == 4 ? 3 : 1>) + 2 * sizeof(Scores);
    // a function attribute belongs to the current device: set it on every launch
    if (cudaFuncSetAttribute(delta_token_kernel<T, TO, DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return KDA_ERR_CUDA;
    const dim3 grid((unsigned)(p.n_seqs * p.H), (unsigned)ceil_div(p.dv, COLS));
    delta_token_kernel<T, TO, DK><<<grid, kThreads, bytes, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <typename T, typename TO>
int launch(const Args &p, cudaStream_t stream)
{
    if (p.dk <= 64) return launch_size<T, TO, 64>(p, stream);
    if (p.dk <= 128) return launch_size<T, TO, 128>(p, stream);
    return launch_size<T, TO, 256>(p, stream);
}

}  // namespace

int run_token_path(const Args &p, int dtype, int out_dtype, cudaStream_t stream)
{
    if (dtype == KDA_BF16)
        return out_dtype == KDA_BF16 ? launch<__nv_bfloat16, __nv_bfloat16>(p, stream) : launch<__nv_bfloat16, float>(p, stream);
    return out_dtype == KDA_BF16 ? launch<float, __nv_bfloat16>(p, stream) : launch<float, float>(p, stream);
}

// Whether the kernel of kda_delta_tc.cu takes these operands: from a mean length on at which it is the faster (us, here
// and there, with initial states.  128 x 128: 32 heads, one sequence of 32 tokens 8.5, 13.9, of 64 12.1, 12.9, 16 of 16 34,
// 54, of 32 53, 55, of 64 82, 53; 96 heads, one of 32 15, 14, 16 of 32 176, 149.  64 x 64: 16 heads, one of 64 9.1, 11.1,
// of 128 14.2, 14.2, 16 of 64 13, 22, of 128 21, 29; 64 heads, 64 sequences of 64 167, 288, 16 of 128 80, 100).
// The lengths themselves are on the device, so the rule does not see a long prompt among many short sequences: 4096 tokens and
// 200 single ones, 128 x 128, 681 for 32 heads (257 and 291 in calls of their own) and 1479 for 96 (289, 844); with 200
// empty ones in place of the tokens 593 and 1064.
bool tc_path(int n_seqs, int64_t T, int d_k, int d_v, int dtype)
{
    return dtype == KDA_BF16 && d_k <= 128 && d_v <= 128 && T >= (d_k <= 64 ? 128 : 32) * (int64_t)n_seqs;
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
