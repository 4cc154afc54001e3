// kda_delta_tc.cu -- the gated delta rule with one decay per head for bf16 operands: chunks of 64 tokens
// on the tensor cores (tcgen05).
//
//     S' = exp(g_t) S_(t-1),   S_t = S' + beta_t k_t (v_t - S'^T k_t)^T,   o_t = scale S_t^T q_t
//
// For a chunk that starts from state S (i, j = its tokens, G_i = sum of the log decays up to i):
//     A_ij = beta_i e^(G_i - G_j) (k_i . k_j)  for j < i,   T = (I + A)^-1 diag(beta)
//     U    = T V + T R,          R_i = -e^(G_i) S^T k_i
//     o_i  = scale (e^(G_i) S^T q_i + sum_(j <= i) e^(G_i - G_j) (q_i . k_j) u_j)
//     S   <- e^(G_C) S + sum_j e^(G_C - G_j) k_j u_j^T
// T, T V and the weighted q . k do not depend on the state, so they are made ahead of the chain
// S -> X = S^T K^T -> R -> U -> S, which is all that is serial.
//
// One CTA a (sequence, head), all of an SM's tensor memory.  Everything is held transposed, value channels as lanes, so
// that the state, R and U are A operands from tensor memory as the warps write them and k, q, v, T and the scores are B
// operands from shared memory.  Two warpgroups are the chain (a thread has half of a lane's columns), one makes outputs,
// two take the chunks in turn and make T and the scores (8 x 8 substitutions, then three joins of halves by mma.sync), and
// three warps issue loads, the Gram products and the chain's products.  Registers are moved to the chain.
// Precision: states shall be good to 1e-6, which bf16 operands (4e-3) miss and tf32's miss too.  S, R, U and T are therefore
// three bf16 parts each (24 bits), six products where both sides have parts and three where one is an input; outputs
// take two parts of S and of U and one of the scores.  fp16 parts would do with two, but k and v are bf16 of any size.
// The products of one chunk: 3 x 8 for X, 6 x 4 for T R, 3 x 8 for the update, 3 x 4 for T V, 2 x 8 for S^T q, 2 x 4 for
// the scores with U, 8 for the Gram, of [128 x 64 x 16] each at 43 cycles: some 5,000 cycles.
//
// Bound by that chain, and by instruction fetch: a chunk takes some 7,900 cycles alone (8 heads).  Products that a chain needs
// (X, T R, update: 3,100) and the passes between them (R, U and S out of tensor memory, into parts and back) follow one
// another; the rest runs beside them, in the gaps.  Left out, to time the rest: preparation 15 % less, the splits 8 %, T V,
// Gram and S^T q 7 %, all but the bare chain 33 %.  The loops' 80 KB of code, a product being 220 bytes of it, do not stay in
// an SM's instruction cache, and what SMs share behind it slows them down together: warps without an instruction, per one
// issued, 0.35 with 8 SMs at work, 0.6 with 96, 3.7 with 152.  T = 8192: 8 heads of 128 x 128 0.49-0.50 ms, 96 heads 0.56,
// 152 heads 0.69, 96 of 64 x 64 0.48, on each of four GPUs at 2070 MHz throughout (one measured before: 0.484, 0.510, 0.681,
// 0.438).  The token-by-token kernel before it took 7.2 ms, the first version of this one 0.86.
// Tried (on that one): all products in loops 0.636, 0.646 and 0.659 ms for 8, 96 and 152 heads (their issue is on the chain), those beside
// the chain in loops 0.532, 0.574, 0.689, by a warp of their own 0.503, 0.576, 0.704; waits without a first look 0.571,
// 0.576, 0.660; before T V stood once and the joins' and R's loops were rolled 0.492, 0.528, 0.720.  Without gain: the
// chain's loads 32 columns at a time or ahead (spills), tf32 rounding by cvt.rna (6 % slower).  T folded into k, so
// that the chain would lose a pass, needs a second operand of three parts a chunk, 48 KB more than shared memory has.
#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

#include "kda_delta.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace delta {
namespace {

using namespace ptx;

constexpr int C = 64;                           // tokens of a chunk
constexpr int kThreads = 6 * 128;
// Registers a thread of each warpgroup, 80 at launch.
constexpr int kRegsChain = 128, kRegsOut = 48, kRegsPrep = 72, kRegsIssue = 32;
static_assert(2 * kRegsChain + kRegsOut + 2 * kRegsPrep + kRegsIssue <= 6 * 80, "registers of the block");
template <int N>
__device__ __forceinline__ void set_regs()
{
    if constexpr (N > 80) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

constexpr long long kTimeout = 4000000000ll;    // bounded waits for work in flight at an end: 4e9 SM cycles (~2 s)
constexpr uint32_t kWaitCycles = 2000000000u;   // bounded waits between roles: 2e9 SM cycles (~1 s)
constexpr uint32_t kSleepNs = 100000;           // longest sleep between two looks at the clock

__device__ int g_delta_tc_error;                // sticky device error word of this translation unit

constexpr int STAGES = 3;                       // chunks of k and q
constexpr uint32_t REGION = 128 * 128;          // 64 channels of 64 k rows, then of 64 q rows (odd chunks: q first)
constexpr uint32_t TILE = 64 * 128;             // 64 x 64 bf16
constexpr int PITCH = 68;                       // of the solver's fp32 matrices
// Shared memory: k and q, v, three parts of T (twice), P (three times), A and then T in fp32 (twice)
constexpr int P_TILES = 3;
constexpr uint32_t SQUARE = C * PITCH * 4;
constexpr uint32_t SM_KQ = 0, SM_V = SM_KQ + STAGES * 2 * REGION, SM_T = SM_V + 2 * TILE, SM_P = SM_T + 6 * TILE,
                   SM_TF = SM_P + P_TILES * TILE, SM_SHARED = SM_TF + 2 * SQUARE;
// Tensor memory, lanes = value channels (Gram: tokens).  The state's parts lie 16 key channels at a time, hi and
// mid side by side, where the update that they make room for comes (a thread overwrites only what it has
// read); R over X (its lo over the state's), U's parts over U and over R.
constexpr uint32_t TM_S = 0, TM_DST = 0, TM_SLO = 128, TM_X = 192, TM_U = 256, TM_UX = 320, TM_O = 384, TM_GRAM = 448,
                   TM_COLS = 512;

struct Decays {
    float gh[C], gl[C];         // a token's sum of log decays, in two parts (see prep_role)
    float suf[C];               // e^(sum from it to the end of its 16 tokens)
    float beta[C], neg[C];      // beta, -e^G
    float gam[C];               // scale e^G
    float lat[C];               // e^(G_C - G)
    float total, less;          // e^(G_C), and what its rounding left out
    float pad[2];
};
constexpr int DECS = 4;

// A wait for a phase's parity holds only where the phase before it is known to be over: so barriers that the two
// groups of warps of prep_role take in turn (products of keys and queries, T) are one for each.
enum Bar {
    B_KQ_FULL, B_K_READY = B_KQ_FULL + STAGES, B_K_FREE = B_K_READY + STAGES, B_V_FULL = B_K_FREE + STAGES, B_V_READY, B_V_FREE,
    B_DEC_READY, B_GRAM_DONE = B_DEC_READY + DECS, B_GRAM_FREE = B_GRAM_DONE + 2, B_P_READY, B_P_FREE = B_P_READY + P_TILES,
    B_T_READY = B_P_FREE + P_TILES, B_T_FREE = B_T_READY + 2, B_S_READY = B_T_FREE + 2, B_X_DONE = B_S_READY + 4, B_R_READY,
    B_U_DONE = B_R_READY + 2, B_UP_READY, B_KU_DONE = B_UP_READY + 2, B_O1_DONE = B_KU_DONE + 2, B_O1_READY, B_O2_DONE, B_O2_FREE,
    B_DRAIN, B_COUNT = B_DRAIN + 2
};

struct Shared {
    Decays dec[DECS];
    uint64_t bars[B_COUNT];
    uint32_t tmem;
    int abort;
    int zero;                   // always 0: the abort flag of waits that must not give up early
};
constexpr uint32_t SM_BYTES = SM_SHARED + sizeof(Shared);
static_assert(SM_BYTES <= 232448, "shared memory per block");

// Products.  Two of them are in order only where they accumulate into the same place in the same shape; what else
// one has to find read or written by another waits for its completion.  (So T's and P's zeros above the diagonal are
// multiplied too: products of fewer rows would be another shape.)  Issuing is on the chain, so all but an operand's place in shared memory is known
// when the kernel is compiled: tensor memory is taken whole, so that it starts at 0, and only the lower half
// of a descriptor varies.
constexpr uint32_t NEG_A = 1u << 13, NEG_B = 1u << 14;          // of an instruction descriptor
constexpr uint32_t DESC_HI = (1024 >> 4) | 1u << 14 | 2u << 29;   // see smem_desc: rows in groups of 1024 bytes
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo = 0) { return saddr >> 4 | lbo >> 4 << 16; }

template <uint32_t D, uint32_t A, uint32_t IDESC, bool ACC>
__device__ __forceinline__ void mma_tmem(uint32_t b_lo)   // A from tensor memory
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}"
                 ::"r"(D), "r"(A), "r"(b_lo), "r"(IDESC), "n"((int)ACC), "r"(DESC_HI) : "memory");
}

// Waits for phase `phase` of a barrier, giving up after `cycles` SM cycles: a role that gave up ends, the
// others, which stand at waits of their own by then, give up by the same rule, and the kernel's end records
// it.  As short as it can be, since it stands in some forty places: the roles' loops together have to fit the
// instruction cache.
__device__ __forceinline__ bool wait(Shared *sh, int bar, int phase, uint32_t cycles = kWaitCycles)
{
    if (mbar_try_wait(&sh->bars[bar], phase & 1)) return true;
    const uint32_t from = (uint32_t)clock();
#pragma unroll 1
    do {
        if (mbar_try_wait_sleep(&sh->bars[bar], phase & 1, kSleepNs)) return true;
    } while ((uint32_t)clock() - from < cycles);
    return false;
}

__device__ __forceinline__ void give_up(Shared *sh) { *reinterpret_cast<volatile int *>(&sh->abort) = 1; }

// wait for a whole warp: its lanes leave a loop together.
__device__ __forceinline__ bool wait_warp(Shared *sh, int bar, int phase, uint32_t cycles = kWaitCycles)
{
    return __all_sync(0xffffffffu, wait(sh, bar, phase, cycles));
}

__device__ __forceinline__ void record(Shared *sh)
{
    if (sh->abort) atomicExch(&g_delta_tc_error, KDA_ERR_DEVICE_TIMEOUT);
}

__device__ __forceinline__ void arrive(Shared *sh, int bar, int lane)
{
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->bars[bar]);
}

// stage by stage, since a pair's own operations wait for one another; `two`: the hi parts, then the mid parts
template <int N>
__device__ __forceinline__ void split3(float2 (&y)[N], uint32_t (&two)[2 * N], uint32_t (&lo)[N])
{
#pragma unroll
    for (int e = 0; e < N; ++e) two[e] = pack_bf16x2(y[e].x, y[e].y);
#pragma unroll
    for (int e = 0; e < N; ++e) rest(two[e], y[e]);
#pragma unroll
    for (int e = 0; e < N; ++e) two[N + e] = pack_bf16x2(y[e].x, y[e].y);
#pragma unroll
    for (int e = 0; e < N; ++e) rest(two[N + e], y[e]);
#pragma unroll
    for (int e = 0; e < N; ++e) lo[e] = pack_bf16x2(y[e].x, y[e].y);
}

__device__ __forceinline__ float2 as_pair(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------------------------------------
// loads

__device__ void load_role(const CUtensorMap *mq, const CUtensorMap *mk, const CUtensorMap *mv, uint8_t *smem, Shared *sh,
                          int h, int hk, int regions, long long t0, int nch)
{
    // a tile's loads, and the next one's into L2 (its work begins with its load and has to end in two chunks' time)
    auto kq = [&](int c) {
        if (elect_one()) {
            uint64_t *bar = &sh->bars[B_KQ_FULL + c % STAGES];
            uint8_t *to = smem + SM_KQ + c % STAGES * 2 * REGION;
            const int t = (int)(t0 + (long long)c * C);
            mbar_arrive_expect_tx(bar, regions * REGION);
#pragma unroll 1
            for (int r = 0; r < regions; ++r) {
                tma_load_3d(to + r * REGION + (c & 1) * TILE, mk, bar, 64 * r, hk, t);
                tma_load_3d(to + r * REGION + (~c & 1) * TILE, mq, bar, 64 * r, hk, t);
                if (c + 1 < nch) {
                    tma_prefetch_l2_3d(mk, 64 * r, hk, t + C);
                    tma_prefetch_l2_3d(mq, 64 * r, hk, t + C);
                }
            }
        }
        __syncwarp();
    };
    auto value = [&](int c) {
        if (elect_one()) {
            const int t = (int)(t0 + (long long)c * C);
            mbar_arrive_expect_tx(&sh->bars[B_V_FULL], 2 * TILE);
#pragma unroll 1
            for (int r = 0; r < 2; ++r) {
                tma_load_3d(smem + SM_V + r * TILE, mv, &sh->bars[B_V_FULL], 64 * r, h, t);
                if (c + 1 < nch) tma_prefetch_l2_3d(mv, 64 * r, h, t + C);
            }
        }
        __syncwarp();
    };
    int nk = 0, nv = 0;   // tiles issued
#pragma unroll 1
    for (; nk < nch && nk < STAGES; ++nk) kq(nk);
    bool ok = true;
#pragma unroll 1
    for (; ok && nv < nch; ++nv) {
        if (nv > 0 && !(ok = wait_warp(sh, B_V_FREE, nv - 1))) break;
        value(nv);
        if (nv > 0 && nk < nch) {   // the stage was chunk nv - 1's
            if (!(ok = wait_warp(sh, B_K_FREE + nk % STAGES, nk / STAGES - 1))) {
                ++nv;
                break;
            }
            kq(nk++);
        }
    }
    if (!ok) {   // no copy in flight when the CTA leaves
        for (int c = max(0, nk - STAGES); c < nk; ++c)
            mbar_wait(&sh->bars[B_KQ_FULL + c % STAGES], c / STAGES & 1, &sh->zero, kTimeout);
        if (nv > 0) mbar_wait(&sh->bars[B_V_FULL], (nv - 1) & 1, &sh->zero, kTimeout);
        give_up(sh);
    }
}

// ---------------------------------------------------------------------------------------------
// products: whole warps, one elected lane issuing, so that descriptors stay in uniform registers

__device__ void drain(Shared *sh, int which)
{
    if (elect_one()) mma_commit(&sh->bars[B_DRAIN + which]);
    mbar_wait(&sh->bars[B_DRAIN + which], 0, &sh->zero, kTimeout);
    give_up(sh);
}

template <uint32_t D, uint32_t IDESC, bool ACC>
__device__ __forceinline__ void mma_smem(uint32_t a_lo, uint32_t b_lo)   // both from shared memory
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}"
                 ::"r"(D), "r"(a_lo), "r"(b_lo), "r"(IDESC), "n"((int)ACC), "r"(DESC_HI) : "memory");
}

// the loops over constants
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F f)
{
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        each<N, I + 1>(f);
    }
}

template <int REGIONS>
__device__ void gram_mma_role(uint32_t sb, Shared *sh, int nch)
{
    constexpr uint32_t I = idesc_bf16(128, 64, 0, 0);
    bool ok = true;
    for (int c = 0; c < nch; ++c) {
        ok = wait_warp(sh, B_K_READY + c % STAGES, c / STAGES) && (c == 0 || wait_warp(sh, B_GRAM_FREE, c - 1));
        if (!ok) break;
        tc_fence_after();
        const uint32_t k = desc_lo(sb + SM_KQ + c % STAGES * 2 * REGION);
        if (elect_one()) {
            each<4 * REGIONS>([&](auto x_) {
                constexpr int x = decltype(x_)::value;
                const uint32_t at = k + (((x >> 2) * REGION + (x & 3) * 32) >> 4);
                mma_smem<TM_GRAM, I, (x > 0)>(at, at + ((c & 1) * TILE >> 4));
            });
            mma_commit(&sh->bars[B_GRAM_DONE + (c & 1)]);
        }
        __syncwarp();
    }
    if (!ok) drain(sh, 0);
}

// Key channels come in steps of 16.  A thread of the chain has GROUPS of them, half of each half of the channels, since
// the update comes by halves: group g of the first four warps (w = 0) or the others is step
template <int GROUPS>
__host__ __device__ constexpr int step_of(int w, int g) { return GROUPS * (g / (GROUPS / 2)) + GROUPS / 2 * w + g % (GROUPS / 2); }

template <int REGIONS>
__device__ void chain_mma_role(uint32_t sb, Shared *sh, int nch)
{
    constexpr int STEPS = 4 * REGIONS, GROUPS = STEPS / 2;   // 16 key channels each; those of four warps
    constexpr uint32_t I64 = idesc_bf16(128, 64, 0, 0), I_KU = idesc_bf16(128, 64, 0, 1);
    bool ok = true;
    for (int c = 0; ok && c < nch; ++c) {
        const int st = c % STAGES, half = c & 1;
        const uint32_t tile = sb + SM_KQ + st * 2 * REGION;
        const uint32_t k = desc_lo(tile + half * TILE), q = desc_lo(tile + (half ^ 1) * TILE), t = desc_lo(sb + SM_T + half * 3 * TILE),
                       v = desc_lo(sb + SM_V, TILE), p = desc_lo(sb + SM_P + c % P_TILES * TILE);
        // U = T V, where nothing waits for the pipe: while the state before is worked on (the update reads where U comes)
        ok = (c == 0 || wait_warp(sh, B_KU_DONE + REGIONS - 1, c - 1)) && wait_warp(sh, B_T_READY + half, c >> 1) &&
             wait_warp(sh, B_V_FULL, c) && wait_warp(sh, B_V_READY, c);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
            each<4>([&](auto s_) {
                constexpr int s = decltype(s_)::value;
                constexpr uint32_t I = idesc_bf16(128, 64, 1, 0);
                const uint32_t a = v + (s * 2048 >> 4), hi = t + (s * 32 >> 4);
                mma_smem<TM_U, I, (s > 0)>(a, hi + 2 * (TILE >> 4));
                mma_smem<TM_U, I | NEG_B, true>(a, hi + (TILE >> 4));
                mma_smem<TM_U, I, true>(a, hi);
            });
            mma_commit(&sh->bars[B_V_FREE]);
        }
        __syncwarp();
        // X = S^T K^T, as the state's parts come (over what the last chunk's outputs read)
        ok = wait_warp(sh, B_K_READY + st, c / STAGES) && (c == 0 || wait_warp(sh, B_O2_DONE, c - 1));
        each<GROUPS>([&](auto g_) {
            constexpr int g = decltype(g_)::value;
            if (!ok || !(ok = wait_warp(sh, B_S_READY + g, c))) return;
            tc_fence_after();
            if (elect_one()) {
                each<2>([&](auto w_) {
                    constexpr int x = step_of<GROUPS>(decltype(w_)::value, g);
                    const uint32_t b = k + (((x >> 2) * REGION + (x & 3) * 32) >> 4);
                    mma_tmem<TM_X, TM_S + 16 * x, I64, (x > 0)>(b);
                    mma_tmem<TM_X, TM_S + 16 * x + 8, I64 | NEG_A, true>(b);
                    mma_tmem<TM_X, TM_SLO + 8 * x, I64, true>(b);
                });
                if (g == GROUPS - 1) mma_commit(&sh->bars[B_X_DONE]);
            }
            __syncwarp();
        });
        // U + T R
        each<2>([&](auto g_) {
            constexpr int g = decltype(g_)::value;
            if (!ok || !(ok = wait_warp(sh, B_R_READY + g, c))) return;
            tc_fence_after();
            if (elect_one()) {
                each<2>([&](auto w_) {
                    constexpr int s = 2 * decltype(w_)::value + g;
                    constexpr uint32_t a = TM_X + 16 * s;
                    const uint32_t hi = t + (s * 32 >> 4), mid = hi + (TILE >> 4), lo = mid + (TILE >> 4);
                    mma_tmem<TM_U, TM_SLO + 8 * s, I64, true>(hi);
                    mma_tmem<TM_U, a + 8, I64, true>(mid);
                    mma_tmem<TM_U, a, I64, true>(lo);
                    mma_tmem<TM_U, a + 8, I64 | NEG_A, true>(hi);
                    mma_tmem<TM_U, a, I64 | NEG_B, true>(mid);
                    mma_tmem<TM_U, a, I64, true>(hi);
                });
                if (g == 1) {
                    mma_commit(&sh->bars[B_U_DONE]);
                    mma_commit(&sh->bars[B_T_FREE + half]);
                }
            }
            __syncwarp();
        });
        // S^T Q^T, while U is worked on (the update writes over the state's parts)
        ok = ok && (c == 0 || wait_warp(sh, B_O2_FREE, c - 1));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
            each<STEPS>([&](auto x_) {
                constexpr int x = decltype(x_)::value;
                const uint32_t b = q + (((x >> 2) * REGION + (x & 3) * 32) >> 4);
                mma_tmem<TM_O, TM_S + 16 * x, I64, (x > 0)>(b);
                mma_tmem<TM_O, TM_S + 16 * x + 8, I64 | NEG_A, true>(b);
            });
            mma_commit(&sh->bars[B_O1_DONE]);
        }
        __syncwarp();
        // the update, sum over j of k_j u~_j^T
        ok = wait_warp(sh, B_O1_DONE, c);
        each<2>([&](auto g_) {
            constexpr int g = decltype(g_)::value;
            if (!ok || !(ok = wait_warp(sh, B_UP_READY + g, c))) return;
            tc_fence_after();
            if (elect_one()) {
                each<REGIONS>([&](auto r_) {   // 64 key channels at a time, so that the state's work begins with the first
                    constexpr int r = decltype(r_)::value;
                    each<2>([&](auto w_) {
                        constexpr int s = 2 * decltype(w_)::value + g;
                        const uint32_t b = k + ((r * REGION + s * 2048) >> 4);
                        mma_tmem<TM_DST + 64 * r, TM_U + 16 * s, I_KU, (s > 0)>(b);
                        mma_tmem<TM_DST + 64 * r, TM_U + 16 * s + 8, I_KU | NEG_A, true>(b);
                        mma_tmem<TM_DST + 64 * r, TM_UX + 16 * s, I_KU, true>(b);
                    });
                    if (g == 1) mma_commit(&sh->bars[B_KU_DONE + r]);
                });
                if (g == 1) mma_commit(&sh->bars[B_K_FREE + st]);
            }
            __syncwarp();
        });
        // outputs: U^T P^T onto the scaled S^T Q^T
        ok = ok && wait_warp(sh, B_P_READY + c % P_TILES, c / P_TILES) && wait_warp(sh, B_O1_READY, c);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
            each<4>([&](auto s_) {
                constexpr int s = decltype(s_)::value;
                const uint32_t b = p + (s * 32 >> 4);
                mma_tmem<TM_O, TM_X + 8 * s, I64 | NEG_A, true>(b);
                mma_tmem<TM_O, TM_UX + 16 * s + 8, I64, true>(b);
            });
            mma_commit(&sh->bars[B_O2_DONE]);
            mma_commit(&sh->bars[B_P_FREE + c % P_TILES]);
        }
        __syncwarp();
    }
    if (!ok) drain(sh, 1);
}

// ---------------------------------------------------------------------------------------------
// warps 0-7, the chain: thread = value channel 32 (warp % 4) + lane; warps 0-3 tokens 0-31 and half of the key
// channels (see step_of), warps 4-7 the others

template <int REGIONS>
__device__ void chain_role(const Args &p, uint8_t *smem, Shared *sh, int seq, int h, long long len, int nch)
{
    constexpr int GROUPS = 2 * REGIONS;   // of 16 key channels
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp >> 2, ch = 32 * (warp & 3) + lane;
    const uint32_t tq = (uint32_t)(32 * (warp & 3)) << 16;
    const bool ch_ok = ch < p.dv;
    const long long own = ((long long)seq * p.H + h) * p.dk * p.dv + ch;
    float2 st[8 * GROUPS];
#pragma unroll
    for (int x = 0; x < 8 * GROUPS; ++x) {
        const int i = 16 * step_of<GROUPS>(w, x / 8) + x % 8 * 2;
        st[x] = make_float2(0.f, 0.f);
        if (p.init && ch_ok && i < p.dk)   // (d_k is even)
            st[x] = make_float2(p.init[own + (long long)i * p.dv], p.init[own + (long long)(i + 1) * p.dv]);
    }
    for (int c = 0;; ++c) {
        if (c < nch) {   // v's rows of other sequences: 0 x NaN must not get into the products
            const int n = (int)min(len - (long long)c * C, (long long)C);
            if (n < C) {
                if (!wait_warp(sh, B_V_FULL, c)) return give_up(sh);
#pragma unroll 1
                for (int x = threadIdx.x; x < (C - n) * 16; x += 256)
                    *reinterpret_cast<uint4 *>(smem + SM_V + (x & 1) * TILE + (n + (x >> 4)) * 128 + (x >> 1 & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
            }
            arrive(sh, B_V_READY, lane);
        }
        // the state after chunk c - 1, and its three bf16 parts, all 24 bits
        float2 total = make_float2(0.f, 0.f), less = total;
        if (c > 0) {
            const Decays &d = sh->dec[(c - 1) % DECS];
            total.x = total.y = d.total;
            less.x = less.y = d.less;
        }
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const int x16 = 16 * step_of<GROUPS>(w, g);
            if (c > 0) {
                uint32_t x[16];
                if (g % 2 == 0) {
                    if (!wait_warp(sh, B_KU_DONE + g / 2, c - 1)) return give_up(sh);
                    tc_fence_after();
                }
                tmem_ld16(tq + TM_DST + x16, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    st[8 * g + e] = fma2(st[8 * g + e], total, fma2(st[8 * g + e], less, as_pair(x[2 * e], x[2 * e + 1])));
            }
            if (c == nch) continue;
            uint32_t two[16], lo[8];
            float2 y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = st[8 * g + e];
            split3(y, two, lo);
            if (g > 0) {   // (what was stored before has had the time)
                tmem_wait_st();
                tc_fence_before();
                arrive(sh, B_S_READY + g - 1, lane);
            }
            tmem_st16(tq + TM_S + x16, two);
            tmem_st8(tq + TM_SLO + x16 / 2, lo);
        }
        if (c == nch) break;
        tmem_wait_st();
        tc_fence_before();
        arrive(sh, B_S_READY + GROUPS - 1, lane);
        const Decays &d = sh->dec[c % DECS];
        if (!wait_warp(sh, B_DEC_READY + c % DECS, c / DECS)) return give_up(sh);
        if (!wait_warp(sh, B_X_DONE, c)) return give_up(sh);
        tc_fence_after();
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {   // R = -e^G X, in three parts
            uint32_t x[16], two[16], lo[8];
            float2 y[8];
            const int t = 32 * w + 16 * g;
            tmem_ld16(tq + TM_X + t, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float4 n = *reinterpret_cast<const float4 *>(&d.neg[t + 2 * e]);
                y[e] = make_float2(n.x * __uint_as_float(x[2 * e]), n.y * __uint_as_float(x[2 * e + 1]));
                y[e + 1] = make_float2(n.z * __uint_as_float(x[2 * e + 2]), n.w * __uint_as_float(x[2 * e + 3]));
            }
            split3(y, two, lo);
            tmem_st16(tq + TM_X + t, two);
            tmem_st8(tq + TM_SLO + t / 2, lo);
            tmem_wait_st();
            tc_fence_before();
            arrive(sh, B_R_READY + g, lane);
        }
        if (!wait_warp(sh, B_U_DONE, c)) return give_up(sh);
        tc_fence_after();
#pragma unroll 1
        for (int g = 0; g < 2; ++g) {   // u~ = e^(G_C - G) u in three parts, u in two for the outputs
            uint32_t x[16], two[16], lo[8];
            float2 y[8];
            const int t = 32 * w + 16 * g;
            tmem_ld16(tq + TM_U + t, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float4 f = *reinterpret_cast<const float4 *>(&d.lat[t + 2 * e]);
                y[e] = make_float2(__uint_as_float(x[2 * e]) * f.x, __uint_as_float(x[2 * e + 1]) * f.y);
                y[e + 1] = make_float2(__uint_as_float(x[2 * e + 2]) * f.z, __uint_as_float(x[2 * e + 3]) * f.w);
            }
            split3(y, two, lo);
            tmem_st16(tq + TM_U + t, two);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                two[e] = lo[e];
                y[e] = as_pair(x[2 * e], x[2 * e + 1]);
                two[8 + e] = pack_bf16x2(y[e].x, y[e].y);
                rest(two[8 + e], y[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) lo[e] = pack_bf16x2(y[e].x, y[e].y);
            tmem_st16(tq + TM_UX + t, two);
            tmem_st8(tq + TM_X + t / 2, lo);
            tmem_wait_st();
            tc_fence_before();
            arrive(sh, B_UP_READY + g, lane);
        }
    }
    if (p.final_state && ch_ok) {
#pragma unroll
        for (int x = 0; x < 8 * GROUPS; ++x) {
            const int i = 16 * step_of<GROUPS>(w, x / 8) + x % 8 * 2;
            if (i < p.dk) {
                p.final_state[own + (long long)i * p.dv] = st[x].x;
                p.final_state[own + (long long)(i + 1) * p.dv] = st[x].y;
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------
// warps 8-11, outputs: thread = value channel 32 (warp % 4) + lane

template <typename TO>
__device__ void output_role(const Args &p, Shared *sh, int h, long long t0, long long len, int nch)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ch = 32 * (warp & 3) + lane;
    const uint32_t tq = ((uint32_t)(32 * (warp & 3)) << 16) + TM_O;
    const long long step = (long long)p.H * p.dv;
    const bool odd = lane & 1;
    for (int c = 0; c < nch; ++c) {
        const Decays &d = sh->dec[c % DECS];
        if (!wait_warp(sh, B_DEC_READY + c % DECS, c / DECS) || !wait_warp(sh, B_O1_DONE, c)) return give_up(sh);
        tc_fence_after();
#pragma unroll 1
        for (int x = 0; x < C; x += 16) {   // what the state gives, scaled
            uint32_t r[16];
            tmem_ld16(tq + x, r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(&d.gam[x + e]);
                const float2 y = mul2(as_pair(r[e], r[e + 1]), make_float2(f.x, f.y));
                const float2 z = mul2(as_pair(r[e + 2], r[e + 3]), make_float2(f.z, f.w));
                r[e] = __float_as_uint(y.x);
                r[e + 1] = __float_as_uint(y.y);
                r[e + 2] = __float_as_uint(z.x);
                r[e + 3] = __float_as_uint(z.y);
            }
            tmem_st16(tq + x, r);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(sh, B_O1_READY, lane);
        if (!wait_warp(sh, B_O2_DONE, c)) return give_up(sh);
        tc_fence_after();
        // Two tokens of a channel are packed and turned around with the neighbouring channel's, so that an even
        // lane stores the first token's pair of channels and an odd lane the second's.
        constexpr int ROWS = sizeof(TO) == 2 ? 2 : 1;   // tokens a store step
        const long long first = (long long)c * C + (ROWS == 2 ? odd : 0);
        TO *o = static_cast<TO *>(p.out) + ((t0 + first) * p.H + h) * p.dv + (ROWS == 2 ? ch & ~1 : ch);
        int left = ch < p.dv ? (int)min(len - first, (long long)C) : 0;   // tokens from the lane's first on
#pragma unroll 1
        for (int x = 0; x < C; x += 16) {
            uint32_t r[16];
            tmem_ld16(tq + x, r);
            tmem_wait_ld();
            if (x + 16 >= C) {   // everything is read
                tc_fence_before();
                arrive(sh, B_O2_FREE, lane);
            }
#pragma unroll
            for (int e = 0; e < 16; e += ROWS) {
                if constexpr (ROWS == 1) {
                    if (e < left) *o = __uint_as_float(r[e]);
                } else {
                    const uint32_t mine = pack_bf16x2(__uint_as_float(r[e]), __uint_as_float(r[e + 1]));
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, mine, 1);
                    if (e < left) *reinterpret_cast<uint32_t *>(o) = __byte_perm(mine, got, odd ? 0x3276 : 0x5410);
                }
                o += ROWS * step;
            }
            left -= 16;
        }
    }
}

// ---------------------------------------------------------------------------------------------
// warps 12-15 and 16-19, in turn a chunk each: what does not depend on the state.  The chunk's decays; A (two warps)
// and P (two) from the products of its keys and queries; T = (I + A)^-1.  A and its blocks are the more work:
// the second four warps' are made by the other two schedulers than the first four's.
//
// Sums of log decays keep their differences exact: a token's log decay is a multiple of 2^-10, summed
// in whole numbers, and a rest below 2^-11, summed in fp32, so that G_i - G_j is good to 2^-30 or
// so however large G is.  A log decay below -128 is taken as -128: any span over it weighs nothing.
//
// T in fp32, in A's place, by blocks: 8 x 8 by substitution, then three times
//     [[P, 0], [B, Q]]^-1 = [[P^-1, 0], [-Q^-1 B P^-1, Q^-1]]
// The products of the joins run on warp-wide tensor instructions with tf32 operands in two parts each (what is left
// out is some 2^-21 of |a| |b|): an operand read by a few narrow loads, where products on the FMA pipe were bound by
// shared memory's path.  Both operands stand along k; what stands on the right is kept transposed, in places above the
// diagonal that nothing else uses.

// hi rounded to tf32 (a conversion instruction for it cost 6 % of the whole kernel), lo what is left, whose last bits
// the product ignores
__device__ __forceinline__ void tf32_parts(float x, uint32_t &hi, uint32_t &lo)
{
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// y[n] = a b_n^T for a of 16 rows and N groups of 8 columns over k of [0, len); lane l holds rows l / 4 and l / 4 + 8
// of columns 2 (l % 4) and the next: (r, c), (r, c + 1), (r + 8, c), (r + 8, c + 1)
template <int N>
__device__ __forceinline__ void products(const float *a, const float *b, int len, float (&y)[N][4])
{
    const int lane = threadIdx.x & 31, at = (lane >> 2) * PITCH + (lane & 3);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[n][e] = 0.f;
#pragma unroll 2
    for (int k = 0; k < len; k += 8) {
        uint32_t ah[4], al[4], bh[2], bl[2];
        tf32_parts(a[at + k], ah[0], al[0]);
        tf32_parts(a[at + k + 8 * PITCH], ah[1], al[1]);
        tf32_parts(a[at + k + 4], ah[2], al[2]);
        tf32_parts(a[at + k + 8 * PITCH + 4], ah[3], al[3]);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            tf32_parts(b[at + k + 8 * n * PITCH], bh[0], bl[0]);
            tf32_parts(b[at + k + 8 * n * PITCH + 4], bh[1], bl[1]);
            mma_tf32(y[n], al, bh);
            mma_tf32(y[n], ah, bl);
            mma_tf32(y[n], ah, bh);
        }
    }
}

// A warp's two 16 x 16 blocks on the diagonal, of rows o .. o + 31
template <typename F>
__device__ __forceinline__ void diagonal(float *A, F turned, int o, int lane)
{
    {   // 8 x 8 blocks, a column per lane
        const int b = lane >> 3, col = lane & 7;
        float *a = A + (o + 8 * b) * (PITCH + 1), t[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = k == col ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < 8; j += 4)   // what four columns' results take from the rows below
#pragma unroll
            for (int k = j + 1; k < 8; ++k) {
                const float4 r = *reinterpret_cast<const float4 *>(a + k * PITCH + j);
                t[k] = fmaf(-r.x, t[j], t[k]);
                if (k > j + 1) t[k] = fmaf(-r.y, t[j + 1], t[k]);
                if (k > j + 2) t[k] = fmaf(-r.z, t[j + 2], t[k]);
                if (k > j + 3) t[k] = fmaf(-r.w, t[j + 3], t[k]);
            }
        __syncwarp();                    // (every lane has read its block)
        const float4 x = make_float4(t[0], t[1], t[2], t[3]), y = make_float4(t[4], t[5], t[6], t[7]);
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k * PITCH + col] = t[k];
        float4 *to = reinterpret_cast<float4 *>(a + col * PITCH + 8);   // transposed, beside the upper block of a pair
        if (!(b & 1)) {
            to[0] = x;
            to[1] = y;
        }
        const int pair = (o >> 4) + (b >> 1);
        to = reinterpret_cast<float4 *>(turned(pair) + (8 * (b & 1) + col) * PITCH);
        if (pair < 3) {
            if (b & 1) to[0] = to[1] = make_float4(0.f, 0.f, 0.f, 0.f);
            to[2 * (b & 1)] = x;
            to[2 * (b & 1) + 1] = y;
        }
        __syncwarp();
    }
    // The joins of both pairs in one: the first pair's rows are a product's upper half, the second's its lower; of a
    // result for the other pair's columns half is of no use.
    const int r = lane >> 2, t = lane & 3;
    float *first = A + o * (PITCH + 1), *second = first + 16 * (PITCH + 1);
    auto product = [&](int left, float (&y0)[4], float (&y1)[4]) {
        uint32_t ah[4], al[4], bh[2], bl[2];
        const int a = (8 + r) * PITCH + left + t, b = r * PITCH + 8 + t;
        tf32_parts(first[a], ah[0], al[0]);
        tf32_parts(second[a], ah[1], al[1]);
        tf32_parts(first[a + 4], ah[2], al[2]);
        tf32_parts(second[a + 4], ah[3], al[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) y0[e] = y1[e] = 0.f;
        tf32_parts(first[b], bh[0], bl[0]);
        tf32_parts(first[b + 4], bh[1], bl[1]);
        mma_tf32(y0, al, bh);
        mma_tf32(y0, ah, bl);
        mma_tf32(y0, ah, bh);
        tf32_parts(second[b], bh[0], bl[0]);
        tf32_parts(second[b + 4], bh[1], bl[1]);
        mma_tf32(y1, al, bh);
        mma_tf32(y1, ah, bl);
        mma_tf32(y1, ah, bh);
        __syncwarp();                    // (every lane has read its operands)
    };
    float y0[4], y1[4];
    product(0, y0, y1);                  // Y = B P^-1, kept transposed over P^-1
    const int at = 2 * t * PITCH + 8 + r;
    first[at] = y0[0];
    first[at + PITCH] = y0[1];
    second[at] = y1[2];
    second[at + PITCH] = y1[3];
    __syncwarp();
    product(8, y0, y1);                  // Q^-1 Y
    *reinterpret_cast<float2 *>(first + (8 + r) * PITCH + 2 * t) = make_float2(-y0[0], -y0[1]);
    *reinterpret_cast<float2 *>(second + (8 + r) * PITCH + 2 * t) = make_float2(-y1[2], -y1[3]);
    *reinterpret_cast<float2 *>(first + r * PITCH + 8 + 2 * t) = make_float2(0.f, 0.f);
    *reinterpret_cast<float2 *>(second + r * PITCH + 8 + 2 * t) = make_float2(0.f, 0.f);
    const int pair = o >> 4;
    turned(pair)[at] = -y0[0];
    turned(pair)[at + PITCH] = -y0[1];
    if (pair + 1 < 3) {
        turned(pair + 1)[at] = -y1[2];
        turned(pair + 1)[at + PITCH] = -y1[3];
    }
}

__device__ void prep_role(const Args &p, uint8_t *smem, Shared *sh, int h, int regions, long long t0, long long len,
                          int nch)
{
    constexpr float LOG2E = 1.4426950408889634f;
    const int par = (threadIdx.x >> 7) - 3, tid = threadIdx.x & 127, warp = tid >> 5, lane = tid & 31;
    const uint32_t tq = ((uint32_t)(32 * warp) << 16) + TM_GRAM, bar = 1 + par;
    uint8_t *parts = smem + SM_T + par * 3 * TILE;
    float *A = reinterpret_cast<float *>(smem + SM_TF + par * SQUARE);
    const int r = lane >> 2, q = (lane & 3) * 2;    // this lane's part of a product's result
    // where a 16 x 16 block's inverse stands transposed (the last one's does not)
    auto turned = [&](int b) { return A + (b ? 16 : 0) * PITCH + (b == 1 ? 48 : 32); };
    const bool lower = (warp >> 1) == par;          // makes A
    const int dec_warp = 2 - 2 * par;               // makes the decays
    float g0 = 0.f, g1 = 0.f, b0 = 0.f, b1 = 0.f;   // of tokens 2 lane, 2 lane + 1
    auto fetch = [&](int c) {
        const long long t = (long long)c * C + 2 * lane;
        g0 = g1 = b0 = b1 = 0.f;
        if (t < len) {
            g0 = p.g[p.g_per_token ? (t0 + t) * p.H + h : h];
            b0 = p.beta[(t0 + t) * p.H + h];
        }
        if (t + 1 < len) {
            g1 = p.g[p.g_per_token ? (t0 + t + 1) * p.H + h : h];
            b1 = p.beta[(t0 + t + 1) * p.H + h];
        }
    };
    auto decays = [&](Decays &d) {
        const float x0 = g0 < -128.f ? -128.f : g0, x1 = g1 < -128.f ? -128.f : g1;
        float h0 = rintf(x0 * 1024.f), h1 = rintf(x1 * 1024.f);
        float l0 = x0 - h0 * (1.f / 1024), l1 = x1 - h1 * (1.f / 1024);
        h1 += h0;
        l1 += l0;
        float hs = h1, ls = l1;   // inclusive sums over lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float a = __shfl_up_sync(0xffffffffu, hs, o), b = __shfl_up_sync(0xffffffffu, ls, o);
            if (lane >= o) {
                hs += a;
                ls += b;
            }
        }
        const float hb = hs - h1, lb = __shfl_up_sync(0xffffffffu, ls, 1);   // before this lane
        const float before = lane ? lb : 0.f;
        const float2 a = make_float2(hb + h0, LOG2E * (before + l0)), b = make_float2(hs, LOG2E * ls);
        const float eh = __shfl_sync(0xffffffffu, b.x, 31), el = __shfl_sync(0xffffffffu, b.y, 31);
        const float bh = __shfl_sync(0xffffffffu, b.x, lane | 7), bl = __shfl_sync(0xffffffffu, b.y, lane | 7);
        auto weight = [](float hh, float ll) { return exp2_fast(fmaf(hh, LOG2E / 1024, ll)); };
        const float e0 = weight(a.x, a.y), e1 = weight(b.x, b.y);
        reinterpret_cast<float2 *>(d.gh)[lane] = make_float2(a.x, b.x);
        reinterpret_cast<float2 *>(d.gl)[lane] = make_float2(a.y, b.y);
        reinterpret_cast<float2 *>(d.suf)[lane] = make_float2(weight(bh - a.x, bl - a.y), weight(bh - b.x, bl - b.y));
        reinterpret_cast<float2 *>(d.beta)[lane] = make_float2(b0, b1);
        reinterpret_cast<float2 *>(d.neg)[lane] = make_float2(-e0, -e1);
        reinterpret_cast<float2 *>(d.gam)[lane] = make_float2(p.scale * e0, p.scale * e1);
        reinterpret_cast<float2 *>(d.lat)[lane] = make_float2(weight(eh - a.x, el - a.y), weight(eh - b.x, el - b.y));
        // The state's own decay in two parts: rounded to fp32 itself, a decay that stays the same would be off the
        // same way chunk after chunk (8192 tokens of g = -7.6e-4: 3.8e-6 of the state, 65536 of -1e-4: 4.2e-5).  Near 1
        // it is 1 + m, m by Taylor's series (what is left of it, G^9 / 9!, is below 6e-9; expm1f and expf here cost 1.5 % of
        // the kernel, this at most 0.6 %); a decay far from 1 is forgotten within two chunks.
        if (lane == 31) {
            const float G = fmaf(hs, 1.f / 1024, ls);
            float y = fmaf(G, 1.f / 40320, 1.f / 5040);
            y = fmaf(G, y, 1.f / 720);
            y = fmaf(G, y, 1.f / 120);
            y = fmaf(G, y, 1.f / 24);
            y = fmaf(G, y, 1.f / 6);
            y = fmaf(G, y, 0.5f);
            const float m = fmaf(G * G, y, G);
            const bool near = fabsf(G) < 0.5f;
            const float total = near ? 1.f + m : e1;
            d.total = total;
            d.less = near ? m - (total - 1.f) : 0.f;
        }
    };
    if (warp == dec_warp && par < nch) fetch(par);
    bool ok = true;
    for (int c = par; c < nch; c += 2) {
        const int stage = c % STAGES;
        Decays &d = sh->dec[c % DECS];
        ok = ok && wait_warp(sh, B_KQ_FULL + stage, c / STAGES);
        const long long n = len - (long long)c * C;
        if (ok && n < C) {   // rows of other sequences: 0 x NaN must not get into the products
            uint8_t *tile = smem + SM_KQ + stage * 2 * REGION;
#pragma unroll 1
            for (int x = tid; x < (C - (int)n) * 8 * 2 * regions; x += 128) {
                const int r = x / (16 * (C - (int)n)), y = x % (16 * (C - (int)n));   // region; k then q rows
                const int row = (int)n + y / 8 % (C - (int)n), q = y / (8 * (C - (int)n));
                *reinterpret_cast<uint4 *>(tile + r * REGION + q * TILE + row * 128 + y % 8 * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
        }
        if (ok) arrive(sh, B_K_READY + stage, lane);
        if (warp == dec_warp) {
            decays(d);
            if (c + 2 < nch) fetch(c + 2);
            if (ok) arrive(sh, B_DEC_READY + c % DECS, lane);
        }
        if (!bar_and(bar, 128, ok)) break;   // the four warps leave together (and the last T of theirs is read)
        ok = wait_warp(sh, B_GRAM_DONE + par, c >> 1);
        if (!lower) ok = ok && (c < P_TILES || wait_warp(sh, B_P_FREE + c % P_TILES, c / P_TILES - 1));
        if (ok) {
            tc_fence_after();
            const int row = 32 * (warp & 1), i = row + lane;
            const float gh = d.gh[i], gl = d.gl[i];
            const float f = lower ? d.beta[i] : p.scale;
            float *arow = A + i * PITCH;
            uint8_t *ptile = smem + SM_P + c % P_TILES * TILE;
#pragma unroll 1
            for (int x = 0; x < row + 32; x += 16) {
                uint32_t r[16];
                tmem_ld16(tq + x, r);
                float y[16];
                const int last = i - x - lower;   // A is strictly lower, P has its diagonal
                // w_ij through the end of j's 16 tokens: in i's own 16 a factor above 1 and one below, as long
                // as neither nears the end of its range
                if (x < row || d.gh[x] - d.gh[x + 15] < 64.f * 1024) {
                    const float to = f * exp2_fast(fmaf(gh - d.gh[x + 15], LOG2E / 1024, gl - d.gl[x + 15]));
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 s = *reinterpret_cast<const float4 *>(&d.suf[x + e]);
                        const float2 a = mul2(mul2(make_float2(s.x, s.y), make_float2(to, to)), as_pair(r[e], r[e + 1]));
                        const float2 b = mul2(mul2(make_float2(s.z, s.w), make_float2(to, to)), as_pair(r[e + 2], r[e + 3]));
                        y[e] = a.x; y[e + 1] = a.y; y[e + 2] = b.x; y[e + 3] = b.y;
                    }
                } else {
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const float4 jh = *reinterpret_cast<const float4 *>(&d.gh[x + e]), jl = *reinterpret_cast<const float4 *>(&d.gl[x + e]);
                        const float hs[4] = {jh.x, jh.y, jh.z, jh.w}, ls[4] = {jl.x, jl.y, jl.z, jl.w};
#pragma unroll
                        for (int m = 0; m < 4; ++m)
                            y[e + m] = exp2_fast(fmaf(gh - hs[m], LOG2E / 1024, gl - ls[m])) * (f * __uint_as_float(r[e + m]));
                    }
                }
                if (x >= row) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) y[e] = e <= last ? y[e] : 0.f;
                }
                if (x >= row + 16 && lane < 16) continue;   // above the diagonal's block
                if (lower) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<float4 *>(arow + x + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; e += 8)
                        *reinterpret_cast<uint4 *>(ptile + sw128(i, 2 * (x + e))) =
                            make_uint4(pack_bf16x2(y[e], y[e + 1]), pack_bf16x2(y[e + 2], y[e + 3]), pack_bf16x2(y[e + 4], y[e + 5]),
                                       pack_bf16x2(y[e + 6], y[e + 7]));
                }
            }
            __syncwarp();
            tc_fence_before();
            if (!lower) fence_proxy_async_smem();
            arrive(sh, B_GRAM_FREE, lane);
            if (!lower && lane == 0) mbar_arrive(&sh->bars[B_P_READY + c % P_TILES]);
            if (lower) diagonal(A, turned, 32 * (warp & 1), lane);
        }
        if (!bar_and(bar, 128, ok)) break;
        {   // the 32 x 32 blocks, two warps each: Y = B P^-1, and Q^-1 Y
            const int o = 32 * (warp >> 1), n = 8 * (warp & 1);
            float y[1][4];
            products(A + (o + 16) * PITCH + o, turned(o >> 4) + n * PITCH, 16, y);
            float *to = A + (o + n + q) * PITCH + o + 16 + r;
            to[0] = y[0][0];
            to[PITCH] = y[0][1];
            to[8] = y[0][2];
            to[PITCH + 8] = y[0][3];
            named_bar_sync(bar, 128);
            products(A + (o + 16) * PITCH + o + 16, A + (o + n) * PITCH + o + 16, 16, y);
            to = A + (o + 16 + r) * PITCH + o + n + q;
            *reinterpret_cast<float2 *>(to) = make_float2(-y[0][0], -y[0][1]);
            *reinterpret_cast<float2 *>(to + 8 * PITCH) = make_float2(-y[0][2], -y[0][3]);
            if (o == 0) {
                to = A + (n + q) * PITCH + 48 + r;
                to[0] = -y[0][0];
                to[PITCH] = -y[0][1];
                to[8] = -y[0][2];
                to[PITCH + 8] = -y[0][3];
            }
        }
        named_bar_sync(bar, 128);
        {   // the 64 x 64 block, 16 rows and columns a warp
            const int m = 16 * (warp & 1), n = 16 * (warp >> 1);
            float y[2][4];
            products(A + (32 + m) * PITCH + n, A + n * PITCH + 32 + n, 32 - n, y);   // (P^-1 is 0 above its diagonal)
            named_bar_sync(bar, 128);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float *to = A + (n + 8 * x + q) * PITCH + 32 + m + r;
                to[0] = y[x][0];
                to[PITCH] = y[x][1];
                to[8] = y[x][2];
                to[PITCH + 8] = y[x][3];
            }
            named_bar_sync(bar, 128);
            products(A + (32 + m) * PITCH + 32, A + n * PITCH + 32, 16 + m, y);      // (nor is Q^-1)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float *to = A + (32 + m + r) * PITCH + n + 8 * x + q;
                *reinterpret_cast<float2 *>(to) = make_float2(-y[x][0], -y[x][1]);
                *reinterpret_cast<float2 *>(to + 8 * PITCH) = make_float2(-y[x][2], -y[x][3]);
            }
        }
        ok = c < 2 || wait_warp(sh, B_T_FREE + par, (c >> 1) - 1);
        if (!bar_and(bar, 128, ok)) break;
        // Columns times beta, in three bf16 parts, eight columns at a time up to the diagonal's: nine such units in rows
        // i and 63 - i together.
#pragma unroll 1
        for (int u = warp; u < 9; u += 4) {
            const int m = (lane >> 3) + 1, i = u < m ? lane : 63 - lane, j = 8 * (u < m ? u : u - m);
            const float4 a = *reinterpret_cast<const float4 *>(A + i * PITCH + j), b = *reinterpret_cast<const float4 *>(A + i * PITCH + j + 4);
            const float4 f = *reinterpret_cast<const float4 *>(&d.beta[j]), g = *reinterpret_cast<const float4 *>(&d.beta[j + 4]);
            float2 y[4] = {make_float2(a.x * f.x, a.y * f.y), make_float2(a.z * f.z, a.w * f.w),
                           make_float2(b.x * g.x, b.y * g.y), make_float2(b.z * g.z, b.w * g.w)};
            uint32_t two[8], lo[4];
            split3(y, two, lo);
            const uint32_t at = sw128(i, 2 * j);
            *reinterpret_cast<uint4 *>(parts + at) = make_uint4(two[0], two[1], two[2], two[3]);
            *reinterpret_cast<uint4 *>(parts + TILE + at) = make_uint4(two[4], two[5], two[6], two[7]);
            *reinterpret_cast<uint4 *>(parts + 2 * TILE + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async_smem();
        arrive(sh, B_T_READY + par, lane);
    }
    if (!ok) give_up(sh);
}

template <typename TO, int REGIONS>
__global__ void __launch_bounds__(kThreads, 1)
delta_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv, const Args p)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared *sh = reinterpret_cast<Shared *>(smem + SM_SHARED);
    const int warp = threadIdx.x >> 5;
    const int seq = blockIdx.x / p.H, h = blockIdx.x % p.H;
    if ((smem_u32(smem) & 1023u) != 0) {   // the swizzle's atoms; the runtime honours the declaration
        if (threadIdx.x == 0) atomicExch(&g_delta_tc_error, KDA_ERR_DEVICE_BOUNDS);
        return;
    }
    if (threadIdx.x == 0) {
        for (int b = 0; b < B_COUNT; ++b) {
            int n = 1;
            if (b >= B_K_READY && b < B_K_FREE) n = 4;
            if (b == B_V_READY || b == B_R_READY || b == B_R_READY + 1 || b == B_UP_READY || b == B_UP_READY + 1) n = 8;
            if (b >= B_S_READY && b < B_X_DONE) n = 8;
            if (b == B_GRAM_FREE || b == B_O1_READY || b == B_O2_FREE) n = 4;
            if (b >= B_P_READY && b < B_P_FREE) n = 2;
            if (b == B_T_READY || b == B_T_READY + 1) n = 4;
            mbar_init(&sh->bars[b], n);
        }
        sh->abort = 0;
        sh->zero = 0;
        fence_barrier_init();
        tma_prefetch_desc(&mq);
        tma_prefetch_desc(&mk);
        tma_prefetch_desc(&mv);
    }
    // what stands above the diagonals of T's parts and of P stays 0
    static_assert(SM_P == SM_T + 6 * TILE, "one range");
    for (int x = threadIdx.x; x < (6 + P_TILES) * (int)TILE / 16; x += kThreads) reinterpret_cast<uint4 *>(smem + SM_T)[x] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    if (warp == 20) {
        tmem_alloc(&sh->tmem, TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (sh->tmem != 0) {   // (the whole of it starts at 0)
        if (threadIdx.x == 0) atomicExch(&g_delta_tc_error, KDA_ERR_DEVICE_BOUNDS);
        if (warp == 20) tmem_dealloc(sh->tmem, TM_COLS);
        return;
    }
    long long t0, t1;
    bounds(p, seq, t0, t1);
    const long long len = t1 - t0;
    const int nch = (int)((len + C - 1) / C);
    if (warp < 8) {
        set_regs<kRegsChain>();
        chain_role<REGIONS>(p, smem, sh, seq, h, len, nch);
    } else if (warp < 12) {
        set_regs<kRegsOut>();
        output_role<TO>(p, sh, h, t0, len, nch);
    } else if (warp < 20) {
        set_regs<kRegsPrep>();
        prep_role(p, smem, sh, h, REGIONS, t0, len, nch);
    } else {
        set_regs<kRegsIssue>();
        if (warp == 20) load_role(&mq, &mk, &mv, smem, sh, h, h / p.group, REGIONS, t0, nch);
        if (warp == 21) gram_mma_role<REGIONS>(smem_u32(smem), sh, nch);
        if (warp == 22) chain_mma_role<REGIONS>(smem_u32(smem), sh, nch);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 20) tmem_dealloc(0, TM_COLS);
    if (threadIdx.x == 0) record(sh);
}

// One warp whose wait is for a phase that nothing completes: it gives up after `cycles`, and the end
// records it, both as in the kernel above.
__global__ void delta_timeout_probe_kernel(uint32_t cycles)
{
    __shared__ Shared sh;
    if (threadIdx.x == 0) {
        mbar_init(&sh.bars[B_KQ_FULL], 1);
        sh.abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (!wait_warp(&sh, B_KQ_FULL, 0, cycles)) give_up(&sh);
    __syncthreads();
    if (threadIdx.x == 0) record(&sh);
}

// ---------------------------------------------------------------------------------------------
// host side

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// [T, heads, d] bf16: box = 64 channels x 1 head x 64 tokens, 128-byte swizzle; channels past d and tokens past T
// read as zeros
bool make_map(CUtensorMap *map, const void *base, int heads, int d, long long T)
{
    auto enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)heads * d * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)C}, es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename TO, int REGIONS>
int launch(const CUtensorMap *m, const Args &p, cudaStream_t stream)
{
    // a function attribute belongs to the current device: set it on every launch
    if (cudaFuncSetAttribute(delta_tc_kernel<TO, REGIONS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SM_BYTES) !=
        cudaSuccess)
        return KDA_ERR_CUDA;
    delta_tc_kernel<TO, REGIONS><<<(unsigned)(p.n_seqs * p.H), kThreads, SM_BYTES, stream>>>(m[0], m[1], m[2], p);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

int run_tc_path(const Args &p, int out_dtype, cudaStream_t stream)
{
    CUtensorMap m[3];
    if (!make_map(&m[0], p.q, p.H / p.group, p.dk, p.T) ||
        !make_map(&m[1], p.k, p.H / p.group, p.dk, p.T) ||
        !make_map(&m[2], p.v, p.H, p.dv, p.T))
        return KDA_ERR_CUDA;
    if (p.dk <= 64) return out_dtype == KDA_BF16 ? launch<__nv_bfloat16, 1>(m, p, stream) : launch<float, 1>(m, p, stream);
    return out_dtype == KDA_BF16 ? launch<__nv_bfloat16, 2>(m, p, stream) : launch<float, 2>(m, p, stream);
}

}  // namespace delta

int launch_delta_timeout_probe(uint32_t cycles, cudaStream_t stream)
{
    delta::delta_timeout_probe_kernel<<<1, 32, 0, stream>>>(cycles);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int *status_word_delta()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, delta::g_delta_tc_error) == cudaSuccess ? static_cast<int *>(p) : nullptr;
}

}  // namespace kda
