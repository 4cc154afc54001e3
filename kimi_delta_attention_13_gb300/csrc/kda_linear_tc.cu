// kda_linear_tc.cu -- linear attention with one decay per head for bf16 operands: chunks of 128
// tokens on the tensor cores.
//
//     S_t = exp(g_t) S_(t-1) + k_t v_t^T,     o_t = scale S_t^T q_t
//
// With a_t = exp(g_t) and a chunk that starts from state S (rows i, j = tokens of the chunk):
//     o_i = scale ( p_i S^T q_i  +  sum_(j <= i) w_ij (q_i . k_j) v_j )
//     S  <- (prod a) S  +  sum_j c_j k_j v_j^T
//     p_i = prod_(l <= i) a_l,   w_ij = prod_(j < l <= i) a_l,   c_j = prod_(l > j) a_l
// Four products a chunk, M = 128 each, accumulated in fp32 in TMEM:
//     scores = Q K^T         A, B = q, k tiles in shared memory
//     D2 = P V               A = P = w . scores (bf16, TMEM), B = v tile
//     D1 = Q S               B = the state as bf16 (shared memory)
//     Dst = K^T V~           B = V~ = c . v, split in three bf16 parts (three passes)
// The state itself stays in fp32 registers: S <- (prod a) S + Dst.  Its update must be good to fp32,
// so V~ keeps the 24 bits of its fp32 products (two parts, 16 bits, left states 4e-6 off against 1e-7, and
// took 188 us in place of 210 at T = 8192, H = 96); P and the state's copy are rounded to bf16 once each
// (their products make the outputs, to which a bf16 rounding of the result is added anyway).
//
// Every weight is made of the decays of the very tokens it spans, never as a quotient or a difference of
// sums, so any decay in [0, 1] is safe: w_ij = (suffix of j's 32-token block after j) x (whole blocks
// between) x (prefix of i's block up to i).  What goes into the state (suffixes and whole blocks) is the
// exponential of a block's own sum of log decays: a product of 32 rounded factors is off by all their
// roundings, which for a constant decay are alike (a memory of 256 tokens: 2.7e-6 of the state, so 5e-7).
// What a bf16 operand or output takes (prefixes, and inside a block a running product from the
// diagonal down) is a product.
//
// One CTA works through the chunks of one (segment, head).  Roles, joined by mbarriers:
//   warps 0-7    the state update: 64 (dv = 128) state columns of one key channel per thread, and the
//                state's bf16 copy
//   warps 8-15   the chunk's outputs, scale (p D1 + D2) -> global
//   warps 16-19  scores -> P, one token row per thread
//   warps 20-23  the chunk's decays, and V~
//   warp 24      TMA loads: q and k one tile, v two;  warps 25, 26, 27  issue Q K^T and P V;  K^T V~;  Q S
// Three issuing warps, because scores, state and outputs of neighbouring chunks overlap.
//
// What bounds it.  Bytes: 1 KB a token and head at d = 128 (T = 8192, H = 96: 815 MB, 120 us at the
// measured copy rate).  Measured: 0.210 ms there (0.57 of that rate) on 96 of the 152 SMs, 6300 cycles a
// chunk.  Shared memory's data path is 81 % busy: a product of two tiles in shared memory reads 8 KB in its
// 64 cycles, all that the path carries, and the row work (V~, the state's copy, v) moves as much again
// as a third of that.  The tensor pipe is 45 % busy.  With outputs TMEM is full (scores and P 128
// columns, D1, D2, Dst 128 each), so scores have one buffer, and shared memory leaves room for one tile of
// q and k and two pieces of V~, so two cycles of about a chunk's time run side by side: Q K^T -> P -> P V ->
// Q K^T, and V~ -> K^T V~ -> V~, joined by the one K tile (the next one is fetched after K^T V~).
// What was tried: one more set of warps on V~ (32 warps): 0.224 ms; pieces made by pairs of warps:
// 0.240; k fetched by quarters as they fall free: 0.219; decays in four buffers: 0.213; V~ split in
// packed bf16 arithmetic, 12 instructions a pair: 0.245; pieces made before their place is free: 0.229;
// outputs staged for TMA stores, polling or sleeping waits: no gain; the roles' loops unrolled: 1.2 times
// the time, with six times the instruction-cache misses, so loops here are rolled where registers allow
// and waits are a few instructions.
// Few heads: the sequences are cut so that up to 152 CTAs work side by side, which costs a second read
// of k and v (T = 65536, H = 8: 0.173 ms, with an initial state 0.181, 71 us of it the states, against
// 1.51 ms uncut).
#include <cudaTypedefs.h>

#include <mutex>

#include "kda_linear.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace lin {
namespace {

using namespace ptx;

constexpr int C = 128;                          // tokens of a chunk
constexpr int kThreads = 7 * 128;
// Registers a thread of each warpgroup, 72 at launch: 2 x 88 + 2 x 56 + 64 + 88 + 64 = 7 x 72 with
// outputs, 2 x 104 + 2 x 24 + 88 + 88 + 64 < 7 x 72 for states alone.  What does not fit spills to local
// memory (8 to 16 bytes in the builds that have any), and with this much
// shared memory nearly every reload of it comes from L2.
constexpr int kRegsState[2] = {104, 88}, kRegsOut[2] = {24, 56}, kRegsScore[2] = {88, 64};
constexpr int kRegsValue[2] = {88, 88}, kRegsIssue = 64;
template <int N>
__device__ __forceinline__ void set_regs()
{
    if constexpr (N > 72) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

constexpr long long kTimeout = 4000000000ll;    // bounded waits for work in flight at an end: 4e9 SM cycles (~2 s)
constexpr uint32_t kWaitCycles = 2000000000u;   // bounded waits between roles: 2e9 SM cycles (~1 s)
constexpr uint32_t kSleepNs = 100000;           // longest sleep between two looks at the clock
constexpr uint32_t REGION = C * 128;            // 64 channels x 128 tokens
constexpr int kQuarter = 32;                    // tokens of a piece of V~
constexpr uint32_t PIECE = kQuarter * 128;      // 64 channels of them

__device__ int g_linear_tc_error;               // sticky device error word of this translation unit

struct Decays {
    float a[C];        // decay of a token (1 past the segment's end)
    float suf[C];      // product of the decays after it in its block of 32
    float blk[4];      // a block's product
};

enum Bar {
    B_QFULL, B_KFULL, B_VFULL = B_KFULL + 2, B_SC_DONE = B_VFULL + 2, B_P_READY, B_PV_DONE, B_QS_DONE = B_PV_DONE + 2, B_VT_READY,
    B_VT_FREE = B_VT_READY + 3, B_KV_DONE = B_VT_FREE + 3, B_K_FREE, B_ST_READY = B_K_FREE + 2, B_DST_FREE,
    B_D2_FREE = B_DST_FREE + 2, B_DEC_READY = B_D2_FREE + 2, B_DRAIN = B_DEC_READY + 2, B_COUNT = B_DRAIN + 3
};

struct Shared {
    Decays dec[2];
    uint64_t bars[B_COUNT];
    uint32_t tmem;
    int abort;
    int zero;          // always 0: the abort flag of waits that must not give up early
};

// Shared memory: tiles of q (with outputs), k (two for states alone), v (two), places for V~'s pieces, the
// state's copy (with outputs).
template <int DK, int DV, bool OUT>
struct Layout {
    static constexpr uint32_t KT = DK / 64 * REGION, VT = DV / 64 * REGION;
    static constexpr int KS = OUT ? 1 : 2, PLACES = OUT ? 2 : 3;
    static constexpr uint32_t PART = DV / 64 * PIECE, PLACE = 3 * PART;   // the hi, mid and lo parts of a piece
    static constexpr uint32_t Q = 0, K = OUT ? KT : 0, V = K + KS * KT, W = V + 2 * VT, S = W + PLACES * PLACE;
    static constexpr uint32_t SREG = DK * 128;   // the state copy: 64 value channels x DK key channels
    static constexpr uint32_t SHARED = OUT ? S + DV / 64 * SREG : S;
    static constexpr uint32_t BYTES = SHARED + sizeof(Shared);
};
static_assert(Layout<128, 128, true>::BYTES <= 232448 && Layout<128, 128, false>::BYTES <= 232448, "shared memory per block");
static_assert(Layout<128, 128, true>::PLACES <= 3 && Layout<128, 128, false>::PLACES <= 3, "barriers of the places");

constexpr uint32_t TM_SC = 0, TM_D2 = 128, TM_D1 = 256, TM_DST = 384, TM_COLS = 512;

__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

// Waits for phase `phase` of a barrier, giving up after `cycles` SM cycles (the clock's lower half, which
// takes 2^32 to come round): a role that gave up ends, the others, which stand at waits of their own by
// then, give up by the same rule, and the kernel's end records it.  As short as it can be, since it
// stands in some thirty places: the roles' loops together have to fit the instruction cache.
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

// How a role ends that a wait gave up in.
__device__ __forceinline__ void give_up(Shared *sh) { *reinterpret_cast<volatile int *>(&sh->abort) = 1; }

// wait for a whole warp: its lanes leave a loop together.
__device__ __forceinline__ bool wait_warp(Shared *sh, int bar, int phase, uint32_t cycles = kWaitCycles)
{
    return __all_sync(0xffffffffu, wait(sh, bar, phase, cycles));
}

// The kernel's end: one thread tells the device error word that a role gave up.
__device__ __forceinline__ void record(Shared *sh)
{
    if (sh->abort) atomicExch(&g_linear_tc_error, KDA_ERR_DEVICE_TIMEOUT);
}

// inclusive product over lanes 0 .. lane
__device__ __forceinline__ float scan_up(float x, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x *= y;
    }
    return x;
}

__device__ __forceinline__ uint4 zero4() { return make_uint4(0u, 0u, 0u, 0u); }

// products of two pairs (one instruction)
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    unsigned long long r, x, y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
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

// Two bf16 values times w as hi + mid + lo, exactly the fp32 products: 8 of their 24 bits a part, cut off,
// so that what a part leaves is exact.
__device__ __forceinline__ void split3(uint32_t x, float2 w, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    const float2 p = mul2(make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)), w);
    const uint32_t px = __float_as_uint(p.x), py = __float_as_uint(p.y);
    hi = __byte_perm(px, py, 0x7632);
    const float rx = p.x - __uint_as_float(px & 0xffff0000u), ry = p.y - __uint_as_float(py & 0xffff0000u);
    const uint32_t ux = __float_as_uint(rx), uy = __float_as_uint(ry);
    mid = __byte_perm(ux, uy, 0x7632);
    lo = __byte_perm(__float_as_uint(rx - __uint_as_float(ux & 0xffff0000u)),
                     __float_as_uint(ry - __uint_as_float(uy & 0xffff0000u)), 0x7632);
}

template <int DK, int DV, bool OUT>
__device__ void load_role(const CUtensorMap *mq, const CUtensorMap *mk, const CUtensorMap *mv, uint8_t *smem,
                          Shared *sh, int h, int hk, long long t0, int nch)
{
    using L = Layout<DK, DV, OUT>;
    auto load = [&](const CUtensorMap *m, uint32_t off, int bar, int regions, int head, int c) {
        if (elect_one()) {
            mbar_arrive_expect_tx(&sh->bars[bar], regions * REGION);
            for (int r = 0; r < regions; ++r)
                tma_load_3d(smem + off + r * REGION, m, &sh->bars[bar], 64 * r, head, (int)(t0 + (long long)c * C));
        }
        __syncwarp();
    };
    auto ahead = [&](const CUtensorMap *m, int regions, int head, int c) {   // into L2
        if (c < nch && elect_one())
            for (int r = 0; r < regions; ++r) tma_prefetch_l2_3d(m, 64 * r, head, (int)(t0 + (long long)c * C));
        __syncwarp();
    };
    auto value = [&](int c) { load(mv, L::V + (c & 1) * L::VT, B_VFULL + (c & 1), DV / 64, hk, c); };
    int nk = 0, nq = 0, nv = 1;   // tiles issued
    value(0);
    for (int c = 0; c < nch; ++c) {
        if constexpr (OUT) {
            if (c > 0 && !(wait_warp(sh, B_SC_DONE, c - 1) && wait_warp(sh, B_QS_DONE, c - 1))) break;
            load(mq, L::Q, B_QFULL, DK / 64, h, c);
            nq = c + 1;
            ahead(mq, DK / 64, h, c + 1);
        }
        if (OUT && c > 0 && !wait_warp(sh, B_K_FREE, c - 1)) break;   // (states alone: waited for with the last v)
        load(mk, L::K + c % L::KS * L::KT, B_KFULL + c % L::KS, DK / 64, hk, c);
        nk = c + 1;
        ahead(mk, DK / 64, hk, c + 1);
        if (c + 1 < nch) {
            if (c > 0 && !(OUT ? wait_warp(sh, B_PV_DONE + ((c - 1) & 1), (c - 1) >> 1)
                               : wait_warp(sh, B_K_FREE + ((c - 1) & 1), (c - 1) >> 1))) break;
            value(c + 1);
            nv = c + 2;
            ahead(mv, DV / 64, hk, c + 2);
        }
    }
    if (nk < nch || nv < nch) {   // no copy in flight when the CTA leaves
        for (int c = max(0, nk - L::KS); c < nk; ++c)
            mbar_wait(&sh->bars[B_KFULL + c % L::KS], c / L::KS & 1, &sh->zero, kTimeout);
        for (int c = max(0, nv - 2); c < nv; ++c)
            mbar_wait(&sh->bars[B_VFULL + (c & 1)], (c >> 1) & 1, &sh->zero, kTimeout);
        if (nq > 0) mbar_wait(&sh->bars[B_QFULL], (nq - 1) & 1, &sh->zero, kTimeout);
        return give_up(sh);
    }
}

// The issuing roles run as whole warps, one elected lane issuing, so that the descriptors stay in
// uniform registers: computed by a single lane they cost some 100 cycles a product.
template <int DK, int DV>
__device__ void score_mma_role(uint32_t sb, Shared *sh, uint32_t tm, int nch)
{
    using L = Layout<DK, DV, true>;
    constexpr uint32_t I_QK = idesc_bf16(128, 128, 0, 0), I_PV = idesc_bf16(128, DV, 0, 1);
    const uint64_t q = smem_desc(sb + L::Q, 0, 1024), k = smem_desc(sb + L::K, 0, 1024);
    bool ok = true;
    for (int c = 0; c < nch; ++c) {
        const int s = c & 1;
        // The scores take the columns of the last chunk's P, which its product with V reads as an operand.
        // Products that accumulate into different places are ordered by completion alone.
        ok = wait_warp(sh, B_QFULL, c) && wait_warp(sh, B_KFULL, c) &&
             (c == 0 || wait_warp(sh, B_PV_DONE + (s ^ 1), (c - 1) >> 1));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll 1
            for (int x = 0; x < DK / 16; ++x)
                mma_ss(tm + TM_SC, desc_at(q, (x >> 2) * REGION + (x & 3) * 32),
                       desc_at(k, (x >> 2) * REGION + (x & 3) * 32), I_QK, x > 0);
            mma_commit(&sh->bars[B_SC_DONE]);
        }
        __syncwarp();
        ok = wait_warp(sh, B_P_READY, c) && wait_warp(sh, B_VFULL + s, c >> 1) &&
             (c == 0 || wait_warp(sh, B_D2_FREE + (s ^ 1), (c - 1) >> 1));
        if (!ok) break;
        tc_fence_after();
        const uint64_t v = smem_desc(sb + L::V + s * L::VT, REGION, 1024);
        if (elect_one()) {
#pragma unroll 1
            for (int x = 0; x < C / 16; ++x)
                mma_ts(tm + TM_D2, tm + TM_SC + 8 * x, desc_at(v, x * 2048), I_PV, x > 0);
            mma_commit(&sh->bars[B_PV_DONE + s]);
        }
        __syncwarp();
    }
    if (!ok) {
        if (elect_one()) mma_commit(&sh->bars[B_DRAIN]);
        mbar_wait(&sh->bars[B_DRAIN], 0, &sh->zero, kTimeout);
        give_up(sh);
    }
}

template <int DK, int DV, bool OUT>
__device__ void update_mma_role(uint32_t sb, Shared *sh, uint32_t tm, int nch)
{
    using L = Layout<DK, DV, OUT>;
    constexpr uint32_t I_KV = idesc_bf16(128, DV, 1, 1);
    const uint64_t k = smem_desc(sb + L::K, REGION, 1024), w = smem_desc(sb + L::W, PIECE, 1024);
    bool ok = true;
    for (int n = 0; n < 4 * nch; ++n) {
        const int c = n >> 2, y = 3 - (n & 3), place = n % L::PLACES;   // piece y of chunk c
        if ((n & 3) == 0)
            ok = wait_warp(sh, B_KFULL + c % L::KS, c / L::KS) &&
                 (c == 0 || wait_warp(sh, B_DST_FREE + ((c - 1) & 1), (c - 1) >> 1));
        ok = ok && wait_warp(sh, B_VT_READY + place, n / L::PLACES);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll 1
            for (int x = 0; x < kQuarter / 16; ++x) {
                const uint64_t a = desc_at(k, c % L::KS * L::KT + (y * (kQuarter / 16) + x) * 2048);
                const uint64_t b = desc_at(w, place * L::PLACE + x * 2048);
                mma_ss(tm + TM_DST, a, desc_at(b, 2 * L::PART), I_KV, (n & 3) + x > 0);
                mma_ss(tm + TM_DST, a, desc_at(b, L::PART), I_KV, 1);
                mma_ss(tm + TM_DST, a, b, I_KV, 1);
            }
            mma_commit(&sh->bars[B_VT_FREE + place]);
            if ((n & 3) == 3) {
                mma_commit(&sh->bars[B_KV_DONE]);
                mma_commit(&sh->bars[B_K_FREE + c % L::KS]);
            }
        }
        __syncwarp();
    }
    if (!ok) {
        if (elect_one()) mma_commit(&sh->bars[B_DRAIN + 1]);
        mbar_wait(&sh->bars[B_DRAIN + 1], 0, &sh->zero, kTimeout);
        give_up(sh);
    }
}

template <int DK, int DV>
__device__ void read_mma_role(uint32_t sb, Shared *sh, uint32_t tm, int nch)
{
    using L = Layout<DK, DV, true>;
    constexpr uint32_t I_QS = idesc_bf16(128, DV, 0, 1);
    const uint64_t q = smem_desc(sb + L::Q, 0, 1024), st = smem_desc(sb + L::S, L::SREG, 1024);
    bool ok = true;
    for (int c = 0; c < nch; ++c) {
        ok = wait_warp(sh, B_ST_READY, c) && wait_warp(sh, B_QFULL, c) &&
             (c == 0 || wait_warp(sh, B_D2_FREE + ((c - 1) & 1), (c - 1) >> 1));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll 1
            for (int x = 0; x < DK / 16; ++x)
                mma_ss(tm + TM_D1, desc_at(q, (x >> 2) * REGION + (x & 3) * 32), desc_at(st, x * 2048), I_QS, x > 0);
            mma_commit(&sh->bars[B_QS_DONE]);
        }
        __syncwarp();
    }
    if (!ok) {
        if (elect_one()) mma_commit(&sh->bars[B_DRAIN + 2]);
        mbar_wait(&sh->bars[B_DRAIN + 2], 0, &sh->zero, kTimeout);
        give_up(sh);
    }
}

// warps 16-19: thread = token row 32 blk + lane
template <int DK, int DV>
__device__ void score_role(uint8_t *smem, Shared *sh, uint32_t tm, long long len, int nch)
{
    using L = Layout<DK, DV, true>;
    const int blk = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, row = 32 * blk + lane;
    const uint32_t tq = tm + TM_SC + ((uint32_t)(32 * blk) << 16);
    for (int c = 0; c < nch; ++c) {
        if (!wait_warp(sh, B_SC_DONE, c) || !wait_warp(sh, B_DEC_READY + (c & 1), c >> 1)) return give_up(sh);
        const Decays &d = sh->dec[c & 1];
        tc_fence_after();
        uint32_t r[32], o[16];
        tmem_ld32(tq, r);
        const float pre = scan_up(d.a[row], lane);   // prefix of the row's own block
        float f = pre;
        for (int x = 1; x < blk; ++x) f *= d.blk[x];
        tmem_wait_ld();
        for (int j = 0; j < blk; ++j) {   // whole blocks before the row's own
            const float2 ff = make_float2(f, f);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const float4 w = reinterpret_cast<const float4 *>(d.suf + 32 * j)[x];
                const float2 p = mul2(make_float2(__uint_as_float(r[4 * x]), __uint_as_float(r[4 * x + 1])),
                                      mul2(ff, make_float2(w.x, w.y)));
                const float2 q = mul2(make_float2(__uint_as_float(r[4 * x + 2]), __uint_as_float(r[4 * x + 3])),
                                      mul2(ff, make_float2(w.z, w.w)));
                o[2 * x] = pack_bf16x2(p.x, p.y);
                o[2 * x + 1] = pack_bf16x2(q.x, q.y);
            }
            // P overwrites scores already read: columns 16 j .. 16 j + 15 of blocks <= j
            tmem_st16(tq + 16 * j, o);
            tmem_ld32(tq + 32 * (j + 1), r);
            f = pre;   // the factor of the next block spans one block less
            for (int x = j + 2; x < blk; ++x) f *= d.blk[x];
            tmem_wait_ld();
        }
        {
            float w = 1.f, odd = 0.f;
#pragma unroll
            for (int y = 7; y >= 0; --y) {   // from the diagonal down: w = product of a over (x, lane]
                const float4 a = reinterpret_cast<const float4 *>(d.a + 32 * blk)[y];
                const float ay[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int e = 3; e >= 0; --e) {
                    const int x = 4 * y + e;
                    const float p = x <= lane ? __uint_as_float(r[x]) * w : 0.f;
                    if (x & 1) odd = p;
                    else o[x / 2] = pack_bf16x2(p, odd);
                    if (x <= lane) w *= ay[e];
                }
            }
            tmem_st16(tq + 16 * blk, o);
        }
        if (blk < 3) {
            uint32_t o[16] = {};
            for (int j = blk + 1; j < 4; ++j) tmem_st16(tq + 16 * j, o);
        }
        tmem_wait_st();
        tc_fence_before();
        const long long n = len - (long long)c * C;
        if (n < C) {   // rows of other sequences: their P is 0, and 0 x NaN must not get in
            if (!wait_warp(sh, B_VFULL + (c & 1), c >> 1)) return give_up(sh);
            if (row >= n) {
                uint4 *v = reinterpret_cast<uint4 *>(smem + L::V + (c & 1) * L::VT + row * 128);
#pragma unroll 1
                for (int x = 0; x < DV / 8; ++x) v[(x >> 3) * (REGION / 16) + (x & 7)] = zero4();
            }
            fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->bars[B_P_READY]);
    }
}

// warps 20-23: the chunk's decays, and V~ in pieces of 32 tokens, a token a lane, the channels shared by
// the warps; for states alone warps 16-19 take half of the channels
template <int DK, int DV, bool OUT>
__device__ void value_role(const Args &p, uint8_t *smem, Shared *sh, int h, long long t0, long long len, int nch)
{
    using L = Layout<DK, DV, OUT>;
    constexpr int WARPS = OUT ? 4 : 8;
    constexpr int UNITS = DV / 8 / WARPS, KUNITS = DK / 8 / WARPS;   // 16-byte units of a row for this thread
    const int blk = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const bool main = OUT || threadIdx.x >= 20 * 32;
    const int share = OUT ? blk : (int)(threadIdx.x >> 5) - 16;
    auto log_decay = [&](int c) {
        const long long t = (long long)c * C + 32 * blk + lane;
        return t < len ? (p.g_per_token ? p.g[(t0 + t) * p.H + h] : p.g[h]) : 0.f;
    };
    float a, suf, all;   // of the lane's token and its block, made before their place is free
    auto make = [&](float g) {
        float rest = g;   // sum from this lane up, then without the lane's own
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_down_sync(0xffffffffu, rest, o);
            if (lane + o < 32) rest += y;
        }
        all = expf(rest);   // (of lane 0)
        rest = __shfl_down_sync(0xffffffffu, rest, 1);
        suf = expf(lane == 31 ? 0.f : rest);
        a = expf(g);
    };
    auto put = [&](int c) {
        Decays &d = sh->dec[c & 1];
        if (lane == 0) d.blk[blk] = all;
        d.a[32 * blk + lane] = a;
        d.suf[32 * blk + lane] = suf;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->bars[B_DEC_READY + (c & 1)]);
    };
    // unit x of a row (row % 8 = lane % 8) in a tile whose regions of 64 channels are `region` bytes, in an
    // order that keeps eight rows' accesses in different banks
    auto at = [&](int x, uint32_t region) { return (x >> 3) * (int)(region / 16) + ((x & 7) ^ (lane & 7)); };
    float g = log_decay(0);
    if constexpr (OUT) {
        make(g);
        put(0);
        g = nch > 1 ? log_decay(1) : 0.f;
    }
    for (int c = 0; c < nch; ++c) {
        if (!OUT && main) {   // the place was chunk c - 2's, whose pieces and state are made
            make(g);
            if (c > 1 && !wait_warp(sh, B_DST_FREE + (c & 1), (c - 2) >> 1)) return give_up(sh);
            put(c);
            if (c + 1 < nch) g = log_decay(c + 1);
        }
        if (!wait_warp(sh, B_DEC_READY + (c & 1), c >> 1) || !wait_warp(sh, B_VFULL + (c & 1), c >> 1)) return give_up(sh);
        if ((long long)(c + 1) * C > len && !wait_warp(sh, B_KFULL + c % L::KS, c / L::KS)) return give_up(sh);
        const Decays &d = sh->dec[c & 1];
        float later = 1.f;   // the product over the blocks after the piece
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {   // from the last tokens back
            const int y = 3 - x, n = 4 * c + x, place = n % L::PLACES, row = 32 * y + lane;
            const uint4 *v = reinterpret_cast<const uint4 *>(smem + L::V + (c & 1) * L::VT + row * 128);
            uint4 *to = reinterpret_cast<uint4 *>(smem + L::W + place * L::PLACE + lane * 128);
            const bool live = (long long)c * C + row < len;
            uint4 in[UNITS];
#pragma unroll
            for (int i = 0; i < UNITS; ++i) in[i] = v[at(share * UNITS + i, REGION)];
            const float f = d.suf[row] * later;
            later *= d.blk[y];
            const float2 w = make_float2(f, f);
            if (n >= L::PLACES && !wait_warp(sh, B_VT_FREE + place, n / L::PLACES - 1)) return give_up(sh);
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                uint4 hi, mid, lo;
                if (!live) in[i] = zero4();   // a row of another sequence: 0 x NaN must not get into the state
                split3(in[i].x, w, hi.x, mid.x, lo.x);
                split3(in[i].y, w, hi.y, mid.y, lo.y);
                split3(in[i].z, w, hi.z, mid.z, lo.z);
                split3(in[i].w, w, hi.w, mid.w, lo.w);
                uint4 *u = to + at(share * UNITS + i, PIECE);
                u[0] = hi;
                u[L::PART / 16] = mid;
                u[2 * (L::PART / 16)] = lo;
            }
            if (!live) {
                uint4 *k = reinterpret_cast<uint4 *>(smem + L::K + c % L::KS * L::KT + row * 128);
#pragma unroll
                for (int i = 0; i < KUNITS; ++i) k[at(share * KUNITS + i, REGION)] = zero4();
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->bars[B_VT_READY + place]);
        }
        if constexpr (OUT) {
            if (c + 1 < nch) {   // the place was chunk c - 1's, whose P and outputs are made
                const int s = (c - 1) & 1, e = (c - 1) >> 1;
                make(g);
                if (c > 0 && !(wait_warp(sh, B_D2_FREE + s, e) && wait_warp(sh, B_DST_FREE + s, e))) return give_up(sh);
                put(c + 1);
                if (c + 2 < nch) g = log_decay(c + 2);
            }
        }
    }
}

// 16 bytes of an output row from consecutive fp32 values
template <typename TO>
__device__ __forceinline__ uint4 pack16(const float *v)
{
    if constexpr (sizeof(TO) == 2)
        return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    else
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}

__device__ __forceinline__ uint4 swap16(uint4 a, int mask)
{
    a.x = __shfl_xor_sync(0xffffffffu, a.x, mask);
    a.y = __shfl_xor_sync(0xffffffffu, a.y, mask);
    a.z = __shfl_xor_sync(0xffffffffu, a.z, mask);
    a.w = __shfl_xor_sync(0xffffffffu, a.w, mask);
    return a;
}

// u[x] of lane m holds unit x of row m (rows of a quad of lanes): afterwards unit m of row x.
__device__ __forceinline__ void transpose4(uint4 (&u)[4], int lane)
{
#pragma unroll
    for (int bit = 1; bit <= 2; bit <<= 1) {
        const bool up = lane & bit;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (x & bit) continue;
            const uint4 got = swap16(up ? u[x] : u[x | bit], bit);
            if (up) u[x] = got;
            else u[x | bit] = got;
        }
    }
}

// warps 0-7: thread = key channel 32 (warp % 4) + lane, value channels [DV/2 half, +DV/2)
template <int DK, int DV, bool OUT>
__device__ void state_role(const Args &p, uint8_t *smem, Shared *sh, uint32_t tm, const Item &it, int item, int h,
                           int nch)
{
    using L = Layout<DK, DV, OUT>;
    constexpr int N = DV / 2;
    const int warp = threadIdx.x >> 5, blk = warp & 3, half = warp >> 2, lane = threadIdx.x & 31;
    const int row = 32 * blk + lane, c0 = half * N;
    const uint32_t tq = tm + ((uint32_t)(32 * blk) << 16) + c0;
    const bool row_ok = row < p.dk;
    const long long unit = (long long)p.dk * p.dv, at = (long long)row * p.dv + c0;
    const long long own = ((long long)it.seq * p.H + h) * unit + at, slot = ((long long)item * p.H + h) * unit + at;
    const float *from = it.seg == 0 && p.init ? p.init + own : nullptr;
    if (OUT && it.nseg > 1 && (it.seg > 0 || p.init)) from = p.starts + slot;
    float st[N];
#pragma unroll
    for (int x = 0; x < N; x += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (from && row_ok && c0 + x < p.dv) v = *reinterpret_cast<const float4 *>(from + x);
        st[x] = v.x; st[x + 1] = v.y; st[x + 2] = v.z; st[x + 3] = v.w;
        // a first segment's start is kept: the last segment may overwrite it (final_state = init)
        if (!OUT && it.seg == 0 && p.init && row_ok && c0 + x < p.dv)
            *reinterpret_cast<float4 *>(p.starts + slot + x) = v;
    }
    auto copy_state = [&] {   // bf16 copy, rows = key channels, 64 value channels per region
        if (row < DK) {
#pragma unroll
            for (int x = 0; x < N; x += 8) {
                uint4 u;
                u.x = pack_bf16x2(st[x], st[x + 1]);
                u.y = pack_bf16x2(st[x + 2], st[x + 3]);
                u.z = pack_bf16x2(st[x + 4], st[x + 5]);
                u.w = pack_bf16x2(st[x + 6], st[x + 7]);
                const int col = c0 + x;
                *reinterpret_cast<uint4 *>(smem + L::S + (col >> 6) * L::SREG + sw128(row, (col & 63) * 2)) = u;
            }
        }
        fence_proxy_async_smem();
    };
    auto arrive = [&](int bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->bars[bar]);
    };
    if constexpr (OUT) {
        copy_state();
        arrive(B_ST_READY);
    }
    float whole = 1.f;
    for (int c = 0; c < nch; ++c) {
        if (!wait_warp(sh, B_DEC_READY + (c & 1), c >> 1)) return give_up(sh);
        const Decays &d = sh->dec[c & 1];
        const float tot = d.blk[0] * d.blk[1] * d.blk[2] * d.blk[3];
        whole *= tot;
        if (!wait_warp(sh, B_KV_DONE, c)) return give_up(sh);
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < N; x += 16) {
            uint32_t r[16];
            tmem_ld16(tq + TM_DST + x, r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) st[x + e] = fmaf(st[x + e], tot, __uint_as_float(r[e]));
        }
        tc_fence_before();
        arrive(B_DST_FREE + (c & 1));
        if constexpr (OUT) {
            if (!wait_warp(sh, B_QS_DONE, c)) return give_up(sh);
            if (c + 1 < nch) {
                copy_state();
                arrive(B_ST_READY);
            }
        }
    }
    float *to = nullptr;
    if (OUT) to = it.seg == it.nseg - 1 && p.final_state ? p.final_state + own : nullptr;
    else to = p.starts + slot + (long long)p.H * unit;
    if (to && row_ok) {
#pragma unroll
        for (int x = 0; x < N; x += 4)
            if (c0 + x < p.dv) *reinterpret_cast<float4 *>(to + x) = make_float4(st[x], st[x + 1], st[x + 2], st[x + 3]);
    }
    if (!OUT && threadIdx.x == 0) p.decays[(long long)item * p.H + h] = whole;
}

// warps 8-15: thread = token row 32 (warp % 4) + lane, value channels [DV/2 half, +DV/2)
template <int DV, typename TO>
__device__ void output_role(const Args &p, Shared *sh, uint32_t tm, const Item &it, int h, int nch)
{
    constexpr int N = DV / 2, UNIT = 16 / sizeof(TO), COLS = 4 * UNIT;
    const int warp = threadIdx.x >> 5, blk = warp & 3, lane = threadIdx.x & 31, row = 32 * blk + lane;
    const int c0 = ((warp >> 2) & 1) * N;
    const uint32_t tq = tm + ((uint32_t)(32 * blk) << 16) + c0;
    const long long len = it.t1 - it.t0, step = (long long)p.H * p.dv;
    // Rows leave in pieces of four 16-byte units: a quad of lanes, which holds four rows, turns its
    // units around so that it stores one row's four units side by side.  (A row per lane would touch
    // 32 rows an instruction.)
    long long t = row & ~3;
    TO *o = static_cast<TO *>(p.out) + ((it.t0 + t) * p.H + h) * p.dv + c0 + UNIT * (lane & 3);
    const int cols = p.dv - c0 - UNIT * (lane & 3);
    const float2 scale = make_float2(p.scale, p.scale);
    for (int c = 0; c < nch; ++c, t += C, o += C * step) {
        if (!wait_warp(sh, B_DEC_READY + (c & 1), c >> 1)) return give_up(sh);
        const Decays &d = sh->dec[c & 1];
        float f = p.scale * scan_up(d.a[row], lane);
        for (int x = 0; x < blk; ++x) f *= d.blk[x];
        const float2 pre = make_float2(f, f);
        if (!wait_warp(sh, B_QS_DONE, c) || !wait_warp(sh, B_PV_DONE + (c & 1), c >> 1)) return give_up(sh);
        tc_fence_after();
        const long long left = len - t;   // rows of the quad to store, may be <= 0
#pragma unroll 1
        for (int x = 0; x < N; x += COLS) {
            uint4 u[4];
#pragma unroll
            for (int y = 0; y < COLS; y += 8) {
                uint32_t r1[8], r2[8];
                float v[8];
                tmem_ld8(tq + TM_D1 + x + y, r1);
                tmem_ld8(tq + TM_D2 + x + y, r2);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 s2 = mul2(scale, make_float2(__uint_as_float(r2[e]), __uint_as_float(r2[e + 1])));
                    const float2 w = fma2(pre, make_float2(__uint_as_float(r1[e]), __uint_as_float(r1[e + 1])), s2);
                    v[e] = w.x;
                    v[e + 1] = w.y;
                }
#pragma unroll
                for (int e = 0; e < 8; e += UNIT) u[(y + e) / UNIT] = pack16<TO>(v + e);
            }
            if (x + COLS >= N) {   // everything is read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->bars[B_D2_FREE + (c & 1)]);
            }
            transpose4(u, lane);
#pragma unroll
            for (int y = 0; y < 4; ++y)
                if (y < left && x < cols) *reinterpret_cast<uint4 *>(o + y * step + x) = u[y];
        }
    }
}

template <int DK, int DV, typename TO, bool OUT>
__global__ void __launch_bounds__(kThreads, 1)
linear_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                 const __grid_constant__ CUtensorMap mv, const Args p)
{
    using L = Layout<DK, DV, OUT>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared *sh = reinterpret_cast<Shared *>(smem + L::SHARED);
    const int warp = threadIdx.x >> 5;
    const int h = blockIdx.x % p.H, item = blockIdx.x / p.H;
    const Item it = find_item(p.cu, p.n_seqs, p.T, p.seg_len, item);
    if (it.seq < 0 || (!OUT && (it.seg == it.nseg - 1 || item + 1 >= p.items))) return;   // (a bad table
    // could name more segments than there are places for)
    if ((smem_u32(smem) & 1023u) != 0) {   // the swizzle's atoms; the runtime honours the declaration
        if (threadIdx.x == 0) atomicExch(&g_linear_tc_error, KDA_ERR_DEVICE_BOUNDS);
        return;
    }
    if (threadIdx.x == 0) {
        for (int b = 0; b < B_COUNT; ++b) {
            int n = 1;
            if (b == B_P_READY || b == B_DEC_READY || b == B_DEC_READY + 1) n = 4;
            if (b >= B_VT_READY && b < B_VT_FREE) n = OUT ? 4 : 8;
            if (b >= B_ST_READY && b < B_DEC_READY) n = 8;
            mbar_init(&sh->bars[b], n);
        }
        sh->abort = 0;
        sh->zero = 0;
        fence_barrier_init();
        if (OUT) tma_prefetch_desc(&mq);
        tma_prefetch_desc(&mk);
        tma_prefetch_desc(&mv);
    }
    if (warp == 25) {
        tmem_alloc(&sh->tmem, TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sh->tmem;
    const long long len = it.t1 - it.t0;
    const int nch = (int)((len + C - 1) / C);
    if (warp < 8) {
        set_regs<kRegsState[OUT]>();
        state_role<DK, DV, OUT>(p, smem, sh, tm, it, item, h, nch);
    } else if (warp < 16) {
        set_regs<kRegsOut[OUT]>();
        if constexpr (OUT) output_role<DV, TO>(p, sh, tm, it, h, nch);
    } else if (warp < 20) {
        set_regs<kRegsScore[OUT]>();
        if constexpr (OUT) score_role<DK, DV>(smem, sh, tm, len, nch);
        else if (nch > 0) value_role<DK, DV, OUT>(p, smem, sh, h, it.t0, len, nch);
    } else if (warp < 24) {
        set_regs<kRegsValue[OUT]>();
        if (nch > 0) value_role<DK, DV, OUT>(p, smem, sh, h, it.t0, len, nch);
    } else {
        set_regs<kRegsIssue>();
        if (warp == 24 && nch > 0)
            load_role<DK, DV, OUT>(&mq, &mk, &mv, smem, sh, h, h / p.group, it.t0, nch);
        if (warp == 25 && OUT && nch > 0) score_mma_role<DK, DV>(smem_u32(smem), sh, tm, nch);
        if (warp == 26 && nch > 0) update_mma_role<DK, DV, OUT>(smem_u32(smem), sh, tm, nch);
        if (warp == 27 && OUT && nch > 0) read_mma_role<DK, DV>(smem_u32(smem), sh, tm, nch);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 25) tmem_dealloc(tm, TM_COLS);
    if (threadIdx.x == 0) record(sh);
}

// One warp whose wait is for a phase that nothing completes: it gives up after `cycles`, and the end
// records it, both as in the kernel above.
__global__ void linear_timeout_probe_kernel(uint32_t cycles)
{
    __shared__ Shared sh;
    if (threadIdx.x == 0) {
        mbar_init(&sh.bars[B_KFULL], 1);
        sh.abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (!wait_warp(&sh, B_KFULL, 0, cycles)) give_up(&sh);
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

// [T, heads, d] bf16: box = 64 channels x 1 head x 128 tokens, 128-byte swizzle; channels past d
// and tokens past T read as zeros
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

template <int DK, int DV, typename TO, bool OUT>
bool launch_one(const CUtensorMap *m, const Args &p, cudaStream_t stream)
{
    const int bytes = (int)Layout<DK, DV, OUT>::BYTES;
    // a function attribute belongs to the current device: set it on every launch
    if (cudaFuncSetAttribute(linear_tc_kernel<DK, DV, TO, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
        cudaSuccess)
        return false;
    linear_tc_kernel<DK, DV, TO, OUT><<<(unsigned)(p.items * p.H), kThreads, bytes, stream>>>(m[0], m[1], m[2], p);
    return cudaGetLastError() == cudaSuccess;
}

template <int DK, int DV>
int run_dims(const CUtensorMap *m, const Args &p, int out_dtype, cudaStream_t stream)
{
    if (p.seg_len > 0) {
        if (!launch_one<DK, DV, float, false>(m, p, stream)) return KDA_ERR_CUDA;
        launch_join(p, stream);
    }
    const bool ok = out_dtype == KDA_BF16 ? launch_one<DK, DV, __nv_bfloat16, true>(m, p, stream)
                                          : launch_one<DK, DV, float, true>(m, p, stream);
    return ok ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

int run_tc_path(const Args &p, int out_dtype, cudaStream_t stream)
{
    CUtensorMap m[3];
    if (!make_map(&m[0], p.q, p.H, p.dk, p.T) || !make_map(&m[1], p.k, p.H / p.group, p.dk, p.T) ||
        !make_map(&m[2], p.v, p.H / p.group, p.dv, p.T))
        return KDA_ERR_CUDA;
    if (p.dk <= 64) return p.dv <= 64 ? run_dims<64, 64>(m, p, out_dtype, stream) : run_dims<64, 128>(m, p, out_dtype, stream);
    return p.dv <= 64 ? run_dims<128, 64>(m, p, out_dtype, stream) : run_dims<128, 128>(m, p, out_dtype, stream);
}

}  // namespace lin

int launch_linear_timeout_probe(uint32_t cycles, cudaStream_t stream)
{
    lin::linear_timeout_probe_kernel<<<1, 32, 0, stream>>>(cycles);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int *status_word_linear()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, lin::g_linear_tc_error) == cudaSuccess ? static_cast<int *>(p) : nullptr;
}

}  // namespace kda
