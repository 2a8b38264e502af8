// Tensor-core (tcgen05 + TMEM + TMA) causal grouped-query attention with a
// sliding window and sinks, bf16 and f16, sm_103a.
//
// Query i sits at position p = off + i and sees the keys j <= p with
// j > p - window or j < sinks.  The tile arithmetic is that of the flash kernel
// (tc_flash.cu): a CTA's two 128-row query tiles share a stream of 128-key tiles,
// S and O live in tensor memory, P goes back there in 16 bits (over S at
// D = 128), thread = query row in two softmax warpgroups, one thread issues every
// MMA.  Bound by the exponentials and the tensor pipe at about 1.2 us per step of
// two tiles, plus about 6 us per CTA (set-up, first loads, masked tiles, last
// P V and epilogue), which is what a short window pays for: 4096 tokens, 32 heads
// on 8, window 1024, sinks 4, D 128: 58.1 us = 1039 TFLOP/s; 32768 tokens, window
// 4096: 1225 us = 1684 TFLOP/s for the first 20 calls in a row, then 1310 to 1335 us
// at the clock that the power cap leaves.  (The steps on record below were timed in
// short runs, against the kernel of their time.)  What differs:
//
//  * Key tile list.  A CTA streams the sink tiles and the tiles of its windows
//    only; tiles on an edge (diagonal, window start, sinks) are masked per
//    element, nearly always by one bound.
//  * Pairs of heads.  The two query tiles are the same rows of two query heads
//    of one KV head: one key range, no step that serves one tile alone.  (Pairs
//    of row tiles, which odd groups use, see windows one key tile apart: the
//    leading tile goes first, for the first query tile alone, so that each
//    works in consecutive steps.)  The 4096 tokens above: 86.1 us with row pairs
//    and one general mask, 74.4 us so.
//  * The pairs of a last round that takes at most half of the SMs are split into
//    single query tiles, so that the round ends sooner (1024 tokens, window 256:
//    19.2 us with any remainder split, 13.0 us so).
//  * A tile that holds a few sinks only (32 at most) is a step of 32 keys
//    (74.0 -> 71.4 us), output rows leave through shared memory as whole rows
//    (70.0 -> 66.7 us), and what the first scores wait for comes first: the
//    loaders' item and tensor maps during the set-up, then one query tile and one
//    key tile (66.7 -> 65.7 us; 5 tokens 4.7 -> 4.1 us).
//  * One CTA per item.  A persistent form (K and V of the next pair streaming in
//    behind the current one's, its first scores computed during the epilogue)
//    measured slower: 60.1 against 58.8 us at 4096 tokens, 1272 against 1220 us at
//    32768 tokens with a window of 4096: both query tiles end together, and their
//    epilogue keeps the softmax warps from the next pair.
//  * One thread per row.  Two (16 softmax warps, half of the keys each) took 63.2
//    against 59.3 us, P V in two halves behind the exponentials 58.8 against 58.3.
//
// Roundings: S, the statistics, row sums and O are fp32.  P is rounded to the 16-bit
// type (half a step of each weight) because the tensor core takes it as an
// operand beside V; the sum takes the weights before that.  O is rounded once.
//
// A key that a row does not see does not change its output, whatever it or its
// value holds: a masked score is -inf before anything is made of it, a row's
// running maximum moves by its own scores alone, and the tensor cores meet no
// infinite or NaN value that one of their rows does not see (0 x inf is NaN).  V
// of the sinks comes through a map that ends behind them (zeros follow); in the
// other tiles on an edge a warp that has nothing else to do looks the values over
// while the scores are computed and clears what is not finite, and the rows that
// do see such a value get it back in the epilogue (spoil_rows).  With finite
// inputs 4096 tokens take 58.4 us where 58.1 go without any of it, 32768 tokens
// 1226 and 1222; with one infinite value 8192 tokens, 8 heads on 2, window 2048, took
// 58 ms as long as rows that were not finite were computed again key by key.
//
// All spin-waits are bounded (1 s); on a timeout the CTA raises the device
// error word, drains what it issued, frees TMEM and exits.
#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "packed.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kBM = 128;      // query rows per tile (MMA M)
constexpr int kNQ = 2;        // query tiles per CTA
constexpr int kBN = 128;      // keys per key tile (MMA N of S)
constexpr int kFew = 32;      // keys of the tile that holds a few sinks only

template <int D>
struct WnCfg {
    static constexpr int BN = kBN;                         // keys per key tile
    static constexpr int PANELS = D / 64;                  // 128-byte swizzle panels
    static constexpr int PANEL_Q = kBM * 128;              // bytes per Q panel
    static constexpr int PANEL_KV = BN * 128;              // bytes per K/V panel
    static constexpr int Q_BYTES = PANELS * PANEL_Q;
    static constexpr int KV_BYTES = PANELS * PANEL_KV;     // one K (or V) stage
    static constexpr int BUDGET = 227 * 1024 - 2048;
    static constexpr int NS_ALL = (BUDGET - kNQ * Q_BYTES) / KV_BYTES;
    // K and V rings of equal depth (a third K stage at D = 128 measured slower)
    static constexpr int KS = NS_ALL / 2 > 4 ? 4 : NS_ALL / 2;               // K stages
    static constexpr int VS = NS_ALL - NS_ALL / 2 > 4 ? 4 : NS_ALL - NS_ALL / 2;  // V stages
    static_assert(KS >= 2 && VS >= 2, "at least two K and two V stages");
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = kNQ * Q_BYTES;
    static constexpr int OFF_V = OFF_K + KS * KV_BYTES;
    static constexpr int OFF_BAR = OFF_V + VS * KV_BYTES;
    static constexpr int SMEM = OFF_BAR + 512 + 1024;      // barriers + 1024 B alignment slack
    // Tensor memory (512 columns): S_t at t BN, O_t at kNQ BN + t D; P (16-bit,
    // two per column) over the first half of S_t (D = 128) or in columns of
    // its own after the O's (D = 64).
    static constexpr bool SEP_P = kNQ * (BN + D + BN / 2) <= 512;
    static constexpr uint32_t tm_s(int t) { return t * BN; }
    static constexpr uint32_t tm_o(int t) { return kNQ * BN + t * D; }
    static constexpr uint32_t tm_p(int t) { return SEP_P ? kNQ * BN + kNQ * D + t * (BN / 2) : t * BN; }
    static constexpr uint32_t TM_COLS = 512;
    static_assert(tm_o(kNQ - 1) + D <= TM_COLS && (!SEP_P || tm_p(kNQ) <= TM_COLS),
                  "tensor-memory layout must fit 512 columns");
    static constexpr int NSOFT = 4 * kNQ;
    static constexpr int W_MMA = NSOFT;                   // MMA issuer, TMEM owner
    static constexpr int W_LOAD = NSOFT + 1;              // Q and K copies
    static constexpr int W_LOADV = NSOFT + 2;             // V copies
    static constexpr int W_INIT = NSOFT + 3;              // barrier set-up
    static constexpr int NT = (NSOFT + 4) * 32;            // 3 warpgroups
    // register split: launch 168 x 384 = 64512; 2 x 128 x 216 + 128 x 72 = 64512
    static constexpr int REGS_LAUNCH = 168;
    static constexpr int REGS_SOFTMAX = 216;
    static constexpr int REGS_OTHER = 72;
    static_assert(2 * 128 * REGS_SOFTMAX + 128 * REGS_OTHER <= NT * REGS_LAUNCH,
                  "setmaxnreg split must fit the launch's register file share");
    static constexpr int k_off(int s) { return OFF_K + s * KV_BYTES; }
    static constexpr int v_off(int s) { return OFF_V + s * KV_BYTES; }
};

// Division by a number that a launch knows: n / d by a multiplication (every CTA
// starts with three of them, and everything waits for its loaders).
struct Div {
    unsigned mul;
    int sh, d;
    Div() = default;
    explicit Div(int n) : d(n) {
        int l = 0;
        while ((1ll << l) < d) ++l;
        mul = unsigned((((1ull << l) - d) << 32) / unsigned(d) + 1);
        sh = l - 1;
    }
    __device__ __forceinline__ int operator()(int n) const {
        const unsigned t = __umulhi(mul, unsigned(n));
        return d == 1 ? n : int((t + ((unsigned(n) - t) >> 1)) >> sh);
    }
};

struct WnParams {
    int Nq, Nkv;             // query / key tokens per (batch, head)
    int off, window, sinks;  // query i sits at position off + i
    float c_log2;            // scale * log2(e)
    unsigned *err;
    int pairs;               // query tile pairs
    int whole;               // pairs that are not split
    int by_head;             // a pair is two heads of one KV head (else two row tiles)
    int blocks;              // row blocks
    Div by_hp, by_h, by_group;   // pairs (or heads) per row block, heads, heads per KV head
    PackedSeqs seqs;         // packed: the sequences' starts (Nq, Nkv, off, pairs, whole, blocks unused)
    int sms;                 // packed: SMs
    const void *v;           // with element strides: values cleared from an edge tile
    TensorStrides sv;
    void *o;
    long long o_sb, o_sh, o_sn;
};

// a[t] for a per-query-tile array and a run-time t, by selects
template <typename T>
__device__ __forceinline__ T pick(const T (&a)[kNQ], int t) { return t == 0 ? a[0] : a[1]; }

// One work item: a pair of query tiles, or one tile alone.  Query tile t (rows
// q0 + t dq, head fh + t dh) works in steps [f[t], n[t]) of the item's key tile
// list.
struct Item {
    int q0, fb, fh, fkh, dq, dh;
    int n[kNQ], f[kNQ], steps;
    int w_lo, w_sk;                // first window tile, sink tiles before it
    bool few;                      // step 0 is the sinks' tile and holds at most kFew keys
    int nq, nkv, off;              // the sequence's lengths, its first query's position
    int q_row, k_row;              // packed: its rows in the arrays
    int e0, e1, e2;                // steps of the tiles on an edge: [e0, e1), [e2, steps), a leading one

    // key tile of step j: the leading tile of the first query tile (if any),
    // the sink tiles, the window
    __device__ __forceinline__ int tile(int j) const {
        const int i = j - f[1];
        return i < 0 ? w_lo : i < w_sk ? i : w_lo + j - w_sk;
    }
    // step j is a tile of sinks in front of every row's window
    __device__ __forceinline__ bool sink_tile(int j) const { return j >= f[1] && j < f[1] + w_sk; }
    // some row does not see all keys of step j's tile (sink tiles left out)
    __device__ __forceinline__ bool edge(int j) const {
        return j >= e2 || (j >= e0 && j < e1) || j < f[1];
    }
    // step j's values are looked over (packed: no tensor map ends behind a
    // sequence's sinks)
    template <bool PACKED> __device__ __forceinline__ bool checked(int j) const {
        return edge(j) || (PACKED && sink_tile(j));
    }
};

// Barrier block at OFF_BAR.
template <int KS, int VS>
struct Bars {
    uint64_t q_full[kNQ];
    // v_in: the stage's copies have landed; v_full: the checking warp has passed it on
    uint64_t k_full[KS], k_empty[KS], v_in[VS], v_full[VS], v_empty[VS];
    // per query tile t: s_full its Q K^T has completed, p_ready the softmax
    // has written P, o_done the P V product that read P has completed,
    // s_free (separate P, D = 64) the softmax holds S_t in registers
    uint64_t s_full[kNQ], p_ready[kNQ], o_done[kNQ], s_free[kNQ];
    uint64_t drain, checked;       // checked: every edge tile has been looked over
    uint32_t tmem_base;
    int abort, wild;               // wild: a value was cleared from one of them
    Item item;                     // packed: the CTA's item
};

// Completes an item of query rows q0 of one sequence: its heads are w.fh, of the
// pair or (half >= 0) one tile of it.
__device__ __forceinline__ void plan_item(const WnParams &p, Item &w, int half) {
    const int pos = w.off + w.q0;
    const bool one = w.q0 < w.nq, two = half < 0 && w.q0 + w.dq < w.nq;
    const int ns = cdiv(p.sinks, kBN);
    w.w_lo = imax(0, pos - p.window + 1) / kBN;
    const int lo1 = imax(0, pos + w.dq - p.window + 1) / kBN;
    w.w_sk = imin(ns, w.w_lo);
    w.few = w.w_sk > 0 && p.sinks <= kFew;
    w.f[0] = 0;
    w.f[1] = two && lo1 > w.w_lo && w.w_lo >= ns ? 1 : 0;
    w.few = w.few && w.f[1] == 0;
    // (a single second row tile past the sequence's end has no step)
    w.n[0] = one ? w.w_sk + (w.off + imin(w.q0 + kBM, w.nq) - 1) / kBN - w.w_lo + 1 : 0;
    w.n[1] = two ? w.w_sk + (w.off + imin(w.q0 + w.dq + kBM, w.nq) - 1) / kBN - w.w_lo + 1 : 0;
    w.steps = imax(w.n[0], w.n[1]);
    // the window of the last query tile starts behind its first key, or the first
    // one's diagonal comes before its last
    const int lead = two ? pos + w.dq : pos;
    w.e0 = w.w_sk + w.f[1];
    w.e1 = w.w_sk + cdiv(imax(0, lead + kBM - p.window), kBN) - w.w_lo;
    w.e2 = w.w_sk + imax(0, (pos + 1) / kBN - w.w_lo);
}

// This CTA's item: whole pairs, late queries first, then the rest as single
// tiles.
__device__ __forceinline__ Item get_item(const WnParams &p) {
    Item w;
    const int s = int(blockIdx.x) - p.whole;
    const int pair = s < 0 ? int(blockIdx.x) : p.whole + (s >> 1), half = s < 0 ? -1 : s & 1;
    const int block = p.by_hp(pair), qb = p.blocks - 1 - block;
    const int bh = (pair - block * p.by_hp.d) * (p.by_head ? 2 : 1);
    w.dq = p.by_head ? 0 : kBM;
    w.dh = p.by_head ? 1 : 0;
    w.fb = p.by_h(bh);
    w.fh = bh - w.fb * p.by_h.d + (half > 0 ? w.dh : 0);
    w.fkh = p.by_group(w.fh);
    w.q0 = qb * (p.by_head ? kBM : kNQ * kBM) + (half > 0 ? w.dq : 0);
    w.nq = p.Nq;
    w.nkv = p.Nkv;
    w.off = p.off;
    w.q_row = w.k_row = 0;
    plan_item(p, w, half);
    return w;
}

// The same for packed sequences (one warp): the blocks of all sequences by falling
// level (packed.cuh), the pairs of a last round split by the same rule.  A CTA
// behind the last item has one without steps.
__device__ __forceinline__ Item find_item(const WnParams &p) {
    const BlockFinder finder(p.seqs, p.by_head ? 7 : 8, blockIdx.x == 0, p.err);
    const int pairs = finder.total * p.by_hp.d, rest = pairs % p.sms;
    const int whole = 2 * rest <= p.sms ? pairs - rest : pairs;
    const int s = int(blockIdx.x) - whole;
    const int pair = s < 0 ? int(blockIdx.x) : whole + (s >> 1), half = s < 0 ? -1 : s & 1;
    Item w;
    w.n[0] = w.n[1] = w.f[0] = w.f[1] = w.steps = 0;
    w.w_lo = w.w_sk = w.e0 = w.e1 = w.e2 = 0;
    w.few = false;
    w.q0 = w.nq = w.nkv = w.off = w.q_row = w.k_row = 0;
    w.fb = w.fh = w.fkh = 0;
    w.dq = p.by_head ? 0 : kBM;
    w.dh = p.by_head ? 1 : 0;
    if (pair >= pairs) return w;
    const int block = p.by_hp(pair);
    const PackedBlock b = finder.find(block);
    w.fh = (pair - block * p.by_hp.d) * (p.by_head ? 2 : 1) + (half > 0 ? w.dh : 0);
    w.fkh = p.by_group(w.fh);
    w.q0 = b.q0 + (half > 0 ? w.dq : 0);
    w.nq = b.nq;
    w.nkv = b.nkv;
    w.off = b.nkv - b.nq;
    w.q_row = b.q_row;
    w.k_row = b.k_row;
    plan_item(p, w, half);
    return w;
}

// The bits of a 16-bit value that are all ones if it is infinite or NaN.
template <bool F16> constexpr uint32_t kWild = F16 ? 0x7c00u : 0x7f80u;

template <bool F16>
__device__ __forceinline__ bool wild_pair(uint32_t w) {
    constexpr uint32_t lo = kWild<F16>, hi = lo << 16;
    return (w & lo) == lo || (w & hi) == hi;
}

// a + 0 x in both halves: NaN where x is infinite or NaN.
template <bool F16>
__device__ __forceinline__ uint32_t add_zero_times(uint32_t a, uint32_t x) {
    uint32_t r;
    if constexpr (F16)
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(a));
    else
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(a));
    return r;
}

// Clears the infinite and NaN values of a V stage; returns whether there were
// any.  One warp; the writes are visible to the tensor cores behind the barrier
// that follows.
template <int D, bool F16>
__device__ __forceinline__ bool clear_wild(uint8_t *stage) {
    constexpr int VECS = kBN * D / 8, U = 8;
    constexpr uint32_t lo = kWild<F16>, hi = lo << 16;
    uint4 *at = reinterpret_cast<uint4 *>(stage) + (threadIdx.x & 31);
    uint32_t z[4] = {0u, 0u, 0u, 0u};
#pragma unroll 2
    for (int i = 0; i < VECS; i += U * 32) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = at[i + u * 32];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            z[0] = add_zero_times<F16>(z[0], x[u].x);
            z[1] = add_zero_times<F16>(z[1], x[u].y);
            z[2] = add_zero_times<F16>(z[2], x[u].z);
            z[3] = add_zero_times<F16>(z[3], x[u].w);
        }
    }
    const bool any = ((z[0] | z[1] | z[2] | z[3]) & 0x7fff7fffu) != 0;   // 0 x is +-0
    if (any) {
#pragma unroll 1
        for (int e = 0; e < VECS / 32 * 4; ++e) {
            uint32_t *y = reinterpret_cast<uint32_t *>(at + (e >> 2) * 32) + (e & 3);
            uint32_t w = *y;
            if ((w & lo) == lo) w &= 0xffff0000u;
            if ((w & hi) == hi) w &= 0x0000ffffu;
            *y = w;
        }
        ptx::fence_proxy_async_smem();
    }
    return __any_sync(0xffffffffu, any);
}

// Adds the infinite and NaN values that were cleared from the item's edge tiles to
// the warp's staged output rows that see them: whatever its (positive) weight,
// such a value makes its channel of the row infinite or NaN.  Rare, so the
// values are read again from memory, a row of V at a time.
template <int D, bool F16, bool PACKED>
__device__ __noinline__ void spoil_rows(const WnParams &p, const Item *packed, uint8_t *stage, int first_pos,
                                        int rows) {
    const Item w = PACKED ? *packed : get_item(p);   // (handed over it would live in memory)
    using H = H16<F16>;
    constexpr int CW = D / 64;                       // 32-bit words (two channels) per lane
    constexpr int CH = D / 8, U = 8;
    const int lane = threadIdx.x & 31;
    const uint32_t *v = reinterpret_cast<const uint32_t *>(static_cast<const typename H::T *>(p.v) +
                                                           w.fb * p.sv.b + w.fkh * p.sv.h +
                                                           w.k_row * p.sv.n) + lane * CW;
    for (int j = 0; j < w.steps; ++j) {
        if (!w.template checked<PACKED>(j)) continue;
        const int k0 = w.tile(j) * kBN, keys = imin(kBN, w.nkv - k0);
        for (int i = 0; i < keys; i += U) {
            uint32_t x[U][CW];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int c = 0; c < CW; ++c) x[u][c] = i + u < keys ? v[(k0 + i + u) * (p.sv.n / 2) + c] : 0u;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                bool here = false;
#pragma unroll
                for (int c = 0; c < CW; ++c) here = here || wild_pair<F16>(x[u][c]);
                if (!__any_sync(0xffffffffu, here)) continue;
                const int key = k0 + i + u;
#pragma unroll 1
                for (int r = 0; r < rows; ++r) {
                    const int pos = first_pos + r;
                    if (key > pos || (key <= pos - p.window && key >= p.sinks)) continue;
                    uint32_t *y = reinterpret_cast<uint32_t *>(
                                      stage + (r * CH + ((lane * CW / 4) ^ (r & 7))) * 16) + lane * CW % 4;
#pragma unroll
                    for (int c = 0; c < CW; ++c) {
                        const float a = H::lo(x[u][c]), b = H::hi(x[u][c]);
                        y[c] = H::pack(fabsf(a) < INFINITY ? H::lo(y[c]) : H::lo(y[c]) + a,
                                       fabsf(b) < INFINITY ? H::hi(y[c]) : H::hi(y[c]) + b);
                    }
                }
            }
        }
    }
    __syncwarp();
}

// PACKED: q, k, v and o hold sequences of different lengths one behind the other
// (p.seqs); a warp finds the CTA's item while the rest is set up.
template <int D, bool F16, bool PACKED>
__global__ void __launch_bounds__(WnCfg<D>::NT, 1)
tc_window_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                 const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tvs,
                 const WnParams p) {
    using C = WnCfg<D>;
    using BarsT = Bars<C::KS, C::VS>;
    static_assert(sizeof(BarsT) <= 512, "barrier block must fit its reserved bytes");
    extern __shared__ uint8_t smem_raw[];
    // 1024-byte alignment for the 128-byte swizzle atoms
    uint8_t *smem = smem_raw + ((1024 - (ptx::smem_addr(smem_raw) & 1023)) & 1023);
    BarsT *bars = reinterpret_cast<BarsT *>(smem + C::OFF_BAR);
    volatile int *abort = &bars->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int BNt = C::BN;     // keys per tile

    if (warp == C::W_INIT && lane == 0) {
        for (int s = 0; s < C::KS; ++s) {
            ptx::mbar_init(&bars->k_full[s], 1);
            ptx::mbar_init(&bars->k_empty[s], 1);
        }
        for (int s = 0; s < C::VS; ++s) {
            ptx::mbar_init(&bars->v_in[s], 1);
            ptx::mbar_init(&bars->v_full[s], 1);
            ptx::mbar_init(&bars->v_empty[s], 1);
        }
        for (int t = 0; t < kNQ; ++t) {
            ptx::mbar_init(&bars->q_full[t], 1);
            ptx::mbar_init(&bars->s_full[t], 1);
            ptx::mbar_init(&bars->p_ready[t], 128);
            ptx::mbar_init(&bars->o_done[t], 1);
            ptx::mbar_init(&bars->s_free[t], 128);
        }
        ptx::mbar_init(&bars->drain, 1);
        ptx::mbar_init(&bars->checked, 1);
        bars->abort = bars->wild = 0;
        ptx::fence_barrier_init();
    }
    if (warp == C::W_MMA) {
        ptx::tmem_alloc(&bars->tmem_base, C::TM_COLS);
        ptx::tmem_relinquish();
    }
    Item load_item;                                    // the loaders', while the rest is set up
    if (warp == C::W_LOAD || warp == C::W_LOADV) {
        ptx::prefetch_tmap(warp == C::W_LOAD ? &tk : &tv);
        if (warp == C::W_LOAD) ptx::prefetch_tmap(&tq);
        if constexpr (PACKED) {
            if (warp == C::W_LOAD) {
                ptx::griddep_wait();                   // the starts may be the previous kernel's
                load_item = find_item(p);
                if (lane == 0) bars->item = load_item;
            }
        } else {
            load_item = get_item(p);
            if (warp == C::W_LOADV && load_item.w_sk > 0) ptx::prefetch_tmap(&tvs);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    // programmatic dependent launch: the set-up above touches nothing global
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    auto my_item = [&]() -> Item { return PACKED ? bars->item : get_item(p); };

    if (warp >= C::NSOFT) {
        ptx::regs_decrease<C::REGS_OTHER>();
        if ((warp == C::W_LOAD || warp == C::W_LOADV) && lane == 0) {
            // ============================================= TMA loaders: one
            // thread streams Q and the K ring, another the V ring
            const int which = warp == C::W_LOAD ? 0 : 1;
            const CUtensorMap *tm = which == 0 ? &tk : &tv;
            uint64_t *full = which == 0 ? bars->k_full : bars->v_in;
            uint64_t *empty = which == 0 ? bars->k_empty : bars->v_empty;
            const int NS = which == 0 ? C::KS : C::VS;   // depth of this ring
            const uint64_t pol_kv = ptx::l2_policy_evict_last(), pol_q = ptx::l2_policy_evict_first();
            const Item w = PACKED && which == 1 ? bars->item : load_item;
            int q_out = 0, issued = 0;
            auto load_q = [&](int t) {
                if (t >= (w.n[1] > 0 ? kNQ : 1)) return;
                ++q_out;
                ptx::mbar_arrive_expect_tx(&bars->q_full[t], C::Q_BYTES);
                for (int pn = 0; pn < C::PANELS; ++pn)
                    ptx::tma_load_4d(smem + C::OFF_Q + t * C::Q_BYTES + pn * C::PANEL_Q, &tq, pn * 64,
                                     w.q_row + w.q0 + t * w.dq, w.fh + t * w.dh, w.fb, &bars->q_full[t], pol_q);
            };
            if (which == 0 && w.steps > 0) load_q(0);
            for (int j = 0; j < w.steps; ++j) {
                const int s = j % NS;
                if (j >= NS && !ptx::mbar_wait_or_abort(&empty[s], ((j / NS) - 1) & 1, p.err, abort)) break;
                issued = j + 1;
                ptx::mbar_arrive_expect_tx(&full[s], C::KV_BYTES);
                for (int pn = 0; pn < C::PANELS; ++pn)
                    ptx::tma_load_4d(smem + (which == 0 ? C::k_off(s) : C::v_off(s)) + pn * C::PANEL_KV,
                                     !PACKED && which == 1 && w.sink_tile(j) ? &tvs : tm, pn * 64,
                                     w.k_row + w.tile(j) * kBN, w.fkh, w.fb, &full[s], pol_kv);
                // the first scores need one query tile and the first keys
                if (which == 0 && j == 0) load_q(1);
            }
            // after a timeout elsewhere: let the copies this thread issued land
            // (bounded) before the CTA's shared memory is released
            if (*abort) {
                for (int t = 0; t < q_out; ++t) ptx::mbar_wait(&bars->q_full[t], 0, nullptr);
                for (int j = imax(0, issued - NS); j < issued; ++j)
                    ptx::mbar_wait(&full[j % NS], (j / NS) & 1, nullptr);
            }
        } else if (warp == C::W_MMA) {
            // ============================================= MMA issuer: the whole
            // warp walks the steps, so that all it computes is uniform, and one
            // thread issues (with a single thread in the branch the operands of every
            // MMA passed through vector registers: 65.3 and 1435 us)
            const bool lead = ptx::elect_one();
            const uint32_t id_qk = ptx::idesc_16_f32(kBM, BNt, false, F16);
            const uint32_t id_few = ptx::idesc_16_f32(kBM, kFew, false, F16);
            const uint32_t id_pv = ptx::idesc_16_f32(kBM, D, true, F16);
            // descriptors are built once; a k-step, a stage or a tile only moves
            // the start-address field
            constexpr uint32_t HI128 = ptx::desc_hi_sw128(1024);
            const uint32_t dq0 = ptx::desc_lo_sw128(ptx::smem_addr(smem + C::OFF_Q), 16);
            const uint32_t dk0 = ptx::desc_lo_sw128(ptx::smem_addr(smem + C::k_off(0)), 16);
            const uint32_t dv0 = ptx::desc_lo_sw128(ptx::smem_addr(smem + C::v_off(0)), C::PANEL_KV);
            constexpr int nkv = BNt / 16;                // k-steps of P V
            const Item w = my_item();
            auto issue_qk = [&](int t, int gk) {
                if (!lead) return;
                const uint32_t id = w.few && gk == 0 ? id_few : id_qk;
                const uint32_t a0 = dq0 + uint32_t((t * C::Q_BYTES) >> 4);
                const uint32_t b0 = dk0 + uint32_t(((gk % C::KS) * C::KV_BYTES) >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t oa = ((kk >> 2) * C::PANEL_Q + (kk & 3) * 32) >> 4;
                    const uint32_t ob = ((kk >> 2) * C::PANEL_KV + (kk & 3) * 32) >> 4;
                    ptx::mma_ss(tmem + C::tm_s(t), ptx::desc_join(a0 + oa, HI128),
                                ptx::desc_join(b0 + ob, HI128), id, kk > 0);
                }
                ptx::tc_commit(&bars->s_full[t]);
            };
            auto issue_pv = [&](int t, int gv, bool first) {
                if (!lead) return;
                const uint32_t b0 = dv0 + uint32_t(((gv % C::VS) * C::KV_BYTES) >> 4);
                const uint32_t a0 = tmem + C::tm_p(t);
#pragma unroll
                for (int kk = 0; kk < nkv; ++kk) {
                    if (kk == kFew / 16 && w.few && gv == 0) break;
                    ptx::mma_ts(tmem + C::tm_o(t), a0 + kk * 8,
                                ptx::desc_join(b0 + uint32_t(kk * (2048 >> 4)), HI128), id_pv,
                                (!first || kk > 0) ? 1u : 0u);
                }
                ptx::tc_commit(&bars->o_done[t]);
            };
            bool ok = w.steps > 0, k_seen = false, v_seen = false;
            // a stage barrier is waited on once per step (a completed wait still
            // costs this thread a round trip to shared memory)
            auto wait_k = [&](int j) {
                if (!k_seen) {
                    ok = ok && ptx::mbar_wait_or_abort(&bars->k_full[j % C::KS], (j / C::KS) & 1, p.err, abort);
                    k_seen = true;
                }
            };
            auto wait_v = [&](int j) {
                if (!v_seen) {
                    ok = ok && ptx::mbar_wait_or_abort(&bars->v_full[j % C::VS], (j / C::VS) & 1, p.err, abort);
                    v_seen = true;
                }
            };
            // Q K^T of step j for tile t, once the softmax no longer needs the S it
            // overwrites (separate P: as soon as the softmax holds the S before in
            // registers; P over S: after the P V before, issued already)
            auto qk = [&](int t, int j) {
                wait_k(j);
                if (j >= w.n[t] || j < w.f[t]) return;
                if (C::SEP_P && j > w.f[t])
                    ok = ok && ptx::mbar_wait_or_abort(&bars->s_free[t], (j - 1 - w.f[t]) & 1, p.err, abort);
                if (!ok) return;
                ptx::tc_fence_after();
                issue_qk(t, j);
            };
            // P V of step j for tile t
            auto pv = [&](int t, int j) {
                wait_v(j);
                if (j >= w.n[t] || j < w.f[t]) return;
                ok = ok && ptx::mbar_wait_or_abort(&bars->p_ready[t], (j - w.f[t]) & 1, p.err, abort);
                if (!ok) return;
                ptx::tc_fence_after();
                issue_pv(t, j, j == w.f[t]);
            };
#pragma unroll
            for (int t = 0; t < kNQ; ++t) {
                if (w.n[t] > 0) ok = ok && ptx::mbar_wait_or_abort(&bars->q_full[t], 0, p.err, abort);
                if (ok) qk(t, 0);
            }
            if (ok && lead) ptx::tc_commit(&bars->k_empty[0]);
            for (int j = 0; ok && j < w.steps; ++j) {
                const int jn = j + 1;
                k_seen = v_seen = false;
                if constexpr (C::SEP_P) {
#pragma unroll
                    for (int t = 0; t < kNQ; ++t)
                        if (ok && jn < w.steps) qk(t, jn);
#pragma unroll
                    for (int t = 0; t < kNQ; ++t)
                        if (ok) pv(t, j);
                } else {
#pragma unroll
                    for (int t = 0; t < kNQ; ++t) {
                        if (ok) pv(t, j);
                        if (ok && jn < w.steps) qk(t, jn);
                    }
                }
                if (!ok) break;
                if (lead) {
                    if (jn < w.steps) ptx::tc_commit(&bars->k_empty[jn % C::KS]);
                    ptx::tc_commit(&bars->v_empty[j % C::VS]);
                }
            }
            // drain: every MMA has completed before TMEM is freed
            if (lead) ptx::tc_commit(&bars->drain);
            ptx::mbar_wait(&bars->drain, 0, p.err);
        } else if (warp == C::W_INIT) {
            // ============================================= the V of edge tiles is
            // looked over as it arrives, while the tile's scores are computed and
            // exponentiated; other tiles are passed on at once
            const Item w = my_item();
            for (int j = 0; j < w.steps; ++j) {
                const int s = j % C::VS;
                if (!__all_sync(0xffffffffu, ptx::mbar_wait_or_abort(&bars->v_in[s], (j / C::VS) & 1, p.err, abort)))
                    break;
                const bool any = w.template checked<PACKED>(j) && clear_wild<D, F16>(smem + C::v_off(s));
                __syncwarp();
                if (lane == 0) {
                    if (any) bars->wild = 1;
                    ptx::mbar_arrive(&bars->v_full[s]);
                }
            }
            if (lane == 0) ptx::mbar_arrive(&bars->checked);
        }
    } else {
        // ================================================= softmax warpgroups
        ptx::regs_increase<C::REGS_SOFTMAX>();
        const int t = warp >> 2;                 // query tile
        const int quarter = warp & 3;            // TMEM lanes [32 quarter, 32 quarter + 32)
        const int row = quarter * 32 + lane;     // query row within the tile
        const uint32_t lane_base = tmem + (uint32_t(quarter * 32) << 16);
        const uint32_t o_addr = lane_base + C::tm_o(t);
        const uint32_t s_addr = lane_base + C::tm_s(t);
        const uint32_t p_addr = lane_base + C::tm_p(t);
        const float cl = p.c_log2;
        bool ok = true;
        const Item w = my_item();
        const int f = pick(w.f, t), nt = pick(w.n, t) - f;   // this query tile's key tiles
        const int pos = w.off + w.q0 + w.dq * t;             // position of its first row

        // waits for the P V product of key tile jj of this query tile (and so
        // for every earlier one: one thread's MMAs complete in issue order)
        auto wait_pv = [&](int jj) -> bool {
            if (!__all_sync(0xffffffffu, ptx::mbar_wait_or_abort(&bars->o_done[t], jj & 1, p.err, abort)))
                return false;
            ptx::tc_fence_after();
            return true;
        };

        float m = -INFINITY, l = 0.f;
        int j = 0;
        // the key tile from which on every row of the warp has seen a key before: of
        // the first one the last rows may see nothing, and then see the next
        const int k_first = w.tile(f) * kBN;
        const int seen_from = k_first < p.sinks || pos + quarter * 32 + 32 - p.window < k_first + kBN ? 1 : 2;
        // ---- a first tile of a few sinks, which every row sees: kFew columns
        if (w.few && nt > 0) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait_or_abort(&bars->s_full[t], 0, p.err, abort));
            if (ok) {
                ptx::tc_fence_after();
                float x[kFew];
                ptx::tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
                ptx::tmem_wait_ld();
                if constexpr (C::SEP_P) {
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(&bars->s_free[t]);
                }
                float mx = -INFINITY;
#pragma unroll
                for (int e = 0; e < kFew; ++e) {
                    if (e >= p.sinks) x[e] = -INFINITY;
                    mx = fmaxf(mx, x[e]);
                }
                m = mx * cl;
                const float nmu = m == -INFINITY ? 0.f : -m;
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < kFew; e += 2) {
                    const float p0 = ptx::ex2(fmaf(x[e], cl, nmu)), p1 = ptx::ex2(fmaf(x[e + 1], cl, nmu));
                    l += p0 + p1;
                    pk[e / 2] = H16<F16>::pack(p0, p1);
                }
                ptx::tmem_st16(p_addr, pk);
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                ptx::mbar_arrive(&bars->p_ready[t]);
                j = 1;
            }
        }
        for (; ok && j < nt; ++j) {
            if (!__all_sync(0xffffffffu, ptx::mbar_wait_or_abort(&bars->s_full[t], j & 1, p.err, abort))) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();

            float sv[BNt];
#pragma unroll
            for (int c = 0; c < BNt / 32; ++c)
                ptx::tmem_ld32(s_addr + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[c * 32]));
            ptx::tmem_wait_ld();
            if constexpr (C::SEP_P) {
                // S_t is in registers: the next QK_t may overwrite it
                ptx::tc_fence_before();
                ptx::mbar_arrive(&bars->s_free[t]);
            }

            // ---- masks: rows at positions pos + row; only tiles on an edge of
            //      the window are masked per element
            {
                const int k0 = w.tile(f + j) * BNt;
                const bool late = k0 + BNt - 1 > pos;                    // a key behind the first row
                const bool early = k0 + p.window < pos + kBM;            // one before the last row's window
                if (late || (early && k0 + BNt > p.sinks)) {
                    // key e of the tile is seen iff e <= hi and (e >= lo or e < sk);
                    // all but tiny windows need only one bound per tile: the
                    // diagonal's, the end of the sinks, or the window's start
                    const int hi = pos + row - k0, lo = hi - p.window + 1, sk = p.sinks - k0;
                    if (!early || (!late && k0 + p.window + BNt <= pos + 1)) {
                        const int last = early ? sk - 1 : hi;
#pragma unroll
                        for (int e = 0; e < BNt; ++e)
                            if (e > last) sv[e] = -INFINITY;
                    } else if (!late && sk <= 0) {
#pragma unroll
                        for (int e = 0; e < BNt; ++e)
                            if (e < lo) sv[e] = -INFINITY;
                    } else {
#pragma unroll
                        for (int e = 0; e < BNt; ++e)
                            if (e > hi || (e < lo && e >= sk)) sv[e] = -INFINITY;
                    }
                }
            }

            // P = 2^(x - m) in 16-bit into TMEM; returns the tile's row sum (fp32)
            auto emit_p = [&](float nmu) -> float {
                float acc[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll
                for (int c = 0; c < BNt / 32; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float x0, x1;
                        ptx::ffma2(x0, x1, sv[c * 32 + 2 * e], sv[c * 32 + 2 * e + 1], cl, cl, nmu, nmu);
                        const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
                        ptx::fadd2(acc[(2 * e) & 7], acc[(2 * e + 1) & 7], acc[(2 * e) & 7],
                                   acc[(2 * e + 1) & 7], p0, p1);
                        pk[e] = H16<F16>::pack(p0, p1);
                    }
                    ptx::tmem_st16(p_addr + c * 16, pk);
                }
                return ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
            };

            // ---- P in columns of its own: the P V product that last read them
            //      (key tile j - 1) must be done.  P over S needs no wait: the
            //      Q K^T that wrote this S was issued after the P V that read the
            //      P last held here, and MMAs complete in issue order.
            bool prev_done = false;              // P V of tile j - 1 observed complete
            if (C::SEP_P && j >= 1) {
                if (!wait_pv(j - 1)) {
                    ok = false;
                    break;
                }
                prev_done = true;
            }

            // ---- fast path: exponentiate against the running maximum m as it
            //      stands, with no tile maximum.  P only has to stay finite in its
            //      16-bit type, not below 1: a tile whose row sum exceeds 2^24 (2^15
            //      for f16, whose largest finite value is 65504) or is not finite
            //      is redone below against its own maximum.  After the first tiles
            //      m is close to the row maximum and the redo almost never runs.
            bool fast = false, keep = false;      // this row's maximum may stay
            if (j >= seen_from) {
                const float lt = emit_p(-m);      // infinite or NaN if m is still -inf
                keep = lt <= (F16 ? 32768.f : 16777216.f);
                fast = __all_sync(0xffffffffu, keep);   // else redo the tile (P is rewritten below)
                if (fast) l += lt;
            }

            if (!fast) {
                // ---- tile maximum
                float mx[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) mx[i] = -INFINITY;
#pragma unroll
                for (int e = 0; e < BNt; e += 8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) mx[i] = fmaxf(mx[i], sv[e + i]);
                }
                const float tmax = fmaxf(ptx::fmax3(ptx::fmax3(mx[0], mx[1], mx[2]), ptx::fmax3(mx[3], mx[4], mx[5]),
                                                    mx[6]),
                                         mx[7]);
                const float mt = tmax * cl;      // cl > 0: max commutes with the scaling

                // ---- the previous P V must be done before O is rescaled
                // (a row that a redo for other rows' sake takes along keeps it)
                const bool want = j == 0 || (!keep && mt > m + 8.f);   // this row moves its maximum
                const bool any_want = __any_sync(0xffffffffu, want);
                if (j > 0 && any_want && !prev_done) {
                    if (!wait_pv(j - 1)) {
                        ok = false;
                        break;
                    }
                }
                // ---- running maximum (moved lazily) and O rescale in TMEM
                if (j == 0) {
                    m = mt;
                } else if (any_want) {
                    // rows that move m scale their O row; the others multiply by 1
                    const float f = want ? ptx::ex2(m - mt) : 1.f;   // m == -inf -> 0
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t ov[32];
                        ptx::tmem_ld32(o_addr + c * 32, ov);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float a0, a1;
                            ptx::ffma2(a0, a1, __uint_as_float(ov[e]), __uint_as_float(ov[e + 1]), f,
                                       f, 0.f, 0.f);
                            ov[e] = __float_as_uint(a0);
                            ov[e + 1] = __float_as_uint(a1);
                        }
                        ptx::tmem_st32(o_addr + c * 32, ov);
                    }
                    if (want) {
                        l *= f;
                        m = mt;
                    }
                }
                l += emit_p((m == -INFINITY) ? 0.f : -m);
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            ptx::mbar_arrive(&bars->p_ready[t]);
        }


        // ---- epilogue: O / l -> 16-bit -> global
        if (ok && nt > 0 && wait_pv(nt - 1)) {
            const float inv = 1.f / l;
            int ln = threadIdx.x & 31;           // opaque: nothing of the epilogue is computed ahead
            asm volatile("" : "+r"(ln));
            const int q_first = w.q0 + t * w.dq + quarter * 32, qh = w.fh + t * w.dh;   // the warp's first row
            constexpr int CH = D / 8;            // 16-byte columns of a row
            // the warp's 32 rows pass through the query tile's memory (every Q K^T
            // has completed), column c of row r at c ^ (r & 7), so that whole rows
            // go out instead of 32 rows' 16 bytes
            uint8_t *stage = smem + C::OFF_Q + t * C::Q_BYTES + quarter * 32 * D * 2;
#pragma unroll
            for (int half = 0; half < D / 64; ++half) {
                float ov[64];
                ptx::tmem_ld32(o_addr + half * 64, *reinterpret_cast<uint32_t(*)[32]>(&ov[0]));
                ptx::tmem_ld32(o_addr + half * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&ov[32]));
                ptx::tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[e] = H16<F16>::pack(ov[c * 8 + 2 * e] * inv, ov[c * 8 + 2 * e + 1] * inv);
                    *reinterpret_cast<uint4 *>(stage + (ln * CH + half * 8 + (c ^ (ln & 7))) * 16) =
                        make_uint4(x[0], x[1], x[2], x[3]);
                }
            }
            __syncwarp();
            if (__all_sync(0xffffffffu, ptx::mbar_wait_or_abort(&bars->checked, 0, p.err, abort)) &&
                *reinterpret_cast<volatile int *>(&bars->wild))
                spoil_rows<D, F16, PACKED>(p, &bars->item, stage, w.off + q_first, imin(32, w.nq - q_first));
            typename H16<F16>::T *const o0 = static_cast<typename H16<F16>::T *>(p.o) + w.fb * p.o_sb + qh * p.o_sh;
            const int col = ln % CH;
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += 32 / CH) {
                const int r = r0 + ln / CH;
                const uint4 x = *reinterpret_cast<const uint4 *>(stage + (r * CH + (col ^ (r & 7))) * 16);
                if (q_first + r < w.nq)
                    *reinterpret_cast<uint4 *>(o0 + (w.q_row + q_first + r) * p.o_sn + col * 8) = x;
            }
        }
    }

    // ---- teardown: all TMEM traffic done before the owner warp frees it
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == C::W_MMA) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, C::TM_COLS);
    }
}

template <int D, bool F16, bool PACKED>
attn_status_t launch_window(const Ctx &c, const CUtensorMap &tq, const CUtensorMap &tk,
                            const CUtensorMap &tv, const CUtensorMap &tvs, const WnParams &p, int grid) {
    using C = WnCfg<D>;
    static int done_mask = 0;
    static int regs = -1;
    auto kern = tc_window_kernel<D, F16, PACKED>;
    if (!ensure_smem_attr(reinterpret_cast<const void *>(kern), C::SMEM, c.device, &done_mask))
        return ATTN_ERR_RESOURCE;
    // the setmaxnreg split is only valid for the per-thread count it was computed for
    if (regs < 0) {
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, reinterpret_cast<const void *>(kern)) != cudaSuccess) {
            cudaGetLastError();
            return ATTN_ERR_CUDA;
        }
        regs = fa.numRegs;
    }
    if (regs != C::REGS_LAUNCH) return ATTN_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(C::NT);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, tvs, p) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    return launch_status(kFamTcFlash);
}

}  // namespace

attn_status_t tc_causal_window(const Ctx &c, attn_dtype_t dt, const void *q, const void *k,
                               const void *v, void *o, int B, int Hq, int Hkv, int Nq, int Nkv,
                               int D, int window, int sinks, float scale, const TensorStrides *st) {
    const bool f16 = dt == ATTN_F16;
    // Two heads of a KV head make a pair with one key range: no step for one
    // tile alone, and 128-row blocks.  An odd group pairs row tiles instead.
    const bool by_head = (Hq / Hkv) % 2 == 0;
    const long long pairs = by_head ? (long long)cdiv(Nq, kBM) * (B * Hq / 2)
                                    : (long long)cdiv(Nq, kNQ * kBM) * B * Hq;
    if (pairs > (1 << 29)) return ATTN_ERR_UNSUPPORTED;
    CUtensorMap tq, tk, tv, tvs;
    // a layout the tensor-map encoder refuses goes to the strided SIMT kernel
    if (!make_tmap4(&tq, q, D, Nq, Hq, B, st[0], f16) || !make_tmap4(&tk, k, D, Nkv, Hkv, B, st[1], f16) ||
        !make_tmap4(&tv, v, D, Nkv, Hkv, B, st[2], f16) ||
        // of the sinks' values only: rows behind them are read as zeros
        !make_tmap4(&tvs, v, D, sinks > 0 ? sinks : Nkv, Hkv, B, st[2], f16))
        return ATTN_ERR_UNSUPPORTED;
    WnParams p{};
    p.Nq = Nq;
    p.Nkv = Nkv;
    p.off = Nkv - Nq;
    p.window = window;
    p.sinks = sinks;
    p.c_log2 = scale * kLog2e;
    p.err = c.err;
    p.blocks = cdiv(Nq, by_head ? kBM : kNQ * kBM);
    p.by_hp = Div(by_head ? B * Hq / 2 : B * Hq);
    p.by_h = Div(Hq);
    p.by_group = Div(Hq / Hkv);
    p.pairs = int(pairs);
    p.by_head = by_head;
    // the pairs of a last round that takes at most half of the SMs go out as
    // single tiles, on twice as many
    const int rest = p.pairs % imax(1, c.sm_count);
    p.whole = 2 * rest <= c.sm_count ? p.pairs - rest : p.pairs;
    p.v = v; p.o = o;
    p.sv = st[2];
    p.o_sb = st[3].b; p.o_sh = st[3].h; p.o_sn = st[3].n;
    const int grid = p.whole + 2 * (p.pairs - p.whole);
    if (D == 128)
        return f16 ? launch_window<128, true, false>(c, tq, tk, tv, tvs, p, grid)
                   : launch_window<128, false, false>(c, tq, tk, tv, tvs, p, grid);
    return f16 ? launch_window<64, true, false>(c, tq, tk, tv, tvs, p, grid)
               : launch_window<64, false, false>(c, tq, tk, tv, tvs, p, grid);
}

attn_status_t tc_causal_varlen(const Ctx &c, attn_dtype_t dt, const VarlenArgs &a) {
    const bool f16 = dt == ATTN_F16;
    const bool by_head = (a.Hq / a.Hkv) % 2 == 0;
    const int bs = by_head ? kBM : kNQ * kBM, hp = by_head ? a.Hq / 2 : a.Hq;
    // the most blocks that sequences of Nq queries together can have
    const long long blocks = (a.Nq + (long long)imin(a.B, a.Nq) * (bs - 1)) / bs;
    if (blocks * hp > (1 << 29)) return ATTN_ERR_UNSUPPORTED;
    CUtensorMap tq, tk, tv;
    if (!make_tmap4(&tq, a.q, a.D, a.Nq, a.Hq, 1, a.st[0], f16) ||
        !make_tmap4(&tk, a.k, a.D, a.Nkv, a.Hkv, 1, a.st[1], f16) ||
        !make_tmap4(&tv, a.v, a.D, a.Nkv, a.Hkv, 1, a.st[2], f16))
        return ATTN_ERR_UNSUPPORTED;
    WnParams p{};
    p.seqs = PackedSeqs{a.cu_q, a.cu_k, a.B, a.Nq, a.Nkv};
    p.sms = imax(1, c.sm_count);
    p.window = a.window;
    p.sinks = a.sinks;
    p.c_log2 = a.scale * kLog2e;
    p.err = c.err;
    p.by_hp = Div(hp);
    p.by_group = Div(a.Hq / a.Hkv);
    p.by_head = by_head;
    p.v = a.v; p.o = a.o;
    p.sv = a.st[2];
    p.o_sh = a.st[3].h; p.o_sn = a.st[3].n;
    const int grid = int(blocks * hp) + p.sms / 2;     // and the halves of a split last round
    if (a.D == 128)
        return f16 ? launch_window<128, true, true>(c, tq, tk, tv, tv, p, grid)
                   : launch_window<128, false, true>(c, tq, tk, tv, tv, p, grid);
    return f16 ? launch_window<64, true, true>(c, tq, tk, tv, tv, p, grid)
               : launch_window<64, false, true>(c, tq, tk, tv, tv, p, grid);
}

}  // namespace attn
