// Key tiles of causal attention with a window and sinks on the tensor cores: what
// the kernels for one length (tc_window.cu) and for packed sequences (tc_varlen.cu)
// share.  The reasons stand in tc_window.cu.
#pragma once

#include "common.cuh"
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
    static constexpr int BARS = 1024;
    static constexpr int SMEM = OFF_BAR + BARS + 1024;     // barriers + 1024 B alignment slack
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
};

// The key tiles of an item whose heads, rows and distances (q0, dq, dh) are set: nq
// queries of a sequence from position off on; half >= 0: one tile of the pair.
__device__ __forceinline__ void plan_item(Item &w, int off, int nq, int window, int sinks, int half) {
    const int pos = off + w.q0;
    const bool one = w.q0 < nq, two = half < 0 && w.q0 + w.dq < nq;
    const int ns = cdiv(sinks, kBN);
    w.w_lo = imax(0, pos - window + 1) / kBN;
    const int lo1 = imax(0, pos + w.dq - window + 1) / kBN;
    w.w_sk = imin(ns, w.w_lo);
    w.few = w.w_sk > 0 && sinks <= kFew;
    w.f[0] = 0;
    w.f[1] = two && lo1 > w.w_lo && w.w_lo >= ns ? 1 : 0;
    w.few = w.few && w.f[1] == 0;
    // (a single second row tile past the sequence's end has no step)
    w.n[0] = one ? w.w_sk + (off + imin(w.q0 + kBM, nq) - 1) / kBN - w.w_lo + 1 : 0;
    w.n[1] = two ? w.w_sk + (off + imin(w.q0 + w.dq + kBM, nq) - 1) / kBN - w.w_lo + 1 : 0;
    w.steps = imax(w.n[0], w.n[1]);
    // the window of the last query tile starts behind its first key, or the first
    // one's diagonal comes before its last
    const int lead = two ? pos + w.dq : pos;
    w.e0 = w.w_sk + w.f[1];
    w.e1 = w.w_sk + cdiv(imax(0, lead + kBM - window), kBN) - w.w_lo;
    w.e2 = w.w_sk + imax(0, (pos + 1) / kBN - w.w_lo);
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
// the warp's output rows that see them: whatever its (positive) weight, such a
// value makes its channel of the row infinite or NaN.  Rare, so the values are
// read again from memory, a row of V at a time.  v0: the KV head's values (v_stride
// elements from token to token, nkv tokens); sinks_too: values of sink tiles were cleared
// as well; at(r): where the lane's channels, 2 CW from 2 CW lane on, of row r are.
template <int D, bool F16, typename At>
__device__ __forceinline__ void spoil_rows(const Item &w, const typename H16<F16>::T *v0, long long v_stride, int nkv,
                                           int window, int sinks, bool sinks_too, At at, int first_pos, int rows) {
    using H = H16<F16>;
    constexpr int CW = D / 64;                       // 32-bit words (two channels) per lane
    constexpr int U = 8;
    const int lane = threadIdx.x & 31;
    const uint32_t *v = reinterpret_cast<const uint32_t *>(v0) + lane * CW;
    for (int j = 0; j < w.steps; ++j) {
        if (!w.edge(j) && !(sinks_too && w.sink_tile(j))) continue;
        const int k0 = w.tile(j) * kBN, keys = imin(kBN, nkv - k0);
        for (int i = 0; i < keys; i += U) {
            uint32_t x[U][CW];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int c = 0; c < CW; ++c) x[u][c] = i + u < keys ? v[(k0 + i + u) * (v_stride / 2) + c] : 0u;
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
                    if (key > pos || (key <= pos - window && key >= sinks)) continue;
                    uint32_t *y = at(r);
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

// The n lowest bits (none for n < 0).
__device__ __forceinline__ uint32_t low_bits(int n) {
    uint32_t x;
    asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(x) : "r"(imax(n, 0)));
    return x;
}

// The rows of a softmax warp's query tile: a row per thread, its running maximum m
// and sum l (base 2, scores scaled by cl).  s_read is called when the scores are in
// registers, wait_prev waits for the P V of the tile before (false: gave up).
// BITS: masks as bits of 32 keys, which chunks of keys that a warp sees go without.  Packed
// sequences start anywhere in a tile, so that twice as many are masked (chunks of a window of 1024:
// 66.8 us with one bound per tile, 61.5 with bits; 8 x 1024 tokens 74.6 and 73.1); the
// kernel for one length loses more on plain steps (D 64 0.706 us, 0.762 with bits; 4096
// tokens of D 128 91.5 us, 93.6).
template <int D, bool F16, bool BITS>
struct SoftRows {
    using C = WnCfg<D>;
    static constexpr int BN = kBN;
    static constexpr bool SEP_P = C::SEP_P;
    uint32_t s_addr, p_addr, o_addr;
    float cl;
    float m = -INFINITY, l = 0.f;

    // A first tile that holds a few sinks, which every row sees: kFew columns.
    template <typename Read>
    __device__ __forceinline__ void few_sinks(int sinks, Read s_read) {
        float x[kFew];
        ptx::tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
        ptx::tmem_wait_ld();
        s_read();
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < kFew; ++e) {
            if (e >= sinks) x[e] = -INFINITY;
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
    }

    // Keys k0 .. k0 + 127 (row `row` of the tile is at position pos + row).  first: the
    // item's first tile; seen_before: every row of the warp has seen a key.
    template <typename Read, typename Wait>
    __device__ __forceinline__ bool tile(int k0, int pos, int row, int window, int sinks, bool first, bool seen_before,
                                         Read s_read, Wait wait_prev) {
        float sv[BN];
#pragma unroll
        for (int c = 0; c < BN / 32; ++c)
            ptx::tmem_ld32(s_addr + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[c * 32]));
        ptx::tmem_wait_ld();
        s_read();

        // ---- masks: rows at positions pos + row; only tiles on an edge of
        //      the window are masked per element
        {
            const bool late = k0 + BN - 1 > pos;                    // a key behind the first row
            const bool early = k0 + window < pos + kBM;            // one before the last row's window
            if (late || (early && k0 + BN > sinks)) {
                // key e of the tile is seen iff e <= hi and (e >= lo or e < sk)
                const int hi = pos + row - k0, lo = hi - window + 1, sk = sinks - k0;
                if constexpr (BITS) {
                    // 32 keys at a time, untouched where every row of the warp sees them all
#pragma unroll
                    for (int c = 0; c < BN; c += 32) {
                        const uint32_t seen = low_bits(hi + 1 - c) & (~low_bits(lo - c) | low_bits(sk - c));
                        if (__all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(seen & (1u << e))) sv[c + e] = -INFINITY;
                    }
                } else
                // all but tiny windows need only one bound per tile: the
                // diagonal's, the end of the sinks, or the window's start
                if (!early || (!late && k0 + window + BN <= pos + 1)) {
                    const int last = early ? sk - 1 : hi;
#pragma unroll
                    for (int e = 0; e < BN; ++e)
                        if (e > last) sv[e] = -INFINITY;
                } else if (!late && sk <= 0) {
#pragma unroll
                    for (int e = 0; e < BN; ++e)
                        if (e < lo) sv[e] = -INFINITY;
                } else {
#pragma unroll
                    for (int e = 0; e < BN; ++e)
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
            for (int c = 0; c < BN / 32; ++c) {
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
        if (SEP_P && !first) {
            if (!wait_prev()) return false;
            prev_done = true;
        }

        // ---- fast path: exponentiate against the running maximum m as it
        //      stands, with no tile maximum.  P only has to stay finite in its
        //      16-bit type, not below 1: a tile whose row sum exceeds 2^24 (2^15
        //      for f16, whose largest finite value is 65504) or is not finite
        //      is redone below against its own maximum.  After the first tiles
        //      m is close to the row maximum and the redo almost never runs.
        bool fast = false, keep = false;      // this row's maximum may stay
        if (seen_before) {
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
            for (int e = 0; e < BN; e += 8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) mx[i] = fmaxf(mx[i], sv[e + i]);
            }
            const float tmax = fmaxf(ptx::fmax3(ptx::fmax3(mx[0], mx[1], mx[2]), ptx::fmax3(mx[3], mx[4], mx[5]),
                                                mx[6]),
                                     mx[7]);
            const float mt = tmax * cl;      // cl > 0: max commutes with the scaling

            // ---- the previous P V must be done before O is rescaled
            // (a row that a redo for other rows' sake takes along keeps it)
            const bool want = first || (!keep && mt > m + 8.f);   // this row moves its maximum
            const bool any_want = __any_sync(0xffffffffu, want);
            if (!first && any_want && !prev_done) {
                if (!wait_prev()) return false;
            }
            // ---- running maximum (moved lazily) and O rescale in TMEM
            if (first) {
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
        return true;
    }
};

}  // namespace
}  // namespace attn
