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
#include "ptx.cuh"
#include "window_tiles.cuh"

namespace attn {
namespace {

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
    const void *v;           // with element strides: values cleared from an edge tile
    TensorStrides sv;
    void *o;
    long long o_sb, o_sh, o_sn;
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
};

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
    plan_item(w, p.off, p.Nq, p.window, p.sinks, half);
    return w;
}

// spoil_rows for the CTA's item.
template <int D, bool F16>
__device__ __noinline__ void spoil_item(const WnParams &p, uint8_t *stage, int first_pos, int rows) {
    const Item w = get_item(p);                      // (handed over it would live in memory)
    const int lane = threadIdx.x & 31;
    constexpr int CW = D / 64, CH = D / 8;
    auto at = [&](int r) {
        return reinterpret_cast<uint32_t *>(stage + (r * CH + ((lane * CW / 4) ^ (r & 7))) * 16) + lane * CW % 4;
    };
    spoil_rows<D, F16>(w, static_cast<const typename H16<F16>::T *>(p.v) + w.fb * p.sv.b + w.fkh * p.sv.h, p.sv.n,
                       p.Nkv, p.window, p.sinks, false, at, first_pos, rows);
}

template <int D, bool F16>
__global__ void __launch_bounds__(WnCfg<D>::NT, 1)
tc_window_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                 const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tvs,
                 const __grid_constant__ WnParams p) {
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
        load_item = get_item(p);
        if (warp == C::W_LOADV && load_item.w_sk > 0) ptx::prefetch_tmap(&tvs);
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    // programmatic dependent launch: the set-up above touches nothing global
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

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
            const Item w = load_item;
            int q_out = 0, issued = 0;
            auto load_q = [&](int t) {
                if (t >= (w.n[1] > 0 ? kNQ : 1)) return;
                ++q_out;
                ptx::mbar_arrive_expect_tx(&bars->q_full[t], C::Q_BYTES);
                for (int pn = 0; pn < C::PANELS; ++pn)
                    ptx::tma_load_4d(smem + C::OFF_Q + t * C::Q_BYTES + pn * C::PANEL_Q, &tq, pn * 64,
                                     w.q0 + t * w.dq, w.fh + t * w.dh, w.fb, &bars->q_full[t], pol_q);
            };
            if (which == 0 && w.steps > 0) load_q(0);
            for (int j = 0; j < w.steps; ++j) {
                const int s = j % NS;
                if (j >= NS && !ptx::mbar_wait_or_abort(&empty[s], ((j / NS) - 1) & 1, p.err, abort)) break;
                issued = j + 1;
                ptx::mbar_arrive_expect_tx(&full[s], C::KV_BYTES);
                for (int pn = 0; pn < C::PANELS; ++pn)
                    ptx::tma_load_4d(smem + (which == 0 ? C::k_off(s) : C::v_off(s)) + pn * C::PANEL_KV,
                                     which == 1 && w.sink_tile(j) ? &tvs : tm, pn * 64, w.tile(j) * kBN, w.fkh, w.fb, &full[s], pol_kv);
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
            const Item w = get_item(p);
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
            const Item w = get_item(p);
            for (int j = 0; j < w.steps; ++j) {
                const int s = j % C::VS;
                if (!__all_sync(0xffffffffu, ptx::mbar_wait_or_abort(&bars->v_in[s], (j / C::VS) & 1, p.err, abort)))
                    break;
                const bool any = w.edge(j) && clear_wild<D, F16>(smem + C::v_off(s));
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
        bool ok = true;
        const Item w = get_item(p);
        const int f = pick(w.f, t), nt = pick(w.n, t) - f;   // this query tile's key tiles
        const int pos = p.off + w.q0 + w.dq * t;             // position of its first row

        // waits for the P V product of key tile jj of this query tile (and so
        // for every earlier one: one thread's MMAs complete in issue order)
        auto wait_pv = [&](int jj) -> bool {
            if (!__all_sync(0xffffffffu, ptx::mbar_wait_or_abort(&bars->o_done[t], jj & 1, p.err, abort)))
                return false;
            ptx::tc_fence_after();
            return true;
        };

        SoftRows<D, F16, false> rows{s_addr, p_addr, o_addr, p.c_log2};
        // S_t is in registers: the next QK_t may overwrite it
        auto s_read = [&]() {
            if constexpr (C::SEP_P) {
                ptx::tc_fence_before();
                ptx::mbar_arrive(&bars->s_free[t]);
            }
        };
        int j = 0;
        // the key tile from which on every row of the warp has seen a key before: of
        // the first one the last rows may see nothing, and then see the next
        const int k_first = w.tile(f) * kBN;
        const int seen_from = k_first < p.sinks || pos + quarter * 32 + 32 - p.window < k_first + kBN ? 1 : 2;
        if (w.few && nt > 0) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait_or_abort(&bars->s_full[t], 0, p.err, abort));
            if (ok) {
                ptx::tc_fence_after();
                rows.few_sinks(p.sinks, s_read);
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
            if (!rows.tile(w.tile(f + j) * kBN, pos, row, p.window, p.sinks, j == 0, j >= seen_from, s_read,
                           [&]() { return wait_pv(j - 1); })) {
                ok = false;
                break;
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            ptx::mbar_arrive(&bars->p_ready[t]);
        }


        // ---- epilogue: O / l -> 16-bit -> global
        if (ok && nt > 0 && wait_pv(nt - 1)) {
            const float inv = 1.f / rows.l;
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
                spoil_item<D, F16>(p, stage, p.off + q_first, imin(32, p.Nq - q_first));
            typename H16<F16>::T *const o0 = static_cast<typename H16<F16>::T *>(p.o) + w.fb * p.o_sb + qh * p.o_sh;
            const int col = ln % CH;
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += 32 / CH) {
                const int r = r0 + ln / CH;
                const uint4 x = *reinterpret_cast<const uint4 *>(stage + (r * CH + (col ^ (r & 7))) * 16);
                if (q_first + r < p.Nq)
                    *reinterpret_cast<uint4 *>(o0 + (q_first + r) * p.o_sn + col * 8) = x;
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

template <int D, bool F16>
attn_status_t launch_window(const Ctx &c, const CUtensorMap &tq, const CUtensorMap &tk,
                            const CUtensorMap &tv, const CUtensorMap &tvs, const WnParams &p) {
    using C = WnCfg<D>;
    static int done_mask = 0;
    static int regs = -1;
    auto kern = tc_window_kernel<D, F16>;
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
    cfg.gridDim = dim3(p.whole + 2 * (p.pairs - p.whole));
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
    if (D == 128)
        return f16 ? launch_window<128, true>(c, tq, tk, tv, tvs, p) : launch_window<128, false>(c, tq, tk, tv, tvs, p);
    return f16 ? launch_window<64, true>(c, tq, tk, tv, tvs, p) : launch_window<64, false>(c, tq, tk, tv, tvs, p);
}

}  // namespace attn
