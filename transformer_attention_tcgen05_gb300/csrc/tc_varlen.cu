// Tensor-core (tcgen05 + TMEM + TMA) causal grouped-query attention over packed
// sequences of different lengths, bf16 and f16, sm_103a.
//
// The tile arithmetic is that of the windowed kernel (tc_window.cu, window_tiles.cuh):
// pairs of 128-row query tiles over a list of 128-key tiles, P in tensor memory, a
// row per softmax thread; masks are made of bits (SoftRows).  What differs:
//
//  * Items come from the device.  A block of query rows and the head pair that works on
//    it are found from the sequences' starts (packed.cuh), the longest first for up to 64
//    of them.
//  * A CTA stays on its SM and takes the items of CTAs that have not started off the
//    launch (clusterlaunchcontrol), in the order of the list.  Items differ in length and
//    number of tiles: dealt out in turn, some SMs worked twice as long as others (chunks
//    behind long pasts: 39 to 77 us).
//  * A batch of prompts has many short items: of the 7.4 us that an item of one key tile
//    took as a CTA of its own, 5.7 were start, finding the item, first copies and scores
//    (4.1), and the last P V and the way out (1.6).  Here the loader finds the next item
//    and copies its first keys while the current one is computed, and the MMA warp computes
//    its first scores while the softmax warps write the current rows out: the last rows of
//    an item and the next one's first scores are 1.5 to 3 us apart.
//  * A thread writes its output row itself, in whole sectors (32-byte stores), so that
//    the query tiles are free for the next item as soon as the last scores are computed
//    and nothing of the way out waits (through shared memory it took 2 us per item).
//  * The values of a sequence's sinks cannot come through a tensor map that ends behind
//    them: sink tiles are looked over like the tiles of an edge.
//
// 16-bit, 32 heads on 8, D 128: one prompt of 4096 tokens 95 us (1440 TFLOP/s over the
// visible pairs; 92 in the kernel for one length), 8 of 1024 73 us (79), 64 of 128 43 us
// (50), 16 prompts of 1 to 6000 tokens 190 us (1355 TFLOP/s, 71% of the measured product).  A
// step of two tiles takes 1.18 us for D 128 and 0.77 for D 64 (0.99 and 0.49 at the
// tensor pipe's rate); 1.5 us where all of its rows are on an edge, and 1.1 for a tile
// alone.  Measured and not kept: no exponentials for keys that no row of a warp sees (step
// 0.77 -> 0.87: the exponentials of a tile are no longer one block of instructions; as a
// second copy of them 0.86 and cold instructions), heads in pairs also where the group is
// odd (7 x 2048 tokens 101 -> 109 us).
//
// All spin-waits are bounded (1 s); on a timeout the CTA raises the device error word,
// drains what it issued, frees TMEM and exits.
#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "packed.cuh"
#include "ptx.cuh"
#include "window_tiles.cuh"

namespace attn {
namespace {

struct VlParams {
    PackedSeqs seqs;
    int window, sinks;       // window: wider than any sequence for none
    float c_log2;            // scale * log2(e)
    unsigned *err;
    int by_head;             // a pair is two heads of one KV head (else two row tiles)
    Div by_hp, by_group;     // pairs (or heads) per block of rows, heads per KV head
    Div by_sm;               // SMs
    const void *v;
    void *o;
    long long sv_h, sv_n, o_sh, o_sn;    // element strides (head, token)
    int wide;                // rows of o are 32-byte aligned
};

struct VlItem : Item {
    int nq, nkv, off;        // the sequence's lengths, its first query's position
    int q_row, k_row;        // its rows in the arrays
};

// register split of a launch of 168 per thread: with 216 for the softmax warps, as in
// the windowed kernel, a few of their values would lie in memory
constexpr int kRegsSoftmax = 224, kRegsOther = 56;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsOther <= WnCfg<128>::NT * WnCfg<128>::REGS_LAUNCH,
              "setmaxnreg split must fit the launch's register file share");

// Query tiles for D = 64 lie in two places in turn, so that an item's are copied as soon
// as it is found (7 sequences of 2048, 24 heads, window 1024: 103 us with one place, 100;
// 97 with the masks as bits);
// for D = 128 the rings leave no room, and they follow the last scores of the item before.
template <int D>
struct VlCfg : WnCfg<D> {
    using W = WnCfg<D>;
    static constexpr int QS = D == 64 ? 2 : 1;
    static constexpr int q_off(int slot) { return slot ? W::OFF_BAR : W::OFF_Q; }
    static constexpr int OFF_BAR = W::OFF_BAR + (QS - 1) * kNQ * W::Q_BYTES;
    static constexpr int SMEM = OFF_BAR + W::BARS + 1024;
    static_assert(SMEM <= 227 * 1024, "must fit a CTA's shared memory");
};

constexpr int kItemUsers = 2 + 1 + 4 * kNQ;    // V loader, MMA, check; softmax warps

// Barrier block at OFF_BAR.  Phases run on from item to item.
template <int KS, int VS, int QS>
struct VlBars {
    uint64_t item_full[2], item_empty[2];
    uint64_t q_full[QS][kNQ], q_empty[kNQ];        // q_empty: QS 1 (else the item before the last is)
    // v_in: the stage's copies have landed; v_full: the checking warp has passed it on
    uint64_t k_full[KS], k_empty[KS], v_in[VS], v_full[VS], v_empty[VS];
    // per query tile t: s_full its Q K^T has completed, p_ready the softmax has written P,
    // o_done the P V product that read P has completed, o_free the softmax has read the
    // item's O, s_free (separate P, D = 64) the softmax holds S_t in registers
    uint64_t s_full[kNQ], p_ready[kNQ], o_done[kNQ], o_free[kNQ], s_free[kNQ];
    uint64_t drain, checked[2];    // checked: every value of the item has been looked over
    uint64_t taken;                // the answer has come
    alignas(16) uint64_t answer[2];
    uint32_t tmem_base;
    int abort, wild[2];            // wild: a value was cleared from one of them
    VlItem item[2];                // steps -1: there are no more
};

// An item by its index (one warp): whole pairs, longest first, then the pairs of a last
// round that takes at most half of the SMs as single tiles.  No steps: there is no such
// item, or it is a second row tile past its sequence's end.
__device__ __forceinline__ VlItem find_item(const VlParams &p, const BlockFinder &finder, int index) {
    const int pairs = finder.total * p.by_hp.d, rest = pairs - p.by_sm(pairs) * p.by_sm.d;
    const int whole = 2 * rest <= p.by_sm.d ? pairs - rest : pairs;
    const int s = index - whole;
    const int pair = s < 0 ? index : whole + (s >> 1), half = s < 0 ? -1 : s & 1;
    VlItem w{};
    w.steps = -1;
    if (index < 0 || pair >= pairs) return w;
    const int block = p.by_hp(pair);
    const PackedBlock b = finder.find(block);
    w.dq = p.by_head ? 0 : kBM;
    w.dh = p.by_head ? 1 : 0;
    w.fh = (pair - block * p.by_hp.d) * (p.by_head ? 2 : 1) + (half > 0 ? w.dh : 0);
    w.fkh = p.by_group(w.fh);
    w.q0 = b.q0 + (half > 0 ? w.dq : 0);
    w.nq = b.nq;
    w.nkv = b.nkv;
    w.off = b.nkv - b.nq;
    w.q_row = b.q_row;
    w.k_row = b.k_row;
    plan_item(w, w.off, w.nq, p.window, p.sinks, half);
    return w;
}

// Adds the values cleared from an item's tiles to a warp's rows, which are written:
// o0 is the first, at position first_pos.
template <int D, bool F16>
__device__ __noinline__ void spoil_item(const VlParams &p, const VlItem *item, typename H16<F16>::T *o0, int first_pos,
                                        int rows) {
    const VlItem w = *item;
    auto at = [&](int r) { return reinterpret_cast<uint32_t *>(o0 + r * p.o_sn) + (threadIdx.x & 31) * (D / 64); };
    __syncwarp();
    spoil_rows<D, F16>(w, static_cast<const typename H16<F16>::T *>(p.v) + w.fkh * p.sv_h + w.k_row * p.sv_n, p.sv_n,
                       w.nkv, p.window, p.sinks, true, at, first_pos, rows);
}

// 32 bytes to global memory, 32-byte aligned.
__device__ __forceinline__ void store32(void *at, const uint32_t (&x)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(x[0]), "r"(x[1]),
                 "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

template <int D, bool F16>
__global__ void __launch_bounds__(WnCfg<D>::NT, 1)
tc_varlen_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                 const __grid_constant__ CUtensorMap tv, const __grid_constant__ VlParams p) {
    using C = VlCfg<D>;
    using BarsT = VlBars<C::KS, C::VS, C::QS>;
    static_assert(sizeof(BarsT) <= C::BARS, "barrier block must fit its reserved bytes");
    extern __shared__ uint8_t smem_raw[];
    // 1024-byte alignment for the 128-byte swizzle atoms
    uint8_t *smem = smem_raw + ((1024 - (ptx::smem_addr(smem_raw) & 1023)) & 1023);
    BarsT *bars = reinterpret_cast<BarsT *>(smem + C::OFF_BAR);
    volatile int *abort = &bars->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

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
            for (int s = 0; s < C::QS; ++s) ptx::mbar_init(&bars->q_full[s][t], 1);
            ptx::mbar_init(&bars->q_empty[t], 1);
            ptx::mbar_init(&bars->s_full[t], 1);
            ptx::mbar_init(&bars->p_ready[t], 128);
            ptx::mbar_init(&bars->o_done[t], 1);
            ptx::mbar_init(&bars->o_free[t], 128);
            ptx::mbar_init(&bars->s_free[t], 128);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(&bars->item_full[s], 1);
            ptx::mbar_init(&bars->item_empty[s], kItemUsers);
            ptx::mbar_init(&bars->checked[s], 1);
        }
        ptx::mbar_init(&bars->drain, 1);
        ptx::mbar_init(&bars->taken, 1);
        bars->abort = 0;
        ptx::fence_barrier_init();
    }
    if (warp == C::W_MMA) {
        ptx::tmem_alloc(&bars->tmem_base, C::TM_COLS);
        ptx::tmem_relinquish();
    }
    if (warp == C::W_LOAD) {
        ptx::prefetch_tmap(&tq);
        ptx::prefetch_tmap(&tk);
        ptx::prefetch_tmap(&tv);
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    // programmatic dependent launch: the set-up above touches nothing global
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return ptx::mbar_wait_or_abort(bar, parity, p.err, abort);
    };
    auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {   // a whole warp
        return __all_sync(0xffffffffu, ptx::mbar_wait_or_abort(bar, parity, p.err, abort));
    };

    if (warp >= C::NSOFT) {
        ptx::regs_decrease<kRegsOther>();
        const uint64_t pol_kv = ptx::l2_policy_evict_last(), pol_q = ptx::l2_policy_evict_first();
        if (warp == C::W_LOAD) {
            // ============================================= items, Q and the K ring: the
            // warp finds an item, one thread copies
            const BlockFinder finder(p.seqs, p.by_head ? 7 : 8, blockIdx.x == 0, p.err);
            int g = 0;                                 // key tiles so far
            // per place of a query tile (bit): copied to before, parity of the copies so far
            uint32_t q_used = 0, q_par = 0;
            bool ok = true;
            int index = blockIdx.x, asked = 0;         // -1: every item has been taken
            bool open = false;                         // an answer is on its way
            auto next = [&]() {
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(&bars->taken, 16);
                    ptx::take_block(bars->answer, &bars->taken);
                }
                open = true;
                ok = wait_all(&bars->taken, asked & 1);
                if (!ok) return;
                ++asked;
                open = false;
                index = ptx::taken_block(bars->answer);
                __syncwarp();
                ptx::fence_proxy_async_smem();         // read before the next answer is written
            };
            for (int it = 0; ok; ++it) {
                const int s = it & 1;
                if (it >= 2) ok = wait_all(&bars->item_empty[s], ((it >> 1) - 1) & 1);
                if (!ok) break;
                // (behind the last item, too, every index is taken: no CTA starts for it)
                VlItem w{};
                while (ok) {
                    w = find_item(p, finder, index);
                    if (w.steps > 0 || index < 0) break;
                    next();
                }
                if (!ok) break;
                if (lane == 0) {
                    bars->item[s] = w;
                    bars->wild[s] = 0;
                    ptx::mbar_arrive(&bars->item_full[s]);
                }
                if (w.steps < 0) break;
                if (lane == 0) {
                    auto load_q = [&](int t) {
                        if (w.n[t] <= 0) return;
                        const int slot = C::QS == 1 ? 0 : s;
                        const uint32_t bit = 1u << (slot * kNQ + t);
                        if (C::QS == 1 && (q_used & bit)) ok = ok && wait(&bars->q_empty[t], (q_par & bit) == 0);
                        if (!ok) return;
                        q_used |= bit;
                        q_par ^= bit;
                        uint64_t *const full = &bars->q_full[slot][t];
                        ptx::mbar_arrive_expect_tx(full, C::Q_BYTES);
                        for (int pn = 0; pn < C::PANELS; ++pn)
                            ptx::tma_load_4d(smem + C::q_off(slot) + t * C::Q_BYTES + pn * C::PANEL_Q, &tq, pn * 64,
                                             w.q_row + w.q0 + t * w.dq, w.fh + t * w.dh, 0, full, pol_q);
                    };
                    load_q(0);
                    for (int j = 0; ok && j < w.steps; ++j, ++g) {
                        const int r = g % C::KS;
                        if (g >= C::KS) ok = wait(&bars->k_empty[r], (g / C::KS - 1) & 1);
                        if (!ok) break;
                        ptx::mbar_arrive_expect_tx(&bars->k_full[r], C::KV_BYTES);
                        for (int pn = 0; pn < C::PANELS; ++pn)
                            ptx::tma_load_4d(smem + C::k_off(r) + pn * C::PANEL_KV, &tk, pn * 64,
                                             w.k_row + w.tile(j) * kBN, w.fkh, 0, &bars->k_full[r], pol_kv);
                        // the first scores need one query tile and the first keys
                        if (j == 0) load_q(1);
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                // Only now, with the item's last keys on their way: whoever asks before its
                // item is nearly done has the next one too early, and the SMs end unevenly
                if (ok) next();
            }
            // after a timeout: let the copies this thread issued land (bounded) before
            // the CTA's shared memory is released
            if (*abort && lane == 0) {
                if (open) ptx::mbar_wait(&bars->taken, asked & 1, nullptr);
                for (int i = 0; i < C::QS * kNQ; ++i)
                    if ((q_used >> i) & 1) ptx::mbar_wait(&bars->q_full[0][0] + i, ((q_par >> i) & 1) ^ 1, nullptr);
                for (int i = imax(0, g - C::KS); i < g; ++i)
                    ptx::mbar_wait(&bars->k_full[i % C::KS], (i / C::KS) & 1, nullptr);
            }
        } else if (warp == C::W_LOADV) {
            if (lane == 0) {
                // ========================================= the V ring
                int g = 0;
                bool ok = true;
                for (int it = 0; ok; ++it) {
                    const int s = it & 1;
                    if (!wait(&bars->item_full[s], (it >> 1) & 1)) break;
                    const VlItem w = bars->item[s];
                    if (w.steps < 0) break;
                    for (int j = 0; j < w.steps; ++j, ++g) {
                        const int r = g % C::VS;
                        if (g >= C::VS && !wait(&bars->v_empty[r], (g / C::VS - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        ptx::mbar_arrive_expect_tx(&bars->v_in[r], C::KV_BYTES);
                        for (int pn = 0; pn < C::PANELS; ++pn)
                            ptx::tma_load_4d(smem + C::v_off(r) + pn * C::PANEL_KV, &tv, pn * 64,
                                             w.k_row + w.tile(j) * kBN, w.fkh, 0, &bars->v_in[r], pol_kv);
                    }
                    ptx::mbar_arrive(&bars->item_empty[s]);
                }
                if (*abort)
                    for (int i = imax(0, g - C::VS); i < g; ++i)
                        ptx::mbar_wait(&bars->v_in[i % C::VS], (i / C::VS) & 1, nullptr);
            }
        } else if (warp == C::W_MMA) {
            // ============================================= MMA issuer: the whole warp
            // walks the steps, one thread issues
            const bool lead = ptx::elect_one();
            const uint32_t id_qk = ptx::idesc_16_f32(kBM, kBN, false, F16);
            const uint32_t id_few = ptx::idesc_16_f32(kBM, kFew, false, F16);
            const uint32_t id_pv = ptx::idesc_16_f32(kBM, D, true, F16);
            constexpr uint32_t HI128 = ptx::desc_hi_sw128(1024);
            const uint32_t dq0 = ptx::desc_lo_sw128(ptx::smem_addr(smem + C::q_off(0)), 16);
            const uint32_t dk0 = ptx::desc_lo_sw128(ptx::smem_addr(smem + C::k_off(0)), 16);
            const uint32_t dv0 = ptx::desc_lo_sw128(ptx::smem_addr(smem + C::v_off(0)), C::PANEL_KV);
            // ring slots and their phases' parities; per query tile (bit t) the parities of
            // its scores, weights and items.  (A fresh barrier's phase before the first
            // counts as completed: "free" barriers are waited on with the other parity.)
            int ks = 0, kp = 0, vs = 0, vp = 0;
            uint32_t score_par = 0, weigh_par = 0, item_par = 0, q_par = 0;   // (q_par: per place)
            int slot = 0;                              // place of the item's query tiles
            bool ok = true;
            auto issue_qk = [&](int t, uint32_t id) {
                if (!lead) return;
                const uint32_t a0 = dq0 + uint32_t((slot * (C::q_off(1) - C::q_off(0)) + t * C::Q_BYTES) >> 4);
                const uint32_t b0 = dk0 + uint32_t(ks * (C::KV_BYTES >> 4));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t oa = ((kk >> 2) * C::PANEL_Q + (kk & 3) * 32) >> 4;
                    const uint32_t ob = ((kk >> 2) * C::PANEL_KV + (kk & 3) * 32) >> 4;
                    ptx::mma_ss(tmem + C::tm_s(t), ptx::desc_join(a0 + oa, HI128), ptx::desc_join(b0 + ob, HI128), id,
                                kk > 0);
                }
                ptx::tc_commit(&bars->s_full[t]);
            };
            auto issue_pv = [&](int t, bool first, bool few) {
                if (!lead) return;
                const uint32_t b0 = dv0 + uint32_t(vs * (C::KV_BYTES >> 4));
                const uint32_t a0 = tmem + C::tm_p(t);
#pragma unroll
                for (int kk = 0; kk < kBN / 16; ++kk) {
                    if (kk == kFew / 16 && few) break;
                    ptx::mma_ts(tmem + C::tm_o(t), a0 + kk * 8, ptx::desc_join(b0 + uint32_t(kk * (2048 >> 4)), HI128),
                                id_pv, (!first || kk > 0) ? 1u : 0u);
                }
                ptx::tc_commit(&bars->o_done[t]);
            };
            // Q K^T of a step for tile t, once the softmax no longer needs the S it
            // overwrites (separate P: as soon as the softmax holds the S before in
            // registers; P over S: after the P V before, issued already)
            auto qk = [&](int t, uint32_t id) {
                if (C::SEP_P) ok = ok && wait(&bars->s_free[t], ((score_par >> t) & 1) ^ 1);
                if (!ok) return;
                score_par ^= 1u << t;
                ptx::tc_fence_after();
                issue_qk(t, id);
            };
            // P V of a step for tile t; the item's first overwrites the O of the item before
            auto pv = [&](int t, bool first, bool few) {
                if (first) {
                    ok = ok && wait(&bars->o_free[t], ((item_par >> t) & 1) ^ 1);
                    item_par ^= 1u << t;
                }
                ok = ok && wait(&bars->p_ready[t], (weigh_par >> t) & 1);
                if (!ok) return;
                weigh_par ^= 1u << t;
                ptx::tc_fence_after();
                issue_pv(t, first, few);
            };
            // the scores of a step are issued: its K stage may be overwritten when they are
            // done, and behind the last step the query tiles
            auto next_k = [&](bool last, const int (&n)[kNQ]) {
                if (ok && lead) {
                    ptx::tc_commit(&bars->k_empty[ks]);
                    if (C::QS == 1 && last)
                        for (int t = 0; t < kNQ; ++t)
                            if (n[t] > 0) ptx::tc_commit(&bars->q_empty[t]);
                }
                ks = ks + 1 == C::KS ? 0 : ks + 1;
                kp ^= ks == 0;
            };
            for (int it = 0; ok; ++it) {
                ok = wait(&bars->item_full[it & 1], (it >> 1) & 1);
                if (!ok) break;
                // The fields that a step needs, as values that the compiler knows to be the same
                // in all lanes: MMA operands made of anything else pass through vector registers
                const VlItem &item = bars->item[it & 1];
                auto same = [](int x) { return __reduce_max_sync(0xffffffffu, x); };
                const int steps = same(item.steps), n[kNQ] = {same(item.n[0]), same(item.n[1])}, f1 = same(item.f[1]);
                const bool few = same(item.few) != 0;
                if (steps < 0) break;
                if (C::QS == 2) slot = it & 1;
#pragma unroll
                for (int t = 0; t < kNQ; ++t)
                    if (n[t] > 0) {
                        const int i = slot * kNQ + t;
                        ok = ok && wait(&bars->q_full[0][0] + i, (q_par >> i) & 1);
                        q_par ^= 1u << i;
                    }
                ok = ok && wait(&bars->k_full[ks], kp);
                qk(0, few ? id_few : id_qk);
                if (n[1] > 0 && f1 == 0) qk(1, few ? id_few : id_qk);
                next_k(steps == 1, n);
                for (int j = 0; ok && j < steps; ++j) {
                    // (tile 0 works in steps [0, n[0]), tile 1 in [f1, n[1]))
                    const bool more = j + 1 < steps, few_now = few && j == 0;
                    if constexpr (C::SEP_P) {
                        if (more) {
                            ok = ok && wait(&bars->k_full[ks], kp);
                            if (j + 1 < n[0]) qk(0, id_qk);
                            if (j + 1 < n[1]) qk(1, id_qk);        // f1 is 0 or 1
                            next_k(j + 2 == steps, n);
                        }
                        ok = ok && wait(&bars->v_full[vs], vp);
                        if (j < n[0]) pv(0, j == 0, few_now);
                        if (j >= f1 && j < n[1]) pv(1, j == f1, few_now);
                    } else {
                        ok = ok && wait(&bars->v_full[vs], vp);
                        if (j < n[0]) pv(0, j == 0, few_now);
                        if (more) {
                            ok = ok && wait(&bars->k_full[ks], kp);
                            if (j + 1 < n[0]) qk(0, id_qk);
                        }
                        if (j >= f1 && j < n[1]) pv(1, j == f1, few_now);
                        if (more) {
                            if (j + 1 < n[1]) qk(1, id_qk);
                            next_k(j + 2 == steps, n);
                        }
                    }
                    if (ok && lead) ptx::tc_commit(&bars->v_empty[vs]);
                    vs = vs + 1 == C::VS ? 0 : vs + 1;
                    vp ^= vs == 0;
                }
                __syncwarp();
                if (lead) ptx::mbar_arrive(&bars->item_empty[it & 1]);
            }
            // drain: every MMA has completed before TMEM is freed
            if (lead) ptx::tc_commit(&bars->drain);
            ptx::mbar_wait(&bars->drain, 0, p.err);
        } else {
            // ============================================= the V of edge and sink tiles
            // is looked over as it arrives; other tiles are passed on at once
            int g = 0;
            bool ok = true;
            for (int it = 0; ok; ++it) {
                const int s = it & 1;
                if (!wait_all(&bars->item_full[s], (it >> 1) & 1)) break;
                const VlItem w = bars->item[s];
                if (w.steps < 0) break;
                for (int j = 0; j < w.steps; ++j, ++g) {
                    const int r = g % C::VS;
                    if (!wait_all(&bars->v_in[r], (g / C::VS) & 1)) {
                        ok = false;
                        break;
                    }
                    const bool any = (w.edge(j) || w.sink_tile(j)) && clear_wild<D, F16>(smem + C::v_off(r));
                    __syncwarp();
                    if (lane == 0) {
                        if (any) bars->wild[s] = 1;
                        ptx::mbar_arrive(&bars->v_full[r]);
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(&bars->checked[s]);
                    ptx::mbar_arrive(&bars->item_empty[s]);
                }
            }
        }
    } else {
        // ================================================= softmax warpgroups
        ptx::regs_increase<kRegsSoftmax>();
        const int t = warp >> 2;                 // query tile
        const int quarter = warp & 3;            // TMEM lanes [32 quarter, 32 quarter + 32)
        const int row = quarter * 32 + lane;     // query row within the tile
        const uint32_t lane_base = tmem + (uint32_t(quarter * 32) << 16);
        const uint32_t o_addr = lane_base + C::tm_o(t);
        int base = 0;                            // key tiles of the items before
        // S_t is in registers: the next QK_t may overwrite it
        auto s_read = [&]() {
            if constexpr (C::SEP_P) {
                ptx::tc_fence_before();
                ptx::mbar_arrive(&bars->s_free[t]);
            }
        };
        // waits for the P V product of this query tile's key tile jj, counted from the
        // first item on (and so for every earlier one: one thread's MMAs complete in order)
        auto wait_pv = [&](int jj) -> bool {
            if (!wait_all(&bars->o_done[t], jj & 1)) return false;
            ptx::tc_fence_after();
            return true;
        };
        bool ok = true;
        for (int it = 0; ok; ++it) {
            const int s = it & 1;
            if (!wait_all(&bars->item_full[s], (it >> 1) & 1)) break;
            const VlItem &w = bars->item[s];     // (read where needed: registers are short here)
            if (w.steps < 0) break;
            const int f = w.f[t], nt = w.n[t] - f;               // this query tile's key tiles
            if (nt > 0) {
                const int pos = w.off + w.q0 + w.dq * t;         // position of its first row
                const int lead = f - w.f[1], lo = w.w_lo, sk = w.w_sk;
                auto key_of = [&](int j) {                       // first key of its tile j (Item::tile)
                    const int i = lead + j;
                    return (i < 0 ? lo : i < sk ? i : lo + f + j - sk) * kBN;
                };
                SoftRows<D, F16, true> rows{lane_base + C::tm_s(t), lane_base + C::tm_p(t), o_addr, p.c_log2};
                int j = 0;
                // the key tile from which on every row of the warp has seen a key before: of
                // the first one the last rows may see nothing, and then see the next
                const int k_first = key_of(0);
                const int seen_from = k_first < p.sinks || pos + quarter * 32 + 32 - p.window < k_first + kBN ? 1 : 2;
                if (w.few) {
                    ok = wait_all(&bars->s_full[t], base & 1);
                    if (ok) {
                        ptx::tc_fence_after();
                        rows.few_sinks(p.sinks, s_read);
                        ptx::mbar_arrive(&bars->p_ready[t]);
                        j = 1;
                    }
                }
                for (; ok && j < nt; ++j) {
                    if (!wait_all(&bars->s_full[t], (base + j) & 1)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    if (!rows.tile(key_of(j), pos, row, p.window, p.sinks, j == 0, j >= seen_from, s_read,
                                   [&]() { return wait_pv(base + j - 1); })) {
                        ok = false;
                        break;
                    }
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(&bars->p_ready[t]);
                }
                base += nt;
                // ---- epilogue: O / l -> 16-bit -> global, whole sectors of the thread's row
                if (ok && wait_pv(base - 1)) {
                    float ov[D];
#pragma unroll
                    for (int c = 0; c < D / 32; ++c)
                        ptx::tmem_ld32(o_addr + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&ov[c * 32]));
                    ptx::tmem_wait_ld();
                    // the next item's P V may overwrite O
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(&bars->o_free[t]);
                    const float inv = 1.f / rows.l;
                    const int q_first = w.q0 + t * w.dq + quarter * 32, left = w.nq - q_first;
                    typename H16<F16>::T *const o0 = static_cast<typename H16<F16>::T *>(p.o) +
                                                     (w.fh + t * w.dh) * p.o_sh + (w.q_row + q_first) * p.o_sn;
                    typename H16<F16>::T *const to = o0 + lane * p.o_sn;
                    if (lane < left) {
#pragma unroll
                        for (int c = 0; c < D; c += 16) {
                            uint32_t x[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                x[e] = H16<F16>::pack(ov[c + 2 * e] * inv, ov[c + 2 * e + 1] * inv);
                            if (p.wide) {
                                store32(to + c, x);
                            } else {
                                *reinterpret_cast<uint4 *>(to + c) = make_uint4(x[0], x[1], x[2], x[3]);
                                *reinterpret_cast<uint4 *>(to + c + 8) = make_uint4(x[4], x[5], x[6], x[7]);
                            }
                        }
                    }
                    ok = wait_all(&bars->checked[s], (it >> 1) & 1);
                    if (ok && *reinterpret_cast<volatile int *>(&bars->wild[s]))
                        spoil_item<D, F16>(p, &bars->item[s], o0, w.off + q_first, imin(32, left));
                } else {
                    ok = false;
                }
            }
            __syncwarp();                            // (every lane has read the item)
            if (lane == 0) ptx::mbar_arrive(&bars->item_empty[s]);
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
attn_status_t launch_varlen(const Ctx &c, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                            const VlParams &p, int grid) {
    using C = VlCfg<D>;
    static int done_mask = 0;
    static int regs = -1;
    auto kern = tc_varlen_kernel<D, F16>;
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
    if (cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, p) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    return launch_status(kFamTcFlash);
}

}  // namespace

attn_status_t tc_causal_varlen(const Ctx &c, attn_dtype_t dt, const VarlenArgs &a) {
    const bool f16 = dt == ATTN_F16;
    // pairs of heads where the group is even, else pairs of row tiles (tc_window.cu)
    const bool by_head = (a.Hq / a.Hkv) % 2 == 0;
    const int bs = by_head ? kBM : kNQ * kBM, hp = by_head ? a.Hq / 2 : a.Hq;
    const long long blocks = BlockFinder::most(a.B, a.Nq, bs);
    if (blocks * hp > (1 << 29)) return ATTN_ERR_UNSUPPORTED;
    CUtensorMap tq, tk, tv;
    // a layout the tensor-map encoder refuses goes to the SIMT kernel
    if (!make_tmap4(&tq, a.q, a.D, a.Nq, a.Hq, 1, a.st[0], f16) ||
        !make_tmap4(&tk, a.k, a.D, a.Nkv, a.Hkv, 1, a.st[1], f16) ||
        !make_tmap4(&tv, a.v, a.D, a.Nkv, a.Hkv, 1, a.st[2], f16))
        return ATTN_ERR_UNSUPPORTED;
    VlParams p{};
    p.seqs = PackedSeqs{a.cu_q, a.cu_k, a.B, a.Nq, a.Nkv, int(blocks)};
    p.window = a.window;
    p.sinks = a.sinks;
    p.c_log2 = a.scale * kLog2e;
    p.err = c.err;
    p.by_head = by_head;
    p.by_hp = Div(hp);
    p.by_group = Div(a.Hq / a.Hkv);
    p.by_sm = Div(c.sm_count);
    p.v = a.v;
    p.o = a.o;
    p.sv_h = a.st[2].h; p.sv_n = a.st[2].n;
    p.o_sh = a.st[3].h; p.o_sn = a.st[3].n;
    p.wide = ((reinterpret_cast<uintptr_t>(a.o) | uintptr_t(p.o_sh * 2) | uintptr_t(p.o_sn * 2)) & 31u) == 0;
    // an index for every item that there can be (at most half an SM count of pairs is
    // given out as two single tiles)
    const int grid = int(blocks * hp + (blocks * hp < c.sm_count / 2 ? blocks * hp : c.sm_count / 2));
    if (a.D == 128)
        return f16 ? launch_varlen<128, true>(c, tq, tk, tv, p, grid) : launch_varlen<128, false>(c, tq, tk, tv, p, grid);
    return f16 ? launch_varlen<64, true>(c, tq, tk, tv, p, grid) : launch_varlen<64, false>(c, tq, tk, tv, p, grid);
}

}  // namespace attn
