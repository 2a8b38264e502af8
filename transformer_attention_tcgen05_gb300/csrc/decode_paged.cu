// Grouped-query decode attention over a paged KV cache, with an optional
// sliding window and a few first tokens that stay visible (sinks).
//
// One query token per sequence b attends to the positions
//     K(b) = { j < len_b : j >= len_b - window  or  j < sinks }
// (window <= 0: every j < len_b); position j lives in row j % S of page
// page_table[b][j / S].  Per head, o = sum_j p_j v_j / sum_j p_j with
// p_j = 2^(x_j - max x), x_j = q . k_j * scale * log2(e).
//
// 4 FLOP per cache byte and query head: the work is bound by HBM, so the
// design streams every visible page once and keeps the SMs evenly loaded:
//
//  * Flat work list.  A sequence is cut into chunks of 32 positions (only those
//    that hold a visible one) and all chunks of all (sequence, KV head) units
//    are numbered consecutively; each of 2 CTAs per SM takes one equal
//    contiguous range.  Lengths are read on the device, so ragged batches and
//    a captured graph whose sequences grow stay balanced, and the page table
//    may be far wider than the sequences are long.
//  * A CTA whose range cuts a unit writes a partial (max, sum, O) per head to
//    the workspace; the last CTA of the unit to arrive (ticket) joins the
//    partials in CTA order, so the result does not depend on who is last.
//    (Drawing the tickets of a range's cut units only at its end, so that the
//    next unit need not wait, took 28.1 us for 8 x 4096 tokens when the kernel
//    took 27.1 without; it takes 25.1 now.)
//  * Short units (up to 5 chunks) beside long ones, or units of up to 8 chunks if
//    there are more of them than CTAs and no longer ones, are dealt out whole,
//    warp by warp, to a share of the CTAs that their work deserves: no joining, no
//    barrier.  (In the list of the long ones each
//    would cost its CTA a merge of four warps, 1.3 us, for a chunk or two.)
//  * Every warp streams chunks of its own (chunk f of the range goes to warp
//    f % CW) into shared memory of its own with TMA: a box of up to 32 rows x D
//    channels per copy, the page and the KV head being coordinates of one 5D
//    tensor map, so either memory order of a page costs nothing and addresses
//    are 64-bit.  A warp asks for its next K right after it has read this one
//    and for its next V after this one's P V; no warp waits for another inside
//    a unit.  The 32 lanes look up 32 boxes' pages at once, one group ahead, also
//    across units.  (With a producer warp for K and one for V the first four
//    chunks went out one after the other, 0.3 us each.)
//  * S^T = K q^T (rows x heads) and O^T += V^T P^T with mma.sync m16n8k16.
//    With at most 16 query heads per KV head the product is 8 or 16 columns
//    wide; the warp-level instruction takes the heads as its n = 8 columns,
//    leaves the softmax statistics in registers and P^T one 8 x 8 transpose
//    away from the next operand, where a tcgen05 tile would need 128 rows, a
//    round trip through tensor memory and P staged in shared memory, for a
//    tensor pipe that is mostly idle either way.
//  * P is split into two 16-bit terms (P = hi + lo), so the P V product keeps
//    ~16 bits of P instead of 8 (bf16): a second MMA on operands that are in
//    registers already.  Sums and statistics are fp32; the output is rounded
//    once.
#include <cuda.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "paged_walk.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kCtasPerSm = 2;
constexpr int kMaxCtas = 2 * 192; // workspace slots (2 CTAs on up to 192 SMs)

template <int D, int NT>
struct PgCfg {
    static constexpr int CW = 4;  // warps
    static constexpr int NS = D == 64 ? 2 : 1;              // chunks in flight per warp
    static constexpr int THREADS = CW * 32;
    static constexpr int HP = NT * 8;                       // padded heads per KV head
    static constexpr int PANELS = D / 64;
    static constexpr int TILE = kChunk * D * 2;             // K (or V) bytes of a chunk
    static constexpr int LDM = D + 4;                       // floats per merge row (bank spread)
    static constexpr int MERGE = CW * HP * LDM * 4;
    static constexpr int ML = CW * HP * 2 * 4;
    static constexpr int MISC = 512;                        // barriers, flags
    static constexpr int OFF_K = 0;
    static constexpr int OFF_V = CW * NS * TILE;
    static constexpr int OFF_M = 2 * CW * NS * TILE;
    static constexpr int OFF_ML = OFF_M + MERGE;
    static constexpr int OFF_MISC = OFF_ML + ML;
    static constexpr int SMEM = OFF_MISC + MISC + 1024;
    static_assert(kCtasPerSm * (SMEM + 1024) <= 228 * 1024, "the CTAs of an SM must fit its shared memory");
};

// Barriers of the chunks' copies, and the work list's block.
struct Misc {
    uint64_t full_k[kMaxWarps * 2], full_v[kMaxWarps * 2];   // [warp][slot]
    Schedule sched;
};
static_assert(sizeof(Misc) <= 512, "barrier block must fit its reserved bytes");

template <int D, int NT, bool F16>
__global__ void __launch_bounds__(PgCfg<D, NT>::THREADS, kCtasPerSm)
decode_paged_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                    const PgParams p) {
    using C = PgCfg<D, NT>;
    using H = H16<F16>;
    using T = typename H::T;
    constexpr int CW = C::CW, NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (ptx::smem_addr(smem_raw) & 1023)) & 1023);
    Misc *bars = reinterpret_cast<Misc *>(smem + C::OFF_MISC);
    Schedule *ms = &bars->sched;
    volatile int *abort = &ms->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < CW * NS; ++s) {
            ptx::mbar_init(&bars->full_k[s], 1);
            ptx::mbar_init(&bars->full_v[s], 1);
        }
        ptx::fence_barrier_init();
        ms->abort = 0;
        ptx::prefetch_tmap(&tk);
        ptx::prefetch_tmap(&tv);
    }
    // programmatic dependent launch: nothing global is read or written before
    // the previous kernel (an append, say) has completed
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    // ---- this CTA's range and where it starts
    Range range;
    if (!find_range<D, CW, T>(p, ms, range)) return;
    const bool alone = range.alone;
    const int team = range.team, rank = range.rank, list = range.list, at = range.at;

    Walk w(p, list, ms->start_b[at], ms->start_len[at], ms->start_kvh[at], ms->start_v[at], range.start, range.count);
    int f = 0;                                         // chunk number within the range

    // ---- loads: a walk of its own that runs NS chunks (and a group of page
    //      lookups) ahead of the computation
    const int BR = 1 << p.br_log;                      // rows of a box (1, 2 or 4 boxes per chunk)
    const int box_bytes = BR * D * 2;
    const uint64_t pol = ptx::l2_policy_evict_first();
    uint64_t *full_k = bars->full_k + warp * NS, *full_v = bars->full_v + warp * NS;
    uint8_t *ring_k = smem + C::OFF_K + warp * NS * C::TILE, *ring_v = smem + C::OFF_V + warp * NS * C::TILE;
    Feed feed(p, w, range);
    // this warp's chunks: K asked for, K and V asked for, computed
    int k_out = 0, issued = 0, taken = 0;
    unsigned bad_bits = 0;                             // bit i % 32: chunk i has a bad page
    auto issue_k = [&]() -> bool {                     // K of this warp's next chunk, if there is one
        if (!feed.next()) return false;
        const int s = issued % NS;
        bad_bits = (bad_bits & ~(1u << (issued & 31))) | (unsigned(feed.bad != 0) << (issued & 31));
        if (lane == 0) ptx::mbar_arrive_expect_tx(&full_k[s], __popc(feed.mine) * box_bytes);
        __syncwarp();
        const int box = feed.box(feed.mine);
        if (box >= 0)
            ptx::tma_load_5d(ring_k + s * C::TILE + box * box_bytes, &tk, 0, feed.cur.row, 0, feed.cur.kvh,
                             feed.cur.page, &full_k[s], pol);
        ++k_out;
        return true;
    };
    auto issue_v = [&]() {                             // V of the same chunk
        const int s = issued % NS;
        if (lane == 0) ptx::mbar_arrive_expect_tx(&full_v[s], __popc(feed.mine) * box_bytes);
        __syncwarp();
        const int box = feed.box(feed.mine);
        if (box >= 0)
            ptx::tma_load_5d(ring_v + s * C::TILE + box * box_bytes, &tv, 0, feed.cur.row, 0, feed.cur.kvh,
                             feed.cur.page, &full_v[s], pol);
        ++issued;
    };
    float *mg = reinterpret_cast<float *>(smem + C::OFF_M);
    float *mml = reinterpret_cast<float *>(smem + C::OFF_ML);
    const int quad = lane >> 2, pair = lane & 3;
    // ldmatrix lane addresses (relative to a slot): rows and the swizzled
    // 16-byte column; a k-step moves bits 5-6 of the column, a panel adds psz
    const int psz = BR * 128;
    uint32_t k_row[2], v_row[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int rk = t * 16 + (lane & 15);
        const int rv = t * 16 + (lane & 7) + ((lane >> 4) & 1) * 8;
        k_row[t] = (rk >> p.br_log) * (C::PANELS * psz) + (rk & (BR - 1)) * 128 +
                   ((((lane >> 4) & 1) ^ (lane & 7)) << 4);
        v_row[t] = (rv >> p.br_log) * (C::PANELS * psz) + (rv & (BR - 1)) * 128 +
                   ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
    }
    const uint32_t k_base = ptx::smem_addr(ring_k), v_base = ptx::smem_addr(ring_v);

    // after a timeout a warp computes nothing more but still walks the
    // segments: the other warps meet it at their barriers, and every unit's
    // ticket is counted up and reset as usual
    int dead = 0, warm = 0;
    // q of the unit's heads as MMA B operands (heads are columns); the next
    // segment's are requested before this one's results are merged
    uint32_t qf[NT][D / 16][2];
    auto load_q = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = nt * 8 + quad;
            const T *qp = static_cast<const T *>(p.q) + w.b * p.q_sb +
                          (long long)(w.kvh * p.G + h) * p.q_sh + pair * 2;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qf[nt][kk][0] = h < p.G ? *reinterpret_cast<const uint32_t *>(qp + kk * 16) : 0u;
                qf[nt][kk][1] = h < p.G ? *reinterpret_cast<const uint32_t *>(qp + kk * 16 + 8) : 0u;
            }
        }
    };
    load_q();
    for (bool more = true; more;) {
        float m[NT][2], l[NT][2], acc[NT][D / 16][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
        }
        int bad = dead;

        const int f_end = f + w.cnt;
        // this warp's chunks: the range's chunk number modulo the team.  The
        // first NS rounds of all only ask for chunks.
        int fc = f + ((rank - f) & (team - 1));
#pragma unroll 1
        while ((warm < NS || fc < f_end) && !dead) {
            const int s = taken % NS;
            const uint32_t parity = (taken / NS) & 1;
            const bool go = warm == NS;
            float sc[2][NT][4];
            if (go) {
                if (!__all_sync(0xffffffffu, ptx::mbar_wait_or_abort(&full_k[s], parity, p.err, abort))) {
                    bad = dead = 1;
                    break;
                }
                bad |= (bad_bits >> (taken & 31)) & 1u;
                // ---- S^T = K q^T, a panel's fragments first, then its MMAs
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        sc[t][nt][0] = sc[t][nt][1] = sc[t][nt][2] = sc[t][nt][3] = 0.f;
#pragma unroll
                for (int pn = 0; pn < C::PANELS; ++pn) {
                    uint32_t a[4][2][4];
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            ptx::ldsm4(a[kk][t], k_base + s * C::TILE + pn * psz + (k_row[t] ^ (kk << 5)));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                ptx::mma16816<F16>(sc[t][nt], a[kk][t], qf[nt][pn * 4 + kk][0],
                                              qf[nt][pn * 4 + kk][1]);
                }
            }
            // every lane's fragments have been read: the slot takes the next K
            __syncwarp();
            const bool more_loads = issue_k();
            if (!go) {
                if (more_loads) issue_v();
                ++warm;
                continue;
            }
            const int base = chunk_of(w.plan, w.v0 + (fc - f)) * kChunk;

            // ---- visibility of the chunk's 32 positions
            unsigned vis;
            {
                const int pos = base + lane;
                vis = __ballot_sync(0xffffffffu, pos < w.plan.len && (pos >= w.plan.lo || pos < w.plan.s_end));
            }
            // ---- online softmax (base 2) per head column
            uint32_t ph[2][NT][2], pl[2][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float x[2][4];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[t][i] = (vis >> (t * 16 + quad + (i >> 1) * 8)) & 1u ? sc[t][nt][i] * p.c_log2
                                                                               : -INFINITY;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float mx = fmaxf(fmaxf(x[0][j], x[0][j + 2]), fmaxf(x[1][j], x[1][j + 2]));
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1)
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    const float mn = fmaxf(m[nt][j], mx);
                    const float alpha = mn == -INFINITY ? 1.f : ptx::ex2(m[nt][j] - mn);
                    m[nt][j] = mn;
                    float sum = 0.f;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int i = j; i < 4; i += 2) {
                            const bool v = (vis >> (t * 16 + quad + (i >> 1) * 8)) & 1u;
                            // no finite score so far: -inf weighs nothing, NaN stays NaN
                            x[t][i] = !v || (mn == -INFINITY && x[t][i] == -INFINITY)
                                          ? 0.f : ptx::ex2(x[t][i] - mn);
                            sum += x[t][i];
                        }
                    l[nt][j] = l[nt][j] * alpha + sum;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        acc[nt][i][j] *= alpha;
                        acc[nt][i][j + 2] *= alpha;
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float a = x[t][2 * r], b = x[t][2 * r + 1];
                        const uint32_t hi = H::pack(a, b);
                        ph[t][nt][r] = ptx::transpose8x8(hi);
                        pl[t][nt][r] = ptx::transpose8x8(H::pack(a - H::lo(hi), b - H::hi(hi)));
                    }
            }

            if (!__all_sync(0xffffffffu, ptx::mbar_wait_or_abort(&full_v[s], parity, p.err, abort))) {
                bad = dead = 1;
                break;
            }
            // ---- O^T += V^T P^T.  Rows that are not visible may hold anything
            //      (NaN times a zero weight is NaN): their values are cleared.
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const unsigned v = vis >> (t * 16 + 2 * pair);
                const uint32_t keep0 = (v & 1u ? 0x0000ffffu : 0u) | (v & 2u ? 0xffff0000u : 0u);
                const uint32_t keep1 = (v & 0x100u ? 0x0000ffffu : 0u) | (v & 0x200u ? 0xffff0000u : 0u);
#pragma unroll
                for (int pn = 0; pn < C::PANELS; ++pn) {
                    uint32_t a[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        ptx::ldsm4t(a[i], v_base + s * C::TILE + pn * psz + (v_row[t] ^ (i << 5)));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a[i][0] &= keep0;
                        a[i][1] &= keep0;
                        a[i][2] &= keep1;
                        a[i][3] &= keep1;
                    }
                    // the two terms of P in separate rounds: no MMA waits for the one before
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            ptx::mma16816<F16>(acc[nt][pn * 4 + i], a[i], ph[t][nt][0], ph[t][nt][1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            ptx::mma16816<F16>(acc[nt][pn * 4 + i], a[i], pl[t][nt][0], pl[t][nt][1]);
                    }
                }
            }
            __syncwarp();
            if (more_loads) issue_v();
            ++taken;
            fc += team;
        }
        f = f_end;

        // this segment (the walk goes on to the next one)
        const int seg_b = w.b, seg_kvh = w.kvh, seg_v0 = w.v0, seg_cnt = w.cnt, seg_n = w.plan.n;
        const int u0 = w.flat - w.v0;                  // flat index of the unit's first chunk
        more = w.next();
        if (more) load_q();
        T *const o_unit = static_cast<T *>(p.o) + seg_b * p.o_sb + (long long)seg_kvh * p.G * p.o_sh;

        // ---- the warps' (max, sum, O) -> one per head
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], off);
                const int h = nt * 8 + pair * 2 + j;
                if (quad == 0) {
                    mml[(warp * C::HP + h) * 2] = m[nt][j];
                    mml[(warp * C::HP + h) * 2 + 1] = l[nt][j];
                }
                float *row = mg + (warp * C::HP + h) * C::LDM;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    row[i * 16 + quad] = acc[nt][i][j];
                    row[i * 16 + 8 + quad] = acc[nt][i][j + 2];
                }
            }
        if (alone) {
            store_alone<D, C::HP, C::LDM, 1, F16>(p, mg, mml, bad, o_unit);
            continue;
        }
        join_segment<D, CW, C::HP, C::LDM, 1, F16>(p, ms, mg, mml, range, seg_b * p.Hkv + seg_kvh, seg_v0, seg_cnt,
                                                seg_n, u0, bad, o_unit);
    }
    // after a timeout: let the copies this warp asked for land (bounded) before
    // the CTA's shared memory is released
    if (dead && lane == 0) {
        for (int i = taken; i < k_out; ++i) ptx::mbar_wait(&full_k[i % NS], (i / NS) & 1, nullptr);
        for (int i = taken; i < issued; ++i) ptx::mbar_wait(&full_v[i % NS], (i / NS) & 1, nullptr);
    }
}

// 5D map {64 channels, S rows, D / 64 panels, Hkv, pages} over a cache with
// element strides (page, head, token); box: BR rows x D channels of one head,
// stored as panels of BR 128-byte rows (128-byte swizzle).
bool page_tmap(CUtensorMap *m, const void *base, int P, int Hkv, int S, int D, const long long st[3],
               int BR, bool f16) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t gdim[5] = {64, cuuint64_t(S), cuuint64_t(D / 64), cuuint64_t(Hkv), cuuint64_t(P)};
    const cuuint64_t gstride[4] = {cuuint64_t(st[2]) * 2, 128, cuuint64_t(st[1]) * 2, cuuint64_t(st[0]) * 2};
    const cuuint32_t box[5] = {64, cuuint32_t(BR), cuuint32_t(D / 64), 1, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
              const_cast<void *>(base), gdim, gstride, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NT, bool F16>
attn_status_t launch_paged(const Ctx &c, const CUtensorMap &tk, const CUtensorMap &tv,
                           const PgParams &p) {
    using C = PgCfg<D, NT>;
    static int done_mask = 0;
    auto kern = decode_paged_kernel<D, NT, F16>;
    if (!ensure_smem_attr(reinterpret_cast<const void *>(kern), C::SMEM, c.device, &done_mask))
        return ATTN_ERR_RESOURCE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(imin(kCtasPerSm * c.sm_count, kMaxCtas));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, tk, tv, p) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    return launch_status(kFamDecodePaged);
}

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

// The partials come first, at their largest size, so that the tickets lie at one
// place whatever the call's sizes: one workspace serves calls of several sizes.
constexpr size_t kPartBytes = size_t(2) * kMaxCtas * 16 * 128 * sizeof(float);
constexpr size_t kMlBytes = size_t(2) * kMaxCtas * 16 * 2 * sizeof(float);
static_assert(kPartBytes % 256 == 0 && kMlBytes % 256 == 0, "aligned workspace parts");

size_t decode_paged_workspace_bytes(int B, int Hkv) {
    return kPartBytes + kMlBytes + align256(size_t(B) * Hkv * sizeof(unsigned));
}

attn_status_t decode_paged(const Ctx &c, attn_dtype_t dt, const PagedDecode &a) {
    const bool f16 = dt == ATTN_F16;
    PgParams p = page_params(a.S);
    const int BR = 1 << p.br_log;
    CUtensorMap tk, tv;
    if (!page_tmap(&tk, a.k, a.P, a.Hkv, a.S, a.D, a.k_st, BR, f16) ||
        !page_tmap(&tv, a.v, a.P, a.Hkv, a.S, a.D, a.v_st, BR, f16))
        return ATTN_ERR_UNSUPPORTED;
    p.q = a.q;
    p.o = a.o;
    p.q_sb = a.q_st[0]; p.q_sh = a.q_st[1];
    p.o_sb = a.o_st[0]; p.o_sh = a.o_st[1];
    p.table = a.table;
    p.table_stride = a.table_stride;
    p.seq_len = a.seq_len;
    p.B = a.B; p.Hkv = a.Hkv; p.G = a.G;
    p.max_pages = a.max_pages; p.num_pages = a.P;
    p.window = a.window; p.sinks = a.sinks;
    p.c_log2 = a.scale * kLog2e;
    uint8_t *w = static_cast<uint8_t *>(a.ws);
    p.part_o = reinterpret_cast<float *>(w);
    p.part_ml = reinterpret_cast<float *>(w + kPartBytes);
    p.tickets = reinterpret_cast<unsigned *>(w + kPartBytes + kMlBytes);
    p.err = c.err;
    if (a.D == 128) {
        if (a.G <= 8) return f16 ? launch_paged<128, 1, true>(c, tk, tv, p) : launch_paged<128, 1, false>(c, tk, tv, p);
        return f16 ? launch_paged<128, 2, true>(c, tk, tv, p) : launch_paged<128, 2, false>(c, tk, tv, p);
    }
    if (a.G <= 8) return f16 ? launch_paged<64, 1, true>(c, tk, tv, p) : launch_paged<64, 1, false>(c, tk, tv, p);
    return f16 ? launch_paged<64, 2, true>(c, tk, tv, p) : launch_paged<64, 2, false>(c, tk, tv, p);
}

}  // namespace attn
