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
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kChunk = 32;        // positions per chunk
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

// The chunk counts of a call fit 31 bits (checked by the entry), so the work
// list is kept in ints; the steps of the loop are kept to one copy each and its
// divisions by the page size are multiplications (the kernel is short: a call
// of a few microseconds fetches most of its code once).
struct PgParams {
    const void *q;
    void *o;
    long long q_sb, q_sh, o_sb, o_sh;      // element strides (batch, head)
    const int32_t *table;
    long long table_stride;
    const int32_t *seq_len;
    int B, Hkv, G;
    int S, nb, br_log;                     // page size, TMA boxes per chunk and log2 of their rows
    unsigned s_mul, s_sh;                  // division by S (div_s)
    int max_pages, num_pages;
    int window, sinks;
    float c_log2;
    float *part_o;                         // [2 CTAs][HP][D]
    float *part_ml;                        // [2 CTAs][HP][2]
    unsigned *tickets;                     // [B * Hkv]
    unsigned *err;
};

constexpr int kMaxWarps = 4;
constexpr int kFitted = 20;       // chunks by which a range may grow to be fitted to its units
// The longest unit (chunks) that counts as short: beside long ones (40 sequences of
// 1 to 900 tokens 11.7 us, 13.7 with 8, 11.8 with 4) and in a call without longer
// ones (100 x 250 tokens 20.2 us, 23.1 with 5).
constexpr int kWarpUnit = 5, kAllShort = 8;

struct Misc {
    uint64_t full_k[kMaxWarps * 2], full_v[kMaxWarps * 2];   // [warp][slot]
    int warp_long[kMaxWarps], warp_short[kMaxWarps];
    int warp_parts[kMaxWarps], warp_idle[kMaxWarps];
    int warp_max[kMaxWarps], warp_units[kMaxWarps], warp_units_l[kMaxWarps];
    // where the CTA's range, or each warp's (and the one behind), starts
    int start_flat[kMaxWarps + 1];
    int start_b[kMaxWarps + 1], start_len[kMaxWarps + 1], start_kvh[kMaxWarps + 1], start_v[kMaxWarps + 1];
    int start_count;
    int abort;
    unsigned last;
    int warp_bad[kMaxWarps];
};
static_assert(sizeof(Misc) <= 512, "barrier block must fit its reserved bytes");

// The chunks of one sequence that hold a visible position: chunks [0, n1) for
// the sinks and [c2, ...) for the window (one run from 0 where they touch).
struct Plan {
    int len, lo, s_end, n1, c2, n;
};

__device__ __forceinline__ Plan make_plan(const PgParams &p, int len) {
    Plan r;
    r.len = len;
    r.lo = r.s_end = r.n1 = r.c2 = r.n = 0;
    if (len < 1 || (long long)len > (long long)p.max_pages * p.S) return r;
    if (p.window > 0 && len > p.window) r.lo = len - p.window;
    r.s_end = imin(p.sinks, r.lo);
    const int end = (len - 1) / kChunk + 1;
    r.n1 = r.s_end > 0 ? (r.s_end - 1) / kChunk + 1 : 0;
    r.c2 = r.lo / kChunk;
    if (r.n1 >= r.c2) r.n1 = r.c2 = 0;
    r.n = r.n1 + end - r.c2;
    return r;
}

// n / S for 0 <= n < 2^31 by a multiplication (S >= 2)
__device__ __forceinline__ int div_s(const PgParams &p, int n) {
    const unsigned t = __umulhi(p.s_mul, unsigned(n));
    return int((t + ((unsigned(n) - t) >> 1)) >> p.s_sh);
}

// The plan of a sequence if it belongs to a list of the call: the units of up to
// `list` chunks, or (negative) those of more than -list.
__device__ __forceinline__ Plan plan_in(const PgParams &p, int len, int list) {
    Plan r = make_plan(p, len);
    if ((r.n <= abs(list)) != (list > 0)) r.n = 0;
    return r;
}

__device__ __forceinline__ int chunk_of(const Plan &r, int v) {
    return v < r.n1 ? v : v - r.n1 + r.c2;
}

// One CTA's range of the flat chunk list, a segment (part of one unit) at a time.
struct Walk {
    const PgParams &p;
    int list;
    Plan plan;
    int b, kvh, v0, cnt;
    int left;                              // chunks of the range from this segment on
    int flat;                              // flat index of the segment's first chunk

    int ahead;                             // seq_len[b + 1], loaded before it is needed

    __device__ Walk(const PgParams &pp, int l, int b0, int len0, int kvh0, int v, int f0, int count)
        : p(pp), list(l), b(b0), kvh(kvh0), v0(v), left(count), flat(f0) {
        plan = make_plan(p, len0);
        ahead = b + 1 < p.B ? p.seq_len[b + 1] : 0;
        if (kvh == p.Hkv) next_sequence();
        cnt = imin(left, plan.n - v0);
    }
    __device__ void next_sequence() {       // the range ends inside the list: b stays below B
        kvh = 0;
        do {
            plan = plan_in(p, ahead, list);
            ++b;
            ahead = b + 1 < p.B ? p.seq_len[b + 1] : 0;
        } while (plan.n == 0);
    }
    __device__ bool next() {
        left -= cnt;
        flat += cnt;
        if (left <= 0) return false;
        v0 = 0;
        if (++kvh == p.Hkv) next_sequence();
        cnt = imin(left, plan.n);
        return true;
    }
};

// ------------------------------------------------------- warp-level MMA

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                     "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
                     "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Takes the next ticket: releases what this CTA wrote, acquires what the
// holders of the earlier tickets wrote.
__device__ __forceinline__ unsigned ticket_add(unsigned *t) {
    unsigned old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(t) : "memory");
    return old;
}

// The pages of one warp's next chunks, box by box: lane i holds box i % nb of
// chunk i / nb of the group.
struct Group {
    int page, row;                         // this lane's box
    unsigned needs, bads;                  // boxes to copy; boxes whose entry is no page
    int kvh, cnt;                          // KV head; chunks in the group (0: the range is done)
};

// Rare steps are functions of their own, out of the way of the code that every
// launch fetches.

// The sequences with nothing to attend to among this CTA's share (b0 and every
// step-th from it on): zeros (length 0) by all of its threads, or a report.  4
// sequences of 128 to 700 tokens, 32 heads, D 128, beside 4 idle slots: 8.8 us,
// 8.7 without the slots (45.8 us with one thread writing a slot's zeros).
template <int D, typename T>
__device__ __noinline__ void idle_sequences(const PgParams &p, int b0, int step) {
#pragma unroll 1
    for (int b = b0; b < p.B; b += step) {
        const int len = p.seq_len[b];
        if (len != 0 && make_plan(p, len).n == 0 && threadIdx.x == 0) raise_device_error(p.err, kDevCheck);
        if (len != 0) continue;
        for (int i = threadIdx.x; i < p.Hkv * p.G * (D / 8); i += blockDim.x)
            *reinterpret_cast<uint4 *>(static_cast<T *>(p.o) + b * p.o_sb + (i / (D / 8)) * p.o_sh +
                                       (i % (D / 8)) * 8) = make_uint4(0u, 0u, 0u, 0u);
    }
}

// Where this CTA's range starts (mark i: f0, or the first unit that starts at or
// behind f0 + i per), looked for by the thread of one sequence: n chunks per
// unit of this list, `before` chunks per KV head ahead of it.
__device__ __forceinline__ void mark_starts(const PgParams &p, Misc *ms, int marks, int f0, int per, int b,
                                            int len, int n, int before) {
    const int lo = before * p.Hkv, hi = lo + n * p.Hkv;
#pragma unroll 1
    for (int i = 0; i < marks; ++i) {
        const unsigned x = unsigned(f0) + unsigned(i * per);
        if (x < unsigned(lo) || x >= unsigned(hi)) continue;
        int kvh = int((x - lo) / unsigned(n)), v = int(x - lo) - kvh * n;
        if (marks > 1 && v > 0) {
            ++kvh;                                     // may be Hkv: the next sequence's first
            v = 0;
        }
        ms->start_b[i] = b;
        ms->start_len[i] = len;
        ms->start_kvh[i] = kvh;
        ms->start_v[i] = v;
        ms->start_flat[i] = lo + kvh * n + v;
    }
}

// The same for a batch of more sequences than threads, read again tile by tile.
template <int CW>
__device__ __noinline__ void mark_long_batch(const PgParams &p, Misc *ms, int marks, int f0, int per,
                                             int list) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int carry = 0;                                     // chunks of the sequences before this tile
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += CW * 32) {
        __syncthreads();
        const int b = b0 + threadIdx.x;
        const int len = b < p.B ? p.seq_len[b] : 0;
        const int n = plan_in(p, len, list).n;
        int inc = n;
#pragma unroll 1
        for (int off = 1; off < 32; off <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += up;
        }
        if (lane == 31) ms->warp_long[warp] = inc;
        __syncthreads();
        int before = carry + inc - n;
#pragma unroll
        for (int w = 0; w < CW; ++w) {
            if (w < warp) before += ms->warp_long[w];
            carry += ms->warp_long[w];
        }
        if (n > 0) mark_starts(p, ms, marks, f0, per, b, len, n, before);
    }
}

template <int D, int NT, bool F16>
__global__ void __launch_bounds__(PgCfg<D, NT>::THREADS, kCtasPerSm)
decode_paged_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                    const PgParams p) {
    using C = PgCfg<D, NT>;
    using H = H16<F16>;
    using T = typename H::T;
    constexpr int CW = C::CW, NS = C::NS, kNT = C::THREADS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (ptx::smem_addr(smem_raw) & 1023)) & 1023);
    Misc *ms = reinterpret_cast<Misc *>(smem + C::OFF_MISC);
    volatile int *abort = &ms->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x, ctas = gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < CW * NS; ++s) {
            ptx::mbar_init(&ms->full_k[s], 1);
            ptx::mbar_init(&ms->full_v[s], 1);
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

    // ---- the lists' lengths, this CTA's range and where it starts.
    //      Sequences with nothing to attend to are dealt out over the CTAs, the
    //      last first (a short call leaves those without a range): length 0
    //      writes zeros, a length outside the table is reported and its output
    //      left as it was.
    const bool one_tile = p.B <= kNT;                  // a thread per sequence: read once
    int inc_l = 0, inc_s = 0, n_mine = 0, len_mine = 0, n_max = 0, units = 0, units_l = 0;
    bool idle = false;
#pragma unroll 1
    for (int b = threadIdx.x; b < p.B; b += kNT) {
        len_mine = p.seq_len[b];
        n_mine = make_plan(p, len_mine).n;
        n_max = imax(n_max, n_mine);
        if (n_mine <= kWarpUnit) {
            inc_s += n_mine;
            units += n_mine > 0;
        } else {
            inc_l += n_mine;
            ++units_l;
        }
        idle = idle || (n_mine == 0 && b % ctas == ctas - 1 - cta);
    }
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
        const int up_l = __shfl_up_sync(0xffffffffu, inc_l, off), up_s = __shfl_up_sync(0xffffffffu, inc_s, off);
        if (lane >= off) {
            inc_l += up_l;
            inc_s += up_s;
        }
        n_max = imax(n_max, __shfl_xor_sync(0xffffffffu, n_max, off));
        units += __shfl_xor_sync(0xffffffffu, units, off);
        units_l += __shfl_xor_sync(0xffffffffu, units_l, off);
    }
    idle = __any_sync(0xffffffffu, idle);
    if (lane == 31) {
        ms->warp_idle[warp] = idle;
        ms->warp_long[warp] = inc_l;
        ms->warp_short[warp] = inc_s;
        ms->warp_max[warp] = n_max;
        ms->warp_units[warp] = units;
        ms->warp_units_l[warp] = units_l;
    }
    __syncthreads();
    int total_l = 0, total_s = 0, before_l = inc_l, before_s = inc_s;
    units = units_l = 0;
#pragma unroll
    for (int w = 0; w < CW; ++w) {
        if (w < warp) {
            before_l += ms->warp_long[w];
            before_s += ms->warp_short[w];
        }
        total_l += ms->warp_long[w];
        total_s += ms->warp_short[w];
        n_max = imax(n_max, ms->warp_max[w]);
        units += ms->warp_units[w];
        units_l += ms->warp_units_l[w];
        idle = idle || ms->warp_idle[w];
    }
    if (idle) idle_sequences<D, T>(p, ctas - 1 - cta, ctas);
    if (n_max <= kAllShort) {                          // no long ones: one list
        total_s += total_l;
        before_s += before_l;
        units += units_l;
        total_l = units_l = 0;
    }
    total_l *= p.Hkv;
    total_s *= p.Hkv;
    units *= p.Hkv;                                    // of the short list
    units_l *= p.Hkv;
    // this CTA's list, its number c among the nc CTAs of that list
    bool in_short = total_l == 0, alone = in_short && units > ctas;
    int c = cta, nc = ctas;
    if (total_l > 0 && total_s > 0) {
        const float cost = float(total_s) + float(units);   // a unit costs about a chunk more
        const int ns = imax(1, imin(ctas - 1, int(ctas * (cost / (cost + float(total_l)))) + 1));
        in_short = alone = cta >= ctas - ns;
        nc = in_short ? ns : ctas - ns;
        c = in_short ? cta - (ctas - ns) : cta;
    }
    const int total = in_short ? total_s : total_l;
    const int limit = n_max <= kAllShort ? kAllShort : kWarpUnit, list = in_short ? limit : -limit;
    if ((n_mine <= limit) != in_short) n_mine = 0;
    int before = (in_short ? before_s : before_l) - n_mine;   // chunks of the sequences ahead (one tile)
    // team: the warps that share a range (all of the CTA's, or each its own)
    const int team = alone ? 1 : CW, rank = alone ? 0 : warp;
    const int teams = alone ? nc * CW : nc;
    int per = int((unsigned(total) + teams - 1) / unsigned(teams));
    // at least one chunk per warp, unless every unit is shorter than that: then
    // the units are spread over more CTAs
    if (!alone) per = imax(per, imin(CW, n_max));
    // Where a quarter more chunks per range allow it, or 20, a range holds part of
    // one unit only, and its CTA merges and joins once instead of twice: with q =
    // CTAs / units, parts of the longest unit's q-th give no more parts than CTAs.
    // The list is read as if each unit filled whole parts.  (Equal units that fill
    // whole ranges need no such thing.)  That saves 2 to 3 us and costs what the
    // longest range gains.  Chunks longer: us without and with (32 heads on 8, D 128)
    //    1   8 x 1024 tokens 13.3, 11.6
    //    4   30 x 600 18.3, 15.7
    //    5   8 x 4096 27.2, 25.4
    //   13   40 of 1 to 900 19.6, 17.4
    //   16   30 of 200 to 1000 19.2, 17.4
    //   17   120 of 170 to 1000, 16 heads on 2: 20.2, 17.6
    //   24   one of 2000 beside 15 of 500 14.4, 16.0
    //   30   36 of 170 to 2000 31.3, 30.4
    //   31   20 of 300 to 1500 18.7, 20.1
    //   51   one of 2000 beside 36 of 300 15.8, 24.2
    //   57   one of 2048 beside 24 of 200 13.3, 22.8
    int parts = 0, parts_before = 0, parts_total = 0;
    const int n_units = in_short ? units : units_l;
    const int fit = n_units <= nc ? imax(per, cdiv(n_max, nc / imax(n_units, 1))) : 0;
    if (!alone && one_tile && fit > 0 && fit <= per + imax(kFitted, per / 4) && n_max > per && total < (1 << 30) &&
        !(n_max % per == 0 && (long long)n_units * n_max == total)) {
        per = fit;
        parts = int(unsigned(n_mine + per - 1) / unsigned(per));
        int inc = parts;
#pragma unroll 1
        for (int off = 1; off < 32; off <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += up;
        }
        if (lane == 31) ms->warp_parts[warp] = inc;
        __syncthreads();
        parts_before = inc - parts;
#pragma unroll
        for (int w = 0; w < CW; ++w) {
            if (w < warp) parts_before += ms->warp_parts[w];
            parts_total += ms->warp_parts[w];
        }
        parts_total *= p.Hkv;
    }
    const bool aligned = parts_total > 0;
    const long long f0l = (long long)per * (alone ? c * CW : c);
    if (aligned ? c >= parts_total : f0l >= total) return;
    const int f0 = int(f0l);
    // each warp's range is a run of whole units, between two marks
    const int marks = alone ? CW + 1 : 1;
    if (aligned) {
        const int x = c - parts_before * p.Hkv;        // among the parts of this thread's sequence
        if (parts > 0 && x >= 0 && x < parts * p.Hkv) {
            const int kvh = int(unsigned(x) / unsigned(parts)), v = (x - kvh * parts) * per;
            ms->start_b[0] = threadIdx.x;
            ms->start_len[0] = len_mine;
            ms->start_kvh[0] = kvh;
            ms->start_v[0] = v;
            ms->start_flat[0] = f0;
            ms->start_count = imin(per, n_mine - v);
        }
    } else {
        if (threadIdx.x < marks && f0l + (long long)threadIdx.x * per >= total) ms->start_flat[threadIdx.x] = total;
        if (!one_tile)
            mark_long_batch<CW>(p, ms, marks, f0, per, list);
        else if (n_mine > 0)
            mark_starts(p, ms, marks, f0, per, threadIdx.x, len_mine, n_mine, before);
    }
    __syncthreads();
    const int at = alone ? warp : 0;
    const int start = ms->start_flat[at];
    const int count = alone ? ms->start_flat[warp + 1] - start : aligned ? ms->start_count : imin(per, total - f0);
    if (count <= 0) return;                            // alone: no unit starts in this warp's share

    Walk w(p, list, ms->start_b[at], ms->start_len[at], ms->start_kvh[at], ms->start_v[at], start, count);
    int f = 0;                                         // chunk number within the range

    // ---- loads: a walk of its own that runs NS chunks (and a group of page
    //      lookups) ahead of the computation
    const int nb = p.nb, BR = 1 << p.br_log;           // boxes per chunk (1, 2 or 4), their rows
    const unsigned bits = (1u << nb) - 1u;
    const int box_bytes = BR * D * 2;
    const int group = BR;                              // chunks whose boxes the lanes look up: 32 / nb
    const int sub = lane >> (5 - p.br_log), box = lane & (nb - 1);
    const uint64_t pol = ptx::l2_policy_evict_first();
    uint64_t *full_k = ms->full_k + warp * NS, *full_v = ms->full_v + warp * NS;
    uint8_t *ring_k = smem + C::OFF_K + warp * NS * C::TILE, *ring_v = smem + C::OFF_V + warp * NS * C::TILE;
    Walk lw = w;
    int l_next = rank;                                 // this warp's next chunk within lw's segment
    int l_f = 0;                                       // chunk number of lw's segment start
    bool l_more = true;
    auto lookup = [&]() -> Group {
        Group g;
        g.page = g.row = 0;
        g.needs = g.bads = 0;
        g.kvh = g.cnt = 0;
        while (l_more && l_next >= lw.cnt) {           // no (more) chunk of this warp in the segment
            l_f += lw.cnt;
            l_more = lw.next();
            l_next = (rank - l_f) & (team - 1);
        }
        if (!l_more) return g;
        g.kvh = lw.kvh;
        g.cnt = imin(group, (lw.cnt - l_next + team - 1) >> (alone ? 0 : 2));
        bool need = false;
        if (sub < g.cnt) {
            const int v = lw.v0 + l_next + sub * team;
            const int pos = chunk_of(lw.plan, v) * kChunk + box * BR;
            // a box without a visible position is not read: its page may not
            // exist (past the end) or may be free again
            need = pos < lw.plan.len && (pos + BR > lw.plan.lo || pos < lw.plan.s_end);
            if (need) {
                const int e = div_s(p, pos);
                g.page = p.table[(long long)lw.b * p.table_stride + e];
                g.row = pos - e * p.S;
            }
        }
        g.needs = __ballot_sync(0xffffffffu, need);
        l_next += g.cnt * team;
        return g;
    };
    // checks the entries (when they have arrived) before the group's first copy
    auto check = [&](Group &g) {
        const bool bad = ((g.needs >> lane) & 1u) && (g.page < 0 || g.page >= p.num_pages);
        if (bad) {
            raise_device_error(p.err, kDevCheck);
            g.page = p.num_pages;                      // outside the map: the copy fills zeros
        }
        g.bads = __ballot_sync(0xffffffffu, bad);
    };
    Group cur{}, nxt{};
    int gi = 0;                                        // chunk within cur
    // this warp's chunks: K asked for, K and V asked for, computed
    int k_out = 0, issued = 0, taken = 0;
    unsigned bad_bits = 0;                             // bit i % 32: chunk i has a bad page
    int pg = 0, pr = 0, kvh_v = 0;                     // the chunk whose K went out last
    unsigned mine = 0;
    auto issue_k = [&]() -> bool {                     // K of this warp's next chunk, if there is one
#pragma unroll 1
        while (gi == cur.cnt && (nxt.cnt > 0 || l_more)) {
            cur = nxt;
            gi = 0;
            nxt = lookup();
            check(cur);
        }
        if (gi == cur.cnt) return false;
        const int s = issued % NS;
        mine = (cur.needs >> (gi * nb)) & bits;
        const unsigned b = (cur.bads >> (gi * nb)) & bits;
        bad_bits = (bad_bits & ~(1u << (issued & 31))) | (unsigned(b != 0) << (issued & 31));
        pg = __shfl_sync(0xffffffffu, cur.page, gi * nb + box);
        pr = __shfl_sync(0xffffffffu, cur.row, gi * nb + box);
        kvh_v = cur.kvh;
        if (lane == 0) ptx::mbar_arrive_expect_tx(&full_k[s], __popc(mine) * box_bytes);
        __syncwarp();
        if (lane < nb && ((mine >> lane) & 1u))
            ptx::tma_load_5d(ring_k + s * C::TILE + lane * box_bytes, &tk, 0, pr, 0, kvh_v, pg, &full_k[s], pol);
        ++k_out;
        return true;
    };
    auto issue_v = [&]() {                             // V of the same chunk
        const int s = issued % NS;
        if (lane == 0) ptx::mbar_arrive_expect_tx(&full_v[s], __popc(mine) * box_bytes);
        __syncwarp();
        if (lane < nb && ((mine >> lane) & 1u))
            ptx::tma_load_5d(ring_v + s * C::TILE + lane * box_bytes, &tv, 0, pr, 0, kvh_v, pg, &full_v[s], pol);
        ++issued;
        ++gi;
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
                            ldsm4(a[kk][t], k_base + s * C::TILE + pn * psz + (k_row[t] ^ (kk << 5)));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816<F16>(sc[t][nt], a[kk][t], qf[nt][pn * 4 + kk][0],
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
                        ph[t][nt][r] = transpose8x8(hi);
                        pl[t][nt][r] = transpose8x8(H::pack(a - H::lo(hi), b - H::hi(hi)));
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
                        ldsm4t(a[i], v_base + s * C::TILE + pn * psz + (v_row[t] ^ (i << 5)));
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
                            mma16816<F16>(acc[nt][pn * 4 + i], a[i], ph[t][nt][0], ph[t][nt][1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma16816<F16>(acc[nt][pn * 4 + i], a[i], pl[t][nt][0], pl[t][nt][1]);
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
            // a whole unit in one warp's registers: through its own merge rows
            // to 8-byte stores
            __syncwarp();
#pragma unroll 1
            for (int e = lane; e < p.G * (D / 4) && !bad; e += 32) {
                const int h = e / (D / 4), d = (e % (D / 4)) * 4;
                const float inv = 1.f / mml[(warp * C::HP + h) * 2 + 1];
                const float4 x = *reinterpret_cast<const float4 *>(mg + (warp * C::HP + h) * C::LDM + d);
                *reinterpret_cast<uint2 *>(o_unit + h * p.o_sh + d) =
                    make_uint2(H::pack(x.x * inv, x.y * inv), H::pack(x.z * inv, x.w * inv));
            }
            __syncwarp();
            continue;
        }
        if (lane == 0) ms->warp_bad[warp] = bad;
        ptx::named_barrier_sync(1, kNT);
#pragma unroll
        for (int i = 0; i < CW; ++i) bad |= ms->warp_bad[i];

        const bool whole = seg_v0 == 0 && seg_cnt == seg_n;
        // a range holds at most one segment that starts inside its unit (slot 0)
        // and one that starts at its unit's head and is cut (slot 1)
        const int slot = 2 * cta + (seg_v0 == 0 ? 1 : 0);
        float *po = p.part_o + (size_t)slot * C::HP * D;
        float *pml = p.part_ml + (size_t)slot * C::HP * 2;
#pragma unroll 1
        for (int e = threadIdx.x; e < p.G * (D / 4); e += kNT) {
            const int h = e / (D / 4), d = (e % (D / 4)) * 4;
            float M = -INFINITY;
#pragma unroll
            for (int i = 0; i < CW; ++i) M = fmaxf(M, mml[(i * C::HP + h) * 2]);
            float L = 0.f;
            float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < CW; ++i) {
                const float mi = mml[(i * C::HP + h) * 2], li = mml[(i * C::HP + h) * 2 + 1];
                // a warp that saw nothing, or only scores of -inf, adds nothing
                // (its sum is zero, or NaN if one of its scores was)
                const float wt = mi == -INFINITY ? 0.f : ptx::ex2(mi - M);
                L += mi == -INFINITY ? li : wt * li;
                const float4 x = *reinterpret_cast<const float4 *>(mg + (i * C::HP + h) * C::LDM + d);
                O.x += wt * x.x;
                O.y += wt * x.y;
                O.z += wt * x.z;
                O.w += wt * x.w;
            }
            if (whole) {
                if (!bad) {
                    const float inv = 1.f / L;
                    T *dst = o_unit + h * p.o_sh + d;
                    *reinterpret_cast<uint2 *>(dst) =
                        make_uint2(H::pack(O.x * inv, O.y * inv), H::pack(O.z * inv, O.w * inv));
                }
            } else {
                *reinterpret_cast<float4 *>(po + h * D + d) = O;
                if (d == 0)                            // a NaN maximum marks a segment with a bad page
                    *reinterpret_cast<float2 *>(pml + h * 2) = make_float2(bad ? NAN : M, L);
            }
        }
        if (!whole) {
            const int unit = seg_b * p.Hkv + seg_kvh;
            const int c0 = int(unsigned(u0) / unsigned(per)), c1 = int(unsigned(u0 + seg_n - 1) / unsigned(per));
            // the barrier puts the CTA's partial before thread 0's release; its
            // acquire and the second barrier put the other CTAs' before the reads
            ptx::named_barrier_sync(1, kNT);
            if (threadIdx.x == 0) ms->last = ticket_add(&p.tickets[unit]) == unsigned(c1 - c0);
            ptx::named_barrier_sync(1, kNT);
            if (ms->last) {
#pragma unroll 1
                for (int e = threadIdx.x; e < p.G * (D / 4); e += kNT) {
                    const int h = e / (D / 4), d = (e % (D / 4)) * 4;
                    float M = -INFINITY, L = 0.f;
                    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
                    bool skip = false;
                    constexpr int U = 8;                   // partials in flight
#pragma unroll 1
                    for (int c = c0; c <= c1; c += U) {
                        float2 ml[U];
                        float4 x[U];
#pragma unroll
                        for (int i = 0; i < U; ++i) {
                            ml[i] = make_float2(-INFINITY, 0.f);
                            x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (c + i <= c1) {
                                // the CTA that holds the unit's head left it in slot 1
                                const size_t sl = 2 * size_t(c + i) + (c + i == c0 ? 1 : 0);
                                ml[i] = __ldcg(reinterpret_cast<const float2 *>(p.part_ml + sl * C::HP * 2) + h);
                                x[i] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + sl * C::HP * D + h * D + d));
                            }
                        }
                        float mn = M;
#pragma unroll
                        for (int i = 0; i < U; ++i) {
                            skip = skip || ml[i].x != ml[i].x;
                            mn = fmaxf(mn, ml[i].x);
                        }
                        const float keep = M == -INFINITY ? 1.f : ptx::ex2(M - mn);
                        L *= keep;
                        O.x *= keep;
                        O.y *= keep;
                        O.z *= keep;
                        O.w *= keep;
                        M = mn;
#pragma unroll
                        for (int i = 0; i < U; ++i) {
                            const float wt = ml[i].x == -INFINITY ? 0.f : ptx::ex2(ml[i].x - mn);
                            L += ml[i].x == -INFINITY ? ml[i].y : wt * ml[i].y;
                            O.x += wt * x[i].x;
                            O.y += wt * x[i].y;
                            O.z += wt * x[i].z;
                            O.w += wt * x[i].w;
                        }
                    }
                    if (!skip) {
                        const float inv = 1.f / L;
                        *reinterpret_cast<uint2 *>(o_unit + h * p.o_sh + d) =
                            make_uint2(H::pack(O.x * inv, O.y * inv), H::pack(O.z * inv, O.w * inv));
                    }
                }
                if (threadIdx.x == 0) p.tickets[unit] = 0u;   // ready for the next call
            }
        }
        ptx::named_barrier_sync(1, kNT);               // the merge rows may be written again
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
    PgParams p{};
    const int BR = a.S % 32 == 0 ? 32 : a.S % 16 == 0 ? 16 : 8;
    p.nb = kChunk / BR;
    p.br_log = BR == 32 ? 5 : BR == 16 ? 4 : 3;
    // n / S = (t + (n - t) / 2) >> s_sh with t = high word of s_mul n, for
    // l = ceil(log2 S), s_mul = floor(2^32 (2^l - S) / S) + 1, s_sh = l - 1
    int l = 0;
    while ((1ll << l) < a.S) ++l;
    p.s_mul = unsigned((((1ull << l) - a.S) << 32) / unsigned(a.S) + 1);
    p.s_sh = l - 1;
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
    p.S = a.S;
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
