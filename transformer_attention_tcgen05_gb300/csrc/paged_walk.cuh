// The work list of decode attention over pages: which chunks a CTA computes, and
// how the parts of a unit are joined (device side, shared by the kernels of 16-bit
// pages, decode_paged.cu, and of pages held in 4 bits, decode_paged_q4.cu).
//
// A sequence is cut into chunks of 32 positions (those that hold a visible one);
// the chunks of all (sequence, KV head) units are numbered consecutively and each
// CTA takes one equal contiguous range.  The reasons and what they measured stand
// at decode_paged.cu.
#pragma once

#include <math.h>

#include "common.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kChunk = 32;        // positions per chunk

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

// The parameters that follow from the page size.
inline PgParams page_params(int S) {
    PgParams p{};
    p.S = S;
    const int BR = S % 32 == 0 ? 32 : S % 16 == 0 ? 16 : 8;
    p.nb = kChunk / BR;
    p.br_log = BR == 32 ? 5 : BR == 16 ? 4 : 3;
    // n / S = (t + (n - t) / 2) >> s_sh with t = high word of s_mul n, for
    // l = ceil(log2 S), s_mul = floor(2^32 (2^l - S) / S) + 1, s_sh = l - 1
    int l = 0;
    while ((1ll << l) < S) ++l;
    p.s_mul = unsigned((((1ull << l) - S) << 32) / unsigned(S) + 1);
    p.s_sh = l - 1;
    return p;
}

constexpr int kMaxWarps = 4;
constexpr int kFitted = 20;       // chunks by which a range may grow to be fitted to its units
// The longest unit (chunks) that counts as short: beside long ones (40 sequences of
// 1 to 900 tokens 11.7 us, 13.7 with 8, 11.8 with 4) and in a call without longer
// ones (100 x 250 tokens 20.2 us, 23.1 with 5).
constexpr int kWarpUnit = 5, kAllShort = 8;

struct Schedule {
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
struct WalkState {
    int list;
    Plan plan;
    int b, kvh, v0, cnt;
    int left;                              // chunks of the range from this segment on
    int flat;                              // flat index of the segment's first chunk

    int ahead;                             // seq_len[b + 1], loaded before it is needed
};
struct Walk : WalkState {
    const PgParams &p;

    __device__ Walk(const PgParams &pp, const WalkState &s) : WalkState(s), p(pp) {}
    __device__ Walk(const PgParams &pp, int l, int b0, int len0, int kvh0, int v, int f0, int count) : p(pp) {
        list = l;
        b = b0;
        kvh = kvh0;
        v0 = v;
        left = count;
        flat = f0;
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

// Takes the next ticket: releases what this CTA wrote, acquires what the
// holders of the earlier tickets wrote.
__device__ __forceinline__ unsigned ticket_add(unsigned *t) {
    unsigned old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(t) : "memory");
    return old;
}

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
__device__ __forceinline__ void mark_starts(const PgParams &p, Schedule *ms, int marks, int f0, int per, int b,
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
__device__ __noinline__ void mark_long_batch(const PgParams &p, Schedule *ms, int marks, int f0, int per,
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

// A CTA's (or, `alone`, a warp's) range of one of the call's two lists.
struct Range {
    bool alone;                            // every warp has whole units of its own
    int team, rank;                        // the warps that share the range, this one among them
    int list;                              // which units the list holds (plan_in)
    int per;                               // chunks per range
    int at, start, count;                  // its start's mark, first chunk and chunks
};

// Finds this CTA's range; false if it has none (its idle sequences are done).
// All threads of the CTA; reads the lengths.
template <int D, int CW, typename T>
__device__ __forceinline__ bool find_range(const PgParams &p, Schedule *ms, Range &range) {
    constexpr int kNT = CW * 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x, ctas = gridDim.x;
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
    if (aligned ? c >= parts_total : f0l >= total) return false;
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
    if (count <= 0) return false;                      // alone: no unit starts in this warp's share
    range.alone = alone;
    range.team = team;
    range.rank = rank;
    range.list = list;
    range.per = per;
    range.at = at;
    range.start = start;
    range.count = count;
    return true;
}

// The pages of one warp's next chunks, box by box: lane i holds box i % nb of
// chunk i / nb of the group.
struct Group {
    int page, row;                         // this lane's box
    unsigned needs, bads;                  // boxes to copy; boxes whose entry is no page
    int kvh, cnt;                          // KV head; chunks in the group (0: the range is done)
};

// The chunks that one warp copies, in order: a walk that runs ahead of the
// computation.  The 32 lanes look up the pages of 32 boxes at once, one group
// ahead, and keep them: after next(), the chunk's boxes are those of the nb lanes
// from `first` on, which have each its page (one behind the pool where the entry is
// no page) and row in cur, and copy their boxes themselves.  Bits from 0 on: the
// boxes to copy (`mine`), those without a page (`bad`).
struct Feed {
    const PgParams &p;
    Walk w;
    int team, step, next_chunk, base;      // this warp's next chunk within w's segment; its start
    bool more;
    Group cur, nxt;
    int gi;                                // chunk within cur
    unsigned mine, bad;
    int first;

    __device__ __forceinline__ Feed(const PgParams &pp, const Walk &walk, const Range &r)
        : p(pp), w(walk), team(r.team), step(r.alone ? 0 : 2), next_chunk(r.rank), base(0), more(true), cur{},
          nxt{}, gi(0), mine(0), bad(0), first(0), rank(r.rank) {}
    __device__ __forceinline__ Group lookup() {
        const int lane = threadIdx.x & 31, BR = 1 << p.br_log;
        const int sub = lane >> (5 - p.br_log), box = lane & (p.nb - 1);
        Group g;
        g.page = g.row = 0;
        g.needs = g.bads = 0;
        g.kvh = g.cnt = 0;
        while (more && next_chunk >= w.cnt) {          // no (more) chunk of this warp in the segment
            base += w.cnt;
            more = w.next();
            next_chunk = (rank - base) & (team - 1);
        }
        if (!more) return g;
        g.kvh = w.kvh;
        g.cnt = imin(BR, (w.cnt - next_chunk + team - 1) >> step);   // 32 / nb = BR chunks at most
        bool need = false;
        if (sub < g.cnt) {
            const int v = w.v0 + next_chunk + sub * team;
            const int pos = chunk_of(w.plan, v) * kChunk + box * BR;
            // a box without a visible position is not read: its page may not
            // exist (past the end) or may be free again
            need = pos < w.plan.len && (pos + BR > w.plan.lo || pos < w.plan.s_end);
            if (need) {
                const int e = div_s(p, pos);
                g.page = p.table[(long long)w.b * p.table_stride + e];
                g.row = pos - e * p.S;
            }
        }
        g.needs = __ballot_sync(0xffffffffu, need);
        next_chunk += g.cnt * team;
        return g;
    }
    // checks the entries (when they have arrived) before the group's first copy
    __device__ __forceinline__ void check(Group &g) {
        const bool wrong = ((g.needs >> (threadIdx.x & 31)) & 1u) && (g.page < 0 || g.page >= p.num_pages);
        if (wrong) {
            raise_device_error(p.err, kDevCheck);
            g.page = p.num_pages;
        }
        g.bads = __ballot_sync(0xffffffffu, wrong);
    }
    __device__ __forceinline__ bool next() {           // false: the range is done
#pragma unroll 1
        while (gi == cur.cnt && (nxt.cnt > 0 || more)) {
            cur = nxt;
            gi = 0;
            nxt = lookup();
            check(cur);
        }
        if (gi == cur.cnt) return false;
        const unsigned bits = (1u << p.nb) - 1u;
        first = gi * p.nb;
        mine = (cur.needs >> first) & bits;
        bad = (cur.bads >> first) & bits;
        ++gi;
        return true;
    }
    // this lane's box of the chunk, if it is one to copy (`of`: mine, or some of it), else -1
    __device__ __forceinline__ int box(unsigned of) const {
        const unsigned i = (threadIdx.x & 31) - unsigned(first);
        return i < 32u && ((of >> i) & 1u) ? int(i) : -1;
    }

  private:
    int rank;
};

// A whole unit in one warp's registers: through its own merge rows to 8-byte
// stores.  A head has ROWS partials per warp, HP / ROWS rows apart.
template <int D, int HP, int LDM, int ROWS, bool F16>
__device__ __forceinline__ void store_alone(const PgParams &p, const float *mg, const float *mml, int bad,
                                            typename H16<F16>::T *o_unit) {
    using H = H16<F16>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll 1
    for (int e = lane; e < p.G * (D / 4) && !bad; e += 32) {
        const int h = e / (D / 4), d = (e % (D / 4)) * 4, row = warp * HP + h;
        float L = mml[row * 2 + 1];
        float4 x = *reinterpret_cast<const float4 *>(mg + row * LDM + d);
        if constexpr (ROWS == 2) {
            const int row2 = row + HP / 2;
            const float m1 = mml[row * 2], m2 = mml[row2 * 2], M = fmaxf(m1, m2);
            const float w1 = m1 == -INFINITY ? 0.f : ptx::ex2(m1 - M), w2 = m2 == -INFINITY ? 0.f : ptx::ex2(m2 - M);
            const float l2 = mml[row2 * 2 + 1];
            L = (m1 == -INFINITY ? L : w1 * L) + (m2 == -INFINITY ? l2 : w2 * l2);
            const float4 y = *reinterpret_cast<const float4 *>(mg + row2 * LDM + d);
            x = make_float4(w1 * x.x + w2 * y.x, w1 * x.y + w2 * y.y, w1 * x.z + w2 * y.z, w1 * x.w + w2 * y.w);
        }
        const float inv = 1.f / L;
        *reinterpret_cast<uint2 *>(o_unit + h * p.o_sh + d) =
            make_uint2(H::pack(x.x * inv, x.y * inv), H::pack(x.z * inv, x.w * inv));
    }
    __syncwarp();
}

// Joins a segment's warps (their maxima and sums in mml, their sums of values in
// the rows of mg) and, where the range cuts the unit, the segment with the
// unit's others: chunks [v0, v0 + cnt) of a unit of n chunks whose first has the
// flat index u0.  HP: rows per warp, LDM: floats per row of mg, ROWS: partials of a
// head per warp, HP / ROWS rows apart.  All threads of
// the CTA; `bad`: the segment has a page that is none.
template <int D, int CW, int HP, int LDM, int ROWS, bool F16>
__device__ __forceinline__ void join_segment(const PgParams &p, Schedule *ms, const float *mg, const float *mml,
                                             const Range &range, int unit, int v0, int cnt, int n, int u0,
                                             int bad, typename H16<F16>::T *o_unit) {
    using H = H16<F16>;
    using T = typename H::T;
    constexpr int kNT = CW * 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x, per = range.per;
    if (lane == 0) ms->warp_bad[warp] = bad;
    ptx::named_barrier_sync(1, kNT);
#pragma unroll
    for (int i = 0; i < CW; ++i) bad |= ms->warp_bad[i];

    const bool whole = v0 == 0 && cnt == n;
    // a range holds at most one segment that starts inside its unit (slot 0)
    // and one that starts at its unit's head and is cut (slot 1)
    const int slot = 2 * cta + (v0 == 0 ? 1 : 0);
    float *po = p.part_o + (size_t)slot * HP * D;
    float *pml = p.part_ml + (size_t)slot * HP * 2;
#pragma unroll 1
    for (int e = threadIdx.x; e < p.G * (D / 4); e += kNT) {
        const int h = e / (D / 4), d = (e % (D / 4)) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int i = 0; i < CW * ROWS; ++i) M = fmaxf(M, mml[(i * (HP / ROWS) + h) * 2]);
        float L = 0.f;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < CW * ROWS; ++i) {
            const float mi = mml[(i * (HP / ROWS) + h) * 2], li = mml[(i * (HP / ROWS) + h) * 2 + 1];
            // a warp that saw nothing, or only scores of -inf, adds nothing
            // (its sum is zero, or NaN if one of its scores was)
            const float wt = mi == -INFINITY ? 0.f : ptx::ex2(mi - M);
            L += mi == -INFINITY ? li : wt * li;
            const float4 x = *reinterpret_cast<const float4 *>(mg + (i * (HP / ROWS) + h) * LDM + d);
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
        const int c0 = int(unsigned(u0) / unsigned(per)), c1 = int(unsigned(u0 + n - 1) / unsigned(per));
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
                            ml[i] = __ldcg(reinterpret_cast<const float2 *>(p.part_ml + sl * HP * 2) + h);
                            x[i] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + sl * HP * D + h * D + d));
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

}  // namespace
}  // namespace attn
