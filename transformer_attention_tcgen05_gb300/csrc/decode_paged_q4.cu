// Grouped-query decode attention over a paged KV cache held in 4 bits, with an
// optional sliding window and sinks.
//
// The operation, the work list over the SMs and the joining of its parts are those
// of the 16-bit kernel (decode_paged.cu, paged_walk.cuh).  A token and KV head is a
// row of D + D / 8 bytes (rotary.cuh): 9/32 of the 16-bit cache's bytes, so the
// arithmetic, not HBM, decides here, and above all the instructions that turn codes
// into operands:
//
//  * Codes are multiplied as integers.  With q scaled by a power of two into f16 (bf16
//    values are exact there, down to 2^-24 of the head's largest) a group's
//    q . (n + M) runs on mma.sync m16n8k16, and s (q . n - 8 sum q) follows in
//    fp32, the constants M and 8 as the MMA's initial accumulator.  No code is
//    ever converted: a mask and an OR put it into the mantissa of 16 + n or 256 + n.
//  * A 16-bit word holds four codes rotated by two bits, so that two of them are
//    in place as they are and two after swapping the bytes: K's 8 codes cost one
//    byte permutation and four LOP3.  V's are needed in pairs of two tokens; the
//    permutation that pairs them swaps the bytes as well (two and four for 8).
//  * The channels of the MMA's k axis (K) and m axis (V) may come in any order, so a
//    row is laid out such that a lane's operands are consecutive: one 16-byte read
//    per token for K, one 8-byte read for V, no ldmatrix, no swizzle.
//  * V's scale belongs to the token, so it is multiplied into the weight:
//    w_jg = r_g p_j s_jg is the P operand of channel group g, f16, and a second MMA with a
//    matrix of -24 (16 + 8) and -264 (256 + 8) takes the constants out again with the very
//    same rounded weights.  r_g, a power of two per head and group, puts the group's
//    largest |p_j s_jg| so far into [2^7, 2^14), so that a product loses 2^-11 of itself
//    down to 2^-21 of that one, and 2^-32 of that one below, however far apart the scales
//    of a token's groups are.  (One reference for all groups of a token, their largest
//    scale, left a group 2^-14 of it at the edge of f16's normal range.)  The token
//    at the running maximum of the scores weighs 1, so that its products, and often most
//    of the sum, lose nothing (f16 outputs are 1.1 times as far from 64 bits as one rounding
//    is, 1.4 with the maximum rounded up to a whole power of two).  Where the maximum
//    moves, r_g rises by the power of two that weights fall by or the next one, so that the
//    largest product stays in that range; the sums of P V are divided by r_g at a segment's
//    end.
//  * The rows of a (page, head) are contiguous: a chunk of 32 tokens is one to four
//    plain bulk copies (4.6 KB at D = 128) for K, V and scales together.
//  * Up to 4 heads fill half of an MMA's 8 columns.  Then (SPLIT) the columns are heads by
//    two halves of a chunk's tokens: half the scales, exponentials and weights per lane
//    (8 x 4096 tokens, 32 heads on 8: 17.4 -> 16.2 us, before r_g).
//  * 3 CTAs of 4 warps per SM (2 for 9 to 16 heads of D 128); what a warp keeps of its
//    range beside the chunk at hand lies in shared memory, so that the registers suffice
//    (12 documents of 9000 to 60 000 tokens, 64 heads on 8, before r_g: 2 CTAs 88.9 us, 3
//    84.9, 4 88.5).
//
// Measured (bf16, D 128): 8 x 4096 tokens, 32 heads on 8, 16.4 us (2.3 TB/s; 26 us from
// 16-bit pages); 12 documents, 64 heads on 8, 85 us (4.38 TB/s; 55 at the copy rate), 128
// heads on 8, 131 us.  Of the first two, 12.2 and 64 are the copies, the work list, the
// merges and joins alone; the rest is arithmetic that does not hide behind them: a chunk
// takes a warp 469 instructions with up to 4 heads, 548 with 5 to 8, 744 with 9 to 16.  For
// the documents those are 36 us of issue slots: the chains within a chunk, which three
// warps per scheduler do not cover, count for more.  r_g and its check cost 0.3, 1 and 8 us.
// (Before them, leaving out V's part took the documents from 86 to 68 us, K's to 70, the
// softmax to 76, the MMAs of the constants to 79.5.)
//
// Sums and statistics are fp32; the output is rounded once.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "paged_walk.cuh"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kMaxSms = 192;               // workspace slots

template <int D, int NT>
struct Q4Cfg {
    static constexpr int CW = 4;                            // warps
    // CTAs: 168 registers per thread, which 16 heads of D 128 do not fit (12 documents, 128
    // heads on 8, before r_g: 132 us so, 122 with 2)
    static constexpr int PER_SM = NT == 2 && D == 128 ? 2 : 3;
    static constexpr int NS = D == 64 ? 4 : 2;              // chunks in flight per warp
    static constexpr int THREADS = CW * 32;
    static constexpr int HP = NT * 8;                       // padded heads per KV head
    static constexpr int NG = D / 32;                       // groups of channels with a scale each
    static constexpr int ROW = D + D / 8;
    static constexpr int TILE = kChunk * ROW;
    static constexpr int LDM = D + 4;                       // floats per merge row (bank spread)
    static constexpr int MERGE = CW * HP * LDM * 4;
    static constexpr int ML = CW * HP * 2 * 4;
    static constexpr int MISC = 2560;
    static constexpr int OFF_M = CW * NS * TILE;
    static constexpr int OFF_ML = OFF_M + MERGE;
    static constexpr int OFF_MISC = OFF_ML + ML;
    static constexpr int OFF_ZERO = OFF_MISC + MISC;        // SPLIT: zeros in the place of queries
    static constexpr int SMEM = OFF_ZERO + NG * 512 + 128;
    static_assert(NT * NG * 32 * 24 <= HP * LDM * 4, "the queries must fit a warp's merge rows");
    static_assert(PER_SM * (SMEM + 1024) <= 228 * 1024, "the CTAs of an SM must fit its shared memory");
};

// What a warp keeps of its range apart from the chunk it computes: where the loads
// are, where the computation is (both change once in many chunks), and the visible
// positions of the chunks asked for.
struct WarpRange {
    WalkState feed, work;
    int feed_next, feed_base, feed_more;   // the next chunk within feed's segment, its start in the range
    int work_f;                            // start of work's segment in the range
    uint32_t seen[64];                     // of chunk i at i % 64: a bit per position; 0: it has a bad page
};

struct MiscQ4 {
    uint64_t full[kMaxWarps * 4];          // [warp][slot]
    WarpRange warp[kMaxWarps];
    Schedule sched;
};
static_assert(sizeof(MiscQ4) <= 2560, "barrier block must fit its reserved bytes");

// The visible positions of the 32 from `base` on.
__device__ __forceinline__ uint32_t seen_bits(const Plan &r, int base) {
    auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
    return below(r.len - base) & (~below(r.lo - base) | below(r.s_end - base));
}

// Fields of two 16-bit words as f16 pairs: bits 6-9 as 16 + n, bits 2-5 as 256 + n;
// one instruction each.
__device__ __forceinline__ uint32_t code16(uint32_t w) { return ptx::and_or(w, 0x03c003c0u, 0x4c004c00u); }
__device__ __forceinline__ uint32_t code256(uint32_t w) { return ptx::and_or(w, 0x003c003cu, 0x5c005c00u); }
constexpr uint32_t kMinus24 = 0xce00ce00u, kMinus264 = 0xdc20dc20u;   // f16 pairs

// Powers of two.  2^n for an integer n in [-126, 126].
__device__ __forceinline__ float pow2(float n) { return __int_as_float((127 + int(n)) << 23); }
// a b / c, zero where it is too small.
__device__ __forceinline__ float pow2_ratio(float a, float b, float c) {
    return __int_as_float(imax(__float_as_int(a) + (__float_as_int(b) - __float_as_int(c)), 0));
}
// The larger values of two pairs of bf16 (NaN left out).
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
constexpr float kMostUp = 0x1p126f;        // the largest r_g (and where it starts)
constexpr float kFull = 0x1p14f;           // from here on r_g moves

// N 32-bit words of shared memory (the widest load that fits)
template <int N> __device__ __forceinline__ void read_words(const uint8_t *p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else if constexpr (N == 2) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        w[0] = u.x; w[1] = u.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

struct PagesQ4 {
    const uint8_t *base;
    long long page, head;                  // byte strides
};

// SPLIT (up to 4 heads per KV head): the 8 columns are the heads of the first 16
// tokens of a chunk and, again, of the other 16.  The queries of the columns that a
// token is not for are zeros, so that one accumulator fragment holds all 32 tokens and
// a lane has the scores, scales and weights of 4 instead of 8 pairs of token and head.
template <int D, int NT, bool SPLIT, bool F16>
__global__ void __launch_bounds__(Q4Cfg<D, NT>::THREADS, Q4Cfg<D, NT>::PER_SM)
decode_paged_q4_kernel(const PgParams p, const PagesQ4 pages) {
    using C = Q4Cfg<D, NT>;
    using H = H16<F16>;
    using T = typename H::T;
    static_assert(!SPLIT || NT == 1, "two halves of 8 columns");
    constexpr int CW = C::CW, NS = C::NS, NG = C::NG;
    constexpr int TT = SPLIT ? 1 : 2;                  // blocks of 16 tokens that a lane has weights of
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((128 - (ptx::smem_addr(smem_raw) & 127)) & 127);
    MiscQ4 *bars = reinterpret_cast<MiscQ4 *>(smem + C::OFF_MISC);
    Schedule *ms = &bars->sched;
    volatile int *abort = &ms->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int w = 0; w < CW; ++w)
            for (int s = 0; s < NS; ++s) ptx::mbar_init(&bars->full[w * 4 + s], 1);
        ptx::fence_barrier_init();
        ms->abort = 0;
    }
    if constexpr (SPLIT)
        for (int i = threadIdx.x; i < NG * 32; i += C::THREADS)
            reinterpret_cast<uint4 *>(smem + C::OFF_ZERO)[i] = make_uint4(0u, 0u, 0u, 0u);
    // programmatic dependent launch: nothing global is read or written before
    // the previous kernel (an append, say) has completed
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    Range range;
    if (!find_range<D, CW, T>(p, ms, range)) return;
    const bool alone = range.alone;
    const int team = range.team, rank = range.rank, at = range.at;
    WarpRange *mine = &bars->warp[warp];
    {
        const Walk w(p, range.list, ms->start_b[at], ms->start_len[at], ms->start_kvh[at], ms->start_v[at],
                     range.start, range.count);
        if (lane == 0) {
            mine->feed = mine->work = w;
            mine->feed_next = rank;
            mine->feed_base = mine->work_f = 0;
            mine->feed_more = 1;
        }
        __syncwarp();
    }

    // ---- loads: NS chunks ahead of the computation.  The lanes look up the pages of
    //      32 boxes (of up to 32 chunks of one segment) at once and keep their own box
    const int step = alone ? 0 : 2;                    // log2 of the team
    const uint64_t pol = ptx::l2_policy_evict_first();
    uint64_t *full = bars->full + warp * 4;
    uint8_t *ring = smem + warp * NS * C::TILE;
    int issued = 0, taken = 0, slot_in = 0;            // this warp's chunks: asked for, computed; issued % NS
    int left = 0;                                      // chunks of the group not asked for yet
    int first = 0;                                     // lane of the next one's first box
    const uint8_t *src = nullptr;                      // this lane's box; null: none
    int bytes = 0;                                     // of its chunk's boxes
    auto lookup = [&]() {
        Walk w(p, mine->feed);
        int next = mine->feed_next, base = mine->feed_base;
        bool more = mine->feed_more != 0;
        while (more && next >= w.cnt) {                // no (more) chunk of this warp in the segment
            base += w.cnt;
            more = w.next();
            next = (rank - base) & (team - 1);
        }
        left = first = 0;
        if (more) {
            const int BR = 1 << p.br_log, sub = lane >> (5 - p.br_log), box = lane & (p.nb - 1);
            left = imin(BR, (w.cnt - next + team - 1) >> step);   // 32 / nb = BR chunks at most
            const int at = chunk_of(w.plan, w.v0 + next + sub * team) * kChunk, pos = at + box * BR;
            // a box without a visible position is not read: its page may not
            // exist (past the end) or may be free again
            const bool need = sub < left && pos < w.plan.len && (pos + BR > w.plan.lo || pos < w.plan.s_end);
            int page = 0, row = 0;
            if (need) {
                const int e = div_s(p, pos);
                page = p.table[(long long)w.b * p.table_stride + e];
                row = pos - e * p.S;
            }
            const bool wrong = page < 0 || page >= p.num_pages;
            if (wrong) raise_device_error(p.err, kDevCheck);
            const unsigned bits = (1u << p.nb) - 1u, chunk0 = lane & ~(p.nb - 1);
            const unsigned bad = (__ballot_sync(0xffffffffu, wrong) >> chunk0) & bits;
            const unsigned go = (__ballot_sync(0xffffffffu, need && !wrong) >> chunk0) & bits;
            if (sub < left && box == 0) mine->seen[(issued + sub) & 63] = bad ? 0u : seen_bits(w.plan, at);
            bytes = __popc(go) * (C::ROW << p.br_log);
            src = need && !wrong ? pages.base + page * pages.page + w.kvh * pages.head + row * C::ROW : nullptr;
            next += left * team;
        }
        __syncwarp();
        if (lane == 0) {
            mine->feed = w;
            mine->feed_next = next;
            mine->feed_base = base;
            mine->feed_more = more;
        }
        __syncwarp();
    };
    auto issue = [&]() {
        if (left == 0) lookup();
        if (left == 0) return;
        const unsigned box = lane - first;
        if (box == 0) ptx::mbar_arrive_expect_tx(&full[slot_in], bytes);
        __syncwarp();
        if (box < unsigned(p.nb) && src)
            ptx::bulk_g2s(ring + slot_in * C::TILE + box * (C::ROW << p.br_log), src, C::ROW << p.br_log,
                          &full[slot_in], pol);
        --left;
        first += p.nb;
        ++issued;
        slot_in = slot_in + 1 == NS ? 0 : slot_in + 1;
    };

    float *mg = reinterpret_cast<float *>(smem + C::OFF_M);
    float *mml = reinterpret_cast<float *>(smem + C::OFF_ML);
    const int quad = lane >> 2, pair = lane & 3;

    // q of the unit's heads as MMA B operands (heads are columns) and the constants of
    // the codes times q per group, which wait in the warp's merge rows (they are read
    // again for every chunk: a register more per thread is a warp less per SM); and
    // what turns sums into base-2 exponents
    float qs[NT][2];
    uint4 *const qf = reinterpret_cast<uint4 *>(mg + warp * C::HP * C::LDM) + lane;              // [nt][g][lane]
    float2 *const qb = reinterpret_cast<float2 *>(mg + warp * C::HP * C::LDM + NT * NG * 128) + lane;
    // what the lane multiplies the first 16 tokens by, and the others
    const uint4 *const zero = reinterpret_cast<const uint4 *>(smem + C::OFF_ZERO);
    const uint4 *const q0 = SPLIT && quad >= 4 ? zero : qf, *const q1 = SPLIT && quad < 4 ? zero : qf;
    const uint32_t keep0 = quad < 4 ? 0xffffffffu : 0u, keep1 = ~keep0;
    const int own = SPLIT ? (pair >> 1) * 16 : 0;      // the lane's tokens of a chunk: block (t * 16 + own)
    auto load_q = [&]() {
        const int b = mine->work.b, kvh = mine->work.kvh;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = SPLIT ? quad & 3 : nt * 8 + quad;
            const T *qp = static_cast<const T *>(p.q) + b * p.q_sb + (long long)(kvh * p.G + h) * p.q_sh + pair * 8;
            uint4 raw[NG];
            float top = 0.f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                raw[g] = h < p.G ? *reinterpret_cast<const uint4 *>(qp + g * 32) : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t v[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(H::lo(v[i])), fabsf(H::hi(v[i]))));
            }
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            // the power of two that puts the head's largest value into [2^13, 2^14)
            const int e = imax(int(__float_as_uint(top) >> 23) - 127, -100);
            const float up = __uint_as_float(unsigned(127 + 13 - e) << 23);
            float sum[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint32_t v[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
                float x[8];
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = H::lo(v[i]) * up;
                    x[2 * i + 1] = H::hi(v[i]) * up;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) u[i] = pack_f16x2(x[i], x[i + 4]);
                qf[(nt * NG + g) * 32] = make_uint4(u[0], u[1], u[2], u[3]);
                sum[g] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum[g] = fmaf(i & 1 ? -264.f : -24.f, f16_lo(u[i]) + f16_hi(u[i]), sum[g]);
#pragma unroll
                for (int off = 1; off < 4; off <<= 1) sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], off);
            }
            // (not 0, which a score of -inf would make NaN; scores times so little vanish)
            const float sc = fmaxf(p.c_log2 * __uint_as_float(unsigned(127 - 13 + e) << 23), 0x1p-126f);
            // of the lane's two columns
#pragma unroll
            for (int j = 0; j < 2; ++j) qs[nt][j] = __shfl_sync(0xffffffffu, sc, (pair * 2 + j) * 4);
#pragma unroll
            for (int g = 0; g < NG; ++g)
                qb[(nt * NG + g) * 32] = make_float2(__shfl_sync(0xffffffffu, sum[g], pair * 8),
                                                     __shfl_sync(0xffffffffu, sum[g], pair * 8 + 4));
        }
    };
    // a lane's row of a block of 8 tokens in K and its two rows in V: with these the
    // reads of 8 lanes fall on all banks (rows are 16 bytes more than a multiple of
    // 128 at D = 128)
    const int tok = (quad >> 1) + 4 * (quad & 1);
    const int tv0 = pair, tv1 = pair + 4;              // columns 2 pair and 2 pair + 1 of P

    // after a timeout a warp computes nothing more but still walks the
    // segments: the other warps meet it at their barriers, and every unit's
    // ticket is counted up and reset as usual
    int dead = 0, s = 0, warm = 0;
    uint32_t parity = 0;
    for (bool more = true; more;) {
        // m: the running maximum, and what weights are taken against (0 while it is -inf);
        // up: r_g
        float m[NT][2], mu[NT][2], l[NT][2], up[NT][NG][2], acc[NT][2 * NG][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            mu[nt][0] = mu[nt][1] = l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int g = 0; g < NG; ++g) up[nt][g][0] = up[nt][g][1] = kMostUp;
#pragma unroll
            for (int i = 0; i < 2 * NG; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
        }
        int bad = dead;
        bool fresh = true, empty = true;               // a column, all of them without a score yet

        // this warp's chunks of the segment: the range's chunk number modulo the team.
        // The first NS rounds of all only ask for chunks; then come the segment's queries.
        int todo = (mine->work.cnt - ((rank - mine->work_f) & (team - 1)) + team - 1) >> step;
        bool have_q = false;
#pragma unroll 1
        while ((warm < NS || todo > 0) && !dead) {
            if (warm < NS) {
                issue();
                ++warm;
                continue;
            }
            if (!have_q) {
                load_q();
                have_q = true;
            }
            if (!__all_sync(0xffffffffu, ptx::mbar_wait_or_abort(&full[s], parity, p.err, abort))) {
                bad = dead = 1;
                break;
            }
            const uint32_t seen = mine->seen[taken & 63];
            const uint8_t *tile = ring + s * C::TILE;

            // ---- S^T = K q^T, group by group; x in base-2 exponents
            float x[TT][NT][4];
            uint32_t vs[TT][2][NG / 2];                // V's scales of the lane's tokens
            {
                uint32_t kw[2][2][NG], ks[TT][2][NG / 2];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        read_words<NG>(tile + (t * 16 + r * 8 + tok) * C::ROW + pair * (D / 8), kw[t][r]);
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint8_t *row = tile + (t * 16 + own + r * 8 + tok) * C::ROW;
                        read_words<NG / 2>(row + D, ks[t][r]);
                        read_words<NG / 2>(row + D + D / 16, vs[t][r]);
                    }
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) x[t][nt][0] = x[t][nt][1] = x[t][nt][2] = x[t][nt][3] = 0.f;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    uint32_t a0[2][4], a1[2][4];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint32_t w0 = kw[t][0][g], w1 = kw[t][1][g];
                        const uint32_t y0 = __byte_perm(w0, 0, 0x2301), y1 = __byte_perm(w1, 0, 0x2301);
                        a0[t][0] = code16(y0); a0[t][1] = code16(y1); a0[t][2] = code256(w0); a0[t][3] = code256(w1);
                        a1[t][0] = code16(w0); a1[t][1] = code16(w1); a1[t][2] = code256(y0); a1[t][3] = code256(y1);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint4 u0 = q0[(nt * NG + g) * 32], u1 = SPLIT ? q1[(nt * NG + g) * 32] : u0;
                        const float2 qc = qb[(nt * NG + g) * 32];
                        float c[TT][4];
                        ptx::mma16816_f16(c[0], a0[0], u0.x, u0.y, qc.x, qc.y, qc.x, qc.y);
                        ptx::mma16816<true>(c[0], a1[0], u0.z, u0.w);
                        if constexpr (SPLIT)
                            ptx::mma16816<true>(c[0], a0[1], u1.x, u1.y);
                        else
                            ptx::mma16816_f16(c[TT - 1], a0[1], u1.x, u1.y, qc.x, qc.y, qc.x, qc.y);
                        ptx::mma16816<true>(c[TT - 1], a1[1], u1.z, u1.w);
#pragma unroll
                        for (int t = 0; t < TT; ++t)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const float sc = g & 1 ? H::hi(ks[t][r][g / 2]) : H::lo(ks[t][r][g / 2]);
                                ptx::ffma2(x[t][nt][2 * r], x[t][nt][2 * r + 1], sc, sc, c[t][2 * r], c[t][2 * r + 1],
                                           x[t][nt][2 * r], x[t][nt][2 * r + 1]);
                            }
                    }
                }
            }
            // ---- positions that are not seen: their scales may be NaN
            if (seen != 0xffffffffu) {
                if (seen == 0u) bad = 1;
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (!((seen >> (t * 16 + own + r * 8 + tok)) & 1u)) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) x[t][nt][2 * r] = x[t][nt][2 * r + 1] = -INFINITY;
#pragma unroll
                            for (int g = 0; g < NG / 2; ++g) vs[t][r][g] = 0u;
                        }
            }
            // scales a group's sums of one column
            auto scale_sums = [&](int nt, int g, int j, float f) {
                acc[nt][2 * g][j] *= f;
                acc[nt][2 * g][j + 2] *= f;
                acc[nt][2 * g + 1][j] *= f;
                acc[nt][2 * g + 1][j + 2] *= f;
            };
            // ---- weights against the running maximum as it stands (a score of -inf weighs
            //      nothing, NaN stays NaN); returns the largest (NaN left out)
            float w[TT][NT][4];
            auto exponentials = [&]() {
                float top = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int t = 0; t < TT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            float a, b;
                            ptx::ffma2(a, b, x[t][nt][i], x[t][nt][i + 1], qs[nt][0], qs[nt][1], -mu[nt][0],
                                       -mu[nt][1]);
                            w[t][nt][i] = ptx::ex2(a);
                            w[t][nt][i + 1] = ptx::ex2(b);
                            top = ptx::fmax3(w[t][nt][i], w[t][nt][i + 1], top);
                        }
                return top;
            };
            // the running maximum of this chunk's scores too
            auto move_maximum = [&]() {
                bool none = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float top = -INFINITY;
#pragma unroll
                        for (int t = 0; t < TT; ++t) top = ptx::fmax3(top, x[t][nt][j], x[t][nt][j + 2]);
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1)
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                        const float mn = fmaxf(m[nt][j], top * qs[nt][j]);
                        // (both infinite: NaN, and then 0)
                        const float d = fmaxf(mn - m[nt][j], 0.f), less = ptx::ex2(-d);
                        const float more = pow2(ceilf(fminf(d, 126.f)));
                        m[nt][j] = mn;
                        mu[nt][j] = mn == -INFINITY ? 0.f : mn;
                        none = none || mn == -INFINITY;
                        l[nt][j] *= less;
                        // weights fall and r_g rises, so far as it may
                        if (!empty) {
#pragma unroll
                            for (int g = 0; g < NG; ++g) {
                                const float r = fminf(up[nt][g][j] * more, kMostUp);
                                scale_sums(nt, g, j, less * pow2_ratio(1.f, r, up[nt][g][j]));
                                up[nt][g][j] = r;
                            }
                        }
                    }
                fresh = __any_sync(0xffffffffu, none);
            };
            float most = exponentials();
            // ---- O^T += V^T P^T, a weight's scale in P
            const uint32_t minus[4] = {kMinus24, kMinus264, kMinus24, kMinus264};
            uint32_t ph[NT][NG][2];                    // of one block (SPLIT: both, side by side)
            // a token pair's weights times their scales, of the lane's two columns
            auto products = [&](int t, int nt, int g, float (&y)[4]) {
                const float s0 = g & 1 ? H::hi(vs[t][0][g / 2]) : H::lo(vs[t][0][g / 2]);
                const float s1 = g & 1 ? H::hi(vs[t][1][g / 2]) : H::lo(vs[t][1][g / 2]);
                ptx::ffma2(y[0], y[1], w[t][nt][0], w[t][nt][1], s0, s0, -0.f, -0.f);
                ptx::ffma2(y[2], y[3], w[t][nt][2], w[t][nt][3], s1, s1, -0.f, -0.f);
            };
            auto fill = [&](int t) {                   // returns the largest magnitude (NaN left out)
                float top = 0.f;
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float y[4];
                        products(t, nt, g, y);
                        ptx::ffma2(y[0], y[1], y[0], y[1], up[nt][g][0], up[nt][g][1], -0.f, -0.f);
                        ptx::ffma2(y[2], y[3], y[2], y[3], up[nt][g][0], up[nt][g][1], -0.f, -0.f);
                        top = ptx::fmax3(fabsf(y[0]), fabsf(y[1]), top);
                        top = ptx::fmax3(fabsf(y[2]), fabsf(y[3]), top);
                        ph[nt][g][0] = ptx::transpose8x8(pack_f16x2(y[0], y[1]));
                        ph[nt][g][1] = ptx::transpose8x8(pack_f16x2(y[2], y[3]));
                    }
                return top;
            };
            auto weigh = [&](int t) {
                if ((t == 0 && fresh) ||
                    __any_sync(0xffffffffu, fmaxf(fill(t), t == 0 ? most * (kFull / 256.f) : 0.f) >= kFull)) {
                    if (t == 0) {
                        move_maximum();
                        most = exponentials();
                    }
                    // r_g: the largest product of the block's tokens into [2^7, 2^8)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            float y[4];
                            products(t, nt, g, y);
                            uint32_t top = pack_bf16x2(fmaxf(fabsf(y[0]), fabsf(y[2])), fmaxf(fabsf(y[1]), fabsf(y[3])));
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1)
                                top = max_bf16x2(top, __shfl_xor_sync(0xffffffffu, top, off));
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int e = int(j ? top >> 23 : (top >> 7) & 0xffu);
                                const float r = fminf(__int_as_float(imin(127 + 7 + 127 - e, 253) << 23), up[nt][g][j]);
                                scale_sums(nt, g, j, pow2_ratio(1.f, r, up[nt][g][j]));
                                up[nt][g][j] = r;
                            }
                        }
                    fill(t);
                    empty = false;
                }
                if (t == 0) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int u = 0; u < TT; ++u) {
                            ptx::fadd2(l[nt][0], l[nt][1], l[nt][0], l[nt][1], w[u][nt][0], w[u][nt][1]);
                            ptx::fadd2(l[nt][0], l[nt][1], l[nt][0], l[nt][1], w[u][nt][2], w[u][nt][3]);
                        }
                }
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        ptx::mma16816<true>(acc[nt][2 * g], minus, ph[nt][g][0], ph[nt][g][1]);
                        ptx::mma16816<true>(acc[nt][2 * g + 1], minus, ph[nt][g][0], ph[nt][g][1]);
                    }
            };
            if constexpr (SPLIT) weigh(0);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t vw[2][2][NG / 2];             // [block of 8][token of the pair]
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    read_words<NG / 2>(tile + (t * 16 + r * 8 + tv0) * C::ROW + D / 2 + quad * (D / 16), vw[r][0]);
                    read_words<NG / 2>(tile + (t * 16 + r * 8 + tv1) * C::ROW + D / 2 + quad * (D / 16), vw[r][1]);
                }
                if constexpr (!SPLIT) weigh(t < TT ? t : 0);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    uint32_t u[2], y[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        u[r] = __byte_perm(vw[r][0][g / 2], vw[r][1][g / 2], g & 1 ? 0x7632 : 0x5410);
                        y[r] = __byte_perm(vw[r][0][g / 2], vw[r][1][g / 2], g & 1 ? 0x6723 : 0x4501);
                    }
                    const uint32_t a0[4] = {code16(y[0]), code256(u[0]), code16(y[1]), code256(u[1])};
                    const uint32_t a1[4] = {code16(u[0]), code256(y[0]), code16(u[1]), code256(y[1])};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint32_t keep = !SPLIT ? 0xffffffffu : t == 0 ? keep0 : keep1;
                        const uint32_t b0 = ph[nt][g][0] & keep, b1 = ph[nt][g][1] & keep;
                        ptx::mma16816<true>(acc[nt][2 * g], a0, b0, b1);
                        ptx::mma16816<true>(acc[nt][2 * g + 1], a1, b0, b1);
                    }
                }
            }
            // every lane has read the slot: it takes the next chunk
            __syncwarp();
            issue();
            ++taken;
            --todo;
            s = s + 1 == NS ? 0 : s + 1;
            parity ^= s == 0;
        }
        // this segment (the walk goes on to the next one)
        const WalkState seg = mine->work;
        const int u0 = seg.flat - seg.v0;              // flat index of the unit's first chunk
        {
            Walk w(p, seg);
            more = w.next();
            __syncwarp();
            if (lane == 0) {
                mine->work = w;
                mine->work_f += seg.cnt;
            }
            __syncwarp();
        }
        T *const o_unit = static_cast<T *>(p.o) + seg.b * p.o_sb + (long long)seg.kvh * p.G * p.o_sh;

        // ---- the warps' (reference, sum, O) -> one per head
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], off);
                const int h = nt * 8 + pair * 2 + j;
                if (quad == 0) {
                    mml[(warp * C::HP + h) * 2] = m[nt][j];
                    mml[(warp * C::HP + h) * 2 + 1] = l[nt][j];
                }
                float *row = mg + (warp * C::HP + h) * C::LDM + quad * 4;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float f = pow2_ratio(1.f, 1.f, up[nt][g][j]);
                    *reinterpret_cast<float4 *>(row + g * 32) =
                        make_float4(acc[nt][2 * g][j] * f, acc[nt][2 * g][j + 2] * f, acc[nt][2 * g + 1][j] * f,
                                    acc[nt][2 * g + 1][j + 2] * f);
                }
            }
        if (alone)
            store_alone<D, C::HP, C::LDM, SPLIT ? 2 : 1, F16>(p, mg, mml, bad, o_unit);
        else
            join_segment<D, CW, C::HP, C::LDM, SPLIT ? 2 : 1, F16>(p, ms, mg, mml, range, seg.b * p.Hkv + seg.kvh,
                                                                   seg.v0, seg.cnt, seg.plan.n, u0, bad, o_unit);
    }
    // after a timeout: let the copies this warp asked for land (bounded) before
    // the CTA's shared memory is released
    if (dead && lane == 0)
        for (int i = taken; i < issued; ++i) ptx::mbar_wait(&full[i % NS], (i / NS) & 1, nullptr);
}

// As in the 16-bit kernel the partials come first, at their largest size (3 CTAs per SM
// with 16 heads), so that the tickets lie at one place.
constexpr size_t kSlots = size_t(2) * kMaxSms * 48;    // slots x heads
constexpr size_t kPartBytes = kSlots * 128 * sizeof(float);
constexpr size_t kMlBytes = kSlots * 2 * sizeof(float);
static_assert(kPartBytes % 256 == 0 && kMlBytes % 256 == 0, "aligned workspace parts");

template <int D, int NT, bool SPLIT, bool F16>
attn_status_t launch_q4(const Ctx &c, const PgParams &p, const PagesQ4 &pages) {
    using C = Q4Cfg<D, NT>;
    static int done_mask = 0;
    static_assert(2 * C::PER_SM * kMaxSms * C::HP <= kSlots, "the partials must fit the workspace");
    auto kern = decode_paged_q4_kernel<D, NT, SPLIT, F16>;
    if (!ensure_smem_attr(reinterpret_cast<const void *>(kern), C::SMEM, c.device, &done_mask))
        return ATTN_ERR_RESOURCE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C::PER_SM * imin(c.sm_count, kMaxSms));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, p, pages) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    return launch_status(kFamDecodePaged);
}

template <int D>
attn_status_t launch_d(const Ctx &c, const PgParams &p, const PagesQ4 &pages, bool f16) {
    if (p.G <= 4) return f16 ? launch_q4<D, 1, true, true>(c, p, pages) : launch_q4<D, 1, true, false>(c, p, pages);
    if (p.G <= 8) return f16 ? launch_q4<D, 1, false, true>(c, p, pages) : launch_q4<D, 1, false, false>(c, p, pages);
    return f16 ? launch_q4<D, 2, false, true>(c, p, pages) : launch_q4<D, 2, false, false>(c, p, pages);
}

}  // namespace

size_t decode_paged_q4_workspace_bytes(int B, int Hkv) {
    return kPartBytes + kMlBytes + ((size_t(B) * Hkv * sizeof(unsigned) + 255) & ~size_t(255));
}

attn_status_t decode_paged_q4(const Ctx &c, attn_dtype_t dt, const PagedDecodeQ4 &a) {
    const bool f16 = dt == ATTN_F16;
    PgParams p = page_params(a.S);
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
    const PagesQ4 pages{static_cast<const uint8_t *>(a.pages), a.p_st[0], a.p_st[1]};
    return a.D == 128 ? launch_d<128>(c, p, pages, f16) : launch_d<64>(c, p, pages, f16);
}

}  // namespace attn
