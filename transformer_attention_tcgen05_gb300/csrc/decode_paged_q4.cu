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
//    w_jg = p_j s_jg is the P operand of channel group g, f16 (a rounding of 2^-12 of
//    each weight), and a second MMA with a matrix of -24 (16 + 8) and -264 (256 + 8)
//    takes the constants out again with the very same rounded weights.  The running
//    reference of the softmax is the maximum of x_j + log2 max_g |s_jg|, which keeps
//    every w_jg below 1 in any cache (below 2^8: the reference moves only when it must).
//  * The rows of a (page, head) are contiguous: a chunk of 32 tokens is one to four
//    plain bulk copies (4.6 KB at D = 128) for K, V and scales together.
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
    static constexpr int PER_SM = NT == 1 ? 3 : 2;          // CTAs
    static constexpr int NS = D == 64 ? 4 : 3;              // chunks in flight per warp
    static constexpr int THREADS = CW * 32;
    static constexpr int HP = NT * 8;                       // padded heads per KV head
    static constexpr int NG = D / 32;                       // groups of channels with a scale each
    static constexpr int ROW = D + D / 8;
    static constexpr int TILE = kChunk * ROW;
    static constexpr int LDM = D + 4;                       // floats per merge row (bank spread)
    static constexpr int MERGE = CW * HP * LDM * 4;
    static constexpr int ML = CW * HP * 2 * 4;
    static constexpr int MISC = 512;
    static constexpr int OFF_M = CW * NS * TILE;
    static constexpr int OFF_ML = OFF_M + MERGE;
    static constexpr int OFF_MISC = OFF_ML + ML;
    static constexpr int SMEM = OFF_MISC + MISC + 128;
    static_assert(PER_SM * (SMEM + 1024) <= 228 * 1024, "the CTAs of an SM must fit its shared memory");
};

struct MiscQ4 {
    uint64_t full[kMaxWarps * 4];          // [warp][slot]
    Schedule sched;
};
static_assert(sizeof(MiscQ4) <= 512, "barrier block must fit its reserved bytes");

// Fields of two 16-bit words as f16 pairs: bits 6-9 as 16 + n, bits 2-5 as 256 + n.
__device__ __forceinline__ uint32_t code16(uint32_t w) { return (w & 0x03c003c0u) | 0x4c004c00u; }
__device__ __forceinline__ uint32_t code256(uint32_t w) { return (w & 0x003c003cu) | 0x5c005c00u; }
constexpr uint32_t kMinus24 = 0xce00ce00u, kMinus264 = 0xdc20dc20u;   // f16 pairs

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

template <int D, int NT, bool F16>
__global__ void __launch_bounds__(Q4Cfg<D, NT>::THREADS, Q4Cfg<D, NT>::PER_SM)
decode_paged_q4_kernel(const PgParams p, const PagesQ4 pages) {
    using C = Q4Cfg<D, NT>;
    using H = H16<F16>;
    using T = typename H::T;
    constexpr int CW = C::CW, NS = C::NS, NG = C::NG;
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
    // programmatic dependent launch: nothing global is read or written before
    // the previous kernel (an append, say) has completed
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    Range range;
    if (!find_range<D, CW, T>(p, ms, range)) return;
    const bool alone = range.alone;
    const int team = range.team, rank = range.rank, at = range.at;
    Walk w(p, range.list, ms->start_b[at], ms->start_len[at], ms->start_kvh[at], ms->start_v[at], range.start,
           range.count);
    int f = 0;                                         // chunk number within the range

    // ---- loads: NS chunks ahead of the computation
    const int box_bytes = (1 << p.br_log) * C::ROW;
    const uint64_t pol = ptx::l2_policy_evict_first();
    uint64_t *full = bars->full + warp * 4;
    uint8_t *ring = smem + warp * NS * C::TILE;
    Feed feed(p, w, range);
    int issued = 0, taken = 0, slot_in = 0;            // this warp's chunks: asked for, computed; issued % NS
    unsigned bad_bits = 0;                             // bit i % 32: chunk i has a bad page
    auto issue = [&]() {
        if (!feed.next()) return;
        const unsigned go = feed.mine & ~feed.bad;
        bad_bits = (bad_bits & ~(1u << (issued & 31))) | (unsigned(feed.bad != 0) << (issued & 31));
        if (lane == 0) ptx::mbar_arrive_expect_tx(&full[slot_in], __popc(go) * box_bytes);
        __syncwarp();
        const int box = feed.box(go);
        if (box >= 0)
            ptx::bulk_g2s(ring + slot_in * C::TILE + box * box_bytes,
                          pages.base + feed.cur.page * pages.page + feed.cur.kvh * pages.head + feed.cur.row * C::ROW,
                          box_bytes, &full[slot_in], pol);
        ++issued;
        slot_in = slot_in + 1 == NS ? 0 : slot_in + 1;
    };
    float *mg = reinterpret_cast<float *>(smem + C::OFF_M);
    float *mml = reinterpret_cast<float *>(smem + C::OFF_ML);
    const int quad = lane >> 2, pair = lane & 3;

    // q of the unit's heads as MMA B operands (heads are columns), the constants of
    // the codes times q per group, and what turns sums into base-2 exponents
    uint32_t qf[NT][NG][4];
    float qb[NT][NG][2], qs[NT][2];
    auto load_q = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = nt * 8 + quad;
            const T *qp = static_cast<const T *>(p.q) + w.b * p.q_sb + (long long)(w.kvh * p.G + h) * p.q_sh + pair * 8;
            uint4 u[NG];
            float top = 0.f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                u[g] = h < p.G ? *reinterpret_cast<const uint4 *>(qp + g * 32) : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t v[4] = {u[g].x, u[g].y, u[g].z, u[g].w};
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
                const uint32_t v[4] = {u[g].x, u[g].y, u[g].z, u[g].w};
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = H::lo(v[i]) * up;
                    x[2 * i + 1] = H::hi(v[i]) * up;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) qf[nt][g][i] = pack_f16x2(x[i], x[i + 4]);
                sum[g] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum[g] = fmaf(i & 1 ? -264.f : -24.f, f16_lo(qf[nt][g][i]) + f16_hi(qf[nt][g][i]), sum[g]);
#pragma unroll
                for (int off = 1; off < 4; off <<= 1) sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], off);
            }
            const float sc = p.c_log2 * __uint_as_float(unsigned(127 - 13 + e) << 23);
            // of the lane's two columns
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                qs[nt][j] = __shfl_sync(0xffffffffu, sc, (pair * 2 + j) * 4);
#pragma unroll
                for (int g = 0; g < NG; ++g) qb[nt][g][j] = __shfl_sync(0xffffffffu, sum[g], (pair * 2 + j) * 4);
            }
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
        // m: the running reference, and what weights are taken against (0 while it is -inf)
        float m[NT][2], mu[NT][2], l[NT][2], acc[NT][2 * NG][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            mu[nt][0] = mu[nt][1] = l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * NG; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
        }
        int bad = dead;

        const int f_end = f + w.cnt;
        // this warp's chunks: the range's chunk number modulo the team.  The first
        // NS rounds of all only ask for chunks; then come the segment's queries.
        int fc = f + ((rank - f) & (team - 1));
        bool have_q = false;
#pragma unroll 1
        while ((warm < NS || fc < f_end) && !dead) {
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
            bad |= (bad_bits >> (taken & 31)) & 1u;
            const uint8_t *tile = ring + s * C::TILE;
            const int base = chunk_of(w.plan, w.v0 + (fc - f)) * kChunk;

            // ---- S^T = K q^T, group by group; x in base-2 exponents
            float x[2][NT][4];
            uint32_t vs[2][2][NG / 2];                 // V's scales of the lane's four tokens
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t kw[2][NG], ks[2][NG / 2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint8_t *row = tile + (t * 16 + r * 8 + tok) * C::ROW;
                    read_words<NG>(row + pair * (D / 8), kw[r]);
                    read_words<NG / 2>(row + D, ks[r]);
                    read_words<NG / 2>(row + D + D / 16, vs[t][r]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) x[t][nt][0] = x[t][nt][1] = x[t][nt][2] = x[t][nt][3] = 0.f;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const uint32_t y0 = __byte_perm(kw[0][g], 0, 0x2301), y1 = __byte_perm(kw[1][g], 0, 0x2301);
                    const uint32_t a0[4] = {code16(y0), code16(y1), code256(kw[0][g]), code256(kw[1][g])};
                    const uint32_t a1[4] = {code16(kw[0][g]), code16(kw[1][g]), code256(y0), code256(y1)};
                    const float s0 = g & 1 ? H::hi(ks[0][g / 2]) : H::lo(ks[0][g / 2]);
                    const float s1 = g & 1 ? H::hi(ks[1][g / 2]) : H::lo(ks[1][g / 2]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float c[4];
                        ptx::mma16816_f16(c, a0, qf[nt][g][0], qf[nt][g][1], qb[nt][g][0], qb[nt][g][1], qb[nt][g][0],
                                          qb[nt][g][1]);
                        ptx::mma16816<true>(c, a1, qf[nt][g][2], qf[nt][g][3]);
                        x[t][nt][0] = fmaf(s0, c[0], x[t][nt][0]);
                        x[t][nt][1] = fmaf(s0, c[1], x[t][nt][1]);
                        x[t][nt][2] = fmaf(s1, c[2], x[t][nt][2]);
                        x[t][nt][3] = fmaf(s1, c[3], x[t][nt][3]);
                    }
                }
            }
            // ---- the reference of a token: the logarithm of its largest scale
            float ref[2][2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float top = fmaxf(fabsf(H::lo(vs[t][r][0])), fabsf(H::hi(vs[t][r][0])));
                    if constexpr (NG == 4)
                        top = ptx::fmax3(fabsf(H::lo(vs[t][r][NG / 2 - 1])), fabsf(H::hi(vs[t][r][NG / 2 - 1])), top);
                    ref[t][r] = fmaxf(ptx::lg2(top), -60.f);
                }
            // ---- positions that are not seen: their scales may be NaN
            if (base + kChunk > w.plan.len || (base < w.plan.lo && base + kChunk > w.plan.s_end)) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int pos = base + t * 16 + r * 8 + tok;
                        if (pos >= w.plan.len || (pos < w.plan.lo && pos >= w.plan.s_end)) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) x[t][nt][2 * r] = x[t][nt][2 * r + 1] = -INFINITY;
#pragma unroll
                            for (int g = 0; g < NG / 2; ++g) vs[t][r][g] = 0u;
                        }
                    }
            }
            // ---- the running reference moves if a weight could pass 2^8, or is NaN
            float mx[NT][2];
            bool far = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        y[i] = fmaf(x[i >> 1][nt][j + (i & 1) * 2], qs[nt][j], ref[i >> 1][i & 1]);
                    mx[nt][j] = fmaxf(ptx::fmax3(y[0], y[1], y[2]), y[3]);
                    // (fmax leaves NaN out: a NaN score shows in its weight)
                    far = far || !(mx[nt][j] <= m[nt][j] + 8.f) || m[nt][j] == -INFINITY;
                }
            if (__any_sync(0xffffffffu, far)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float top = mx[nt][j];
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1)
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                        const float mn = fmaxf(m[nt][j], top);
                        const float alpha = mn == -INFINITY ? 1.f : ptx::ex2(m[nt][j] - mn);
                        m[nt][j] = mn;
                        mu[nt][j] = mn == -INFINITY ? 0.f : mn;
                        l[nt][j] *= alpha;
#pragma unroll
                        for (int i = 0; i < 2 * NG; ++i) {
                            acc[nt][i][j] *= alpha;
                            acc[nt][i][j + 2] *= alpha;
                        }
                    }
            }
            // ---- weights (a score of -inf weighs nothing, NaN stays NaN)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[t][nt][i] = ptx::ex2(fmaf(x[t][nt][i], qs[nt][i & 1], -mu[nt][i & 1]));
                        l[nt][i & 1] += x[t][nt][i];
                    }
            // ---- O^T += V^T P^T, a weight's scale in P
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t vw[2][2][NG / 2];             // [block of 8][token of the pair]
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    read_words<NG / 2>(tile + (t * 16 + r * 8 + tv0) * C::ROW + D / 2 + quad * (D / 16), vw[r][0]);
                    read_words<NG / 2>(tile + (t * 16 + r * 8 + tv1) * C::ROW + D / 2 + quad * (D / 16), vw[r][1]);
                }
                const uint32_t minus[4] = {kMinus24, kMinus264, kMinus24, kMinus264};
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
                    const float s0 = g & 1 ? H::hi(vs[t][0][g / 2]) : H::lo(vs[t][0][g / 2]);
                    const float s1 = g & 1 ? H::hi(vs[t][1][g / 2]) : H::lo(vs[t][1][g / 2]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint32_t b0 = ptx::transpose8x8(pack_f16x2(x[t][nt][0] * s0, x[t][nt][1] * s0));
                        const uint32_t b1 = ptx::transpose8x8(pack_f16x2(x[t][nt][2] * s1, x[t][nt][3] * s1));
                        ptx::mma16816<true>(acc[nt][2 * g], a0, b0, b1);
                        ptx::mma16816<true>(acc[nt][2 * g + 1], a1, b0, b1);
                        ptx::mma16816<true>(acc[nt][2 * g], minus, b0, b1);
                        ptx::mma16816<true>(acc[nt][2 * g + 1], minus, b0, b1);
                    }
                }
            }
            // every lane has read the slot: it takes the next chunk
            __syncwarp();
            issue();
            ++taken;
            fc += team;
            s = s + 1 == NS ? 0 : s + 1;
            parity ^= s == 0;
        }
        f = f_end;

        // this segment (the walk goes on to the next one)
        const int seg_b = w.b, seg_kvh = w.kvh, seg_v0 = w.v0, seg_cnt = w.cnt, seg_n = w.plan.n;
        const int u0 = w.flat - w.v0;                  // flat index of the unit's first chunk
        more = w.next();
        T *const o_unit = static_cast<T *>(p.o) + seg_b * p.o_sb + (long long)seg_kvh * p.G * p.o_sh;

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
                for (int g = 0; g < NG; ++g)
                    *reinterpret_cast<float4 *>(row + g * 32) =
                        make_float4(acc[nt][2 * g][j], acc[nt][2 * g][j + 2], acc[nt][2 * g + 1][j],
                                    acc[nt][2 * g + 1][j + 2]);
            }
        if (alone)
            store_alone<D, C::HP, C::LDM, F16>(p, mg, mml, bad, o_unit);
        else
            join_segment<D, CW, C::HP, C::LDM, F16>(p, ms, mg, mml, range, seg_b * p.Hkv + seg_kvh, seg_v0, seg_cnt,
                                                    seg_n, u0, bad, o_unit);
    }
    // after a timeout: let the copies this warp asked for land (bounded) before
    // the CTA's shared memory is released
    if (dead && lane == 0)
        for (int i = taken; i < issued; ++i) ptx::mbar_wait(&full[i % NS], (i / NS) & 1, nullptr);
}

template <int D, int NT, bool F16>
attn_status_t launch_q4(const Ctx &c, const PgParams &p, const PagesQ4 &pages) {
    using C = Q4Cfg<D, NT>;
    static int done_mask = 0;
    auto kern = decode_paged_q4_kernel<D, NT, F16>;
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

// As in the 16-bit kernel the partials come first, at their largest size (3 CTAs
// per SM with 8 heads, or 2 with 16), so that the tickets lie at one place.
constexpr size_t kSlots = size_t(2) * kMaxSms * 32;    // slots x heads
constexpr size_t kPartBytes = kSlots * 128 * sizeof(float);
constexpr size_t kMlBytes = kSlots * 2 * sizeof(float);
static_assert(kPartBytes % 256 == 0 && kMlBytes % 256 == 0, "aligned workspace parts");

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
    if (a.D == 128) {
        if (a.G <= 8) return f16 ? launch_q4<128, 1, true>(c, p, pages) : launch_q4<128, 1, false>(c, p, pages);
        return f16 ? launch_q4<128, 2, true>(c, p, pages) : launch_q4<128, 2, false>(c, p, pages);
    }
    if (a.G <= 8) return f16 ? launch_q4<64, 1, true>(c, p, pages) : launch_q4<64, 1, false>(c, p, pages);
    return f16 ? launch_q4<64, 2, true>(c, p, pages) : launch_q4<64, 2, false>(c, p, pages);
}

}  // namespace attn
