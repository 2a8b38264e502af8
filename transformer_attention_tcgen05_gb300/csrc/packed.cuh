// Blocks of query rows of packed sequences of different lengths, found on the
// device from the sequences' starts (shared by the packed forms of the tensor-core
// and the SIMT attention kernels).
//
// Sequence b has n queries, the last of its t keys.  Its rows are cut into blocks
// of BS; block i starts at position t - n + i BS.
//
// Up to 64 sequences, which a warp holds in registers: a block has the level (t - n) / BS
// + i, which grows with the keys that it reads.  Blocks are numbered by falling level,
// and within one by sequence, so that the longest start first.  The block of a number
// is found by bisection: with F(L) the blocks of level L or more, it lies in the
// largest L with F(L) > number (16 sequences: 1.0 to 1.4 us to a block's rows, which a
// kernel hides behind the block before).
//
// More of them: in the order of the sequences, from the last one's last block back, so
// that the longest blocks of each start first (99 prompts of 50 tokens and then one of
// 8000: 357 us, 390 from the front); those of b from number cu_q[b] / BS + b on.
// That leaves each at least as many numbers as it has blocks, and one at most empty, so
// that a search among the starts themselves finds a number, 32 probes at a time (two to
// four rounds).  (By levels, where every step of the bisection goes over all sequences,
// 4096 prompts of 20 tokens, 32 heads, took 8054 us; now 1845.)
//
// No list is written, so a call needs no workspace and one launch.  Sequences whose
// starts do not rise have no rows and are reported; others of such a call may go without
// theirs, where they overlap or stand behind those.
#pragma once

#include "common.cuh"

namespace attn {

struct PackedSeqs {
    const int32_t *cu_q, *cu_k;
    int B, Nq, Nkv;
    int most;                              // numbers that disjoint sequences can need (BlockFinder::most)
};

struct PackedBlock {
    int q_row, nq, k_row, nkv;             // the sequence's rows
    int q0;                                // first query of the block, within the sequence (>= nq: none)
};

class BlockFinder {
  public:
    static constexpr int kFew = 64;

    // The numbers that sequences of Nq queries together can need.
    static long long most(int B, int Nq, int bs) {
        return B > kFew ? (long long)Nq / bs + B : (Nq + (long long)imin(B, Nq) * (bs - 1)) / bs;
    }

    // All lanes of a warp; report: invalid sequences set the device error word.
    __device__ __forceinline__ BlockFinder(const PackedSeqs &s, int bs_log, bool report, unsigned *err)
        : s_(s), log_(bs_log), lane_(threadIdx.x & 31) {
        bool wrong = false;
        int sum;
        first_ = load(lane_, wrong);
        second_ = load(lane_ + 32, wrong);
        if (s_.B <= kFew) {
            top_ = __reduce_max_sync(0xffffffffu,
                                     imax(first_.level + first_.blocks, second_.level + second_.blocks));
            sum = __reduce_add_sync(0xffffffffu, first_.blocks + second_.blocks);
        } else {
            top_ = 0;
            sum = number_of(s_.B);
            if (report)
#pragma unroll 4
                for (int b = lane_ + kFew; b < s_.B; b += 32) load(b, wrong);
        }
        if (report && wrong) raise_device_error(err, kDevCheck);
        total = imax(0, imin(sum, s_.most));           // (starts that do not rise: anything)
    }

    int total;                             // numbers given out

    // The block of a number below `total`; q0 >= nq: there is none.
    __device__ __forceinline__ PackedBlock find(int number) const {
        int b, q0;
        if (s_.B <= kFew) {
            int lo = 0, hi = top_;         // F(lo) > number >= F(hi)
            int behind = 0;                // F(hi)
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                const int f = __reduce_add_sync(0xffffffffu, from(first_, mid) + from(second_, mid));
                if (f > number) {
                    lo = mid;
                } else {
                    hi = mid;
                    behind = f;
                }
            }
            int left = number - behind;    // blocks of this level before ours
            unsigned here = __ballot_sync(0xffffffffu, has(first_, lo));
            const int n = __popc(here);
            b = 0;
            if (left >= n) {
                left -= n;
                here = __ballot_sync(0xffffffffu, has(second_, lo));
                b = 32;
            }
            b = imin(b + (__fns(here, 0, left + 1) & 31), s_.B - 1);
            const int level = __shfl_sync(0xffffffffu, b < 32 ? first_.level : second_.level, b & 31);
            q0 = (lo - level) << log_;
        } else {
            number = total - 1 - number;
            b = 0;
            int end = s_.B;                // number_of(b) <= number < number_of(end)
            while (end - b > 1) {
                const int step = (end - b + 31) >> 5, at = b + lane_ * step;
                const unsigned ahead = __ballot_sync(0xffffffffu, at < end && (lane_ == 0 || number_of(at) <= number));
                b += (31 - __clz(ahead)) * step;
                end = imin(end, b + step);
            }
            q0 = (number - number_of(b)) << log_;
        }
        bool wrong = false;
        load(b, wrong);
        PackedBlock r{0, 0, 0, 0, 0};
        if (wrong || q0 < 0) return r;
        r.q_row = s_.cu_q[b];
        r.nq = s_.cu_q[b + 1] - r.q_row;
        r.k_row = s_.cu_k[b];
        r.nkv = s_.cu_k[b + 1] - r.k_row;
        r.q0 = q0;
        return r;
    }

  private:
    struct Seq {
        int level, blocks;                 // of its first block; how many
    };
    __device__ __forceinline__ Seq load(int b, bool &wrong) const {
        Seq q{0, 0};
        if (b >= s_.B) return q;
        const int q0 = s_.cu_q[b], q1 = s_.cu_q[b + 1], k0 = s_.cu_k[b], k1 = s_.cu_k[b + 1];
        if (q0 < 0 || q1 < q0 || q1 > s_.Nq || k0 < 0 || k1 < k0 || k1 > s_.Nkv || k1 - k0 < q1 - q0) {
            wrong = true;
            return q;
        }
        q.level = (k1 - k0 - (q1 - q0)) >> log_;
        q.blocks = (q1 - q0 + (1 << log_) - 1) >> log_;
        return q;
    }
    // The first number of a sequence's blocks (more than kFew sequences).
    __device__ __forceinline__ int number_of(int b) const { return (s_.cu_q[b] >> log_) + b; }
    static __device__ __forceinline__ int from(const Seq &q, int level) {
        return imin(imax(q.level + q.blocks - level, 0), q.blocks);
    }
    static __device__ __forceinline__ bool has(const Seq &q, int level) {
        return level >= q.level && level < q.level + q.blocks;
    }
    const PackedSeqs &s_;
    int log_, lane_, top_;
    Seq first_, second_;
};

}  // namespace attn
