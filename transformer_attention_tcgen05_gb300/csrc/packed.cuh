// Blocks of query rows of packed sequences of different lengths, found on the
// device from the sequences' starts (shared by the packed forms of the tensor-core
// and the SIMT attention kernels).
//
// Sequence b has n queries, the last of its t keys.  Its rows are cut into blocks
// of BS; block i starts at position t - n + i BS and has the level (t - n) / BS + i,
// which grows with the keys that it reads.  Blocks are numbered by falling level, and
// within one by sequence, so that the longest start first.  The block of a number
// is found by bisection: with F(L) the blocks of level L or more, it lies in the
// largest L with F(L) > number.  One warp, 32 sequences at a time, of which the first
// 64 stay in registers (16 sequences: 1.0 to 1.4 us to a block's rows, which a kernel
// hides behind the block before).  No list is written, so a call needs no workspace and
// one launch.
//
// Sequences whose starts do not rise have no rows and are reported.  Such starts may
// make others overlap, in any number: no sum passes kMost per lane, and no more blocks
// are given out than disjoint sequences can have.
#pragma once

#include "common.cuh"

namespace attn {

struct PackedSeqs {
    const int32_t *cu_q, *cu_k;
    int B, Nq, Nkv;
    int most;                              // blocks that disjoint sequences can have, at most kMost
};

struct PackedBlock {
    int q_row, nq, k_row, nkv;             // the sequence's rows
    int q0;                                // first query of the block, within the sequence
};

class BlockFinder {
    static constexpr int kMost = 1 << 25;  // (of 32 lanes together: 2^30)

  public:
    // All lanes of a warp; report: invalid sequences set the device error word.
    __device__ __forceinline__ BlockFinder(const PackedSeqs &s, int bs_log, bool report, unsigned *err)
        : s_(s), log_(bs_log), lane_(threadIdx.x & 31) {
        bool wrong = false;
        int top = 0, sum = 0;
        first_ = load(lane_, wrong);
        second_ = load(lane_ + 32, wrong);
        top = imax(first_.level + first_.blocks, second_.level + second_.blocks);
        sum = first_.blocks + second_.blocks;
        for (int b = lane_ + 64; b < s_.B; b += 32) {
            const Seq q = load(b, wrong);
            top = imax(top, q.level + q.blocks);
            sum = imin(sum + q.blocks, kMost);
        }
        if (report && wrong) raise_device_error(err, kDevCheck);
        top_ = __reduce_max_sync(0xffffffffu, top);
        total = imin(__reduce_add_sync(0xffffffffu, sum), s_.most);
    }

    int total;                             // blocks to work on

    // The block of a number below `total`.
    __device__ __forceinline__ PackedBlock find(int number) const {
        int lo = 0, hi = top_;             // F(lo) > number >= F(hi)
        int behind = 0;                    // F(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1, f = from_level(mid);
            if (f > number) {
                lo = mid;
            } else {
                hi = mid;
                behind = f;
            }
        }
        int left = number - behind;        // blocks of this level before ours
        for (int b0 = 0;; b0 += 32) {      // one of the sequences has it
            const Seq q = get(b0 + lane_);
            const unsigned here = __ballot_sync(0xffffffffu, lo >= q.level && lo < q.level + q.blocks);
            const int n = __popc(here);
            if (left >= n && b0 + 32 < s_.B) {
                left -= n;
                continue;
            }
            const int at = __fns(here, 0, left + 1) & 31;
            const int b = imin(b0 + at, s_.B - 1);
            PackedBlock r;
            r.q_row = s_.cu_q[b];
            r.nq = s_.cu_q[b + 1] - r.q_row;
            r.k_row = s_.cu_k[b];
            r.nkv = s_.cu_k[b + 1] - r.k_row;
            r.q0 = (lo - ((r.nkv - r.nq) >> log_)) << log_;
            return r;
        }
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
    __device__ __forceinline__ Seq get(int b) const {
        bool wrong = false;
        return b == lane_ ? first_ : b == lane_ + 32 ? second_ : load(b, wrong);
    }
    static __device__ __forceinline__ int from(const Seq &q, int level) {
        return imin(imax(q.level + q.blocks - level, 0), q.blocks);
    }
    __device__ __forceinline__ int from_level(int level) const {
        int sum = from(first_, level) + from(second_, level);
        bool wrong = false;
        for (int b = lane_ + 64; b < s_.B; b += 32) sum = imin(sum + from(load(b, wrong), level), kMost);
        return __reduce_add_sync(0xffffffffu, sum);
    }
    const PackedSeqs &s_;
    int log_, lane_, top_;
    Seq first_, second_;
};

}  // namespace attn
