// Rotary positions: rows of any tensor (attn_rope_fwd), and of the new tokens on
// their way into a paged cache, 16-bit / fp32 or held in 4 bits, with the reader
// that gives a 4-bit cache's rows back.
//
// Rows that stay 16-bit or fp32 are bound by memory: a thread owns two times eight
// channels of a row (both halves of eight pairs, two 16-byte vectors of a 16-bit type),
// walks the heads of its token and has the vectors of four rows in flight.  A row belongs
// to D / 16 lanes and nothing of it passes through shared memory, so it may be rotated in place.
// The angles of a tile of tokens are computed once into shared memory while the first
// rows arrive.  (Eight channels per thread with the partners read a second time, and
// the angles computed by every thread for itself, executed four times the
// instructions.)  bf16, 8192 x 32 rows of D 128: 22.5 us, 6.0 TB/s (29.2 that way);
// append of 20 000 tokens, 32 heads on 8: 78.5 us, 6.3 TB/s (193); 64 tokens 2.9 us.
//
// Rows coded in 4 bits are bound by instructions (320 per warp and two rows, a quarter of
// them angles; 63% of the issue slots): 20 000 tokens 37.4 us for K and V alone, 76 with
// their queries, whose CTAs they run beside; 64 tokens 3.1 us.  Extrema in packed pairs
// and with NaN carried along, the next heads' rows on the way and the scales of K and V in
// different lanes brought K and V of 5000 tokens from 15.8 to 12.9 us; a fourth CTA per SM
// leaves too few registers (18.3).  The reader: 22 500 rows 21.7 us, 5.4 TB/s.
#include "kernels.h"
#include "ptx.cuh"
#include "rotary.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;

template <typename... P, typename... A>
attn_status_t launch(const Ctx &c, int family, void (*kern)(P...), dim3 grid, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = c.stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, P(args)...) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    return launch_status(family);
}

constexpr int kPerSm = 3;                              // CTAs
constexpr int kTile = 16;                              // most tokens of a tile

// How a CTA's threads are laid over a tile: 2^lane_log lanes per row, 2^tb_log tokens,
// the rest over heads.
struct Tile {
    int lane_log, tb_log;
    __host__ __device__ int vec(int t) const { return t & ((1 << lane_log) - 1); }
    __host__ __device__ int token(int t) const { return (t >> lane_log) & ((1 << tb_log) - 1); }
    __host__ __device__ int lane(int t) const { return t >> (lane_log + tb_log); }
    __host__ __device__ int lanes() const { return kThreads >> (lane_log + tb_log); }
    __host__ __device__ int tokens() const { return 1 << tb_log; }
    // rows of 8 channels per lane instead of 16
    __host__ __device__ Tile finer() const { return Tile{lane_log + 1, tb_log}; }
};

// The most tokens per CTA (fewest angles computed) that leave `want` CTAs, but no fewer
// than give every lane one of a token's `rows` (8 heads, 1030 tokens of D 64 in fp32:
// 3.4 us, 4.5 with a token per CTA).
Tile make_tile(int D, long long tokens, int rows, long long want) {
    Tile t;
    t.lane_log = D == 128 ? 3 : D == 64 ? 2 : 1;
    t.tb_log = 4;
    while (t.tb_log > 0 && (tokens >> t.tb_log) < want && t.lanes() < rows) --t.tb_log;
    return t;
}

// The channels of a thread: [a, a + 8) and [b, b + 8), its row's pairs 8 vec .. 8 vec + 7
// if they are rotated.
struct Channels {
    int a, b;
    bool turns;
    __device__ __forceinline__ Channels(const Rotation &r, int vec) {
        turns = vec * 16 < r.rot;
        const bool half = turns && !r.interleaved;
        a = half ? vec * 8 : vec * 16;
        b = half ? a + r.rot / 2 : a + 8;
    }
};

// -------------------------------------------------------------------- rope

struct RopeRows {
    const void *x;
    void *y;
    const int32_t *pos;
    long long pos_stride;                              // between batches
    TensorStrides sx, sy;
    int H, N, slice;                                   // slice: heads per CTA
    long long tokens;                                  // B * N
    Rotation rot;
    Tile tile;
};

template <typename T>
__global__ void __launch_bounds__(kThreads, kPerSm) rope_rows_kernel(const RopeRows p) {
    constexpr int U = sizeof(T) == 4 ? 2 : 4;
    __shared__ __align__(16) float2 tab[kTile * 64];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x, hl = p.tile.lanes(), tl = p.tile.token(tid);
    const Channels ch(p.rot, p.tile.vec(tid));
    const long long t0 = (long long)blockIdx.x << p.tile.tb_log, t = t0 + tl;
    const bool here = t < p.tokens;
    const long long b = here ? t / p.N : 0, n = here ? t % p.N : 0;
    const int h_end = imin(p.H, (blockIdx.y + 1) * p.slice);
    const T *x = static_cast<const T *>(p.x) + b * p.sx.b + n * p.sx.n;
    T *y = static_cast<T *>(p.y) + b * p.sy.b + n * p.sy.n;
    Row8<T> va[U], vb[U];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (here && h0 + u * hl < h_end) {
                const T *src = x + (h0 + u * hl) * p.sx.h;
                va[u].load(src + ch.a);
                vb[u].load(src + ch.b);
            }
    };
    int h = blockIdx.y * p.slice + p.tile.lane(tid);
    load(h);                                           // on the way while the angles are computed
    fill_turns(p.rot, tab, p.tile.tokens(), [&](int i) {
        const long long u = t0 + i < p.tokens ? t0 + i : 0;
        return p.pos[u / p.N * p.pos_stride + u % p.N];
    });
    __syncthreads();
    const int step = p.rot.rot / 16;                   // lanes that rotate
    const float4 *turns = reinterpret_cast<const float4 *>(tab) + tl * (p.rot.rot / 4) + p.tile.vec(tid);
#pragma unroll 1
    for (; h < h_end; h += U * hl) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (here && h + u * hl < h_end) {
                if (ch.turns) rotate16<T>(turns, step, p.rot.interleaved, va[u], vb[u]);
                T *dst = y + (h + u * hl) * p.sy.h;
                va[u].store(dst + ch.a);
                vb[u].store(dst + ch.b);
            }
        if (h + U * hl < h_end) load(h + U * hl);
    }
}

// ------------------------------------------------------------------ append

struct AppendRows {
    const void *kn, *vn, *q;
    void *qo;
    long long kn_st[2], vn_st[2], q_st[2], qo_st[2];   // (token, head)
    void *k, *v;                                       // 4-bit: k alone
    long long k_st[3], v_st[3];                        // (page, head, token); 4-bit: bytes
    const int32_t *table;
    long long table_stride;
    int32_t *seq_len;
    const int32_t *cu;                                 // null: token b is the next one of sequence b
    int B, N, Hq, Hkv, D, S, P, max_pages, advance;
    int apart;                                         // 4-bit: q, and K and V, in CTAs of their own
    Rotation rot;
    Tile tile;
    unsigned *err;
};

// Where a tile's tokens go.
struct Dest {
    int seq[kTile], first[kTile], count[kTile];        // sequence (-1: none), its first row and rows
    int pos[kTile];                                    // length so far or first position, then the
                                                       // position (-1: the request does not fit)
    int page[kTile], row[kTile];                       // page -1: none
};

// Sequence, first row and row count of the tile's tokens [t0, t0 + n), from the
// starts cu[0..B] of the packed sequences, and the sequence's `base` (null: 0).  The first
// CTA reports sequences that cannot be, and empty ones whose base is not `valid` (others'
// rows tell).
template <typename F>
__device__ __forceinline__ void find_sequences(Dest &d, const int32_t *cu, const int32_t *base, int B, int N, int t0,
                                               int n, unsigned *err, F valid) {
    if (threadIdx.x < kTile) d.seq[threadIdx.x] = -1;
    __syncthreads();
    for (int b = threadIdx.x; b < B; b += kThreads) {
        const int lo = cu[b], hi = cu[b + 1], from = base ? base[b] : 0;
        const bool wrong = lo < 0 || hi < lo || hi > N;
        if (blockIdx.x == 0 && (wrong || (hi == lo && !valid(from)))) raise_device_error(err, kDevCheck);
        if (wrong) continue;
        for (int t = imax(lo, t0); t < imin(hi, t0 + n); ++t) {
            d.seq[t - t0] = b;
            d.first[t - t0] = lo;
            d.count[t - t0] = hi - lo;
            d.pos[t - t0] = from;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ bool append_fits(const AppendRows &p, int len, int n) {
    return len >= 0 && (long long)len + n <= (long long)p.max_pages * p.S;
}

// Looks up where the tile's tokens go, and the angles of their positions.
__device__ __forceinline__ void find_places(const AppendRows &p, Dest &d, float2 *tab, int t0) {
    const int tid = threadIdx.x, TB = p.tile.tokens();
    if (p.cu) {
        find_sequences(d, p.cu, p.seq_len, p.B, p.N, t0, TB, p.err, [&](int len) { return append_fits(p, len, 0); });
    } else if (tid < TB) {
        d.seq[tid] = t0 + tid < p.N ? t0 + tid : -1;
        d.first[tid] = t0 + tid;
        d.count[tid] = 1;
        if (t0 + tid < p.N) d.pos[tid] = p.seq_len[t0 + tid];
    }
    if (tid < TB) {
        int pos = -1, page = -1, row = 0;
        const int b = d.seq[tid];
        if (b >= 0) {
            const int len = d.pos[tid];
            if (append_fits(p, len, d.count[tid])) {
                // (of sequences that overlap, which takes starts that do not rise, a row
                // may hold one's length and another's start)
                const long long at = (long long)len + t0 + tid - d.first[tid];
                if (at >= 0 && at < (long long)p.max_pages * p.S) pos = int(at);
            }
            if (pos >= 0) {
                row = pos % p.S;
                page = p.table[b * p.table_stride + pos / p.S];
                if (page < 0 || page >= p.P) page = -1;
            }
            if (page < 0) raise_device_error(p.err, kDevCheck);
        }
        d.pos[tid] = pos;
        d.page[tid] = page;
        d.row[tid] = row;
    }
    __syncthreads();
    if (p.rot.rot > 0) {
        fill_turns(p.rot, tab, TB, [&](int i) { return d.pos[i]; });
        __syncthreads();
    }
}

// Rows of K and V into a cache held in 4 bits: D / 8 lanes each, so that 4 neighbours
// hold a group of 32 channels; the partners of a rotated half are read a second time.
// The rows of a thread's next two heads are on the way while one's are coded.
template <typename T>
struct CodedRows {
    const AppendRows &p;
    const T *kn, *vn;
    int c0, token, first, step, other;                 // channels, token, heads of the thread
    bool in, rotated;
    Row8<T> k[2], kp[2], v[2];

    __device__ __forceinline__ CodedRows(const AppendRows &p_, int t0) : p(p_) {
        const Tile fine = p.tile.finer();
        c0 = fine.vec(threadIdx.x) * 8;
        token = fine.token(threadIdx.x);
        first = fine.lane(threadIdx.x);
        step = fine.lanes();
        in = t0 + token < p.N;
        rotated = c0 < p.rot.rot;
        const int half = p.rot.rot / 2;
        other = !rotated || p.rot.interleaved ? 0 : c0 >= half ? -half : half;
        kn = static_cast<const T *>(p.kn) + (t0 + token) * p.kn_st[0] + first * p.kn_st[1] + c0;
        vn = static_cast<const T *>(p.vn) + (t0 + token) * p.vn_st[0] + first * p.vn_st[1] + c0;
        load(0, first);
        load(1, first + step);
    }
    __device__ __forceinline__ void load(int u, int h) {
        if (in && h < p.Hkv) {
            k[u].load(kn);
            if (other != 0) kp[u].load(kn + other);
            v[u].load(vn);
        }
        kn += step * p.kn_st[1];
        vn += step * p.vn_st[1];
    }
    // All lanes take every step: their neighbours' values pass by shuffles.
    __device__ __forceinline__ void run(const Dest &d, const float2 *tab) {
        const int rot = p.rot.rot, g = c0 >> 5, pl = (c0 >> 3) & 3;
        const bool inter = p.rot.interleaved, upper = other < 0;
        // y = x c + partner s, s of either sign
        float c[8], s[8];
        if (rotated) {
            const float2 *w = tab + token * (rot / 2);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 x = w[turn_at(rot, inter ? (c0 + i) / 2 : (upper ? c0 + other : c0) + i)];
                c[i] = x.x;
                s[i] = (inter ? i & 1 : upper) ? x.y : -x.y;
            }
        }
        const long long page = d.page[token];
        const bool keep = in && page >= 0;
        uint8_t *to = static_cast<uint8_t *>(p.k) + (keep ? page * p.k_st[0] + d.row[token] * p.k_st[2] : 0) +
                      first * p.k_st[1];
        const int at_k = pl * (p.D / 8) + 4 * g, at_v = p.D / 2 + (2 * pl + (g & 1)) * (p.D / 16) + 2 * (g & ~1);
        const uint32_t order = g & 1 ? 0x3276u : 0x5410u;
        auto code = [&](int u, int h) {
            float x[8], inv;
            k[u].get(x);
            if (rotated) {
                float y[8];
                if (inter) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
                } else {
                    kp[u].get(y);
                }
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    ptx::ffma2(x[i], x[i + 1], x[i], x[i + 1], c[i], c[i + 1], -0.f, -0.f);
                    ptx::ffma2(x[i], x[i + 1], y[i], y[i + 1], s[i], s[i + 1], x[i], x[i + 1]);
                }
            }
            // the even lanes of a group work out K's scale, the odd ones V's
            const float best_k = q4_best(x), best_v = q4_best<T>(v[u].u);
            const T scale = q4_scale<T>(pl & 1 ? best_v : best_k, inv);
            const float inv2 = __shfl_xor_sync(0xffffffffu, inv, 1);
            const uint32_t wk = q4_codes<H16F<T>::f16>(x, pl & 1 ? inv2 : inv);
            v[u].get(x);
            const uint32_t wv = q4_codes<H16F<T>::f16>(x, pl & 1 ? inv : inv2);
            // V: words of two neighbouring groups, one of this lane's own and one of the
            // lane of the other group that holds the same channels of it
            const uint32_t o = __shfl_xor_sync(0xffffffffu, wv, 4);
            if (keep && h < p.Hkv) {
                *reinterpret_cast<uint32_t *>(to + at_k) = wk;
                *reinterpret_cast<uint32_t *>(to + at_v) = __byte_perm(wv, o, order);
                if (pl < 2) *reinterpret_cast<T *>(to + p.D + pl * (p.D / 16) + 2 * g) = scale;
            }
            to += step * p.k_st[1];
        };
#pragma unroll 1
        for (int h = first; h - first < p.Hkv; h += 2 * step) {
            code(0, h);
            if (h + step - first >= p.Hkv) break;
            load(0, h + 2 * step);
            code(1, h + step);
            load(1, h + 3 * step);
        }
    }
};

// Rows of q, and of K and V into a 16-bit or fp32 cache: D / 16 lanes each.  Q4: K and V
// as CodedRows, in CTAs of their own where no CTA may see another's new lengths.
template <typename T, bool Q4>
__global__ void __launch_bounds__(kThreads, kPerSm) append_rows_kernel(const AppendRows p) {
    constexpr int U = sizeof(T) == 4 ? 2 : 4;
    __shared__ Dest d;
    __shared__ __align__(16) float2 tab[kTile * 64];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x, TB = p.tile.tokens();
    const bool two = Q4 && p.apart;                    // odd CTAs: K and V, even ones: q
    const int t0 = (two ? blockIdx.x >> 1 : blockIdx.x) * TB;
    if (Q4 && (p.Hq == 0 || (two && (blockIdx.x & 1)))) {
        if constexpr (Q4) {
            CodedRows<T> rows(p, t0);                  // on the way while their places are looked up
            find_places(p, d, tab, t0);
            rows.run(d, tab);
        }
    } else {
        const int hl = p.tile.lanes(), tl = p.tile.token(tid), t = t0 + tl;
        const bool in = t < p.N;
        const Channels ch(p.rot, p.tile.vec(tid));
        const int heads = Q4 ? p.Hq : p.Hq + 2 * p.Hkv;    // of q, then K, then V
        // row h is at base + h stride of its tensor
        const T *const sq = static_cast<const T *>(p.q) + t * p.q_st[0] + ch.a;
        const T *const sk = static_cast<const T *>(p.kn) + t * p.kn_st[0] - p.Hq * p.kn_st[1] + ch.a;
        const T *const sv = static_cast<const T *>(p.vn) + t * p.vn_st[0] - (p.Hq + p.Hkv) * p.vn_st[1] + ch.a;
        const int apart = ch.b - ch.a;
        Row8<T> va[U], vb[U];
        auto load = [&](int h0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * hl;
                if (!in || h >= heads) continue;
                const bool is_q = Q4 || h < p.Hq, is_k = h < p.Hq + p.Hkv;
                const T *src = (is_q ? sq : is_k ? sk : sv) + h * (is_q ? p.q_st[1] : is_k ? p.kn_st[1] : p.vn_st[1]);
                va[u].load(src);
                vb[u].load(src + apart);
            }
        };
        load(p.tile.lane(tid));                        // on the way while their places are looked up
        find_places(p, d, tab, t0);
        const bool known = in && d.pos[tl] >= 0;
        const long long page = d.page[tl], row = d.row[tl];
        const bool stored = in && page >= 0;
        const int step = p.rot.rot / 16;               // lanes that rotate
        const float4 *turns = reinterpret_cast<const float4 *>(tab) + tl * (p.rot.rot / 4) + p.tile.vec(tid);
        T *const dq = static_cast<T *>(p.qo) + t * p.qo_st[0] + ch.a;
        T *const dk = static_cast<T *>(p.k) + page * p.k_st[0] + row * p.k_st[2] - p.Hq * p.k_st[1] + ch.a;
        T *const dv = static_cast<T *>(p.v) + page * p.v_st[0] + row * p.v_st[2] - (p.Hq + p.Hkv) * p.v_st[1] + ch.a;
#pragma unroll 1
        for (int h0 = p.tile.lane(tid); h0 < heads; h0 += U * hl) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * hl;
                const bool is_q = Q4 || h < p.Hq, is_k = h < p.Hq + p.Hkv;
                if (h >= heads || !(is_q ? known : stored)) continue;
                if (ch.turns && (is_q || is_k)) rotate16<T>(turns, step, p.rot.interleaved, va[u], vb[u]);
                T *dst = (is_q ? dq : is_k ? dk : dv) + h * (is_q ? p.qo_st[1] : is_k ? p.k_st[1] : p.v_st[1]);
                va[u].store(dst);
                vb[u].store(dst + apart);
            }
            if (h0 + U * hl < heads) load(h0 + U * hl);
        }
        if constexpr (Q4) {
            if (!two) CodedRows<T>(p, t0).run(d, tab);
        }
    }
    // one token per sequence: no other CTA reads this length
    if (!p.cu && p.advance && tid < TB && d.page[tid] >= 0) p.seq_len[d.seq[tid]] = d.pos[tid] + 1;
}

// Advances the lengths after an append of packed sequences (every tile has read
// them by now): one warp per sequence, which stays where it was if one of its
// pages was bad.
__global__ void __launch_bounds__(kThreads) advance_rows_kernel(const AppendRows p) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int b = (blockIdx.x * kThreads + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    if (b >= p.B) return;
    const int lo = p.cu[b], n = p.cu[b + 1] - lo, len = p.seq_len[b];
    if (lo < 0 || n < 0 || lo + n > p.N) return;
    bool ok = append_fits(p, len, n);
    if (!ok || n == 0) return;
    for (int i = len / p.S + lane; i <= (len + n - 1) / p.S; i += 32) {
        const int page = p.table[b * p.table_stride + i];
        ok = ok && page >= 0 && page < p.P;
    }
    if (__all_sync(0xffffffffu, ok) && lane == 0) p.seq_len[b] = len + n;
}

// ------------------------------------------------------------------ gather

struct GatherRows {
    const uint8_t *pages;
    long long p_st[2];                                 // bytes (page, head)
    const int32_t *table;
    long long table_stride;
    const int32_t *start, *cu;                         // start null: 0
    void *k, *v;
    long long k_st[2], v_st[2];                        // (token, head)
    int B, N, Hkv, D, S, P, max_pages;
    Tile tile;
    unsigned *err;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) gather_rows_kernel(const GatherRows p) {
    constexpr int U = 8;
    __shared__ Dest d;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x, TB = p.tile.tokens(), hl = p.tile.lanes();
    const int t0 = blockIdx.x * TB, tl = p.tile.token(tid);
    find_sequences(d, p.cu, p.start, p.B, p.N, t0, TB, p.err, [](int) { return true; });
    if (tid < TB) {
        int page = -1, row = 0;
        const int b = d.seq[tid];
        if (b >= 0) {
            const long long pos = (long long)d.pos[tid] + (t0 + tid - d.first[tid]);
            if (pos >= 0 && pos < (long long)p.max_pages * p.S) {
                page = p.table[b * p.table_stride + int(pos) / p.S];
                row = int(pos) % p.S;
            }
            if (page < 0 || page >= p.P) {
                page = -1;
                raise_device_error(p.err, kDevCheck);
            }
        }
        d.page[tid] = page;
        d.row[tid] = row;
    }
    __syncthreads();
    const int vec = p.tile.vec(tid), g = vec >> 2, pl = vec & 3;
    const bool here = d.page[tl] >= 0;
    const uint8_t *from = p.pages + (here ? d.page[tl] * p.p_st[0] + (long long)d.row[tl] * q4_row_bytes(p.D) : 0);
    const int at_k = pl * (p.D / 8) + 4 * g;
    const int at_v = p.D / 2 + (2 * pl + (g & 1)) * (p.D / 16) + 2 * (g & ~1), at_s = p.D + 2 * g;
    for (int h0 = 0; h0 < p.Hkv; h0 += U * hl) {
        uint32_t kw[U], vw[U];
        T ks[U], vs[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + p.tile.lane(tid) + u * hl;
            kw[u] = vw[u] = 0;
            if (here && h < p.Hkv) {
                const uint8_t *r = from + h * p.p_st[1];
                kw[u] = *reinterpret_cast<const uint32_t *>(r + at_k);
                vw[u] = *reinterpret_cast<const uint32_t *>(r + at_v);
                ks[u] = *reinterpret_cast<const T *>(r + at_s);
                vs[u] = *reinterpret_cast<const T *>(r + at_s + p.D / 16);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + p.tile.lane(tid) + u * hl;
            // a lane of an even group has read the first four channels of both
            // groups, the lane of the odd one the last four
            const uint32_t o = __shfl_xor_sync(0xffffffffu, vw[u], 4);
            const uint32_t w = g & 1 ? __byte_perm(o, vw[u], 0x7632) : __byte_perm(vw[u], o, 0x5410);
            if (here && h < p.Hkv) {
                Row8<T> r;
                r.u = q4_values<T>(kw[u], ks[u]);
                r.store(static_cast<T *>(p.k) + (t0 + tl) * p.k_st[0] + h * p.k_st[1] + vec * 8);
                r.u = q4_values<T>(w, vs[u]);
                r.store(static_cast<T *>(p.v) + (t0 + tl) * p.v_st[0] + h * p.v_st[1] + vec * 8);
            }
        }
    }
}

Rotation rotation_of(const RotaryArgs &a) {
    return Rotation{a.freq, a.rot, a.interleaved, a.inverse, a.mscale};
}

}  // namespace

attn_status_t rope_rows(const Ctx &c, attn_dtype_t dt, const void *x, void *y, const int32_t *pos,
                        long long pos_stride, int B, int H, int N, int D, const TensorStrides &sx,
                        const TensorStrides &sy, const RotaryArgs &rot) {
    RopeRows p{};
    p.x = x; p.y = y; p.pos = pos; p.pos_stride = pos_stride;
    p.sx = sx; p.sy = sy;
    p.H = H; p.N = N;
    p.tokens = (long long)B * N;
    p.rot = rotation_of(rot);
    // as many tokens per CTA as the heads, cut into slices, leave CTAs enough
    p.tile = make_tile(D, p.tokens, H, 8ll * c.sm_count);
    const long long cols = (p.tokens + p.tile.tokens() - 1) >> p.tile.tb_log;
    int slices = 1;
    while (slices < H && slices < 32768 && cols * slices < 2ll * c.sm_count) slices *= 2;
    p.slice = cdiv(H, slices);
    if (cols > 0x7fffffffll) return ATTN_ERR_UNSUPPORTED;
    const dim3 grid(unsigned(cols), unsigned(cdiv(H, p.slice)));
    if (dt == ATTN_F32) return launch(c, kFamRope, rope_rows_kernel<float>, grid, p);
    if (dt == ATTN_F16) return launch(c, kFamRope, rope_rows_kernel<__half>, grid, p);
    return launch(c, kFamRope, rope_rows_kernel<__nv_bfloat16>, grid, p);
}

attn_status_t append_rows(const Ctx &c, attn_dtype_t dt, const RowsAppend &a) {
    AppendRows p{};
    p.kn = a.kn; p.vn = a.vn; p.q = a.q; p.qo = a.qo;
    p.k = a.k; p.v = a.v;
    for (int i = 0; i < 2; ++i) {
        p.kn_st[i] = a.kn_st[i];
        p.vn_st[i] = a.vn_st[i];
        p.q_st[i] = a.q_st[i];
        p.qo_st[i] = a.qo_st[i];
    }
    for (int i = 0; i < 3; ++i) {
        p.k_st[i] = a.k_st[i];
        p.v_st[i] = a.v_st[i];
    }
    p.table = a.table; p.table_stride = a.table_stride;
    p.seq_len = a.seq_len; p.cu = a.cu;
    p.B = a.B; p.N = a.N; p.Hq = a.q ? a.Hq : 0; p.Hkv = a.Hkv; p.D = a.D;
    p.S = a.S; p.P = a.P; p.max_pages = a.max_pages;
    p.advance = a.advance;
    p.rot = rotation_of(a.rot);
    // (a 4-bit row costs more per token than its angles do)
    p.tile = make_tile(a.D, a.N, a.q4 ? imax(a.Hq, 2 * a.Hkv) : a.Hq + 2 * a.Hkv, (a.q4 ? 2ll : 8ll) * c.sm_count);
    p.err = c.err;
    p.apart = a.q4 && a.q && (a.cu || !a.advance);     // (else a CTA advances the lengths it has read)
    const dim3 grid(unsigned(cdiv(a.N, p.tile.tokens())) * (p.apart ? 2 : 1));
    attn_status_t st;
    if (a.q4)
        st = dt == ATTN_F16 ? launch(c, kFamKvPages, append_rows_kernel<__half, true>, grid, p)
                            : launch(c, kFamKvPages, append_rows_kernel<__nv_bfloat16, true>, grid, p);
    else if (dt == ATTN_F32)
        st = launch(c, kFamKvPages, append_rows_kernel<float, false>, grid, p);
    else
        st = dt == ATTN_F16 ? launch(c, kFamKvPages, append_rows_kernel<__half, false>, grid, p)
                            : launch(c, kFamKvPages, append_rows_kernel<__nv_bfloat16, false>, grid, p);
    if (st != ATTN_OK || !p.cu || !p.advance) return st;
    return launch(c, kFamKvPages, advance_rows_kernel, dim3(unsigned(cdiv(a.B, kThreads / 32))), p);
}

attn_status_t gather_rows(const Ctx &c, attn_dtype_t dt, const RowsGather &a) {
    GatherRows p{};
    p.pages = static_cast<const uint8_t *>(a.pages);
    p.table = a.table; p.table_stride = a.table_stride;
    p.start = a.start; p.cu = a.cu;
    p.k = a.k; p.v = a.v;
    for (int i = 0; i < 2; ++i) {
        p.p_st[i] = a.p_st[i];
        p.k_st[i] = a.k_st[i];
        p.v_st[i] = a.v_st[i];
    }
    p.B = a.B; p.N = a.N; p.Hkv = a.Hkv; p.D = a.D;
    p.S = a.S; p.P = a.P; p.max_pages = a.max_pages;
    p.tile = make_tile(a.D, a.N, 2 * a.Hkv, 2ll * c.sm_count).finer();
    p.err = c.err;
    const dim3 grid(unsigned(cdiv(a.N, p.tile.tokens())));
    return dt == ATTN_F16 ? launch(c, kFamKvPages, gather_rows_kernel<__half>, grid, p)
                          : launch(c, kFamKvPages, gather_rows_kernel<__nv_bfloat16>, grid, p);
}

}  // namespace attn
