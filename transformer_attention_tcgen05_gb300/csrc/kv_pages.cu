// The pages of a paged KV cache: appending rows, and the allocator (reserve,
// free, fork, compact) with the page copies it asks for.
//
// The allocator's whole state is on the device: page_table [B][max_pages]
// (-1: no page) and page_refs [P], the number of table entries that name a
// page (0: free).  The lowest free page is always taken first and requests are
// served in (row, entry) order, so the result of a call depends on its inputs
// alone, never on the order in which threads or atomics run, and a captured
// graph can allocate.  Nothing here is read back by the host.
//
// These calls move a few kilobytes of tables, so they are bound by latency,
// not bandwidth: a call that has to number its requests (reserve, fork,
// compact) is one CTA, or for a large pool one cluster of 8, whose barriers and
// distributed shared memory replace a grid-wide scan in several launches.  An append and a page
// copy move cache rows and are bound by HBM: 16-byte vectors, several in
// flight per thread.
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

// Launches with the programmatic-dependent attribute: the kernel may start
// while the one before it finishes, and waits for it (griddep_wait) before its
// first global access.
template <typename... P, typename... A>
attn_status_t launch_pdl(const Ctx &c, void (*kern)(P...), dim3 grid, int threads, int cluster,
                         size_t smem, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, P(args)...) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_CUDA;
    }
    return launch_status(kFamKvPages);
}

// ------------------------------------------------------------------ append

struct AppendParams {
    uint8_t *k, *v;
    const uint8_t *kn, *vn;
    const int32_t *table;
    int32_t *seq_len;
    const int32_t *new_len;
    int T, Hkv, S, P, max_pages;
    long long table_stride;
    long long k_st[3], v_st[3], kn_st[3], vn_st[3];   // bytes
    int vpr_log;                                      // log2 of the 16-byte vectors per row
    int tiles;                                        // token tiles per sequence
    int advance;
    unsigned *err;
};

// Rows the call appends to sequence b at position `len`, or -1 if the request
// does not fit the table.
__device__ __forceinline__ int append_count(const AppendParams &p, int b, int len) {
    const int n = p.new_len ? p.new_len[b] : p.T;
    if (len < 0 || n < 0 || n > p.T || (long long)len + n > (long long)p.max_pages * p.S) return -1;
    return n;
}

// One CTA copies a tile of TB tokens (all KV heads, K and V) of one sequence.
// ONE: a single tile per sequence; the CTA that wrote it advances the length.
template <int TB, bool ONE>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    __shared__ long long s_k[TB], s_v[TB];             // byte offset of a token's row of head 0, -1: none
    __shared__ int s_bad;
    const int b = blockIdx.x / p.tiles, t0 = (blockIdx.x % p.tiles) * TB;
    const int len = p.seq_len[b];
    const int n = append_count(p, b, len);
    if (n < 0) {
        if (threadIdx.x == 0 && t0 == 0) raise_device_error(p.err, kDevCheck);
        return;
    }
    if (t0 >= n) return;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    const int nt = imin(TB, n - t0);
    if (threadIdx.x < TB) {
        long long ok = -1, ov = -1;
        if (int(threadIdx.x) < nt) {
            const int pos = len + t0 + threadIdx.x;
            const int page = p.table[b * p.table_stride + pos / p.S], row = pos % p.S;
            if (page >= 0 && page < p.P) {
                ok = page * p.k_st[0] + row * p.k_st[2];
                ov = page * p.v_st[0] + row * p.v_st[2];
            } else {
                raise_device_error(p.err, kDevCheck);
                s_bad = 1;
            }
        }
        s_k[threadIdx.x] = ok;
        s_v[threadIdx.x] = ov;
    }
    __syncthreads();
    // vector e of the tile: column e % VPR of token (e / VPR) % TB of head e / (VPR TB)
    const int vpr = 1 << p.vpr_log, total = (TB * p.Hkv) << p.vpr_log;
    const uint8_t *kn = p.kn + b * p.kn_st[0] + (long long)t0 * p.kn_st[2];
    const uint8_t *vn = p.vn + b * p.vn_st[0] + (long long)t0 * p.vn_st[2];
    constexpr int U = 4;
    for (int e0 = threadIdx.x; e0 < total; e0 += U * 256) {
        uint4 xk[U], xv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + u * 256;
            const int c = e & (vpr - 1), t = (e >> p.vpr_log) % TB, h = (e >> p.vpr_log) / TB;
            if (e < total && s_k[t] >= 0) {
                xk[u] = *reinterpret_cast<const uint4 *>(kn + h * p.kn_st[1] + t * p.kn_st[2] + c * 16);
                xv[u] = *reinterpret_cast<const uint4 *>(vn + h * p.vn_st[1] + t * p.vn_st[2] + c * 16);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = e0 + u * 256;
            const int c = e & (vpr - 1), t = (e >> p.vpr_log) % TB, h = (e >> p.vpr_log) / TB;
            if (e < total && s_k[t] >= 0) {
                *reinterpret_cast<uint4 *>(p.k + s_k[t] + h * p.k_st[1] + c * 16) = xk[u];
                *reinterpret_cast<uint4 *>(p.v + s_v[t] + h * p.v_st[1] + c * 16) = xv[u];
            }
        }
    }
    if (ONE && p.advance && threadIdx.x == 0 && !s_bad) p.seq_len[b] = len + n;
}

// Advances the lengths after a tiled append (every tile has read them by now):
// one warp per sequence, which stays where it was if one of its pages was bad.
__global__ void __launch_bounds__(128) advance_kernel(const AppendParams p, int B) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int b = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (b >= B) return;
    const int len = p.seq_len[b];
    const int n = append_count(p, b, len);
    if (n <= 0) return;
    bool ok = true;
    for (int i = len / p.S + lane; i <= (len + n - 1) / p.S; i += 32) {
        const int page = p.table[b * p.table_stride + i];
        ok = ok && page >= 0 && page < p.P;
    }
    if (__all_sync(0xffffffffu, ok) && lane == 0) p.seq_len[b] = len + n;
}

// -------------------------------------------------------------------- copy

struct CopyParams {
    uint8_t *k, *v;
    const int32_t *src, *dst, *count;
    int n, P;
    int vecs;                                          // 16-byte vectors of a page side
    int pieces;                                        // pieces of kPiece vectors per page side
    int sides, two;                                    // layers * 2; two: K and V are arrays of their own
    int vpr, S;                                        // vectors per row, rows per head
    long long k_st[4], v_st[4];                        // bytes (layer, page, head, token)
    unsigned *err;
};

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kPiece = kCopyThreads * kCopyUnroll;     // 16 KB

// A persistent grid walks the pieces (16 KB of one page of one layer's K or V)
// of all pairs.  DENSE: a page is one contiguous block.
template <bool DENSE>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyParams p) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int n = p.count ? imax(0, imin(*p.count, p.n)) : p.n;
    const int per_pair = p.sides * p.pieces;
    const long long total = (long long)n * per_pair;
    for (long long it = blockIdx.x; it < total; it += gridDim.x) {
        const int pair = int(it / per_pair), rest = int(it % per_pair);
        const int side = rest / p.pieces, piece = rest % p.pieces;
        const int s = p.src[pair], d = p.dst[pair];
        if (s == -1 && d == -1) continue;
        if (s < 0 || s >= p.P || d < 0 || d >= p.P) {
            if (rest == 0 && threadIdx.x == 0) raise_device_error(p.err, kDevCheck);
            continue;
        }
        if (s == d) continue;
        const bool is_v = side & p.two;
        uint8_t *base = (is_v ? p.v : p.k) + (side >> p.two) * (is_v ? p.v_st[0] : p.k_st[0]);
        const long long pst = is_v ? p.v_st[1] : p.k_st[1];
        const uint8_t *from = base + s * pst;
        uint8_t *to = base + d * pst;
        uint4 x[kCopyUnroll];
        long long off[kCopyUnroll];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u) {
            const int e = piece * kPiece + u * kCopyThreads + threadIdx.x;
            if (DENSE) {
                off[u] = (long long)e * 16;
            } else {
                const int row = e / p.vpr;
                off[u] = (row / p.S) * (is_v ? p.v_st[2] : p.k_st[2]) +
                         (row % p.S) * (is_v ? p.v_st[3] : p.k_st[3]) + (e % p.vpr) * 16;
            }
            if (e < p.vecs) x[u] = *reinterpret_cast<const uint4 *>(from + off[u]);
        }
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (piece * kPiece + u * kCopyThreads + int(threadIdx.x) < p.vecs)
                *reinterpret_cast<uint4 *>(to + off[u]) = x[u];
    }
}

// --------------------------------------------------------------- allocator


constexpr int kClu = 8;                                // CTAs of a large call's cluster
constexpr int kAT = 1024;                              // threads per CTA
constexpr int kMaxRows = 16384;                        // rows of a table (shared-memory prefix)
constexpr int kMaxForks = 8192;

struct AllocShared {
    int warp[3][32];
    int val[8];                                        // one word per cluster exchange
    int chunk[2][32], base[2][32];                     // pages of the warps' chunks, pages before them
    int got[3][kClu];                                  // the CTAs' words of an exchange
};

// Exclusive prefix of x over the CTA's threads; *total: the CTA's sum.
__device__ __forceinline__ int block_scan(AllocShared &sh, int x, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += up;
    }
    if (lane == 31) sh.warp[0][warp] = inc;
    __syncthreads();
    const int s = sh.warp[0][lane];
    int ws = s;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, ws, off);
        if (lane >= off) ws += up;
    }
    __syncthreads();
    *total = __shfl_sync(0xffffffffu, ws, 31);
    return __shfl_sync(0xffffffffu, ws - s, warp) + inc - x;
}

// Sums of three words over the CTA.
__device__ __forceinline__ void block_sum3(AllocShared &sh, int &x, int &y, int &z) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    x = __reduce_add_sync(0xffffffffu, x);
    y = __reduce_add_sync(0xffffffffu, y);
    z = __reduce_add_sync(0xffffffffu, z);
    if (lane == 0) {
        sh.warp[0][warp] = x;
        sh.warp[1][warp] = y;
        sh.warp[2][warp] = z;
    }
    __syncthreads();
    x = __reduce_add_sync(0xffffffffu, sh.warp[0][lane]);
    y = __reduce_add_sync(0xffffffffu, sh.warp[1][lane]);
    z = __reduce_add_sync(0xffffffffu, sh.warp[2][lane]);
    __syncthreads();
}

// Cluster barrier (arrive / wait are warp-collective); orders global and
// distributed shared memory between the CTAs.  A small call is one CTA.
__device__ __forceinline__ void cluster_barrier() {
    if (gridDim.x == 1) {
        __syncthreads();
    } else {
        __syncwarp();
        ptx::cluster_sync();
    }
}

// Publishes one word per CTA; after the cluster barrier that follows,
// cluster_gather returns the sum over the lower ranks and over all.
__device__ __forceinline__ void cluster_put(AllocShared &sh, int word, int x) {
    if (threadIdx.x == 0) sh.val[word] = x;
}
__device__ __forceinline__ int cluster_gather(AllocShared &sh, int word, int *total) {
    const int rank = blockIdx.x, ranks = gridDim.x, lane = threadIdx.x & 31;
    const uint32_t a = ptx::smem_addr(&sh.val[word]);
    int x = 0;
    if (lane < ranks)
        x = ranks == 1 ? sh.val[word] : __float_as_int(ptx::ld_cluster_f32(ptx::cluster_map(a, lane)));
    __syncwarp();
    *total = __reduce_add_sync(0xffffffffu, x);
    return __reduce_add_sync(0xffffffffu, lane < rank ? x : 0);
}

struct AllocParams {
    int32_t *table;
    long long stride;
    int B, M, P, S;
    int32_t *seq_len;
    const int32_t *add;
    int32_t *refs;
    const int32_t *src, *dst;
    int n;
    int32_t *copy_src, *copy_dst, *count;
    int32_t *new_refs, *new_table;
    long long new_stride;
    int32_t *ws;                                       // [P]
    int quads;                                         // 16-byte reads of a chunk's counts per lane
    unsigned *err;
};

// This CTA's share [i0, i1) of n items.
__device__ __forceinline__ void share(int n, int *i0, int *i1) {
    const long long per = ((long long)n + gridDim.x - 1) / gridDim.x;
    *i0 = int(per * blockIdx.x < n ? per * blockIdx.x : n);
    *i1 = int(*i0 + per < n ? *i0 + per : n);
}

// The pool is looked at in chunks of 128 `quads` pages, one per warp and dealt
// out over the CTAs in turn (the lowest pages are taken first: contiguous shares
// would leave that to one CTA), a bit per page: bits 4 k .. 4 k + 3 of a lane are
// pages 4 lane .. 4 lane + 3 of the chunk's k-th 128.  A pool of one span (up to
// 32,768 pages per CTA) is read once; the bits stay in a register from the count
// to the hand-out.
__device__ __forceinline__ int span(const AllocParams &p) { return int(gridDim.x) * (kAT / 32) * 128 * p.quads; }

__device__ __forceinline__ int quad_page(const AllocParams &p, int at, int k) {
    const int chunk = int(threadIdx.x >> 5) * int(gridDim.x) + int(blockIdx.x);
    return at + (chunk * p.quads + k) * 128 + int(threadIdx.x & 31) * 4;
}

// Bits of this lane's pages below `limit`.
__device__ __forceinline__ unsigned below(const AllocParams &p, int at, int limit) {
    unsigned m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int n = k < p.quads ? imax(0, imin(4, limit - quad_page(p, at, k))) : 0;
        m |= ((1u << n) - 1u) << (4 * k);
    }
    return m;
}

// Bits of this lane's pages whose count is positive (ANY: not zero).
template <bool ANY = false>
__device__ __forceinline__ unsigned live_bits(const AllocParams &p, int at) {
    int4 r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int i = quad_page(p, at, k);
        r[k] = make_int4(0, 0, 0, 0);
        if (k >= p.quads) continue;
        if (i + 4 <= p.P) {
            r[k] = *reinterpret_cast<const int4 *>(p.refs + i);
        } else if (i < p.P) {
            r[k].x = p.refs[i];
            if (i + 1 < p.P) r[k].y = p.refs[i + 1];
            if (i + 2 < p.P) r[k].z = p.refs[i + 2];
        }
    }
    auto on = [](int n) { return ANY ? n != 0 : n > 0; };
    unsigned m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        m |= (unsigned(on(r[k].x)) | unsigned(on(r[k].y)) << 1 | unsigned(on(r[k].z)) << 2 |
              unsigned(on(r[k].w)) << 3) << (4 * k);
    return m;
}

// Bits of this lane's free pages.
__device__ __forceinline__ unsigned free_bits(const AllocParams &p, int at) {
    return ~live_bits<true>(p, at) & below(p, at, p.P);
}

// Pages (bits) of this warp's chunk, for all to see after a cluster barrier.  Two
// counts may be under way at once, in different slots.
__device__ __forceinline__ void put_chunk(AllocShared &sh, int slot, unsigned bits) {
    const int n = __reduce_add_sync(0xffffffffu, __popc(bits));
    if ((threadIdx.x & 31) == 0) sh.chunk[slot][threadIdx.x >> 5] = n;
}
// Pages in the chunks before this warp's; *total: in all chunks.  Ends with a
// cluster barrier.
__device__ __forceinline__ int chunk_base(AllocShared &sh, int slot, int *total) {
    const int ranks = gridDim.x, t = threadIdx.x;
    int x = 0;
    if (t < 32 * ranks) {
        const int *word = &sh.chunk[slot][t / ranks];
        x = ranks == 1 ? *word
                       : __float_as_int(ptx::ld_cluster_f32(ptx::cluster_map(ptx::smem_addr(word), t % ranks)));
    }
    const int pre = block_scan(sh, x, total);
    if (t < 32 * ranks && t % ranks == int(blockIdx.x)) sh.base[slot][t / ranks] = pre;
    cluster_barrier();                                 // chunk has been read everywhere
    return sh.base[slot][t >> 5];
}

// Calls f(page, number) for the pages of this lane's bits, numbered in page
// order over the chunk from `base` on.
template <typename F>
__device__ __forceinline__ void each_page(const AllocParams &p, unsigned bits, int at, int base, F f) {
    // per k the pages of the lower lanes: a prefix over the lanes of 8 counts,
    // at most 128 each, a byte apiece (k even, k odd)
    unsigned x = bits - ((bits >> 1) & 0x55555555u);
    x = (x & 0x33333333u) + ((x >> 2) & 0x33333333u);
    const unsigned c[2] = {x & 0x0f0f0f0fu, (x >> 4) & 0x0f0f0f0fu};
    unsigned inc[2] = {c[0], c[1]};
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned up0 = __shfl_up_sync(0xffffffffu, inc[0], off), up1 = __shfl_up_sync(0xffffffffu, inc[1], off);
        if (int(threadIdx.x & 31) >= off) {
            inc[0] += up0;
            inc[1] += up1;
        }
    }
    const unsigned tot[2] = {__shfl_sync(0xffffffffu, inc[0], 31), __shfl_sync(0xffffffffu, inc[1], 31)};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (k >= p.quads) break;
        const int sh = 8 * (k >> 1), page = quad_page(p, at, k);
        const unsigned q = bits >> (4 * k);
        int n = base + int(((inc[k & 1] - c[k & 1]) >> sh) & 0xffu);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if ((q >> j) & 1u) f(page + j, n++);
        base += int((tot[k & 1] >> sh) & 0xffu);
    }
}

// This lane's free pages, and their bits if the pool is one span.
__device__ __forceinline__ int count_free(const AllocParams &p, unsigned *bits) {
    int n = 0;
    for (int at = 0; at < p.P; at += span(p)) {
        *bits = free_bits(p, at);
        n += __popc(*bits);
    }
    return n;
}

// One exchange of all that the CTAs have to know of each other: each gives three
// words (put before in val[0 .. 2]) and its chunks' free pages (slot 0).  One
// barrier and one round of remote reads, about 1.1 us at 8 CTAs; a word at a time
// cost 0.5 us each.  sum: the words' sums; *before: word 0 of the lower CTAs.
__device__ __forceinline__ int exchange(AllocShared &sh, int (&sum)[3], int *before) {
    const int ranks = gridDim.x, t = threadIdx.x, w = t / ranks, r = t % ranks;
    cluster_barrier();
    int x = 0;
    if (w < 35) {
        const int *word = w < 32 ? &sh.chunk[0][w] : &sh.val[w - 32];
        x = ranks == 1 ? *word : __float_as_int(ptx::ld_cluster_f32(ptx::cluster_map(ptx::smem_addr(word), r)));
        if (w >= 32) {
            sh.got[w - 32][r] = x;
            x = 0;
        }
    }
    int all;
    const int pre = block_scan(sh, x, &all);
    if (w < 32 && r == int(blockIdx.x)) sh.base[0][w] = pre;
    __syncthreads();
    sum[0] = sum[1] = sum[2] = *before = 0;
    for (int i = 0; i < ranks; ++i) {
        if (i < int(blockIdx.x)) *before += sh.got[0][i];
        sum[0] += sh.got[0][i];
        sum[1] += sh.got[1][i];
        sum[2] += sh.got[2][i];
    }
    return sh.base[0][t >> 5];
}

// Takes the `need` lowest free pages: list[i] = page, refs[page] = 1.  bits, base:
// from count_free and the exchange behind it.
__device__ __forceinline__ void take_free(const AllocParams &p, AllocShared &sh, int need, unsigned bits,
                                          int base) {
    int taken = 0;
    for (int at = 0; at < p.P && taken < need; at += span(p)) {   // the same in every CTA
        int all = need;
        if (p.P > span(p)) {
            bits = free_bits(p, at);
            cluster_barrier();                         // the slot has been read
            put_chunk(sh, 0, bits);
            cluster_barrier();
            base = taken + chunk_base(sh, 0, &all);
        }
        if (base < need)
            each_page(p, bits, at, base, [&](int page, int k) {
                if (k < need) {
                    p.ws[k] = page;
                    p.refs[page] = 1;
                }
            });
        taken += all;
    }
}

// *to += x if `take`; what it was (1 if not).  Predicated: the call's atomics go
// out together (as branches each was waited for, 8 x 0.5 us).
__device__ __forceinline__ int add_if(bool take, int32_t *to, int x) {
    int was;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %3, 0;\n\tmov.s32 %0, 1;\n\t"
        "@p atom.global.add.s32 %0, [%1], %2;\n\t}"
        : "=&r"(was)
        : "l"(to), "r"(x), "r"(int(take))
        : "memory");
    return was;
}

// Reserve: entry i of row b is needed if it covers a position of
// [seq_len[b], seq_len[b] + add[b]) and holds no page yet.  The entries that
// the rows ask about, one after the other, are numbered by a prefix over the
// rows and dealt out evenly over the threads, however long the rows are.
__global__ void __launch_bounds__(kAT, 1) reserve_kernel(const AllocParams p) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    __shared__ AllocShared sh;
    extern __shared__ int dyn[];
    int *const pre = dyn, *const e0 = dyn + p.B + 1;   // entries before row b; its first entry
    unsigned bits = 0;
    int my_free = count_free(p, &bits);
    int bad = 0, ask = 0;
    for (int b0 = 0; b0 < p.B; b0 += kAT) {
        const int b = b0 + threadIdx.x;
        int n = 0, first = 0;
        if (b < p.B) {
            const int len = p.seq_len[b], add = p.add[b];
            if (len < 0 || add < 0 || (long long)len + add > (long long)p.M * p.S) {
                bad = 1;
            } else if (add > 0) {
                first = len / p.S;
                n = (len + add - 1) / p.S + 1 - first;
            }
        }
        int all;
        const int at = ask + block_scan(sh, n, &all);
        if (b < p.B) {
            pre[b] = at;
            e0[b] = first;
        }
        ask += all;
    }
    if (threadIdx.x == 0) pre[p.B] = ask;
    __syncthreads();
    // the table entry of number x: the last row whose entries start at or before it
    auto entry = [&](int x) -> int32_t * {
        int lo = 0, hi = p.B;                          // pre[lo] <= x < pre[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= x)
                lo = mid;
            else
                hi = mid;
        }
        return p.table + lo * p.stride + e0[lo] + (x - pre[lo]);
    };
    int x0, x1;
    share(ask, &x0, &x1);
    int need = 0;
    if (x1 - x0 <= kAT) {
        if (x0 + int(threadIdx.x) < x1) need = *entry(x0 + threadIdx.x) < 0;
    } else {
        for (int x = x0 + threadIdx.x; x < x1; x += kAT) need += *entry(x) < 0;
    }
    const int mine = need;
    put_chunk(sh, 0, bits);
    block_sum3(sh, need, bad, my_free);
    cluster_put(sh, 0, need);
    cluster_put(sh, 1, bad);
    cluster_put(sh, 2, my_free);
    int sum[3], base;
    const int free0 = exchange(sh, sum, &base);
    const bool refuse = sum[1] > 0 || sum[0] > sum[2]; // the same in every CTA
    if (!refuse) take_free(p, sh, sum[0], bits, free0);
    cluster_barrier();                                 // the list is complete; no CTA left early
    if (refuse) {
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_device_error(p.err, kDevCheck);
        return;
    }
    for (int x = x0; x < x1; x += kAT) {
        int32_t *e = nullptr;
        int n = 0;
        if (x + int(threadIdx.x) < x1) {
            e = entry(x + threadIdx.x);
            n = x1 - x0 <= kAT ? mine : *e < 0;
        }
        int all;
        const int k = base + block_scan(sh, n, &all);
        if (n) *e = p.ws[k];
        base += all;
    }
}

// Free: an entry whose page holds no visible token of its row lets go of it.
__global__ void __launch_bounds__(256) free_kernel(const AllocParams p, int blocks, int window,
                                                   int sinks) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int b = blockIdx.x / blocks, j0 = (blockIdx.x % blocks) * 1024;
    const int len = p.seq_len[b];
    if (len < 0 || len > (long long)p.M * p.S) {
        if (threadIdx.x == 0 && j0 == 0) raise_device_error(p.err, kDevCheck);
        return;
    }
    const int lo = window > 0 && len > window ? len - window : 0;
    const int s_end = imin(sinks, len);
    int32_t *row = p.table + b * p.stride;
    int page[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int i = j0 + u * 256 + threadIdx.x;
        page[u] = i < p.M ? row[i] : -1;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int i = j0 + u * 256 + threadIdx.x;
        if (page[u] == -1) continue;
        const long long at = (long long)i * p.S;
        if (at < len && (at + p.S > lo || at < s_end)) continue;
        if (page[u] < 0 || page[u] >= p.P) {
            raise_device_error(p.err, kDevCheck);
            continue;
        }
        if (atomicSub(&p.refs[page[u]], 1) <= 0) {     // not counted: the entry stays
            atomicAdd(&p.refs[page[u]], 1);
            raise_device_error(p.err, kDevCheck);
            continue;
        }
        row[i] = -1;
    }
}

// Fork: row dst[i] becomes a copy of row src[i].  Full pages are shared; a last
// page that is partly filled gets a page of its own and a copy order.
__global__ void __launch_bounds__(kAT, 1) fork_kernel(const AllocParams p) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    __shared__ AllocShared sh;
    extern __shared__ int dyn[];
    int *const s_src = dyn, *const s_dst = dyn + p.n, *const s_len = dyn + 2 * p.n;
    int *const s_tail = dyn + 3 * p.n, *const s_rank = dyn + 4 * p.n;       // last page, its number
    unsigned *const is_dst = reinterpret_cast<unsigned *>(dyn + 5 * p.n);   // one bit per row
    const int rank = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    // ---- the lists: rows in range, no row twice a target, none target and source
    int bad = 0, zero = 0, wrong = 0;
    for (int i = threadIdx.x; i < (p.B + 31) / 32; i += kAT) is_dst[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < p.n; i += kAT) {
        const int s = p.src[i], d = p.dst[i];
        int len = 0, tail = -1;
        if (s < 0 || s >= p.B || d < 0 || d >= p.B) {
            bad = 1;
        } else {
            if (atomicOr(&is_dst[d >> 5], 1u << (d & 31)) >> (d & 31) & 1u) bad = 1;
            len = p.seq_len[s];
            if (len < 0 || len > (long long)p.M * p.S) {
                bad = 1;
            } else if (len % p.S != 0) {
                // a partly filled last page, to be copied from
                tail = p.table[s * p.stride + len / p.S];
                if (tail < -1 || tail >= p.P) bad = 1;
            }
        }
        s_tail[i] = tail;
        s_src[i] = s;
        s_dst[i] = d;
        s_len[i] = len;
    }
    __syncthreads();
    if (!bad)
        for (int i = threadIdx.x; i < p.n; i += kAT) {
            const int s = s_src[i];
            if (s >= 0 && s < p.B && (is_dst[s >> 5] >> (s & 31) & 1u)) bad = 1;
        }
    block_sum3(sh, bad, zero, wrong);                  // the same in every CTA
    // ---- counts: the targets' old pages are let go, and what is left is looked
    //      at: a page that a source names must still be counted, or it would be
    //      handed out.  An entry that is no counted page makes the call fail; the
    //      counts are put back then.  No count rises before all have fallen, so
    //      the verdict does not depend on which CTA is first.
    //      Work item: 128 entries of one fork, a warp each.
    const int blocks = cdiv(p.M, 128);
    const long long items = (long long)p.n * blocks;
    const int w0 = warp * int(gridDim.x) + rank, wn = int(gridDim.x) * (kAT / 32);
    auto let_go = [&](int sign) {
        for (long long it = w0; it < items; it += wn) {
            const int f = int(it / blocks), j0 = int(it % blocks) * 128;
            const int32_t *rd = p.table + s_dst[f] * p.stride;
            int old[4], was[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = j0 + u * 32 + lane;
                old[u] = j < p.M ? rd[j] : -1;
            }
            // the counts change together; what they were is looked at behind
#pragma unroll
            for (int u = 0; u < 4; ++u) was[u] = add_if(old[u] >= 0 && old[u] < p.P, p.refs + old[u], -sign);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (old[u] < -1 || old[u] >= p.P || (sign > 0 && was[u] <= 0)) wrong = 1;
        }
    };
    if (!bad) let_go(1);
    int tails = 0;                                     // last pages to copy, numbered in list order
    for (int b0 = 0; b0 < p.n && !bad; b0 += kAT) {
        const int f = b0 + threadIdx.x;
        const int t = f < p.n && s_tail[f] >= 0;
        int all;
        const int k = tails + block_scan(sh, t, &all);
        if (f < p.n) s_rank[f] = k;
        tails += all;
    }
    cluster_barrier();                                 // every page is let go
    for (long long it = w0; it < items && !bad; it += wn) {
        const int f = int(it / blocks), j0 = int(it % blocks) * 128;
        const int32_t *rs = p.table + s_src[f] * p.stride;
        const int full = s_len[f] / p.S;
        int e[4], n[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + u * 32 + lane;
            e[u] = j < full ? rs[j] : j == full ? s_tail[f] : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) n[u] = e[u] >= 0 && e[u] < p.P ? p.refs[e[u]] : 1;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (e[u] < -1 || e[u] >= p.P || n[u] <= 0) wrong = 1;
    }
    unsigned bits = 0;
    int my_free = bad ? 0 : count_free(p, &bits);
    put_chunk(sh, 0, bits);
    block_sum3(sh, my_free, wrong, zero);
    cluster_put(sh, 0, 0);
    cluster_put(sh, 1, wrong + bad);
    cluster_put(sh, 2, my_free);
    int sum[3], none;
    const int free0 = exchange(sh, sum, &none);
    const bool refuse = sum[1] || tails > sum[2];      // the same in every CTA
    if (refuse) {
        if (!bad) let_go(-1);                          // nothing has changed but the counts
    } else {
        take_free(p, sh, tails, bits, free0);
    }
    cluster_barrier();
    if (refuse) {
        for (int i = rank * kAT + threadIdx.x; i < p.n; i += int(gridDim.x) * kAT)
            p.copy_src[i] = p.copy_dst[i] = -1;
        if (rank == 0 && threadIdx.x == 0) raise_device_error(p.err, kDevCheck);
        return;
    }
    // ---- the rows
    for (long long it = w0; it < items; it += wn) {
        const int f = int(it / blocks), j0 = int(it % blocks) * 128;
        const int32_t *rs = p.table + s_src[f] * p.stride;
        int32_t *rd = p.table + s_dst[f] * p.stride;
        const int full = s_len[f] / p.S;
        int e[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + u * 32 + lane;
            e[u] = j < full ? rs[j] : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + u * 32 + lane;
            if (e[u] >= 0) atomicAdd(&p.refs[e[u]], 1);     // a shared full page
            if (j >= p.M) continue;
            if (j == full) {                           // the last page, or the first entry behind it
                if (s_tail[f] >= 0) e[u] = p.ws[s_rank[f]];
                p.copy_src[f] = s_tail[f];
                p.copy_dst[f] = e[u];
            }
            rd[j] = e[u];
        }
        if (j0 == 0 && lane == 0) {
            p.seq_len[s_dst[f]] = s_len[f];
            if (full == p.M) p.copy_src[f] = p.copy_dst[f] = -1;   // no entry behind a full table
        }
    }
}

// A table entry behind a compaction (the map is complete).
__device__ __forceinline__ int moved(const AllocParams &p, int e) {
    if (e == -1) return -1;
    const int to = e >= 0 && e < p.P ? p.ws[e] : -1;
    if (to < 0) raise_device_error(p.err, kDevCheck);
    return to;
}

// Compact: with L live pages, the k-th live page at or above L moves to the
// k-th free page below L.  Lists the moves, fills the map old -> new (ws[page],
// -1 for a page that is not live) and writes the new counts, and the new table
// too if it is short (TABLE).
template <bool TABLE>
__global__ void __launch_bounds__(kAT, 1) compact_kernel(const AllocParams p) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    __shared__ AllocShared sh;
    const int cap = p.P / 2;
    int live = 0, one = 0, zero = 0;
    unsigned bits = 0;                                 // of one span
    for (int at = 0; at < p.P; at += span(p)) {
        bits = live_bits(p, at);
        live += __popc(bits);
    }
    block_sum3(sh, live, zero, one);
    cluster_put(sh, 0, live);
    cluster_barrier();
    int L, moves = 0, holes = 0;
    cluster_gather(sh, 0, &L);
    for (int at = 0; at < p.P; at += span(p)) {
        if (p.P > span(p)) bits = live_bits(p, at);
        // live pages at or above L (movers), free ones below (holes)
        const unsigned low = below(p, at, L), mov = bits & ~low, hole = ~bits & low;
        put_chunk(sh, 0, mov);
        put_chunk(sh, 1, hole);
        cluster_barrier();
        int n_m, n_h;
        const int bm = moves + chunk_base(sh, 0, &n_m), bh = holes + chunk_base(sh, 1, &n_h);
        each_page(p, mov, at, bm, [&](int page, int k) { p.copy_src[k] = page; });
        each_page(p, hole, at, bh, [&](int page, int k) { p.copy_dst[k] = page; });
        // the map: a live page stays (a mover's new place is filled in below); an
        // entry that names no live page is wrong
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k >= p.quads) break;
            const int i = quad_page(p, at, k);
            const unsigned q = bits >> (4 * k);
            const int4 to = make_int4(q & 1u ? i : -1, q & 2u ? i + 1 : -1, q & 4u ? i + 2 : -1, q & 8u ? i + 3 : -1);
            if (i + 4 <= p.P) {
                *reinterpret_cast<int4 *>(p.ws + i) = to;
            } else if (i < p.P) {
                p.ws[i] = to.x;
                if (i + 1 < p.P) p.ws[i + 1] = to.y;
                if (i + 2 < p.P) p.ws[i + 2] = to.z;
            }
        }
        moves += n_m;
        holes += n_h;
    }
    cluster_barrier();
    const int t = blockIdx.x * kAT + threadIdx.x, step = int(gridDim.x) * kAT;
    for (int k = t; k < cap; k += step) {
        if (k < moves) {
            const int s = p.copy_src[k], d = p.copy_dst[k];
            p.ws[s] = d;
            p.new_refs[d] = p.refs[s];
        } else {
            p.copy_src[k] = p.copy_dst[k] = -1;
        }
    }
    if (t == 0) {
        *p.count = moves;
    }
    cluster_barrier();                                 // the movers' counts have been read
    for (int i = t; i < p.P; i += step) {
        if (i >= L)
            p.new_refs[i] = 0;
        else if (p.refs[i] > 0)
            p.new_refs[i] = p.refs[i];
    }
    if (TABLE) {
        constexpr int U = 2;                           // entries per thread
        const int n = p.B * p.M;
        for (int x0 = t; x0 < n; x0 += U * step) {
            int e[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int x = x0 + u * step;
                e[u] = x < n ? p.table[x / p.M * p.stride + x % p.M] : -1;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int x = x0 + u * step;
                e[u] = moved(p, e[u]);
                if (x < n) p.new_table[x / p.M * p.new_stride + x % p.M] = e[u];
            }
        }
    }
}

// The table of a large call.
__global__ void __launch_bounds__(256) remap_kernel(const AllocParams p, int blocks) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int b = blockIdx.x / blocks, j0 = (blockIdx.x % blocks) * 1024;
    int e[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int i = j0 + u * 256 + threadIdx.x;
        e[u] = i < p.M ? p.table[b * p.stride + i] : -1;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int i = j0 + u * 256 + threadIdx.x;
        if (i < p.M) p.new_table[b * p.new_stride + i] = moved(p, e[u]);
    }
}

AllocParams alloc_params(const Ctx &c, const PageTable &t) {
    AllocParams p{};
    p.table = t.table;
    p.stride = t.stride;
    p.B = t.B; p.M = t.max_pages; p.P = t.P; p.S = t.S;
    p.err = c.err;
    return p;
}

// CTAs of a call that scans n words: one CTA reads 16,384 in about the time of
// the cluster barriers that a larger call needs.
int cluster_size(long long n) { return n <= 16384 ? 1 : kClu; }

// Chunks as short as the pool allows, so that every warp has one.
int chunk_quads(int P, int ctas) { return imax(1, imin(8, cdiv(P, ctas * (kAT / 32) * 128))); }

// A page is one block if its rows follow one another in either order.
// st: element strides (head, token).
bool dense_page(const long long *st, int Hkv, int S, int D) {
    const long long h = st[0], t = st[1];
    return (t == D && (Hkv == 1 || h == (long long)S * D)) ||
           (h == D && t == (long long)Hkv * D);
}

}  // namespace

attn_status_t kv_append_paged(const Ctx &c, attn_dtype_t dt, const PagedAppend &a) {
    const int es = dt == ATTN_F32 ? 4 : 2;
    AppendParams p{};
    p.k = static_cast<uint8_t *>(a.k);
    p.v = static_cast<uint8_t *>(a.v);
    p.kn = static_cast<const uint8_t *>(a.kn);
    p.vn = static_cast<const uint8_t *>(a.vn);
    p.table = a.table;
    p.seq_len = a.seq_len;
    p.new_len = a.new_len;
    p.T = a.T; p.Hkv = a.Hkv; p.S = a.S; p.P = a.P; p.max_pages = a.max_pages;
    p.table_stride = a.table_stride;
    for (int i = 0; i < 3; ++i) {
        p.k_st[i] = a.k_st[i] * es;
        p.v_st[i] = a.v_st[i] * es;
        p.kn_st[i] = a.kn_st[i] * es;
        p.vn_st[i] = a.vn_st[i] * es;
    }
    for (int vpr = a.D * es / 16; vpr > 1; vpr >>= 1) ++p.vpr_log;
    p.advance = a.advance;
    p.err = c.err;
    if (a.T == 1) {
        p.tiles = 1;
        return launch_pdl(c, append_kernel<1, true>, dim3(a.B), 256, 1, 0, p);
    }
    constexpr int TB = 16;
    p.tiles = cdiv(a.T, TB);
    if ((long long)a.B * p.tiles > 0x7fffffffll) return ATTN_ERR_UNSUPPORTED;
    if (p.tiles == 1) return launch_pdl(c, append_kernel<TB, true>, dim3(a.B), 256, 1, 0, p);
    const attn_status_t st = launch_pdl(c, append_kernel<TB, false>, dim3(a.B * p.tiles), 256, 1, 0, p);
    if (st != ATTN_OK || !a.advance) return st;
    return launch_pdl(c, advance_kernel, dim3(cdiv(a.B, 4)), 128, 1, 0, p, a.B);
}

attn_status_t kv_pages_copy(const Ctx &c, attn_dtype_t dt, const PagesCopy &a) {
    const int es = dt == ATTN_F32 ? 4 : 2;
    CopyParams p{};
    p.k = static_cast<uint8_t *>(a.k);
    p.v = static_cast<uint8_t *>(a.v);
    p.src = a.src; p.dst = a.dst; p.count = a.count;
    p.n = a.n; p.P = a.P;
    p.vpr = a.D * es / 16;
    p.S = a.S;
    p.vecs = a.Hkv * a.S * p.vpr;
    p.pieces = cdiv(p.vecs, kPiece);
    p.sides = 2 * a.layers;
    p.two = 1;
    for (int i = 0; i < 4; ++i) {
        p.k_st[i] = a.k_st[i] * es;
        p.v_st[i] = a.v_st[i] * es;
    }
    p.err = c.err;
    const long long items = (long long)a.n * p.sides * p.pieces;
    const int grid = int(items < 8ll * c.sm_count ? items : 8ll * c.sm_count);
    const bool dense = dense_page(a.k_st + 2, a.Hkv, a.S, a.D) && dense_page(a.v_st + 2, a.Hkv, a.S, a.D);
    return dense ? launch_pdl(c, copy_kernel<true>, dim3(grid), kCopyThreads, 1, 0, p)
                 : launch_pdl(c, copy_kernel<false>, dim3(grid), kCopyThreads, 1, 0, p);
}

// A (page, head) of a cache held in 4 bits is one block of bytes: one row of the
// copy above, in one array.
attn_status_t kv_pages_copy_q4(const Ctx &c, const PagesCopyQ4 &a) {
    CopyParams p{};
    p.k = p.v = static_cast<uint8_t *>(a.pages);
    p.src = a.src; p.dst = a.dst; p.count = a.count;
    p.n = a.n; p.P = a.P;
    p.vpr = int(a.block / 16);
    p.S = 1;
    p.vecs = a.Hkv * p.vpr;
    p.pieces = cdiv(p.vecs, kPiece);
    p.sides = a.layers;
    for (int i = 0; i < 3; ++i) p.k_st[i] = p.v_st[i] = a.st[i];
    p.err = c.err;
    const long long items = (long long)a.n * p.sides * p.pieces;
    const int grid = int(items < 8ll * c.sm_count ? items : 8ll * c.sm_count);
    return a.Hkv == 1 || a.st[2] == a.block ? launch_pdl(c, copy_kernel<true>, dim3(grid), kCopyThreads, 1, 0, p)
                                            : launch_pdl(c, copy_kernel<false>, dim3(grid), kCopyThreads, 1, 0, p);
}

size_t kv_pages_workspace_bytes(int P) { return (size_t(P) * 4 + 255) & ~size_t(255); }

attn_status_t kv_pages_reserve(const Ctx &c, const PageTable &t, const int32_t *seq_len,
                               const int32_t *add, int32_t *refs, void *ws) {
    AllocParams p = alloc_params(c, t);
    p.seq_len = const_cast<int32_t *>(seq_len);        // read only
    p.add = add;
    p.refs = refs;
    p.ws = static_cast<int32_t *>(ws);
    if (t.B > kMaxRows) return ATTN_ERR_UNSUPPORTED;
    static int done_mask = 0;
    if (!ensure_smem_attr(reinterpret_cast<const void *>(reserve_kernel), (2 * kMaxRows + 1) * 4, c.device,
                          &done_mask))
        return ATTN_ERR_RESOURCE;
    const int ctas = cluster_size(t.P);
    p.quads = chunk_quads(t.P, ctas);
    return launch_pdl(c, reserve_kernel, dim3(ctas), kAT, ctas, size_t(2 * t.B + 1) * 4, p);
}

attn_status_t kv_pages_free(const Ctx &c, const PageTable &t, const int32_t *seq_len, int32_t *refs,
                            int window, int sinks) {
    AllocParams p = alloc_params(c, t);
    p.seq_len = const_cast<int32_t *>(seq_len);        // read only
    p.refs = refs;
    const int blocks = cdiv(t.max_pages, 1024);
    if ((long long)t.B * blocks > 0x7fffffffll) return ATTN_ERR_UNSUPPORTED;
    return launch_pdl(c, free_kernel, dim3(t.B * blocks), 256, 1, 0, p, blocks, window, sinks);
}

attn_status_t kv_pages_fork(const Ctx &c, const PageTable &t, int32_t *seq_len, int32_t *refs,
                            const int32_t *src, const int32_t *dst, int n, int32_t *copy_src,
                            int32_t *copy_dst, void *ws) {
    AllocParams p = alloc_params(c, t);
    p.seq_len = seq_len;
    p.refs = refs;
    p.src = src; p.dst = dst; p.n = n;
    p.copy_src = copy_src; p.copy_dst = copy_dst;
    p.ws = static_cast<int32_t *>(ws);
    if (t.B > kMaxRows || n > kMaxForks) return ATTN_ERR_UNSUPPORTED;
    static int done_mask = 0;
    if (!ensure_smem_attr(reinterpret_cast<const void *>(fork_kernel), 5 * kMaxForks * 4 + kMaxRows / 8, c.device,
                          &done_mask))
        return ATTN_ERR_RESOURCE;
    // an entry is read three times and costs two atomics on the counts (16 rows of
    // 254 entries: 12.4 us in one CTA, 9.8 in eight; 21 of 52: 9.4 and 9.5)
    const int ctas = cluster_size(8ll * n * t.max_pages + t.P);
    p.quads = chunk_quads(t.P, ctas);
    return launch_pdl(c, fork_kernel, dim3(ctas), kAT, ctas, size_t(5 * n + cdiv(t.B, 32)) * 4, p);
}

attn_status_t kv_pages_compact(const Ctx &c, const PageTable &t, const int32_t *refs,
                               int32_t *new_table, long long new_stride, int32_t *new_refs,
                               int32_t *copy_src, int32_t *copy_dst, int32_t *count, void *ws) {
    AllocParams p = alloc_params(c, t);
    p.refs = const_cast<int32_t *>(refs);              // written only where new_refs is the same array
    p.new_refs = new_refs;
    p.copy_src = copy_src; p.copy_dst = copy_dst; p.count = count;
    p.ws = static_cast<int32_t *>(ws);
    const int blocks = cdiv(t.max_pages, 1024);
    if ((long long)t.B * blocks > 0x7fffffffll) return ATTN_ERR_UNSUPPORTED;
    const int ctas = cluster_size(t.P);
    p.quads = chunk_quads(t.P, ctas);
    p.new_table = new_table;
    p.new_stride = new_stride;
    // a table of up to 2 entries per thread saves a launch (host side of a call
    // 7.2 -> 5.5 us); with 8 each the launch is faster (72.3 against 75.5 us with
    // the copy of 1440 pages)
    if ((long long)t.B * t.max_pages <= 2ll * kAT * ctas)
        return launch_pdl(c, compact_kernel<true>, dim3(ctas), kAT, ctas, 0, p);
    const attn_status_t st = launch_pdl(c, compact_kernel<false>, dim3(ctas), kAT, ctas, 0, p);
    if (st != ATTN_OK) return st;
    return launch_pdl(c, remap_kernel, dim3(t.B * blocks), 256, 1, 0, p, blocks);
}

}  // namespace attn
