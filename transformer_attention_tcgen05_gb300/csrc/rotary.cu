// Rotary positions: rows of any tensor (attn_rope_fwd), and of the new tokens on
// their way into a paged cache, 16-bit / fp32 or held in 4 bits, with the reader
// that gives a 4-bit cache's rows back.
//
// All of it is bound by memory: 16 or 32 bytes per thread and load, several loads
// in flight.  A thread keeps its token and channels and walks the heads, so the
// angles of a (token, pair) are computed once for all heads where there are
// tokens enough to fill the GPU; a short call spreads its heads over the threads
// of a CTA instead and computes them several times over.  A thread reads its
// partners' channels beside its own (a second read of a line that is in L1),
// so no row passes through shared memory, and a row may be rotated in place: the
// lanes of one warp own it, and all of them read before any writes.
#include <math.h>

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

// How a CTA's threads are laid over a tile: D / 8 lanes per row, 2^tb_log tokens,
// the rest over heads.
struct Tile {
    int vpr_log, tb_log;
    __host__ __device__ int vec(int t) const { return t & ((1 << vpr_log) - 1); }
    __host__ __device__ int token(int t) const { return (t >> vpr_log) & ((1 << tb_log) - 1); }
    __host__ __device__ int lane(int t) const { return t >> (vpr_log + tb_log); }
    __host__ __device__ int lanes() const { return kThreads >> (vpr_log + tb_log); }
    __host__ __device__ int tokens() const { return 1 << tb_log; }
};

// The most tokens per CTA (fewest angles computed) that leave `want` CTAs.
Tile make_tile(int D, long long tokens, long long want) {
    Tile t;
    t.vpr_log = D == 128 ? 4 : D == 64 ? 3 : 2;
    t.tb_log = 8 - t.vpr_log;
    while (t.tb_log > 0 && (tokens >> t.tb_log) < want) --t.tb_log;
    return t;
}

// -------------------------------------------------------------------- rope

struct RopeRows {
    const void *x;
    void *y;
    const int32_t *pos;
    long long pos_stride;                              // between batches
    TensorStrides sx, sy;
    int H, N, D, slice;                                // slice: heads per CTA
    long long tokens;                                  // B * N
    Rotation rot;
    Tile tile;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) rope_rows_kernel(const RopeRows p) {
    constexpr int U = sizeof(T) == 4 ? 2 : 4;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x, c0 = p.tile.vec(tid) * 8, hl = p.tile.lanes();
    const long long t = ((long long)blockIdx.x << p.tile.tb_log) + p.tile.token(tid);
    const bool here = t < p.tokens, turns = c0 < p.rot.rot;
    const long long b = here ? t / p.N : 0, n = here ? t % p.N : 0;
    const int h_end = imin(p.H, (blockIdx.y + 1) * p.slice);
    const T *x = static_cast<const T *>(p.x) + b * p.sx.b + n * p.sx.n;
    T *y = static_cast<T *>(p.y) + b * p.sy.b + n * p.sy.n + c0;
    const bool inter = p.rot.interleaved;
    Turn tr;
    bool ready = false;
#pragma unroll 1
    for (int h0 = blockIdx.y * p.slice; h0 < h_end; h0 += U * hl) {
        Row8<T> own[U], other[U];
        const int h = h0 + p.tile.lane(tid);
        if (!ready)
            tr.partner = inter ? c0 : c0 < p.rot.rot / 2 ? c0 + p.rot.rot / 2 : c0 - p.rot.rot / 2;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (here && h + u * hl < h_end) {
                own[u].load(x + (h + u * hl) * p.sx.h + c0);
                if (turns && !inter) other[u].load(x + (h + u * hl) * p.sx.h + tr.partner);
            }
        if (!ready && turns && here) make_turn(p.rot, p.pos[b * p.pos_stride + n], c0, tr);
        ready = true;
        __syncwarp();                                  // the row has been read by all its lanes
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (here && h + u * hl < h_end) {
                if (turns) {
                    float z[8];
                    rotate8<T>(tr, own[u], other[u], inter, z);
                    own[u].set(z);
                }
                own[u].store(y + (h + u * hl) * p.sy.h);
            }
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
    Rotation rot;
    Tile tile;
    unsigned *err;
};

// Where a tile's tokens go.
struct Dest {
    int seq[64], first[64], count[64];                 // sequence (-1: none), its first row and rows
    int pos[64];                                       // position (-1: the request does not fit)
    int page[64], row[64];                             // page -1: none
};

// Sequence, first row and row count of the tile's tokens [t0, t0 + n), from the
// starts cu[0..B] of the packed sequences.
__device__ __forceinline__ void find_sequences(Dest &d, const int32_t *cu, int B, int N, int t0, int n,
                                               unsigned *err) {
    if (threadIdx.x < 64) d.seq[threadIdx.x] = -1;
    __syncthreads();
    for (int b = threadIdx.x; b < B; b += kThreads) {
        const int lo = cu[b], hi = cu[b + 1];
        if (lo < 0 || hi < lo || hi > N) {
            if (blockIdx.x == 0) raise_device_error(err, kDevCheck);
            continue;
        }
        for (int t = imax(lo, t0); t < imin(hi, t0 + n); ++t) {
            d.seq[t - t0] = b;
            d.first[t - t0] = lo;
            d.count[t - t0] = hi - lo;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ bool append_fits(const AppendRows &p, int len, int n) {
    return len >= 0 && (long long)len + n <= (long long)p.max_pages * p.S;
}

template <typename T, bool Q4>
__global__ void __launch_bounds__(kThreads) append_rows_kernel(const AppendRows p) {
    constexpr int U = sizeof(T) == 4 ? 2 : 4;
    __shared__ Dest d;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x, TB = p.tile.tokens(), hl = p.tile.lanes();
    const int t0 = blockIdx.x * TB, tl = p.tile.token(tid), t = t0 + tl;
    const int vec = p.tile.vec(tid), c0 = vec * 8;
    const bool in = t < p.N, turns = c0 < p.rot.rot, inter = p.rot.interleaved;
    const int other_c = inter ? c0 : c0 < p.rot.rot / 2 ? c0 + p.rot.rot / 2 : c0 - p.rot.rot / 2;
    const int heads = p.Hq + 2 * p.Hkv;                // of q, then K, then V
    // the first rows are read while their places are looked up
    Row8<T> own[U], other[U];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * hl;
            if (!in || h >= heads) continue;
            const T *src;
            if (h < p.Hq)
                src = static_cast<const T *>(p.q) + t * p.q_st[0] + h * p.q_st[1];
            else if (h < p.Hq + p.Hkv)
                src = static_cast<const T *>(p.kn) + t * p.kn_st[0] + (h - p.Hq) * p.kn_st[1];
            else
                src = static_cast<const T *>(p.vn) + t * p.vn_st[0] + (h - p.Hq - p.Hkv) * p.vn_st[1];
            own[u].load(src + c0);
            if (turns && !inter && h < p.Hq + p.Hkv) other[u].load(src + other_c);
        }
    };
    load(p.tile.lane(tid));
    if (p.cu) {
        find_sequences(d, p.cu, p.B, p.N, t0, TB, p.err);
    } else if (tid < TB) {
        d.seq[tid] = t0 + tid < p.N ? t0 + tid : -1;
        d.first[tid] = t0 + tid;
        d.count[tid] = 1;
    }
    if (tid < TB) {
        int pos = -1, page = -1, row = 0;
        const int b = d.seq[tid];
        if (b >= 0) {
            const int len = p.seq_len[b];
            if (append_fits(p, len, d.count[tid])) {
                pos = len + t0 + tid - d.first[tid];
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
    const int pos = d.pos[tl], page = d.page[tl], row = d.row[tl];
    const bool known = in && pos >= 0, stored = in && page >= 0;
    Turn tr;
    if (turns && known) make_turn(p.rot, pos, c0, tr);
    for (int h0 = 0; h0 < heads; h0 += U * hl) {
        const int hb = h0 + p.tile.lane(tid);
        if (h0 > 0) load(hb);
        __syncwarp();                                  // the rows have been read by all their lanes
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = hb + u * hl;
            const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
            const int hk = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
            float z[8];
            if (known && h < heads && turns && !is_v) {
                rotate8<T>(tr, own[u], other[u], inter, z);
                if (!Q4 || is_q) own[u].set(z);
            } else if (Q4) {
                own[u].get(z);
            }
            if (is_q && known && h < heads)
                own[u].store(static_cast<T *>(p.qo) + t * p.qo_st[0] + h * p.qo_st[1] + c0);
            if constexpr (!Q4) {
                if (!is_q && stored && h < heads)
                    own[u].store(static_cast<T *>(is_v ? p.v : p.k) + page * (is_v ? p.v_st[0] : p.k_st[0]) +
                                 hk * (is_v ? p.v_st[1] : p.k_st[1]) + row * (is_v ? p.v_st[2] : p.k_st[2]) + c0);
            } else if (__any_sync(0xffffffffu, !is_q && h < heads)) {
                float inv;
                const T s = q4_scale<T>(z, inv);
                const uint32_t w = q4_codes(z, inv);
                // V: this lane's words of two neighbouring groups, one of its own and one
                // of the lane of the other group (which holds the same four channels)
                const int g = vec >> 2, pl = vec & 3;
                const uint32_t o = __shfl_xor_sync(0xffffffffu, w, 4);
                if (!is_q && stored && h < heads) {
                    uint8_t *to = static_cast<uint8_t *>(p.k) + page * p.k_st[0] + hk * p.k_st[1] + row * p.k_st[2];
                    if (!is_v)
                        *reinterpret_cast<uint32_t *>(to + pl * (p.D / 8) + 4 * g) = w;
                    else if (g & 1)
                        *reinterpret_cast<uint32_t *>(to + p.D / 2 + (2 * pl + 1) * (p.D / 16) + 2 * (g - 1)) =
                            (o >> 16) | (w & 0xffff0000u);
                    else
                        *reinterpret_cast<uint32_t *>(to + p.D / 2 + 2 * pl * (p.D / 16) + 2 * g) =
                            (w & 0xffffu) | (o << 16);
                    if (pl == 0)
                        *reinterpret_cast<T *>(to + p.D + (is_v ? p.D / 16 : 0) + 2 * g) = s;
                }
            }
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
    if (!ok && n == 0 && lane == 0) raise_device_error(p.err, kDevCheck);
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
    constexpr int U = 4;
    __shared__ Dest d;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x, TB = p.tile.tokens(), hl = p.tile.lanes();
    const int t0 = blockIdx.x * TB, tl = p.tile.token(tid);
    find_sequences(d, p.cu, p.B, p.N, t0, TB, p.err);
    if (tid < TB) {
        int page = -1, row = 0;
        const int b = d.seq[tid];
        if (b >= 0) {
            const long long pos = (long long)(p.start ? p.start[b] : 0) + (t0 + tid - d.first[tid]);
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
            const uint32_t w = g & 1 ? (o >> 16) | (vw[u] & 0xffff0000u) : (vw[u] & 0xffffu) | (o << 16);
            if (here && h < p.Hkv) {
                float z[8];
                Row8<T> r;
                q4_values(kw[u], Elem<T>::load(&ks[u]), z);
                r.set(z);
                r.store(static_cast<T *>(p.k) + (t0 + tl) * p.k_st[0] + h * p.k_st[1] + vec * 8);
                q4_values(w, Elem<T>::load(&vs[u]), z);
                r.set(z);
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
    p.H = H; p.N = N; p.D = D;
    p.tokens = (long long)B * N;
    p.rot = rotation_of(rot);
    // as many tokens per CTA as the heads, cut into slices, leave CTAs enough
    p.tile = make_tile(D, p.tokens * H, 4ll * c.sm_count);
    const long long cols = (p.tokens + p.tile.tokens() - 1) >> p.tile.tb_log;
    int slices = 1;
    while (slices < H && slices < 32768 && cols * slices < 8ll * c.sm_count) slices *= 2;
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
    p.tile = make_tile(a.D, a.N, 2ll * c.sm_count);
    p.err = c.err;
    const dim3 grid(unsigned(cdiv(a.N, p.tile.tokens())));
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
    p.tile = make_tile(a.D, a.N, 2ll * c.sm_count);
    p.err = c.err;
    const dim3 grid(unsigned(cdiv(a.N, p.tile.tokens())));
    return dt == ATTN_F16 ? launch(c, kFamKvPages, gather_rows_kernel<__half>, grid, p)
                          : launch(c, kFamKvPages, gather_rows_kernel<__nv_bfloat16>, grid, p);
}

// theta_i as 64-bit fractions of a turn.  double has 53 bits: the error at
// position t is t 2^-55 of a turn.
attn_status_t rope_frequencies(uint64_t *freq, int rot, double theta, attn_rope_scaling_t scaling, double factor,
                               double original_len, double alpha, double beta) {
    constexpr double two_pi = 6.283185307179586476925;
    for (int i = 0; i < rot / 2; ++i) {
        const double e = 2.0 * i / rot;
        double f = pow(theta, -e);
        if (scaling == ATTN_ROPE_LINEAR) {
            f /= factor;
        } else if (scaling == ATTN_ROPE_NTK) {
            f = pow(theta * pow(factor, double(rot) / (rot - 2)), -e);
        } else if (scaling == ATTN_ROPE_BY_PARTS) {
            const double turns = original_len * f / two_pi;
            const double share = fmin(1.0, fmax(0.0, (turns - alpha) / (beta - alpha)));
            f = (1.0 - share) * f / factor + share * f;
        }
        f = f / two_pi;
        if (!(f < 0.5)) return ATTN_ERR_INVALID_ARG;   // half a turn per position, or NaN
        freq[i] = uint64_t(ldexp(f, 64) + 0.5);
    }
    return ATTN_OK;
}

}  // namespace attn
