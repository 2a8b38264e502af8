// Exact-FFMA causal attention with a sliding window and sinks: the fp32 path of
// attn_causal_gqa_window_fwd (and the 16-bit types at D = 32).
//
// Query i sits at position p = off + i and sees the keys j <= p with
// j > p - window or j < sinks.  One CTA owns 32 query rows of one (batch, head)
// and streams the keys that one of them sees, the sinks and the window, as one
// list in tiles of 64.
//
// Both products are register-tiled: a thread holds 8 rows x 2 keys of S and 8
// rows x D / 32 channels of O and multiplies in pairs (two FMAs an instruction:
// even and odd channels of S, two rows of O), the vectors of the next step read
// ahead.  A warp owns 8 rows, so what it shares (q, P) is read as broadcasts.
// Bound by shared-memory latency and the FMA pipe (3.4 cycles per pair
// instruction and warp, 2 at best) and, for short prompts, by the three or four
// tiles that each CTA goes through one after the other: 32-row tiles give a
// 515-token prompt of 16 heads 272 CTAs (B 2, 8 heads on 2 KV heads, D 64,
// window 128, sinks 4: 15.4 us; 2048 tokens, 8 heads, D 128, window 512: 121 us
// = 31.4 TFLOP/s).  4 rows x 4 keys per thread, scalar FMAs and nothing read
// ahead: 20.6 and 187 us; 4 rows x 2 keys in twice the warps: 17.6 and 146 us;
// one row per thread, as in the entries without a window: 57 and 334 us.
//
// Every product is an fp32 FMA (never TF32), statistics and sums are fp32 and
// the output is rounded once.  A key that a row does not see never enters the
// row's sums, whatever its value holds: on a masked tile that holds an infinite
// or NaN value (noticed when it is loaded) its weight is left out of the P V
// product instead of multiplying by zero.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kBM = 32;      // query rows per CTA
constexpr int kBN = 64;      // keys per tile
constexpr int kThreads = 128;
constexpr int kR = 8;        // query rows per warp

struct WinParams {
    const void *q, *k, *v;
    void *o;
    int Nq, Nkv, off, window, sinks, H, group;
    float qscale;            // scale * log2(e)
    TensorStrides sq, sk, sv, so;
};

template <int D>
struct WinSmem {
    static constexpr int LD = D + 4;                   // floats per row: conflict-free row reads
    static constexpr int LP = kBM + 4;
    static constexpr int Q = 0, K = kBM * LD, V = K + kBN * LD, P = V + kBN * LD;
    static constexpr int BYTES = (P + kBN * LP) * 4;
};

template <typename T> __device__ __forceinline__ float4 load4(const T *p);
template <> __device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}
template <> __device__ __forceinline__ float4 load4<__half>(const __half *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(f16_lo(u.x), f16_hi(u.x), f16_lo(u.y), f16_hi(u.y));
}

// 16 bytes global -> shared without passing registers; src is read only if `take`
// (zeros otherwise).
__device__ __forceinline__ void cp_async16(float *dst, const void *src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(take ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// waits until at most one group of this thread is outstanding
__device__ __forceinline__ void cp_wait1() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// the largest x of a warp (NaN ignored)
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// N consecutive floats of shared memory (the widest load that fits)
template <int N> __device__ __forceinline__ void read(const float *p, float (&x)[N]) {
    if constexpr (N == 1) {
        x[0] = *p;
    } else if constexpr (N == 2) {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        x[0] = v.x;
        x[1] = v.y;
    } else {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
    }
}

// Warp w owns rows 8 w .. 8 w + 7; a lane keys lane and lane + 32 of a tile and
// channels lane CH .. lane CH + CH - 1 of O.  What all lanes read (q, P) costs
// shared memory one cycle a vector, what each reads for itself (k, V) four.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, D == 128 ? 2 : 3) simt_window_kernel(const WinParams p) {
    using S = WinSmem<D>;
    constexpr int CH = D / 32;
    extern __shared__ float sm[];
    float *Qs = sm + S::Q, *Ks = sm + S::K, *Vs = sm + S::V, *Ps = sm + S::P;
    const int tid = threadIdx.x, lane = tid & 31, row0 = (tid >> 5) * kR;
    const int q0 = (gridDim.x - 1 - blockIdx.x) * kBM;
    const long long b = blockIdx.y / p.H, h = blockIdx.y % p.H, hk = h / p.group;
    const T *qg = static_cast<const T *>(p.q) + (b * p.sq.b + h * p.sq.h);
    const T *kg = static_cast<const T *>(p.k) + (b * p.sk.b + hk * p.sk.h);
    const T *vg = static_cast<const T *>(p.v) + (b * p.sv.b + hk * p.sv.h);
    T *og = static_cast<T *>(p.o) + (b * p.so.b + h * p.so.h);

    const int pos0 = p.off + q0;                       // position of the first row
    const int rows = imin(kBM, p.Nq - q0);
    const int end = pos0 + rows;                       // keys past the last row are seen by none
    const int win0 = imax(0, pos0 - p.window + 1);
    const int sink1 = imin(p.sinks, win0);

#pragma unroll
    for (int e = tid; e < kBM * D / 4; e += kThreads) {
        const int r = (e * 4) / D, d = (e * 4) % D;
        const T *src = qg + (r < rows ? (q0 + r) * p.sq.n + d : 0);
        if constexpr (sizeof(T) == 4)
            cp_async16(Qs + r * S::LD + d, src, r < rows);
        else
            *reinterpret_cast<float4 *>(Qs + r * S::LD + d) = r < rows ? load4<T>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
    }

    float acc[kR][CH], m[kR], l[kR];
#pragma unroll
    for (int i = 0; i < kR; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int e = 0; e < CH; ++e) acc[i][e] = 0.f;
    }

    // key u of the list: the sinks before the window, then the window
    const int total = sink1 + end - win0;
    auto key_of = [&](int u) { return u < sink1 ? u : u - sink1 + win0; };
    // One tile of K or V.  fp32 goes to shared memory asynchronously: the next
    // K while this tile's P V runs, the next V while the next S does.
    auto stage = [&](float *dst, const T *base, long long sn, int kb) {
        constexpr int VPR = D / 4, STEP = kThreads / VPR;      // vectors per row, rows per round
        const int r0 = tid / VPR, d = (tid % VPR) * 4;
        float *to = dst + r0 * S::LD + d;
        const T *from = base + d;
#pragma unroll 8
        for (int r = 0; r < kBN; r += STEP) {
            const int u = kb + r0 + r;
            const bool in = u < total;
            const T *src = from + (in ? key_of(u) : 0) * sn;
            if constexpr (sizeof(T) == 4) {
                cp_async16(to + r * S::LD, src, in);
            } else {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (in) x = load4<T>(src);
                *reinterpret_cast<float4 *>(to + r * S::LD) = x;
            }
        }
        cp_commit();
    };
    stage(Ks, kg, p.sk.n, 0);
    stage(Vs, vg, p.sv.n, 0);
    for (int kb = 0; kb < total; kb += kBN) {
        const int keys = imin(kBN, total - kb);
        cp_wait1();                                    // K is here
        __syncthreads();

        // ---- S: kR rows x 2 keys per thread, sums over even and odd channels;
        //      the next step's vectors are read while this one's are multiplied
        float s[kR][2], s2[kR][2][2];
#pragma unroll
        for (int i = 0; i < kR; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) s2[i][c][0] = s2[i][c][1] = 0.f;
        float qn[kR][4], kn[2][4];
        auto read_qk = [&](int d) {
#pragma unroll
            for (int c = 0; c < 2; ++c) read<4>(Ks + (lane + 32 * c) * S::LD + d, kn[c]);
#pragma unroll
            for (int i = 0; i < kR; ++i) read<4>(Qs + (row0 + i) * S::LD + d, qn[i]);
        };
        read_qk(0);
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            float qv[kR][4], kv[2][4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
#pragma unroll
                for (int i = 0; i < kR; ++i) qv[i][x] = qn[i][x];
                kv[0][x] = kn[0][x];
                kv[1][x] = kn[1][x];
            }
            read_qk(d + 4);                            // the last one reads the rows' padding
#pragma unroll
            for (int x = 0; x < 4; x += 2)
#pragma unroll
                for (int i = 0; i < kR; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        ptx::ffma2(s2[i][c][0], s2[i][c][1], qv[i][x], qv[i][x + 1], kv[c][x], kv[c][x + 1],
                                   s2[i][c][0], s2[i][c][1]);
        }

        __syncthreads();                               // K has been read
        if (kb + kBN < total)
            stage(Ks, kg, p.sk.n, kb + kBN);
        else
            cp_commit();
        cp_wait1();                                    // V is here
        const int k_first = key_of(kb), k_last = key_of(kb + keys - 1);
        const bool edge = keys < kBN || k_last > pos0 ||
                          (k_first <= pos0 + kBM - 1 - p.window && k_last >= p.sinks);
        // an infinite or NaN value in a masked tile: 0 x is not 0
        float z0 = 0.f, z1 = 0.f;
        if (edge)
#pragma unroll 4
            for (int e = tid; e < kBN * D / 4; e += kThreads) {
                const float4 v = *reinterpret_cast<const float4 *>(Vs + (e * 4) / D * S::LD + (e * 4) % D);
                ptx::ffma2(z0, z1, v.x, v.y, 0.f, 0.f, z0, z1);
                ptx::ffma2(z0, z1, v.z, v.w, 0.f, 0.f, z0, z1);
            }
        const int wild = __syncthreads_or(z0 + z1 != 0.f);

        // ---- masks (every row sees the whole tile, or it is tested key by key)
        //      and online softmax
        unsigned seen = 0xffffu;                       // bit kR c + i
        if (edge) {
            seen = 0;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int u = lane + 32 * c, key = key_of(kb + u), ahead = key - (pos0 + row0);
#pragma unroll
                for (int i = 0; i < kR; ++i)
                    seen |= unsigned(u < keys && ahead <= i && (ahead > i - p.window || key < p.sinks))
                            << (kR * c + i);
            }
        }
#pragma unroll
        for (int i = 0; i < kR; ++i) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
                s[i][c] = (seen >> (kR * c + i)) & 1u ? (s2[i][c][0] + s2[i][c][1]) * p.qscale : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            const float mn = fmaxf(m[i], warp_max(fmaxf(s[i][0], s[i][1])));
            const float alpha = mn == -INFINITY ? 1.f : ptx::ex2(m[i] - mn);
            m[i] = mn;
            l[i] *= alpha;                             // of this lane's keys; joined at the end
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                // no finite score yet: -inf weighs nothing, NaN stays NaN
                const float w = s[i][c] == -INFINITY ? 0.f : ptx::ex2(s[i][c] - mn);
                l[i] += w;
                s[i][c] = wild && !((seen >> (kR * c + i)) & 1u) ? -1.f : w;
            }
#pragma unroll
            for (int e = 0; e < CH; ++e) acc[i][e] *= alpha;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < kR; i += 4)
                *reinterpret_cast<float4 *>(Ps + (lane + 32 * c) * S::LP + row0 + i) =
                    make_float4(s[i][c], s[i + 1][c], s[i + 2][c], s[i + 3][c]);
        __syncwarp();                                  // a warp reads its own rows of P

        // ---- O += P V, two rows per FFMA2
        if (wild) {
#pragma unroll 1
            for (int c = 0; c < keys; ++c) {
                float v[CH];
                read<CH>(Vs + c * S::LD + lane * CH, v);
#pragma unroll
                for (int i = 0; i < kR; ++i) {
                    const float w = Ps[c * S::LP + row0 + i];
#pragma unroll
                    for (int e = 0; e < CH; ++e)
                        if (!(w < 0.f)) acc[i][e] = fmaf(w, v[e], acc[i][e]);
                }
            }
        } else {
            // NK keys at a time, the next NK read ahead; weights (and V) of
            // keys past the end are zeros
            constexpr int NK = 4;
            float wn[NK][kR], vn[NK][CH];
            auto read_pv = [&](int c) {
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    read<CH>(Vs + (c + k) * S::LD + lane * CH, vn[k]);
#pragma unroll
                    for (int i = 0; i < kR; i += 4) {
                        float x[4];
                        read<4>(Ps + (c + k) * S::LP + row0 + i, x);
#pragma unroll
                        for (int e = 0; e < 4; ++e) wn[k][i + e] = x[e];
                    }
                }
            };
            read_pv(0);
#pragma unroll 2
            for (int c = 0; c < keys; c += NK) {
                float w[NK][kR], v[NK][CH];
#pragma unroll
                for (int k = 0; k < NK; ++k) {
#pragma unroll
                    for (int i = 0; i < kR; ++i) w[k][i] = wn[k][i];
#pragma unroll
                    for (int e = 0; e < CH; ++e) v[k][e] = vn[k][e];
                }
                read_pv(imin(c + NK, kBN - NK));
#pragma unroll
                for (int k = 0; k < NK; ++k)
#pragma unroll
                    for (int e = 0; e < CH; ++e)
#pragma unroll
                        for (int i = 0; i < kR; i += 2)
                            ptx::ffma2(acc[i][e], acc[i + 1][e], w[k][i], w[k][i + 1], v[k][e], v[k][e], acc[i][e],
                                       acc[i + 1][e]);
            }
        }
        __syncthreads();                               // V has been read
        if (kb + kBN < total)
            stage(Vs, vg, p.sv.n, kb + kBN);
        else
            cp_commit();
    }

#pragma unroll
    for (int off = 1; off < 32; off <<= 1)
#pragma unroll
        for (int i = 0; i < kR; ++i) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
        if (row0 + i >= rows) continue;
        const float inv = 1.f / l[i];
        T *orow = og + (q0 + row0 + i) * p.so.n + lane * CH;
        alignas(16) T x[CH];
#pragma unroll
        for (int e = 0; e < CH; ++e) Elem<T>::store(x + e, acc[i][e] * inv);
        if constexpr (CH * sizeof(T) == 16)
            *reinterpret_cast<uint4 *>(orow) = *reinterpret_cast<const uint4 *>(x);
        else if constexpr (CH * sizeof(T) == 8)
            *reinterpret_cast<uint2 *>(orow) = *reinterpret_cast<const uint2 *>(x);
        else if constexpr (CH * sizeof(T) == 4)
            *reinterpret_cast<uint32_t *>(orow) = *reinterpret_cast<const uint32_t *>(x);
        else
            *orow = x[0];
    }
}

template <typename T, int D>
attn_status_t launch_win(const Ctx &c, const WinParams &p, int tiles, int BH) {
    static int done_mask = 0;
    auto kern = simt_window_kernel<T, D>;
    if (!ensure_smem_attr(reinterpret_cast<const void *>(kern), WinSmem<D>::BYTES, c.device, &done_mask))
        return ATTN_ERR_RESOURCE;
    kern<<<dim3(tiles, BH), kThreads, WinSmem<D>::BYTES, c.stream>>>(p);
    return launch_status(kFamSimt);
}

template <typename T>
attn_status_t dispatch_win(const Ctx &c, int D, const WinParams &p, int tiles, int BH) {
    if (D == 32) return launch_win<T, 32>(c, p, tiles, BH);
    if (D == 64) return launch_win<T, 64>(c, p, tiles, BH);
    return launch_win<T, 128>(c, p, tiles, BH);
}

}  // namespace

attn_status_t simt_causal_window(const Ctx &c, attn_dtype_t dt, const void *q, const void *k,
                                 const void *v, void *o, int B, int Hq, int Hkv, int Nq, int Nkv,
                                 int D, int window, int sinks, float scale,
                                 const TensorStrides *st) {
    WinParams p{};
    p.q = q; p.k = k; p.v = v; p.o = o;
    p.Nq = Nq;
    p.Nkv = Nkv;
    p.off = Nkv - Nq;
    p.window = window;
    p.sinks = sinks;
    p.H = Hq;
    p.group = Hq / Hkv;
    p.qscale = scale * kLog2e;
    p.sq = st[0]; p.sk = st[1]; p.sv = st[2]; p.so = st[3];
    const int tiles = cdiv(Nq, kBM);
    if (dt == ATTN_F32) return dispatch_win<float>(c, D, p, tiles, B * Hq);
    if (dt == ATTN_F16) return dispatch_win<__half>(c, D, p, tiles, B * Hq);
    return dispatch_win<__nv_bfloat16>(c, D, p, tiles, B * Hq);
}

}  // namespace attn
