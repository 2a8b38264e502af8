// Exact-FFMA causal attention with a sliding window and sinks: the fp32 path of
// attn_causal_gqa_window_fwd (and the 16-bit types at D = 32).
//
// Query i sits at position p = off + i and sees the keys j <= p with
// j > p - window or j < sinks.  One CTA owns 32 query rows of one (batch, head)
// and streams the keys that one of them sees, the sinks and the window, as one
// list in tiles of 64.
//
// Both products are register-tiled: a thread holds 4 rows x 4 keys of S and 4
// rows x D / 16 channels of O, so that 8 shared-memory vectors feed 64 FMAs
// (S) and 2 feed 16 (P V); the one-row-per-thread kernel that the unwindowed
// entries use reads one vector per 4 FMAs and has a quarter of the warps.
// Bound by the FMA pipe and, for short prompts, by latency: 32-row tiles give a
// 515-token prompt of 16 heads 272 CTAs (B 2, 8 heads on 2 KV heads, D 64,
// window 128, sinks 4: 21.8 us, 57 us in the one-row-per-thread form; 2048
// tokens, 8 heads, D 128, window 512: 188 us = 20.2 TFLOP/s, was 334 us).
// Sinks and window as two runs of tiles cost one tile more (27.9 us), synchronous
// copies 22.9 us.
//
// Every product is an fp32 FMA (never TF32), statistics and sums are fp32 and
// the output is rounded once.  A key that a row does not see never enters the
// row's sums, whatever its value holds: on a masked tile that holds an infinite
// or NaN value (noticed when it is loaded) its weight is left out of the P V
// product instead of multiplying by zero.
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace attn {
namespace {

constexpr int kBM = 32;      // query rows per CTA
constexpr int kBN = 64;      // keys per tile
constexpr int kThreads = 128;

struct WinParams {
    const void *q, *k, *v;
    void *o;
    int Nq, Nkv, off, window, sinks, H, group;
    float qscale;            // scale * log2(e), folded into q
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
template <> __device__ __forceinline__ float4 load4<float>(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
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

// Thread (ty, tx) = (tid / 16, tid % 16): rows 4 ty + i, keys tx + 16 c,
// channels tx * D / 16 + e.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) simt_window_kernel(const WinParams p) {
    using S = WinSmem<D>;
    constexpr int CH = D / 16;
    extern __shared__ float sm[];
    float *Qs = sm + S::Q, *Ks = sm + S::K, *Vs = sm + S::V, *Ps = sm + S::P;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
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

    for (int e = tid; e < kBM * D / 4; e += kThreads) {
        const int r = (e * 4) / D, d = (e * 4) % D;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) x = load4<T>(qg + (q0 + r) * p.sq.n + d);
        x.x *= p.qscale;
        x.y *= p.qscale;
        x.z *= p.qscale;
        x.w *= p.qscale;
        *reinterpret_cast<float4 *>(Qs + r * S::LD + d) = x;
    }

    float acc[4][CH], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
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
        const int keys = imin(kBN, total - kb);
#pragma unroll 4
        for (int e = tid; e < kBN * D / 4; e += kThreads) {
            const int r = (e * 4) / D, d = (e * 4) % D;
            const bool in = r < keys;
            const T *src = base + (in ? key_of(kb + r) * sn + d : 0);
            if constexpr (sizeof(T) == 4) {
                cp_async16(dst + r * S::LD + d, src, in);
            } else {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (in) x = load4<T>(src);
                *reinterpret_cast<float4 *>(dst + r * S::LD + d) = x;
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

        // ---- S: 4 rows x 4 keys per thread
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[i][c] = 0.f;
#pragma unroll 4
        for (int d = 0; d < D; d += 4) {
            float4 qv[4], kv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4 *>(Qs + (4 * ty + i) * S::LD + d);
#pragma unroll
            for (int c = 0; c < 4; ++c) kv[c] = *reinterpret_cast<const float4 *>(Ks + (tx + 16 * c) * S::LD + d);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    s[i][c] = fmaf(qv[i].x, kv[c].x, s[i][c]);
                    s[i][c] = fmaf(qv[i].y, kv[c].y, s[i][c]);
                    s[i][c] = fmaf(qv[i].z, kv[c].z, s[i][c]);
                    s[i][c] = fmaf(qv[i].w, kv[c].w, s[i][c]);
                }
        }

        __syncthreads();                               // K has been read
        if (kb + kBN < total)
            stage(Ks, kg, p.sk.n, kb + kBN);
        else
            cp_commit();
        cp_wait1();                                    // V is here
        int wild = 0;                                  // an infinite or NaN value in the tile
#pragma unroll 4
        for (int e = tid; e < kBN * D / 4; e += kThreads) {
            const float4 v = *reinterpret_cast<const float4 *>(Vs + (e * 4) / D * S::LD + (e * 4) % D);
            wild |= !(fabsf(v.x) < INFINITY && fabsf(v.y) < INFINITY && fabsf(v.z) < INFINITY &&
                      fabsf(v.w) < INFINITY);
        }
        wild = __syncthreads_or(wild);

        // ---- masks (every row sees the whole tile, or it is tested key by key)
        //      and online softmax
        const int k_first = key_of(kb), k_last = key_of(kb + keys - 1);
        const bool edge = keys < kBN || k_last > pos0 ||
                          (k_first <= pos0 + kBM - 1 - p.window && k_last >= p.sinks);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int pos = pos0 + 4 * ty + i;
            unsigned seen = 0xfu;
            if (edge) {
                seen = 0;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int u = tx + 16 * c, key = key_of(kb + u);
                    const bool ok = u < keys && key <= pos && (key > pos - p.window || key < p.sinks);
                    seen |= unsigned(ok) << c;
                    if (!ok) s[i][c] = -INFINITY;
                }
            }
            float mx = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float mn = fmaxf(m[i], mx);
            const float alpha = mn == -INFINITY ? 1.f : exp2f(m[i] - mn);
            m[i] = mn;
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const bool ok = (seen >> c) & 1u;
                // no finite score yet: -inf weighs nothing, NaN stays NaN
                const float w = mn == -INFINITY && s[i][c] == -INFINITY ? 0.f : exp2f(s[i][c] - mn);
                if (ok) sum += w;
                s[i][c] = ok ? w : (wild ? -1.f : 0.f);
            }
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l[i] = l[i] * alpha + sum;
#pragma unroll
            for (int e = 0; e < CH; ++e) acc[i][e] *= alpha;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<float4 *>(Ps + (tx + 16 * c) * S::LP + 4 * ty) =
                make_float4(s[0][c], s[1][c], s[2][c], s[3][c]);
        // rows 4 ty .. 4 ty + 3 of P are written and read by the same half warp
        __syncwarp();

        // ---- O += P V
        if (edge && wild) {
#pragma unroll 1
            for (int c = 0; c < keys; ++c) {
                const float4 w = *reinterpret_cast<const float4 *>(Ps + c * S::LP + 4 * ty);
                const float wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < CH; ++e) {
                    const float v = Vs[c * S::LD + tx * CH + e];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!(wv[i] < 0.f)) acc[i][e] = fmaf(wv[i], v, acc[i][e]);
                }
            }
        } else {
#pragma unroll 4
            for (int c = 0; c < keys; ++c) {
                const float4 w = *reinterpret_cast<const float4 *>(Ps + c * S::LP + 4 * ty);
                float v[CH];
                if constexpr (CH == 2) {
                    const float2 x = *reinterpret_cast<const float2 *>(Vs + c * S::LD + tx * 2);
                    v[0] = x.x;
                    v[1] = x.y;
                } else {
#pragma unroll
                    for (int e = 0; e < CH; e += 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(Vs + c * S::LD + tx * CH + e);
                        v[e] = x.x;
                        v[e + 1] = x.y;
                        v[e + 2] = x.z;
                        v[e + 3] = x.w;
                    }
                }
#pragma unroll
                for (int e = 0; e < CH; ++e) {
                    acc[0][e] = fmaf(w.x, v[e], acc[0][e]);
                    acc[1][e] = fmaf(w.y, v[e], acc[1][e]);
                    acc[2][e] = fmaf(w.z, v[e], acc[2][e]);
                    acc[3][e] = fmaf(w.w, v[e], acc[3][e]);
                }
            }
        }
        __syncthreads();                               // V has been read
        if (kb + kBN < total)
            stage(Vs, vg, p.sv.n, kb + kBN);
        else
            cp_commit();
    }

#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (r >= rows) continue;
        const float inv = 1.f / l[i];
        T *orow = og + (q0 + r) * p.so.n + tx * CH;
#pragma unroll
        for (int e = 0; e < CH; ++e) Elem<T>::store(orow + e, acc[i][e] * inv);
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
