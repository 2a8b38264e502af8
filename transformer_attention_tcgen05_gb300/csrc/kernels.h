// Host-side launchers of libattn's kernels (internal; the public ABI is include/libattn.h).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "libattn.h"

namespace attn {

struct Ctx {
    cudaStream_t stream;
    unsigned *err;      // device error word of the current device
    int device;
    int sm_count;
};

enum KernelFamily : int {
    kFamSimt = 0,
    kFamTcFlash = 1,
    kFamDecode = 2,
    kFamRope = 3,
    kFamNaStarts = 4,
    kFamTcNa = 5,
    kFamKvAppend = 6,
    kFamDebug = 7,
    kFamDecodePaged = 8,
    kFamKvPages = 9,
    kFamCount = 10,
};

void count_launch(int family);

// The per-device context (stream, device error word, SM count) of a call.
attn_status_t context_for(void *stream, Ctx *c);

// Converts the result of a launch into a status (and counts it on success).
attn_status_t launch_status(int family);

// Sets the dynamic shared-memory limit of `func` once per device.
bool ensure_smem_attr(const void *func, size_t bytes, int device, int *done_mask);

// 16-bit (bf16 or f16) TMA tensor map with 128-byte swizzle; dims and box
// innermost first (dims[0] = D), the tensor packed.  False if the driver's
// encoder is unavailable or rejects the map.
bool make_tmap(CUtensorMap *m, const void *base, int rank, const uint64_t *dims, const uint32_t *box,
               bool f16 = false);
bool tma_encode_available();
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();   // nullptr if the driver has none

// Element strides of a [B, heads, N, D] tensor with D contiguous.
struct TensorStrides {
    long long b, h, n;
};

// 4D map {D, N, heads, B} over such a tensor; 128-byte swizzle, box {64, 128, 1, 1}.
bool make_tmap4(CUtensorMap *m, const void *base, int D, int N, int heads, int B,
                const TensorStrides &st, bool f16);

// fp32 / generic SIMT flash attention (exact FFMA for fp32 storage).
attn_status_t simt_full(const Ctx &c, attn_dtype_t dt, const void *q, const void *k,
                        const void *v, void *o, int B, int H, int Nq, int Nkv, int D,
                        float scale, const TensorStrides *st = nullptr);
attn_status_t simt_na3d(const Ctx &c, attn_dtype_t dt, const void *q, const void *k,
                        const void *v, void *o, int B, int H, int T, int Hg, int W, int D,
                        const int kernel[3], float scale, const TensorStrides *st = nullptr);
attn_status_t na_starts(const Ctx &c, int T, int Hg, int W, const int kernel[3],
                        int32_t *starts);

// RoPE prologue: rotated copies of q and k into qr / kr (same dtype).
attn_status_t rope_rotate_qk(const Ctx &c, attn_dtype_t dt, const void *q, const void *k,
                             void *qr, void *kr, int BH, int N, int D, const int32_t *pos,
                             const int axes_dim[4], float theta);

// KV-cache append at the device-side position seq_len[b] (optionally advancing it);
// ring: the cache keeps the last Lmax tokens, token t in row t % Lmax.
attn_status_t kv_append(const Ctx &c, attn_dtype_t dt, void *kc, void *vc, const void *kn,
                        const void *vn, int32_t *seq_len, int B, int Hkv, int Lmax, int D,
                        int advance, bool ring = false);

// Split-KV GQA decode (bf16 or f16 cache).
size_t decode_workspace_bytes(int B, int Hq, int Hkv, int Lmax, int D);
attn_status_t decode_gqa(const Ctx &c, attn_dtype_t dt, const void *q, const void *k,
                         const void *v, const int32_t *seq_len, void *o, int B, int Hq, int Hkv,
                         int Lmax, int D, float scale, void *ws, size_t ws_bytes,
                         bool ring = false);

// Paged KV cache.  Strides are element strides; pages [P][Hkv][S][D] in any
// order of (page, head, token) with D contiguous.
struct PagedDecode {
    const void *q, *k, *v;
    void *o;
    const int32_t *table, *seq_len;
    int B, G, Hkv, D, P, S, max_pages;
    long long table_stride;
    long long q_st[2], o_st[2];          // (batch, head)
    long long k_st[3], v_st[3];          // (page, head, token)
    int window, sinks;
    float scale;
    void *ws;
};
size_t decode_paged_workspace_bytes(int B, int Hkv);
attn_status_t decode_paged(const Ctx &c, attn_dtype_t dt, const PagedDecode &a);

struct PagedAppend {
    void *k, *v;
    const void *kn, *vn;
    const int32_t *table;
    int32_t *seq_len;
    const int32_t *new_len;              // nullptr: T rows for every sequence
    int B, T, Hkv, D, P, S, max_pages;
    long long table_stride;
    long long k_st[3], v_st[3];          // (page, head, token)
    long long kn_st[3], vn_st[3];        // (batch, head, token)
    int advance;
};
attn_status_t kv_append_paged(const Ctx &c, attn_dtype_t dt, const PagedAppend &a);

struct PagesCopy {
    void *k, *v;
    const int32_t *src, *dst, *count;    // count: nullptr for n
    int n, layers, Hkv, S, D, P;
    long long k_st[4], v_st[4];          // (layer, page, head, token)
};
attn_status_t kv_pages_copy(const Ctx &c, attn_dtype_t dt, const PagesCopy &a);

struct PageTable {
    int32_t *table;
    long long stride;
    int B, max_pages, P, S;
};
size_t kv_pages_workspace_bytes(int P);
attn_status_t kv_pages_reserve(const Ctx &c, const PageTable &t, const int32_t *seq_len,
                               const int32_t *add, int32_t *refs, void *ws);
attn_status_t kv_pages_free(const Ctx &c, const PageTable &t, const int32_t *seq_len,
                            int32_t *refs, int window, int sinks);
attn_status_t kv_pages_fork(const Ctx &c, const PageTable &t, int32_t *seq_len, int32_t *refs,
                            const int32_t *src, const int32_t *dst, int n, int32_t *copy_src,
                            int32_t *copy_dst, void *ws);
attn_status_t kv_pages_compact(const Ctx &c, const PageTable &t, const int32_t *refs,
                               int32_t *new_table, long long new_stride, int32_t *new_refs,
                               int32_t *copy_src, int32_t *copy_dst, int32_t *count, void *ws);

// tcgen05 (tensor-core) flash attention, bf16 or f16: full and neighborhood.
// st: strides of q, k, v, o (nullptr: contiguous).
attn_status_t tc_full(const Ctx &c, attn_dtype_t dt, const void *q, const void *k, const void *v,
                      void *o, int B, int H, int Nq, int Nkv, int D, float scale,
                      const TensorStrides *st = nullptr);
bool tc_full_supported(int B, int H, int Nq, int Nkv, int D);
attn_status_t tc_causal_gqa(const Ctx &c, attn_dtype_t dt, const void *q, const void *k,
                            const void *v, void *o, int B, int Hq, int Hkv, int N, int D,
                            float scale, const TensorStrides *st = nullptr);
attn_status_t simt_causal_gqa(const Ctx &c, attn_dtype_t dt, const void *q, const void *k,
                              const void *v, void *o, int B, int Hq, int Hkv, int N, int D,
                              float scale, const TensorStrides *st = nullptr);
// Sliding window with sinks: queries are the last Nq of Nkv positions.
attn_status_t tc_causal_window(const Ctx &c, attn_dtype_t dt, const void *q, const void *k,
                               const void *v, void *o, int B, int Hq, int Hkv, int Nq, int Nkv,
                               int D, int window, int sinks, float scale, const TensorStrides *st);
attn_status_t simt_causal_window(const Ctx &c, attn_dtype_t dt, const void *q, const void *k,
                                 const void *v, void *o, int B, int Hq, int Hkv, int Nq, int Nkv,
                                 int D, int window, int sinks, float scale,
                                 const TensorStrides *st);
attn_status_t tc_na3d(const Ctx &c, attn_dtype_t dt, const void *q, const void *k, const void *v,
                      void *o, int B, int H, int T, int Hg, int W, int D, const int kernel[3],
                      float scale);
bool tc_na3d_supported(int B, int H, int T, int Hg, int W, int D, const int kernel[3]);
// One 128 x 128 tile through both tcgen05 MMA forms (testing).
attn_status_t tc_selftest(const Ctx &c, const void *q, const void *k, const void *v,
                          const void *P, float *S, float *O, int D);

}  // namespace attn
