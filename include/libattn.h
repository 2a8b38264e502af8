/*
 * libattn -- multi-head scaled-dot-product attention for NVIDIA GB300 (sm_103a).
 *
 * The operation, in every entry point, for each query row i and its admitted
 * key set K(i):
 *     S = Q K^T * scale,  P = row softmax(S) over K(i),  O = P V
 * ("cuBLAS matmuls for ... attention scores" plus a softmax kernel, iris.c
 * issue #15 "CUDA codepath !"; the windowed score / softmax / accumulate of
 * candle PR #11's neighborhood attention; the single-token decode attention
 * over a device-resident KV cache of fak "GPU - the in-kernel forward pass",
 * sections 0 and 4).
 *
 * Conventions shared by all entry points
 *   - Tensors are DEVICE pointers to contiguous row-major arrays with the head
 *     dimension innermost.  Attention tensors are heads-major [B, H, N, D].
 *   - dtype ATTN_F32: float32 storage, exact fp32 FMA arithmetic (no TF32).
 *     dtype ATTN_BF16 / ATTN_F16: bfloat16 / IEEE half storage (candle's
 *     F32 / BF16 / F16 trio); the contractions run on the tensor cores
 *     (tcgen05) with fp32 accumulation where the shapes allow (else the exact
 *     SIMT kernel), the softmax in fp32, P rounded to the storage type for the
 *     P V product; the output is rounded to the storage type (to nearest even).
 *   - D (head dimension) is 32, 64 or 128.
 *   - scale <= 0 selects 1/sqrt(D).
 *   - Inputs are never written.  The output must not alias any input.
 *   - The caller owns every buffer.  No entry point allocates device memory
 *     and none synchronises: work is enqueued on `stream` (a cudaStream_t;
 *     NULL = the legacy default stream) and the call returns.
 *   - Errors: arguments are validated on the host before any launch; a failed
 *     check returns ATTN_ERR_INVALID_ARG / ATTN_ERR_UNSUPPORTED /
 *     ATTN_ERR_RESOURCE and launches nothing.  A launch failure returns
 *     ATTN_ERR_CUDA.  Device-side waits are bounded: a wait that runs out sets
 *     a device error word that attn_device_status() reports.  Nothing is
 *     thrown across this interface.
 *   - Thread safety: calls may come from several host threads; each call only
 *     reads its arguments and enqueues work.
 */
#ifndef LIBATTN_H
#define LIBATTN_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define ATTN_API __attribute__((visibility("default")))
#else
#define ATTN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ATTN_F32 = 0,
    ATTN_BF16 = 1,
    ATTN_F16 = 2
} attn_dtype_t;

typedef enum {
    ATTN_ROPE_UNSCALED = 0,
    ATTN_ROPE_LINEAR = 1,
    ATTN_ROPE_NTK = 2,
    ATTN_ROPE_BY_PARTS = 3
} attn_rope_scaling_t;

typedef enum {
    ATTN_OK = 0,
    ATTN_ERR_INVALID_ARG = 1,   /* null pointer, bad shape, bad kernel, ...       */
    ATTN_ERR_UNSUPPORTED = 2,   /* valid request this build has no kernel for     */
    ATTN_ERR_RESOURCE = 3,      /* shared memory / workspace too small            */
    ATTN_ERR_CUDA = 4,          /* a CUDA runtime call or launch failed           */
    ATTN_ERR_TIMEOUT = 5,       /* a bounded device wait ran out (device word)    */
    ATTN_ERR_DEVICE_CHECK = 6   /* a device-side consistency check failed         */
} attn_status_t;

/*
 * Full (unmasked, non-causal) attention.
 *   q [B, H, Nq, D], k and v [B, H, Nkv, D], o [B, H, Nq, D]; dtype for all.
 *   Every query attends to all Nkv keys of its (batch, head).
 *   Requires B, H, Nq, Nkv >= 1 and D in {32, 64, 128}.
 * Passage: iris.c issue #15, the reply listing "attention scores" among the
 * cuBLAS matmuls and softmax among the custom kernels.
 */
ATTN_API attn_status_t attn_full_fwd(const void *q, const void *k, const void *v, void *o,
                            int B, int H, int Nq, int Nkv, int D,
                            attn_dtype_t dtype, float scale, void *stream);

/*
 * Full attention on strided views: the operation of attn_full_fwd, with each
 * of q, k, v and o addressed through its own element strides instead of the
 * contiguous [B, H, N, D] layout, so that transposed [B, N, H, D] tensors,
 * slices of a packed QKV projection or a column block of a wider output are
 * used in place, with no copy.
 *   x_strides[3] = element strides of (batch, head, row); D is contiguous
 *   (stride 1).  Element (b, h, n, d) of x is x[b*s[0] + h*s[1] + n*s[2] + d].
 *   Every stride is >= 1 and a multiple of 16 bytes (8 elements for bf16 and
 *   f16, 4 for f32), as the tensor-memory-access unit requires; a stride
 *   whose extent is 1 is ignored.  Base pointers are 16-byte aligned.
 *   q, k and v are read only and may overlap one another; o must not
 *   overlap them, and its (batch, head, row) rows must be disjoint (checked:
 *   sorted by stride, each stride covers the extent below it).
 *   Same sizes, dtypes, scale and status codes as attn_full_fwd.
 * Passage: the unmasked attention of attn_full_fwd; the layout is an
 * addressing choice with no counterpart in the pages.
 */
ATTN_API attn_status_t attn_full_fwd_strided(const void *q, const void *k, const void *v,
                                            void *o, int B, int H, int Nq, int Nkv, int D,
                                            const int64_t q_strides[3],
                                            const int64_t k_strides[3],
                                            const int64_t v_strides[3],
                                            const int64_t o_strides[3],
                                            attn_dtype_t dtype, float scale, void *stream);

/*
 * Joint text+image attention with a multi-axis rotary embedding on Q and K.
 *   q, k, v, o [B, H, N, D]; N = text + image tokens in the caller's order.
 *   pos: DEVICE int32 [N, 4], the 4 position ids of each token.
 *   axes_dim: HOST int[4], channel widths of the 4 axis blocks; each even and
 *   sum == D.  In the block of axis a starting at channel c_a, the adjacent
 *   pair (c_a + 2i, c_a + 2i + 1) rotates by phi = pos[t][a] * theta^(-2i/axes_dim[a]):
 *       x0' = x0 cos(phi) - x1 sin(phi),   x1' = x0 sin(phi) + x1 cos(phi).
 *   V is not rotated.  Then full attention over all N tokens.
 *   workspace: DEVICE scratch of at least attn_rope_joint_workspace_bytes(...)
 *   bytes, 256-byte aligned, that no other call uses concurrently; the rotated
 *   copies of Q and K (in the storage dtype) live there during the call.
 * Passage: iris.c issue #15, GGML lessons item 3 (FLUX's custom RoPE: 4 axes
 * [32,32,32,32], separate text/image positions, repeat_interleave) and the
 * closing "AdaLN + custom RoPE + joint attention" remark.
 */
ATTN_API attn_status_t attn_rope_joint_fwd(const void *q, const void *k, const void *v, void *o,
                                  int B, int H, int N, int D,
                                  const int32_t *pos, const int axes_dim[4], float theta,
                                  attn_dtype_t dtype, float scale,
                                  void *workspace, size_t workspace_bytes, void *stream);

ATTN_API size_t attn_rope_joint_workspace_bytes(int B, int H, int N, int D, attn_dtype_t dtype);

/*
 * Causal grouped-query prefill (self-attention over a prompt).
 *   q, o [B, Hq, N, D]; k, v [B, Hkv, N, D]; Hq % Hkv == 0.  Query head hq
 *   reads KV head hq / (Hq / Hkv); query position i attends to key positions
 *   j <= i.  bf16 and f16 run on the tensor cores for D in {64, 128}; fp32
 *   (and the 16-bit types with D = 32) on the exact-FFMA SIMT kernel.
 * Passage: fak "GPU - the in-kernel forward pass", section 3 (Llama prefill
 * workloads pp64 .. pp512 of a grouped-query model).
 */
ATTN_API attn_status_t attn_causal_gqa_fwd(const void *q, const void *k, const void *v, void *o,
                                           int B, int Hq, int Hkv, int N, int D,
                                           attn_dtype_t dtype, float scale, void *stream);

/*
 * Causal grouped-query prefill on strided views: the operation of
 * attn_causal_gqa_fwd with q, k, v and o addressed through element strides
 * of (batch, head, row) as in attn_full_fwd_strided (D contiguous, every
 * stride a multiple of 16 bytes, extent-1 axes' strides ignored, o's rows
 * disjoint), so a Llama layer's [B, N, Hq, D] query projection and a packed
 * [B, N, 2, Hkv, D] key/value projection are read in place.
 * Passage: as attn_causal_gqa_fwd; the layout is an addressing choice with
 * no counterpart in the pages.
 */
ATTN_API attn_status_t attn_causal_gqa_fwd_strided(const void *q, const void *k, const void *v,
                                                  void *o, int B, int Hq, int Hkv, int N, int D,
                                                  const int64_t q_strides[3],
                                                  const int64_t k_strides[3],
                                                  const int64_t v_strides[3],
                                                  const int64_t o_strides[3],
                                                  attn_dtype_t dtype, float scale, void *stream);

/*
 * Single-token grouped-query decode attention over a KV cache.
 *   q [B, Hq, D], o [B, Hq, D]; k_cache, v_cache [B, Hkv, Lmax, D].
 *   seq_len: DEVICE int32 [B], 1 <= seq_len[b] <= Lmax (checked on the device;
 *   a violation sets ATTN_ERR_DEVICE_CHECK and that batch's output is left
 *   unwritten).  Query head hq reads KV head hq / (Hq / Hkv) and attends to
 *   cache rows j < seq_len[b]; rows at or beyond seq_len[b] are never used.
 *   Requires Hq % Hkv == 0, Hq / Hkv in {1, 2, 4, 8}, D in {64, 128}, dtype
 *   ATTN_BF16 or ATTN_F16 (q, caches and o alike).
 *   workspace: DEVICE scratch of attn_decode_gqa_workspace_bytes(...) bytes,
 *   256-byte aligned, ZERO-FILLED before its first use.  It holds per-split
 *   partial results and per-(batch, kv-head) arrival counters when the splits
 *   merge through global memory; when the splits of every (batch, kv-head)
 *   fit on the GPU at once as thread-block clusters they merge through
 *   distributed shared memory instead and the workspace is not touched.
 *   Every call that completes leaves the counters at zero, so the same workspace serves
 *   the next call without clearing.  Calls that share a workspace must not
 *   overlap on the GPU.  After a call that reported a device error, zero it
 *   again.
 * Passage: fak "GPU - the in-kernel forward pass", section 0 (device-resident
 * KV cache) and section 4 (naive decode attention: per-call scratch, one block
 * per head, no flash/paged attention).
 */
ATTN_API attn_status_t attn_decode_gqa(const void *q, const void *k_cache, const void *v_cache,
                              const int32_t *seq_len, void *o,
                              int B, int Hq, int Hkv, int Lmax, int D,
                              attn_dtype_t dtype, float scale,
                              void *workspace, size_t workspace_bytes, void *stream);

ATTN_API size_t attn_decode_gqa_workspace_bytes(int B, int Hq, int Hkv, int Lmax, int D);

/*
 * attn_decode_gqa without a workspace argument, for callers that cannot hand
 * this library any device memory beyond the tensors themselves: a host that
 * owns all device memory through its own allocator and gives plugins only
 * inputs and outputs, or a steady-state decode loop that must not call
 * cudaMalloc (it can synchronise the whole device) between tokens.  There is
 * no counterpart on the pages; this is an interface convenience only.
 *
 * Arguments, layouts, math and results are those of attn_decode_gqa.  The
 * split partials and arrival counters live in a 4 MiB array that is part of
 * the library's device image: every GPU that loads the library holds it until
 * the process exits.  Nothing is allocated per call.
 *   - Limit: the call needs about B*Hkv*splits*G'*(D+2)*4 bytes (G' = Hq/Hkv
 *     rounded up to a power of two; splits <= 3*SMs/(B*Hkv), at least 1); a
 *     problem that does not fit the 4 MiB returns ATTN_ERR_RESOURCE.
 *   - Every call on a device shares the array and leaves its contents behind;
 *     each call zeroes the counters it uses first.  Calls that may overlap on
 *     the GPU (other streams, other host threads) race: serialise them.
 *   - The first call on a device looks up the array's device address; make
 *     that first call outside any stream capture.
 *   - `stream` must belong to the current device (the array used is the
 *     current device's); a stream of another device returns
 *     ATTN_ERR_INVALID_ARG and launches nothing.
 */
ATTN_API attn_status_t attn_decode_gqa_noalloc(const void *q, const void *k_cache,
                                               const void *v_cache, const int32_t *seq_len,
                                               void *o, int B, int Hq, int Hkv, int Lmax, int D,
                                               attn_dtype_t dtype, float scale, void *stream);

/*
 * Appends one token's K and V rows to a KV cache at the position the device
 * holds, for a decode step that is captured once as a CUDA graph and replayed
 * per token with unchanged arguments.
 *   k_cache, v_cache [B, Hkv, Lmax, D] (written: row seq_len[b] of every KV
 *   head of batch b); k_new, v_new [B, Hkv, D] (read).  seq_len: DEVICE int32
 *   [B], the write position; if advance != 0 the kernel then sets
 *   seq_len[b] += 1 (so a following attn_decode_gqa sees the new token).
 *   A position outside [0, Lmax) writes nothing and sets ATTN_ERR_DEVICE_CHECK.
 *   dtype ATTN_F32, ATTN_BF16 or ATTN_F16; D in {32, 64, 128}.
 * Passage: fak "GPU - the in-kernel forward pass", section 3b, step 3 (a
 * kernel-form KV append with a scalar offset replaces the cudaMemcpy whose
 * moving destination forced a graph re-instantiation every token).
 */
ATTN_API attn_status_t attn_kv_append(void *k_cache, void *v_cache, const void *k_new,
                                      const void *v_new, int32_t *seq_len, int B, int Hkv,
                                      int Lmax, int D, attn_dtype_t dtype, int advance,
                                      void *stream);

/*
 * Ring KV cache: the pair attn_kv_append_ring / attn_decode_gqa_ring keeps the
 * most recent Lmax tokens of a sequence in a cache of Lmax rows, so a decode
 * loop captured once as a CUDA graph runs past the cache capacity instead of
 * stopping at it (a sliding attention window of Lmax tokens).
 *   seq_len[b] counts every token appended to sequence b so far (it may
 *   exceed Lmax); token t lives in row t % Lmax until token t + Lmax
 *   overwrites it.
 *   attn_kv_append_ring: as attn_kv_append, writing row seq_len[b] % Lmax;
 *   seq_len[b] must be >= 0 and below INT32_MAX, else nothing is written and
 *   ATTN_ERR_DEVICE_CHECK is set.
 *   attn_decode_gqa_ring: as attn_decode_gqa, attending to the
 *   min(seq_len[b], Lmax) rows that hold tokens, i.e. to tokens
 *   [seq_len[b] - Lmax, seq_len[b]) once the ring has wrapped; seq_len[b] >= 1
 *   with no upper bound.  The row order does not change the result: the
 *   softmax-weighted sum runs over a set of keys, whose positions are already
 *   in their rotated K rows.  Same workspace contract as attn_decode_gqa.
 * Passage: fak "GPU - the in-kernel forward pass", section 3b (the device KV
 * of fixed capacity, with a dynamic / ring device KV named as the follow-up).
 * With Lmax a call argument, a larger capacity is a new cache and a new
 * capture; the ring is what lets one capture run indefinitely.
 */
ATTN_API attn_status_t attn_kv_append_ring(void *k_cache, void *v_cache, const void *k_new,
                                           const void *v_new, int32_t *seq_len, int B, int Hkv,
                                           int Lmax, int D, attn_dtype_t dtype, int advance,
                                           void *stream);
ATTN_API attn_status_t attn_decode_gqa_ring(const void *q, const void *k_cache,
                                            const void *v_cache, const int32_t *seq_len,
                                            void *o, int B, int Hq, int Hkv, int Lmax, int D,
                                            attn_dtype_t dtype, float scale, void *workspace,
                                            size_t workspace_bytes, void *stream);

/*
 * Causal grouped-query prefill with a sliding window and sinks.
 *   q, o [B, Hq, Nq, D]; k, v [B, Hkv, Nkv, D]; Hq % Hkv == 0, Nq <= Nkv.  The
 *   queries are the last Nq of the Nkv positions: query i sits at position
 *   p = Nkv - Nq + i and attends to
 *       { j <= p : j > p - window  or  j < sinks },
 *   i.e. its newest `window` positions (itself among them) and the first
 *   `sinks` tokens.  window <= 0: no window (plain causal attention).
 *   sinks >= 0.  Nq < Nkv continues a prompt whose first keys are cached.
 *   x_strides[3] as in attn_full_fwd_strided (NULL: contiguous).
 *   A key that a query does not attend to does not change a bit of its output,
 *   whatever it or its value holds (infinities and NaN included).  An infinity
 *   or NaN that it does attend to makes what it reaches infinite or NaN.
 *   bf16 and f16 run on the tensor cores for D in {64, 128}; fp32 (and the
 *   16-bit types with D = 32) on the exact-FFMA SIMT kernel.  Work grows with
 *   Nq * (window + sinks), not with Nq * Nkv.
 *   Requires Nkv <= 2^30.
 * Passage: fak "GPU - the in-kernel forward pass", section 3 (Llama prefill
 * of a grouped-query model); the window is that of attn_decode_gqa_paged.
 */
ATTN_API attn_status_t attn_causal_gqa_window_fwd(const void *q, const void *k, const void *v,
                                                  void *o, int B, int Hq, int Hkv, int Nq,
                                                  int Nkv, int D, const int64_t q_strides[3],
                                                  const int64_t k_strides[3],
                                                  const int64_t v_strides[3],
                                                  const int64_t o_strides[3], int window,
                                                  int sinks, attn_dtype_t dtype, float scale,
                                                  void *stream);

/*
 * Causal grouped-query attention over packed sequences of different lengths.
 *   q, o [Nq, Hq, D], k, v [Nkv, Hkv, D], element strides (token, head) in
 *   x_strides[2] (NULL: contiguous).  cu_q, cu_k: DEVICE int32 [B + 1]: sequence b
 *   has the queries [cu_q[b], cu_q[b + 1]) and the keys [cu_k[b], cu_k[b + 1]);
 *   cu_k may be cu_q.  The queries of a sequence are the last of its positions,
 *   as in attn_causal_gqa_window_fwd, whose window, sinks and rules for infinities
 *   and NaN hold within each sequence: what lies in other sequences' rows, or
 *   between them, does not change a bit of its output.
 *   Sequences may be empty, and so may cu_q's (keys without queries).  Rows of o
 *   outside every sequence are left as they were.  A sequence with more queries
 *   than keys, or whose starts do not rise or pass Nq / Nkv, sets
 *   ATTN_ERR_DEVICE_CHECK and its rows of o are left as they were (but for rows
 *   that another sequence, whose own starts rise, claims as well).  Starts that
 *   fall may leave other sequences' rows as they were, too.
 *   The lengths are read on the device: Nq and Nkv are the arrays' extents, and
 *   a captured call serves any lengths within them.  bf16 and f16 run on the
 *   tensor cores for D in {64, 128}; fp32 (and the 16-bit types with D = 32) on
 *   the exact-FFMA SIMT kernel.  B <= 65535, Nq and Nkv <= 2^26.
 * Passage: fak "GPU - the in-kernel forward pass", section 3 (Llama prefill of
 * a grouped-query model), for a batch of prompts without padding.
 */
ATTN_API attn_status_t attn_causal_gqa_varlen_fwd(const void *q, const void *k, const void *v,
                                                  void *o, const int32_t *cu_q,
                                                  const int32_t *cu_k, int B, int Nq, int Nkv,
                                                  int Hq, int Hkv, int D,
                                                  const int64_t q_strides[2],
                                                  const int64_t k_strides[2],
                                                  const int64_t v_strides[2],
                                                  const int64_t o_strides[2], int window,
                                                  int sinks, attn_dtype_t dtype, float scale,
                                                  void *stream);

/*
 * Paged KV cache.  Many sequences share one pool of pages of `page_size`
 * tokens; a page table names each sequence's pages.  Conventions of all
 * entries below:
 *   k_pages, v_pages [num_pages, Hkv, page_size, D], any order of the three
 *     outer axes given by k_strides / v_strides[3] = element strides of (page,
 *     head, token); D is contiguous, strides are multiples of 16 bytes, a
 *     stride whose extent is 1 is ignored, NULL means contiguous in the order
 *     above.  page_size is a multiple of 8.
 *   page_table: DEVICE int32 [B, max_pages], rows table_stride entries apart
 *     (>= max_pages).  Position j of sequence b lives in row j % page_size of
 *     page page_table[b][j / page_size]; -1 means no page.  Requires
 *     max_pages * page_size < 2^31 and B <= 2^20.
 *   seq_len: DEVICE int32 [B], tokens held by each sequence.
 *   page_refs: DEVICE int32 [num_pages], 16-byte aligned: how many table
 *     entries name the page; 0 means free.  A page named by several rows
 *     (after a fork) is only read.  page_table and page_refs are the whole
 *     state of the allocator; a new pool is refs = 0 and table = -1.
 *   The values are read on the device when the call runs, so every call can be
 *   captured in a CUDA graph and replayed as sequences grow.
 */

/*
 * Appends the K and V rows of new tokens to the sequences' pages.
 *   k_new, v_new [B, Hkv, T, D], element strides (batch, head, token) in
 *   kn_strides / vn_strides[3] (NULL: contiguous), e.g. slices of a packed
 *   projection.  new_len: DEVICE int32 [B], rows to append per sequence, 0 <=
 *   new_len[b] <= T; NULL means T.  Row t goes to position seq_len[b] + t; if
 *   advance != 0, seq_len[b] += new_len[b] afterwards.
 *   The pages must exist (attn_kv_pages_reserve) and be named by this sequence
 *   alone.  A request that does not fit the table writes nothing; a token whose
 *   table entry is no page of the pool is not written; either sets
 *   ATTN_ERR_DEVICE_CHECK and leaves that sequence's seq_len as it was.
 *   The cache's (page, head, token) rows must be disjoint (checked).
 *   dtype ATTN_F32, ATTN_BF16 or ATTN_F16; D in {32, 64, 128}.
 * Passage: fak "GPU - the in-kernel forward pass", section 3b (the kernel-form
 * KV append with a device-held position), on pages.
 */
ATTN_API attn_status_t attn_kv_append_paged(void *k_pages, void *v_pages, const void *k_new,
                                            const void *v_new, const int32_t *page_table,
                                            int32_t *seq_len, const int32_t *new_len, int B, int T,
                                            int Hkv, int D, int num_pages, int page_size,
                                            int max_pages, int64_t table_stride,
                                            const int64_t k_strides[3], const int64_t v_strides[3],
                                            const int64_t kn_strides[3],
                                            const int64_t vn_strides[3], attn_dtype_t dtype,
                                            int advance, void *stream);

/*
 * Single-token grouped-query decode attention over a paged KV cache.
 *   q, o [B, Hq, D] with element strides (batch, head) in q_strides /
 *   o_strides[2] (NULL: contiguous).  Query head hq of sequence b reads KV head
 *   hq / (Hq / Hkv) and attends to the positions
 *       { j < seq_len[b] : j >= seq_len[b] - window  or  j < sinks };
 *   window <= 0: all of them.  sinks >= 0.
 *   seq_len[b] == 0 (an idle slot) writes zeros.  Table entries of pages that
 *   hold no visible position are not needed, so those pages may be free.  Rows of a page
 *   behind seq_len[b], or outside the window, do not change the result,
 *   whatever they hold.  An infinity or NaN that is visible makes what it
 *   reaches infinite or NaN.
 *   A seq_len[b] outside [0, max_pages * page_size], or a needed entry that is
 *   no page of the pool, sets ATTN_ERR_DEVICE_CHECK and leaves that sequence's
 *   output unwritten; other sequences' are not affected.
 *   Requires Hq % Hkv == 0, Hq / Hkv <= 16, D in {64, 128}, dtype ATTN_BF16 or
 *   ATTN_F16 (q, pages and o alike), B * Hkv * (max_pages * page_size + 32) < 2^36.  For one set of inputs the result does not
 *   depend on timing.
 *   workspace: DEVICE scratch of attn_decode_gqa_paged_workspace_bytes(...)
 *   bytes, 256-byte aligned, ZERO-FILLED before its first use.  Every call that
 *   completes leaves it ready for the next one, of any sizes it is large enough
 *   for.  Calls (and replays of captured ones) that share a workspace must not
 *   overlap on the GPU.
 * Passage: fak "GPU - the in-kernel forward pass", section 4 (naive decode
 * attention, "no flash/paged attention").
 */
ATTN_API attn_status_t attn_decode_gqa_paged(const void *q, const void *k_pages,
                                             const void *v_pages, const int32_t *page_table,
                                             const int32_t *seq_len, void *o, int B, int Hq,
                                             int Hkv, int D, int num_pages, int page_size,
                                             int max_pages, int64_t table_stride,
                                             const int64_t q_strides[2],
                                             const int64_t k_strides[3],
                                             const int64_t v_strides[3],
                                             const int64_t o_strides[2], int window, int sinks,
                                             attn_dtype_t dtype, float scale, void *workspace,
                                             size_t workspace_bytes, void *stream);

ATTN_API size_t attn_decode_gqa_paged_workspace_bytes(int B, int Hq, int Hkv, int D);

/*
 * Rotary positions.  The first rotary_dim channels of a row at position t are
 * rotated in pairs (a, b) by the angle t theta_i, i < rotary_dim / 2:
 *     a' = m (a cos - b sin),   b' = m (b cos + a sin);
 * pair i is channels (i, i + rotary_dim / 2), or (2i, 2i + 1) if interleaved.
 * The other channels are copied.  rotary_dim is a multiple of 16, at most D.
 *   freq: DEVICE uint64 [rotary_dim / 2], theta_i as a fraction of a turn per
 *     position, 2^64 theta_i / (2 pi) (8-byte aligned).  The angle is the product
 *     modulo 2^64, within 2^-31 of a turn at every 32-bit position where the table
 *     holds nearest integers, as attn_rope_frequencies' does.
 *   mscale: the factor m (1 for plain rotary positions; not for the copied
 *     channels).  Must be finite.
 *
 * attn_rope_frequencies fills freq (HOST memory here; the caller copies it to
 * the device, once) with theta_i = theta^(-2i / rotary_dim), scaled for contexts
 * `factor` times the original length:
 *   ATTN_ROPE_UNSCALED  as it is;
 *   ATTN_ROPE_LINEAR    theta_i / factor;
 *   ATTN_ROPE_NTK       with theta factor^(rotary_dim / (rotary_dim - 2)) in
 *                       the place of theta;
 *   ATTN_ROPE_BY_PARTS  (1 - g) theta_i / factor + g theta_i, where a pair that
 *                       makes r = original_len theta_i / (2 pi) turns within the
 *                       original length has g = (r - alpha) / (beta - alpha),
 *                       held to [0, 1].
 *   theta > 0 and factor > 0 finite; by parts also original_len > 0 and beta >
 *   alpha.  A theta_i of half a turn or more is refused.
 *
 * attn_rope_fwd: y = the rotated rows of x, both [B, H, N, D] with element
 *   strides (batch, head, token) in x_strides / y_strides[3] (NULL: contiguous).
 *   positions: DEVICE int32 [B, N], rows pos_stride entries apart (at least N, or 0:
 *   one row for all batches); any value, negative ones too.  inverse != 0: the transposed
 *   rotation (angles negated), which is the gradient of the call with respect
 *   to x.  y may be x itself, with x's strides (in place); it must not overlap x
 *   otherwise.  All dtypes, D in {32, 64, 128}, H <= 2^30; fp32 arithmetic, rounded
 *   once.
 * Passage: iris.c issue #15 "CUDA codepath !" (custom RoPE kernel) and fak
 * "GPU - the in-kernel forward pass", section 3 (the rotary step of a Llama
 * layer); the scalings are published extensions of it.
 */
ATTN_API attn_status_t attn_rope_frequencies(uint64_t *freq, int rotary_dim, double theta,
                                             attn_rope_scaling_t scaling, double factor,
                                             double original_len, double alpha, double beta);

ATTN_API attn_status_t attn_rope_fwd(const void *x, void *y, const uint64_t *freq,
                                     const int32_t *positions, int64_t pos_stride, int B, int H,
                                     int N, int D, int rotary_dim, int interleaved, int inverse,
                                     float mscale, const int64_t x_strides[3],
                                     const int64_t y_strides[3], attn_dtype_t dtype, void *stream);

/*
 * attn_kv_append_paged for packed new tokens, K rotated on the way.
 *   k_new, v_new [N, Hkv, D] (read), q, q_out [N, Hq, D], element strides (token,
 *   head) in kn_strides / vn_strides / q_strides / qo_strides[2] (NULL: contiguous),
 *   e.g. column blocks of one packed projection.
 *   cu_new: DEVICE int32 [B + 1], sequence b's new tokens are rows [cu_new[b],
 *   cu_new[b + 1]); rows outside every sequence are not touched.  NULL: one token
 *   per sequence, row b (N == B).
 *   Row cu_new[b] + t goes to position seq_len[b] + t: K is rotated for that
 *   position (freq, rotary_dim, interleaved and mscale as in attn_rope_fwd) and
 *   rounded once, V is copied.  q, if not NULL, is rotated likewise into q_out
 *   (which may be q itself, with q's strides).  If advance != 0, seq_len[b] +=
 *   the sequence's new tokens afterwards.
 *   Pages, errors and their effects as for attn_kv_append_paged: a request that
 *   does not fit the table, or starts that do not rise or pass N, writes nothing
 *   for that sequence (its rows of q_out neither); a token whose entry is no
 *   page is not written.  Either sets ATTN_ERR_DEVICE_CHECK and leaves that
 *   sequence's seq_len as it was.
 *   All dtypes, D in {32, 64, 128}; Hkv and Hq at most 65535.
 * Passage: fak "GPU - the in-kernel forward pass", section 3b (kernel-form KV
 * append), with the rotary step before it.
 */
ATTN_API attn_status_t attn_kv_append_paged_rope(
    void *k_pages, void *v_pages, const void *k_new, const void *v_new, const void *q, void *q_out,
    const int32_t *page_table, int32_t *seq_len, const int32_t *cu_new, const uint64_t *freq, int B,
    int N, int Hq, int Hkv, int D, int rotary_dim, int interleaved, float mscale, int num_pages,
    int page_size, int max_pages, int64_t table_stride, const int64_t k_strides[3],
    const int64_t v_strides[3], const int64_t kn_strides[2], const int64_t vn_strides[2],
    const int64_t q_strides[2], const int64_t qo_strides[2], attn_dtype_t dtype, int advance,
    void *stream);

/*
 * Paged KV cache held in 4 bits.  One array kv_pages holds K and V: a page is
 * [Hkv, page_size] rows of attn_kv_q4_row_bytes(D) = D + D / 8 bytes, one token
 * and KV head each; the rows of a (page, head) are contiguous, pages_strides[2]
 * are the BYTE strides of (page, head) (NULL: contiguous), multiples of 16.
 * Page table, lengths and allocator are those of the paged cache above.
 *   Values are held in groups of 32 channels as s (n - 8), n in [0, 15].  With
 *   x* the group's largest or its least value, whichever is further from zero
 *   (the largest if both are), s = -x* / 8, rounded to `dtype` (ATTN_BF16 or
 *   ATTN_F16; below 2^-126: 0), and n = rint(x (1 / s)) + 8, held to [0, 15], in
 *   fp32 (s = 0: n = 8).  A group that holds an infinity or NaN, or whose s does
 *   not fit, is NaN throughout.  A cache is read with the dtype it was written with.
 *   A row is: the codes of K (D / 2 bytes), those of V (D / 2), the scales of K's
 *   groups (D / 16), those of V's (D / 16).  The codes of four consecutive channels
 *   form a 16-bit word, channel i's at bit 4 i, rotated right by two bits
 *   (little-endian).  Channel c = 32 g + r: K's word lies at byte (r / 8) D / 8 +
 *   4 g + 2 (r / 4 mod 2), V's at D / 2 + (r / 4) D / 16 + 2 g.
 *   D in {64, 128}, dtype ATTN_BF16 or ATTN_F16.
 *
 * attn_kv_append_paged_q4: attn_kv_append_paged_rope into such pages.  freq NULL
 *   (rotary_dim 0): neither K nor q is rotated (q is copied to q_out).
 * attn_kv_gather_paged_q4: the reader.  k, v [N, Hkv, D] (written, strides (token,
 *   head)); row cu_len[b] + t receives position start[b] + t of sequence b
 *   (DEVICE int32; start NULL: 0), t < cu_len[b + 1] - cu_len[b], rounded once to
 *   dtype.  Rows outside every sequence are left as they were.  A position
 *   outside the table, or whose entry is no page, is left as it was and sets
 *   ATTN_ERR_DEVICE_CHECK; so are all rows of a sequence whose starts do not
 *   rise or pass N.  It gives the cached keys and values of a prompt
 *   that is continued to attn_causal_gqa_varlen_fwd.
 * attn_kv_pages_copy_q4: attn_kv_pages_copy for such pages; strides[3]: BYTE
 *   strides of (layer, page, head) (NULL: contiguous).
 * attn_decode_gqa_paged_q4: attn_decode_gqa_paged over such pages: the same
 *   arguments, visibility, errors and workspace rules, with a workspace of
 *   attn_decode_gqa_paged_q4_workspace_bytes(...) bytes.  Codes are multiplied as they are and
 *   scaled in fp32; a weight times its value's scale is rounded to 11 bits for
 *   the P V product (below 2^-21 of the largest such product of its head and group
 *   of 32 channels, to a multiple of 2^-31 of that one).  Outputs are finite for
 *   scales of up to 2^100.
 * Passage: fak "GPU - the in-kernel forward pass", section 3b (the device KV
 * cache), section 4 (decode attention), and candle PR #11's int8 rows with a scale
 * for the idea of holding rows in fewer bits.
 */
ATTN_API size_t attn_kv_q4_row_bytes(int D);

ATTN_API attn_status_t attn_kv_append_paged_q4(
    void *kv_pages, const void *k_new, const void *v_new, const void *q, void *q_out,
    const int32_t *page_table, int32_t *seq_len, const int32_t *cu_new, const uint64_t *freq, int B,
    int N, int Hq, int Hkv, int D, int rotary_dim, int interleaved, float mscale, int num_pages,
    int page_size, int max_pages, int64_t table_stride, const int64_t pages_strides[2],
    const int64_t kn_strides[2], const int64_t vn_strides[2], const int64_t q_strides[2],
    const int64_t qo_strides[2], attn_dtype_t dtype, int advance, void *stream);

ATTN_API attn_status_t attn_kv_gather_paged_q4(
    const void *kv_pages, const int32_t *page_table, const int32_t *start, const int32_t *cu_len,
    void *k, void *v, int B, int N, int Hkv, int D, int num_pages, int page_size, int max_pages,
    int64_t table_stride, const int64_t pages_strides[2], const int64_t k_strides[2],
    const int64_t v_strides[2], attn_dtype_t dtype, void *stream);

ATTN_API attn_status_t attn_kv_pages_copy_q4(void *kv_pages, const int32_t *copy_src,
                                             const int32_t *copy_dst, int n, const int32_t *count,
                                             int layers, int num_pages, int Hkv, int page_size,
                                             int D, const int64_t strides[3], void *stream);

ATTN_API attn_status_t attn_decode_gqa_paged_q4(
    const void *q, const void *kv_pages, const int32_t *page_table, const int32_t *seq_len, void *o,
    int B, int Hq, int Hkv, int D, int num_pages, int page_size, int max_pages,
    int64_t table_stride, const int64_t q_strides[2], const int64_t pages_strides[2],
    const int64_t o_strides[2], int window, int sinks, attn_dtype_t dtype, float scale,
    void *workspace, size_t workspace_bytes, void *stream);

ATTN_API size_t attn_decode_gqa_paged_q4_workspace_bytes(int B, int Hq, int Hkv, int D);

/*
 * The page allocator.  Each call takes its pages lowest number first and
 * serves requests in (row, entry) order, so its result depends on its inputs
 * alone (but for free where a page's count is too low: which of the entries that
 * name it keep it).  A request that cannot be met, or an argument on the device that is
 * out of range, sets ATTN_ERR_DEVICE_CHECK and changes nothing (free: the
 * entry, or the row of that seq_len, stays; compact: an entry that names no live page becomes
 * -1).  page_refs must count the table's entries, as these calls keep it; calls
 * that change the same pool are ordered by their stream.
 *   workspace: DEVICE scratch of attn_kv_pages_workspace_bytes(num_pages)
 *   bytes, 256-byte aligned, contents irrelevant, not used by another call at
 *   the same time.  reserve and fork take B <= 16384, reserve B * max_pages < 2^31.
 *
 * reserve: pages for the add_len[b] tokens (DEVICE int32 [B], >= 0) behind
 *   seq_len[b]: every entry that covers a position in [seq_len[b], seq_len[b] +
 *   add_len[b]) and holds no page gets one.
 * free: lets go of every page that holds no token sequence b can still see:
 *   entries whose positions are all >= seq_len[b], or (window > 0) all < seq_len[b] -
 *   window and >= sinks.  With seq_len[b] = 0 that is the whole row.  Pages
 *   reserved ahead of seq_len[b] are let go too.
 * fork: for i < n, row dst[i] becomes a copy of row src[i] (DEVICE int32 [n]),
 *   seq_len[dst[i]] = seq_len[src[i]]; what dst[i] held is let go first.  Full
 *   pages are shared; a partly filled last page gets a page of its own, and
 *   (copy_src[i], copy_dst[i]) (DEVICE int32 [n]) names the copy that
 *   attn_kv_pages_copy must make before either row is appended to; (-1, -1) if
 *   there is none.  No row may be a target twice, or both target and source; a
 *   source may be named many times.  1 <= n <= B, n <= 8192.
 * compact: moves the live pages to the lowest numbers.  With L live pages the
 *   k-th live page >= L goes to the k-th free page < L.  Writes the new table
 *   and counts to new_table (rows new_stride apart) and new_refs, either of
 *   which may be the old array; copy_src / copy_dst (DEVICE int32
 *   [num_pages / 2], NULL allowed only if num_pages is 1) hold *count (DEVICE
 *   int32) moves and -1 behind them.
 * copy: copies pages copy_src[i] -> copy_dst[i], i < n (and < *count, if count
 *   is not NULL), K and V, in each of `layers` caches that share one table:
 *   strides[4] of (layer, page, head, token), NULL = contiguous.  A pair
 *   (-1, -1) is skipped; another number outside the pool sets
 *   ATTN_ERR_DEVICE_CHECK and that pair is skipped.  The pairs are copied in no
 *   order, so no page may be a target twice, or both target and source (the
 *   lists of fork and compact are so).  All dtypes, D in {32, 64, 128}.
 * Passage: fak "GPU - the in-kernel forward pass", section 3b (device KV of a
 * dynamic capacity, named there as the follow-up).
 */
ATTN_API size_t attn_kv_pages_workspace_bytes(int num_pages);

ATTN_API attn_status_t attn_kv_pages_reserve(int32_t *page_table, const int32_t *seq_len,
                                             const int32_t *add_len, int32_t *page_refs, int B,
                                             int num_pages, int page_size, int max_pages,
                                             int64_t table_stride, void *workspace,
                                             size_t workspace_bytes, void *stream);

ATTN_API attn_status_t attn_kv_pages_free(int32_t *page_table, const int32_t *seq_len,
                                          int32_t *page_refs, int B, int num_pages, int page_size,
                                          int max_pages, int64_t table_stride, int window,
                                          int sinks, void *stream);

ATTN_API attn_status_t attn_kv_pages_fork(int32_t *page_table, int32_t *seq_len,
                                          int32_t *page_refs, const int32_t *src,
                                          const int32_t *dst, int n, int32_t *copy_src,
                                          int32_t *copy_dst, int B, int num_pages, int page_size,
                                          int max_pages, int64_t table_stride, void *workspace,
                                          size_t workspace_bytes, void *stream);

ATTN_API attn_status_t attn_kv_pages_compact(const int32_t *page_table, const int32_t *page_refs,
                                             int32_t *new_table, int32_t *new_refs,
                                             int32_t *copy_src, int32_t *copy_dst, int32_t *count,
                                             int B, int num_pages, int max_pages,
                                             int64_t table_stride, int64_t new_stride,
                                             void *workspace, size_t workspace_bytes,
                                             void *stream);

ATTN_API attn_status_t attn_kv_pages_copy(void *k_pages, void *v_pages, const int32_t *copy_src,
                                          const int32_t *copy_dst, int n, const int32_t *count,
                                          int layers, int num_pages, int Hkv, int page_size, int D,
                                          const int64_t k_strides[4], const int64_t v_strides[4],
                                          attn_dtype_t dtype, void *stream);

/*
 * 3D neighborhood attention with NATTEN boundary windows.
 *   q, k, v, o [B, heads, N, D] with N = T * Hg * W tokens in row-major
 *   (t, h, w) order.  kernel: HOST int[3], the requested window per axis; each
 *   must be positive and odd, and may exceed the axis extent.  Per axis of
 *   extent n and request k: k_eff = min(k, n); query coordinate i attends to
 *   [s, s + k_eff) with s = clamp(i - k/2, 0, n - k_eff); the 3D window is the
 *   Cartesian product of the three intervals.  A window at least as wide as
 *   its axis is full attention along that axis.
 * Passage: candle PR #11, the "Line-for-line port of neighborhood_attention.metal"
 * commit and the "kernel exceeds grid extent" commit (effective_kernel() clamp,
 * validate() only requires a positive odd triple).
 */
ATTN_API attn_status_t attn_na3d_fwd(const void *q, const void *k, const void *v, void *o,
                            int B, int heads, int T, int Hg, int W, int D,
                            const int kernel[3], attn_dtype_t dtype, float scale,
                            void *stream);

/*
 * 3D neighborhood attention on strided views: the operation of
 * attn_na3d_fwd with q, k, v and o addressed through element strides of
 * (batch, head, token) as in attn_full_fwd_strided (D contiguous, every
 * stride a multiple of 16 bytes, extent-1 axes' strides ignored, o's rows
 * disjoint); tokens keep their row-major (t, h, w) order at a uniform token
 * stride, so a [B, T*Hg*W, heads, D] projection is read in place.  A
 * non-contiguous layout runs on the exact SIMT kernel; contiguous strides
 * take the tensor-core kernel of attn_na3d_fwd.
 * Passage: as attn_na3d_fwd; the layout is an addressing choice with no
 * counterpart in the pages.
 */
ATTN_API attn_status_t attn_na3d_fwd_strided(const void *q, const void *k, const void *v, void *o,
                                            int B, int heads, int T, int Hg, int W, int D,
                                            const int kernel[3], const int64_t q_strides[3],
                                            const int64_t k_strides[3],
                                            const int64_t v_strides[3],
                                            const int64_t o_strides[3], attn_dtype_t dtype,
                                            float scale, void *stream);

/*
 * Window starts as the neighborhood kernels compute them (same device
 * function), for testing: starts = DEVICE int32 [T*Hg*W, 3], the (t, h, w)
 * start of each query's window.  Same validation as attn_na3d_fwd.
 */
ATTN_API attn_status_t attn_na3d_window_starts(int T, int Hg, int W, const int kernel[3],
                                      int32_t *starts, void *stream);

/*
 * Tensor-core building-block check (testing): one CTA computes, for a single
 * tile, S = q k^T + q[:, :16] k[:, :16]^T and O = P v with the same tcgen05
 * MMA forms, shared-memory layouts (128-byte swizzle for q, k, v; 32-byte
 * swizzle for the 16-channel term, as used by the neighborhood kernel's
 * window-penalty channels) and TMEM placement the bf16 attention kernels use.
 *   q, k, v: DEVICE bf16 [128, D]; P: DEVICE bf16 [128, 128];
 *   S: DEVICE f32 [128, 128]; O: DEVICE f32 [128, D]; D in {64, 128}.
 * No counterpart on the pages: it isolates the matrix-descriptor and
 * tensor-memory conventions so a layout error shows up as a wrong tile here.
 */
ATTN_API attn_status_t attn_debug_tc_tile(const void *q, const void *k, const void *v,
                                          const void *P, float *S, float *O, int D,
                                          void *stream);

/*
 * Bounded-wait check (testing): launches one thread that waits on a
 * shared-memory barrier nothing ever completes, with a wait limit of
 * limit_ns nanoseconds (1000 .. 1000000000; outside that range
 * ATTN_ERR_INVALID_ARG and nothing launches).  The wait runs out, sets the
 * device error word to the timeout code and the thread returns, so the
 * next attn_device_status() on this stream returns ATTN_ERR_TIMEOUT (and
 * clears the word) with the context still usable.  Every spin-wait in the
 * attention kernels is this same bounded wait with a limit of one second.
 * No counterpart on the pages: it exercises the library's failure reporting
 * without faulting or hanging a GPU.
 */
ATTN_API attn_status_t attn_debug_wait_test(uint64_t limit_ns, void *stream);

/* Human-readable name of a status code (static storage). */
ATTN_API const char *attn_status_string(attn_status_t status);

/*
 * Synchronises `stream`, then reads and clears the device error word that
 * bounded waits and device-side checks set on the current device.
 * Returns ATTN_OK, ATTN_ERR_TIMEOUT, ATTN_ERR_DEVICE_CHECK or ATTN_ERR_CUDA.
 */
ATTN_API attn_status_t attn_device_status(void *stream);

/*
 * Number of kernel launches this process has made through the given kernel
 * family, for tests that must prove the path under test really ran.
 * ids: 0 = fp32/SIMT flash, 1 = tcgen05 flash, 2 = decode split-KV,
 *      3 = RoPE prologue, 4 = window-start export, 5 = tcgen05 neighborhood,
 *      6 = KV-cache append, 7 = bounded-wait check, 8 = paged decode,
 *      9 = paged append, page allocator and page copies.
 * Returns 0 for an unknown id.
 */
ATTN_API uint64_t attn_launch_count(int kernel_family);

/* Library version string, e.g. "libattn 0.1 sm_103a". */
ATTN_API const char *attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LIBATTN_H */
