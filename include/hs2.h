/*
 * hs2.h — C ABI of the group-shared top-k sparse attention library (libhs2).
 *
 * One Cross group of a HySparse2 model = one FA layer + its SA layers over one
 * shared paged KV cache. The FA layer attends causally to every visible key and
 * emits, per query and KV head, the top-k positions outside a forced recent
 * window; each SA layer reuses that KV and those positions with its own query,
 * attending to window ∪ top-k under one softmax. The CSA2 variant replaces the
 * FA selection by a hierarchical lightning indexer (Full / Reindex / Reuse).
 *
 * Pages this interface restates (cited by title and section):
 *   [HS2]  "HySparse2：整体架构、KV 生命周期与 PD 分离"
 *          §5 (KV Reuse), §7.1-7.4 (forced window + out-of-window top-k, one
 *          normalisation, direct access to paged KV).
 *   [CSA2] "2.3.1 · CSA、HCA 与 CSA2: 压缩序列上的稀疏检索和跨层复用"
 *          §3.1 (Full / Reindex / Reuse), §3.2 (hierarchical sparse indexer).
 *   [L10]  "Lecture 10 · 混合架构与稀疏注意力：Mamba、Marconi 与 DeepSeek-V3.2"
 *          §5.1 (lightning indexer score), §5.5 (paged gather through a block table).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Positions are 0-based. A query that sees t keys sits at position t-1; its
 *   own key is already in the cache. Window W(t) = [max(0,t-w), t-1]; far range
 *   F(t) = [0, t-w-1]; the FA selects min(k, max(0, t-w)) positions of F(t).
 * - GQA: query head h reads KV head g = h / (Hq / Hkv).
 * - All pointers are DEVICE pointers unless stated otherwise. The caller owns
 *   every buffer (inputs, outputs, workspace, dev_err). The library never
 *   allocates, frees or synchronises; every call is asynchronous on `stream`
 *   (a cudaStream_t passed as void*; NULL = the legacy default stream).
 * - Return value: host-side validation and launch status. HS2_ERR_ARG means
 *   nothing was launched. HS2_ERR_CUDA means a launch failed (the CUDA error is
 *   cleared and reported by hs2_last_cuda_error()).
 * - dev_err (optional, may be NULL): int32 device word the kernels OR error bits
 *   into (HS2_DEV_*) when they meet an out-of-range block-table entry or index,
 *   or give up a bounded wait. Bad accesses are skipped, never performed. The
 *   caller zeroes it and reads it after synchronising.
 * - Outputs are float32 whatever the input dtype (fp32 accumulation); hs2_fa_chunk, hs2_kv_read
 *   and the latent operators take the output type as an argument.
 * - Index sets are written sorted ascending, padded with -1, with a count array.
 *   Among equal scores the lower position (or lower block id) wins.
 */
#ifndef HS2_H
#define HS2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define HS2_ABI_VERSION 6

typedef enum {
  HS2_OK = 0,
  HS2_ERR_ARG = -1,         /* invalid shape, pointer, alignment or workspace size */
  HS2_ERR_UNSUPPORTED = -2, /* valid but not implemented combination (e.g. head_dim 96) */
  HS2_ERR_CUDA = -3,        /* a CUDA launch / runtime call failed */
  HS2_ERR_DEVICE = -4,      /* reserved for callers that fold dev_err into a status */
  HS2_ERR_SCRATCH_LIMIT = -5 /* problem needs more scratch than hs2_fa_select_noalloc holds */
} hs2_status;

/* device-side error bits (ORed into *dev_err) */
#define HS2_DEV_BAD_PAGE 1    /* block-table entry outside [0, num_pages) */
#define HS2_DEV_BAD_INDEX 2   /* selected position outside F(t) (or outside [0,t) with w=0) */
#define HS2_DEV_TIMEOUT 4     /* a bounded wait (mbarrier / TMA / MMA) gave up */
#define HS2_DEV_BAD_LENGTH 8  /* seq_len < 1 or beyond max_pages * page_size */
#define HS2_DEV_SELECT 16     /* reserved: no longer raised. A prefill row whose streamed
                                 candidates cannot prove its top-k is recomputed exactly over
                                 its whole far range inside hs2_fa_select */

typedef enum { HS2_F32 = 0, HS2_BF16 = 1, HS2_FP8_E4M3 = 2, HS2_FP4_E2M1 = 3 } hs2_dtype;

/* Paged KV of ONE group, shared by its FA and SA layers ([HS2] §5, §7.2).
 * k, v:        [num_pages][Hkv][page_size][d] elements of `dtype`, 16-byte aligned.
 *              v may be NULL for an indexer-key cache (hs2_hier_reindex).
 * block_table: int32 [batch][max_pages]; entry j of sequence b is the physical page
 *              holding logical positions [j*page_size, (j+1)*page_size).
 * seq_len:     int32 [batch], keys visible to the query (its own included), >= 1.
 * k_scale, v_scale: HS2_FP8_E4M3 and HS2_FP4_E2M1 only (else NULL): float32
 *              [num_pages][Hkv]; FP8: a stored E4M3 code c of page p, KV head g stands for
 *              c * scale[p][g].
 * k_sf, v_sf:  HS2_FP4_E2M1 only (else NULL): uint8 E4M3 codes [num_pages][Hkv][page_size]
 *              [d/16], one per 16 channels of a row ([CSA2] §3, "KV 字节与 FP4": E2M1 main KV
 *              with an E4M3 scale per 16 channels). k and v then hold [num_pages][Hkv]
 *              [page_size][d/2] bytes, channel 2i in the low nibble of byte i (E2M1: sign,
 *              2 exponent bits with bias 1, 1 mantissa bit); channel c of a row stands for
 *              e2m1(code) * e4m3(sf[c / 16]) * scale[p][g].
 *              FP8 and FP4 caches are written and read back by hs2_kv_write / hs2_kv_read,
 *              and read by hs2_fa_select (decode), hs2_sa_reuse (decode) and hs2_fa_chunk;
 *              queries are bf16; the prefill selection and the KV append refuse them.
 * page_size must be 64; d must be 64 or 128, in a latent cache 576 or 320 (hs2_latent_write;
 *              hs2_pages_fork and hs2_pages_compact take those too).                    */
typedef struct {
  const void* k;
  const void* v;
  const int32_t* block_table;
  const int32_t* seq_len;
  int32_t batch;
  int32_t num_pages;
  int32_t max_pages;
  int32_t page_size;
  int32_t Hkv;
  int32_t d;
  hs2_dtype dtype;
  const float* k_scale;
  const float* v_scale;
  const uint8_t* k_sf;
  const uint8_t* v_sf;
} hs2_kv;

/* ---------------------------------------------------------------------------
 * FA layer + window-excluding top-k selection  ([HS2] §5, §7.2; the "oracle"
 * selection of the appendix: the FA's own exactly computed attention scores).
 *
 * decode (prefill = 0): one query per sequence; q is [batch][Hq][d] of kv->dtype,
 *   B_or_n must equal kv->batch; query b sees t_b = seq_len[b] keys.
 * prefill (prefill = 1): one sequence (kv->batch == 1), n = B_or_n query rows,
 *   q is [n][Hq][d]; row i sees t_i = i + 1 keys; requires n <= seq_len[0].
 *
 * Per query and head h: x_h(s) = scale * q_h . k_g(s) for s < t;
 *   o[..][h][:] = sum_s softmax(x_h)(s) v_g(s);  lse[..][h] = log sum_s exp x_h(s).
 * Per query and KV head g: score_g(s) = sum_{h in g} exp(x_h(s) - lse_h) over
 *   s in F(t); idx[..][g][:] = the min(k, |F|) best positions (score descending,
 *   lower position first on ties), ascending, -1 padded; idx_cnt[..][g] = count.
 * Outputs: o float32 [B_or_n][Hq][d]; lse float32 [B_or_n][Hq] (may be NULL);
 *   idx int32 [B_or_n][Hkv][k]; idx_cnt int32 [B_or_n][Hkv].
 * workspace: device scratch of at least hs2_fa_select_workspace(...) bytes,
 *   256-byte aligned; contents on entry are ignored.
 * max_t: the largest seq_len of the call (decode) or n (prefill).
 * Requirements: Hq % Hkv == 0, Hq / Hkv <= 32, k >= 0, w >= 0.                     */
size_t hs2_fa_select_workspace(int B_or_n, int Hq, const hs2_kv* kv, int max_t, int k, int prefill);
hs2_status hs2_fa_select(const void* q, int B_or_n, int Hq, const hs2_kv* kv, int max_t, int w,
                         int k, float scale, int prefill, float* o, float* lse, int32_t* idx,
                         int32_t* idx_cnt, void* workspace, size_t ws_bytes, int32_t* dev_err,
                         void* stream);

/* hs2_fa_select with block-level selection, the first HySparse version's scheme ([HS2] §2:
 * 16 blocks of 64 tokens = 1024 positions). sel_block = 1 is hs2_fa_select. sel_block > 1
 * (decode only; sel_block a multiple of 4, at most 4096, and k a multiple of sel_block): far position s belongs to
 * block s / sel_block, a block's key is the largest selection score among its far
 * positions, and the min(k / sel_block, #blocks) best blocks by (key descending, block
 * ascending) are taken whole: idx holds their far positions ascending (-1 padded),
 * idx_cnt their number. Prefill with sel_block > 1: HS2_ERR_UNSUPPORTED. The workspace
 * size is hs2_fa_select_workspace's. */
hs2_status hs2_fa_select_ex(const void* q, int B_or_n, int Hq, const hs2_kv* kv, int max_t, int w,
                            int k, float scale, int prefill, int sel_block, float* o, float* lse,
                            int32_t* idx, int32_t* idx_cnt, void* workspace, size_t ws_bytes,
                            int32_t* dev_err, void* stream);

/* ---------------------------------------------------------------------------
 * Decode KV append  ([HS2] §10.1, step 3: once the source hidden state is ready, each
 * Cross group's cache gains one entry; §4.2: the groups' KV branches are independent).
 * The new token is the last visible key of its sequence: for every cache c < n_caches and
 * sequence b < kvs[c].batch, with t = kvs[c].seq_len[b] (already counting the new token),
 *   K row t-1 of KV head g  <-  k_new[c][b][g][:]   (and V likewise from v_new[c]),
 * i.e. slot (t-1) % 64 of page block_table[b][(t-1) / 64]. One launch for all caches.
 * kvs: host array of n_caches descriptors (1 <= n_caches <= 8), bf16 or f32 pools; an FP8
 *   or FP4 pool returns HS2_ERR_UNSUPPORTED (hs2_kv_write quantises). A key-only
 *   cache (v = NULL, e.g. a CSA2 indexer-key cache) takes k_new only.
 * k_new, v_new: host arrays of n_caches device pointers, each [batch][Hkv][d] in the
 *   cache's dtype, 16-byte aligned; v_new may be NULL when every cache is key-only.
 * The pools are written through the descriptors' k / v pointers, which must therefore be
 *   writable device memory owned by the caller. The page holding position t-1 must belong
 *   to that sequence alone for the duration of the call.
 * Device-side: t < 1 or t > 64 * max_pages sets HS2_DEV_BAD_LENGTH, a block-table entry
 *   outside [0, num_pages) sets HS2_DEV_BAD_PAGE; that sequence's rows are not written. */
hs2_status hs2_kv_append(int n_caches, const hs2_kv* kvs, const void* const* k_new, const void* const* v_new,
                         int32_t* dev_err, void* stream);

/* Decode FA + selection with the current token's K/V append fused in (hs2_fa_select_ex,
 * decode only, plus hs2_kv_append of one cache): k_new / v_new [batch][Hq / G = Hkv][d]
 * (device, kv->dtype, 16-byte aligned) are written to position t-1 as hs2_kv_append does,
 * and the scan uses them for key t-1. On the bf16 tensor-core scan the write happens inside
 * the scan kernel, which takes key t-1 from k_new / v_new rather than the pool; otherwise
 * (f32, or a head-sharing factor that path does not take) a separate append kernel runs
 * first on the same stream. Outputs equal those of hs2_kv_append followed by
 * hs2_fa_select_ex. FP8 pools: HS2_ERR_UNSUPPORTED. The workspace size is
 * hs2_fa_select_workspace(B, Hq, kv, max_t, k, 0). */
hs2_status hs2_fa_select_append(const void* q, int B, int Hq, const hs2_kv* kv, int max_t, int w, int k,
                                float scale, int sel_block, const void* k_new, const void* v_new, float* o,
                                float* lse, int32_t* idx, int32_t* idx_cnt, void* workspace, size_t ws_bytes,
                                int32_t* dev_err, void* stream);

/* ---------------------------------------------------------------------------
 * hs2_fa_select_noalloc — hs2_fa_select for callers that cannot allocate device
 * memory (an engine that has reserved nearly all HBM for its KV pool and forbids
 * further cudaMalloc, or a latency-critical thread that must not call cudaMalloc /
 * cudaFree because they can synchronise the device). It takes no workspace: its
 * scratch is a file-scope device array of hs2_fa_select_noalloc_capacity() bytes
 * (64 MiB) that every GPU loading the library holds until the process exits. The
 * pages have no counterpart to this entry point; it is a deployment convenience.
 * Arguments, outputs and results are exactly those of hs2_fa_select.
 * - Returns HS2_ERR_SCRATCH_LIMIT, launching nothing, when
 *   hs2_fa_select_workspace(...) of the call exceeds the capacity.
 * - The first call on a device looks up the array's device address on that device
 *   (it must be the current device); make that first call before any stream capture.
 *   The address is looked up again when the device's current context has changed since
 *   (after a cudaDeviceReset, say); make the first call after such a change before any
 *   stream capture too.
 * - All calls share the one array: calls that overlap on the GPU (concurrent streams
 *   or host threads) race and corrupt each other's results; serialise them.
 * - It allocates nothing and calls no cudaMalloc / cudaFree.                        */
size_t hs2_fa_select_noalloc_capacity(void);
hs2_status hs2_fa_select_noalloc(const void* q, int B_or_n, int Hq, const hs2_kv* kv, int max_t, int w,
                                 int k, float scale, int prefill, float* o, float* lse, int32_t* idx,
                                 int32_t* idx_cnt, int32_t* dev_err, void* stream);

/* ---------------------------------------------------------------------------
 * SA layer: KV and index reuse with the layer's own query  ([HS2] §5, §7.2, §7.4).
 * For each query and head h of KV head g:
 *   U = W(t) ∪ {idx[..][g][j] : j < idx_cnt[..][g]}   (the caller guarantees the
 *   indices lie in F(t), i.e. outside the window; with w = 0 any s < t),
 *   o[..][h][:] = sum_{s in U} softmax_U(scale * q_h . k_g(s)) v_g(s), one softmax.
 * Shapes and the decode / prefill convention are those of hs2_fa_select; idx and
 * idx_cnt have the layout hs2_fa_select writes ([B_or_n][Hkv][k], [B_or_n][Hkv]).
 * workspace: at least hs2_sa_reuse_workspace(...) bytes, 256-byte aligned, no
 *   initialisation needed; calls that run at the same time need workspaces of their own. */
size_t hs2_sa_reuse_workspace(int B_or_n, int Hq, const hs2_kv* kv, int w, int k, int prefill);
hs2_status hs2_sa_reuse(const void* q, int B_or_n, int Hq, const hs2_kv* kv, int w,
                        const int32_t* idx, const int32_t* idx_cnt, int k, float scale, int prefill,
                        float* o, void* workspace, size_t ws_bytes, int32_t* dev_err, void* stream);

/* hs2_sa_reuse with the SA layers' per-head sink bias and output sigmoid gate
 * ([HS2] §17.1). sink: float32 [Hq] natural-log logits, or NULL: one more key per head
 * with logit sink[h] and a zero value, i.e. the single softmax denominator over W ∪ S
 * gains exp(sink[h]) (-inf = no sink). gate: float32 [B_or_n][Hq][d] logits, or NULL:
 * the output is multiplied elementwise by 1 / (1 + exp(-gate)). Both are read-only,
 * device memory, owned by the caller.
 * flags: 0 or HS2_SA_OVERLAP. The decode kernel is always launched so that it may start
 *   while the previous launch on `stream` finishes (programmatic dependent launch), and
 *   waits for that launch before it reads anything. HS2_SA_OVERLAP (decode) is for the SA
 *   layers of a group after the first, each issued right after the one before it:
 *   - the call reads idx, idx_cnt, kv->block_table and kv->seq_len before that wait, so
 *     those four must have been complete before the previous launch on the stream began
 *     (not written by it);
 *   - `workspace` must be the one the previous hs2_sa_reuse call on this stream used,
 *     with the same B_or_n, Hq, kv sizes, w and k: the call keeps the state that call
 *     left in it instead of clearing it, and makes no launch but its kernel.
 *   Prefill ignores the flag; other bits: HS2_ERR_ARG.
 * Everything else as hs2_sa_reuse (which is this call with sink = gate = NULL, flags = 0);
 * the workspace size does not change. */
#define HS2_SA_OVERLAP 1
hs2_status hs2_sa_reuse_ex(const void* q, int B_or_n, int Hq, const hs2_kv* kv, int w,
                           const int32_t* idx, const int32_t* idx_cnt, int k, float scale, int prefill,
                           const float* sink, const float* gate, int flags, float* o, void* workspace,
                           size_t ws_bytes, int32_t* dev_err, void* stream);

/* ---------------------------------------------------------------------------
 * CSA2 hierarchical sparse indexer  ([CSA2] §3.1-3.2; score from [L10] §5.1).
 * I(s) = sum_j w_idx[b][j] * max(0, q_idx[b][j] . k_idx(s)), unscaled, where k_idx(s)
 * is row s of the indexer-key cache k_idx (Hkv = 1, d = di, v = NULL), shared by
 * all Hi indexer heads.
 * HS2_FULL: score every s < t; idx[b] = top-min(k_top, t) positions; block maxima
 *   over blocks [blk*j, blk*j+blk) ∩ [0,t); pool_blocks[b] = top-min(max_blocks,
 *   ceil(t/blk)) block ids (maximum descending, lower id first), ascending, -1
 *   padded; pool_cnt[b] = count.  (pool_blocks / pool_cnt are outputs.)
 * HS2_REINDEX: score only the positions of the given pool (inputs pool_blocks /
 *   pool_cnt); idx[b] = top-min(k_top, |pool positions|), ascending.
 * (Reuse layers call nothing: they pass the previous idx to hs2_sa_reuse.)
 * q_idx: [batch][Hi][di] of k_idx->dtype; w_idx: float32 [batch][Hi];
 * idx: int32 [batch][k_top]; idx_cnt: int32 [batch]; blk must divide page_size.
 * workspace: at least hs2_hier_reindex_workspace(...) bytes, 256-byte aligned.     */
typedef enum { HS2_FULL = 0, HS2_REINDEX = 1 } hs2_idx_mode;
size_t hs2_hier_reindex_workspace(hs2_idx_mode mode, int Hi, const hs2_kv* k_idx, int max_t,
                                  int k_top, int blk, int max_blocks);
hs2_status hs2_hier_reindex(hs2_idx_mode mode, const void* q_idx, const float* w_idx, int Hi,
                            const hs2_kv* k_idx, int max_t, int k_top, int blk, int max_blocks,
                            int32_t* pool_blocks, int32_t* pool_cnt, int32_t* idx, int32_t* idx_cnt,
                            void* workspace, size_t ws_bytes, int32_t* dev_err, void* stream);

/* ---------------------------------------------------------------------------
 * Rows into and out of a paged cache, for prompts and single tokens.
 * A call covers a ragged batch: row_start is int32 [batch + 1] (device), ascending from
 * row_start[0] >= 0; rows [row_start[b], row_start[b+1]) of the packed row arrays belong to
 * sequence b and are its LAST n_b = row_start[b+1] - row_start[b] positions, t_b - n_b ..
 * t_b - 1 with t_b = seq_len[b] (already counting them; n_b = 0 is a sequence that takes no
 * part, whatever its length and table). n_rows is the number of rows the arrays hold; rows
 * outside [row_start[0], row_start[batch]) are neither read nor written.
 * k_rows, v_rows: [n_rows][Hkv][d] of row_dtype (HS2_F32 or HS2_BF16), token r at
 *   r * row_stride elements (row_stride >= Hkv * d: slices of a fused projection's output
 *   fit), 16-byte aligned, row_stride * sizeof(element) a multiple of 16. v_rows is ignored
 *   for a key-only cache (kv->v = NULL); K and V rows of different strides take two calls,
 *   each on one side as a key-only cache.
 *
 * hs2_kv_write stores the rows in the cache's type:
 *   F32 / BF16: the value, rounded to nearest even where bfloat16 is narrower.
 *   FP8: code = E4M3(x / S), S = scale[page][g], nearest even, saturating at +-448; NaN is NaN.
 *   FP4: per group of 16 channels the scale s = the smallest E4M3 value with 6 s S >= max|x|
 *     (448 where none is), then code = E2M1(x / (s S)), nearest even, saturating at +-6. A
 *     group holding a NaN stores s = NaN, i.e. all its 16 values read as NaN.
 *   Every code is the one exact arithmetic gives. k_scale / v_scale (one per page and KV
 *   head) are inputs: they are set before rows are written and apply to a page's older rows
 *   too. S outside [2^-60, 2^60] (or NaN): HS2_DEV_BAD_PAGE, and the row's part under that
 *   scale (its KV head's K, or V) is not written.
 *   The pages written must belong to their sequence alone.
 * hs2_kv_read writes the values those positions stand for to k_rows / v_rows (FP8 / FP4:
 *   code * scales in float32, rounded once; then to bfloat16 where that is row_dtype).
 * Device-side: t_b beyond max_pages * page_size, n_b > t_b, a sequence with rows outside
 *   [0, n_rows) or a descending row_start sets HS2_DEV_BAD_LENGTH, a table entry outside
 *   [0, num_pages) HS2_DEV_BAD_PAGE; such sequences' rows are left as they were (in the
 *   cache, or in k_rows / v_rows; of a bad entry the rows of its page; where a start falls,
 *   all or only some rows of the sequences about it are). */
hs2_status hs2_kv_write(const hs2_kv* kv, const void* k_rows, const void* v_rows, hs2_dtype row_dtype,
                        int64_t row_stride, const int32_t* row_start, int n_rows, int32_t* dev_err, void* stream);
hs2_status hs2_kv_read(const hs2_kv* kv, void* k_rows, void* v_rows, hs2_dtype row_dtype, int64_t row_stride,
                       const int32_t* row_start, int n_rows, int32_t* dev_err, void* stream);

/* ---------------------------------------------------------------------------
 * Attention of a ragged batch of query chunks over the cache: a prompt chunk, draft tokens
 * under verification, single tokens, or any mixture ([HS2] §8: prompt rows pass through the
 * Self-Decoder's FA and sliding-window layers, which select nothing). Rows are laid out as
 * in hs2_kv_write: q is [n_rows][Hq][d] (bf16; float32 with an F32 cache), row r of sequence
 * b is its position p = t_b - n_b + (r - row_start[b]), whose key is already in the cache.
 * Head h of KV head g attends to the keys s in (p - w, p] (w = 0: s in [0, p]):
 *   x(s) = scale * q_h . k_g(s);  Z = sum_s exp x(s) + exp(sink[h]);
 *   o = sum_s exp x(s) v_g(s) / Z;  lse = log Z.
 * max_n, max_t: at least the largest n_b and t_b of the call. sink: float32 [Hq] natural-log
 * logits, or NULL (no sink). o: [n_rows][Hq][d] of o_dtype (HS2_F32 or HS2_BF16); lse:
 * float32 [n_rows][Hq], may be NULL. scale > 0. All cache types; d 64 or 128; Hq / Hkv a
 * power of two up to 32.
 * Keys in pages whose table entry is bad are left out (HS2_DEV_BAD_PAGE; a row with no key
 * left and no sink gets o = 0, lse = -inf). A sequence whose n_b > max_n, t_b > max_t,
 * n_b > t_b, or rows beyond n_rows, sets HS2_DEV_BAD_LENGTH and its rows are not written
 * (a descending row_start: none or only some rows are). With n_rows = 0 or max_n = 0 nothing
 * is launched and nothing flagged. HS2_ERR_UNSUPPORTED: pools of 2^31 rows (num_pages * Hkv *
 * 64) or more, and declared sizes of more than 2^30 tiles (max_t / 128 + 2 for every 16 to 256
 * of the n_rows * Hq rows and every sequence's KV head).
 * The weights enter P.V rounded to 16 bits whatever o_dtype is (float32 caches: not rounded): to
 * bfloat16, or, with few rows per KV head over an FP8 / FP4 cache, weight times V scale to float16
 * relative to the row's largest, of which 2^-30 and less is lost. Their sum and lse are float32.
 * V scales may differ from page to page; magnitudes in [2^-60, 2^60], or 0.
 * Logits x(s) of finite inputs are taken to stay below 2^26 in magnitude (float32 caches: any):
 * beyond, their float32 form has no fraction left and a row can come out as NaN or 0.
 * A V row that is not finite can make every row of its sequence in the call undefined, as a
 * weight of zero does not cancel it in the rows that share its tile; values behind seq_len do
 * not matter. A NaN in a K row or a query, or a logit of +inf, gives NaN in the rows that see
 * it; a logit of -inf is a weight of 0.
 * workspace: at least hs2_fa_chunk_workspace(...) bytes, 256-byte aligned, contents ignored;
 * what it gives for some n_rows, max_n and max_t also suffices where any of them is smaller
 * (same Hq, kv and w). Calls that run at the same time need workspaces of their own.
 * Calls of many rows over an FP8 / FP4 cache keep bf16 copies of the pages there: up to
 * batch * min(max_t, max_n + w) * Hkv * d * 4 bytes (w = 0: batch * max_t ...), so max_n and
 * max_t are best kept close to what the batch holds.                                     */
size_t hs2_fa_chunk_workspace(int n_rows, int Hq, const hs2_kv* kv, int max_n, int max_t, int w);
hs2_status hs2_fa_chunk(const void* q, const int32_t* row_start, int n_rows, int max_n, int Hq, const hs2_kv* kv,
                        int max_t, int w, float scale, const float* sink, void* o, hs2_dtype o_dtype, float* lse,
                        void* workspace, size_t ws_bytes, int32_t* dev_err, void* stream);

/* ---------------------------------------------------------------------------
 * Rows rotated by their positions on the way into a cache (rotary position embedding).
 * hs2_rot: table float32 [n_pos][dim] (device, 16-byte aligned): row p has the cosines of position
 * p's dim / 2 angles, then their sines. The first dim channels of a head are rotated (dim a
 * multiple of 32 up to d), in pairs (a, b) = (x_i, x_{i + dim/2}), with pairs = 1 (x_2i, x_2i+1):
 *   a' = a cos_i - b sin_i,  b' = b cos_i + a sin_i,
 * every product and sum rounded to float32 by itself, then the result to where it goes. */
typedef struct {
  const float* table;
  int32_t n_pos;
  int32_t dim;
  int32_t pairs;
} hs2_rot;

/* hs2_kv_write with K, and optionally the queries of the same rows, rotated: rows, positions, types
 * and errors as there; K and V rows have a token stride each (strides here and below: at most 2^31
 * elements). q: [n_rows][Hq][d] of row_dtype, token r
 * at r * q_stride elements, or NULL with Hq = 0; q_out: the rotated queries as hs2_fa_chunk takes
 * them, float32 for an F32 cache, else bfloat16, [n_rows][Hq][d] at q_out_stride; it may be q itself
 * (same type and stride) and overlaps nothing else. Rows that are flagged or outside every sequence have
 * neither their cache rows nor their q_out written; but under a slab scale out of range only the part
 * that hs2_kv_write leaves out is, not the row's other heads, its other side or its q_out. A position
 * of n_pos or more sets HS2_DEV_BAD_INDEX. n_rows = 0: nothing to do, q and q_out may be NULL. All cache types. */
hs2_status hs2_kv_write_rot(const hs2_kv* kv, const void* k_rows, int64_t k_stride, const void* v_rows, int64_t v_stride,
                            hs2_dtype row_dtype, const int32_t* row_start, int n_rows, const hs2_rot* rot, const void* q,
                            int64_t q_stride, int Hq, void* q_out, int64_t q_out_stride, int32_t* dev_err, void* stream);

/* ---------------------------------------------------------------------------
 * Latent attention: keys and values of all heads from one latent vector a token, plus a key part
 * that carries the position.
 * A latent cache is an hs2_kv with v = NULL, Hkv = 1 and d = dc + 64, dc 512 or 256: a row is dc
 * latent channels c and 64 rotated channels r. F32 or BF16; FP8 / FP4: HS2_ERR_UNSUPPORTED.
 *
 * hs2_latent_write stores c_rows ([n_rows][dc]) as they are and r_rows ([n_rows][64]) rotated (rot->dim
 * must be 64), and writes the queries' rotated part q ([n_rows][Hq][64], or NULL with Hq = 0) to
 * q_out, of the cache's type. Token r of an array is at r times its stride (elements), head h of q and
 * q_out at h times q_head / q_out_head; all 16-byte aligned with strides of a multiple of 16 bytes.
 * q_out is typically the last 64 channels of [n_rows][Hq][dc + 64]; it may be q itself.
 * hs2_latent_read gets rows back (c and r of row_dtype; r as stored, rotated), e.g. to expand them.
 * Rows, positions and errors as in hs2_kv_write / hs2_kv_read / hs2_kv_write_rot. */
hs2_status hs2_latent_write(const hs2_kv* kv, const void* c_rows, int64_t c_stride, const void* r_rows, int64_t r_stride,
                            hs2_dtype row_dtype, const int32_t* row_start, int n_rows, const hs2_rot* rot, const void* q,
                            int64_t q_stride, int64_t q_head, int Hq, void* q_out, int64_t q_out_stride,
                            int64_t q_out_head, int32_t* dev_err, void* stream);
hs2_status hs2_latent_read(const hs2_kv* kv, void* c_rows, int64_t c_stride, void* r_rows, int64_t r_stride,
                           hs2_dtype row_dtype, const int32_t* row_start, int n_rows, int32_t* dev_err, void* stream);

/* hs2_latent_chunk, the absorbed form: causal attention of a ragged batch of query chunks over a
 * latent cache, rows as in hs2_fa_chunk. q: [n_rows][Hq][dc + 64] of the cache's type, the queries
 * taken into the latent space and their rotated part. Row at position p, head h:
 *   x(s) = scale * q_h . [c_s, r_s], s <= p;  o = sum_s softmax(x)(s) c_s;  lse = log sum_s exp x(s).
 * o: [n_rows][Hq][dc] of o_dtype (HS2_F32 or HS2_BF16), lse float32 [n_rows][Hq] or NULL. Hq a power
 * of two up to 128. max_n and max_t, bad pages and lengths, values that are not finite, sizes and
 * workspace (hs2_latent_chunk_workspace(...) bytes): as hs2_fa_chunk. BF16 caches: the weights enter the
 * second product rounded to bfloat16; float32 caches: not rounded. */
size_t hs2_latent_chunk_workspace(int n_rows, int Hq, const hs2_kv* kv, int max_n, int max_t);
hs2_status hs2_latent_chunk(const void* q, const int32_t* row_start, int n_rows, int max_n, int Hq, const hs2_kv* kv,
                            int max_t, float scale, void* o, hs2_dtype o_dtype, float* lse, void* workspace,
                            size_t ws_bytes, int32_t* dev_err, void* stream);

/* hs2_latent_prefill, the expanded form: the same attention with K and V of every head expanded from
 * the latents, for prompts (a fifth to a third of the absorbed form's operations per key). Keys are
 * packed like rows: sequence b has keys [key_start[b], key_start[b+1]) and its rows
 * [row_start[b], row_start[b+1]) are its LAST positions. Head h:
 *   x(s) = scale * (q_h[0:128] . k_{s,h} + q_h[128:192] . r_s),  o = sum_s softmax(x)(s) v_{s,h}.
 * hs2_latent_keys: k, v [n_keys][Hq][128] with token and head strides (elements; slices of the
 * expansion's output fit), r [n_keys][64] shared by the heads; HS2_F32 or HS2_BF16, 16-byte aligned
 * with strides of a multiple of 16 bytes. q: [n_rows][Hq][192] of the same type; o:
 * [n_rows][Hq][128] of o_dtype. A sequence with n_b > max_n, more keys than max_t, fewer keys than rows,
 * or rows or keys outside the arrays sets HS2_DEV_BAD_LENGTH and its rows are not written (a
 * descending row_start or key_start: none or only some rows are). Precision as hs2_latent_chunk; a V row
 * that is not finite can make every row of its sequence undefined, what lies outside every sequence
 * does not matter. HS2_ERR_UNSUPPORTED: n_keys above 2^31 - 257, and declared sizes of more than 2^30
 * tiles (max_t / 128 + 2 for every 256 of the n_rows rows and every sequence, times Hq). workspace: at
 * least hs2_latent_prefill_workspace(...) bytes, as there. */
typedef struct {
  const void* k;
  const void* r;
  const void* v;
  int64_t k_token, k_head, r_token, v_token, v_head;
  const int32_t* key_start; /* [batch + 1] */
  int32_t n_keys;
  hs2_dtype dtype;
} hs2_latent_keys;
size_t hs2_latent_prefill_workspace(int n_rows, int Hq, int batch, int max_n, int max_t);
hs2_status hs2_latent_prefill(const void* q, const int32_t* row_start, int n_rows, int max_n, int Hq, int batch,
                              const hs2_latent_keys* keys, int max_t, float scale, void* o, hs2_dtype o_dtype, float* lse,
                              void* workspace, size_t ws_bytes, int32_t* dev_err, void* stream);

/* ---------------------------------------------------------------------------
 * Pages of a pool: room for sequences, branches that share pages, defragmentation. All on
 * the device: no call returns a count to the host, and results do not depend on timing.
 * hs2_pages: device arrays of the caller's; ref[p] is the number of table entries that hold
 * page p (0: free), free_list[0 .. *n_free) the free pages, taken from its end. The caches
 * whose pages are numbered alike (the K/V pools of several groups) share one hs2_pages and
 * one block table: kvs lists them (1 <= n_caches <= 8), with the same block_table, seq_len,
 * batch, max_pages, num_pages (= pages->num_pages) and page_size.
 * A call runs alone on its pool's books: calls on one hs2_pages are issued on one stream or
 * ordered by events. All are captured and replayed like any launch. */
typedef struct {
  int32_t* ref;       /* [num_pages] */
  int32_t* free_list; /* [num_pages] */
  int32_t* n_free;    /* [1] */
  int32_t num_pages;
} hs2_pages;

/* hs2_pages_grow: seq_len[b] += n_new[b] (n_new >= 0) for every sequence, and entries
 * [ceil(old / 64), ceil(new / 64)) of block_table[b] ([batch][max_pages]) take free pages
 * (ref 1) in order of (b, entry). All or nothing: where the free pages do not suffice for
 * every sequence, HS2_DEV_BAD_PAGE is set and nothing changes. A sequence with n_new < 0, a
 * negative length, or a new length beyond max_pages * 64 sets HS2_DEV_BAD_LENGTH and stays
 * as it was. */
hs2_status hs2_pages_grow(const hs2_pages* pages, int32_t* block_table, int32_t* seq_len, const int32_t* n_new,
                          int batch, int max_pages, int32_t* dev_err, void* stream);
/* hs2_pages_free: every page of block_table[b][0 .. ceil(seq_len[b] / 64)) loses a reference
 * where drop[b] != 0; pages left with none go to the end of the free list in ascending
 * order. Tables and lengths are not written. An entry outside [0, num_pages) or without a
 * reference left sets HS2_DEV_BAD_PAGE and is skipped; a length outside [0, max_pages * 64]
 * sets HS2_DEV_BAD_LENGTH and its sequence is skipped. */
hs2_status hs2_pages_free(const hs2_pages* pages, const int32_t* block_table, const int32_t* seq_len,
                          const int32_t* drop, int batch, int max_pages, int32_t* dev_err, void* stream);
/* hs2_pages_fork: branch c < n_child becomes a sequence of its own with the keys of sequence
 * src[c] of the caches (several branches may have one source; src[c] = -1: none, length 0).
 * child_table ([n_child][max_pages]) shares the source's full pages (ref + 1); the rows of a
 * last, partly filled page, and its scales, are copied in every cache to a page taken from
 * the free list, in order of c. child_len[c] = seq_len[src[c]]; other table entries are -1.
 * child_table and child_len do not overlap the sources'. Where the free pages do not
 * suffice, HS2_DEV_BAD_PAGE is set and every branch has length 0 and no pages. src outside
 * [-1, batch) sets HS2_DEV_BAD_INDEX, a source length outside [0, max_pages * 64]
 * HS2_DEV_BAD_LENGTH: that branch is none. A source's bad table entry (out of range, or a
 * page without a reference) sets HS2_DEV_BAD_PAGE and is -1 in the branch (a bad last page:
 * nothing is copied to the branch's own). */
hs2_status hs2_pages_fork(const hs2_pages* pages, int n_caches, const hs2_kv* kvs, const int32_t* src, int n_child,
                          int32_t* child_table, int32_t* child_len, int32_t* dev_err, void* stream);
/* hs2_pages_compact: with L referenced pages, moves every referenced page >= L into a free
 * page < L, in place (i-th free page ascending takes the i-th such page ascending), in every
 * cache with its scales, and updates the references, the free list (the pages >= L, the
 * lowest taken first; entries behind are -1) and the entries of the caches' block table
 * below ceil(seq_len[b] / 64). That table must hold every sequence that has pages of the
 * pool. Bad entries (out of range, or of a free page: HS2_DEV_BAD_PAGE) and the rows of
 * sequences with a bad length (HS2_DEV_BAD_LENGTH) are left as they are.
 * workspace: at least hs2_pages_compact_workspace(pages) bytes, 256-byte aligned, contents
 * ignored. */
size_t hs2_pages_compact_workspace(const hs2_pages* pages);
hs2_status hs2_pages_compact(const hs2_pages* pages, int n_caches, const hs2_kv* kvs, void* workspace,
                             size_t ws_bytes, int32_t* dev_err, void* stream);

/* ---------------------------------------------------------------------------
 * Diagnostics.
 * hs2_profile_next: the next call on this host thread that runs `stage` records the
 * cudaEvent_t handles `start` and `stop` (passed as void*, created by the caller) on
 * that call's stream immediately before and after the stage's main kernel; one-shot,
 * NULL events clear it. Lets a caller time the dominant kernel inside a running step. */
typedef enum {
  HS2_STAGE_FA_SCAN = 0,    /* FA scan over all visible keys (hs2_fa_select) */
  HS2_STAGE_SA_GATHER = 1,  /* SA gather-attention (hs2_sa_reuse) */
  HS2_STAGE_INDEXER = 2     /* lightning-indexer scan (hs2_hier_reindex) */
} hs2_stage;
void hs2_profile_next(hs2_stage stage, void* start, void* stop);
/* hs2_selftest_wait_timeout: launches one warp that waits, through the library's bounded
 * mbarrier wait and with a limit of timeout_us microseconds (1 .. 2000000), on a barrier nothing
 * arrives on; the wait gives up, HS2_DEV_TIMEOUT is set in *dev_err (device memory) and the
 * kernel finishes. Lets a caller check the device-side timeout path without a fault. */
hs2_status hs2_selftest_wait_timeout(int timeout_us, int32_t* dev_err, void* stream);
/* hs2_fa_select_launches / hs2_sa_reuse_launches: how many kernels hs2_fa_select_ex (with
 * append != 0: hs2_fa_select_append) and hs2_sa_reuse_ex launch for these arguments (device
 * memsets not counted), or -1 for arguments they reject on the host. Lets a caller account
 * for the library's launches inside a step; launches nothing (it may query the current
 * device's properties, as the calls themselves do to plan their grids). */
int hs2_fa_select_launches(int B_or_n, int Hq, const hs2_kv* kv, int max_t, int w, int k, int prefill,
                           int sel_block, int append);
int hs2_sa_reuse_launches(int B_or_n, int Hq, const hs2_kv* kv, int w, int k, int prefill);
const char* hs2_strerror(hs2_status st);
int hs2_last_cuda_error(void); /* cudaError_t of the last HS2_ERR_CUDA, 0 if none */
int hs2_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* HS2_H */
