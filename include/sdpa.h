/*
 * sdpa.h -- C ABI of the GB300 (sm_103a) fused scaled dot-product attention
 * forward.
 *
 * OPERATION.  For every (batch b, head h) and query row i:
 *
 *     out[b,h,i,:] = sum_j softmax_j( scale * q[b,h,i,:] . k[b,h,j,:]
 *                                     with removed keys at -inf ) * v[b,h,j,:]
 *
 * i.e. the five steps matmul(q, k^T), times scale, masked_fill(mask, -inf),
 * softmax over keys, matmul(attn, v) of the NaiveCausalAttention module in
 * "Profiling attention in PyTorch: kernels, backends and where the time goes"
 * (news.bpdata.com), section "Naiv causal attention", and of section 1 of
 * "PyTorch attention profiling: Flash, cuDNN and Math backends compared"
 * (dev.smart-guide.co.kr).  The user-facing call there is
 * F.scaled_dot_product_attention(q, k, v, is_causal=True) (same pages, SDPA
 * sections); this ABI takes the same arguments as raw device pointers.
 *
 *   - causal (is_causal != 0): query i sees keys j <= i.
 *   - explicit mask: mask[i*L + j] != 0 removes key j for query i, the
 *     masked_fill polarity (1 = masked out).  One [L, L] mask serves every
 *     (b, h).
 *   - a query with no admissible key yields a zero row (the math backend's
 *     "safe softmax", same pages, math-backend sections), never NaN.
 *   - rank-3 inputs [H, L, D] are treated as rank-4 [1, H, L, D] and reach the
 *     same fused kernel ("PyTorch 2.14 SDPA: rank-3 inputs now take the fused
 *     kernels", daker.dacon.io, sections on the rank-3 problem and on what
 *     changed in 2.14); results are bit-identical to the rank-4 call.
 *
 * Computation: one GPU kernel launch per call, launched with programmatic
 * stream serialization (its set-up overlaps the previous kernel in the
 * stream, its first global-memory access waits for that kernel); 16-bit
 * inputs on tensor cores
 * with fp32 accumulation, the softmax in fp32, probabilities rounded to the
 * input type before the second product, output rounded to nearest even.
 */
#ifndef SDPA_GB300_H
#define SDPA_GB300_H

#include <stdint.h>

#if defined(__GNUC__)
#define SDPA_API __attribute__((visibility("default")))
#else
#define SDPA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum sdpa_status {
  SDPA_OK = 0,
  SDPA_ERR_NULL = 1,            /* a required pointer argument is NULL */
  SDPA_ERR_RANK = 2,            /* rank is not 3 or 4 */
  SDPA_ERR_SHAPE = 3,           /* D not 64 or 128, or a dimension < 1, or too large */
  SDPA_ERR_DTYPE = 4,           /* dtype is not SDPA_BF16 / SDPA_FP16 */
  SDPA_ERR_LAYOUT = 5,          /* inner stride != 1, other strides not multiples of 8
                                   elements (16 bytes), zero stride on a dimension > 1,
                                   or a pointer not 16-byte aligned */
  SDPA_ERR_ARG = 6,             /* causal and mask both given, or out overlaps q/k/v/mask,
                                   or a NaN/inf scale other than the NaN default */
  SDPA_ERR_CUDA = 7,            /* the CUDA runtime/driver reported an error (launch,
                                   tensor-map encoding, no device) */
  SDPA_ERR_DEVICE_TIMEOUT = 8,  /* a kernel barrier wait ran out of time (see
                                   sdpa_last_device_status) */
  SDPA_ERR_DEVICE = 9           /* the current device is not an sm_103 GPU */
} sdpa_status;

typedef enum sdpa_dtype {
  SDPA_BF16 = 0,
  SDPA_FP16 = 1
} sdpa_dtype;

/*
 * sdpa_forward -- launch the fused attention forward on `stream`.
 *
 * q, k, v, out : DEVICE pointers to 16-bit elements of type `dtype`; all four
 *                share one logical shape.  The caller owns them; the call
 *                neither frees nor retains them.
 * rank         : 3 for [H, L, D], 4 for [B, H, L, D].
 * shape        : `rank` extents (host array).  D must be 64 or 128; L >= 1
 *                (any value, including ragged ones not divisible by 128).
 * *_stride     : `rank` strides in ELEMENTS (host arrays), so any strided view
 *                (for example a [B, L, H, D] buffer viewed as [B, H, L, D])
 *                is consumed in place with no transpose.  The innermost (D)
 *                stride must be 1; every other stride must be a multiple of
 *                8 elements and non-zero unless its extent is 1.
 * is_causal    : nonzero for the causal triangle.
 * mask         : NULL, or a DEVICE pointer to a dense row-major [L, L] byte
 *                matrix (nonzero = removed).  Not allowed together with
 *                is_causal.
 * scale        : multiplier of q.k; NaN selects the default 1/sqrt(D) (the
 *                module's scale on both profiling pages).
 * stream       : a cudaStream_t (NULL = legacy default stream).
 *
 * Returns SDPA_OK once the kernel is enqueued (asynchronous: results are
 * ready when the stream reaches it), or an error code.  Argument errors are
 * detected on the host before any CUDA call and launch nothing.  No device
 * memory is allocated per call.  Thread-compatible: concurrent calls must use
 * different streams.
 */
SDPA_API sdpa_status sdpa_forward(const void* q, const void* k, const void* v, void* out,
                         sdpa_dtype dtype, int rank, const int64_t* shape,
                         const int64_t* q_stride, const int64_t* k_stride,
                         const int64_t* v_stride, const int64_t* o_stride,
                         int is_causal, const uint8_t* mask, float scale, void* stream);

/*
 * Plans -- validate and encode once, launch many times.
 *
 * sdpa_forward validates its arguments and encodes three TMA descriptors on
 * every call.  A plan does that work once for a fixed shape, dtype, strides,
 * mask mode and scale (the same arguments and the same errors as
 * sdpa_forward); sdpa_plan_launch then only launches the kernel, which keeps
 * the host cost of a call to a few microseconds.  (The pages measure 117-214
 * us of CPU time per forward for the fused PyTorch backends, most of it
 * per-call plan selection for cuDNN: "Profiling attention in PyTorch:
 * kernels, backends and where the time goes", news.bpdata.com, section
 * "cuDNN backend".)
 *
 * sdpa_plan_create      : *plan receives a new plan (host memory owned by the
 *                         caller until sdpa_plan_destroy), or NULL on error.
 *                         Binds the plan to the current device.
 * sdpa_plan_set_pointers: rebinds q, k, v, out (and mask, which must be
 *                         present iff it was at creation) to new DEVICE
 *                         buffers of the same shape and strides; validated
 *                         like sdpa_forward.  Not thread-safe with a
 *                         concurrent launch of the same plan.
 * sdpa_plan_launch      : enqueues the forward on `stream` (asynchronous);
 *                         SDPA_ERR_ARG if the current device is not the
 *                         plan's.  Safe to call from several threads on
 *                         different streams, and inside CUDA graph capture.
 *                         A plan with a mask first launches the mask summary
 *                         (see sdpa_mask_tiles) into device memory the plan
 *                         allocated at creation (n^2 * 2049 bytes for n =
 *                         ceil(L / 128); SDPA_ERR_CUDA from sdpa_plan_create
 *                         when that allocation fails), then the forward,
 *                         which skips the key tiles that remove every key
 *                         for both query tiles of its job and reads 16 bytes
 *                         of mask per row and tile.  Concurrent launches of
 *                         one plan write identical summary bytes as long as
 *                         the mask's contents do not change meanwhile.
 * sdpa_plan_destroy     : frees the plan (NULL is ignored).  Work already
 *                         enqueued is unaffected.
 */
typedef struct sdpa_plan sdpa_plan;

SDPA_API sdpa_status sdpa_plan_create(sdpa_plan** plan, const void* q, const void* k,
                                      const void* v, void* out, sdpa_dtype dtype, int rank,
                                      const int64_t* shape, const int64_t* q_stride,
                                      const int64_t* k_stride, const int64_t* v_stride,
                                      const int64_t* o_stride, int is_causal,
                                      const uint8_t* mask, float scale);
SDPA_API sdpa_status sdpa_plan_set_pointers(sdpa_plan* plan, const void* q, const void* k,
                                            const void* v, void* out, const uint8_t* mask);
SDPA_API sdpa_status sdpa_plan_launch(const sdpa_plan* plan, void* stream);
SDPA_API void sdpa_plan_destroy(sdpa_plan* plan);

/*
 * sdpa_forward_masked_noalloc -- a masked forward that allocates nothing.
 *
 * The pages have no counterpart: this entry point is for callers that
 * cannot allocate device memory -- code that runs inside another runtime
 * whose memory pool has already reserved the device's memory, or a serving
 * loop that must not call cudaMalloc/cudaFree (they can synchronise the
 * whole device) -- but still want the masked fast path that a masked plan
 * gets from its summary buffer.  Here the mask summary (see sdpa_mask_tiles)
 * lives in one fixed array inside the library instead: 2,098,176 bytes of
 * device memory on every GPU that loads the library, held until the process
 * exits, enough for L <= SDPA_NOALLOC_MAX_L.
 *
 * Arguments as sdpa_forward with an explicit mask (no is_causal): mask must
 * be non-NULL (else SDPA_ERR_NULL); L > SDPA_NOALLOC_MAX_L returns
 * SDPA_ERR_SHAPE, the scratch array's limit; other errors as sdpa_forward.
 * The caller passes and owns q, k, v, out and mask; the call allocates no
 * device or pinned memory.  The first call on a device looks up the array's
 * device address on that device (it must be current, as for every call) and
 * caches it; make that first call before any stream capture.  The cached
 * address belongs to the device's context: after cudaDeviceReset the next
 * call finds that the context changed and looks the address up again (so
 * that call, too, belongs before any capture).  Every call
 * on a device uses the same array and leaves its last summary in it:
 * nothing there needs to start at zero, because each call rewrites every
 * byte it then reads, but calls whose work overlaps on the GPU (different
 * streams, or different threads) race on the array and must be ordered by
 * the caller.
 */
#define SDPA_NOALLOC_MAX_L 4096
SDPA_API sdpa_status sdpa_forward_masked_noalloc(const void* q, const void* k, const void* v,
                                                 void* out, sdpa_dtype dtype, int rank,
                                                 const int64_t* shape, const int64_t* q_stride,
                                                 const int64_t* k_stride,
                                                 const int64_t* v_stride,
                                                 const int64_t* o_stride, const uint8_t* mask,
                                                 float scale, void* stream);

/*
 * sdpa_mask_tiles -- the tile summary of an explicit mask (the mask-tile
 * skip bitmap masked plans use), written into caller-owned memory.
 *
 * The [L, L] mask (DEVICE, row-major bytes, nonzero = removed: the
 * masked_fill polarity of "Profiling attention in PyTorch: kernels, backends
 * and where the time goes", news.bpdata.com, section "Naiv causal attention") is cut
 * into n x n tiles of 128 x 128, n = ceil(L / 128).  For tile (qt, kt):
 *   tile_bits  : DEVICE, 16-byte aligned, n*n*128*16 bytes.  Row r of the
 *                tile is four 32-bit words at byte ((qt*n + kt)*128 + r)*16;
 *                bit c of word w is 1 when key kt*128 + 32w + c is removed
 *                for query qt*128 + r.  Keys and rows past L read as removed.
 *   tile_class : DEVICE, n*n bytes at qt*n + kt: 0 = no entry inside [L, L]
 *                is removed, 1 = some are, 2 = all are.
 * Asynchronous on `stream` (PDL launch: it waits for the previous kernel in
 * the stream before reading the mask).  Errors: SDPA_ERR_NULL,
 * SDPA_ERR_SHAPE (L < 1 or n > 65535), SDPA_ERR_LAYOUT (tile_bits not 16-byte
 * aligned), SDPA_ERR_CUDA.
 */
SDPA_API sdpa_status sdpa_mask_tiles(const uint8_t* mask, int64_t L, void* tile_bits,
                                     uint8_t* tile_class, void* stream);

/*
 * sdpa_forward_lse -- sdpa_forward that also writes, per query row, the
 * log-sum-exp of the scaled, masked scores, log(sum_j exp(scale * q_i . k_j))
 * over the admissible keys (-inf for a row with none): the log of the
 * softmax denominator, the second output of the fused forward on the
 * FlashInfer pull-request page (`out, lse = fwd(...)`), which a backward
 * pass or a merge of partial results needs.
 *
 * lse        : DEVICE float32 buffer of shape [B, H, L] (rank 4) or [H, L]
 *              (rank 3), 4-byte aligned, not overlapping any other operand.
 * lse_stride : rank - 1 strides in ELEMENTS (host array); positive unless
 *              the extent is 1.
 * Everything else as sdpa_forward; SDPA_ERR_NULL if lse or lse_stride is
 * NULL.  The LSE is computed in fp32 from the same running maximum and sum
 * the softmax uses.
 */
SDPA_API sdpa_status sdpa_forward_lse(const void* q, const void* k, const void* v, void* out,
                                      float* lse, sdpa_dtype dtype, int rank,
                                      const int64_t* shape, const int64_t* q_stride,
                                      const int64_t* k_stride, const int64_t* v_stride,
                                      const int64_t* o_stride, const int64_t* lse_stride,
                                      int is_causal, const uint8_t* mask, float scale,
                                      void* stream);

/*
 * sdpa_forward_varlen -- packed variable-length sequences.  Several
 * documents are stored one after another along the token axis and
 * described by cumulative offsets, the cu_seqlens arrays that the varlen
 * kernels on the FlashInfer pull-request page take ("FlashInfer, Cake DSA
 * kernel optimization", blog.secrett2633.cloud, section 3 on varlen index
 * preparation).  Each document attends only to itself: sequence i is rows
 * [cu_seqlens[i], cu_seqlens[i+1]) of q, k and v, and its output rows are
 * exactly what sdpa_forward returns for that slice alone (the same kernel
 * and per-tile arithmetic, so bit-identical).  Queries and keys share one
 * offsets array (self-attention; causal means key j <= query i within the
 * document).
 *
 * q, k, v, out : DEVICE [total, H, D] 16-bit tensors of type `dtype`.
 * *_stride     : 3 strides in ELEMENTS in (token, head, dim) order; the dim
 *                stride must be 1, the others multiples of 8 elements.
 * lse          : NULL, or DEVICE fp32 [H, total] (lse_stride: 2 strides, head
 *                then token), the per-row log-sum-exp as in sdpa_forward_lse.
 * cu_seqlens   : DEVICE int32 [n_seqs + 1], 4-byte aligned, nondecreasing,
 *                cu_seqlens[0] = 0 and cu_seqlens[n_seqs] = total.  The
 *                kernel uses the running maximum of the offsets clamped to
 *                [0, total] (the identity for valid offsets), so bad offsets
 *                cannot make it read or write outside the buffers or make
 *                two sequences overlap; rows covered by no sequence are
 *                left unwritten.
 * max_seqlen   : an upper bound on the sequence lengths; it only sizes the
 *                grid (a smaller value gives fewer CTAs, never missed work).
 * Explicit masks are not supported here (is_causal or no mask).  Errors as
 * sdpa_forward, plus SDPA_ERR_SHAPE for n_seqs < 1 or max_seqlen < 1 and
 * SDPA_ERR_ARG when out or lse overlaps cu_seqlens.
 */
SDPA_API sdpa_status sdpa_forward_varlen(const void* q, const void* k, const void* v, void* out,
                                         float* lse, sdpa_dtype dtype, int64_t total,
                                         int64_t n_heads, int64_t head_dim,
                                         const int64_t* q_stride, const int64_t* k_stride,
                                         const int64_t* v_stride, const int64_t* o_stride,
                                         const int64_t* lse_stride, const int32_t* cu_seqlens,
                                         int64_t n_seqs, int64_t max_seqlen, int is_causal,
                                         float scale, void* stream);

/*
 * sdpa_sparse_forward -- sparse top-k attention: query row i, every head,
 * attends only to the key rows idx[i, 0 .. len_i) of one key/value head
 * shared by all query heads, len_i = topk_length[i] clamped to [0, topk]
 * (topk when topk_length is NULL).  The DeepSeek sparse attention forward
 * of "FlashInfer, Cake DSA kernel optimization" (blog.secrett2633.cloud):
 * `out, lse = fwd(q, kv, idx, topk_length=...)` over hole-free index rows
 * (sections 1 and 3 of that page); pass the same pointer as k and v for one
 * shared kv tensor.
 *
 * q, out     : DEVICE [total_q, H, D] 16-bit of type `dtype`; q_stride and
 *              o_stride give 2 strides in ELEMENTS (token, head), multiples
 *              of 8; the D stride is 1.
 * k, v       : DEVICE [total_k, D]; k_stride, v_stride = row strides in
 *              ELEMENTS (multiples of 8).  16-byte aligned pointers.
 * lse        : NULL or DEVICE fp32 [total_q, H] (lse_stride: token, head).
 * idx        : DEVICE int32 [total_q, topk] (row stride idx_stride >= topk)
 *              of global key rows; entries outside [0, total_k) inside the
 *              first len_i are treated as removed keys (no fault).
 * topk_length: NULL or DEVICE int32 [total_q].
 * A row with no admissible key gives zeros and lse = -inf.  Computation as
 * sdpa_forward (16-bit tensor-core products, fp32 softmax).  Errors: NULL,
 * DTYPE, SHAPE (D not 64/128, an extent < 1), LAYOUT (alignment, strides),
 * ARG (out or lse overlapping an input, infinite scale), CUDA, DEVICE.
 * Asynchronous on `stream`; one kernel launch.
 */
SDPA_API sdpa_status sdpa_sparse_forward(const void* q, const void* k, const void* v, void* out,
                                         float* lse, sdpa_dtype dtype, int64_t total_q,
                                         int64_t total_k, int64_t n_heads, int64_t head_dim,
                                         const int64_t* q_stride, int64_t k_stride,
                                         int64_t v_stride, const int64_t* o_stride,
                                         const int64_t* lse_stride, const int32_t* idx,
                                         int64_t idx_stride, int64_t topk,
                                         const int32_t* topk_length, float scale, void* stream);

/*
 * sdpa_sparse_compact -- the index preparation of the same page (sections 1
 * and 3) in one launch: per-document key positions become global key rows
 * with the holes removed.  Query row r of document b (rows
 * [cu_seqlens_q[b], cu_seqlens_q[b+1])) keeps, in order, every entry l of
 * idx_local[r, :] with 0 <= l < (cu_seqlens_k[b+1] - cu_seqlens_k[b]) and,
 * if is_causal, l <= r - cu_seqlens_q[b]; it is written as
 * cu_seqlens_k[b] + l to idx_global[r, 0 .. n), the rest of the row is -1,
 * and topk_length[r] = n.  Rows outside every document get n = 0.
 * All arrays DEVICE int32, 4-byte aligned; offsets nondecreasing.  Errors:
 * NULL, SHAPE, LAYOUT, ARG (outputs overlapping inputs or each other), CUDA.
 */
SDPA_API sdpa_status sdpa_sparse_compact(const int32_t* idx_local, int64_t idx_local_stride,
                                         int32_t* idx_global, int64_t idx_global_stride,
                                         int32_t* topk_length, int64_t total_q, int64_t topk,
                                         const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                                         int64_t n_docs, int is_causal, void* stream);

/*
 * Paged key/value caches.  The pages' text has no counterpart: these are the
 * operators that a program needs to answer with a model token by token, next
 * to the forwards above.  A cache is a pool of pages of page_size tokens; a
 * sequence's tokens [i * page_size, ...) lie in page table[i], in any order
 * and shared between sequences at will.  sdpa_cache_append writes new tokens'
 * keys and values, sdpa_paged_forward attends to them.
 *
 * k, v         : DEVICE [n_pages, page_size, n_kv_heads, head_dim], strides in
 *                ELEMENTS for (page, token, head); the last stride is 1, the
 *                others are multiples of 16 bytes.  16-byte aligned.
 * elem         : SDPA_CACHE_BF16, SDPA_CACHE_FP16 (the type of the tokens and
 *                queries used with it), or SDPA_CACHE_E4M3: 8-bit codes, used
 *                with tokens and queries of either 16-bit type.
 * k_scale,
 * v_scale      : SDPA_CACHE_E4M3: DEVICE fp32 [n_pages, n_kv_heads]; the
 *                values are code * scale.  Scales are positive, in [2^-50,
 *                2^50]; others are taken as the nearest of these (0 and NaN as
 *                the least).  NULL for 16-bit caches.
 * page_size    : 16, 32, 64, 128, 256, 512 or 1024.
 * head_dim     : 64 or 128.
 */
typedef enum sdpa_cache_elem {
  SDPA_CACHE_BF16 = 0,
  SDPA_CACHE_FP16 = 1,
  SDPA_CACHE_E4M3 = 2
} sdpa_cache_elem;

typedef struct sdpa_paged_cache {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t n_pages, page_size, n_kv_heads, head_dim;
  int64_t k_stride[3], v_stride[3];
  int32_t elem;
} sdpa_paged_cache;

/*
 * sdpa_cache_append -- write new tokens' keys and values into a paged cache,
 * the keys rotated by their positions on the way, and the queries of the same
 * tokens if they are given.  One kernel launch, asynchronous on `stream`.
 *
 * k, v         : DEVICE [total, n_kv_heads, head_dim] of `dtype`; 2 strides in
 *                ELEMENTS (token, head), multiples of 8.  Sequence b's new
 *                tokens are rows [cu_seqlens[b], cu_seqlens[b+1]).
 * cu_seqlens   : DEVICE int32 [n_seqs + 1], nondecreasing, or NULL: every
 *                sequence has total / n_seqs new tokens (which must divide).
 * kv_lens      : DEVICE int32 [n_seqs], the sequences' lengths WITH the new
 *                tokens: token i of n has position kv_lens[b] - n + i.
 * page_table   : DEVICE int32 [n_seqs, max_pages], row stride
 *                page_table_stride >= max_pages.  No two entries with new
 *                tokens may name one page, in one sequence or in two.
 * cos, sin     : both NULL (no rotation), or DEVICE fp32 [n_pos, rot_dim / 2]
 *                contiguous, 16-byte aligned: entry (pos, j) turns pair j of
 *                every key (and query) head: (x1, x2) -> (x1 cos - x2 sin,
 *                x2 cos + x1 sin).  rot_dim: a multiple of 8 up to head_dim;
 *                later elements are left as they are.  Pair j is elements
 *                (j, j + rot_dim / 2), or (2j, 2j + 1) when interleaved != 0.
 * q, q_out     : both NULL, or DEVICE [total, n_heads, head_dim] of `dtype`
 *                (2 strides each): q_out receives the rotated queries.  q_out
 *                may be q with q's strides (in place).
 *
 * A token whose position is negative or not below max_pages * page_size or
 * n_pos is left out: none of its rows is written, in q_out neither.  A page entry outside [0,
 * n_pages) leaves the token's key and value out.  Rows of tokens beyond the
 * last sequence are not touched.
 *
 * 16-bit caches: the rotated key is rounded once.  SDPA_CACHE_E4M3: the scale
 * of a (page, head) is the least power of two, in range, under which every
 * finite value appended to it so far fits into +-448; a page's first token
 * (row 0) starts it anew.  When it grows, the page's earlier codes are
 * multiplied by old / new in place (exact but for codes below the type's
 * least normal).  Values beyond the range become +-448, NaN stays NaN.
 *
 * Errors: NULL; DTYPE (elem of a 16-bit cache is not dtype); SHAPE (an extent
 * < 1 or too large, page_size, head_dim, rot_dim, total not divisible);
 * LAYOUT; ARG (an output overlaps an input or the cache; pages of keys are pages
 * of values, which attention may read but an append would write twice); CUDA;
 * DEVICE.
 */
SDPA_API sdpa_status sdpa_cache_append(
    const sdpa_paged_cache* cache, const void* k, const void* v, sdpa_dtype dtype, int64_t total,
    const int64_t* k_stride, const int64_t* v_stride, const int32_t* page_table,
    int64_t page_table_stride, int64_t max_pages, const int32_t* kv_lens,
    const int32_t* cu_seqlens, int64_t n_seqs, const float* cos, const float* sin, int64_t n_pos,
    int64_t rot_dim, int interleaved, const void* q, void* q_out, int64_t n_heads,
    const int64_t* q_stride, const int64_t* q_out_stride, void* stream);

/*
 * sdpa_paged_forward -- attention of each sequence's new tokens over its pages.
 *
 * q, out       : DEVICE [total_q, n_heads, head_dim] of `dtype`; 2 strides in
 *                ELEMENTS (token, head), multiples of 8.  n_heads is a
 *                multiple of the cache's n_kv_heads; query head h reads
 *                key/value head h / (n_heads / n_kv_heads).
 * cu_seqlens_q : DEVICE int32 [n_seqs + 1] (rows of q of each sequence,
 *                nondecreasing), or NULL: total_q / n_seqs rows each.
 * kv_lens      : DEVICE int32 [n_seqs], cached tokens of each sequence (the
 *                new ones among them), clamped to [0, max_pages * page_size].
 * is_causal    : nonzero: row i of n sees keys j <= kv_lens[b] - n + i, i.e.
 *                the new tokens are the sequence's last ones; zero: all keys.
 * lse          : NULL or DEVICE fp32 [total_q, n_heads] (2 strides).
 * max_seqlen_q : an upper bound on the sequences' rows, used to choose a
 *                kernel; a smaller value costs time, and results differ by
 *                roundings only.
 * scale        : multiplier of q.k; NaN selects 1/sqrt(head_dim).
 * workspace    : DEVICE scratch, 16-byte aligned, of at least
 *                sdpa_paged_workspace_bytes(...) bytes, whatever it holds.
 *                Calls that may run at the same time need one each.
 *
 * A row that sees no key gives zeros and lse = -inf; rows of q outside every
 * sequence are not written.  A page entry outside [0, n_pages) removes its
 * tokens' keys.  What pages hold beyond a sequence's length is not used (it
 * may be anything, NaN too).  A key within the length that a causal row does
 * not see has the weight zero in that row, times its value, which therefore
 * has to be finite for the row to be.  Products on tensor cores with fp32
 * sums, softmax in fp32; each key's weight, times its value's scale, is
 * rounded to 16 bits (bf16 for a bf16 cache, else fp16, an fp16 one to within
 * 2^-36 of the row's largest) before the second product.  With an
 * 8-bit cache, elements of a query row down to 2^-13 of the row's largest are
 * exact; with more than 16 rows a key/value head (max_seqlen_q * n_heads /
 * n_kv_heads) smaller ones are taken to within 2^-21 (bf16) or 2^-24 (fp16) of
 * it, with fewer bf16 ones to within 2^-39 and fp16 ones are all exact.  Results do not depend on timing.  Asynchronous on
 * `stream`; two kernel launches.  The kernel for many rows a head waits on
 * barriers, each for a bounded time (sdpa_last_device_status).  Errors as
 * above; ARG for an infinite scale or too small a workspace, SHAPE also when
 * (total_q * n_heads / n_kv_heads / 16 + n_seqs) * n_kv_heads * max_pages *
 * page_size / 16 exceeds about 2^31.
 */
SDPA_API sdpa_status sdpa_paged_forward(
    const void* q, void* out, float* lse, sdpa_dtype dtype, const sdpa_paged_cache* cache,
    int64_t total_q, int64_t n_heads, const int64_t* q_stride, const int64_t* o_stride,
    const int64_t* lse_stride, const int32_t* page_table, int64_t page_table_stride,
    int64_t max_pages, const int32_t* kv_lens, const int32_t* cu_seqlens_q, int64_t n_seqs,
    int64_t max_seqlen_q, int is_causal, float scale, void* workspace, uint64_t workspace_bytes,
    void* stream);

/* Bytes of workspace that sdpa_paged_forward needs on the current device (a
 * bound that depends on the device and these arguments alone, not on lengths
 * or batch); 0 when there is no sm_103 device or an argument is out of range. */
SDPA_API uint64_t sdpa_paged_workspace_bytes(int64_t head_dim, int64_t n_heads,
                                             int64_t n_kv_heads, int64_t max_seqlen_q);

/* Adds (lse != NULL) or removes (lse == NULL) the log-sum-exp output of a
 * plan; same layout rules as sdpa_forward_lse. */
SDPA_API sdpa_status sdpa_plan_set_lse(sdpa_plan* plan, float* lse, const int64_t* lse_stride);

/* Human-readable name of a status code (static storage, never NULL). */
SDPA_API const char* sdpa_status_string(sdpa_status status);

/*
 * sdpa_last_device_status -- synchronise `stream`, then report whether any
 * kernel since the previous query gave up on a barrier wait (every wait in
 * the kernel is bounded in time; on expiry the kernel stops, frees its
 * resources and sets a device status word instead of hanging).  Returns
 * SDPA_OK, SDPA_ERR_DEVICE_TIMEOUT (the word is then cleared), or
 * SDPA_ERR_CUDA.
 *
 * sdpa_last_device_status_detail -- the same query; when `detail` is not
 * NULL it also receives the raw status bits (bit 0: a wait ran out of time;
 * the higher bits name the kind of wait), for diagnostics.
 */
SDPA_API sdpa_status sdpa_last_device_status(void* stream);
SDPA_API sdpa_status sdpa_last_device_status_detail(void* stream, uint32_t* detail);

/* ABI version: major * 10000 + minor * 100 + patch. */
SDPA_API int sdpa_version(void);

/*
 * Test hooks (not for production use).
 * sdpa_debug_set_wait_limit_ns: bound on a single barrier wait inside the
 *   kernel (default 1e9 ns); 0 restores the default.
 * sdpa_debug_withhold_q_load: when nonzero, subsequent launches (dense,
 *   packed-document and sparse forwards) never load the query tile, so every
 *   consumer wait runs out before any product is issued: the kernel must return
 *   with SDPA_ERR_DEVICE_TIMEOUT reported by sdpa_last_device_status and the
 *   context must stay usable.
 */
SDPA_API void sdpa_debug_set_wait_limit_ns(uint64_t ns);
SDPA_API void sdpa_debug_withhold_q_load(int enable);

#ifdef __cplusplus
}
#endif

#endif /* SDPA_GB300_H */
