/*
 * mlora.h -- C ABI of libmlora: gathered multi-LoRA shrink / expand on NVIDIA GB300 (sm_103a).
 *
 * THE OPERATION
 *   A LoRA-adapted projection computes y = x·W + s·(x·A)·B with a per-adapter A (d_in x r),
 *   B (r x d_out) and scale s = alpha / r ("Multi-LoRA Serving, in depth", section "The
 *   computation, unmerged"). The adapters' calls do not compute the shared base product x·W: the
 *   caller passes its result as y (lora_fp8_matmul makes it from 8-bit weights), and the
 *   library adds the low-rank delta in place.
 *   Punica (arXiv 2310.18547), section 3.4 "The SGMV Operator", splits the delta into
 *       shrink   v = x·A        (d_in -> r; v starts from zero)
 *       expand   y += v·B       (r -> d_out, in place)
 *   and batches rows that use different adapters. For every row i whose adapter slot s is
 *   not -1 this library computes
 *       v[i][j] = sum_k x[i][k] · A_s[k][j]                                  j < rank[s]
 *       y[i][n] = round( y[i][n] + scale[s] · sum_{j<rank[s]} v[i][j] · B_s[j][n] )
 *   with fp32 accumulation, bf16/fp16 inputs, and one round-to-nearest-even of y.
 *
 *   Two ways to say which row uses which adapter:
 *     SGMV  segments: rows off[t] .. off[t+1]-1 use slot seg_slot[t], with
 *           0 = off[0] <= off[1] <= ... <= off[n] = num_rows (Punica section 3.4, segment
 *           boundaries s_0 = 0 < ... < s_n; the "sgmv" semantics quoted in the zh-TW Punica
 *           digest, section 5.4: y[s[i]:s[i+1]] += x[s[i]:s[i+1]] @ w[i]).
 *     BGMV  a slot per row, row_slot[i], -1 = no adapter (the "add_lora_bgmv" semantics in
 *           the zh-TW Punica digest, section 5.5; the reference loop of "Multi-LoRA Serving,
 *           in depth", section "Why a mixed batch needs special kernels").
 *   Empty segments are allowed and do nothing; the same slot may appear in several segments.
 *
 * ADAPTER POOLS  (mlora_pool, a host struct of device pointers; see below)
 *   stacked  A^T [num_slots][num_layers][r_max][d_in]   row j of A^T = column j of A
 *            B   [num_slots][num_layers][r_max][d_out]  row j of B
 *            (Punica's LoraWeight, zh-TW digest section 5.4: wa [layers, r, in_features],
 *            wb [layers, r, out_features]; slots padded to the largest rank as in the
 *            reference loop). Rows j >= rank[s] are never read.
 *   paged    S-LoRA (arXiv 2311.03285) "Unified Paging": a page is one vector of
 *            page_elems elements (one H-vector). A of rank R is R vectors of d_in elements
 *            (its columns), B is R vectors of d_out elements (its rows); pages sit anywhere
 *            in one pool of num_pages x page_elems elements. A vector longer than a page
 *            spans ceil(d / page_elems) pages (d = d_in for A, d_out for B), so the page
 *            tables are [num_slots][num_layers][r_max][ceil(d / page_elems)] int32: element
 *            k of vector j is element k % page_elems of page table[..][j][k / page_elems].
 *            With page_elems >= d this is one page per vector ([..][r_max][1]). Ranks differ
 *            per adapter and nothing is padded. Page elements past a vector's end are never
 *            read.
 *
 * CONVENTIONS FOR EVERY CALL
 *   - All array pointers are DEVICE pointers unless stated; the mlora_pool / mlora_problem
 *     structs themselves are read on the host during the call and may be freed afterwards.
 *   - The caller owns all memory (inputs, outputs, the pool, v). The library allocates no
 *     device memory in any call.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy default stream)
 *     and never synchronise the host.
 *   - x [num_rows][ldx], y [num_rows][ldy]: row-major bf16/fp16 (the pool's dtype), ldx >=
 *     d_in, ldy >= d_out. v [num_rows][r_max]: fp32, written by shrink at columns < rank[s]
 *     of adapted rows (other entries unspecified), read by expand.
 *   - Alignment (16-byte rows for bulk copies): x, y, a_t, b, pages 16-byte aligned; ldx,
 *     ldy, d_in, d_out, page_elems multiples of 8 elements; v 4-byte aligned.
 *   - Limits: 1 <= r_max <= MLORA_MAX_RANK; d_in, d_out >= 8; num_rows >= 0; 0 <= layer <
 *     num_layers; num_segments >= 0. num_rows == 0 is a no-op that launches nothing; then x,
 *     y, v and row_slot may be NULL (empty arrays), the pool is still validated.
 *   - Host-detectable errors return a negative MLORA_ERR_* code BEFORE anything is launched
 *     (nothing is written). A failed launch returns MLORA_ERR_CUDA (text: lora_error_string).
 *   - Device-detectable metadata errors never trap: the kernel ORs an MLORA_STATUS_* bit
 *     into *dev_status (if dev_status is not NULL) and skips the affected rows, leaving
 *     their y and v untouched:
 *        offsets not 0 = off[0] <= ... <= off[n] = num_rows   -> BAD_OFFSETS, whole call skipped
 *        slot < -1 or slot >= num_slots                      -> BAD_SLOT, rows skipped
 *        rank[s] outside [1, r_max]                          -> BAD_RANK, rows skipped
 *        a page id of a vector j < rank[s] outside [0, num_pages) -> BAD_PAGE, rows skipped
 *     A wait that exceeds its time limit inside a kernel sets MLORA_STATUS_TIMEOUT.
 *   - Slot -1 rows are never written (their y keeps its exact bits).
 *   - Calls whose outputs overlap on the device must be ordered by the caller (one stream).
 */
#ifndef MLORA_H
#define MLORA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define MLORA_API __attribute__((visibility("default")))
#else
#define MLORA_API
#endif

#define MLORA_ABI_VERSION 1
#define MLORA_MAX_RANK 128

/* Return codes. */
#define MLORA_OK 0
#define MLORA_ERR_NULL (-1)        /* a required pointer is NULL */
#define MLORA_ERR_DTYPE (-2)       /* dtype is not MLORA_BF16 / MLORA_FP16 */
#define MLORA_ERR_SHAPE (-3)       /* a size or index is out of range */
#define MLORA_ERR_ALIGN (-4)       /* a pointer, leading dimension or size breaks the alignment rule */
#define MLORA_ERR_POOL (-5)        /* malformed pool descriptor */
#define MLORA_ERR_CUDA (-6)        /* a CUDA call failed; see lora_error_string(MLORA_ERR_CUDA) */
#define MLORA_ERR_TOO_LARGE (-7)   /* the call needs more than the built-in scratch of lora_sgmv_noalloc */
#define MLORA_ERR_WORKSPACE (-8)   /* the workspace is smaller than the call needs */

/* Device status bits, OR-ed into *dev_status. */
#define MLORA_STATUS_BAD_OFFSETS 1
#define MLORA_STATUS_BAD_SLOT 2
#define MLORA_STATUS_BAD_RANK 4
#define MLORA_STATUS_BAD_PAGE 8
#define MLORA_STATUS_TIMEOUT 16
#define MLORA_STATUS_NO_PAGES 32      /* lora_kv_layout: more pages needed than are free */
#define MLORA_STATUS_BAD_LENGTH 64    /* a length, a position or the free ring's state is out of range */
#define MLORA_STATUS_BAD_TOKEN 128    /* lora_logits_adjust: a token id outside the vocabulary */
#define MLORA_STATUS_BAD_REQUEST 256  /* a row's request outside [0, num_requests) */

typedef enum { MLORA_BF16 = 0, MLORA_FP16 = 1, MLORA_FP32 = 2 /* logits only */ } mlora_dtype;
typedef enum { MLORA_POOL_STACKED = 0, MLORA_POOL_PAGED = 1 } mlora_pool_kind;

/* One adapter pool for one projection shape (d_in -> d_out), every layer, every slot.
 * Host struct; every pointer in it is a device pointer owned by the caller. */
typedef struct {
  int32_t kind;        /* mlora_pool_kind */
  int32_t dtype;       /* mlora_dtype: the element type of the pool, x and y */
  int32_t num_slots;   /* adapters resident in the pool (slot ids 0 .. num_slots-1) */
  int32_t num_layers;
  int32_t r_max;       /* stride of the rank dimension (stacked) / of the page tables */
  int32_t d_in;        /* h1: columns of x, rows of A */
  int32_t d_out;       /* h2: columns of y and of B */
  const void *a_t;     /* stacked: A^T [num_slots][num_layers][r_max][d_in]  (NULL when paged) */
  const void *b;       /* stacked: B   [num_slots][num_layers][r_max][d_out] (NULL when paged) */
  const void *pages;   /* paged: [num_pages][page_elems]                     (NULL when stacked) */
  int64_t page_elems;  /* paged: elements per page, a multiple of 8, at least 8 */
  int64_t num_pages;   /* paged */
  const int32_t *a_page_table; /* paged: [num_slots][num_layers][r_max][ceil(d_in/page_elems)], pages of column j of A */
  const int32_t *b_page_table; /* paged: [num_slots][num_layers][r_max][ceil(d_out/page_elems)], pages of row j of B */
  const int32_t *rank;  /* [num_slots], each in [1, r_max] */
  const float *scale;   /* [num_slots], alpha / rank, applied by the expand */
} mlora_pool;

/* Launch flags of the _ex calls. */
#define MLORA_LAUNCH_PROGRAMMATIC 1u /* programmatic dependent launch for this call (see
                                        lora_set_programmatic_launch) */

/* ---- two-phase form (Punica section 3.4: one shrink launch, one expand launch) --------- */

/* SGMV shrink: v[i][j] = sum_k x[i][k] A_s[k][j] for rows of segments with slot s != -1.
 * seg_offsets [num_segments+1] and seg_slot [num_segments] are int32 device arrays. */
MLORA_API int lora_sgmv_shrink(float *v, const void *x, int64_t ldx, const mlora_pool *pool, const int32_t *seg_offsets,
                     const int32_t *seg_slot, int32_t num_segments, int32_t num_rows, int32_t layer,
                     int32_t *dev_status, void *stream);

/* SGMV expand: y[i][n] = round(y[i][n] + scale[s] sum_j v[i][j] B_s[j][n]), in place. */
MLORA_API int lora_sgmv_expand(void *y, int64_t ldy, const float *v, const mlora_pool *pool, const int32_t *seg_offsets,
                     const int32_t *seg_slot, int32_t num_segments, int32_t num_rows, int32_t layer,
                     int32_t *dev_status, void *stream);

/* BGMV shrink: as lora_sgmv_shrink with slot row_slot[i] per row (int32 [num_rows], -1 = none). */
MLORA_API int lora_bgmv_shrink(float *v, const void *x, int64_t ldx, const mlora_pool *pool, const int32_t *row_slot,
                     int32_t num_rows, int32_t layer, int32_t *dev_status, void *stream);

/* BGMV expand: as lora_sgmv_expand with slot row_slot[i] per row. */
MLORA_API int lora_bgmv_expand(void *y, int64_t ldy, const float *v, const mlora_pool *pool, const int32_t *row_slot,
                     int32_t num_rows, int32_t layer, int32_t *dev_status, void *stream);

/* ---- fused form: shrink and expand of one projection in one call ------------------------
 * Same result as shrink followed by expand. For decode-sized segments both phases run in one
 * launch and v stays on chip (a cluster of CTAs splits d_in, sums its partial v through
 * distributed shared memory, then splits d_out). v_scratch [num_rows][r_max] fp32 is
 * caller-owned scratch that the library may use when it runs the two phases as separate
 * launches (long prefill segments); its contents afterwards are unspecified. It is required. */
MLORA_API int lora_sgmv(void *y, int64_t ldy, const void *x, int64_t ldx, const mlora_pool *pool, const int32_t *seg_offsets,
              const int32_t *seg_slot, int32_t num_segments, int32_t num_rows, int32_t layer, float *v_scratch,
              int32_t *dev_status, void *stream);

MLORA_API int lora_bgmv(void *y, int64_t ldy, const void *x, int64_t ldx, const mlora_pool *pool, const int32_t *row_slot,
              int32_t num_rows, int32_t layer, float *v_scratch, int32_t *dev_status, void *stream);

/* lora_bgmv with launch flags. Device-side grouping of the rows (Punica section 3.4, "Batch
 * Layout Construction": rows that share an adapter form one group; "Multi-LoRA Serving, in
 * depth", section "The decode cost model": each adapter read once per step): a first small
 * kernel orders the rows by (rank descending, slot) on the GPU, the main kernel then walks the
 * rows in that order. Rows of one adapter run side by side, so the adapter comes from HBM once;
 * the heaviest rows start first. The caller's row order, x and y are unchanged; the order is
 * kept in v_scratch (2 x num_rows int32). On pools of r_max 32 to 128 (S-LoRA section 3,
 * "Heterogeneous Batching Kernels": adapters of many ranks in one pool) the grouped order is
 * also cut into segments of up to 4 rows that share a slot (num_rows + 1 more int32 of
 * v_scratch), and a streaming kernel takes over: a cluster of CTAs per segment streams the
 * adapter's A^T and B rank-rows through shared-memory rings once for the segment's rows,
 * segments in snake order over the clusters, largest first. lora_bgmv groups batches of at least
 * 128 rows (up to 4096 rows, r_max >= 2); the flags override that:
 *   MLORA_LAUNCH_GROUP_ROWS   group (when num_rows <= 4096 and r_max >= 2)
 *   MLORA_LAUNCH_NO_GROUPING  never group
 *   MLORA_LAUNCH_PROGRAMMATIC programmatic dependent launch for the first kernel of the call
 * Other bits are rejected with MLORA_ERR_SHAPE. Grouped on the main kernel, results are the same
 * bits as ungrouped (every row's arithmetic is the same); streamed, the sums run in another fixed
 * order (the same bits on every call, within the same tolerance of the exact result). */
#define MLORA_LAUNCH_GROUP_ROWS 2u
#define MLORA_LAUNCH_NO_GROUPING 4u
MLORA_API int lora_bgmv_ex(void *y, int64_t ldy, const void *x, int64_t ldx, const mlora_pool *pool,
                           const int32_t *row_slot, int32_t num_rows, int32_t layer, float *v_scratch, uint32_t flags,
                           int32_t *dev_status, void *stream);

/* ---- fused form without a scratch argument -------------------------------------------------
 * lora_sgmv_noalloc: lora_sgmv for callers that cannot hand the library a device buffer --
 * code that may not allocate device memory, such as a plugin running inside a host engine
 * that owns all device memory and passes the plugin only its inputs and outputs, or a
 * latency-critical path where cudaMalloc (which can synchronise the device) is not acceptable.
 * Instead of v_scratch it uses an array built into the library: MLORA_NOALLOC_MAX_FLOATS fp32
 * values (4 MiB) in device memory, which every GPU that loads the library holds until the
 * process exits. The call itself allocates nothing (no cudaMalloc, no cudaFree, no library
 * allocator).
 *   - Limit: num_rows * pool->r_max <= MLORA_NOALLOC_MAX_FLOATS; a larger call returns
 *     MLORA_ERR_TOO_LARGE and launches nothing.
 *   - The first call on a device, with that device current, looks up the array's device
 *     address (cudaGetSymbolAddress); make that first call before any stream capture.
 *   - Every call shares the one array, and it keeps the last call's contents. Nothing in it
 *     must start at zero: the shrink writes every entry the expand later reads.
 *   - Calls whose kernels may run at the same time on the GPU (other streams, other host
 *     threads) race on the array; order them, e.g. on one stream.
 * Same arguments, results and errors as lora_sgmv otherwise. (No counterpart on the pages:
 * an interface convenience of this library.) */
#define MLORA_NOALLOC_MAX_FLOATS (1 << 20)
MLORA_API int lora_sgmv_noalloc(void *y, int64_t ldy, const void *x, int64_t ldx, const mlora_pool *pool,
                                const int32_t *seg_offsets, const int32_t *seg_slot, int32_t num_segments,
                                int32_t num_rows, int32_t layer, int32_t *dev_status, void *stream);

/* ---- grouped form: several projections over the same rows in one call --------------------
 * Punica builds the segments once per batch and reuses them for all 7 projections of every
 * layer (section 3.4, "Batch Layout Construction"). A group runs the fused op of each problem
 * in one launch: typically the projections that read the same x (q, k, v; or gate, up).
 * Each problem has its own x, y, pool, layer and v_scratch; all share the rows' metadata.
 * The mlora_problem array is a host array of at most MLORA_MAX_GROUP entries, and every pool
 * in a group must have the same dtype. */
#define MLORA_MAX_GROUP 8
typedef struct {
  void *y;
  int64_t ldy;
  const void *x;
  int64_t ldx;
  const mlora_pool *pool; /* host pointer */
  int32_t layer;
  float *v_scratch;       /* [num_rows][pool->r_max] fp32 */
} mlora_problem;

MLORA_API int lora_sgmv_grouped(const mlora_problem *problems, int32_t num_problems, const int32_t *seg_offsets,
                      const int32_t *seg_slot, int32_t num_segments, int32_t num_rows, int32_t *dev_status,
                      void *stream);

/* lora_sgmv_grouped with launch flags given per call instead of taken from the calling thread's
 * setting (lora_set_programmatic_launch). flags: 0 or MLORA_LAUNCH_PROGRAMMATIC; other bits are
 * rejected with MLORA_ERR_SHAPE. (No counterpart on the pages: a launch-latency measure for
 * GB300.) */
MLORA_API int lora_sgmv_grouped_ex(const mlora_problem *problems, int32_t num_problems, const int32_t *seg_offsets,
                                   const int32_t *seg_slot, int32_t num_segments, int32_t num_rows, uint32_t flags,
                                   int32_t *dev_status, void *stream);

/* ---- sequence form: the grouped calls of a whole step in one call ------------------------
 * A decoder step issues one grouped call per dependent stage of every layer (q,k,v; o;
 * gate,up; down for a Llama layer: 4 x num_layers calls). lora_sgmv_sequence issues such a
 * list of grouped calls, in order, on `stream`, from native code: the same launches as
 * num_groups calls of lora_sgmv_grouped_ex, for one call's host cost. Every group is validated
 * before anything is launched (a host-detectable error in any group returns its code and
 * launches nothing). flags: MLORA_LAUNCH_PROGRAMMATIC gives every call after the first
 * programmatic dependent launch (the first keeps an ordinary dependency on whatever ran
 * before); the groups then must not write each other's metadata or pools, which this
 * library's calls never do. Each group's problems must not write the x of a later group
 * while that group may read it -- as in a real step, where x of the next stage comes from
 * other kernels. (No counterpart on the pages: Punica issues 7 x L launches per step from
 * the host; this is the same schedule issued natively.) */
typedef struct {
  const mlora_problem *problems; /* host array of num_problems entries */
  int32_t num_problems;          /* 1 .. MLORA_MAX_GROUP */
  const int32_t *seg_offsets;    /* device [num_segments + 1] */
  const int32_t *seg_slot;       /* device [num_segments] */
  int32_t num_segments;
  int32_t num_rows;
} mlora_group;

MLORA_API int lora_sgmv_sequence(const mlora_group *groups, int32_t num_groups, uint32_t flags, int32_t *dev_status,
                                 void *stream);

/* ---- the step around the adapters: cache layout, append, attention, logits -----------------
 * A decode or mixed step of many tenants' requests, besides the adapted projections: where each new
 * row goes in a paged key-value cache, the write of its k and v, the attention that reads the
 * cache, and each request's own adjustment of its logits. The paged cache is S-LoRA's (section 3,
 * "Unified Paging": the key-value pages live in the same pool as the adapters' pages, one list of
 * free pages); any strided view of one allocation serves, an adapter pool's `pages` included.
 *
 * The calls share the conventions above, and these:
 *   - Each takes a host struct that may be built once and used for every step (the lengths are in
 *     device memory, so a captured graph can be replayed). num_rows is the capacity of the row
 *     arrays; a row that stands for nothing has -1 as its request, position and cache slot, and no
 *     call reads or writes anything for it but where said.
 *   - Where an output may be an input (said at the call), its rows are as far apart as the input's. Outputs overlap inputs
 *     in no other way.
 *   - Every kernel waits for the work before it in the stream before it reads or writes any memory,
 *     whether or not it was launched programmatically. lora_kv_layout writes the segments that the adapters' calls
 *     read before such a wait: the first of them after it is launched without MLORA_LAUNCH_PROGRAMMATIC. */

#define MLORA_KV_MAX_REQUESTS 8192
#define MLORA_KV_MAX_HEAD_DIM 256
#define MLORA_LOGITS_MAX_VOCAB (INT32_MAX - 65536) /* a slice of a row ends at most 32768 + 8 tokens behind it */

/* lora_kv_layout: from the requests' lengths, on the GPU, the pages they take or give back, and the
 * places of the step's rows. With n = new_tokens[r] and len = kv_len[r] of request r:
 *   n >= 0  the request gets rows for tokens len .. len+n-1 (n = 0: none; a decoding request: 1; a
 *           prompt: its length). Its page table entries 0 .. ceil(len/page_tokens)-1 are in place;
 *           the entries up to ceil((len+n)/page_tokens)-1 are popped off the free ring, requests in
 *           order. kv_len_out[r] = len + n.
 *   n = -1  the request leaves: its ceil(len/page_tokens) pages are pushed onto the ring, requests
 *           in order, for later calls (this call's new entries come from the pages that were free
 *           before it). kv_len_out[r] = 0; its page table row is left as it is.
 * The ring is free_ring[num_pages] with free_state = {head, count}: the free pages are entries
 * head, head+1, .. head+count-1 (mod num_pages); pops move the head, pushes go behind the last.
 * Rows follow in request order, then padding up to num_rows:
 *   row_request[i], position[i] (the token's index in its request), cache_slot[i] (page *
 *   page_tokens + position % page_tokens), row_slot[i] (the request's adapter): -1 in padding;
 *   seg_offsets[num_requests+2], seg_slot[num_requests+1]: the rows as SGMV segments, one per
 *   request with its adapter slot and a last one for the padding with slot -1.
 * Sums are over whole numbers and every place is determined by the inputs.
 * Errors, in which case the call changes no page and no length (kv_len_out = kv_len,
 * free_state_out = free_state) and lays every row out as padding:
 *   NO_PAGES    the ring holds fewer pages than the requests need
 *   BAD_LENGTH  kv_len[r] < 0, n < -1, len + n > max_pages * page_tokens, more than num_rows rows,
 *               head outside [0, num_pages), count outside [0, num_pages] or pushed beyond num_pages
 *   BAD_PAGE    (only this row) the row's page id is outside [0, num_pages): its cache_slot is -1 */
typedef struct {
  int32_t num_requests;        /* 0 .. MLORA_KV_MAX_REQUESTS */
  int32_t num_rows;            /* entries of the row arrays */
  int32_t page_tokens;         /* tokens of a page */
  int32_t max_pages;           /* entries of a page table row; max_pages * page_tokens < 2^31 */
  int32_t num_pages;           /* entries of free_ring; page ids are 0 .. num_pages-1 */
  int64_t table_stride;        /* page table: int32 from one request's row to the next, >= max_pages */
  const int32_t *new_tokens;   /* [num_requests] */
  const int32_t *kv_len;       /* [num_requests] tokens in the cache before this step */
  int32_t *kv_len_out;         /* [num_requests] tokens after it; may be kv_len */
  int32_t *page_table;         /* [num_requests][table_stride], in and out */
  int32_t *free_ring;          /* [num_pages], in and out */
  const int32_t *free_state;   /* [2] head, count */
  int32_t *free_state_out;     /* [2]; may be free_state */
  const int32_t *adapter_slot; /* [num_requests], or NULL: every adapter slot written is -1 */
  int32_t *row_request;        /* [num_rows] */
  int32_t *position;           /* [num_rows] */
  int64_t *cache_slot;         /* [num_rows] */
  int32_t *row_slot;           /* [num_rows], or NULL */
  int32_t *seg_offsets;        /* [num_requests + 2], or NULL */
  int32_t *seg_slot;           /* [num_requests + 1], or NULL */
} mlora_kv_batch;

MLORA_API int lora_kv_layout(const mlora_kv_batch *batch, int32_t *dev_status, void *stream);

/* A paged key-value cache. Element d of token t of head h in page p of a layer is at
 *   k + p * page_stride + layer * layer_stride + t * token_stride + h * head_stride + d
 * and v likewise (strides in elements, multiples of 8; k and v 16-byte aligned). Token j of request r
 * is token j % page_tokens of page page_table[r][j / page_tokens]. */
typedef struct {
  int32_t dtype;        /* MLORA_BF16 or MLORA_FP16: the type of the cache, q, k, v and the output */
  int32_t num_layers;
  int32_t num_kv_heads;
  int32_t head_dim;     /* a multiple of 8, 8 .. MLORA_KV_MAX_HEAD_DIM */
  int32_t page_tokens;
  int32_t num_pages;
  void *k, *v;
  int64_t page_stride, layer_stride, token_stride, head_stride;
} mlora_kv_cache;

/* lora_kv_append: for every row i with cache_slot[i] >= 0, store its k and v heads in the cache, k
 * rotated by the row's position, and its q heads, rotated likewise, in q_out (no q: q = NULL, num_q_heads
 * = 0). Rotary positions: with c, s = rope_cos, rope_sin[position[i]][m], 0 <= m < rotary_dim / 2,
 *   (a, b) -> (a c - b s, b c + a s),  in fp32, rounded once to the cache's type, for
 *   (a, b) = elements (m, m + rotary_dim/2) of a head, or (2m, 2m+1) with rope_interleaved;
 * the elements from rotary_dim on, and all of them without tables (rope_cos = NULL), are copied.
 * Two rows with the same cache slot leave either's values there. q_out may be q. Rows are
 * ldk, ldv, ldq, ldq_out elements apart (multiples of 8; pointers 16-byte aligned). All num_rows rows of k, v and q have to
 * be there: those of rows without a slot are loaded with the others, before the slots are known, and not used.
 * Skipped rows, with their status: a slot < -1 or >= num_pages * page_tokens (BAD_SLOT), a position
 * outside [0, max_position) where there are tables (BAD_LENGTH). */
typedef struct {
  int32_t num_rows, num_q_heads;
  const int64_t *cache_slot; /* [num_rows] */
  const int32_t *position;   /* [num_rows]; NULL without tables */
  const void *k, *v, *q;     /* [num_rows][ldk >= num_kv_heads * head_dim], .. */
  void *q_out;
  int64_t ldk, ldv, ldq, ldq_out;
  const float *rope_cos, *rope_sin; /* [max_position][rotary_dim / 2] fp32, contiguous, 16-byte aligned, or both NULL */
  int32_t rotary_dim;        /* a multiple of 16, at most head_dim; 0 without tables */
  int32_t max_position, rope_interleaved;
} mlora_kv_rows;

MLORA_API int lora_kv_append(const mlora_kv_cache *cache, const mlora_kv_rows *rows, int32_t layer,
                             int32_t *dev_status, void *stream);

/* lora_kv_attention: for every row i and query head h, over the tokens t of its request
 * row_request[i] that it sees, max(0, position[i] + 1 - window) <= t <= position[i] (window = 0: from
 * token 0),
 *   w_t = exp(scale q[i][h] . K[t][h / G]) / sum of these,   out[i][h] = sum_t w_t V[t][h / G],
 *   lse[i][h] = log of that sum,   G = num_q_heads / num_kv_heads,
 * the scores, the sums and the softmax's statistics in fp32 (accumulated by matrix instructions; a weight enters the second
 * sum to 2^-16 of itself with bf16, 2^-22 with fp16), the output rounded once. A row with
 * position -1 sees nothing: its output is 0 and its lse -inf. Several rows of one request (a drafted
 * continuation, the rows of a prompt) are rows of their own. Cache contents outside the tokens that a
 * row sees, NaN included, do not reach its output. An element of V that is an infinity makes the output's that infinity,
 * however small the token's weight; a NaN, or infinities of both signs, make it NaN. A row whose every score is -inf has
 * no weights: its output is 0 and its lse -inf. out may be q. The long rows' tokens are split over the whole GPU
 * and joined in a fixed order: the same call gives the same bits.
 * workspace: lora_kv_attention_workspace bytes of device memory, 16-byte aligned, zeroed by the
 * caller before its first use; every call leaves the part that has to be zero at zero. Calls that may
 * run at the same time need workspaces of their own.
 * Status: a row_request outside [0, num_requests) (BAD_REQUEST) or a position outside [-1, max_pages *
 * page_tokens) (BAD_LENGTH): the row's output and lse are left untouched. A page id outside [0, num_pages)
 * (BAD_PAGE): the page's tokens count as not seen. */
typedef struct {
  int32_t num_rows, num_q_heads; /* num_q_heads a multiple of the cache's num_kv_heads */
  const void *q;                 /* [num_rows][ldq >= num_q_heads * head_dim] */
  void *out;                     /* [num_rows][ldo] */
  int64_t ldq, ldo;              /* multiples of 8 */
  const int32_t *position;       /* [num_rows] */
  const int32_t *row_request;    /* [num_rows], or NULL: row i is request i */
  const int32_t *page_table;     /* [num_requests][table_stride] */
  int64_t table_stride;
  int32_t num_requests, max_pages; /* max_pages * page_tokens < 2^31, times num_kv_heads (and every 16 query heads
                                      of a group) below 2^34 */
  int32_t window;
  float scale;
  float *lse;                    /* [num_rows][num_q_heads], or NULL */
  void *workspace;
  int64_t workspace_bytes;
} mlora_kv_attn;

/* Bytes of workspace that lora_kv_attention needs on this cache, whatever the batch. */
MLORA_API int64_t lora_kv_attention_workspace(const mlora_kv_cache *cache, int32_t num_q_heads);
MLORA_API int lora_kv_attention(const mlora_kv_cache *cache, const mlora_kv_attn *args, int32_t layer,
                                int32_t *dev_status, void *stream);
/* The same, told how many rows a request has at most in this call (1: a decode step; a prompt's or a draft's length; 0: not
 * known). It decides how many rows are taken through the cache together, which changes the time and the rounding, not
 * what is computed; a wrong number is only slower. Without it the call goes by num_rows / num_requests, which says little where
 * the rows are padded or the page table has places without a request. */
MLORA_API int lora_kv_attention_ex(const mlora_kv_cache *cache, const mlora_kv_attn *args, int32_t layer,
                                   int32_t rows_per_request, int32_t *dev_status, void *stream);

/* lora_logits_adjust: out[i][t] from logits[i][t], for row i of request r = row_request[i] (-1: the row's
 * output is left untouched), in fp32 and rounded once to the logits' type. With the request's history
 * tokens[r][0 .. total_len[r]), of which the first prompt_len[r] are its prompt,
 *   x = logits[i][t]
 *   t in the history:              x = x > 0 ? x / repetition[r] : x * repetition[r]
 *   t c > 0 times past the prompt: x = x - frequency[r] * c - presence[r]
 *   t in the request's bias list:  x = x + its value (of several entries with one id, the last)
 *   temperature[r] > 0:            x = x / temperature[r]
 *   mask_index[r] >= 0 and bit t % 32 of mask[mask_index[r]][t / 32] is 0: x = -inf
 * Every array may be NULL and then has no part (tokens, prompt_len and total_len together; bias_offsets,
 * bias_token and bias_value; mask and mask_index). logits and out are rows ld, ldo elements apart, aligned
 * to their element; out may be logits. Every id of a row of tokens may be read, those behind its total_len included (a
 * matrix that is part of a wider one has its own width as tokens_len).
 * Status: a token id outside [0, vocab) in a history or a bias list (BAD_TOKEN): that entry has no
 * part. total_len[r] outside [0, tokens_len] or prompt_len[r] outside [0, total_len[r]] or bias offsets
 * that decrease or leave [0, num_bias] (BAD_LENGTH), mask_index[r] outside [-1, num_masks) (BAD_SLOT), row_request[i]
 * outside [-1, num_requests) (BAD_REQUEST): the row is skipped. */
typedef struct {
  int32_t num_rows, vocab, dtype; /* 1 <= vocab <= MLORA_LOGITS_MAX_VOCAB; dtype: MLORA_FP32, MLORA_BF16 or MLORA_FP16 */
  int32_t num_requests;
  const void *logits;
  void *out;
  int64_t ld, ldo;
  const int32_t *row_request;     /* [num_rows], or NULL: row i is request i */
  const int32_t *tokens;          /* [num_requests] rows of tokens_len ids, tokens_stride apart */
  int64_t tokens_stride;
  const int32_t *prompt_len, *total_len;                        /* [num_requests] */
  const float *repetition, *presence, *frequency, *temperature; /* [num_requests] each */
  const int32_t *bias_offsets;    /* [num_requests + 1] */
  const int32_t *bias_token;
  const float *bias_value;
  int32_t num_bias;               /* entries of bias_token and bias_value */
  const uint32_t *mask;           /* [num_masks][mask_stride >= ceil(vocab / 32)] */
  int64_t mask_stride;
  const int32_t *mask_index;      /* [num_requests] */
  int32_t num_masks;
  int32_t tokens_len;             /* ids in a row of tokens, at most tokens_stride; 0: tokens_stride of them */
} mlora_logits;

MLORA_API int lora_logits_adjust(const mlora_logits *args, int32_t *dev_status, void *stream);

/* ---- the step around the adapters: norm, 8-bit rows, base product, next token ---------------
 * What stands between the adapted projections of a step whose base weights are held in 8 bits: the norm with the
 * residual's addition, the base products x W that the adapters add to, and the choice of the next token. The
 * adapters read x in 16 bits, the base product reads it in 8, so the calls that make x write both.
 *
 * 8-bit rows: e4m3 values (1 sign, 4 exponent, 3 mantissa bits, largest 448) q [num_rows][ldq] with an fp32 scale for
 * every block of MLORA_FP8_BLOCK columns of a row (the last may be shorter), scale [num_rows][lds]; an element
 * stands for q * scale. Those of values v are
 *   scale = max(max |v| of the block / 448, 2^-126),   q = v / scale, in fp32, rounded to the nearest e4m3, ties to even;
 * a NaN makes its block's scale and values NaN, an infinity makes the scale an infinity, its own value NaN and the
 * others 0. The conventions above hold: pointers of 16-bit and 8-bit arrays 16-byte aligned, their widths and
 * leading dimensions multiples of 8 unless said, fp32 and int32 arrays 4-byte aligned. */

#define MLORA_FP8_BLOCK 128
#define MLORA_ROW_MAX_WIDTH 32768     /* lora_rms_norm */
#define MLORA_SAMPLE_MAX_VOCAB 393216

/* lora_rms_norm: with h = x + residual (x without one),
 *   residual_out = round(h),   v = weight * h / sqrt(mean of h^2 over the row + eps),   out = round(v),
 *   (q, q_scale) = v as 8-bit rows,
 * in fp32 from the unrounded h, each output rounded once. residual and residual_out come together, and q and q_scale; out
 * or q may be NULL, not both. residual_out may be residual or x, and out may be x or residual, with equal leading dimensions; every
 * other output is an array of its own. Sums and squares may pass fp32's range: finite rows of x and residual have a
 * finite norm (residual_out is rounded as any sum is). */
typedef struct {
  int32_t num_rows, width, dtype; /* width a multiple of 8, 8 .. MLORA_ROW_MAX_WIDTH; dtype of x, residual, weight, out */
  float eps;                      /* at least 2^-126, finite */
  const void *x;                  /* [num_rows][ldx] */
  const void *residual;           /* [num_rows][ldr], or NULL */
  const void *weight;             /* [width], or NULL: 1 */
  void *residual_out;             /* [num_rows][ldro] */
  void *out;                      /* [num_rows][ldo], or NULL */
  void *q;                        /* [num_rows][ldq], or NULL */
  float *q_scale;                 /* [num_rows][lds >= ceil(width / 128)] */
  int64_t ldx, ldr, ldro, ldo, ldq, lds;
} mlora_norm;

MLORA_API int lora_rms_norm(const mlora_norm *args, void *stream);

/* lora_quantize: v = x, or x * gate / (1 + exp(-gate)) with a gate, in fp32;
 *   (q, q_scale) = v as 8-bit rows,   out = round(v)
 * q (with q_scale) or out may be NULL, not both. out may be x or gate, with equal leading dimensions; the other outputs are arrays
 * of their own. gate and x may be column blocks of one array. 1 / (1 + exp(-gate)) is held to 2^-149. */
typedef struct {
  int32_t num_rows, width, dtype; /* width a multiple of 8, at least 8; dtype of x, gate, out */
  const void *x;                  /* [num_rows][ldx] */
  const void *gate;               /* [num_rows][ldg], or NULL */
  void *out;                      /* [num_rows][ldo], or NULL */
  void *q;                        /* [num_rows][ldq], or NULL */
  float *q_scale;                 /* [num_rows][lds >= ceil(width / 128)] */
  int64_t ldx, ldg, ldo, ldq, lds;
} mlora_quant;

MLORA_API int lora_quantize(const mlora_quant *args, void *stream);

/* lora_fp8_matmul: y[i][n] = round( sum over blocks b of 128 columns of
 *     x_scale[i][b] * w_scale[n / 128][b] * sum over k in b of x[i][k] w[n][k] ),
 * the base product that lora_sgmv and lora_bgmv then add to. x: 8-bit rows; w: e4m3 [d_out][ldw >= d_in], the layout
 * (out_features, in_features), with a scale for every block of 128 x 128. A block's products are summed by the tensor
 * cores in fp32, the blocks in fp32 in a fixed order: the same call gives the same bits. The two scales are multiplied first, in
 * fp32, whose range their product must not leave. y is no other array.
 * TIMEOUT as for the adapters' calls. */
typedef struct {
  int32_t num_rows, d_in, d_out, dtype; /* d_in a multiple of 16, d_out of 8 and below 2^31 - 256;
                                           ceil(num_rows / 16) ceil(d_out / 128) below 2^28 */
  const void *x;                        /* [num_rows][ldx], ldx a multiple of 16 */
  const float *x_scale;                 /* [num_rows][ldxs >= ceil(d_in / 128)] */
  const void *w;                        /* [d_out][ldw], ldw a multiple of 16 */
  const float *w_scale;                 /* [ceil(d_out / 128)][ldws >= ceil(d_in / 128)] */
  void *y;                              /* [num_rows][ldy] */
  int64_t ldx, ldxs, ldw, ldws, ldy;
} mlora_matmul;

MLORA_API int lora_fp8_matmul(const mlora_matmul *args, int32_t *dev_status, void *stream);

/* lora_sample: the next token of row i, of request r = row_request[i] (-1: the row's outputs are left untouched), from a
 * uniform random number in [0, 1). The tokens in the order of their logits, the largest first, equal ones by their
 * id; with T = temperature[r], w_t = exp((logit_t - the largest logit) / T). A prefix of the order is kept, the shortest of
 *   top_k[r] > 0:     the first top_k[r] tokens
 *   top_p[r] < 1:     the fewest whose w sum to at least top_p[r] times the sum over those that top_k leaves
 *   min_p[r] > 0:     the tokens with w_t >= min_p[r]
 * and at least one token; token[i] is the first of the order at which the running sum of w exceeds uniform[i] times the sum
 * over those kept, logprob[i] = log(its w / that sum). T <= 0: the first token of the order; 0 < T < 2^-126 counts as
 * 2^-126. A difference of logits beyond fp32's range has w = 0. Every array of the requests may be NULL and then has no
 * part (T = 1). Behind lora_logits_adjust, the temperature is given to one of the two calls.
 * A NaN logit counts as -inf; -inf has w = 0; of logits of +inf each has w = 1 and all others 0. A row with nothing but
 * -inf gets token -1 and logprob -inf. uniform outside [0, 1) is taken to the nearer end, NaN as 0.
 * The sums are of whole numbers, 2^-44 of the largest w each (w to 2^-36 of itself, below 2^-18
 * of the largest to 2^-40 of that): the same bits on every call.
 * token and logprob are arrays of their own.
 * Status: row_request[i] outside [-1, num_requests) (BAD_REQUEST): the row is skipped. */
typedef struct {
  int32_t num_rows, vocab, dtype; /* 1 <= vocab <= MLORA_SAMPLE_MAX_VOCAB; dtype: MLORA_FP32, MLORA_BF16 or MLORA_FP16 */
  int32_t num_requests;
  const void *logits;             /* [num_rows][ld >= vocab], aligned to their element */
  int64_t ld;
  const int32_t *row_request;     /* [num_rows], or NULL: row i is request i */
  const float *uniform;           /* [num_rows] */
  const float *temperature;       /* [num_requests] each, or NULL */
  const int32_t *top_k;
  const float *top_p, *min_p;
  int32_t *token;                 /* [num_rows] */
  float *logprob;                 /* [num_rows], or NULL */
} mlora_sampling;

MLORA_API int lora_sample(const mlora_sampling *args, int32_t *dev_status, void *stream);

/* ---- utilities --------------------------------------------------------------------------- */

/* Static text for a return code; for MLORA_ERR_CUDA it names the last CUDA error this thread saw. */
MLORA_API const char *lora_error_string(int code);

/* Programmatic dependent launch (off by default), for the calling host thread. When on, every
 * later call from this thread launches its kernels so that they may start while the previous
 * kernel in the stream is still running: before waiting for that kernel a kernel reads only its
 * rows' metadata (offsets, slots), the pool descriptor arrays (rank, scale, page tables) and the
 * adapter weights, and it requests the weights; x, y, v and dev_status are touched only after
 * the wait. Turn it on only where the kernel launched just before each call does not write those
 * inputs -- e.g. a sequence of this library's calls, or calls whose inputs were written by copies
 * or at least one kernel earlier. Other host threads keep their own setting. Returns this
 * thread's previous setting. (No counterpart on the pages: a launch-latency measure for GB300.) */
MLORA_API int lora_set_programmatic_launch(int enable);

/* MLORA_ABI_VERSION of the loaded library. */
MLORA_API int lora_abi_version(void);

/* Number of kernel launches the library has issued from this process (all threads). */
MLORA_API int64_t lora_launch_count(void);

/* Testing hook for the time-out path: limit, in nanoseconds, of the waits inside the CUDA-core
 * kernels and lora_fp8_matmul's launched later by the calling thread (the waits for their own bulk
 * copies, for their cluster peers' partial sums and between a product's loads, MMAs and sums). 0 restores the default of 2 s. With a limit of a few
 * nanoseconds a wait gives up unless its data has already landed, the kernel sets
 * MLORA_STATUS_TIMEOUT and skips the work that needed the data, and copies still in flight are
 * drained (with the default limit) before the kernel exits. Not for production use: results of
 * rows whose waits gave up are left unwritten. (No counterpart on the pages.) */
MLORA_API void lora_test_set_wait_limit_ns(uint64_t limit_ns);

#ifdef __cplusplus
}
#endif

#endif /* MLORA_H */
