/*
 * pa.h -- C ABI of libpagedfp8: paged decode attention over an FP8 (e4m3) KV cache
 * with per-token or scalar K/V scales (and a BF16-KV control), for grouped-query
 * attention with ragged speculative-decode query lengths, split-K over long contexts
 * with a log-sum-exp merge, and a sparse selected-page variant; with the two steps next
 * to it: the per-token FP8 quantise-and-write that fills the cache
 * (pa_kv_quantize_write) and the indexer's page scores and top-k that choose the sparse
 * variant's pages (pa_index_topk); the log-sum-exp merge that combines the parts of a
 * context split across GPUs (pa_lse_merge); and what happens to the cache between two
 * decode steps: eviction by accumulated attention weight (pa_attn_mass, pa_evict_select,
 * pa_kv_compact) and beam search (pa_beam_select, pa_beam_reorder); and a prompt's way into the
 * cache: pages and slots for its tokens (pa_page_assign, pa_page_release), rotary positions (pa_rope)
 * and causal attention over whole packed prompts (pa_prompt_attn).  sm_103a (GB300).
 *
 * Sources of the operation (the pages are pull-request threads):
 *  - ROCm/ATOM PR 2614, "Change": dense max-q-len-1 per-token FP8 decode and sparse
 *    decode share one paged-decode contract; "Validation": the per-token kernel
 *    needs split-K.
 *  - ROCm/ATOM PR 2710, review "Must fix" 1 and "Should fix" 2: scratch is sized
 *    from a bounded set of capacity buckets and reused; an unsupported call is
 *    refused at set-up, not raised mid-run; "Smaller": partition scratch
 *    (exp_sums, max_logits, temporary_output).
 *  - ROCm/ATOM PR 2122 ("fix(minimax-m3): unblock fp8 KV cache and EAGLE3 spec decode
 *    on the vLLM plugin"), section 1: FP8 caches are raw bytes; section 2: a decode
 *    segment must be measured as uniform, rows map to requests through
 *    cu_seqlens_q, and row tok attends positions < seq_len - q_len + tok + 1.
 *  - vLLM PR 52060 ("[ROCm][Perf] Fold scalar KV scales in MiniMax-M3 sparse
 *    attention"), "Suggested Fix": a scalar K scale folds into the score scale and a
 *    scalar V scale is applied once to the normalised fp32 accumulator; per-token
 *    scales stay per token.
 *
 * Conventions for every call:
 *  - Device pointers are caller-owned device memory; the library allocates no device
 *    memory at any time.  Its only scratch is the caller's workspace, sized once per
 *    plan by pa_plan_workspace_size.
 *  - Errors are returned as pa_status_t; no call aborts, throws or prints.
 *  - pa_decode performs no host synchronisation and no allocation, and returns as
 *    soon as its kernel is enqueued on the given stream.
 */
#ifndef PAGEDFP8_PA_H
#define PAGEDFP8_PA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pa_status {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = 1,   /* a null pointer, a negative size or a value out of range */
  PA_ERR_UNSUPPORTED = 2,   /* a shape or mode this library does not implement */
  PA_ERR_CAPACITY = 3,      /* a call larger than its plan's capacity bucket */
  PA_ERR_RAGGED = 4,        /* a uniform plan given ragged (or miscounted) query rows */
  PA_ERR_ALIGN = 5,         /* a pointer without the required 16-byte alignment */
  PA_ERR_CUDA = 6,          /* a CUDA runtime or driver call failed */
  PA_ERR_DEVICE_DATA = 7,   /* the kernel flagged bad data (see PA_DEV_* flags) */
  PA_ERR_WORKSPACE = 8      /* the workspace is null, misaligned or too small */
} pa_status_t;

enum { PA_KV_FP8_E4M3 = 0, PA_KV_BF16 = 1 };
enum { PA_SCALE_NONE = 0, PA_SCALE_SCALAR = 1, PA_SCALE_PER_TOKEN = 2 };
enum { PA_Q_UNIFORM = 0, PA_Q_RAGGED = 1 };
enum { PA_OUT_BF16 = 0, PA_OUT_F32 = 1 };

/* Device status flags, OR-ed into the plan's workspace by the kernels.  A flagged
 * work item is skipped (its pages are not read); nothing traps.  Read them with
 * pa_plan_get_device_status. */
#define PA_DEV_BAD_PAGE      0x01u  /* a block-table entry outside [0, num_pages) */
#define PA_DEV_BAD_CONTEXT   0x02u  /* context_len < 0, > max_context_len, or more pages than the block-table stride */
#define PA_DEV_BAD_QLEN      0x04u  /* a request's q_len < 0 or > the plan's q_len, or context_len < q_len */
#define PA_DEV_NOT_UNIFORM   0x08u  /* uniform plan, but cu_seqlens_q[r] != r * q_len */
#define PA_DEV_BAD_SELECTED  0x10u  /* num_selected outside [0, selected_stride], or a selected page outside [-1, pages of the request) */
#define PA_DEV_Q_RANGE       0x20u  /* a query value outside the f16 range (|q| > 65504) */
#define PA_DEV_TIMEOUT       0x40u  /* a bounded wait inside a kernel gave up (the output is incomplete) */
#define PA_DEV_DUMP_RANGE    0x80u  /* pa_debug_gather's buffer was too small for the schedule */
#define PA_DEV_BAD_SLOT      0x100u /* pa_kv_quantize_write: a slot >= num_pages * page_size */

/* Plan flags.
 * PA_PLAN_NO_PDL: launch pa_decode as an ordinary kernel.  By default it is launched
 *   with programmatic dependent launch: its CTAs may start while the kernel before it
 *   in the stream is finishing, and read the index inputs (block_table, context_lens,
 *   cu_seqlens_q, selected_pages, num_selected) before that kernel has completed; they
 *   wait for it to complete before reading q, the caches or the scales, and before
 *   writing anything (before the wait they only ask L2 to prefetch the first pages,
 *   which reads nothing into the kernel).  So with PDL on, the kernel enqueued immediately before pa_decode
 *   must not write those index inputs (copies and host writes are unaffected), nor may the one before
 *   that if it was such a pa_decode.  Set this flag if they do. */
#define PA_PLAN_NO_PDL 0x1
/* PA_PLAN_TCGEN05: for an FP8 plan with q_len 1, run the tcgen05 kernel, which feeds the
 *   cache bytes to the tensor core (QK^T and PV as kind::f8f6f4 MMAs with accumulators
 *   in tensor memory), instead of the default mma.sync kernel, which widens e4m3 to f16
 *   on the SM sub-partitions.  Both give the same results within the library's
 *   tolerances.  On GB300 the default kernel is currently the faster of the two; the
 *   flag is ignored for other plans. */
#define PA_PLAN_TCGEN05 0x2

/* Plan descriptor: the capacity bucket and the fixed shape of every call on the plan
 * (ROCm/ATOM PR 2710 review, "Must fix" 1: size the plan by a capacity bucket).
 * Supported: head_dim 128, group_size 16, page_size in {16, 32, 64, 128},
 * kv_dtype FP8 with scale_mode SCALAR or PER_TOKEN, or BF16 with scale_mode NONE;
 * q_len 1..8; max_batch 1..4096. */
typedef struct pa_plan_desc {
  int32_t num_kv_heads;       /* Hkv >= 1; query heads = Hkv * group_size, head j uses KV head j / group_size */
  int32_t group_size;         /* query heads sharing one KV head */
  int32_t head_dim;           /* D */
  int32_t page_size;          /* tokens per page */
  int32_t kv_dtype;           /* PA_KV_* */
  int32_t scale_mode;         /* PA_SCALE_* */
  int32_t q_mode;             /* PA_Q_UNIFORM: every request has q_len rows; PA_Q_RAGGED: rows from cu_seqlens_q */
  int32_t q_len;              /* uniform: rows per request; ragged: the most rows one request may have */
  int32_t max_batch;          /* most requests per call */
  int32_t max_rows;           /* most query rows per call */
  int32_t max_context_len;    /* longest context (tokens, counting the request's own q_len new tokens) */
  int32_t max_selected_pages; /* 0: dense-only plan; else the most selected pages per request in sparse calls */
  int32_t partition_tokens;   /* 0: balanced persistent schedule (one CTA per SM, equal tile counts);
                                 else fixed split-K partitions of this many tokens (multiple of 128) */
  int32_t out_dtype;          /* PA_OUT_BF16 (round to nearest even) or PA_OUT_F32 */
  int32_t num_sms;            /* 0: the current device's SM count; > 0: use this count (sizing without a GPU) */
  int32_t flags;              /* PA_PLAN_* bits */
  int32_t reserved[2];        /* must be 0 */
} pa_plan_desc_t;

/* One decode call.  Layouts are dense row-major; rows = query tokens. */
typedef struct pa_decode_args {
  const void *q;                   /* device bf16 [num_rows, Hkv*group, head_dim], 16-B aligned */
  const void *k_cache;             /* device [num_pages, Hkv, page_size, head_dim]: e4m3 bytes (raw uint8 or
                                      float8_e4m3fn storage, ROCm/ATOM PR 2122 section 1) or bf16; 16-B aligned */
  const void *v_cache;             /* same layout as k_cache */
  const float *k_scale;            /* device fp32 [num_pages, Hkv, page_size]; PER_TOKEN only, 16-B aligned */
  const float *v_scale;            /* same; PER_TOKEN only */
  float k_scale_scalar;            /* SCALAR only: one K scale for the whole cache */
  float v_scale_scalar;            /* SCALAR only: one V scale */
  int64_t num_pages;               /* physical pages in each cache (bounds every block-table entry) */
  const int32_t *block_table;      /* device int32 [num_seqs, block_table_stride]: logical page -> physical page */
  int32_t block_table_stride;      /* entries per block-table row */
  int32_t num_seqs;                /* requests in this call (<= max_batch) */
  const int32_t *context_lens;     /* device int32 [num_seqs]: tokens in each request's cache, own q_len included */
  const int32_t *cu_seqlens_q;     /* device int32 [num_seqs + 1]: request r owns rows [cu[r], cu[r+1]);
                                      required by RAGGED plans, optional for UNIFORM (then checked on device) */
  const int32_t *cu_seqlens_q_host;/* host int32 [num_seqs + 1], optional: validated before launch */
  const int32_t *selected_pages;   /* device int32 [num_seqs, selected_stride] logical page indices, -1 = padding;
                                      NULL for a dense call */
  const int32_t *num_selected;     /* device int32 [num_seqs]: entries used per row of selected_pages */
  int32_t selected_stride;         /* entries per selected_pages row (<= max_selected_pages) */
  int32_t num_rows;                /* query rows in this call (<= max_rows) */
  float sm_scale;                  /* softmax scale, > 0 (1/sqrt(head_dim) for the workloads) */
  int32_t reserved0;               /* must be 0 */
  void *out;                       /* device [num_rows, Hkv*group, head_dim], bf16 or fp32 per the plan; 16-B aligned */
  float *lse;                      /* device fp32 [num_rows, Hkv*group], optional: natural-log sum of exp of the
                                      scores (-inf for an empty key set) */
} pa_decode_args_t;

/* Facts about a created plan (for tests and benchmarks). */
typedef struct pa_plan_info {
  int32_t grid_ctas;          /* CTAs per decode launch (balanced: the SM count) */
  int32_t stages;             /* KV tiles in flight per CTA */
  int32_t threads_per_cta;
  int32_t tile_tokens;        /* tokens per KV tile (128) */
  int64_t smem_bytes;         /* dynamic shared memory per CTA */
  int64_t workspace_bytes;
  int64_t partial_slots;      /* split-K partial (m, l, o) slots in the workspace */
  int32_t kernel;             /* decode kernel of the plan: 0 mma.sync, 1 tcgen05 (PA_PLAN_TCGEN05) */
  int32_t reserved;
} pa_plan_info_t;

typedef struct pa_plan pa_plan_t;

/* Validates a descriptor without touching a GPU.  PA_ERR_UNSUPPORTED for an
 * unimplemented shape or mode, PA_ERR_INVALID_ARG for an out-of-range field. */
pa_status_t pa_plan_validate(const pa_plan_desc_t *desc);

/* Workspace bytes a plan with this descriptor needs (a multiple of 256), or 0 if the
 * descriptor is refused.  Queries the current device when desc->num_sms == 0. */
size_t pa_plan_workspace_size(const pa_plan_desc_t *desc);

/* Creates a plan bound to a caller-owned device workspace of at least
 * pa_plan_workspace_size bytes (256-B aligned).  The workspace holds the split-K
 * partials, per-request merge counters and the device status word; this call
 * zero-fills its control part with a synchronous cudaMemset on the current device.
 * The plan is immutable and reusable by any call within its bucket; calls that share
 * a plan (and so its workspace) must be serialised on one stream.  On error *plan is
 * set to NULL.  With d_workspace == NULL and workspace_bytes == 0 the plan is
 * check-only: it makes no CUDA call, serves pa_decode_check (for refusing a serving
 * configuration at start-up), and pa_decode on it returns PA_ERR_WORKSPACE. */
pa_status_t pa_plan_create(const pa_plan_desc_t *desc, void *d_workspace, size_t workspace_bytes,
                           pa_plan_t **plan);

/* Host-only check of a call against its plan (capacity, mode, pointers, alignment,
 * the host mirror of cu_seqlens_q).  Launches nothing.  pa_decode runs it first. */
pa_status_t pa_decode_check(const pa_plan_t *plan, const pa_decode_args_t *args);

/* Enqueues one decode on `stream` (a cudaStream_t; NULL = the legacy default stream).
 * Refusals (PA_ERR_CAPACITY, PA_ERR_RAGGED, ...) happen before anything is enqueued.
 * Rows of requests with an empty key set are written as zeros (lse -inf).  Data errors
 * found on the device set PA_DEV_* flags instead of faulting. */
pa_status_t pa_decode(pa_plan_t *plan, const pa_decode_args_t *args, void *stream);

/* Synchronises the device, copies the plan's PA_DEV_* flags to *flags and, if clear
 * is non-zero, resets them.  For tests and diagnostics, never on the hot path. */
pa_status_t pa_plan_get_device_status(pa_plan_t *plan, uint32_t *flags, int clear);

pa_status_t pa_plan_get_info(const pa_plan_t *plan, pa_plan_info_t *info);

/* Frees the host-side plan (the workspace stays the caller's).  NULL is a no-op. */
void pa_plan_destroy(pa_plan_t *plan);

/* A static string naming the status. */
const char *pa_status_string(pa_status_t status);

/* Size of the fixed device scratch that pa_decode_noalloc uses (8 MiB per GPU). */
#define PA_NOALLOC_SCRATCH_BYTES (8u << 20)

/* pa_decode for callers that cannot allocate device memory when they set up or run a
 * decode -- for example an engine plugin whose enqueue step must not allocate, or a
 * runtime whose device memory pool is fixed before the first request -- and so cannot
 * hand pa_plan_create a workspace.  No source page has a counterpart of this call: it
 * is a convenience of this library.
 *
 * It takes the plan descriptor directly and runs the same decode as pa_decode, with the
 * split-K scratch in one fixed array of PA_NOALLOC_SCRATCH_BYTES that the library
 * reserves on every GPU that loads it, for the life of the process.  It calls no
 * cudaMalloc, cudaFree or other allocating routine, host or device.
 *  - Descriptors whose workspace (pa_plan_workspace_size) exceeds the array are
 *    refused with PA_ERR_CAPACITY (on 152 SMs a balanced plan fits for q_len <= 3);
 *    other refusals are those of pa_plan_create and pa_decode_check.
 *  - The first call on a device looks up the array's device address and sets the
 *    kernels' shared-memory limit for that device; make that first call before any
 *    stream capture on the device.
 *  - Each call first clears the scratch's status word and arrival counters on `stream`.
 *    All calls on a device share the one array, so calls that may overlap on the GPU
 *    (different streams without ordering between them) race and corrupt each other.
 *  - Device-side data flags (PA_DEV_*) of these calls are not reported. */
pa_status_t pa_decode_noalloc(const pa_plan_desc_t *desc, const pa_decode_args_t *args,
                              void *stream);

/* ---- the producer of the cache: per-token FP8 quantise-and-write ---- */

/* Arguments of pa_kv_quantize_write.  All pointers are device pointers. */
typedef struct pa_kv_write_args {
  const void *k_new;             /* bf16 [num_tokens, num_kv_heads, head_dim], 16-B aligned */
  const void *v_new;             /* bf16, same shape */
  const int64_t *slot_mapping;   /* [num_tokens]: cache slot page * page_size + offset of each
                                    token; a negative slot skips the token */
  void *k_cache;                 /* e4m3 bytes [num_pages, num_kv_heads, page_size, head_dim], 16-B aligned */
  void *v_cache;
  float *k_scale;                /* fp32 [num_pages, num_kv_heads, page_size], 4-B aligned */
  float *v_scale;
  uint32_t *status;              /* nullable; PA_DEV_BAD_SLOT is OR-ed in when a slot is past the cache */
  int64_t num_tokens;            /* >= 0; 0 enqueues nothing */
  int64_t num_pages;
  int32_t num_kv_heads;          /* >= 1 */
  int32_t head_dim;              /* 128 */
  int32_t page_size;             /* 16, 32, 64 or 128 */
  int32_t reserved;              /* 0 */
} pa_kv_write_args_t;

/* Quantises new K and V rows to the per-token FP8 cache that pa_decode reads (ROCm/ATOM
 * PR 2614: MiniMax-M3 writes FP8 KV plus per-token K/V scales, checked by a
 * producer-to-consumer operator test; ROCm/ATOM PR 2710, "Smaller": the cache-write
 * branch).  For every token t with slot s = slot_mapping[t] >= 0 and every KV head h,
 * with row = (s / page_size * num_kv_heads + h) * page_size + s % page_size:
 *   scale = max_d |x[d]| / 448 in fp32 (448 being the largest finite e4m3fn value),
 *   code[d] = x[d] / scale taken as the fp32 product x[d] * (448 / amax), the reciprocal
 *   rounded to fp32 once per row (the fp32 quotient where it overflows), then rounded to
 *   the nearest e4m3fn value (ties to even) and saturated to +-448 (all codes 0 when
 *   amax is 0),
 *   k_scale[row] = scale, k_cache[row][d] = code[d]; V the same.
 * Inputs must be finite (codes of NaN or infinite inputs are unspecified).  Slots past
 * the cache are skipped and reported through *status.  Rows of different tokens must
 * not share a slot.  One kernel launch on `stream`; no host synchronisation, no
 * allocation.  Returns PA_ERR_INVALID_ARG for a missing pointer or a bad size (also
 * num_tokens * num_kv_heads above 2^31 - 1), PA_ERR_ALIGN for a misaligned pointer,
 * PA_ERR_UNSUPPORTED for head_dim or page_size outside the list, PA_ERR_CUDA when the
 * launch fails. */
pa_status_t pa_kv_quantize_write(const pa_kv_write_args_t *args, void *stream);

/* ---- the indexer: block score and top-k page selection for the sparse decode ---- */

#define PA_DEV_BAD_INDEX_ROW 0x200u /* pa_index_topk: q_len < 0 or > max_q_len, context_len < q_len, rows past num_rows, or more pages than the stride (the request's rows are skipped) */

/* Arguments of pa_index_topk.  All pointers are device pointers. */
typedef struct pa_index_args {
  const void *q;                 /* bf16 [num_rows, index_heads, head_dim], 16-B aligned */
  const void *k_cache;           /* index cache, e4m3 bytes [num_pages, page_size, head_dim], 16-B aligned */
  const float *k_scale;          /* fp32 [num_pages, page_size], or NULL: codes read at scale 1 */
  const int32_t *block_table;    /* [num_seqs, block_table_stride] physical page of each logical page */
  const int32_t *context_lens;   /* [num_seqs] */
  const int32_t *cu_seqlens_q;   /* [num_seqs + 1]: rows of request r are [cu[r], cu[r+1]) */
  int32_t *selected;             /* out: [num_rows, topk] logical pages, -1 after num_selected */
  int32_t *num_selected;         /* out: [num_rows] */
  float *scores;                 /* out: [num_rows, block_table_stride] page scores (log2 units),
                                    -inf where a page holds no attended position; 16-B aligned */
  uint32_t *status;              /* nullable: PA_DEV_BAD_PAGE, PA_DEV_BAD_INDEX_ROW are OR-ed in */
  int64_t num_pages;
  int32_t num_seqs;
  int32_t num_rows;
  int32_t index_heads;           /* >= 1; max_q_len * index_heads <= 16 */
  int32_t head_dim;              /* 128 */
  int32_t page_size;             /* 16, 32, 64 or 128 */
  int32_t topk;                  /* 1 .. 1024 */
  int32_t block_table_stride;    /* 1 .. 16384 */
  int32_t max_q_len;             /* bound on any request's q_len, >= 1 */
  float sm_scale;                /* > 0 */
  int32_t reserved;              /* 0 */
} pa_index_args_t;

/* The indexer step before the sparse decode (ROCm/ATOM PR 2122, section 1: the index
 * cache of (num_blocks, 128, 128) e4m3 codes and the block score q . k * sm_scale * log2(e);
 * section 2: rows map to requests through cu_seqlens_q, and row tok of a request with
 * context L and q_len rows attends positions < L - q_len + tok + 1).  For each row:
 *   s[h][p] = sm_scale * log2(e) * sum_d q[row][h][d] * k[p][d] * k_scale[p] over the
 *     attended positions p, where k is the index key at p (through the block table);
 *   scores[row][b] = log2 sum_h sum_{attended p in page b} 2^s[h][p] (-inf if none);
 *   selected[row] = the row's last attended page, then the other candidates by descending
 *     score (equal scores: lower page first), topk entries at most, -1 after.
 * With q_len 1 rows are requests, and selected / num_selected are pa_decode's
 * selected_pages / num_selected.  Inputs must be finite.  Two kernel launches on
 * `stream`; no host synchronisation, no allocation.  PA_ERR_INVALID_ARG for a missing
 * pointer or a value out of range, PA_ERR_ALIGN for a misaligned pointer,
 * PA_ERR_UNSUPPORTED for head_dim, page_size or max_q_len * index_heads outside the
 * limits above, PA_ERR_CUDA when a launch fails. */
pa_status_t pa_index_topk(const pa_index_args_t *args, void *stream);

/* ---- the merge of a context split across GPUs ---- */

/* Arguments of pa_lse_merge.  All pointers are device pointers. */
typedef struct pa_lse_merge_args {
  const float *part_out;   /* fp32 [num_parts, num_rows, num_heads, head_dim]: each part's normalised
                              attention output (pa_decode with PA_OUT_F32), 16-B aligned */
  const float *part_lse;   /* fp32 [num_parts, num_rows, num_heads]: each part's natural-log LSE
                              (pa_decode's lse; -inf where the part attended no position) */
  void *out;               /* [num_rows, num_heads, head_dim], bf16 or fp32 per out_dtype, 16-B aligned */
  float *lse;              /* fp32 [num_rows, num_heads] merged LSE, or NULL */
  int32_t num_parts;       /* 1 .. 64 */
  int32_t num_rows;        /* >= 0; 0 enqueues nothing */
  int32_t num_heads;       /* >= 1 */
  int32_t head_dim;        /* 128 */
  int32_t out_dtype;       /* PA_OUT_BF16 (round to nearest even) or PA_OUT_F32 */
  int32_t reserved;        /* 0 */
} pa_lse_merge_args_t;

/* Merges attention partials computed over disjoint parts of each request's positions: the
 * combine step of a long context split across GPUs (each GPU decodes its own pages with
 * pa_decode, PA_OUT_F32 and an lse; the parts are gathered, then merged here).  It is the
 * merge of the split-K partition triple -- maximum logit, exponential sum and partial
 * output per partition, ROCm/ATOM PR 2710, "Smaller" -- with each part's (max, sum) carried
 * as its lse; MiniMax-M3 is served across four GPUs (ROCm/ATOM PR 2614, "Validation").
 * For every (row, head) v, over the parts i with lse_i > -inf:
 *   M = max_i lse_i, w_i = exp(lse_i - M),
 *   out[v] = sum_i w_i part_out_i[v] / sum_i w_i,   lse[v] = M + log sum_i w_i;
 * no such part gives out = 0 and lse = -inf (an empty part's output is never read).
 * One kernel launch on `stream`; no host synchronisation, no allocation.
 * PA_ERR_INVALID_ARG for a missing pointer or a bad size, PA_ERR_ALIGN for a misaligned
 * pointer, PA_ERR_UNSUPPORTED for head_dim other than 128 or more than 64 parts,
 * PA_ERR_CUDA when the launch fails. */
pa_status_t pa_lse_merge(const pa_lse_merge_args_t *args, void *stream);

/* ---- attention mass: what each cached token has been worth to the queries so far ---- */

/* Arguments of pa_attn_mass.  All pointers are device pointers. */
typedef struct pa_attn_mass_args {
  const void *q;                 /* bf16 [num_rows, num_kv_heads * group_size, head_dim], 16-B aligned */
  const void *k_cache;           /* [num_pages, num_kv_heads, page_size, head_dim], e4m3 or bf16; 16-B aligned */
  const float *k_scale;          /* fp32 [num_pages, num_kv_heads, page_size]; PER_TOKEN only, 16-B aligned */
  const int32_t *block_table;    /* [num_seqs, block_table_stride] */
  const int32_t *context_lens;   /* [num_seqs]: tokens in each request's cache, own q_len included */
  const int32_t *cu_seqlens_q;   /* [num_seqs + 1]: rows of request r are [cu[r], cu[r+1]) */
  const float *lse;              /* fp32 [num_rows, num_kv_heads * group_size]: lse of the same step's pa_decode over
                                    the whole context (not of a sparse plan; natural log; -inf: no weight) */
  const float *mass;             /* fp32 [num_seqs, num_kv_heads, mass_stride]; may be NULL when decay is 0 */
  float *mass_out;               /* same shape; may be `mass` itself (any other overlap, also with q, lse or the index
                                    inputs, is refused) */
  uint32_t *status;              /* nullable: PA_DEV_BAD_PAGE, PA_DEV_BAD_CONTEXT, PA_DEV_BAD_QLEN,
                                    PA_DEV_TIMEOUT are OR-ed in */
  int64_t num_pages;
  int32_t num_seqs;              /* 0 .. 4096; 0 enqueues nothing */
  int32_t num_rows;
  int32_t num_kv_heads;          /* 1 .. 64 */
  int32_t group_size;            /* 16 */
  int32_t head_dim;              /* 128 */
  int32_t page_size;             /* 16, 32, 64 or 128 */
  int32_t kv_dtype;              /* PA_KV_* */
  int32_t scale_mode;            /* FP8: SCALAR or PER_TOKEN; BF16: NONE */
  int32_t block_table_stride;
  int32_t mass_stride;           /* positions per (request, KV head) row of the mass */
  int32_t max_q_len;             /* bound on any request's q_len, 1 .. 64 */
  float k_scale_scalar;          /* SCALAR only */
  float sm_scale;                /* > 0 */
  float decay;                   /* 0 .. 1: what the mass so far is multiplied by */
  int32_t reserved;              /* 0 */
} pa_attn_mass_args_t;

/* Adds one dense decode step's attention weights to the mass of the cached tokens, the quantity
 * by which pa_evict_select keeps them.  The lse of a decode over selected pages covers those alone, while every
 * position is weighed here: tokens that nobody attended would gain weight, even above one.  For request r with context L, q_len rows and KV head
 * h, and every position p < L:
 *   w[p] = sum over its rows t and the 16 query heads g of h, where p < L - q_len + t + 1,
 *          of exp(sm_scale * q[t][g] . k[p] * k_scale[p] - lse[t][g]),
 *   mass_out[r][h][p] = (p < L - q_len ? decay * mass[r][h][p] : 0) + w[p].
 * The step's own tokens start from zero, so a slot's earlier owner leaves nothing behind, and
 * with decay 0 `mass` is not read.  Positions >= L, and requests without rows, are left as they are
 * (in mass_out).  A position on a bad page gets w = 0.  A request with a bad length is skipped.
 * The mass belongs to the request, not to the page: requests may share pages (a common prefix,
 * beams).  Sums and exponentials are fp32 and always in the same order; with an e4m3 cache a query row is held
 * as pairs of e4m3 numbers, exactly for elements within 2^-14 of the row's largest and to 2^-22 of that for
 * smaller ones.  Inputs other than lse's -inf must be finite.  One kernel launch on `stream`; no host synchronisation, no allocation.
 * PA_ERR_INVALID_ARG for a missing pointer, a value out of range or an overlap of mass and
 * mass_out other than equality, PA_ERR_ALIGN for a misaligned pointer, PA_ERR_UNSUPPORTED for
 * a shape or mode outside the limits above, PA_ERR_CAPACITY when num_pages * num_kv_heads *
 * page_size passes 2^31 - 1, PA_ERR_CUDA when the launch fails. */
pa_status_t pa_attn_mass(const pa_attn_mass_args_t *args, void *stream);

/* ---- eviction: which tokens a bounded cache keeps, and their move to the front ---- */

/* A pa_decode on a plan without PA_PLAN_NO_PDL reads its index inputs before the kernel enqueued
 * just before it has completed (see the flag).  pa_evict_select writes new_lens and
 * pa_beam_reorder writes block_table_out, which are such inputs: another kernel has to lie between
 * them and that decode (the write of the step's new tokens does; a second pa_decode does not, it may let
 * the next one start before it has waited itself), or the plan has to have the flag.
 * The indexer's key cache is neither compacted nor reordered by these calls: see pa_kv_compact and pa_beam_reorder. */

#define PA_DEV_BAD_KEEP 0x400u /* pa_kv_compact: new_lens outside [0, keep_stride] or past the tables, or a keep row
                                  that is not ascending positions of the request's cache */

/* Arguments of pa_evict_select.  All pointers are device pointers. */
typedef struct pa_evict_select_args {
  const float *mass;             /* fp32 [num_seqs, num_kv_heads, mass_stride] */
  const int32_t *context_lens;   /* [num_seqs] */
  int32_t *keep;                 /* out: [num_seqs, num_kv_heads, budget] kept positions, ascending, -1 after */
  int32_t *new_lens;             /* out: [num_seqs] min(context_len, budget) */
  uint32_t *status;              /* nullable: PA_DEV_BAD_CONTEXT, PA_DEV_TIMEOUT are OR-ed in */
  int32_t num_seqs;              /* >= 0, num_seqs * num_kv_heads <= 65535; 0 enqueues nothing */
  int32_t num_kv_heads;          /* 1 .. 64 */
  int32_t mass_stride;           /* 1 .. 2^30 */
  int32_t budget;                /* >= 1: most tokens kept per (request, KV head) */
  int32_t keep_first;            /* >= 0: positions [0, keep_first) always stay */
  int32_t keep_recent;           /* >= 0: the last keep_recent positions always stay;
                                    keep_first + keep_recent <= budget */
  int32_t reserved;              /* 0 */
} pa_evict_select_args_t;

/* Chooses, for every (request, KV head), the positions that stay when its cache is cut to
 * `budget` tokens.  With context L <= budget all of them stay.  Else the first keep_first, the
 * last keep_recent, and of those between the ones with the largest mass until there are budget
 * of them; equal masses (0 and -0 are equal) stay lowest position first, and a NaN counts as less
 * than any number.  The result is exact, whatever the values.  A request whose context is negative
 * or beyond mass_stride is flagged: its keep rows are all -1 and its new_lens 0.  keep and new_lens
 * share no byte with each other, mass or context_lens.  One kernel
 * launch on `stream`; no host synchronisation, no allocation.  PA_ERR_INVALID_ARG for a missing
 * pointer, a value out of range or such an overlap, PA_ERR_ALIGN for a pointer not aligned to 4 bytes,
 * PA_ERR_UNSUPPORTED for a shape beyond the limits above, PA_ERR_CUDA when the launch fails. */
pa_status_t pa_evict_select(const pa_evict_select_args_t *args, void *stream);

/* Arguments of pa_kv_compact.  All pointers are device pointers. */
typedef struct pa_kv_compact_args {
  const int32_t *keep;           /* [num_seqs, num_kv_heads, keep_stride] positions, strictly ascending per row */
  const int32_t *new_lens;       /* [num_seqs]: entries of every keep row of the request */
  const int32_t *block_table;    /* [num_seqs, block_table_stride]: where the cache is */
  const int32_t *dst_block_table;/* [num_seqs, dst_block_table_stride]: where it goes; NULL moves it in place, to
                                    the front of its own pages */
  void *k_cache;                 /* [num_pages, num_kv_heads, page_size, head_dim], e4m3 or bf16; 16-B aligned */
  void *v_cache;
  float *k_scale;                /* fp32 [num_pages, num_kv_heads, page_size]; PER_TOKEN only, 4-B aligned */
  float *v_scale;
  const float *mass;             /* nullable: fp32 [num_seqs, num_kv_heads, mass_stride] */
  float *mass_out;               /* where the kept tokens' mass goes: [num_seqs, num_kv_heads, mass_out_stride]; in place
                                    `mass` itself with the same stride, with dst_block_table not overlapping it; and
                                    not overlapping keep, new_lens or the tables */
  uint32_t *status;              /* nullable: PA_DEV_BAD_KEEP, PA_DEV_BAD_PAGE are OR-ed in */
  int64_t num_pages;
  int32_t num_seqs;              /* >= 0, num_seqs * num_kv_heads <= 65535; 0 enqueues nothing */
  int32_t num_kv_heads;          /* 1 .. 64 */
  int32_t head_dim;              /* 128 */
  int32_t page_size;             /* 16, 32, 64 or 128 */
  int32_t kv_dtype;              /* PA_KV_* */
  int32_t scale_mode;            /* FP8: SCALAR or PER_TOKEN; BF16: NONE */
  int32_t keep_stride;           /* >= 1 */
  int32_t block_table_stride;
  int32_t dst_block_table_stride;
  int32_t mass_stride;
  int32_t mass_out_stride;
  int32_t reserved;              /* 0 */
} pa_kv_compact_args_t;

/* Moves the kept tokens to the front: for every (request r, KV head h) and i < new_lens[r],
 * slot i of r's destination pages takes the K and V rows, the scales and the mass of position
 * keep[r][h][i], bit for bit; afterwards new_lens is the request's context_lens.  Positions
 * keep their order, so causal cutoffs and recency stay meaningful.  The indexer's keys and scales are not moved: page
 * scores of pa_index_topk belong to the tokens that were there before, until the caller has moved its index cache
 * by the same keep (or written it anew).
 * In place nothing but the request's own first pages is written, and pages all of whose tokens
 * stay are not; slots past new_lens are left as they are.  Pages that another request reads
 * as well (a common prefix, beams) must not be compacted in place: give dst_block_table, whose pages
 * are then written and must be nobody else's (not the source's either).  An entry that is not above the one before it
 * or lies past the tables, and a bad page, are flagged and that token is not moved.  One kernel launch
 * on `stream`; no host synchronisation, no allocation.  PA_ERR_INVALID_ARG for a missing pointer,
 * a value out of range, or mass_out against the rule above, PA_ERR_ALIGN for a misaligned pointer,
 * PA_ERR_UNSUPPORTED for a shape or mode outside the limits above, PA_ERR_CAPACITY when num_pages *
 * num_kv_heads * page_size passes 2^31 - 1, PA_ERR_CUDA when the launch fails. */
pa_status_t pa_kv_compact(const pa_kv_compact_args_t *args, void *stream);

/* ---- beam search over the paged cache ---- */

#define PA_DEV_BAD_BEAM 0x800u /* pa_beam_reorder: a parent outside [0, num_beams), or beams of one request with
                                  different lengths (the request's rows are carried over as they are) */

enum { PA_LOGITS_BF16 = 0, PA_LOGITS_F32 = 1 };

/* Arguments of pa_beam_select.  All pointers are device pointers; beams of request n are
 * [n * num_beams, (n + 1) * num_beams). */
typedef struct pa_beam_select_args {
  const void *logits;            /* [num_reqs * num_beams, logits_stride], the first `vocab` of each row; aligned to
                                    its element (rows need no 16-byte alignment) */
  const float *scores;           /* fp32 [num_reqs, num_beams]: sum of log-probabilities so far (-inf: no such beam yet) */
  const uint8_t *finished;       /* nullable [num_reqs, num_beams]: non-zero for a beam that has ended */
  const int32_t *lengths;        /* nullable [num_reqs, num_beams]: tokens of each beam; needed when
                                    length_penalty is not 0 */
  int32_t *tokens;               /* out: [num_reqs, num_beams] token that continues each new beam */
  int32_t *parents;              /* out: [num_reqs, num_beams] beam (of the same request) that it continues */
  float *scores_out;             /* out: its sum of log-probabilities; may be `scores` */
  uint8_t *finished_out;         /* nullable out: may be `finished` */
  int32_t *lengths_out;          /* nullable out: may be `lengths`; needs lengths */
  int64_t logits_stride;         /* elements between rows, >= vocab */
  int32_t num_reqs;              /* 0 .. 65535; 0 enqueues nothing */
  int32_t num_beams;             /* 1 .. 32 */
  int32_t vocab;                 /* 1 .. 2^24 */
  int32_t logits_dtype;          /* PA_LOGITS_* */
  int32_t eos_token;             /* the token that ends a beam, or -1: none; needed (>= 0) with finished */
  float length_penalty;          /* >= 0; the exponent is this fp32 number (0.6f is 0.60000002384) */
  int32_t reserved;              /* 0 */
} pa_beam_select_args_t;

/* One step of beam search: the num_beams best continuations of each request's beams, best first.
 * A live beam b continues with every token v at total = scores[b] + logits[b][v] - logsumexp(logits[b])
 * and length lengths[b] + 1; a finished one only with eos_token, at its own score and length.
 * Candidates are ranked by total / max(length, 1)^length_penalty, equal ranks by the lower beam,
 * then the lower token.  A candidate that does not exist or whose total is NaN (a row of -inf
 * logits, a NaN or +inf among them) counts as -inf and is taken, lowest beam and token first, only
 * where nothing better is left; its scores_out is -inf.  finished_out is set where the parent
 * had ended or the token is eos_token.  Totals and ranks are fp64.  The
 * log-sum-exp in them adds fp32 exponentials, off by 2^-22 of themselves at most, in fp32 over a thread's share of
 * a row and in steps of 2^-36 across threads; it measures some 1e-7 from fp64's, and totals of two beams that
 * are closer than that may come in either order unless their rows are equal.  The power of a length is CUDA's pow, within
 * two units of its last place, and with a length_penalty of 1 the length itself.  Ranks that round to the same number
 * are equal, also those of different logits.  scores_out is rounded once.  One kernel launch on `stream`;
 * no host synchronisation, no allocation.  Outputs share no byte with each other or an input, but for an output
 * that begins where its own input does.  PA_ERR_INVALID_ARG for a missing pointer, a value out
 * of range or another overlap, PA_ERR_ALIGN for a misaligned pointer, PA_ERR_UNSUPPORTED for more than 32 beams,
 * 65535 requests or 2^24 tokens, PA_ERR_CUDA when the launch fails. */
pa_status_t pa_beam_select(const pa_beam_select_args_t *args, void *stream);

#define PA_MAX_BEAM_STATES 4

/* Arguments of pa_beam_reorder.  All pointers but state_in and state_out themselves are device pointers. */
typedef struct pa_beam_reorder_args {
  const int32_t *parents;        /* [num_reqs, num_beams]: pa_beam_select's */
  const int32_t *context_lens;   /* [num_reqs * num_beams]: tokens in each beam's cache, equal within a request */
  const int32_t *block_table;    /* [num_reqs * num_beams, block_table_stride] */
  int32_t *block_table_out;      /* same shape; must not overlap block_table, parents, context_lens or a state */
  void *k_cache;                 /* [num_pages, num_kv_heads, page_size, head_dim], e4m3 or bf16; 16-B aligned */
  void *v_cache;
  float *k_scale;                /* fp32 [num_pages, num_kv_heads, page_size]; PER_TOKEN only, 4-B aligned */
  float *v_scale;
  uint32_t *status;              /* nullable: PA_DEV_BAD_BEAM, PA_DEV_BAD_CONTEXT, PA_DEV_BAD_PAGE are OR-ed in */
  const void *state_in[PA_MAX_BEAM_STATES];  /* num_states device arrays of num_reqs * num_beams rows of */
  void *state_out[PA_MAX_BEAM_STATES];       /*   state_bytes bytes each; outs overlap nothing else */
  int64_t state_bytes[PA_MAX_BEAM_STATES];   /* > 0 */
  int64_t num_pages;
  int32_t num_states;            /* 0 .. 4 */
  int32_t num_reqs;              /* 0 .. 65535; 0 enqueues nothing */
  int32_t num_beams;             /* 1 .. 32; num_reqs * num_beams <= 65535 */
  int32_t num_kv_heads;          /* 1 .. 64 */
  int32_t head_dim;              /* 128 */
  int32_t page_size;             /* 16, 32, 64 or 128 */
  int32_t kv_dtype;              /* PA_KV_* */
  int32_t scale_mode;            /* FP8: SCALAR or PER_TOKEN; BF16: NONE */
  int32_t block_table_stride;
  int32_t reserved;              /* 0 */
} pa_beam_reorder_args_t;

/* Lets every beam's history follow its parent without copying whole caches.  With L = the
 * request's context length and f = L / page_size full pages, row j of block_table_out holds the
 * parent's first f entries, shared by reference; then, if L is not a multiple of page_size, the page
 * that the beam's next token goes to; then row j's own later entries as they were.  That
 * partial page is never shared: the first child (lowest j) of a parent takes the parent's, and every further
 * child takes the partial page of a beam that has no children (there are as many of those as
 * further children, in ascending order), into which the L % page_size tokens of the parent's page are
 * copied (K, V and scales of all KV heads).  So the partial pages of a request's beams must be its own
 * and distinct before the call, and are afterwards; nothing is allocated.  With parents all 0
 * the call also spreads a prompt, cached once in beam 0's pages, over all beams.  Each state's row j becomes
 * its parent's row (mass, token history).  The indexer's keys are not copied: the page that a further child takes
 * keeps the childless beam's, and pa_index_topk scores it by them until the caller has copied the parent's.  A flagged request keeps its rows, as if each beam were its
 * own parent.  One kernel launch on `stream`; no host synchronisation, no allocation.
 * PA_ERR_INVALID_ARG for a missing pointer, a value out of range or an overlap, PA_ERR_ALIGN for
 * a misaligned pointer, PA_ERR_UNSUPPORTED for a shape or mode outside the limits above,
 * PA_ERR_CAPACITY when num_pages * num_kv_heads * page_size passes 2^31 - 1, PA_ERR_CUDA when the
 * launch fails. */
pa_status_t pa_beam_reorder(const pa_beam_reorder_args_t *args, void *stream);

/* ---- a prompt's way into the cache: pages and slots, rotary positions, attention ---- */

#define PA_DEV_PAGE_POOL 0x1000u /* pa_page_assign: a request needed more pages than were left; pa_page_release: the
                                    stack has no room for a request's pages */

/* Arguments of pa_page_assign.  All pointers are device pointers. */
typedef struct pa_page_assign_args {
  const int32_t *context_lens;   /* [num_seqs]: tokens in each request's cache before the step */
  const int32_t *cu_seqlens_q;   /* [num_seqs + 1]: the new tokens of request r are rows [cu[r], cu[r+1]) */
  int32_t *block_table;          /* [num_seqs, block_table_stride]: the new pages are entered */
  const int32_t *free_pages;     /* [free_capacity]: a stack of free pages, its top at num_free - 1 */
  const int32_t *num_free;       /* [1] */
  int32_t *num_free_out;         /* [1]; may be num_free */
  int32_t *new_lens;             /* out: [num_seqs] context lengths with the new tokens; may be context_lens */
  int64_t *slot_mapping;         /* out: [num_rows] slot of every row, -1 where it has none (pa_kv_quantize_write's) */
  int32_t *positions;            /* nullable out: [num_rows] position of every row in its request (pa_rope's) */
  uint32_t *status;              /* nullable: PA_DEV_BAD_CONTEXT, PA_DEV_BAD_QLEN, PA_DEV_BAD_PAGE, PA_DEV_PAGE_POOL */
  int64_t num_pages;             /* 1 .. 2^31 - 1: pages of the cache */
  int32_t num_seqs;              /* 0 .. 2^30 */
  int32_t num_rows;              /* >= 0: rows of the step, padding behind the last request's among them */
  int32_t block_table_stride;
  int32_t page_size;             /* 16, 32, 64 or 128 */
  int32_t free_capacity;         /* >= 1 */
  int32_t reserved;              /* 0 */
} pa_page_assign_args_t;

/* Gives requests that grow their pages, and their new tokens slots and positions.  With L = context_lens[r] and
 * q = cu[r+1] - cu[r], request r needs ceil((L + q) / page_size) - ceil(L / page_size) pages.  In the order of the
 * requests each takes its pages off the top of the stack, lower positions first, as long as the pool lasts: from
 * the first request on that needs more than is left, those that need a page are not served (PA_DEV_PAGE_POOL), and
 * those that need none still are.  A served request's row of position p gets the slot
 * block_table[r][p / page_size] * page_size + p % page_size, and new_lens[r] = L + q; one that is not served gets no
 * page, slots of -1 and new_lens[r] = L.  positions are L + row - cu[r] for both.  Rows of no request (before cu[0], behind
 * cu[num_seqs]) get slot -1 and position 0.  Entries of the block table other than the new pages', and the
 * stack, are left as they are; num_free_out is what is left.  So the table's partial pages must be the request's own, as they are
 * after pa_beam_reorder.  A request with a negative context or one whose tokens pass the table or 2^31 - 1 is not served
 * (PA_DEV_BAD_CONTEXT).  If cu does not ascend from 0 or more to num_rows or fewer, no request is served and every position
 * is 0 (PA_DEV_BAD_QLEN).  num_free is taken as within 0 .. free_capacity.  A page outside [0, num_pages), off the stack or in
 * the table, gives its rows slot -1 (PA_DEV_BAD_PAGE); off the stack it is entered as it stands, and the decode flags it again.
 * Outputs share no byte with each other or with an input, but for the two pairs above at the same address.
 * One kernel launch on `stream`, two for more than 16384 rows with lengths or count updated in place, none where there is nothing to
 * write (no requests, no rows, num_free_out at num_free; pointers to nothing may be NULL); no host synchronisation, no allocation.  A pa_decode on a plan without PA_PLAN_NO_PDL
 * reads new_lens and block_table before the kernel enqueued just before it has completed: another kernel that is no decode
 * has to lie between (pa_rope and pa_kv_quantize_write do).  PA_ERR_INVALID_ARG for a missing pointer, a value out of range or an overlap,
 * PA_ERR_ALIGN for a misaligned pointer, PA_ERR_UNSUPPORTED for another page size, PA_ERR_CUDA when the launch fails. */
pa_status_t pa_page_assign(const pa_page_assign_args_t *args, void *stream);

/* Arguments of pa_page_release.  All pointers are device pointers. */
typedef struct pa_page_release_args {
  const int32_t *context_lens;   /* [num_seqs]: tokens that the request's pages were taken for */
  const int32_t *new_lens;       /* [num_seqs]: tokens that stay; 0 for a request that has ended */
  const int32_t *block_table;    /* [num_seqs, block_table_stride] */
  int32_t *free_pages;           /* [free_capacity]: the stack, its top at num_free - 1 */
  const int32_t *num_free;       /* [1] */
  int32_t *num_free_out;         /* [1]; may be num_free */
  uint32_t *status;              /* nullable: PA_DEV_BAD_CONTEXT, PA_DEV_BAD_PAGE, PA_DEV_PAGE_POOL */
  int64_t num_pages;             /* 1 .. 2^31 - 1 */
  int32_t num_seqs;              /* 0 .. 2^30 */
  int32_t block_table_stride;
  int32_t page_size;             /* 16, 32, 64 or 128 */
  int32_t free_capacity;         /* >= 1 */
  int32_t reserved;              /* 0 */
} pa_page_release_args_t;

/* Takes pages back: entries [ceil(new_lens[r] / page_size), ceil(context_lens[r] / page_size)) of row r of the block
 * table go on top of the stack, request by request, lower positions first.  A request that does not shrink gives none.  The
 * table is left as it is (what lies behind a context length is not read).  Pages that another request reads as well (a
 * common prefix, beams) must not be given back: who counts references is the caller.  From the first request on whose pages
 * pass free_capacity, those that have pages to give back keep them (PA_DEV_PAGE_POOL: such a pool has been given a page twice).  A request with a
 * negative length or a context beyond the table gives none back (PA_DEV_BAD_CONTEXT).  A page outside [0, num_pages) goes on
 * the stack as it stands and is flagged (PA_DEV_BAD_PAGE).  num_free is taken as within 0 .. free_capacity.  Outputs share no byte with each
 * other or with an input, but for num_free_out at num_free.  One kernel launch on `stream`, two where more than 16384 pages could be
 * given back (by the table's and the stack's sizes) and num_free_out is num_free, none without requests and with num_free_out at num_free; no host synchronisation, no allocation.  PA_ERR_INVALID_ARG for a missing pointer, a value out of range or an overlap, PA_ERR_ALIGN for a misaligned pointer,
 * PA_ERR_UNSUPPORTED for another page size, PA_ERR_CUDA when the launch fails. */
pa_status_t pa_page_release(const pa_page_release_args_t *args, void *stream);

enum { PA_ROPE_BF16 = 0, PA_ROPE_F32 = 1 };
enum { PA_ROPE_HALF = 0, PA_ROPE_PAIRS = 1 };

/* Arguments of pa_rope.  All pointers are device pointers; strides are elements between tokens, and a token's heads lie
 * one behind the other, so that views of one projection's output can be given. */
typedef struct pa_rope_args {
  const void *q;                 /* [num_tokens, num_q_heads, head_dim], aligned to its element */
  const void *k;                 /* [num_tokens, num_kv_heads, head_dim]; NULL with num_kv_heads 0 */
  const int32_t *positions;      /* [num_tokens], of either sign */
  const int64_t *freqs;          /* [rot_dim / 2]: turns per position of each pair, times 2^64, modulo 2^64 */
  void *q_out;                   /* as q; may be q with q's stride */
  void *k_out;                   /* as k; may be k with k's stride */
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;  /* >= heads * head_dim */
  int32_t num_tokens;            /* >= 0; 0 enqueues nothing */
  int32_t num_q_heads;           /* >= 1 */
  int32_t num_kv_heads;          /* >= 0 */
  int32_t head_dim;              /* 128 */
  int32_t rot_dim;               /* even, 2 .. 128: the head's first rot_dim elements turn, the others are carried over */
  int32_t dtype;                 /* PA_ROPE_* */
  int32_t layout;                /* PA_ROPE_HALF: pair i is elements (i, i + rot_dim / 2); PA_ROPE_PAIRS: (2i, 2i + 1) */
  int32_t inverse;               /* 1 turns back: the gradient of the rotation, or a key that is to be moved; else 0 */
  float scale;                   /* finite; what the turned elements are multiplied by (1, or that of a stretched context) */
  int32_t reserved;              /* 0 */
} pa_rope_args_t;

/* Rotary positions: pair i = (a, b) of every head of a token at position p becomes
 *   (a cos t - b sin t, b cos t + a sin t) * scale,   t = 2 pi p freqs[i] / 2^64   (-t with inverse),
 * in fp32, rounded once to the type.  The angle is reduced in 64-bit integers: p * freqs[i] modulo 2^64 is the fraction of
 * a turn, exactly, however far the position, so far positions are as exact as near ones.  One kernel launch on `stream`; no host
 * synchronisation, no allocation.  Outputs share no byte with each other or another input (rows of one buffer interleave only
 * with equal strides).  PA_ERR_INVALID_ARG for a missing pointer, a value out of range or an overlap, PA_ERR_ALIGN for a misaligned pointer, PA_ERR_UNSUPPORTED for
 * head_dim other than 128 or more than 65535 heads of both together, PA_ERR_CUDA when the launch fails. */
pa_status_t pa_rope(const pa_rope_args_t *args, void *stream);

/* Arguments of pa_prompt_attn.  All pointers are device pointers; strides are elements between tokens, and a token's heads
 * lie one behind the other, so that views of one projection's output can be given. */
typedef struct pa_prompt_attn_args {
  const void *q;                 /* bf16 [num_rows, num_kv_heads * group_size, head_dim], 16-B aligned */
  const void *k;                 /* bf16 [num_rows, num_kv_heads, head_dim], 16-B aligned */
  const void *v;                 /* as k */
  const int32_t *cu_seqlens;     /* [num_seqs + 1]: sequence s is rows [cu[s], cu[s+1]) */
  void *out;                     /* [num_rows, num_kv_heads * group_size, head_dim], bf16 or fp32 per out_dtype, dense, 16-B aligned */
  float *lse;                    /* nullable: fp32 [num_rows, num_kv_heads * group_size], natural log */
  uint32_t *status;              /* nullable: PA_DEV_BAD_QLEN, PA_DEV_TIMEOUT are OR-ed in */
  int64_t q_stride, k_stride, v_stride;  /* multiples of 8, >= heads * head_dim */
  int32_t num_seqs;              /* 0 .. 4096; 0 enqueues nothing */
  int32_t num_rows;              /* 0 .. 2^24; 0 enqueues nothing */
  int32_t num_kv_heads;          /* 1 .. 64 */
  int32_t group_size;            /* 1 .. 64 */
  int32_t head_dim;              /* 128 */
  int32_t out_dtype;             /* PA_OUT_BF16 or PA_OUT_F32 */
  float sm_scale;                /* > 0 */
  int32_t reserved;              /* 0 */
} pa_prompt_attn_args_t;

/* Causal attention over whole prompts, packed one behind the other: row t of sequence s (its t-th token) and query head j
 * of KV head h = j / group_size attend the sequence's tokens 0 .. t,
 *   out[t][j] = sum_i softmax_i(sm_scale * q[t][j] . k[i][h]) v[i][h],   lse[t][j] = log sum_i exp(sm_scale * q[t][j] . k[i][h]).
 * Scores, maxima, sums and accumulators are fp32; the softmax weights are rounded to bf16 for the second product (their sum is
 * taken before), so an fp32 output is good to 2^-8 of its terms and serves pa_lse_merge, which joins it with the part of a context
 * that is already cached (a decode over the cached pages with an fp32 output and lse).  What a row does not attend has no effect on it,
 * infinities and NaN included: later tokens, other sequences, rows of no sequence; rows of no sequence are left as they are.
 * A row whose scores are all -inf has an output of NaN (0 / 0) and an lse of -inf; one with a score of +inf or NaN has NaN in both.  An infinite
 * value whose weight is 0 in fp32 (a score of -inf, or 2^-126 of the row's largest) gives an attending row the infinity or NaN (0 * inf),
 * and which of them may differ with what else the call has; any other weight counts as in the formula.  Weights exceed 1 by 2^8 at most before
 * the division, so values beyond 2^120 / (number of tokens) may overflow.  Many values that are not finite are slow: each row adds those
 * of its last blocks one by one.
 * A sequence whose cu does not lie in order within 0 .. num_rows is left out (PA_DEV_BAD_QLEN); where others then overlap, rows may be left
 * unwritten.  A sequence's last bits may depend on how many rows the call has besides: equal calls give equal bits.  One kernel launch on
 * `stream`; no host synchronisation, no allocation.  out and lse share no byte with each other or an input.  PA_ERR_INVALID_ARG
 * for a missing pointer, a value out of range or an overlap, PA_ERR_ALIGN for a misaligned pointer or stride, PA_ERR_UNSUPPORTED for a shape outside the limits
 * above, PA_ERR_CUDA when the launch fails. */
pa_status_t pa_prompt_attn(const pa_prompt_attn_args_t *args, void *stream);

/* ---- test hooks: exact integer / byte outputs of the row map and the page gather ---- */

/* For every query row: (request, query token, causal cutoff) as int32 triples into the
 * device buffer row_map [num_rows, 3], computed by the same device code that maps rows
 * in pa_decode (ROCm/ATOM PR 2122, section 2).  Rows no request owns are left as is. */
pa_status_t pa_debug_row_map(pa_plan_t *plan, const pa_decode_args_t *args, int32_t *row_map,
                             void *stream);

/* Bytes per KV tile in pa_debug_gather's output. */
size_t pa_debug_gather_tile_bytes(const pa_plan_t *plan);

/* Runs pa_decode's schedule and page-gather path (block table, selected pages, tile
 * loads into shared memory) and, instead of attending, writes every tile it loaded to
 * `dump` at its global tile index: a 128-byte header of int32 (request, KV head, tile,
 * flags, context_len, q_len, first row, valid pages, then 8 first-positions and 8
 * physical pages, -1 where a page slot is empty), the K tile and the V tile as
 * [128 tokens][head_dim] elements with the swizzle undone, then (FP8 per-token) the
 * 128 K and 128 V scales.  Tiles are numbered request-major, then KV head, then tile;
 * dump must hold (number of tiles) * pa_debug_gather_tile_bytes bytes, given as
 * dump_bytes (tiles past it set PA_DEV_DUMP_RANGE and are skipped). */
pa_status_t pa_debug_gather(pa_plan_t *plan, const pa_decode_args_t *args, void *dump,
                            size_t dump_bytes, void *stream);

/* Launch trace of the mma.sync decode kernel, a diagnostic: the GPU global timer (ns) at
 * fixed points of each CTA's run, kept for each CTA's last 16 launches on the current
 * device.  Copies min(bytes, 2 MiB) of the array uint64 [16 slots][1024 CTAs][16 marks]
 * to host memory; slot = the CTA's launch count mod 16.  Marks: 0 entry, 1 prologue (the
 * schedule) done, 2 producer past the dependency wait, 3 consumers past it, 4 first tile
 * in warp 0, 5 warp 0 through the CTA's range, 6 partial stored, 7 arrival counted,
 * 8 / 9 merge start / end, 10 exit, 11 the CTA's launch count, 12 / 13 its tile range
 * [a, b), 14 merge duty bits; marks a launch does not reach keep older values.  Returns
 * PA_ERR_UNSUPPORTED unless the library was built with tracing (its kernels carry no
 * trace code otherwise), PA_ERR_CUDA if the copy fails. */
pa_status_t pa_debug_trace(void *host, size_t bytes);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDFP8_PA_H */
