/*
 * spec_attn.h -- C ABI of a GB300 (sm_103a) library for the attention of
 * speculative-decoding windows against a paged KV cache.
 *
 * The operation.  A batch holds P requests.  Request r brings a window of
 * W_r = q_indptr[r+1] - q_indptr[r] query rows (0 <= W_r <= 16: the seed
 * token plus k proposed tokens) and owns seq_len[r] keys in a paged K/V cache
 * shared by all requests.  The window's own W_r keys are already in the
 * cache as its last W_r keys, so ctx_r = seq_len[r] - W_r keys precede it.
 * Every window row attends to its request's cache under one of two masks:
 *
 *   causal-in-block: window row i sees keys 0 .. ctx_r + i (inclusive)
 *   non-causal:      every window row sees all seq_len[r] keys
 *
 * optionally narrowed, for causal calls, by a sliding window: with
 * window_left = n > 0, row i sees only keys max(0, ctx_r + i - n + 1) ..
 * ctx_r + i.  (The first page below names an attention window that its
 * non-causal draft layers leave unapplied, without defining it; this is the
 * plainest reading, and non-causal calls take no window.)
 *
 * and outputs are produced for window rows only, never for context rows.
 * Sources (titles of the pages this library restates):
 *   - "DFlash2 leaves the paged graph fast path at every c>1 and re-attends
 *     the whole batch context every decode step", sections "The route
 *     change" (paged store, Tq = 1+k rows, graph-captured), "The cost" (no
 *     outputs for context rows; non-causal draft layers see their request's
 *     whole span) and "Scope" (one shared paged pool, a batched block table,
 *     per-request seq_lens, P x (1+k) query rows).
 *   - "ChunkedSmallT re-streams full KV per query chunk (DFlash K>=8 verify
 *     at long context)", sections "Finding" (key-splitting plus a reduce
 *     kernel; the K/V sweep must not repeat per query chunk) and
 *     "Measurement" (q24 verify windows W = 8 and 16, bf16 and nvfp4 KV).
 *   - "perf(dflash): widen the verify window past the compact graph's
 *     four-row limit", section "What changed" (an unsupported width must not
 *     silently truncate; attention reads only seq_len entries).
 *
 * For each query row and head h (KV head h / (Hq/Hkv)):
 *   s_j = sm_scale * <q, k_j>,  O = sum_j softmax(s)_j v_j,
 *   LSE = max_j s_j + ln(sum_j exp(s_j - max_j s_j))     (natural log)
 * with fp32 accumulation; O is written as bf16 (round to nearest even),
 * LSE as fp32.
 *
 * Layouts (row-major; the pools may have a page stride, everything else is
 * dense):
 *   Q, O       [total_q_rows, Hq, head_dim] bf16; the rows of request r are
 *              q_indptr[r] .. q_indptr[r+1]-1, in window order.
 *   LSE        [total_q_rows, Hq] fp32.
 *   K/V pools  num_pages pages, page p at byte offset p * kv_page_stride
 *              (default: dense), each page [Hkv, page_size, row] with
 *              bf16:  row = head_dim bf16 values;
 *              NVFP4: row = head_dim/2 code bytes (two e2m1 codes per byte,
 *                     low nibble = even element), and scale pools laid out
 *                     the same way with page stride scale_page_stride and
 *                     row = head_dim/16 bytes (one OCP e4m3 scale per 16
 *                     contiguous elements), plus one fp32 global scale per
 *                     tensor: value = e2m1(code) * e4m3(scale) * gscale.
 *              A page stride lets K and V (and their scales) share one
 *              allocation, e.g. [num_pages, 2, Hkv, page_size, row].
 *   block_table [P, block_table_stride] int32: key j of request r lives in
 *              page block_table[r][j / page_size], slot j % page_size.
 *              Entries past ceil(seq_len[r] / page_size) are never read.
 *   seq_lens   [P] int32;  q_indptr [P+1] int32 (q_indptr[0] == 0).
 *
 * Ownership: every buffer is allocated and owned by the caller.  The library
 * allocates no device memory, makes no host<->device copy and never
 * synchronises inside spec_attn_run / spec_attn_run_traced, so both may be
 * captured into a CUDA graph.  A plan is a host object owned by the library
 * between spec_attn_plan_create() and spec_attn_plan_destroy().
 *
 * Errors: every function returns a spec_attn_status.  Host-side checks run
 * in spec_attn_plan_create() (shapes, limits, host copies of seq_lens and
 * q_indptr when given) and spec_attn_run() (null or misaligned pointers,
 * workspace size).  Device-side checks (a page id outside [0, num_pages), a
 * seq_len above the plan's max_seq_len or below its window, a window wider
 * than max_w) never fault: the kernels clamp the access, set a sticky error
 * word in the workspace and go on; spec_attn_check_device_status() reads and
 * clears it.
 */
#ifndef SPEC_ATTN_H
#define SPEC_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; declared here so this header needs no CUDA
 * include.  NULL means the legacy default stream. */
typedef struct CUstream_st* spec_attn_stream_t;

typedef enum spec_attn_status {
    SPEC_ATTN_OK = 0,
    SPEC_ATTN_E_INVALID_ARG = -1,          /* bad shape, pointer, alignment or value */
    SPEC_ATTN_E_UNSUPPORTED = -2,          /* valid but outside the library's limits */
    SPEC_ATTN_E_WORKSPACE_TOO_SMALL = -3,  /* workspace_bytes below the plan's need */
    SPEC_ATTN_E_CUDA = -4,                 /* a CUDA runtime call failed; see spec_attn_last_cuda_error */
    SPEC_ATTN_E_DEVICE_CHECK = -5          /* a device-side check tripped (check_device_status) */
} spec_attn_status;

typedef enum spec_attn_mask_mode {
    SPEC_ATTN_MASK_CAUSAL_IN_BLOCK = 0,
    SPEC_ATTN_MASK_NON_CAUSAL = 1
} spec_attn_mask_mode;

typedef enum spec_attn_kv_dtype {
    SPEC_ATTN_KV_BF16 = 0,
    SPEC_ATTN_KV_NVFP4 = 1
} spec_attn_kv_dtype;

typedef enum spec_attn_kernel_variant {
    SPEC_ATTN_VARIANT_AUTO = 0,       /* the library's choice for the shape */
    SPEC_ATTN_VARIANT_CUDA_CORE = 1,  /* fp32 FMA on CUDA cores */
    SPEC_ATTN_VARIANT_TCGEN05 = 2     /* 5th-generation tensor cores, TMEM accumulators */
} spec_attn_kernel_variant;

/* Device-status bits set by the kernels (spec_attn_check_device_status). */
#define SPEC_ATTN_DEV_BAD_PAGE      0x1u  /* block-table entry outside [0, num_pages) */
#define SPEC_ATTN_DEV_BAD_SEQ_LEN   0x2u  /* seq_len > max_seq_len or table capacity, or < W_r */
#define SPEC_ATTN_DEV_BAD_WINDOW    0x4u  /* W_r < 0, W_r > max_w, or rows past total_q_rows */
#define SPEC_ATTN_DEV_WAIT_TIMEOUT  0x8u  /* a pipeline wait gave up (bounded spin) */
#define SPEC_ATTN_DEV_OUT_OF_PAGES  0x10u /* spec_attn_build_tables: fewer free pages than the step needs */
#define SPEC_ATTN_DEV_BAD_FREE_LIST 0x20u /* spec_attn_build_tables: free and held pages exceed the pool */

/* Limits of the library. */
#define SPEC_ATTN_MAX_W 16
#define SPEC_ATTN_MAX_GROUP 16       /* Hq / Hkv */
#define SPEC_ATTN_MIN_PAGE_SIZE 16   /* page_size is 16, 32 or 64 */
#define SPEC_ATTN_MAX_PAGE_SIZE 64

typedef struct spec_attn_problem {
    int32_t num_reqs;            /* P >= 0 */
    int32_t total_q_rows;        /* rows of Q and O (sum of all W_r) */
    int32_t max_w;               /* upper bound on every W_r, 1..16 */
    int32_t num_q_heads;         /* Hq */
    int32_t num_kv_heads;        /* Hkv; Hq % Hkv == 0, Hq / Hkv <= 16 */
    int32_t head_dim;            /* 64, 128 or 256 */
    int32_t page_size;           /* keys per page: 16, 32 or 64 */
    int32_t num_pages;           /* pages in each pool (device bounds check); >= 1 when
                                    num_reqs > 0, even if no key is cached */
    int32_t block_table_stride;  /* int32 entries per block-table row; a row's capacity,
                                    stride x page_size keys, at most 2^31 - 1 */
    int32_t mask_mode;           /* spec_attn_mask_mode */
    int32_t kv_dtype;            /* spec_attn_kv_dtype */
    float sm_scale;              /* softmax scale; 0 selects 1/sqrt(head_dim) */
    int64_t max_seq_len;         /* upper bound on every seq_len the plan will see,
                                    at most 2^31 - 1 */
    int32_t force_splits;        /* 0: heuristic; n > 0: split the longest request's keys n ways */
    int32_t kernel_variant;      /* spec_attn_kernel_variant */
    int32_t w_invariant;         /* 1: W-invariant mode (below); 0: off */
    int32_t fixed_keys_per_split;/* W-invariant mode: keys per split, a multiple of 64
                                    (0 selects 64 x ceil(max_seq_len / 2048), at least
                                    512); ignored otherwise */
    int32_t window_left;         /* causal sliding window in keys; 0 = none (required
                                    for the non-causal mask) */
    int64_t kv_page_stride;      /* bytes from a K (or V) page to the next: 0 = dense
                                    (Hkv * page_size * row bytes); else a multiple of 16
                                    and at least the dense size */
    int64_t scale_page_stride;   /* NVFP4 scale pools, likewise (dense: Hkv * page_size
                                    * head_dim/16 bytes); ignored for bf16 */
    int32_t dense_block_kv;      /* 1: the window's own keys come from dense block
                                    tensors (spec_attn_run_dense_block), not the cache;
                                    bf16 caches only, not with w_invariant */
    int32_t early_metadata;      /* 1: the caller vouches that no kernel still running
                                    when a run starts in its stream (the one launched
                                    just before it, and any earlier one that kernel
                                    overlaps through a programmatic launch) writes
                                    seq_lens, q_indptr or block_table (true of every
                                    layer of a decode step that fills them once per
                                    step); the attention kernel then reads them while
                                    that kernel drains.  0: it waits first (safe). */
    int32_t test_stall;          /* testing only (needs kernel_variant TCGEN05): 1 makes
                                    the K producer issue nothing, so its consumers'
                                    bounded waits run out after about a second; the
                                    call then sets SPEC_ATTN_DEV_WAIT_TIMEOUT, frees its
                                    tensor memory and returns, leaving O undefined and
                                    the context usable.  0 in every real call. */
    int32_t early_context_kv;    /* 1 (needs early_metadata = 1): the caller also
                                    vouches that no such kernel writes a cached key
                                    below its request's ctx_r (the window's own keys
                                    may be written, e.g. by spec_attn_append_kv just
                                    before); the bf16 tensor-core kernel then starts
                                    the copies of each split's first K and V tile
                                    (when it holds context keys only, and with no
                                    sliding window or dense block operand) while that
                                    kernel drains.  Results are bit-identical either
                                    way.  0: it waits first (safe). */
} spec_attn_problem;

/*
 * W-invariant mode (w_invariant = 1).  Every output row comes out bit-identical
 * to the same row computed alone: window row i of request r equals the W = 1
 * call on the same cache with seq_len = ctx_r + i + 1, whatever W, P or the
 * other rows are -- the exactness rule of the page "perf(dflash): widen the
 * verify window past the compact graph's four-row limit" (section
 * "Exactness"), which greedy speculative decoding needs for its output to
 * match plain decoding.  The plan then uses split boundaries that depend only
 * on key positions (every fixed_keys_per_split keys), always writes split
 * partials and always merges them in a fold order fixed by the split index
 * alone (split s in group s mod G, G a constant of head_dim).  It
 * needs the tensor-core kernel (E_UNSUPPORTED if the CUDA-core one is
 * forced) and ignores force_splits.  Rows computed in W-invariant mode match
 * rows computed in W-invariant mode with the same fixed_keys_per_split; the
 * default mode's splits are chosen for speed and may round differently.  The
 * cost is the split count this fixes: one CTA per (split, KV head, request),
 * so the call is fastest when fixed_keys_per_split is near the typical
 * context length x P x Hkv / (number of SMs), e.g. 512 for one request with
 * 4 KV heads at 16K keys, 2048 at 64K.  The default (0) derives it from
 * max_seq_len (512 up to 16K keys, 2048 at 64K): plans that must agree
 * bitwise with each other pass the same explicit value, or have max_seq_len
 * values that round up to the same multiple of 2048 (or are both at most
 * 16384).
 */

typedef struct spec_attn_plan spec_attn_plan;   /* opaque */

/* What a plan decided; for tests, benches and logs. */
typedef struct spec_attn_plan_info {
    int32_t kernel_variant;      /* the variant that will run (never AUTO) */
    int32_t keys_per_split;      /* keys of one request one CTA sweeps (multiple of 64) */
    int32_t max_splits;          /* splits of the longest request */
    int32_t row_groups;          /* CTAs sharing one (request, KV head, split), each with
                                    its own rows; tcgen05: > 1 only above 128 query rows
                                    per KV head (groups of whole window rows) */
    int32_t grid_x, grid_y, grid_z;
    int32_t block_threads;
    int32_t smem_bytes;          /* dynamic shared memory of the split kernel */
    int32_t uses_merge;          /* 1 when a second (LSE-merge) kernel runs */
    int32_t num_sms;
    size_t workspace_bytes;
} spec_attn_plan_info;

/*
 * Validate a problem and choose the split count (keys per split) and the
 * kernel variant (the plan step of the scope table; its spec_attn_plan).
 * The split count restates the key-splitting of the page "ChunkedSmallT
 * re-streams full KV per query chunk (DFlash K>=8 verify at long context)",
 * section "Finding", without its width cap: every CTA holds all W x G rows of
 * one KV head, so widths up to 16 keep one sweep; wider ones fail here
 * rather than truncate (page "perf(dflash): widen the verify window past the
 * compact graph's four-row limit", section "What changed").  Host only; no
 * device allocation.  h_seq_lens [P] and
 * h_q_indptr [P+1] are optional host copies: when given they are checked
 * and used by the split heuristic; otherwise max_seq_len and max_w stand in
 * for every request.  A plan may be reused for every layer of a step and
 * replayed inside a CUDA graph while every device seq_len stays at or below
 * max_seq_len.  *out receives the plan; *workspace_bytes (nullable) receives
 * the bytes spec_attn_run needs.  The CUDA device current at this call is
 * the one the plan targets.
 */
int spec_attn_plan_create(const spec_attn_problem* problem, const int32_t* h_seq_lens,
                          const int32_t* h_q_indptr, spec_attn_plan** out,
                          size_t* workspace_bytes);

/* Free a plan (host memory only).  NULL is accepted. */
int spec_attn_plan_destroy(spec_attn_plan* plan);

int spec_attn_plan_get_info(const spec_attn_plan* plan, spec_attn_plan_info* info);

/*
 * Run one attention call asynchronously on `stream`: the block attention of
 * the page "DFlash2 leaves the paged graph fast path at every c>1 and
 * re-attends the whole batch context every decode step" (sections "The
 * route change" and "Scope": P x W rows over a shared paged pool through a
 * batched block table, outputs for window rows only), swept once over each
 * request's keys however wide its window (page "ChunkedSmallT re-streams full
 * KV per query chunk (DFlash K>=8 verify at long context)", section
 * "Finding"), reading only seq_len entries (page "perf(dflash): widen the
 * verify window past the compact graph's four-row limit", section "What
 * changed").
 *   q         [total_q_rows, Hq, d] bf16, 16-byte aligned
 *   k_pool, v_pool   pools as above, 16-byte aligned (NVFP4: code pools)
 *   k_scales, v_scales  NVFP4 scale pools, 16-byte aligned; NULL for bf16
 *   k_gscale, v_gscale  NVFP4 global scales; ignored for bf16
 *   block_table [P, block_table_stride] int32, seq_lens [P], q_indptr [P+1]
 *   o         [total_q_rows, Hq, d] bf16 output, 16-byte aligned
 *   lse       [total_q_rows, Hq] fp32 output, or NULL
 *   workspace caller-owned device scratch of at least the plan's
 *             workspace_bytes, 256-byte aligned; its first 256 bytes hold the
 *             sticky device-status word, which the caller zeroes once after
 *             allocating it (spec_attn_reset_device_status).  One workspace
 *             must not be shared by runs that may overlap on the GPU.
 * All device pointers must belong to the plan's device.  Returns
 * SPEC_ATTN_E_CUDA if a launch fails.
 */
int spec_attn_run(const spec_attn_plan* plan, const void* q, const void* k_pool,
                  const void* v_pool, const void* k_scales, const void* v_scales,
                  float k_gscale, float v_gscale, const int32_t* block_table,
                  const int32_t* seq_lens, const int32_t* q_indptr, void* o, float* lse,
                  void* workspace, size_t workspace_bytes, spec_attn_stream_t stream);

/*
 * spec_attn_run plus an index/mask trace: trace [total_q_rows, Hq, 2] int64
 * (zeroed by the caller) receives, for every output (row, head), the number
 * of keys the kernels let into its softmax and the sum of their physical
 * slot ids (page * page_size + slot), accumulated over all splits.  This is
 * the floating-point-free check that every row saw exactly its mask's keys
 * through the block table.  Slower than spec_attn_run; for validation.
 */
int spec_attn_run_traced(const spec_attn_plan* plan, const void* q, const void* k_pool,
                         const void* v_pool, const void* k_scales, const void* v_scales,
                         float k_gscale, float v_gscale, const int32_t* block_table,
                         const int32_t* seq_lens, const int32_t* q_indptr, void* o,
                         float* lse, int64_t* trace, void* workspace,
                         size_t workspace_bytes, spec_attn_stream_t stream);

/*
 * Dense block operand (dense_block_kv = 1).  The window's own W_r keys are
 * not in the cache: they come from dense tensors block_k, block_v
 * [total_q_rows, Hkv, head_dim] bf16 (16-byte aligned), row q_indptr[r] + i
 * holding key ctx_r + i = seq_len[r] - W_r + i.  The cache holds the context
 * keys 0 .. ctx_r - 1 only, and the block table need cover just those.  This
 * is the "Narrow" shape of the page "DFlash2 leaves the paged graph fast path
 * at every c>1 and re-attends the whole batch context every decode step"
 * (section "Scope"): the draft's block K/V are discarded after the step, so
 * they are kept apart from the paged context.  Masks, window and outputs are
 * as for spec_attn_run, over the keys 0 .. seq_len[r] - 1 so formed.  trace
 * (nullable, as spec_attn_run_traced) counts a block key with slot id
 * -(1 + its row).  A plan made with dense_block_kv = 1 runs only here, and
 * this entry point needs such a plan (else SPEC_ATTN_E_INVALID_ARG).
 */
int spec_attn_run_dense_block(const spec_attn_plan* plan, const void* q, const void* block_k,
                              const void* block_v, const void* k_pool, const void* v_pool,
                              const int32_t* block_table, const int32_t* seq_lens,
                              const int32_t* q_indptr, void* o, float* lse, int64_t* trace,
                              void* workspace, size_t workspace_bytes, spec_attn_stream_t stream);

/*
 * KV append: write the window's new key and value rows into their cache slots
 * (page "perf(dflash): widen the verify window past the compact graph's
 * four-row limit", section "What changed": the window's rows go into the
 * cache, later steps overwrite the rows a rejected tail leaves stale, and
 * attention reads only seq_len entries).  seq_len_r already counts the
 * window, so window row i of request r is written at key position
 * pos = seq_len_r - W_r + i: page block_table[r][pos / page_size], slot
 * pos % page_size, for every KV head.
 *   k_new, v_new  [total_q_rows, Hkv, d] bf16, rows in q_indptr order,
 *                 16-byte aligned; read only
 *   k_pool, v_pool, k_scales, v_scales, k_gscale, v_gscale, block_table,
 *   seq_lens, q_indptr   as for spec_attn_run; the pools (and, for NVFP4,
 *                 the scale pools) are written at the window's slots only
 *   workspace     as for spec_attn_run; spec_attn_append_kv uses only its
 *                 device-status word (workspace_bytes >= 256)
 * bf16 caches receive the bits unchanged.  NVFP4 caches receive each run of
 * 16 head_dim elements quantised against the cache's decode scale g (k_gscale
 * or v_gscale): amax = max |x|; scale byte = E4M3(amax / (6 g)); den =
 * scale * g; code = E2M1(x / den), or +0 throughout when den = 0; every
 * product and quotient in binary32 rounded to nearest even in that order, the
 * conversions to nearest even, saturating at 448 and 6 and keeping the sign.
 * Values beyond 6 * 448 * g clip.  NaN or infinite inputs give unspecified
 * codes.  Device-side checks (bad window, seq_len or page id) set the same
 * status bits as spec_attn_run and skip the row; nothing else is written.
 * Asynchronous on `stream`, allocation-free, graph capturable.
 */
int spec_attn_append_kv(const spec_attn_plan* plan, const void* k_new, const void* v_new, void* k_pool,
                        void* v_pool, void* k_scales, void* v_scales, float k_gscale, float v_gscale,
                        const int32_t* block_table, const int32_t* seq_lens, const int32_t* q_indptr,
                        void* workspace, size_t workspace_bytes, spec_attn_stream_t stream);

/*
 * spec_attn_append_kv followed by spec_attn_run on the same stream: the step
 * a verify layer takes once it has the window's K and V.  Every argument is
 * checked before either kernel is launched, so a rejected call writes
 * nothing.  The attention kernel is launched as a programmatic dependent of
 * the append and reads the cache only after the append has completed.
 * workspace as for spec_attn_run (the plan's workspace_bytes).
 */
int spec_attn_run_append(const spec_attn_plan* plan, const void* q, const void* k_new, const void* v_new,
                         void* k_pool, void* v_pool, void* k_scales, void* v_scales, float k_gscale,
                         float v_gscale, const int32_t* block_table, const int32_t* seq_lens,
                         const int32_t* q_indptr, void* o, float* lse, void* workspace, size_t workspace_bytes,
                         spec_attn_stream_t stream);

/*
 * Optional timing hooks: when set (both non-NULL; cudaEvent_t values), every
 * later run records `split_begin` on its stream just before the split-KV
 * kernel launch and `split_end` just after it, so a caller can time that
 * kernel alone with cudaEventElapsedTime.  Pass NULLs to clear.
 */
int spec_attn_plan_set_timing_events(spec_attn_plan* plan, void* split_begin, void* split_end);

/* Zero the workspace's device-status word (asynchronous on `stream`). */
int spec_attn_reset_device_status(void* workspace, spec_attn_stream_t stream);

/* Synchronise `stream`, read the device-status word into *bits (nullable)
 * and clear it.  Returns SPEC_ATTN_E_DEVICE_CHECK when any bit was set. */
int spec_attn_check_device_status(void* workspace, spec_attn_stream_t stream, uint32_t* bits);

/* Name of a status code; never NULL. */
const char* spec_attn_status_string(int status);

/* The last CUDA error code this thread saw inside the library (0 if none). */
int spec_attn_last_cuda_error(void);

/* Library version: major * 10000 + minor * 100 + patch. */
int spec_attn_version(void);

/*
 * spec_attn_run without a workspace argument, for callers that cannot
 * allocate device memory (code running where cudaMalloc is not allowed, such
 * as inside an allocator hook or a host callback, or a plugin handed only its
 * input and output buffers).  No counterpart on the pages this library
 * restates: it is a convenience of this library.
 *
 * Scratch comes from one array of SPEC_ATTN_NOALLOC_SCRATCH_BYTES (32 MiB) in
 * the library's own device memory; every GPU that loads the library holds it
 * until the process exits.  A plan whose workspace_bytes exceeds that size is
 * rejected with SPEC_ATTN_E_WORKSPACE_TOO_SMALL.  Every call on a device
 * shares the array, so calls that may overlap on the GPU race and must be
 * serialised by the caller; each call clears the device-status word at the
 * head of the array once its host checks have passed (a rejected call writes
 * nothing), and spec_attn_noalloc_check_device_status reads what the last
 * call left.  The first call on each device looks up the array's device
 * address (with that device current) and caches it with the id of the
 * context it belongs to; make that first call before any stream capture.  A
 * call made in another context of the device (after cudaDeviceReset, which
 * creates the primary context anew) looks the address up again, so make the
 * first call after a reset outside stream capture too.  Allocates nothing;
 * other arguments and errors as spec_attn_run.
 */
#define SPEC_ATTN_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
int spec_attn_run_noalloc(const spec_attn_plan* plan, const void* q, const void* k_pool,
                          const void* v_pool, const void* k_scales, const void* v_scales,
                          float k_gscale, float v_gscale, const int32_t* block_table,
                          const int32_t* seq_lens, const int32_t* q_indptr, void* o, float* lse,
                          spec_attn_stream_t stream);

/*
 * Device-status bits of the last spec_attn_run_noalloc call on the current
 * device (read and cleared, synchronising `stream` like
 * spec_attn_check_device_status); 0 in *bits, and SPEC_ATTN_OK, before any
 * such call.  Returns SPEC_ATTN_E_DEVICE_CHECK when a bit is set.  Also no
 * counterpart on the pages: it completes the no-alloc entry point.
 */
int spec_attn_noalloc_check_device_status(spec_attn_stream_t stream, uint32_t* bits);

/*
 * Step tables.  spec_attn_build_tables makes, on the GPU and from the
 * requests' lengths alone, everything the other entry points take: seq_lens,
 * q_indptr, the grown block table, and each row's position and cache slot.  A
 * verify step's accepted lengths are known on the GPU only; with this call no
 * step needs them on the host.
 *
 * Request r has prev_seq_lens[r] keys' worth of pages in its block-table row,
 * held_r = ceil(prev_seq_lens[r] / page_size), of which ctx_lens[r] keys are
 * kept (ctx_lens[r] <= prev_seq_lens[r]: a rejected tail is dropped), and
 * brings window_lens[r] new rows:
 *   seq_lens[r] = ctx_lens[r] + window_lens[r],  need_r = ceil(seq_lens[r] / page_size)
 *   q_indptr    = exclusive sum of window_lens, q_indptr[P] the total
 *   row i of request r (row q_indptr[r] + i): position ctx_lens[r] + i and
 *   slot = page * page_size + position % page_size, page its table entry.
 * A request with ctx 0 and window 0 ends (its pages go back); one with
 * prev_seq_lens 0 joins.  Rows from q_indptr[P] to max_rows (a padded batch)
 * get position 0 and slot -1, which spec_attn_norm_rope_append skips.
 *
 * Pages.  free_pages[0 .. free_count) is a stack of free page ids.  Pages past
 * need_r go back on top of it, in request and then table order; requests that
 * grow then take from its top, in the same order, into their table entries
 * held_r .. need_r - 1.  Other table entries, and stack entries outside the
 * new part, are left as they were, so a call repeated on the same
 * inputs writes the same values.  A page belongs to one request or to the
 * stack, never to two (pages shared between requests are not counted).
 *
 * seq_lens may be prev_seq_lens or ctx_lens, and free_count may be
 * prev_free_count (the state of a decode loop updated in place: captured once
 * and replayed every step); no other buffer may overlap another.
 *
 * Device-side checks: a window below 0 or above max_w, more than max_rows rows
 * in all (SPEC_ATTN_DEV_BAD_WINDOW); a length below 0, above max_seq_len or the
 * table row's capacity, or ctx above prev (SPEC_ATTN_DEV_BAD_SEQ_LEN); free and
 * held pages that exceed the pool (SPEC_ATTN_DEV_BAD_FREE_LIST); too few free
 * pages (SPEC_ATTN_DEV_OUT_OF_PAGES).  After any of them the step is empty:
 * q_indptr is all zero, every slot -1, every position 0, seq_lens and
 * free_count equal their previous values (prev_seq_lens and prev_free_count),
 * table and stack are untouched, so later calls of the step do nothing and the
 * caller may try again (where seq_lens is ctx_lens, with ctx_lens set anew: it
 * holds prev_seq_lens now).  A page id
 * outside [0, num_pages) sets SPEC_ATTN_DEV_BAD_PAGE and gives its rows slot -1.
 *
 * workspace: 256 bytes, 256-byte aligned, zeroed once (spec_attn_reset_device_
 * status); it may be a spec_attn_run workspace used on the same stream.  Calls
 * that may overlap on the GPU need workspaces of their own.  Asynchronous on
 * `stream`, one kernel, allocation-free, graph capturable.
 */
#define SPEC_ATTN_TABLES_MAX_REQS 16384
typedef struct spec_attn_tables_problem {
    int32_t num_reqs;            /* P: 0 .. SPEC_ATTN_TABLES_MAX_REQS */
    int32_t max_rows;            /* entries of positions and slot_map */
    int32_t page_size;           /* 16, 32 or 64 */
    int32_t num_pages;           /* pages of the pool and entries of free_pages */
    int32_t block_table_stride;  /* entries per block-table row */
    int32_t max_w;               /* upper bound on every window, >= 1 (prompts may be long) */
    int64_t max_seq_len;         /* upper bound on every seq_len, at most 2^31 - 1 */
} spec_attn_tables_problem;

int spec_attn_build_tables(const spec_attn_tables_problem* problem, const int32_t* ctx_lens,
                           const int32_t* window_lens, const int32_t* prev_seq_lens,
                           const int32_t* prev_free_count, int32_t* free_pages, int32_t* block_table,
                           int32_t* seq_lens, int32_t* q_indptr, int32_t* free_count, int32_t* positions,
                           int64_t* slot_map, void* workspace, size_t workspace_bytes,
                           spec_attn_stream_t stream);

/*
 * Norm and rotation of q and k in one pass.  For each row and head with
 * elements x_0 .. x_{d-1} (bf16, arithmetic in fp32):
 *   y_e = x_e * w_e / sqrt(mean_e x_e^2 + eps)     (without weights: y = x)
 *   (a, b) -> (a cos t - b sin t, a sin t + b cos t)   for each rotated pair,
 *   t = positions[axis_j][row] * inv_freq_j,  cos and sin times rot_scale,
 * written as bf16, rounded once.  Pair j < rot_dim / 2 is elements
 * (j, j + rot_dim / 2), or (2 j, 2 j + 1) with interleaved = 1; elements from
 * rot_dim on are not rotated.  Positions with several axes (time, height and
 * width of an image or a video) give each pair the axis h_pair_axis names.
 * The angle is reduced exactly: t in turns is a 64-bit fraction times the
 * position, modulo one turn, so far positions lose nothing (the fp32 product
 * would be off by up to 2^-24 of the whole angle).
 *
 * The plan holds the frequencies; it is a host object, reusable for any rows
 * and layers.  The device current at its creation is the one it targets.
 */
typedef struct spec_attn_norm_rope_problem {
    int32_t num_q_heads;         /* Hq >= 0 */
    int32_t num_kv_heads;        /* Hkv >= 0; Hq + Hkv >= 1, each at most 4096 */
    int32_t head_dim;            /* 64, 128 or 256 */
    int32_t rot_dim;             /* rotated elements: 0 .. head_dim, a multiple of 16 */
    int32_t interleaved;         /* pairs (2 j, 2 j + 1) instead of (j, j + rot_dim / 2) */
    int32_t num_axes;            /* position axes, 1 .. 4 */
    float eps;                   /* of the norm, >= 0 */
    float rot_scale;             /* factor of cos and sin; 0 selects 1 */
    int64_t q_row_stride;        /* elements from a row of q (k, v) to the next; 0 = dense; else a */
    int64_t k_row_stride;        /* multiple of 8 and at least the dense row (the heads of a row */
    int64_t v_row_stride;        /* are adjacent), e.g. views of one fused projection's output */
    int64_t q_out_row_stride;    /* likewise for the outputs */
    int64_t k_out_row_stride;
    int32_t kv_dtype;            /* spec_attn_norm_rope_append only: spec_attn_kv_dtype, */
    int32_t page_size;           /* 16, 32 or 64 (0: the plan has no cache), */
    int32_t num_pages;           /* pages of each pool, */
    int32_t reserved;            /* 0 */
    int64_t kv_page_stride;      /* and page strides in bytes, as spec_attn_problem */
    int64_t scale_page_stride;
} spec_attn_norm_rope_problem;

typedef struct spec_attn_norm_rope_plan spec_attn_norm_rope_plan;   /* opaque */

/* h_inv_freq [rot_dim / 2]: radians per position, finite and >= 0, below 2^20;
 * h_pair_axis [rot_dim / 2]: axis of each pair, below num_axes (NULL: axis 0).
 * Host only; both are copied. */
int spec_attn_norm_rope_plan_create(const spec_attn_norm_rope_problem* problem, const double* h_inv_freq,
                                    const uint8_t* h_pair_axis, spec_attn_norm_rope_plan** out);
int spec_attn_norm_rope_plan_destroy(spec_attn_norm_rope_plan* plan);

/*
 * q [num_rows, Hq, d], k [num_rows, Hkv, d] -> q_out, k_out of the same shapes,
 * rows at the plan's strides, all 16-byte aligned.  q_weight, k_weight [d] fp32
 * or NULL (no norm of q, of k); positions [num_axes, num_rows] int32 (any
 * value).  q_out may be q, and k_out k, at equal strides; otherwise an output
 * shares no byte with an input or another output (SPEC_ATTN_E_INVALID_ARG; rows
 * that lie between each other, as views of one fused projection do, are
 * apart).  Asynchronous on `stream`, allocation-free, graph capturable.
 */
int spec_attn_norm_rope(const spec_attn_norm_rope_plan* plan, int32_t num_rows, const void* q, const void* k,
                        const float* q_weight, const float* k_weight, const int32_t* positions, void* q_out,
                        void* k_out, spec_attn_stream_t stream);

/*
 * The same pass with K and V going straight into the paged cache: row i's key
 * heads (normalised, rotated, rounded to bf16) and value heads (v [num_rows,
 * Hkv, d], unchanged) are written at slot slot_map[i] = page * page_size + slot
 * within the page -- any number of rows, windows and prompts alike.  The cache
 * bytes equal spec_attn_norm_rope followed by spec_attn_append_kv (NVFP4
 * caches are quantised by the same rule from the bf16 values).  A row whose
 * slot is negative is skipped whole: neither q_out nor the cache is written
 * for it.  A slot at or past num_pages * page_size sets
 * SPEC_ATTN_DEV_BAD_PAGE and skips the row.  Rows must have distinct slots.
 * Pools, scales and decode scales as spec_attn_append_kv; workspace: 256 bytes
 * holding the device-status word.  q_out may be q at equal strides; otherwise
 * q_out, pools, scales and workspace share no byte with an input or with each
 * other (SPEC_ATTN_E_INVALID_ARG; pages of K and V may alternate in one
 * allocation).
 */
int spec_attn_norm_rope_append(const spec_attn_norm_rope_plan* plan, int32_t num_rows, const void* q,
                               const void* k, const void* v, const float* q_weight, const float* k_weight,
                               const int32_t* positions, const int64_t* slot_map, void* q_out, void* k_pool,
                               void* v_pool, void* k_scales, void* v_scales, float k_gscale, float v_gscale,
                               void* workspace, size_t workspace_bytes, spec_attn_stream_t stream);

/*
 * Cross attention: query rows of any number (a verify window, one token, a
 * whole prompt) attend to an encoder's states of another length.  Request r's
 * rows q_indptr[r] .. q_indptr[r+1]-1 see the kv_len[r] state rows from
 * kv_start[r] on, all of them:
 *   s_j = sm_scale * <q, k_j>,  O = sum_j softmax(s)_j v_j,  LSE natural log
 * with fp32 accumulation, O bf16, LSE fp32.  kv_len[r] = 0 gives O = 0 and
 * LSE = -infinity.  Scores of -infinity weigh nothing; a row of nothing else, or
 * with a score of +infinity, has O = NaN and LSE = -infinity or +infinity; a NaN
 * score makes both NaN.  K and V are dense rows [total_kv_rows, Hkv, head_dim] bf16
 * (not the paged cache: an encoder's states are written once and do not
 * grow), kv_row_stride elements apart, so that a fused projection's [rows, 2,
 * Hkv, head_dim] is taken as it is; packed states, a padded batch and states
 * shared by several requests are all ranges of rows.  Rows outside every range
 * may hold anything.
 *
 * Device-side checks: a window below 0 or above max_q_rows, or rows past
 * total_q_rows (SPEC_ATTN_DEV_BAD_WINDOW); a range not inside the state rows, or
 * longer than max_kv_len (SPEC_ATTN_DEV_BAD_SEQ_LEN): such a request is skipped,
 * its rows left as they were, like rows of no request.
 */
typedef struct spec_attn_cross_problem {
    int32_t num_reqs;            /* P, 0 .. 65535 */
    int32_t total_q_rows;        /* rows of Q and O, at most 2^30 */
    int32_t max_q_rows;          /* upper bound on a request's rows, >= 1 */
    int32_t num_q_heads;         /* Hq */
    int32_t num_kv_heads;        /* Hkv; Hq % Hkv == 0, Hq / Hkv <= 16 */
    int32_t head_dim;            /* 64, 128 or 256 */
    int32_t total_kv_rows;       /* rows of K and V, at most 2^30 */
    int32_t max_kv_len;          /* upper bound on every kv_len */
    float sm_scale;              /* 0 selects 1/sqrt(head_dim) */
    int32_t force_splits;        /* 0: the library's choice; 1 .. 8: cut the longest range n ways */
    int64_t kv_row_stride;       /* elements; 0 = dense; else a multiple of 8, at least the dense row */
} spec_attn_cross_problem;

typedef struct spec_attn_cross_plan spec_attn_cross_plan;   /* opaque */

/* Host only; the current device is the one the plan targets.
 * *workspace_bytes (nullable) receives what spec_attn_run_cross needs. */
int spec_attn_cross_plan_create(const spec_attn_cross_problem* problem, spec_attn_cross_plan** out,
                                size_t* workspace_bytes);
int spec_attn_cross_plan_destroy(spec_attn_cross_plan* plan);

/*
 * q [total_q_rows, Hq, d], o likewise, k and v at the plan's row stride, all
 * bf16 and 16-byte aligned; q_indptr [P+1], kv_start [P], kv_len [P] int32;
 * lse [total_q_rows, Hq] fp32 or NULL; workspace: 256 bytes, 256-byte aligned,
 * holding the device-status word (zeroed once).  o, lse and workspace share no
 * byte with an input or with each other (SPEC_ATTN_E_INVALID_ARG).
 * Asynchronous on `stream`, allocation-free, graph capturable.
 */
int spec_attn_run_cross(const spec_attn_cross_plan* plan, const void* q, const void* k, const void* v,
                        const int32_t* q_indptr, const int32_t* kv_start, const int32_t* kv_len, void* o,
                        float* lse, void* workspace, size_t workspace_bytes, spec_attn_stream_t stream);

/*
 * Attention of windows of any width over the paged cache under wider masks than
 * spec_attn_run's: drafted trees, where each row sees its ancestors among the
 * window's keys, and a sliding window whose first keys stay visible (sinks), for
 * chains (one token, a verify window, a chunk of a prompt) and trees alike.  The
 * pages of spec_attn_run restate one drafted chain a request; these are the same
 * step with more of it kept.
 *
 * As for spec_attn_run, request r's W_r = q_indptr[r+1] - q_indptr[r] rows are its
 * last W_r keys, already in the cache, and ctx_r = seq_len[r] - W_r.  Row i has
 * position pos_i: ctx_r + i for a chain (tree = 0); for a tree (tree = 1) the
 * greater of ctx_r and positions[row], read only with window_left > 0.  It sees
 *   context keys j < ctx_r:   all; with window_left = n > 0 those with
 *                             j > pos_i - n or j < sink_keys
 *   the window's key ctx_r + j, chain:  j <= i (and in the window or a sink, as above)
 *                               tree:   bit j of the row's mask, alone
 * row_mask [total_q_rows, mask_row_words] int32: bit j of a row is bit j mod 32 of
 * its word j / 32; bits from W_r on are ignored.  spec_attn_build_tree makes masks and
 * positions from parent pointers.  A row that sees nothing has O = 0 and LSE =
 * -infinity, like one whose scores are all -infinity.  A score of +infinity makes
 * O = NaN and LSE = +infinity, a NaN score both NaN.
 *
 * With a window, the keys from sink_keys to max(0, ctx_r - n + 1) are seen by no
 * row: pages that hold only such keys are not read and their table entries may be
 * anything, so a streaming cache may free them.  K and V of keys that no row of the
 * request sees by these bounds, and of slots past seq_len, may be anything; V of the
 * keys within them has to be finite (a row's weight 0 does not take out an infinity
 * or a NaN that other rows see), K may be anything where a row does not see it.
 *
 * Pools, scales, lengths, tables, layouts and device checks are as for
 * spec_attn_run; a request that fails a check is skipped, its rows left as they were,
 * like rows of no request.
 */
typedef struct spec_attn_masked_problem {
    int32_t num_reqs;            /* P, 0 .. 65535 */
    int32_t total_q_rows;        /* rows of Q and O, at most 2^30 */
    int32_t max_w;               /* upper bound on a request's rows, >= 1 */
    int32_t num_q_heads;         /* Hq */
    int32_t num_kv_heads;        /* Hkv, at most 65535; Hq % Hkv == 0, Hq / Hkv <= 16 */
    int32_t head_dim;            /* 64, 128 or 256 */
    int32_t page_size;           /* 16, 32 or 64 */
    int32_t num_pages;           /* pages in each pool; >= 1 when num_reqs > 0 */
    int32_t block_table_stride;  /* entries per block-table row, stride x page_size <= 2^31 - 1 */
    int32_t kv_dtype;            /* spec_attn_kv_dtype */
    float sm_scale;              /* 0 selects 1/sqrt(head_dim) */
    int32_t tree;                /* 1: the window's keys by row_mask; 0: a chain */
    int32_t window_left;         /* sliding window in keys, the row's own among them; 0: none */
    int32_t sink_keys;           /* first keys that stay visible behind the window, >= 0 */
    int32_t mask_row_words;      /* words from a row of row_mask to the next; 0: ceil(max_w / 32) */
    int32_t force_splits;        /* 0: the library's choice; n > 0: cut the longest span n ways */
    int64_t max_seq_len;         /* upper bound on every seq_len, at most 2^31 - 1 */
    int64_t kv_page_stride;      /* page strides in bytes, as spec_attn_problem */
    int64_t scale_page_stride;
} spec_attn_masked_problem;

typedef struct spec_attn_masked_plan spec_attn_masked_plan;   /* opaque */

/* Host only, some 5 to 12 us (it asks the driver how many clusters of a size fit the GPU);
 * the current device is the one the plan targets.
 * *workspace_bytes (nullable) receives what spec_attn_run_masked needs. */
int spec_attn_masked_plan_create(const spec_attn_masked_problem* problem, spec_attn_masked_plan** out,
                                 size_t* workspace_bytes);
int spec_attn_masked_plan_destroy(spec_attn_masked_plan* plan);

/* What a plan decided; for tests, benches and logs. */
typedef struct spec_attn_masked_plan_info {
    int32_t query_tiles;         /* query tiles of 128 (row, head) pairs of a CTA: 1, or 2 that share its K and V tiles */
    int32_t key_streams;         /* softmax groups that take a query tile's key tiles in turn: 1 or 2 */
    int32_t ctas_per_sm;         /* 1 or 2 */
    int32_t tiles_per_split;     /* tiles of 64 keys */
    int32_t max_splits;          /* splits of the longest span */
    int32_t join;                /* how splits are joined: 0 (one split), 1 (in a cluster), 2 (by a second kernel) */
    int32_t longest_first;       /* 1: the requests with the most keys go first */
    int32_t grid_x, grid_y, grid_z;
    int32_t block_threads;
    int32_t smem_bytes;          /* dynamic shared memory of the attention kernel */
    int32_t num_sms;
    size_t workspace_bytes;
} spec_attn_masked_plan_info;

int spec_attn_masked_plan_get_info(const spec_attn_masked_plan* plan, spec_attn_masked_plan_info* info);

/* Testing only: with stall = 1 the plan's calls copy no K, so that the bounded waits behind
 * it run out after about a second; a call then sets SPEC_ATTN_DEV_WAIT_TIMEOUT, frees its
 * tensor memory and returns, leaving O undefined and the context usable.  0: as ever. */
int spec_attn_masked_plan_set_test_stall(spec_attn_masked_plan* plan, int stall);

/*
 * Arguments as spec_attn_run, the NVFP4 global scales positive and finite, and so in
 * fp32 sm_scale x log2(e) (x k_gscale); row_mask
 * for trees only (ignored for chains), positions [total_q_rows] int32 for trees with
 * a window only (ignored otherwise).  lse may be NULL.  o, lse and workspace share no
 * byte with an input or with each other (SPEC_ATTN_E_INVALID_ARG).  Up to 8 splits need
 * 256 bytes of workspace, the device-status word; more leave partial rows in it, and
 * runs that may overlap on the GPU then need workspaces of their own.  Asynchronous on
 * `stream`, allocation-free, graph capturable.
 *
 * What is held in 16 bits, beside O itself:
 *   weights: bf16 in O's sum, unrounded in its divisor and in LSE.  NVFP4 caches: fp16
 *     of the weight relative to a running reference that is at most a factor 256 below
 *     the largest weight so far; what is below 2^-25 of it counts in the divisor but not
 *     in O, which moves O by up to 2^-25 sum_j |v_j| of a split's keys.
 *   q over NVFP4 caches: fp16; elements beyond +-65504 count as that, those below 2^-14
 *     are rounded to multiples of 2^-24 (below 2^-25: to 0).
 *   partial rows of more than 8 splits: fp16 of the row's largest element (or of 2^-126,
 *     if that is larger), 2^-12 of which each split may be off; up to 8 splits keep fp32.
 *     The number of splits is the plan's choice, or force_splits.
 */
int spec_attn_run_masked(const spec_attn_masked_plan* plan, const void* q, const void* k_pool, const void* v_pool,
                         const void* k_scales, const void* v_scales, float k_gscale, float v_gscale,
                         const int32_t* block_table, const int32_t* seq_lens, const int32_t* q_indptr,
                         const int32_t* row_mask, const int32_t* positions, void* o, float* lse, void* workspace,
                         size_t workspace_bytes, spec_attn_stream_t stream);

/*
 * Drafted trees.  A request's window is a tree of W_r nodes in an order that puts
 * parents before children: parents[row] is the parent's place in the window, or -1
 * for a root.  Node 0 is the seed token, the last one already accepted.  A parent
 * below -1 or not before its child sets SPEC_ATTN_DEV_BAD_TREE and counts as -1.
 *
 * spec_attn_build_tree writes, for the rows of every request,
 *   positions[row] = ctx_r + depth (a root's depth is 0), and
 *   row_mask[row]: the node and its ancestors -- with window_left = n > 0 only those
 *   fewer than n levels above the node, or at a position below sink_keys --
 * in mask_row_words words a row (0: ceil(max_w / 32)), unused bits 0.  The rows from
 * q_indptr[P] on get position 0 and an empty mask, unless the last window is below 0.
 * ctx_r = seq_lens[r] - W_r.
 *
 * spec_attn_accept_tree walks each tree from node 0: the next node is the lowest
 * child whose draft token is the target token of its parent (the token that the
 * model takes after that node).
 *   path [P, path_stride]: the nodes, node 0 first, -1 behind the last
 *   accept_lens[r]: their number, at most path_stride (0 for a request without rows)
 *   next_tokens[r]: the target token of the last (-1 without rows)
 *   ctx_lens[r] = ctx_r + accept_lens[r], the ctx_lens of the next step's
 *                 spec_attn_build_tables (whose prev_seq_lens are these seq_lens)
 * draft_tokens [total_rows], target_tokens [total_rows] and next_tokens [P] int64.
 * ctx_lens may be seq_lens, for a caller that keeps those lengths elsewhere: what
 * comes next takes them as they were, window included -- spec_attn_move_kv as its
 * seq_lens, the next step's spec_attn_build_tables as its prev_seq_lens.
 *
 * A window below 0, above max_w or past total_rows sets SPEC_ATTN_DEV_BAD_WINDOW, a
 * seq_len below its window SPEC_ATTN_DEV_BAD_SEQ_LEN; such a request's rows are left
 * as they were, its path is empty, accept_lens 0, next_tokens -1 and ctx_lens its
 * seq_len.  Outputs share no byte with an input (ctx_lens apart) or with each other
 * (SPEC_ATTN_E_INVALID_ARG).  workspace: 256 bytes holding the device-status word.
 * Asynchronous on `stream`, one kernel, allocation-free, graph capturable.
 */
#define SPEC_ATTN_TREE_MAX_W 1024
#define SPEC_ATTN_DEV_BAD_TREE      0x40u /* a parent that is no earlier node; a path that does not ascend */
typedef struct spec_attn_tree_problem {
    int32_t num_reqs;            /* P, 0 .. 65535 */
    int32_t total_rows;          /* entries of parents (a padded batch may have more than q_indptr[P]) */
    int32_t max_w;               /* upper bound on a tree's nodes, 1 .. SPEC_ATTN_TREE_MAX_W */
    int32_t mask_row_words;      /* spec_attn_build_tree: at least ceil(max_w / 32), or 0 */
    int32_t window_left;         /* spec_attn_build_tree, >= 0 */
    int32_t sink_keys;           /* spec_attn_build_tree, >= 0 */
    int32_t path_stride;         /* spec_attn_accept_tree: entries of a row of path, >= 1 */
    int32_t reserved;            /* 0 */
} spec_attn_tree_problem;

int spec_attn_build_tree(const spec_attn_tree_problem* problem, const int32_t* parents, const int32_t* seq_lens,
                         const int32_t* q_indptr, int32_t* positions, int32_t* row_mask, void* workspace,
                         size_t workspace_bytes, spec_attn_stream_t stream);
int spec_attn_accept_tree(const spec_attn_tree_problem* problem, const int32_t* parents, const int64_t* draft_tokens,
                          const int64_t* target_tokens, const int32_t* seq_lens, const int32_t* q_indptr, int32_t* path,
                          int32_t* accept_lens, int64_t* next_tokens, int32_t* ctx_lens, void* workspace,
                          size_t workspace_bytes, spec_attn_stream_t stream);

/*
 * Move the accepted nodes' keys and values together, in the caches of several
 * layers at once: for i < accept_lens[r], key ctx_r + path[r][i] of request r goes to
 * key ctx_r + i, for every KV head (NVFP4 caches: codes and scales, byte for byte).
 * Afterwards the request's first ctx_r + accept_lens[r] keys are its accepted text; a
 * chain needs no such call.  Nothing else is written.
 *
 * seq_lens are those that spec_attn_accept_tree took, window included: ctx_r =
 * seq_lens[r] - W_r.  (Not the ctx_lens that it wrote, in a buffer of their own or over
 * seq_lens: every key would be taken from and put W_r - accept_lens[r] places too low,
 * over accepted text, and unless that lies before key 0 no check can tell.)
 *
 * h_k_pools, h_v_pools, h_k_scales, h_v_scales: host arrays of num_layers device
 * pointers, read before the call returns (the scales' NULL for bf16).  All layers
 * have the same shapes, strides and block table; no pool shares a byte with another
 * (not checked between layers) or with the index arrays.
 *
 * Device checks: those of spec_attn_append_kv; a path of request r that does not
 * ascend from 0 or more within the window, or an accept_lens[r] below 0 or above
 * path_stride or W_r, sets SPEC_ATTN_DEV_BAD_TREE.  Such a request is skipped whole; a
 * bad page skips its keys' moves.
 */
typedef struct spec_attn_move_problem {
    int32_t num_reqs;            /* P, 0 .. 65535 */
    int32_t num_layers;          /* >= 0 */
    int32_t num_kv_heads;        /* Hkv, 1 .. 65535 */
    int32_t head_dim;            /* 64, 128 or 256 */
    int32_t page_size;           /* 16, 32 or 64 */
    int32_t num_pages;           /* pages of each pool */
    int32_t block_table_stride;
    int32_t kv_dtype;            /* spec_attn_kv_dtype */
    int32_t path_stride;         /* entries of a row of path, >= 1 */
    int32_t reserved;            /* 0 */
    int64_t max_seq_len;         /* at most 2^31 - 1 */
    int64_t kv_page_stride;      /* page strides in bytes, as spec_attn_problem */
    int64_t scale_page_stride;
} spec_attn_move_problem;

int spec_attn_move_kv(const spec_attn_move_problem* problem, void* const* h_k_pools, void* const* h_v_pools,
                      void* const* h_k_scales, void* const* h_v_scales, const int32_t* block_table,
                      const int32_t* seq_lens, const int32_t* q_indptr, const int32_t* path,
                      const int32_t* accept_lens, void* workspace, size_t workspace_bytes,
                      spec_attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_ATTN_H */
