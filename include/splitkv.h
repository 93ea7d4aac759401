/*
 * splitkv.h -- C ABI of libsplitkv: split-KV decode attention with an exact
 * LSE-weighted merge of partial states, on one GB300 (sm_103a).
 *
 * The method (LiquidCP Section 2.1 and Section 3, Eq. 1; Helix Parallelism,
 * "Attention-Phase Configuration", steps 2-3): the KV history of each
 * request is cut into independent ranges ("splits"); each split yields a
 * partial attention state -- an output normalised over the split and the
 * log-sum-exp (LSE) of its scores -- and the partial states of a query row
 * are merged exactly,
 *      o = sum_r exp(lse_r) o_r / sum_r exp(lse_r),  lse = log sum_r exp(lse_r).
 * On one GPU the splits play the role of the KV-parallel ranks: they are
 * regions of the same HBM, processed by different SMs.
 *
 * Conventions shared by every entry point
 *  - Memory: pointers documented "device" must be device (or managed)
 *    memory of the current CUDA device; "host" pointers are ordinary host
 *    memory.  The caller allocates and frees every buffer; the library
 *    allocates only the host-side plan object, freed by splitkv_plan_destroy.
 *  - Streams: every call that touches the GPU is asynchronous on the given
 *    stream (0 = legacy default stream).  Argument errors are detected on the
 *    host and returned synchronously before anything is enqueued.
 *  - Device-side errors (a page id outside the pool, a bounded wait that ran
 *    out) are written to a caller-visible 32-bit error word; read it with
 *    splitkv_read_device_error after the stream has been synchronised.  The
 *    library never aborts the process and its kernels never trap or assert.
 *  - Threads: all functions are thread-safe except that one plan object must
 *    not be destroyed while another thread uses it.  splitkv_last_error_message
 *    is per thread.
 *  - Query rows: request b owns tokens qo_indptr[b] .. qo_indptr[b+1]-1 of q;
 *    its q_len = qo_indptr[b+1] - qo_indptr[b] appended tokens are the last
 *    q_len of its seq_len cached tokens, and its query row i (0-based) sees
 *    keys 0 .. seq_len - q_len + i (causal over the appended chunk; a decode
 *    row with q_len 1 sees the whole history).
 *  - GQA head map: query head h reads KV head h / (num_q_heads / num_kv_heads).
 *  - Output rows: out and lse_out hold total_q * num_q_heads rows, row
 *    x = token * num_q_heads + head, out row width head_dim_v.
 */
#ifndef SPLITKV_H
#define SPLITKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPLITKV_ABI_VERSION 1

/* a cudaStream_t, passed as an opaque handle so this header needs no CUDA headers */
typedef void *splitkv_stream;

typedef enum {
    SPLITKV_OK = 0,
    SPLITKV_ERR_INVALID_ARG = 1,   /* a pointer, size or length is invalid */
    SPLITKV_ERR_UNSUPPORTED = 2,   /* valid, but no kernel covers this shape/dtype */
    SPLITKV_ERR_WORKSPACE = 3,     /* workspace too small or misaligned */
    SPLITKV_ERR_CUDA = 4,          /* a CUDA runtime call failed */
    SPLITKV_ERR_TIMEOUT = 5,       /* (device) a bounded wait ran out */
    SPLITKV_ERR_DEVICE_CHECK = 6,  /* (device) a page id or index failed its range check */
} splitkv_status;

typedef enum { SPLITKV_GQA = 0, SPLITKV_MLA = 1 } splitkv_kind;
typedef enum { SPLITKV_F32 = 0, SPLITKV_BF16 = 1 } splitkv_dtype;

/*
 * One batch of attention over a paged KV cache (LiquidCP Section 2.1,
 * decode and mixed batches; paged KV as in SPLASH Appendix F.1).
 *
 * kind SPLITKV_GQA: q [total_q][num_q_heads][head_dim_qk]; k_cache and
 *   v_cache [num_pages][num_kv_heads][page_size][head_dim] ("HND": each
 *   (page, KV head) block of page_size x head_dim elements is contiguous);
 *   head_dim_qk == head_dim_v.
 * kind SPLITKV_MLA (absorbed MLA, SPLASH Section 2 Eq. 1 and Appendix A:
 *   one latent row of d_c + d_r = 512 + 64 per token shared by all heads):
 *   q [total_q][num_q_heads][576]; k_cache [num_pages][page_size][576];
 *   v_cache NULL -- values are the first head_dim_v = 512 columns of k_cache;
 *   num_kv_heads == 1.
 * page_table [batch][max_pages_per_req]: token j of request b is at page
 *   page_table[b][j / page_size], offset j % page_size.  Entries past a
 *   request's last page are never read.
 * dtype: storage type of q, k_cache and v_cache (SPLITKV_F32 or SPLITKV_BF16);
 *   arithmetic is float32 with float32 accumulation either way.
 * scale: multiplies q.k (e.g. 1/sqrt(head_dim)); the exported LSE is the
 *   natural log of sum exp(scale * q.k).
 * seq_lens_host / qo_indptr_host: host copies of seq_lens / qo_indptr, read
 *   by the planner (splitkv_plan) and by argument checks; the device copies
 *   are read by the kernels.  Both must hold the same values.
 */
typedef struct {
    int32_t kind;                    /* splitkv_kind */
    int32_t dtype;                   /* splitkv_dtype */
    int32_t batch;                   /* >= 1 */
    int32_t num_q_heads;
    int32_t num_kv_heads;
    int32_t head_dim_qk;
    int32_t head_dim_v;
    int32_t page_size;
    int32_t num_pages;               /* pages in the pool; page ids must be < num_pages */
    int32_t max_pages_per_req;       /* row stride of page_table */
    float scale;
    const void *q;                   /* device */
    const void *k_cache;             /* device */
    const void *v_cache;             /* device, NULL for MLA */
    const int32_t *page_table;       /* device */
    const int32_t *seq_lens;         /* device [batch], 1 <= seq_len, q_len <= seq_len */
    const int32_t *qo_indptr;        /* device [batch + 1], qo_indptr[0] == 0, non-decreasing */
    const int32_t *seq_lens_host;    /* host [batch] */
    const int32_t *qo_indptr_host;   /* host [batch + 1] */
    int32_t kv_fp8;                  /* 0: k_cache / v_cache hold `dtype` values.  1: they hold
                                        8-bit E4M3 codes (OCP FP8, the variant without
                                        infinities), the value of code c being e4m3(c) * k_scale
                                        in k_cache and e4m3(c) * v_scale in v_cache: an FP8 KV
                                        cache with one scale per tensor (SPLASH Appendix C.1).
                                        For MLA the latent rows are keys and values, so both
                                        take k_scale (v_scale is checked, not used).  Needs dtype
                                        BF16 (q and outputs).  GQA with head_dim 128 and
                                        page_size 64 or 128 runs on the GQA engine, which
                                        multiplies f16 operands, so query entries must lie
                                        within the f16 range (|q| <= 65504).  MLA of the tcgen05
                                        kernel's shape (128 heads, 576 / 512, page 64, contiguous
                                        splits) runs on that kernel over a bf16 copy of the
                                        batch's latent pages (exact), written into the workspace
                                        by a pre-pass: the workspace grows by 73,728 bytes per
                                        page of the batch.  Other shapes with head_dim_qk a
                                        multiple of 16 and head_dim_v 64, 128 or 512 run on the
                                        CUDA-core path in float32.  Other problems with
                                        kv_fp8 = 1 are UNSUPPORTED.
                                        2: E4M3 codes with a scale for each block of scale_block
                                        tokens and KV head (the fields below), GQA only; what
                                        else kv_fp8 = 1 asks for holds here too.  Requests with
                                        more than 64 query rows per KV head run on the chunk tiles
                                        where these apply otherwise (splitkv_plan_num_chunk_tasks),
                                        over a bf16 and f16 copy of their pages' codes (exact) that
                                        a pre-pass writes into the workspace: 512 bytes per cached
                                        token and KV head of theirs. */
    float k_scale;                   /* kv_fp8 1: finite, > 0 */
    float v_scale;                   /* kv_fp8 1: finite, > 0 */
    int32_t reserved0;               /* 0 */
    /* Read only when kv_fp8 is 2 (a caller without these fields passes 0 or 1).  The value of a
       code in slot s of page p and KV head h is e4m3(code) * scales[p][h][s / scale_block].
       Scales are 0 or from 2^-126 to 2^120, as splitkv_kv_append writes them; those of blocks that no
       visible token lies in may be anything.  Scores take a key's scale in float32; a weight meets its value's
       scale in float32 and is rounded to f16 relative to the largest such product of its row
       (of the keys that one warp has met), so that blocks of very different scales keep their bits.
       Scores, weights and sums of weighted values have float32's range, as over other caches: a key
       whose score is more than 87 (126 binary orders) below its row's largest may count for nothing, whatever its value's scale,
       and sums from 2^128 on are infinite.
       The NaN code of a new token's value may reach the rows of the new tokens before it. */
    const float *k_block_scales;     /* device [num_pages][num_kv_heads][page_size / scale_block] */
    const float *v_block_scales;     /* the same */
    int32_t scale_block;             /* 16, 32, 64 or 128; divides page_size */
    int32_t reserved1;               /* 0 */
} splitkv_problem;

typedef enum { SPLITKV_PLAN_UNIFORM = 0, SPLITKV_PLAN_CRITICAL_WAVE = 1 } splitkv_plan_mode;

/*
 * Planner settings.  Critical-wave model of LiquidCP Section 5.2 (Eq. 5:
 * tau(k) = max(rho, k/K); Eq. 6: c_red = delta_red + gamma * v_u * s_u;
 * c_attn = n_t + delta_attn).  A negative rho, delta_attn, delta_red or
 * gamma takes the constant calibrated on GB300 for the kernel the plan
 * targets (LiquidCP Appendix A.2 "Calibration", redone for this library's
 * kernels; LiquidCP Table 2's H100 values where no fit exists).
 */
typedef struct {
    int32_t mode;             /* splitkv_plan_mode */
    int32_t uniform_splits;   /* UNIFORM: splits per request; a history with fewer pages gets empty splits */
    int32_t min_splits;       /* CRITICAL_WAVE: lower bound per request (>= 1) */
    int32_t max_splits;       /* CRITICAL_WAVE: upper bound per request */
    int32_t num_ctas;         /* K of the model; 0 = the engine's CTA count on the current device */
    int32_t warps_per_cta;    /* reduction warps per scheduling unit in the model; 0 = the engine's own
                                 (GQA engine 7, or 4 with 16-token pages; MLA task slot 1,
                                 its merge being a separate kernel; CUDA-core path 16) */
    int32_t tile_tokens;      /* tokens per model KV tile; 0 = page_size */
    int32_t decode_qlen_max;  /* requests with q_len <= this are decode requests; 0 = 16 */
    double rho;               /* per-tile time floor; < 0: calibrated */
    double delta_attn;        /* fixed work per attention task, in tile units; < 0: calibrated */
    double delta_red;         /* fixed cost per reduction task; < 0: calibrated */
    double gamma;             /* cost per merged partial vector; < 0: calibrated */
    double adopt_margin;      /* adopt a split plan only if >= this fraction below NoSplit */
    int32_t interleave;       /* 0: split r of a request is a contiguous page range (the cut of
                                 LiquidCP Figure 8).  1: split r takes the request's pages r,
                                 r + n, r + 2n, ... (n = its split count): Helix Parallelism's
                                 staggered round-robin KV layout (Section 2.3, step 4), one page
                                 per round-robin block (16-token pages give the paper's 16-token
                                 blocks).  Split sizes are the same as with contiguous ranges.
                                 Interleaved plans run on the GQA engine (row blocks of up to 64
                                 rows: no chunk or paired tiles), on the MLA tcgen05 kernel and
                                 on the CUDA-core path. */
    int32_t partial_dtype;    /* storage type of the partial outputs o_r (splitkv_dtype):
                                 SPLITKV_F32 (default; SGLang's exchange precision) or
                                 SPLITKV_BF16 -- each o_r rounded to nearest even once, the
                                 precision vLLM and MegaDCP exchange partial states in
                                 (LiquidCP Section 7); half the partial-state bytes.  The
                                 LSE of every partial state stays float32.  Applies to the
                                 workspace of splitkv_decode and to splitkv_partial's o_part. */
    int32_t trace;            /* 1: the workspace gets a trace region and the persistent kernels
                                 record every task (see splitkv_trace_read); 0: off */
    int32_t reserved;         /* 0 */
} splitkv_plan_params;

/* Fill *p with the defaults: critical-wave mode, min 1 / max 64 splits, K =
 * engine scheduling units, the engine's reduction warps, tile = page, model
 * constants calibrated for the target kernel (negative values), margin 0.10
 * (LiquidCP Section 5.2). */
void splitkv_plan_params_default(splitkv_plan_params *p);

/* Opaque host-side plan: per-request split counts, the ordered task list and
 * the partial-state layout.  Built once per batch and reusable by every layer
 * that shares the batch's lengths (LiquidCP Section 7, planner runs once per
 * decoding step). */
typedef struct splitkv_plan_s splitkv_plan_t;

/*
 * splitkv_plan -- choose splits and build the task list (host only, no GPU
 * work; LiquidCP Section 5.2 "Plan selection" and "Task ordering", Appendix
 * A.2 "Split planning").
 *  prob:   problem; only shapes, seq_lens_host and qo_indptr_host are read.
 *  params: NULL for defaults.
 *  out:    receives a new plan; free with splitkv_plan_destroy.
 * Splits are contiguous, page-aligned ranges: with N pages and n splits,
 * split r holds floor(N/n) pages, plus one for r < N mod n (LiquidCP
 * Figure 8 cuts 176 tiles as 59/59/58).  Errors: INVALID_ARG (bad lengths,
 * shapes), UNSUPPORTED (no kernel for the shape).
 */
splitkv_status splitkv_plan(const splitkv_problem *prob, const splitkv_plan_params *params,
                            splitkv_plan_t **out);

void splitkv_plan_destroy(splitkv_plan_t *plan);

/* Plan queries (host). */
int32_t splitkv_plan_num_tasks(const splitkv_plan_t *plan);
/* Tasks that run on the tcgen05 chunk-tile kernel (up to 256 query rows each, as two
 * 128-row tiles): GQA bf16 requests with more than 128 query rows per KV head, D 64/128,
 * page 64/128, group size dividing 128, scale > 0, contiguous splits, bf16 cache; or an E4M3
 * cache with block scales, D 128, from 65 rows on.
 * Included in splitkv_plan_num_tasks.  -1 on NULL. */
int32_t splitkv_plan_num_chunk_tasks(const splitkv_plan_t *plan);
/* Tasks that run on the tcgen05 paired-tile kernel: GQA requests of the same shapes
 * with 33..128 query rows per KV head (speculative decode blocks, short appended
 * chunks).  Each of the request's (KV head, split) pairs is one block of up to 128 rows;
 * a task is two blocks, run side by side on one CTA (each in its own 128-row
 * tensor-memory tile), paired longest first.  Included in splitkv_plan_num_tasks.
 * -1 on NULL. */
int32_t splitkv_plan_num_pair_tasks(const splitkv_plan_t *plan);
/* flags[b] = 1 when request b runs on the chunk-tile kernel, 2 when on the paired-tile
 * kernel, else 0 (the decode engine or the CUDA-core path); INVALID_ARG on NULL. */
splitkv_status splitkv_plan_chunk_requests(const splitkv_plan_t *plan, int32_t *flags);
int64_t splitkv_plan_num_states(const splitkv_plan_t *plan);     /* partial states (rows of o_part) */
int32_t splitkv_plan_num_rows(const splitkv_plan_t *plan);       /* total_q * num_q_heads */
/* n_splits[b] for every request; returns INVALID_ARG on NULL. */
splitkv_status splitkv_plan_splits(const splitkv_plan_t *plan, int32_t *n_splits);
/* state_indptr[x], x = 0 .. num_rows: partial states of output row x are
 * rows state_indptr[x] .. state_indptr[x+1]-1 of o_part / lse_part, split r
 * at state_indptr[x] + r. */
splitkv_status splitkv_plan_state_indptr(const splitkv_plan_t *plan, int32_t *state_indptr);
/* key ranges [begin, end) of each split of request b (n_splits[b] pairs);
 * UNSUPPORTED for an interleaved plan, whose splits are not ranges: split r
 * holds the keys of pages r, r + n, r + 2n, ... below seq_len. */
splitkv_status splitkv_plan_split_ranges(const splitkv_plan_t *plan, int32_t b, int32_t *begin_end);
/* 1 if the plan's splits are page-interleaved (splitkv_plan_params.interleave), else 0. */
int32_t splitkv_plan_interleaved(const splitkv_plan_t *plan);
/* splitkv_dtype of the plan's partial outputs (splitkv_plan_params.partial_dtype); -1 on NULL. */
int32_t splitkv_plan_partial_dtype(const splitkv_plan_t *plan);
/* model scores: [0] NoSplit (or min-split) baseline, [1] chosen plan,
 * [2] search result, [3] reference plan (all 0 in uniform mode). */
splitkv_status splitkv_plan_scores(const splitkv_plan_t *plan, double *scores4);
/* Which kernel the plan targets: 0 CUDA-core float32 path, 1 bf16 GQA
 * tensor-core engine, 2 bf16 MLA tcgen05 path. */
int32_t splitkv_plan_kernel_path(const splitkv_plan_t *plan);

/*
 * Device workspace needed by splitkv_partial / splitkv_decode for this plan:
 * the task descriptors, request table, state_indptr, completion counters and
 * (for splitkv_decode) the float32 partial states.  Must be 256-byte aligned.
 */
size_t splitkv_workspace_bytes(const splitkv_plan_t *plan);

/*
 * splitkv_plan_upload -- copy the plan's descriptors into the workspace and
 * zero its counters (asynchronous on stream; the plan must outlive the copy).
 * Call once per plan and workspace before splitkv_partial / splitkv_decode;
 * again after any call that returned a device error.
 */
splitkv_status splitkv_plan_upload(const splitkv_plan_t *plan, void *workspace, size_t ws_bytes,
                                   splitkv_stream stream);

/*
 * splitkv_partial -- partial attention states of every split (Helix step 2:
 * attention of each query row over its local KV range, producing the
 * normalised output and the LSE; LiquidCP Section 3 "Attention Regions").
 *  o_part:   device [num_states][head_dim_v] (output): float32, 16-byte aligned,
 *            or bf16, 8-byte aligned, when the plan's partial_dtype is BF16
 *  lse_part: device float32 [num_states] (output; natural log)
 *  state layout: see splitkv_plan_state_indptr.  A split that holds no key a
 *  row may see (empty split, or entirely past the row's causal limit) writes
 *  o = 0 and lse = -inf.
 *  dev_error_word: device int32, or NULL to use the workspace's own word.
 */
splitkv_status splitkv_partial(const splitkv_problem *prob, const splitkv_plan_t *plan,
                               void *workspace, size_t ws_bytes, void *o_part, float *lse_part,
                               int32_t *dev_error_word, splitkv_stream stream);

/*
 * merge_states -- LSE-weighted merge of partial states (LiquidCP Eq. 1;
 * Helix step 3: rescale each partial by exp(lse_r - lse) and sum).
 *  o_part [num_states][head_dim] float32, lse_part [num_states] float32,
 *  state_indptr [num_rows + 1] int32: all device.
 *  out [num_rows][head_dim] of out_dtype (float32, or bf16 rounded to nearest
 *  even once at the end); lse_out [num_rows] float32 (may be NULL).
 *  Partials with lse = -inf contribute nothing; a row with none finite gets
 *  o = 0, lse = -inf.  Splits are combined in index order, so results do not
 *  depend on timing.  head_dim must be a multiple of 4 and <= 1024.
 */
splitkv_status merge_states(const float *o_part, const float *lse_part, const int32_t *state_indptr,
                            int32_t num_rows, int32_t head_dim, void *out, int32_t out_dtype,
                            float *lse_out, splitkv_stream stream);

/*
 * merge_states_typed -- merge_states over partial outputs stored as
 * o_part_dtype: SPLITKV_F32 (16-byte aligned; the same as merge_states) or
 * SPLITKV_BF16 (8-byte aligned: the bf16 partial states of a plan made with
 * partial_dtype BF16, LiquidCP Section 7).  The weights, the sum and the
 * LSE are float32 either way.  Errors as merge_states, plus INVALID_ARG for
 * another dtype or a misaligned o_part.
 */
splitkv_status merge_states_typed(const void *o_part, int32_t o_part_dtype, const float *lse_part,
                                  const int32_t *state_indptr, int32_t num_rows, int32_t head_dim, void *out,
                                  int32_t out_dtype, float *lse_out, splitkv_stream stream);

/*
 * splitkv_decode -- the fused path: one persistent kernel claims the plan's
 * tasks from a device queue in plan order, computes each split's partial
 * state into the workspace, and the last task to finish for a (request, KV
 * head, row block) merges its splits in index order and writes out/lse_out
 * (LiquidCP Section 6.2: attention tasks publish partial results, the
 * dependent reduction runs as soon as its inputs are complete).  The
 * CUDA-core path (kernel path 0) works the same way in one launch: each
 * request's last task to finish merges the request's splits.  The tcgen05 MLA
 * path (kernel path 2) runs its partial kernel, then the merge kernel.
 *  out: device [total_q][num_q_heads][head_dim_v], bf16 for bf16 problems,
 *  float32 for float32 problems.  lse_out: device float32 [total_q *
 *  num_q_heads] (may be NULL).
 * Requires splitkv_plan_upload on this workspace first.  Calls on the same
 * workspace must be stream-ordered (they share the counters).
 * When splitkv_plan_overlap_ctas(plan) > 0 the chunk tiles run on a second
 * stream of the library's own (one per device, created with its fork and join
 * events by the first such call on the device and kept until exit), forked from
 * `stream` and joined back into it: work enqueued on `stream` afterwards still
 * follows the whole call.  The same holds for splitkv_partial.
 */
splitkv_status splitkv_decode(const splitkv_problem *prob, const splitkv_plan_t *plan,
                              void *workspace, size_t ws_bytes, void *out, float *lse_out,
                              int32_t *dev_error_word, splitkv_stream stream);

/*
 * splitkv_decode_static -- splitkv_decode without a caller-provided
 * workspace, for callers that cannot allocate device memory: code that runs
 * where the GPU's memory is already fully reserved by another allocator (a
 * serving framework's caching pool, where an extra cudaMalloc fails or
 * fragments it), latency-critical loops in which cudaMalloc / cudaFree would
 * synchronise the device, and plugin or foreign-language callers that have no
 * access to the host framework's allocator.  The pages describe no such
 * variant; it exists only for these callers.
 *
 * Scratch: a fixed device array of SPLITKV_STATIC_SCRATCH_BYTES inside the
 * library (file-scope device storage).  Every GPU on which the library's
 * device code is loaded holds this array until the process exits.  The call
 * allocates nothing: no cudaMalloc, no cudaFree, no allocating library call.
 *  - Size limit: plans with splitkv_workspace_bytes(plan) above
 *    SPLITKV_STATIC_SCRATCH_BYTES are rejected with SPLITKV_ERR_WORKSPACE
 *    before anything is enqueued; use splitkv_decode with your own workspace
 *    for them.
 *  - Set-up: the first call on a device (with that device current) looks up
 *    the array's device address once.
 *  - No stream capture: every call copies the plan's descriptors from the
 *    plan's own (pageable) host memory with cudaMemcpyAsync, which a CUDA graph
 *    could not replay once the plan is gone; call it outside capture (to put a
 *    decode in a graph, use splitkv_plan_upload once and splitkv_decode).
 *  - Sharing: every call uses the same array and it keeps the last call's
 *    contents.  Each call re-uploads its plan's descriptors and zeroes the
 *    counters and error word it needs (asynchronously, on `stream`), so calls
 *    ordered on the GPU are independent; calls that overlap on the GPU (other
 *    streams, other threads) race on the array and give undefined results.
 *  - Arguments and results are those of splitkv_decode.  Every argument is
 *    checked on the host before anything is written to the array, so a call
 *    that returns an argument error has queued nothing.  With dev_error_word
 *    NULL, device errors go to the array's own error word: read it with
 *    splitkv_read_static_device_error before the next call, which clears it.
 */
#define SPLITKV_STATIC_SCRATCH_BYTES ((size_t)32 << 20)
splitkv_status splitkv_decode_static(const splitkv_problem *prob, const splitkv_plan_t *plan, void *out,
                                     float *lse_out, int32_t *dev_error_word, splitkv_stream stream);

/*
 * Read the error word of the static array used by splitkv_decode_static
 * calls made with dev_error_word NULL on the current device: synchronises
 * `stream`, then behaves as splitkv_read_device_error (status, raw word,
 * optional clear).  Allocates nothing.
 */
splitkv_status splitkv_read_static_device_error(int32_t clear, int32_t *raw, splitkv_stream stream);

/*
 * Read the device error word (dev_error_word, or the workspace's own word
 * when dev_error_word is NULL and workspace is given): synchronises the
 * stream, returns SPLITKV_OK, SPLITKV_ERR_TIMEOUT or SPLITKV_ERR_DEVICE_CHECK,
 * and stores the raw word in *raw if raw is non-NULL.  clear != 0 zeroes it.
 */
splitkv_status splitkv_read_device_error(int32_t *dev_error_word, void *workspace, int32_t clear,
                                         int32_t *raw, splitkv_stream stream);

/*
 * Rows of tokens outside the cache, as splitkv_kv_append reads and
 * splitkv_kv_gather writes them.  Strides are in elements; a row's innermost
 * elements are contiguous.
 *  GQA: k and v are [rows][num_kv_heads][head_dim].
 *  MLA: k is [rows][head_dim_v], the latent columns, and v is
 *    [rows][head_dim_qk - head_dim_v], the rotary columns; or v is NULL and k is
 *    [rows][head_dim_qk], whole cache rows.  Head strides are not used.
 * 16-byte aligned pointers (the cache's too) with strides that keep every row
 * 16-byte aligned, and widths that are multiples of 8, move in pieces of 16 or 32
 * bytes, others element by element.
 */
typedef struct {
    void *k;
    void *v;
    int64_t k_token_stride;
    int64_t k_head_stride;
    int64_t v_token_stride;
    int64_t v_head_stride;
    int32_t dtype;                   /* splitkv_dtype of k and v; need not be the cache's */
    int32_t reserved;                /* 0 */
} splitkv_kv_rows;

/*
 * splitkv_kv_append -- write the K/V rows of new tokens into the paged cache
 * that splitkv_decode reads (the appended tokens of LiquidCP Section 2.1), and
 * quantise them there when the cache is E4M3 (SPLASH Appendix C.1).
 *  prob: the same description that the attention call takes (q is not read).
 *    k_cache and v_cache are written.  Row qo_indptr[b] + i of `rows` is token
 *    seq_lens[b] - q_len + i of request b: the rows of its q_len new tokens, in
 *    the slots where the attention expects them.
 *  Entries: float32 caches take the value, bf16 caches the value rounded to
 *    nearest even, E4M3 caches the code of sat(x / k_scale) (or v_scale; MLA
 *    rows take k_scale): the quotient in float32, rounded to nearest even,
 *    magnitudes above 448 (infinities too) to 448, NaN to the NaN code.
 *  Block scales (kv_fp8 2) are written too.  A block whose first slot is among the new
 *    tokens gets the smallest power of two (from 2^-126) whose 448-fold reaches its
 *    tokens' largest finite magnitude.  A block that holds older tokens of the request
 *    keeps its scale while 448 times it reaches the new tokens' largest magnitude;
 *    otherwise it gets the power of two of those, and the older codes become those
 *    of sat(e4m3(code) * old / new).  Powers of two divide exactly, so that a code
 *    changes only where it falls below E4M3's smallest normal.  No other request may
 *    read or append to such a block's slots meanwhile (requests share whole blocks only).
 *  Positions come from the device arrays seq_lens and qo_indptr, so a captured
 *    call follows lengths updated in place; the host arrays give the number of
 *    rows and the argument checks.  Rows behind the device qo_indptr's last
 *    entry are left alone.
 *  dev_error_word: device int32 or NULL (errors are then not reported).  A row
 *    whose position or page id is out of range is not written and reports
 *    DEVICE_CHECK.  Two requests that share a page must not append to one slot.
 */
splitkv_status splitkv_kv_append(const splitkv_problem *prob, const splitkv_kv_rows *rows,
                                 int32_t *dev_error_word, splitkv_stream stream);

/*
 * splitkv_kv_gather -- read cached tokens back as rows (to hand a request to
 * another cache or another KV layout, or to compute on its cached values).
 *  kv_indptr: device [batch + 1], non-decreasing from 0; kv_begin: device
 *    [batch] or NULL (0).  Row kv_indptr[b] + i of `rows` is token
 *    kv_begin[b] + i of request b, which must lie below seq_lens[b].
 *  num_rows: rows that `rows` holds, >= kv_indptr[batch]; rows behind
 *    kv_indptr[batch] are left as they were.
 *  Values: E4M3 codes times k_scale / v_scale, or their block's scale, in float32,
 *    rounded once to the row type; other entries are converted to it.
 *  dev_error_word: as splitkv_kv_append; a refused row is written as zeros.
 */
splitkv_status splitkv_kv_gather(const splitkv_problem *prob, const int32_t *kv_indptr, const int32_t *kv_begin,
                                 int32_t num_rows, const splitkv_kv_rows *rows, int32_t *dev_error_word,
                                 splitkv_stream stream);

/*
 * Latent attention from the model's own queries (SPLASH Section 2 Eq. 1): each
 * head has 192-wide queries (128 + 64 rotary columns) and weights W_uk, W_uv
 * (128 x 512 each) that raise a latent row c of the cache to the head's key
 * (W_uk c, c's rotary columns) and value W_uv c.  Two forms of the same result:
 *  expanded -- every cached token's keys and values are computed, then
 *    attended: 2 * 512 * 256 operations per cached token and head, 640 per
 *    (query, key) pair.  For prompts and chunks of new tokens.
 *  absorbed -- W_uk is applied to the queries and W_uv to the outputs, and the
 *    latent rows themselves are attended (splitkv_partial on a
 *    576-wide problem).  For few query tokens per request.
 * The problem describes the latent cache and the batch: kind MLA, dtype BF16,
 * head_dim_qk 576, head_dim_v 512, scale > 0 (1 / sqrt(192) for these widths);
 * E4M3 caches with k_scale.
 */
typedef struct {
    const void *q;                   /* device bf16 [total_q][num_q_heads][192], heads contiguous */
    int64_t q_token_stride;          /* elements, a multiple of 8, >= num_q_heads * 192 */
    const void *w_kv_b;              /* device bf16 [num_q_heads][256][512]: per head W_uk's 128 rows, then W_uv's */
    void *out;                       /* device bf16 [total_q][num_q_heads][128] */
    float *lse_out;                  /* device float32 [total_q][num_q_heads] or NULL */
} splitkv_latent_layer;

/* Opaque host-side plan of the expanded form: its tasks, splits and workspace.  Built once per
 * batch of lengths, reusable by every layer. */
typedef struct splitkv_latent_plan_s splitkv_latent_plan_t;

/*
 * splitkv_latent_plan -- tasks of up to 256 query tokens of one (request, head).
 * A batch with fewer tasks than SMs has its histories split; the partial
 * states are merged as splitkv_decode's are.  Errors: INVALID_ARG,
 * UNSUPPORTED (float32, other widths, scale <= 0).  Free with
 * splitkv_latent_plan_destroy.
 */
splitkv_status splitkv_latent_plan(const splitkv_problem *prob, splitkv_latent_plan_t **out);
void splitkv_latent_plan_destroy(splitkv_latent_plan_t *plan);
/* Device workspace of splitkv_latent_expanded: descriptors, the batch's latent rows (1152 bytes per
 * token) and keys and values (512 bytes per token and head, 8 bytes per 64 of them) of all heads or,
 * where those exceed 8 GiB, of as many at a time as fit that, but at least two; partial states.
 * Must be 256-byte aligned. */
size_t splitkv_latent_workspace_bytes(const splitkv_latent_plan_t *plan);
int32_t splitkv_latent_plan_num_tasks(const splitkv_latent_plan_t *plan);
/* Splits of every request, n_splits[batch]; INVALID_ARG on NULL. */
splitkv_status splitkv_latent_plan_splits(const splitkv_latent_plan_t *plan, int32_t *n_splits);
/* As splitkv_plan_upload: once per plan and workspace, and after a device error. */
splitkv_status splitkv_latent_upload(const splitkv_latent_plan_t *plan, void *workspace, size_t ws_bytes,
                                     splitkv_stream stream);

/*
 * splitkv_latent_expanded -- out[token][head] of the expanded form; row i of a
 * request sees keys 0 .. seq_len - q_len + i.  prob->q is not read, and the
 * lengths are the plan's.  Keys are rounded to bf16, values and probabilities
 * to f16; scores, sums and outputs are float32 until the one rounding of the
 * result.  The values of a head over 64 tokens (64 j .. 64 j + 63 of a request)
 * are rounded times a power of two (up to 2^60) that brings the largest magnitude
 * among them to 2^14: down to 2^-28 of that one they keep 11 bits, below it
 * the error is at most 2^-39 of it.  A finite expanded value beyond 65504 (of an
 * E4M3 cache: before k_scale) reports DEVICE_CHECK.  A weight smaller than 2^-21
 * of the row's largest (both times their units' powers) enters the product with
 * an absolute error of up to 2^-32 of that one: of a million such keys together,
 * at most 2^-12.
 * Cache slots past a request's last token do not reach the result, whatever
 * they hold; a token's own NaN or infinity may reach the rows before it, where
 * the masked weight 0 meets it, as in the formula's matrix product.  Calls on
 * the same workspace must be stream-ordered.
 */
splitkv_status splitkv_latent_expanded(const splitkv_problem *prob, const splitkv_latent_plan_t *plan,
                                       const splitkv_latent_layer *layer, void *workspace, size_t ws_bytes,
                                       int32_t *dev_error_word, splitkv_stream stream);

/*
 * The two ends of the absorbed form, around splitkv_partial on the 576-wide problem.
 * splitkv_latent_absorb_query: q_abs [total_q][num_q_heads][576] =
 *   (q_nope W_uk, q_rope), the q of that problem; rounded to bf16.  Device
 *   bf16, 16-byte aligned; layer->out and lse_out are not used.
 * splitkv_latent_project: merges the 512-wide partial states of every row (as
 *   merge_states_typed does: o_part of o_part_dtype, lse_part, state_indptr) and
 *   projects them: layer->out [total_q][num_q_heads][128] = o_lat W_uv^T, and
 *   lse_out when it is given.  o_lat is float32 until it meets the weights
 *   (as two bf16 parts).  layer->q is not used.
 * total_q is prob->qo_indptr_host[batch].  dev_error_word: device int32 or NULL.
 */
splitkv_status splitkv_latent_absorb_query(const splitkv_problem *prob, const splitkv_latent_layer *layer, void *q_abs,
                                           int32_t *dev_error_word, splitkv_stream stream);
splitkv_status splitkv_latent_project(const splitkv_problem *prob, const splitkv_latent_layer *layer, const void *o_part,
                                      int32_t o_part_dtype, const float *lse_part, const int32_t *state_indptr,
                                      int32_t *dev_error_word, splitkv_stream stream);

/* 1 when the expanded form is expected to be the faster one for the problem's lengths, 0 for the
 * absorbed one, -1 when the problem is not one of latent attention (host only). */
int32_t splitkv_latent_prefers_expanded(const splitkv_problem *prob);

/*
 * Drafted tokens and the two models' probabilities (speculative decoding: the
 * step after the attention of a drafted block).  The query rows are the
 * attention call's: request b's row qo_indptr[b] fed its last accepted token,
 * the rows after it its q_len - 1 drafts, and row r of target_probs is the
 * target's distribution of the token that follows row r.  All pointers device.
 */
typedef struct {
    int32_t batch;
    int32_t total_q;                 /* rows: qo_indptr[batch] */
    int32_t vocab;
    int32_t reserved;                /* 0 */
    const int32_t *qo_indptr;        /* [batch + 1] */
    const int32_t *tokens;           /* [total_q]: the token that each row fed to the model */
    const float *target_probs;       /* [total_q][vocab], row stride target_stride */
    const float *draft_probs;        /* the same layout: row r, the distribution that the draft of row
                                        r + 1 was drawn from (a request's last row is not read); NULL:
                                        every draft was proposed with certainty */
    int64_t target_stride;           /* elements, >= vocab */
    int64_t draft_stride;
    const float *accept_u;           /* [total_q] random numbers in [0, 1): row r tests the draft of row r + 1 */
    const float *sample_u;           /* [batch] random numbers in [0, 1) for the drawn tokens */
    const int32_t *seq_lens;         /* [batch], or NULL with seq_lens_out */
    int32_t *seq_lens_out;           /* [batch] or NULL: seq_lens without the refused drafts' slots (may be
                                        seq_lens itself) */
    int32_t *out_tokens;             /* [total_q] */
    int32_t *accepted;               /* [batch] */
} splitkv_verify;

/*
 * splitkv_verify_drafts -- accept drafted tokens so that the result follows the
 * target's distribution.  Draft x at row r + 1 is accepted while
 * accept_u[r] * q_r(x) < p_r(x) (compared exactly).  accepted[b] is the number
 * of drafts before the first refusal; at that row one token is drawn from
 * max(p_r - q_r, 0) (from p_r where that is zero everywhere), after the last
 * draft, if all are accepted, from p_r: the lowest token whose cumulative
 * weight exceeds sample_u[b] times the row's total.  Tokens without weight are
 * never drawn; a row without any gives -1.  Weights that are NaN or negative count as
 * 0; probabilities must otherwise be finite.  out_tokens row r of request b: the
 * accepted drafts, then the drawn token, then -1.  seq_lens_out[b] = seq_lens[b] - (q_len - 1) + accepted[b].  A
 * request without rows gets accepted 0 and keeps its length.
 *  dev_error_word: device int32 or NULL.  A draft outside [0, vocab) is refused
 *    and reports DEVICE_CHECK, and so does a qo_indptr entry outside total_q.
 */
splitkv_status splitkv_verify_drafts(const splitkv_verify *v, int32_t *dev_error_word, splitkv_stream stream);

/*
 * The pages of a batch's requests, and where they come from.  All pointers device.
 */
typedef struct {
    int32_t batch;                   /* 1 .. 8192 */
    int32_t page_size;
    int32_t max_pages_per_req;       /* row stride of page_table */
    int32_t capacity;                /* entries of free_pages (a pool's pages all fit where it is num_pages) */
    int32_t *page_table;             /* [batch][max_pages_per_req]: entries 0 .. held[b] - 1 of row b are request b's */
    const int32_t *held;             /* [batch]: pages that each request holds */
    int32_t *held_out;               /* [batch], after the call (may be held itself) */
    const int32_t *seq_lens;         /* [batch]: tokens that each request is to have room for; 0: it has ended */
    int32_t *free_pages;             /* [capacity]: the ids of the free pages, the next one to be taken last */
    const int32_t *free_count;       /* [1]: how many there are */
    int32_t *free_count_out;         /* [1], after the call (may be free_count itself) */
    const int32_t *qo_indptr;        /* [batch + 1], or NULL without slots (not read where num_slots is 0) */
    int64_t *slots;                  /* [num_slots], or NULL: the cache slot, page * page_size + offset, of every new token:
                                        entry qo_indptr[b] + i is that of token seq_lens[b] - q_len + i */
    int32_t num_slots;               /* entries of slots; those from qo_indptr[batch] on are left as they were */
    int32_t reserved;                /* 0 */
} splitkv_pages;

/*
 * splitkv_assign_pages -- give every request the ceil(seq_lens[b] / page_size) pages
 * that its length needs, on the GPU: the page table that the other calls read, from
 * lengths alone (a captured call follows lengths updated in place).
 *  Requests that hold more (ended ones, refused drafts) give the surplus back first:
 *    page_table[b][need .. held - 1] go onto the free list, request after request, in
 *    order.  Those that hold too few then take ids from the list's end, in order.  Table
 *    entries behind a request's pages are left as they were.
 *  dev_error_word: device int32 or NULL.  A request that needs more than
 *    max_pages_per_req, or whose pages together with those of the growing requests before it exceed
 *    the free ones, gets none (it keeps what it holds) and reports DEVICE_CHECK; a
 *    negative length counts as 0 and reports it too, as do a held or free count out of
 *    range (taken as the nearest one in range) and pages given back beyond `capacity`
 *    (dropped).  Slots of tokens without a page are -1, so are all those of a request whose
 *    qo_indptr entries decrease, leave num_slots or exceed its length (reported).  A row that two
 *    requests claim (entries that decrease in between) gets the value of one of them.
 */
splitkv_status splitkv_assign_pages(const splitkv_pages *p, int32_t *dev_error_word, splitkv_stream stream);

/*
 * Logits of the next tokens and each row's settings.  All pointers device; a NULL setting is off
 * for every row.
 */
typedef struct {
    int32_t rows;
    int32_t vocab;                   /* 1 .. 2^19 */
    int32_t dtype;                   /* splitkv_dtype of logits */
    int32_t reserved;                /* 0 */
    const void *logits;              /* [rows][vocab], row stride logits_stride */
    int64_t logits_stride;           /* elements, >= vocab */
    const float *temperature;        /* [rows], >= 0; 0: the most likely token */
    const int32_t *top_k;            /* [rows]; <= 0: off */
    const float *top_p;              /* [rows]; >= 1 (and NaN): off; <= 0: the most likely token */
    const float *min_p;              /* [rows]; <= 0 (and NaN): off; above 1 counts as 1 */
    const float *sample_u;           /* [rows] random numbers in [0, 1); NULL without out_tokens */
    int32_t *out_tokens;             /* [rows] or NULL */
    float *probs;                    /* [rows][vocab] or NULL: the distributions drawn from */
    int64_t probs_stride;            /* elements, >= vocab */
} splitkv_sample;

/*
 * splitkv_sample_tokens -- draw a token from each row of logits x, and / or write the
 * distributions that splitkv_verify_drafts takes.  With m the row's largest logit and T its
 * temperature, the weight of token i is exp((x_i - m) / T).  In turn, each on what the ones before
 * have left: min_p keeps tokens of (x_i - m) / T >= log(min_p); top_k the k largest; top_p
 * the fewest of the largest whose weights reach top_p times the weight that is left.  Equal logits
 * rank in the order of their tokens.  The token drawn is the lowest whose cumulative
 * weight exceeds sample_u times the total; probs are weights over the total, 0 for tokens not kept.
 *  Logits that are NaN or -infinity have no weight; a row without any other gives token -1 and
 *    probabilities of 0.  Infinite logits share all the weight.  T = 0 is the largest logit's
 *    lowest token, whatever the other settings.
 *    Random numbers of 1 and more draw the last token with weight, negative ones and NaN the first.
 *  Weights are whole multiples of a unit (2^-44 of the power of two just above the largest), computed to
 *    2^-40 of themselves (2^-38 where |m| / T is some hundreds), so that their sums do not depend on any order;
 *    probs are float32.
 *  dev_error_word: device int32 or NULL.  A negative or NaN temperature reports
 *    DEVICE_CHECK and gives token -1 and probabilities of 0.
 */
splitkv_status splitkv_sample_tokens(const splitkv_sample *s, int32_t *dev_error_word, splitkv_stream stream);

/* Message for the last error returned on the calling thread. */
const char *splitkv_last_error_message(void);
const char *splitkv_status_string(splitkv_status s);
int32_t splitkv_abi_version(void);

/*
 * Critical-wave model entry points (host only), exposed for calibration and
 * tests.  A sequence has `tiles` KV tiles, `tasks_per_split` attention tasks
 * per split, `vectors` output vectors and `q_len` query tokens.
 */
typedef struct {
    int32_t tiles;
    int32_t tasks_per_split;
    int32_t vectors;
    int32_t q_len;
} splitkv_seq_model;

typedef struct {
    int32_t num_ctas;         /* K */
    int32_t warps_per_cta;
    int32_t q_heads;          /* h_q for the reduction run-length rule */
    int32_t decode_qlen_max;
    double rho, delta_attn, delta_red, gamma, adopt_margin;
} splitkv_model_params;

/* Simulated completion (score) and attention completion of one split plan
 * (LiquidCP Section 5.2, Eqs. 5-6). */
splitkv_status splitkv_model_simulate(const splitkv_seq_model *seqs, int32_t nseq,
                                      const int32_t *splits, const splitkv_model_params *params,
                                      double *score, double *attn_end);

/* Plan search and selection (LiquidCP Section 5.2 "Plan selection", Appendix
 * A.2); splits_out [nseq]; scores_out [4] as in splitkv_plan_scores. */
splitkv_status splitkv_model_plan(const splitkv_seq_model *seqs, int32_t nseq,
                                  const splitkv_model_params *params, int32_t min_splits,
                                  int32_t max_splits, int32_t *splits_out, double *scores_out);

/*
 * Task trace (a measurement aid; LiquidCP Section 3 and Section 7 measure
 * per-SM stage timelines and tail idle the same way).  With
 * splitkv_plan_params.trace = 1 the plan's workspace holds one record per
 * traced unit of work and every splitkv_decode / splitkv_partial launch of the
 * plan rewrites them: the claimer stamps start_ns (%globaltimer), sm (%smid)
 * and cta when it takes the unit from the device queue; end_ns is the last
 * moment a role finished its part of it (its outputs written).  Records, in
 * order:
 *   GQA plans: one per engine task (kind ATTENTION), one per reduction item of
 *   the fused engine (kind REDUCTION; start after its inputs were complete),
 *   one per chunk-tile task (kind CHUNK), one per paired-tile task (kind PAIR);
 *   MLA tcgen05 plans: one per work item, two per task (kind MLA_ITEM);
 *   CUDA-core plans: none.
 * Units a launch did not reach (an error) keep the previous launch's values.
 */
typedef struct {
    uint64_t start_ns;
    uint64_t end_ns;
    int32_t id;       /* index of the unit within its kind */
    int32_t sm;
    int32_t kind;     /* splitkv_trace_kind */
    int32_t cta;
} splitkv_trace_record;

typedef enum {
    SPLITKV_TRACE_ATTENTION = 0,
    SPLITKV_TRACE_REDUCTION = 1,
    SPLITKV_TRACE_CHUNK = 2,
    SPLITKV_TRACE_MLA_ITEM = 3,
    SPLITKV_TRACE_PAIR = 4
} splitkv_trace_kind;

/* CTAs of the chunk-tile kernel when the plan runs it beside the engine on disjoint SMs
 * (0: the two run one after the other; -1 on NULL).  Chosen by splitkv_plan for GQA plans
 * whose chunk-tile requests are all unsplit -- their tiles write final rows, so the
 * engine's reduction phase needs nothing from them -- in proportion to the two kernels'
 * work, when that is expected to save at least 5 %; the engine then gets the other SMs
 * (and the critical-wave model plans its requests over that many units). */
int32_t splitkv_plan_overlap_ctas(const splitkv_plan_t *plan);

/* Records of the plan's trace region (0 when the plan was made without trace). */
int32_t splitkv_plan_trace_records(const splitkv_plan_t *plan);

/* Copy the trace records out of `workspace` into host memory `out`
 * [splitkv_plan_trace_records(plan)]; synchronises `stream`.  Errors:
 * INVALID_ARG (NULL, plan without trace), WORKSPACE, CUDA. */
splitkv_status splitkv_trace_read(const splitkv_plan_t *plan, const void *workspace, size_t ws_bytes,
                                  splitkv_trace_record *out, splitkv_stream stream);

typedef struct {
    int32_t records;          /* records of the selected kinds */
    int32_t sms;              /* SMs counted */
    double begin_ns;          /* first start of the selected records */
    double end_ns;            /* last end: the stage's finish */
    double tail_idle_sm_ns;   /* sum over SMs of (end_ns - the SM's last end) */
    double tail_idle_frac;    /* tail_idle_sm_ns / (sms * (end_ns - begin_ns)) */
} splitkv_trace_stats;

/*
 * Tail idle of one stage (host arithmetic only; LiquidCP Section 3: an SM's
 * wait after its last task in the stage until the stage finishes; the
 * fraction is summed tail idle over total SM-time).  The stage is made of the
 * records whose kind bit is set in kind_mask (bit k = kind k).  num_sms > 0
 * counts that many SMs, those with no record of the stage idle for all of it;
 * num_sms = 0 counts the SMs that appear in the records.  Errors: INVALID_ARG
 * (NULL, no selected record, a record with end < start or an SM id outside
 * [0, num_sms)).
 */
splitkv_status splitkv_trace_tail_idle(const splitkv_trace_record *recs, int32_t n, int32_t kind_mask,
                                       int32_t num_sms, splitkv_trace_stats *out);

/*
 * Launch profiler (host).  The pages describe no such facility: it is a
 * measurement aid.  Between splitkv_profile_begin and splitkv_profile_end,
 * every kernel launch of the library is bracketed by CUDA events recorded on
 * the launching stream (a few microseconds of host time per launch).
 * splitkv_profile_end waits for the recorded events, fills out[k] for each
 * kernel k (launch count, summed device time in ms; NULL to discard) and
 * turns the profiler off.  Process-wide; safe to call from several threads.
 * Errors: CUDA when an event could not be read (that launch is skipped).
 */
typedef enum {
    SPLITKV_KERNEL_GENERIC = 0,      /* CUDA-core float32/bf16 partial attention */
    SPLITKV_KERNEL_GQA_ENGINE = 1,   /* persistent bf16 GQA engine */
    SPLITKV_KERNEL_MLA = 2,          /* tcgen05 absorbed-MLA partial attention */
    SPLITKV_KERNEL_CHUNK = 3,        /* tcgen05 GQA chunk tiles */
    SPLITKV_KERNEL_MERGE = 4,        /* merge_states */
    SPLITKV_KERNEL_CHUNK_VCONV = 5,  /* f16 copy of the chunk requests' value pages, with block scales copies of
                                        their keys' and values' codes (before the chunk tiles) */
    SPLITKV_KERNEL_PAIR = 6,         /* tcgen05 paired row blocks (33..128 rows per KV head) */
    SPLITKV_KERNEL_MLA_LATENT = 7,   /* bf16 copy of an E4M3 latent cache's pages (before the MLA kernel) */
    SPLITKV_KERNEL_KV_APPEND = 8,    /* rows into the paged cache */
    SPLITKV_KERNEL_KV_GATHER = 9,    /* cache entries back to rows */
    SPLITKV_KERNEL_VERIFY = 10,      /* verification of drafted tokens */
    SPLITKV_KERNEL_LATENT_ROWS = 11,       /* bf16 copy of the batch's latent rows */
    SPLITKV_KERNEL_LATENT_EXPAND = 12,     /* keys and values of every head */
    SPLITKV_KERNEL_LATENT_ATTENTION = 13,  /* expanded latent attention */
    SPLITKV_KERNEL_LATENT_ABSORB = 14,     /* queries times W_uk */
    SPLITKV_KERNEL_LATENT_PROJECT = 15,    /* merge of latent outputs, times W_uv^T */
    SPLITKV_KERNEL_ASSIGN_PAGES = 16,      /* page tables and slots from lengths */
    SPLITKV_KERNEL_SAMPLE = 17,            /* the next tokens from logits */
    SPLITKV_KERNEL_COUNT = 18
} splitkv_kernel;

typedef struct {
    int32_t launches;
    int32_t pad;
    double total_ms;
} splitkv_kernel_time;

splitkv_status splitkv_profile_begin(void);
splitkv_status splitkv_profile_end(splitkv_kernel_time *out /* [SPLITKV_KERNEL_COUNT] */);

/*
 * Test hook (host; no counterpart on the pages).  mode 1 makes every
 * persistent kernel launched afterwards (GQA engine, chunk tiles, MLA)
 * withhold its tasks from its own roles: nothing ever signals them, so their
 * bounded waits expire after about 2 s each, the launch records
 * SPLITKV_ERR_TIMEOUT in its device error word and returns normally (no
 * fault, the context stays usable, outputs are not written).  mode 0 (the
 * default) restores normal operation.  Process-wide.  Errors: INVALID_ARG
 * for other modes.
 */
splitkv_status splitkv_debug_set_inject(int32_t mode);

#ifdef __cplusplus
}
#endif

#endif /* SPLITKV_H */
