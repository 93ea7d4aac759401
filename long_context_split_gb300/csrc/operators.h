// Internal types and helpers of the operators around the attention call (cache
// rows, latent attention, verification of drafts).  Not part of the C ABI.
#pragma once

#include <atomic>

#include "internal.h"

namespace skv {

// device error site, beside those of internal.h
enum : int32_t {
    SITE_TOKEN_RANGE = 7 << 8,   // a row, position or token id outside its range
};

// Sets the calling thread's message (printf style) and returns s.
splitkv_status fail_with(splitkv_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// SMs of the current device (0: none visible).
int sm_count();

// Allows `kernel` `bytes` of dynamic shared memory on the current device; `done` is the kernel's own
// record of the devices where that has been done.
cudaError_t allow_smem(const void* kernel, size_t bytes, std::atomic<uint64_t>& done);

// Host-side checks of a problem's shape and lengths (no pointers).
splitkv_status check_problem_lengths(const splitkv_problem* prob);

// ---- cache rows (splitkv_kv_append / splitkv_kv_gather) --------------------
// One part of a token's cache entry: K or V of a GQA cache, or the latent / rotary
// columns of a latent cache.
struct CachePart {
    void* rows;            // [row][heads][width] with the strides below (elements)
    int64_t token_stride;
    int64_t head_stride;
    void* cache;           // [page][heads][page_size][row_width], this part's columns from `col`
    int32_t width;
    int32_t row_width;
    int32_t col;
    float scale;           // E4M3: value = code * scale
    float* scales;         // block scales [page][heads][page_size >> scale_shift] in its place, or null
};

struct CacheRowsArgs {
    CachePart part[2];     // part 1 has width 0 when there is none
    const int32_t* page_table;
    const int32_t* seq_lens;
    const int32_t* indptr;     // append: qo_indptr; gather: kv_indptr
    const int32_t* kv_begin;   // gather: first token per request, or null (0)
    int32_t batch;
    int32_t rows;              // rows of the call (host count)
    int32_t heads;
    int32_t page_size;
    int32_t num_pages;
    int32_t max_pages;
    int32_t scale_shift;       // log2 of the tokens of a block scale
    int32_t* err;              // may be null
};

// ---- pages and slots -------------------------------------------------------
constexpr int32_t kMaxPagesBatch = 8192;
struct PagesArgs {
    int32_t* page_table;
    const int32_t* held;
    int32_t* held_out;
    const int32_t* seq_lens;
    int32_t* free_pages;
    const int32_t* free_count;
    int32_t* free_count_out;
    const int32_t* qo_indptr;  // null without slots
    int64_t* slots;
    int32_t* err;              // may be null
    int32_t batch;
    int32_t page_size;
    int32_t max_pages;
    int32_t capacity;
    int32_t num_slots;
};

// ---- the next tokens from logits ---------------------------------------------
struct SampleArgs {
    const void* logits;
    int64_t logits_stride;
    const float* temperature;  // settings: null where they are off for every row
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* u;            // null without tokens
    int32_t* tokens;
    float* probs;              // may be null
    int64_t probs_stride;
    int32_t* err;              // may be null
    int32_t rows;
    int32_t vocab;
};

// ---- verification of drafted tokens -----------------------------------------
struct VerifyArgs {
    const int32_t* tokens;
    const int32_t* qo_indptr;
    const float* target;
    const float* draft;        // null: each draft was proposed with certainty
    int64_t target_stride;
    int64_t draft_stride;
    const float* accept_u;
    const float* sample_u;
    const int32_t* seq_lens;   // null with seq_lens_out
    int32_t* seq_lens_out;
    int32_t* out_tokens;
    int32_t* accepted;
    int32_t* err;              // may be null
    int32_t batch;
    int32_t total_q;
    int32_t vocab;
};

// cache_kind / rows_f32: 0 f32, 1 bf16, 2 E4M3, 3 (gather) E4M3 with block scales; rows float32 or bf16
cudaError_t launch_kv_append(const CacheRowsArgs& a, int cache_kind, int rows_f32, cudaStream_t s);
cudaError_t launch_kv_gather(const CacheRowsArgs& a, int cache_kind, int rows_f32, cudaStream_t s);
cudaError_t launch_block_append(const CacheRowsArgs& a, int rows_f32, cudaStream_t s);   // kind 3
cudaError_t launch_assign_pages(const PagesArgs& a, cudaStream_t s);
cudaError_t launch_sample_tokens(const SampleArgs& a, int logits_bf16, cudaStream_t s);
cudaError_t launch_verify_drafts(const VerifyArgs& a, cudaStream_t s);

}  // namespace skv
