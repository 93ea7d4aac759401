// Types of the latent-attention operators (expanded form, query absorption,
// value projection) shared by the host entry points and the kernels.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "operators.h"

namespace skv {

constexpr int kLatNope = 128;                      // query / key columns that come from the latent
constexpr int kLatRope = 64;                       // rotary columns, shared by all heads
constexpr int kLatQ = kLatNope + kLatRope;
constexpr int kLatC = 512;                         // latent columns
constexpr int kLatRow = kLatC + kLatRope;          // cache row
constexpr int kLatV = 128;                         // value columns of a head
constexpr int kLatW = kLatNope + kLatV;            // weight rows of a head (key rows, then value rows)

// The expanded keys (bf16) and values (f16) of 64 cached tokens and one head, in the order of the
// shared-memory operands of their products, so that a warp of the expansion stores whole lines (32
// tokens x 32 bytes) and the attention copies 16 KB at a time: eight groups of 16 columns, a
// group 64 rows (tokens) of 32 bytes in the 32-byte swizzle (the two 16-byte halves of a row change
// places where bit 2 of the row is set); the keys' groups, then the values'.
constexpr int kLatUnit = 64;                       // (each request's rows are padded to whole units)
constexpr int kLatGroup = kLatUnit * 32;           // one 16-column group: 2 KB
constexpr int kLatSide = 8 * kLatGroup;            // keys (or values) of a unit: 16 KB
constexpr int kLatImage = 2 * kLatSide;

// The images of all heads take 512 bytes per token and head: 66 GB for a million tokens of 128 heads.  Heads are
// expanded and attended in equal groups whose images fit these bytes (a group has at least two heads).
constexpr size_t kLatImageBytes = (size_t)8 << 30;

// The power of two of a unit's values: f16 holds 2^-exp2 times them, with the largest finite magnitude of the
// unit's 64 x 128 values in [2^14, 2^15).  Values are only scaled up (exp2 <= 0: what f16 does not hold is
// reported) and by at most 2^60, which keeps the softmax's sum in float32.
constexpr int kLatValueTop = 14, kLatValueUp = 60;
struct LatentScale {
    float exp2;
    float back;             // 2^-exp2
};
static_assert(sizeof(LatentScale) == 8, "LatentScale layout");

struct LatentReq {
    int32_t seq_len;
    int32_t q_len;
    int32_t q_start;
    int32_t row_base;       // first of the request's rows in the copies
    int32_t n_splits;
    int32_t state_base;     // partial state of token i, head h, split r: state_base + (i * H + h) * n_splits + r
    int32_t pad[2];
};
static_assert(sizeof(LatentReq) == 32, "LatentReq layout");

// Up to 256 query tokens of one (request, head) over the keys [key_begin, key_end) of one split; with
// heads == 2, all (up to 128) query tokens of two consecutive heads.
struct LatentTask {
    int32_t b;
    int32_t head;
    int32_t row_begin;
    int32_t row_end;
    int32_t key_begin;      // a multiple of 64
    int32_t key_end;
    int32_t split;
    int32_t heads;
};
static_assert(sizeof(LatentTask) == 32, "LatentTask layout");

// 64 rows of the copies: request, first token.
struct LatentBlock {
    int32_t b;
    int32_t token;
};
static_assert(sizeof(LatentBlock) == 8, "LatentBlock layout");

struct LatentArgs {
    const void* q;             // bf16 [total_q][H][192], token stride below
    int64_t q_stride;
    const void* w;             // bf16 [H][256][512]
    const void* cache;         // latent cache, bf16 or E4M3
    const int32_t* page_table;
    const LatentReq* reqs;
    const LatentTask* tasks;
    const LatentBlock* blocks;
    void* rows;                // bf16 [padded rows][576]: the requests' latent rows
    void* kv;                  // [group's heads][padded rows / 64] images of 64 keys and values, 32 KB each
    LatentScale* v_exp;        // the same: each unit's values in `kv`
    void* out;                 // bf16 [total_q][H][128]
    float* lse_out;            // may be null
    float* o_part;             // partial states of a split batch, or null: the tasks write final rows
    float* lse_part;
    Control* ctrl;
    int32_t* err;
    int32_t total_q;
    int32_t heads;
    int32_t head0;             // the group of heads of this launch: first, how many
    int32_t group;
    int32_t num_tasks;         // of the group
    int32_t num_blocks;        // padded rows / 64
    int32_t page_size;
    int32_t num_pages;
    int32_t max_pages;
    int32_t kv_fp8;
    float scale_log2;          // scale * k_scale * log2 e
    float v_scale;             // k_scale: values are codes times it
    int32_t inject;
    int32_t pairs;             // some tasks are of two heads
};

// bf16 (exact) copy of the batch's latent rows, padding rows zero
cudaError_t launch_latent_rows(const LatentArgs& a, cudaStream_t s);
// keys and values of the group's heads from the copy
cudaError_t launch_latent_expand(const LatentArgs& a, cudaStream_t s);
cudaError_t launch_latent_attention(const LatentArgs& a, cudaStream_t s);
// q_abs [total_q][H][576] = (q_nope W_uk | q_rope); a.q, a.w
cudaError_t launch_latent_absorb(const LatentArgs& a, void* q_abs, cudaStream_t s);
// out [total_q][H][128] = (merged latent output) W_uv^T from the 512-wide partial states of row
// x = token * H + head, states indptr[x] .. indptr[x + 1]-1; a.w, a.out, a.lse_out
cudaError_t launch_latent_project(const LatentArgs& a, const void* o_part, int part_bf16, const float* lse_part,
                                  const int32_t* indptr, cudaStream_t s);

}  // namespace skv
