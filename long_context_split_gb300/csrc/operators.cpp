// C-ABI entry points of the operators around the attention call: cache rows in
// and out, and the verification of drafted tokens.  Argument checks only; the
// arithmetic runs in the CUDA kernels.
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "splitkv.h"
#include "internal.h"

using namespace skv;

namespace {

splitkv_status ok() {
    set_last_error_message("");
    return SPLITKV_OK;
}

splitkv_status cuda_fail(cudaError_t e, const char* what) {
    return fail_with(SPLITKV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Device (or managed) memory of the current device.
splitkv_status check_ptr(const void* ptr, const char* name, bool allow_null) {
    if (!ptr) {
        if (allow_null) return SPLITKV_OK;
        return fail_with(SPLITKV_ERR_INVALID_ARG, "%s is NULL", name);
    }
    cudaPointerAttributes at;
    cudaError_t e = cudaPointerGetAttributes(&at, ptr);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail_with(SPLITKV_ERR_INVALID_ARG, "%s: %s", name, cudaGetErrorString(e));
    }
    if (at.type == cudaMemoryTypeManaged) return SPLITKV_OK;
    int dev = 0;
    if (at.type != cudaMemoryTypeDevice) return fail_with(SPLITKV_ERR_INVALID_ARG, "%s is not device memory", name);
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return cuda_fail(e, "current device");
    if (at.device != dev)
        return fail_with(SPLITKV_ERR_INVALID_ARG, "%s is on device %d, the current device is %d", name, at.device, dev);
    return SPLITKV_OK;
}

// The cache side of append and gather from the problem, the rows' side from `r`.
splitkv_status cache_rows_args(const splitkv_problem* p, const splitkv_kv_rows* r, const char* call, CacheRowsArgs* a) {
    splitkv_status s = check_problem_lengths(p);
    if (s) return s;
    if (!r) return fail_with(SPLITKV_ERR_INVALID_ARG, "rows is NULL");
    if (r->dtype != SPLITKV_F32 && r->dtype != SPLITKV_BF16)
        return fail_with(SPLITKV_ERR_INVALID_ARG, "rows dtype %d is not F32 or BF16", r->dtype);
    if (r->reserved != 0) return fail_with(SPLITKV_ERR_INVALID_ARG, "rows reserved must be 0");
    if (p->kv_fp8 && p->dtype != SPLITKV_BF16)
        return fail_with(SPLITKV_ERR_UNSUPPORTED, "an E4M3 cache needs dtype BF16, as the attention call does");
    std::memset(a, 0, sizeof *a);
    const bool mla = p->kind == SPLITKV_MLA;
    const int elem = p->kv_fp8 ? 1 : p->dtype == SPLITKV_BF16 ? 2 : 4;
    a->batch = p->batch;
    a->heads = p->num_kv_heads;
    a->page_size = p->page_size;
    a->num_pages = p->num_pages;
    a->max_pages = p->max_pages_per_req;
    a->page_table = p->page_table;
    a->seq_lens = p->seq_lens;
    a->part[0].rows = r->k;
    a->part[0].token_stride = r->k_token_stride;
    a->part[0].head_stride = mla ? 0 : r->k_head_stride;
    a->part[0].cache = const_cast<void*>(p->k_cache);
    a->part[0].row_width = p->head_dim_qk;
    a->part[0].scale = p->kv_fp8 ? p->k_scale : 1.f;
    a->part[1] = a->part[0];
    a->part[1].rows = r->v;
    a->part[1].token_stride = r->v_token_stride;
    if (mla) {
        a->part[0].width = r->v ? p->head_dim_v : p->head_dim_qk;
        a->part[1].width = r->v ? p->head_dim_qk - p->head_dim_v : 0;
        a->part[1].col = p->head_dim_v;
        if (p->v_cache) return fail_with(SPLITKV_ERR_INVALID_ARG, "an MLA cache has no v_cache");
        if (r->v && a->part[1].width == 0)
            return fail_with(SPLITKV_ERR_INVALID_ARG, "%s: the cache has no rotary columns for v", call);
    } else {
        a->part[0].width = a->part[1].width = p->head_dim_qk;
        a->part[1].head_stride = r->v_head_stride;
        a->part[1].cache = const_cast<void*>(p->v_cache);
        a->part[1].scale = p->kv_fp8 ? p->v_scale : 1.f;
    }
    for (int k = 0; k < 2; ++k) {
        const CachePart& c = a->part[k];
        if (c.width == 0) continue;
        const char* name = k ? "v" : "k";
        if (c.token_stride < 0 || c.head_stride < 0)
            return fail_with(SPLITKV_ERR_INVALID_ARG, "%s strides must not be negative", name);
        if ((uintptr_t)c.rows % (r->dtype == SPLITKV_F32 ? 4 : 2) || (uintptr_t)c.cache % elem)
            return fail_with(SPLITKV_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
    }
    return SPLITKV_OK;
}

splitkv_status check_rows_ptrs(const splitkv_problem* p, const CacheRowsArgs& a, const int32_t* err) {
    splitkv_status s;
    if ((s = check_ptr(p->k_cache, "k_cache", false))) return s;
    if (p->kind == SPLITKV_GQA && (s = check_ptr(p->v_cache, "v_cache", false))) return s;
    if ((s = check_ptr(a.part[0].rows, "rows k", false))) return s;
    if (a.part[1].width > 0 && (s = check_ptr(a.part[1].rows, "rows v", false))) return s;
    if ((s = check_ptr(p->page_table, "page_table", false))) return s;
    if ((s = check_ptr(p->seq_lens, "seq_lens", false))) return s;
    return check_ptr(err, "dev_error_word", true);
}

int cache_kind(const splitkv_problem* p) { return p->kv_fp8 ? 2 : p->dtype == SPLITKV_BF16 ? 1 : 0; }

}  // namespace

extern "C" {

splitkv_status splitkv_kv_append(const splitkv_problem* prob, const splitkv_kv_rows* rows, int32_t* dev_error_word,
                                 splitkv_stream stream) {
    CacheRowsArgs a;
    splitkv_status s = cache_rows_args(prob, rows, "kv_append", &a);
    if (s) return s;
    a.rows = prob->qo_indptr_host[prob->batch];
    a.indptr = prob->qo_indptr;
    a.err = dev_error_word;
    if (a.rows == 0) return ok();
    if ((s = check_rows_ptrs(prob, a, dev_error_word))) return s;
    if ((s = check_ptr(prob->qo_indptr, "qo_indptr", false))) return s;
    cudaError_t e = launch_kv_append(a, cache_kind(prob), rows->dtype == SPLITKV_F32, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "kv_append launch");
    return ok();
}

splitkv_status splitkv_kv_gather(const splitkv_problem* prob, const int32_t* kv_indptr, const int32_t* kv_begin,
                                 int32_t num_rows, const splitkv_kv_rows* rows, int32_t* dev_error_word,
                                 splitkv_stream stream) {
    CacheRowsArgs a;
    splitkv_status s = cache_rows_args(prob, rows, "kv_gather", &a);
    if (s) return s;
    if (num_rows < 0) return fail_with(SPLITKV_ERR_INVALID_ARG, "num_rows %d < 0", num_rows);
    a.rows = num_rows;
    a.indptr = kv_indptr;
    a.kv_begin = kv_begin;
    a.err = dev_error_word;
    if (num_rows == 0) return ok();
    for (int k = 0; k < 2; ++k) {
        // written rows must not overlap: (token, head) rows in either order of nesting
        const CachePart& c = a.part[k];
        if (c.width == 0) continue;
        const int64_t w = c.width, H = a.heads;
        const bool token_outer = (H == 1 || c.head_stride >= w) && c.token_stride >= (H == 1 ? w : (H - 1) * c.head_stride + w);
        const bool head_outer = c.token_stride >= w && (H == 1 || c.head_stride >= ((int64_t)num_rows - 1) * c.token_stride + w);
        if (num_rows > 1 || H > 1) {
            if (!token_outer && !head_outer && !(num_rows == 1 && c.head_stride >= w))
                return fail_with(SPLITKV_ERR_INVALID_ARG, "%s strides make output rows overlap", k ? "v" : "k");
        }
    }
    if ((s = check_rows_ptrs(prob, a, dev_error_word))) return s;
    if ((s = check_ptr(kv_indptr, "kv_indptr", false))) return s;
    if ((s = check_ptr(kv_begin, "kv_begin", true))) return s;
    cudaError_t e = launch_kv_gather(a, cache_kind(prob), rows->dtype == SPLITKV_F32, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "kv_gather launch");
    return ok();
}

splitkv_status splitkv_verify_drafts(const splitkv_verify* v, int32_t* dev_error_word, splitkv_stream stream) {
    if (!v) return fail_with(SPLITKV_ERR_INVALID_ARG, "verify arguments are NULL");
    if (v->batch < 1 || v->batch > (1 << 24)) return fail_with(SPLITKV_ERR_INVALID_ARG, "batch %d", v->batch);
    if (v->total_q < 0) return fail_with(SPLITKV_ERR_INVALID_ARG, "total_q %d < 0", v->total_q);
    if (v->vocab < 1 || v->vocab > (1 << 30)) return fail_with(SPLITKV_ERR_INVALID_ARG, "vocab %d", v->vocab);
    if (v->reserved != 0) return fail_with(SPLITKV_ERR_INVALID_ARG, "reserved must be 0");
    if (v->target_stride < v->vocab || (v->draft_probs && v->draft_stride < v->vocab))
        return fail_with(SPLITKV_ERR_INVALID_ARG, "row strides must be at least vocab");
    if (((uintptr_t)v->target_probs | (uintptr_t)v->draft_probs) & 3)
        return fail_with(SPLITKV_ERR_INVALID_ARG, "probabilities are not aligned to their elements");
    if ((v->seq_lens == nullptr) != (v->seq_lens_out == nullptr))
        return fail_with(SPLITKV_ERR_INVALID_ARG, "seq_lens and seq_lens_out come together");
    const uintptr_t in = (uintptr_t)v->tokens, out = (uintptr_t)v->out_tokens, bytes = (uintptr_t)v->total_q * 4;
    if (in && out && in < out + bytes && out < in + bytes)
        return fail_with(SPLITKV_ERR_INVALID_ARG, "out_tokens overlaps tokens");
    splitkv_status s;
    const bool none = v->total_q == 0;
    if ((s = check_ptr(v->qo_indptr, "qo_indptr", false))) return s;
    if ((s = check_ptr(v->tokens, "tokens", none))) return s;
    if ((s = check_ptr(v->target_probs, "target_probs", none))) return s;
    if ((s = check_ptr(v->draft_probs, "draft_probs", true))) return s;
    if ((s = check_ptr(v->accept_u, "accept_u", none))) return s;
    if ((s = check_ptr(v->sample_u, "sample_u", false))) return s;
    if ((s = check_ptr(v->seq_lens, "seq_lens", true))) return s;
    if ((s = check_ptr(v->seq_lens_out, "seq_lens_out", true))) return s;
    if ((s = check_ptr(v->out_tokens, "out_tokens", none))) return s;
    if ((s = check_ptr(v->accepted, "accepted", false))) return s;
    if ((s = check_ptr(dev_error_word, "dev_error_word", true))) return s;
    VerifyArgs a;
    std::memset(&a, 0, sizeof a);
    a.tokens = v->tokens;
    a.qo_indptr = v->qo_indptr;
    a.target = v->target_probs;
    a.draft = v->draft_probs;
    a.target_stride = v->target_stride;
    a.draft_stride = v->draft_stride;
    a.accept_u = v->accept_u;
    a.sample_u = v->sample_u;
    a.seq_lens = v->seq_lens;
    a.seq_lens_out = v->seq_lens_out;
    a.out_tokens = v->out_tokens;
    a.accepted = v->accepted;
    a.err = dev_error_word;
    a.batch = v->batch;
    a.total_q = v->total_q;
    a.vocab = v->vocab;
    cudaError_t e = launch_verify_drafts(a, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "verify_drafts launch");
    return ok();
}

}  // extern "C"
