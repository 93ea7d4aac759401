// C-ABI entry points of the operators around the attention call: cache rows in
// and out, latent attention from the model's own queries, and the verification
// of drafted tokens.  Argument checks and the expanded form's plan; the
// arithmetic runs in the CUDA kernels.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <vector>

#include <cuda_runtime.h>

#include "splitkv.h"
#include "latent.h"
#include "operators.h"

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

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

int device_sms() {
    const int n = sm_count();
    return n > 0 ? n : 152;   // GB300, where no device is visible
}

splitkv_status check_latent_problem(const splitkv_problem* p) {
    splitkv_status s = check_problem_lengths(p);
    if (s) return s;
    if (p->kind != SPLITKV_MLA) return fail_with(SPLITKV_ERR_INVALID_ARG, "latent attention takes an MLA problem");
    if (p->v_cache) return fail_with(SPLITKV_ERR_INVALID_ARG, "an MLA cache has no v_cache");
    if (p->dtype != SPLITKV_BF16 || p->head_dim_qk != kLatRow || p->head_dim_v != kLatC)
        return fail_with(SPLITKV_ERR_UNSUPPORTED, "latent attention needs BF16, head_dim_qk 576 and head_dim_v 512");
    if (!(p->scale > 0.f)) return fail_with(SPLITKV_ERR_UNSUPPORTED, "latent attention needs scale > 0");
    return SPLITKV_OK;
}

splitkv_status check_layer(const splitkv_problem* p, const splitkv_latent_layer* l, bool need_q, bool need_out) {
    splitkv_status s;
    if (!l) return fail_with(SPLITKV_ERR_INVALID_ARG, "layer is NULL");
    if (need_q && (l->q_token_stride % 8 || l->q_token_stride < (int64_t)p->num_q_heads * kLatQ || l->q_token_stride > (1LL << 38)))
        return fail_with(SPLITKV_ERR_INVALID_ARG, "q_token_stride %lld: need a multiple of 8, at least num_q_heads * 192",
                         (long long)l->q_token_stride);
    if ((need_q && ((uintptr_t)l->q & 15)) || ((uintptr_t)l->w_kv_b & 15) || (need_out && ((uintptr_t)l->out & 15)))
        return fail_with(SPLITKV_ERR_INVALID_ARG, "q, w_kv_b and out must be 16-byte aligned");
    if (need_q && (s = check_ptr(l->q, "q", false))) return s;
    if ((s = check_ptr(l->w_kv_b, "w_kv_b", false))) return s;
    if (need_out && (s = check_ptr(l->out, "out", false))) return s;
    return SPLITKV_OK;
}

LatentArgs layer_args(const splitkv_problem* p, const splitkv_latent_layer* l, int32_t* err) {
    LatentArgs a;
    std::memset(&a, 0, sizeof a);
    a.q = l->q;
    a.q_stride = l->q_token_stride;
    a.w = l->w_kv_b;
    a.out = l->out;
    a.err = err;
    a.total_q = p->qo_indptr_host[p->batch];
    a.heads = p->num_q_heads;
    a.inject = debug_inject();
    return a;
}

int cache_kind(const splitkv_problem* p) { return p->kv_fp8 ? 2 : p->dtype == SPLITKV_BF16 ? 1 : 0; }

}  // namespace

namespace skv {
int sm_count() {
    static std::atomic<int> known[64];   // per device, a constant of the hardware
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (dev >= 0 && dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (dev >= 0 && dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

cudaError_t allow_smem(const void* kernel, size_t bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)) != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_release);
    return cudaSuccess;
}
}  // namespace skv

struct splitkv_latent_plan_s {
    int32_t batch = 0, heads = 0, page = 0, max_pages = 0, kv_fp8 = 0, total_q = 0;
    int32_t pairs = 0;                      // some tasks are of two heads
    std::vector<int32_t> seq_len, qo;
    std::vector<LatentReq> reqs;
    std::vector<LatentTask> tasks;          // group after group of heads
    std::vector<int32_t> group_tasks;       // first task of each group, then their number
    int32_t group = 0;                      // heads of a group (the last one may have fewer)
    std::vector<LatentBlock> blocks;
    std::vector<int32_t> state_indptr;      // empty when nothing is split
    int64_t num_states = 0;
    std::vector<unsigned char> image;       // control block and descriptors
    size_t off_tasks = 0, off_reqs = 0, off_blocks = 0, off_indptr = 0;
    size_t off_rows = 0, off_kv = 0, off_vexp = 0, off_opart = 0, off_lse = 0, ws_bytes = 0;
};

namespace {

splitkv_status build_latent_plan(const splitkv_problem* p, splitkv_latent_plan_t* pl) {
    constexpr int kTaskRows = 256, kTileRows = 128;
    const int B = p->batch, H = p->num_q_heads;
    pl->batch = B;
    pl->heads = H;
    pl->page = p->page_size;
    pl->max_pages = p->max_pages_per_req;
    pl->kv_fp8 = p->kv_fp8;
    pl->seq_len.assign(p->seq_lens_host, p->seq_lens_host + B);
    pl->qo.assign(p->qo_indptr_host, p->qo_indptr_host + B + 1);
    pl->total_q = pl->qo[B];
    long long per_head = 0, units = 0, rows = 0;      // tasks of a head before splits; units of 64 tokens
    for (int b = 0; b < B; ++b) {
        const int t = pl->qo[b + 1] - pl->qo[b];
        per_head += (t + kTaskRows - 1) / kTaskRows;
        if (t > 0) units += (pl->seq_len[b] + kLatUnit - 1) / kLatUnit;
    }
    if (per_head * H > (1 << 28)) return fail_with(SPLITKV_ERR_INVALID_ARG, "too many tasks");
    if ((long long)pl->total_q * H >= (1LL << 31)) return fail_with(SPLITKV_ERR_UNSUPPORTED, "num_q_heads * query tokens exceeds 2^31");
    if (units * kLatUnit >= (1LL << 31) - 256) return fail_with(SPLITKV_ERR_UNSUPPORTED, "cached tokens exceed 2^31");
    // equal groups of an even number of heads (a task may be of two)
    pl->group = H;
    if (units * H > (long long)(kLatImageBytes / kLatImage)) {
        const int most = std::max(2, (int)(kLatImageBytes / kLatImage / units) & ~1), groups = (H + most - 1) / most;
        pl->group = std::min({H, most, ((H + groups - 1) / groups + 1) & ~1});
    }
    const long long unsplit = per_head * pl->group;       // tasks of a group, which run together
    const int sms = device_sms();
    pl->reqs.resize(B);
    for (int b = 0; b < B; ++b) {
        LatentReq& r = pl->reqs[b];
        std::memset(&r, 0, sizeof r);
        r.seq_len = pl->seq_len[b];
        r.q_start = pl->qo[b];
        r.q_len = pl->qo[b + 1] - pl->qo[b];
        r.row_base = (int32_t)rows;
        // fewer tasks than SMs: cut the histories so that the SMs are filled once and no more, in splits of at
        // least 1024 keys (one token after 65,536, 16 heads: 144 tasks 330 us, 160 tasks 400)
        r.n_splits = 1;
        if (unsplit > 0 && unsplit < sms)
            r.n_splits = (int32_t)std::max<long long>(1, std::min<long long>(sms / unsplit, r.seq_len / 1024));
        if (r.q_len == 0) continue;          // nothing to attend: its rows are not copied
        const int blocks = (r.seq_len + kLatUnit - 1) / kLatUnit;
        for (int k = 0; k < blocks; ++k) pl->blocks.push_back(LatentBlock{b, k * kLatUnit});
        rows += (long long)blocks * kLatUnit;
    }
    // The tasks of a (request, head, split) read the same keys and values: together, longest first,
    // so that those stay in L2; the request with the longest task first.
    std::vector<int> order(B);
    for (int b = 0; b < B; ++b) order[b] = b;
    std::stable_sort(order.begin(), order.end(), [&](int x, int y) { return pl->reqs[x].seq_len > pl->reqs[y].seq_len; });
    // A request of one tile of query tokens leaves half of a task's threads idle: two heads per task, when
    // there are more tasks than SMs anyway (attention over 128 heads: 32 prompts of 117 tokens 134 -> 108 us,
    // 64 of 60 162 -> 118, 2 x 96 tokens after 30,000 709 -> 676).
    const bool pairs = unsplit > sms;
    for (int head0 = 0; head0 < H; head0 += pl->group) {
        const int end = std::min(H, head0 + pl->group);
        pl->group_tasks.push_back((int32_t)pl->tasks.size());
        for (int b : order) {
            const LatentReq& r = pl->reqs[b];
            const int together = pairs && r.q_len <= kTileRows ? 2 : 1;
            const int nblk = (r.seq_len + kLatUnit - 1) / kLatUnit, per = nblk / r.n_splits, extra = nblk % r.n_splits;
            for (int h = head0; h < end; h += together)
                for (int s = 0; s < r.n_splits; ++s) {
                    const int first = s * per + std::min(s, extra), count = per + (s < extra ? 1 : 0);
                    for (int row = (r.q_len - 1) / kTaskRows * kTaskRows; r.q_len > 0 && row >= 0; row -= kTaskRows) {
                        LatentTask t;
                        std::memset(&t, 0, sizeof t);
                        t.b = b;
                        t.head = h;
                        t.row_begin = row;
                        t.row_end = std::min(r.q_len, row + kTaskRows);
                        t.key_begin = std::min(first * kLatUnit, r.seq_len);
                        t.key_end = std::min((first + count) * kLatUnit, r.seq_len);
                        t.split = s;
                        t.heads = std::min(together, end - h);
                        pl->pairs |= t.heads - 1;
                        pl->tasks.push_back(t);
                    }
                }
        }
    }
    pl->group_tasks.push_back((int32_t)pl->tasks.size());
    // with any request split, every row of the batch goes through the merge (one state or more)
    bool split = false;
    for (const LatentReq& r : pl->reqs) split = split || (r.n_splits > 1 && r.q_len > 0);
    if (split) {
        for (LatentReq& r : pl->reqs) {
            r.state_base = (int32_t)pl->num_states;
            pl->num_states += (int64_t)r.q_len * H * r.n_splits;
            if (pl->num_states >= (1LL << 31) - 1) return fail_with(SPLITKV_ERR_INVALID_ARG, "too many partial states");
        }
        pl->state_indptr.resize((size_t)pl->total_q * H + 1);
        for (const LatentReq& r : pl->reqs)
            for (int64_t x = 0; x < (int64_t)r.q_len * H; ++x)
                pl->state_indptr[(size_t)r.q_start * H + x] = r.state_base + (int32_t)(x * r.n_splits);
        pl->state_indptr[(size_t)pl->total_q * H] = (int32_t)pl->num_states;
    }
    size_t off = sizeof(Control);
    pl->off_tasks = off;
    off = align256(off + pl->tasks.size() * sizeof(LatentTask));
    pl->off_reqs = off;
    off = align256(off + pl->reqs.size() * sizeof(LatentReq));
    pl->off_blocks = off;
    off = align256(off + pl->blocks.size() * sizeof(LatentBlock));
    pl->off_indptr = off;
    off = align256(off + pl->state_indptr.size() * sizeof(int32_t));
    pl->image.assign(off, 0);
    auto put = [&](size_t at, const void* src, size_t n) {
        if (n) std::memcpy(pl->image.data() + at, src, n);
    };
    put(pl->off_tasks, pl->tasks.data(), pl->tasks.size() * sizeof(LatentTask));
    put(pl->off_reqs, pl->reqs.data(), pl->reqs.size() * sizeof(LatentReq));
    put(pl->off_blocks, pl->blocks.data(), pl->blocks.size() * sizeof(LatentBlock));
    put(pl->off_indptr, pl->state_indptr.data(), pl->state_indptr.size() * sizeof(int32_t));
    pl->off_rows = off;
    off = align256(off + (size_t)rows * kLatRow * 2);
    pl->off_kv = off;
    off = align256(off + (size_t)(rows / kLatUnit) * pl->group * kLatImage);
    pl->off_vexp = off;
    off = align256(off + (size_t)(rows / kLatUnit) * pl->group * sizeof(LatentScale));
    pl->off_opart = off;
    off = align256(off + (size_t)pl->num_states * kLatV * 4);
    pl->off_lse = off;
    off = align256(off + (size_t)pl->num_states * 4);
    pl->ws_bytes = off;
    return SPLITKV_OK;
}

splitkv_status check_latent_workspace(const splitkv_latent_plan_t* pl, const void* ws, size_t bytes) {
    if (!pl) return fail_with(SPLITKV_ERR_INVALID_ARG, "plan is NULL");
    if (!ws) return fail_with(SPLITKV_ERR_WORKSPACE, "workspace is NULL");
    if ((uintptr_t)ws & 255) return fail_with(SPLITKV_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    if (bytes < pl->ws_bytes)
        return fail_with(SPLITKV_ERR_WORKSPACE, "workspace has %zu bytes, plan needs %zu", bytes, pl->ws_bytes);
    return check_ptr(ws, "workspace", false);
}

}  // namespace

extern "C" {

splitkv_status splitkv_latent_plan(const splitkv_problem* prob, splitkv_latent_plan_t** out) {
    if (!out) return fail_with(SPLITKV_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    splitkv_status s = check_latent_problem(prob);
    if (s) return s;
    splitkv_latent_plan_t* pl = nullptr;
    try {
        pl = new splitkv_latent_plan_t();
        if ((s = build_latent_plan(prob, pl))) {
            delete pl;
            return s;
        }
    } catch (...) {   // (no exception leaves a C entry)
        delete pl;
        return fail_with(SPLITKV_ERR_INVALID_ARG, "no host memory for the plan");
    }
    *out = pl;
    return ok();
}

void splitkv_latent_plan_destroy(splitkv_latent_plan_t* plan) { delete plan; }

size_t splitkv_latent_workspace_bytes(const splitkv_latent_plan_t* plan) { return plan ? plan->ws_bytes : 0; }

int32_t splitkv_latent_plan_num_tasks(const splitkv_latent_plan_t* plan) { return plan ? (int32_t)plan->tasks.size() : -1; }

splitkv_status splitkv_latent_plan_splits(const splitkv_latent_plan_t* plan, int32_t* n_splits) {
    if (!plan || !n_splits) return fail_with(SPLITKV_ERR_INVALID_ARG, "NULL argument");
    for (int b = 0; b < plan->batch; ++b) n_splits[b] = plan->reqs[b].n_splits;
    return ok();
}

splitkv_status splitkv_latent_upload(const splitkv_latent_plan_t* plan, void* workspace, size_t ws_bytes,
                                     splitkv_stream stream) {
    splitkv_status s = check_latent_workspace(plan, workspace, ws_bytes);
    if (s) return s;
    cudaError_t e = cudaMemcpyAsync(workspace, plan->image.data(), plan->image.size(), cudaMemcpyHostToDevice,
                                    (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "plan upload");
    return ok();
}

splitkv_status splitkv_latent_expanded(const splitkv_problem* prob, const splitkv_latent_plan_t* plan,
                                       const splitkv_latent_layer* layer, void* workspace, size_t ws_bytes,
                                       int32_t* dev_error_word, splitkv_stream stream) {
    if (!plan) return fail_with(SPLITKV_ERR_INVALID_ARG, "plan is NULL");
    splitkv_status s = check_latent_problem(prob);
    if (s) return s;
    if (prob->batch != plan->batch || prob->num_q_heads != plan->heads || prob->page_size != plan->page ||
        prob->max_pages_per_req != plan->max_pages || prob->kv_fp8 != plan->kv_fp8)
        return fail_with(SPLITKV_ERR_INVALID_ARG, "problem shape differs from the plan's");
    if (std::memcmp(prob->seq_lens_host, plan->seq_len.data(), plan->seq_len.size() * 4) ||
        std::memcmp(prob->qo_indptr_host, plan->qo.data(), plan->qo.size() * 4))
        return fail_with(SPLITKV_ERR_INVALID_ARG, "lengths differ from the plan's");
    if (plan->total_q == 0) return ok();
    if ((s = check_latent_workspace(plan, workspace, ws_bytes))) return s;
    if ((s = check_layer(prob, layer, true, true))) return s;
    if ((uintptr_t)prob->k_cache & 15) return fail_with(SPLITKV_ERR_INVALID_ARG, "k_cache must be 16-byte aligned");
    if ((s = check_ptr(prob->k_cache, "k_cache", false))) return s;
    if ((s = check_ptr(prob->page_table, "page_table", false))) return s;
    if ((s = check_ptr(layer->lse_out, "lse_out", true))) return s;
    if ((s = check_ptr(dev_error_word, "dev_error_word", true))) return s;
    unsigned char* base = (unsigned char*)workspace;
    Control* ctrl = (Control*)base;
    LatentArgs a = layer_args(prob, layer, dev_error_word ? dev_error_word : &ctrl->error_word);
    a.lse_out = layer->lse_out;
    a.cache = prob->k_cache;
    a.page_table = prob->page_table;
    a.reqs = (const LatentReq*)(base + plan->off_reqs);
    a.blocks = (const LatentBlock*)(base + plan->off_blocks);
    a.rows = base + plan->off_rows;
    a.kv = base + plan->off_kv;
    a.v_exp = (LatentScale*)(base + plan->off_vexp);
    if (plan->num_states > 0) {
        a.o_part = (float*)(base + plan->off_opart);
        a.lse_part = (float*)(base + plan->off_lse);
    }
    a.ctrl = ctrl;
    a.pairs = plan->pairs;
    a.num_blocks = (int32_t)plan->blocks.size();
    a.page_size = prob->page_size;
    a.num_pages = prob->num_pages;
    a.max_pages = prob->max_pages_per_req;
    a.kv_fp8 = prob->kv_fp8;
    a.v_scale = prob->kv_fp8 ? prob->k_scale : 1.f;
    a.scale_log2 = (float)((double)prob->scale * a.v_scale * 1.4426950408889634);
    cudaError_t e;
    if ((e = launch_latent_rows(a, (cudaStream_t)stream)) != cudaSuccess) return cuda_fail(e, "latent rows launch");
    for (size_t g = 0; g + 1 < plan->group_tasks.size(); ++g) {
        a.head0 = (int32_t)g * plan->group;
        a.group = std::min(plan->group, plan->heads - a.head0);
        a.tasks = (const LatentTask*)(base + plan->off_tasks) + plan->group_tasks[g];
        a.num_tasks = plan->group_tasks[g + 1] - plan->group_tasks[g];
        if ((e = launch_latent_expand(a, (cudaStream_t)stream)) != cudaSuccess) return cuda_fail(e, "latent expansion launch");
        if ((e = launch_latent_attention(a, (cudaStream_t)stream)) != cudaSuccess) return cuda_fail(e, "latent attention launch");
    }
    if (plan->num_states > 0) {
        e = launch_merge(a.o_part, 0, a.lse_part, (const int32_t*)(base + plan->off_indptr), plan->total_q * plan->heads, kLatV,
                         layer->out, 1, layer->lse_out, (cudaStream_t)stream);
        if (e != cudaSuccess) return cuda_fail(e, "merge launch");
    }
    return ok();
}

splitkv_status splitkv_latent_absorb_query(const splitkv_problem* prob, const splitkv_latent_layer* layer, void* q_abs,
                                           int32_t* dev_error_word, splitkv_stream stream) {
    splitkv_status s = check_latent_problem(prob);
    if (s) return s;
    if (prob->qo_indptr_host[prob->batch] == 0) return ok();
    if ((uintptr_t)q_abs & 15) return fail_with(SPLITKV_ERR_INVALID_ARG, "q_abs must be 16-byte aligned");
    if ((s = check_layer(prob, layer, true, false))) return s;
    if ((s = check_ptr(q_abs, "q_abs", false))) return s;
    if ((s = check_ptr(dev_error_word, "dev_error_word", true))) return s;
    cudaError_t e = launch_latent_absorb(layer_args(prob, layer, dev_error_word), q_abs, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "query absorption launch");
    return ok();
}

splitkv_status splitkv_latent_project(const splitkv_problem* prob, const splitkv_latent_layer* layer, const void* o_part,
                                      int32_t o_part_dtype, const float* lse_part, const int32_t* state_indptr,
                                      int32_t* dev_error_word, splitkv_stream stream) {
    splitkv_status s = check_latent_problem(prob);
    if (s) return s;
    if (o_part_dtype != SPLITKV_F32 && o_part_dtype != SPLITKV_BF16)
        return fail_with(SPLITKV_ERR_INVALID_ARG, "o_part_dtype %d", o_part_dtype);
    if (prob->qo_indptr_host[prob->batch] == 0) return ok();
    if ((uintptr_t)o_part & 15) return fail_with(SPLITKV_ERR_INVALID_ARG, "o_part must be 16-byte aligned");
    if ((s = check_layer(prob, layer, false, true))) return s;
    if ((s = check_ptr(o_part, "o_part", false))) return s;
    if ((s = check_ptr(lse_part, "lse_part", false))) return s;
    if ((s = check_ptr(state_indptr, "state_indptr", false))) return s;
    if ((s = check_ptr(layer->lse_out, "lse_out", true))) return s;
    if ((s = check_ptr(dev_error_word, "dev_error_word", true))) return s;
    LatentArgs a = layer_args(prob, layer, dev_error_word);
    a.lse_out = layer->lse_out;
    cudaError_t e = launch_latent_project(a, o_part, o_part_dtype == SPLITKV_BF16, lse_part, state_indptr, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "value projection launch");
    return ok();
}

int32_t splitkv_latent_prefers_expanded(const splitkv_problem* prob) {
    if (check_latent_problem(prob)) return -1;
    // Without the tcgen05 MLA kernel (128 heads, 64-token pages) the absorbed form attends on the CUDA cores, and
    // the expanded one is faster at every length: in us, expanded against absorbed, one token per
    // request, 8 / 16 / 64 heads: after 4,096 tokens 49 / 53 / 114 against 290 / 508 / 509; after 512k (8 and 16 heads)
    // 1279 / 2840 against 4348 / 7754; 64 requests of 300 tokens 78 / 123 / 380 against 188 / 318 / 611, of 1k to
    // 16k 985 / 1475 / 5676 against 3744 / 6669 / 16,241 (16 new tokens each: 989 / 1483 / 5741 against 21,092 /
    // 36,719 / 137,451); 128 heads on 16-token pages, the same 64 requests, 11,263 against 21,083.
    if (!mla_tc_supports(1, 1, prob->num_q_heads, prob->head_dim_qk, prob->head_dim_v, prob->page_size)) return 1;
    // Operations per head: see splitkv_latent_layer; the absorbed kernel computes its scores in both
    // halves of the output columns and its probabilities as a high part and a residual.  The two meet
    // at 71 tokens per request after a long history (128 heads, 2 x 32,768 tokens, absorbed against
    // expanded: 32 tokens 960 us, 2266; 64 tokens 1896, 2185; 128 tokens 3358, 2135).
    double tokens = 0, pairs = 0;
    for (int b = 0; b < prob->batch; ++b) {
        const double n = prob->seq_lens_host[b], t = prob->qo_indptr_host[b + 1] - prob->qo_indptr_host[b];
        if (t == 0) continue;
        tokens += n;
        pairs += t * (n - t) + t * (t + 1) / 2;
    }
    const double expanded = tokens * 262144 + pairs * 640, absorbed = pairs * 4352;
    return expanded < absorbed ? 1 : 0;
}

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
