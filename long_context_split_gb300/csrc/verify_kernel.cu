// Verification of drafted tokens against the target's probabilities.
//
// What it computes, for request b with query rows r0 .. r0 + n (row 0 fed the
// last accepted token, rows 1 .. n the drafts x_1 .. x_n): draft x_i is
// accepted while u_i q_i(x_i) < p_i(x_i) (rows r0 + i - 1 of the target's p and
// the draft's q).  At the first refusal, row r = r0 + a, one token is drawn
// from max(p_r - q_r, 0); with every draft accepted (a = n) from p_r.  The draw
// inverts the distribution function: the lowest token v with
// sum_{w <= v} weight_w > u sum_w weight_w.
//
// What bounds it: one row of p and q per request, 8 bytes a token of the
// vocabulary, read once.  A cluster of CTAs takes a request, a warp a
// contiguous segment of the vocabulary: one pass sums every segment; the
// segments' sums, shared through distributed shared memory, show which one the
// draw falls in, and that warp reads its own segment again (from L2).
//
// Arithmetic: products and differences of two float32 values are exact in
// float64, but float64 adds run at a small fraction of the float32 rate, so a
// lane sums its weights as an unevaluated pair of float32 (each difference and
// each addition split into a rounded value and its exact error) and the pairs
// become float64 once per lane.  The order of every sum is fixed.
#include <algorithm>

#include "internal.h"

namespace skv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kLoads = 4;          // loads of p and of q in flight per lane

struct Pair {
    float hi = 0.f, lo = 0.f;
};

// s + e = a + b exactly
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
    s = __fadd_rn(a, b);
    const float bb = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}

// the weight of a token, max(p - q, 0), as hi + lo (NaN and negative weigh nothing)
__device__ __forceinline__ Pair weight(float p, float q) {
    Pair w;
    if (p > q) two_sum(p, -q, w.hi, w.lo);
    return w;
}

__device__ __forceinline__ void accumulate(Pair& s, Pair w) {
    float hi, e;
    two_sum(s.hi, w.hi, hi, e);
    s.hi = hi;
    s.lo = __fadd_rn(s.lo, __fadd_rn(e, w.lo));
}

// p and q of VEC tokens (q 0 without a draft row; the excluded token's q is its p)
template <int VEC>
struct Tokens {
    float p[VEC], q[VEC];
};

template <int VEC>
__device__ __forceinline__ void load_tokens(Tokens<VEC>& t, const float* p, const float* q, int v, int end, int excluded) {
    if (VEC == 4 && v + 3 < end) {
        const float4 x = *(const float4*)(p + v);
        t.p[0] = x.x; t.p[1 % VEC] = x.y; t.p[2 % VEC] = x.z; t.p[3 % VEC] = x.w;
        if (q) {
            const float4 y = *(const float4*)(q + v);
            t.q[0] = y.x; t.q[1 % VEC] = y.y; t.q[2 % VEC] = y.z; t.q[3 % VEC] = y.w;
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) t.q[k] = 0.f;
        }
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            t.p[k] = v + k < end ? p[v + k] : 0.f;
            t.q[k] = q && v + k < end ? q[v + k] : 0.f;
        }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k)
        if (v + k == excluded) t.p[k] = 0.f;
}

__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ double remote_double(const double* local, uint32_t rank) {
    uint32_t addr;
    double v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"((uint32_t)__cvta_generic_to_shared(local)), "r"(rank));
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
    return v;
}

template <int VEC>
__global__ void __launch_bounds__(kThreads, 2) verify_drafts_kernel(VerifyArgs a, int cluster) {
    __shared__ double seg_sum[2][kWarps];
    __shared__ int s_accepted;
    const int b = blockIdx.x / cluster, rank = (int)cluster_ctarank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r0 = a.qo_indptr[b], rows = a.qo_indptr[b + 1] - r0, n = rows - 1;
    const int V = a.vocab;
    // the cluster leaves together: every CTA of it sees the same request
    if (rows <= 0 || r0 < 0 || r0 + rows > a.total_q) {
        if (rank == 0 && threadIdx.x == 0) {
            if (rows != 0 && a.err) atomicCAS(a.err, 0, ERR_DEVICE_CHECK | SITE_TOKEN_RANGE);
            a.accepted[b] = 0;
            if (a.seq_lens_out) a.seq_lens_out[b] = a.seq_lens[b];
        }
        return;
    }
    // ---- how many drafts are accepted: 32 tests at a time (every CTA for itself) ----
    if (warp == 0) {
        int acc = n;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane;
            bool take = true;
            if (i < n) {
                const int x = a.tokens[r0 + i + 1];
                if (x < 0 || x >= V) {
                    take = false;
                    if (rank == 0 && a.err) atomicCAS(a.err, 0, ERR_DEVICE_CHECK | SITE_TOKEN_RANGE);
                } else {
                    const double p = a.target[(r0 + i) * a.target_stride + x];
                    const double q = a.draft ? (double)a.draft[(r0 + i) * a.draft_stride + x] : 1.0;
                    take = (double)a.accept_u[r0 + i] * q < p;   // float32 x float32: exact
                }
            }
            const unsigned no = __ballot_sync(0xffffffffu, !take);
            if (no) {
                acc = i0 + __ffs(no) - 1;
                break;
            }
        }
        if (lane == 0) s_accepted = acc;
    }
    __syncthreads();
    const int acc = s_accepted;
    const float* p = a.target + (r0 + acc) * a.target_stride;
    const float* q = acc < n && a.draft ? a.draft + (r0 + acc) * a.draft_stride : nullptr;
    int excluded = acc < n && !a.draft ? a.tokens[r0 + acc + 1] : -1;   // max(p - q, 0) with q certain of it
    // this warp's segment of the vocabulary, a multiple of a step's tokens
    constexpr int kStep = 32 * VEC;
    const int warps = cluster * kWarps;
    const int seg = ((V + warps - 1) / warps + kStep - 1) / kStep * kStep;
    const int w = rank * kWarps + warp;
    const int v0 = (int)min((long long)w * seg, (long long)V), v1 = min(v0 + seg, V);
    int token = -1;
    bool mine = false, none = false;
    // the second pass, over p alone, only where max(p - q, 0) is zero everywhere
    for (int pass = 0; pass < 2; ++pass) {
        Pair s;
        for (int v = v0 + lane * VEC; v < v1; v += kLoads * kStep) {
            Tokens<VEC> t[kLoads];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) load_tokens<VEC>(t[k], p, q, v + k * kStep, v1, excluded);
#pragma unroll
            for (int k = 0; k < kLoads; ++k)
#pragma unroll
                for (int j = 0; j < VEC; ++j) accumulate(s, weight(t[k].p[j], t[k].q[j]));
        }
        double sum = (double)s.hi + (double)s.lo;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) seg_sum[pass][warp] = sum;
        cluster_sync();
        // ---- the segment of the draw: every warp scans all segments' sums the same way ----
        double part[kMaxCluster * kWarps / 32], run = 0.0;
#pragma unroll
        for (int k = 0; k < kMaxCluster * kWarps / 32; ++k) {
            const int i = 32 * k + lane;
            part[k] = i < warps ? remote_double(&seg_sum[pass][i % kWarps], i / kWarps) : 0.0;
        }
        double before = 0.0, total = 0.0;
        int owner = -1, last = -1;
        double incl[kMaxCluster * kWarps / 32];
#pragma unroll
        for (int k = 0; k < kMaxCluster * kWarps / 32; ++k) {
            double x = part[k];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            incl[k] = run + x;
            run = __shfl_sync(0xffffffffu, incl[k], 31);
        }
        total = run;
        if (!(total > 0.0)) {
            if (q == nullptr && excluded < 0) {          // p itself has no mass: no token
                none = true;
                break;
            }
            q = nullptr;
            excluded = -1;
            continue;
        }
        const double at = (double)a.sample_u[b] * total;
#pragma unroll
        for (int k = 0; k < kMaxCluster * kWarps / 32; ++k) {
            const unsigned has = __ballot_sync(0xffffffffu, part[k] > 0.0);
            const unsigned over = __ballot_sync(0xffffffffu, part[k] > 0.0 && incl[k] > at);
            if (has) last = 32 * k + 31 - __clz(has);
            if (over && owner < 0) owner = 32 * k + __ffs(over) - 1;
        }
        if (owner < 0) owner = last;                     // u at the very end of the distribution
        mine = owner == w;
        if (!mine) break;
#pragma unroll
        for (int k = 0; k < kMaxCluster * kWarps / 32; ++k) {
            const double excl = __shfl_sync(0xffffffffu, incl[k] - part[k], owner & 31);
            if (k == owner / 32) before = excl;
        }
        // ---- the token inside the segment: steps of 32 * VEC tokens in order ----
        for (int s0 = v0; s0 < v1; s0 += kStep) {
            const int v = s0 + lane * VEC;
            Tokens<VEC> t;
            load_tokens<VEC>(t, p, q, v, v1, excluded);
            Pair m[VEC];
            Pair sum_lane;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                m[j] = weight(t.p[j], t.q[j]);
                accumulate(sum_lane, m[j]);
            }
            const double own = (double)sum_lane.hi + (double)sum_lane.lo;
            double x = own;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            const unsigned has = __ballot_sync(0xffffffffu, own > 0.0);
            const unsigned over = __ballot_sync(0xffffffffu, own > 0.0 && before + x > at);
            const int pick = over ? __ffs(over) - 1 : has ? 31 - __clz(has) : -1;
            if (pick >= 0) {
                // within the lane: the first token over the draw, else its last one with mass
                double c = before + (x - own);
                int found = -1, tail = -1;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    c += (double)m[j].hi + (double)m[j].lo;
                    if (m[j].hi > 0.f) {
                        tail = v + j;
                        if (found < 0 && c > at) found = v + j;
                    }
                }
                const int cand = over && found >= 0 ? found : tail;
                token = __shfl_sync(0xffffffffu, cand, pick);
            }
            if (over) break;
            before += __shfl_sync(0xffffffffu, x, 31);
        }
        break;
    }
    // ---- outputs: one warp has the token; no mass anywhere gives -1 ----
    if (mine && lane == 0) a.out_tokens[r0 + acc] = token;
    if (rank == 0) {
        if (none && threadIdx.x == 0) a.out_tokens[r0 + acc] = -1;
        for (int i = threadIdx.x; i < rows; i += kThreads)
            if (i != acc) a.out_tokens[r0 + i] = i < acc ? a.tokens[r0 + i + 1] : -1;
        if (threadIdx.x == 0) {
            a.accepted[b] = acc;
            if (a.seq_lens_out) a.seq_lens_out[b] = a.seq_lens[b] - n + acc;
        }
    }
    cluster_sync();   // no CTA leaves while another may still read its sums
}

template <int VEC>
cudaError_t launch(const VerifyArgs& a, int cluster, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.batch * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    ProfileScope ps(SPLITKV_KERNEL_VERIFY, s);
    return cudaLaunchKernelEx(&cfg, verify_drafts_kernel<VEC>, a, cluster);
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs& a, cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    // CTAs per request: while each still has 4096 tokens and the SMs are not full (two CTAs each)
    int cluster = 1;
    while (cluster < kMaxCluster && a.vocab > 4096 * cluster && (long long)a.batch * cluster <= sms) cluster *= 2;
    const bool vec = a.target_stride % 4 == 0 && !((uintptr_t)a.target & 15) &&
                     (!a.draft || (a.draft_stride % 4 == 0 && !((uintptr_t)a.draft & 15)));
    return vec ? launch<4>(a, cluster, s) : launch<1>(a, cluster, s);
}

}  // namespace skv
