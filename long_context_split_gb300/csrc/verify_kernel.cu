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
// draw falls in, and the CTA that owns it reads that segment again (from L2), a step of 128
// tokens per warp, and sums, picks the step and then the token in the same way.
//
// Arithmetic: float64 adds run at 1/64 of the float32 rate here (a scan of 16 sums by every
// warp of a CTA took 7 us), so sums are unevaluated pairs of float32, about 48 bits: each
// difference and each addition is split into a rounded value and its exact error.
// The order of every sum is fixed.
#include <algorithm>

#include "operators.h"

namespace skv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kLoads = 4;          // loads of p and of q in flight per lane

// hi + lo, |lo| at most half a unit in the last place of hi once normalised
struct Pair {
    float hi, lo;
};

// s + e = a + b exactly
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
    s = __fadd_rn(a, b);
    const float bb = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}

__device__ __forceinline__ Pair normal(float s, float e) {
    Pair r;
    r.hi = __fadd_rn(s, e);
    r.lo = __fsub_rn(e, __fsub_rn(r.hi, s));
    return r;
}

__device__ __forceinline__ Pair add(Pair a, Pair b) {
    float s, e;
    two_sum(a.hi, b.hi, s, e);
    return normal(s, __fadd_rn(e, __fadd_rn(a.lo, b.lo)));
}

__device__ __forceinline__ Pair sub(Pair a, Pair b) { return add(a, Pair{-b.hi, -b.lo}); }

__device__ __forceinline__ Pair scale(float u, Pair a) {
    const float p = __fmul_rn(u, a.hi);
    return normal(p, __fmaf_rn(u, a.lo, __fmaf_rn(u, a.hi, -p)));
}

__device__ __forceinline__ bool greater(Pair a, Pair b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }

__device__ __forceinline__ Pair shfl(Pair a, int from) {
    return Pair{__shfl_sync(0xffffffffu, a.hi, from), __shfl_sync(0xffffffffu, a.lo, from)};
}

// the weight of a token, max(p - q, 0) (NaN and negative weigh nothing)
__device__ __forceinline__ Pair weight(float p, float q) {
    Pair w{0.f, 0.f};
    if (p > q) two_sum(p, -q, w.hi, w.lo);
    return w;
}

// s += w without normalising: lo only collects errors far below hi
__device__ __forceinline__ void accumulate(Pair& s, Pair w) {
    float hi, e;
    two_sum(s.hi, w.hi, hi, e);
    s.hi = hi;
    s.lo = __fadd_rn(s.lo, __fadd_rn(e, w.lo));
}

// p and q of VEC tokens (q 0 without a draft row; p 0 past the end and for the excluded token)
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

// by every thread; each warp's lanes come back together first, as the aligned forms need
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ Pair remote_pair(const Pair* local, uint32_t rank) {
    uint32_t addr;
    Pair v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"((uint32_t)__cvta_generic_to_shared(local)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.hi), "=f"(v.lo) : "r"(addr) : "memory");
    return v;
}

// sum over the warp (lane 0's value is the one used)
__device__ __forceinline__ Pair warp_sum(Pair s) {
#pragma unroll
    for (int d = 16; d; d >>= 1)
        s = add(s, Pair{__shfl_xor_sync(0xffffffffu, s.hi, d), __shfl_xor_sync(0xffffffffu, s.lo, d)});
    return s;
}

// sum over the lanes up to this one
__device__ __forceinline__ Pair warp_scan(Pair x, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Pair y{__shfl_up_sync(0xffffffffu, x.hi, d), __shfl_up_sync(0xffffffffu, x.lo, d)};
        if (lane >= d) x = add(y, x);
    }
    return x;
}

struct Pick {
    Pair before;   // sum of the weights before the picked entry
    int index;     // the picked entry; -1: no weight
    bool over;     // its running sum exceeds the draw (else it is the last entry with weight)
};

// The lowest of 32 * N entries (N consecutive ones per lane, `excl` the sum before the
// lane's) whose running sum exceeds `at`, among those with weight; the last one with weight if
// none does.  The same result in every lane.
template <int N>
__device__ __forceinline__ Pick pick(const Pair (&part)[N], Pair excl, Pair at, int lane) {
    Pair c = excl, over_before = excl, last_before = excl;
    int over = -1, last = -1;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const Pair next = add(c, part[k]);
        if (part[k].hi > 0.f) {
            last = k;
            last_before = c;
            if (over < 0 && greater(next, at)) {
                over = k;
                over_before = c;
            }
        }
        c = next;
    }
    const unsigned has = __ballot_sync(0xffffffffu, last >= 0), hit = __ballot_sync(0xffffffffu, over >= 0);
    const int from = hit ? __ffs(hit) - 1 : has ? 31 - __clz(has) : 0;
    Pick d;
    d.over = hit != 0;
    d.before = shfl(hit ? over_before : last_before, from);
    d.index = __shfl_sync(0xffffffffu, hit ? over : last, from);
    if (d.index >= 0) d.index += N * from;
    return d;
}

template <int VEC>
__global__ void __launch_bounds__(kThreads, 2) verify_drafts_kernel(VerifyArgs a, int cluster) {
    __shared__ __align__(8) Pair seg_sum[2][kWarps], step_sum[kWarps];
    __shared__ Pair s_at;
    __shared__ Pick s_seg;
    __shared__ int s_accepted, s_token;
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
        Pair s{0.f, 0.f};
        for (int v = v0 + lane * VEC; v < v1; v += kLoads * kStep) {
            Tokens<VEC> t[kLoads];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) load_tokens<VEC>(t[k], p, q, v + k * kStep, v1, excluded);
#pragma unroll
            for (int k = 0; k < kLoads; ++k)
#pragma unroll
                for (int j = 0; j < VEC; ++j) accumulate(s, weight(t[k].p[j], t[k].q[j]));
        }
        s = warp_sum(s);
        if (lane == 0) seg_sum[pass][warp] = s;
        cluster_sync();
        // ---- the segment of the draw: warp 0 of every CTA scans all segments' sums the same way ----
        if (warp == 0) {
            constexpr int kPer = kMaxCluster * kWarps / 32;      // consecutive segments per lane
            Pair part[kPer], own{0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int i = kPer * lane + k;
                part[k] = i < warps ? remote_pair(&seg_sum[pass][i % kWarps], i / kWarps) : Pair{0.f, 0.f};
                own = add(own, part[k]);
            }
            const Pair incl = warp_scan(own, lane);
            const Pair at = scale(a.sample_u[b], shfl(incl, 31));
            const Pick d = pick<kPer>(part, sub(incl, own), at, lane);
            if (lane == 0) {
                s_at = at;
                s_seg = d;
            }
        }
        __syncthreads();
        const int segment = s_seg.index;
        if (segment < 0) {                                       // no weight at all
            if (q == nullptr && excluded < 0) {
                none = true;
                break;
            }
            q = nullptr;
            excluded = -1;
            __syncthreads();
            continue;
        }
        if (segment / kWarps != rank) break;
        // ---- the token inside the segment, by the CTA that owns it: a step per warp ----
        mine = true;
        const int g0 = segment * seg, g1 = min(g0 + seg, V);
        const Pair at = s_at;
        Pair before = s_seg.before;
        for (int base = g0; base < g1; base += kWarps * kStep) {
            Tokens<VEC> t;
            const int v = base + warp * kStep + lane * VEC;
            load_tokens<VEC>(t, p, q, v, g1, excluded);
            Pair m[VEC], sum{0.f, 0.f};
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                m[j] = weight(t.p[j], t.q[j]);
                sum = add(sum, m[j]);
            }
            const Pair step = warp_sum(sum);
            if (lane == 0) step_sum[warp] = step;
            __syncthreads();
            // every warp picks the step (16 sums, a lane each)
            const Pair part[1] = {lane < kWarps ? step_sum[lane] : Pair{0.f, 0.f}};
            const Pair incl = warp_scan(part[0], lane);
            const Pick d = pick<1>(part, add(before, sub(incl, part[0])), at, lane);
            if (d.index == warp) {
                const Pair own = warp_scan(sum, lane);
                const Pick in = pick<VEC>(m, add(d.before, sub(own, sum)), at, lane);
                if (lane == 0) s_token = base + warp * kStep + in.index;
            }
            before = add(before, shfl(incl, 31));
            __syncthreads();
            if (d.index >= 0) token = s_token;
            if (d.over) break;
        }
        break;
    }
    // ---- outputs: one CTA has the token; no weight anywhere gives -1 ----
    if (mine && threadIdx.x == 0) a.out_tokens[r0 + acc] = token;
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
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // CTAs per request: as many as leave each 4096 tokens and run at once.  An SM takes two, but clusters
    // stay within a GPC, so that 1.6 an SM is what fits (48 requests of 128k tokens: four CTAs each
    // 22.3 us, five 20.5, six -- a second wave -- 30.8)
    const int cluster = std::min({kMaxCluster, (a.vocab + 4095) / 4096, std::max(1, 8 * sms / 5 / a.batch)});
    const bool vec = a.target_stride % 4 == 0 && !((uintptr_t)a.target & 15) &&
                     (!a.draft || (a.draft_stride % 4 == 0 && !((uintptr_t)a.draft & 15)));
    return vec ? launch<4>(a, cluster, s) : launch<1>(a, cluster, s);
}

}  // namespace skv
