// The end of absorbed latent attention in one kernel: the splits' partial states of
// each (token, head) are merged (LiquidCP Eq. 1) and the merged 512-wide latent
// output is projected by the head's W_uv.
//
// What it computes: o_lat = sum_s exp(lse_s - lse) o_s, lse = log sum_s exp(lse_s),
// out = o_lat W_uv^T, a CTA per head and 64 tokens.
//
// What bounds it: bytes (128 KB of weights per head, 2 KB per state) and, for one
// token, the chain index -> log-sum-exps -> states -> product.  So the weights' copy starts
// first (all 128 KB are resident); all rows' weights are computed at once (16 lanes a row); the
// states are read with several 16-byte loads in flight per thread, and up to 16 tokens share
// their splits out over the CTA's sixteen groups of 64 threads.  64 tokens a CTA keep a decode batch of 64 at one CTA per head.  The latent columns
// are merged and multiplied in two halves, so that the operands of one half (64 KB) fit
// beside the weights and the first half's product runs under the second half's merge (with
// the weights in a ring of four boxes instead, the products waited 3 us for the second four).
// The product is taken transposed, D[v][token] = W_uv[v][:] . o_lat[token][:]
// (M = 128 value columns, N = 64 tokens, K = 512), so that few tokens waste little.
//
// o_lat stays float32 until it meets the weights, as a bf16 high part and a bf16
// residual (two products with the same weights, 16 significant bits): rounding it to
// one bf16 would cost as much as the result's own rounding.
#include "latent.h"
#include "tc_issue.cuh"

namespace skv {
namespace {

constexpr int kThreads = 1024;
constexpr int kGroups = kThreads / 64;               // a group covers half of a row's 512 columns, four a thread
constexpr int kTok = 64;                             // tokens per CTA (N of the product)
constexpr int kTable = 64;                           // splits of a row whose weights are kept
constexpr int kBoxes = kLatC / 64;
constexpr int kWBox = kLatV * 128;                   // 128 weight rows x 64 columns
constexpr int kOBox = kTok * 128;                    // 64 tokens x 64 columns

struct Shared {
    unsigned long long w_full[2], done[2];           // per half of the latent columns
    uint32_t tmem_base;
    int abort_flag;
    float lse[kTok];
    int first[kTok], count[kTok];
    float4 part[kGroups][64];
    float weight[kTok][kTable];
};

constexpr size_t kSmemBytes = 1024 + kBoxes * (size_t)kWBox + kBoxes / 2 * (size_t)(2 * kOBox) + sizeof(Shared);
static_assert(kSmemBytes <= 232448, "shared memory budget");

template <bool BF16>
__device__ __forceinline__ float4 load_state(const void* o_part, int state, int col4) {
    if (BF16) {
        const uint2 v = *((const uint2*)((const __nv_bfloat16*)o_part + (size_t)state * kLatC) + col4);
        return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                           __uint_as_float(v.y & 0xFFFF0000u));
    }
    return *((const float4*)((const float*)o_part + (size_t)state * kLatC) + col4);
}

__device__ __forceinline__ void fma4(float4& s, float w, const float4& v) {
    s.x = fmaf(w, v.x, s.x);
    s.y = fmaf(w, v.y, s.y);
    s.z = fmaf(w, v.z, s.z);
    s.w = fmaf(w, v.w, s.w);
}

// the token's four columns (of the half) as bf16 high parts and residuals, in the swizzled operand boxes
__device__ __forceinline__ void put(unsigned char* hi, unsigned char* lo, int tok, int col4, const float4& s) {
    uint32_t h[2], l[2];
    split_bf16(s.x, s.y, h[0], l[0]);
    split_bf16(s.z, s.w, h[1], l[1]);
    const int c = col4 * 4, at = (c >> 6) * kOBox + tok * 128 + ((((c & 63) >> 3) ^ (tok & 7)) << 4) + (c & 7) * 2;
    *(uint2*)(hi + at) = make_uint2(h[0], h[1]);
    *(uint2*)(lo + at) = make_uint2(l[0], l[1]);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
latent_project_kernel(const __grid_constant__ CUtensorMap mw, LatentArgs a, const void* o_part, const float* lse_part,
                      const int32_t* indptr) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sW = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char* sHi = sW + kBoxes * kWBox;              // four boxes: a half of the columns
    unsigned char* sLo = sHi + kBoxes / 2 * kOBox;
    Shared& S = *(Shared*)(sLo + kBoxes / 2 * kOBox);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = blockIdx.x % a.heads, t0 = blockIdx.x / a.heads * kTok;
    const int n = min(kTok, a.total_q - t0);
    if (threadIdx.x == 0) {
        for (int h = 0; h < 2; ++h) {
            mbar_init(smem_u32(&S.w_full[h]), 1);
            mbar_init(smem_u32(&S.done[h]), 1);
        }
        S.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int j = 0; j < kBoxes; ++j) {
            const uint32_t full = smem_u32(&S.w_full[j / (kBoxes / 2)]);
            if (j % (kBoxes / 2) == 0) mbar_expect_tx(full, kBoxes / 2 * kWBox);
            tma_2d(smem_u32(sW + j * kWBox), &mw, 64 * j, head * kLatW + kLatNope, full);
        }
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem_base)), "r"(kTok)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // ---- each row's log-sum-exp over its states, and their weights: 16 lanes per row ----
    {
        const int t = threadIdx.x >> 4, sub = threadIdx.x & 15;
        const bool on = t < n;
        const size_t x = (size_t)(t0 + (on ? t : 0)) * a.heads + head;
        const int s0 = indptr[x], cnt = on ? indptr[x + 1] - s0 : 0;
        // (the first four of a lane's states stay in registers: all of them up to 64 splits)
        float own[4], m = -INFINITY, sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            own[k] = sub + 16 * k < cnt ? lse_part[s0 + sub + 16 * k] : -INFINITY;
            m = fmaxf(m, own[k]);
        }
        for (int s = sub + 64; s < cnt; s += 16) m = fmaxf(m, lse_part[s0 + s]);
#pragma unroll
        for (int d = 8; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float base = m == -INFINITY ? 0.f : m;         // (then every weight is exp(-inf) = 0)
#pragma unroll
        for (int k = 0; k < 4; ++k) sum += sub + 16 * k < cnt ? expf(own[k] - base) : 0.f;
        for (int s = sub + 64; s < cnt; s += 16) sum += expf(lse_part[s0 + s] - base);
#pragma unroll
        for (int d = 8; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const float lse = sum == 0.f ? -INFINITY : m + logf(sum);   // (a NaN among the states makes the sum NaN)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (sub + 16 * k < cnt) S.weight[t][sub + 16 * k] = sum == 0.f ? 0.f : expf(own[k] - lse);
        if (on && sub == 0) {
            S.lse[t] = lse;
            S.first[t] = s0;
            S.count[t] = cnt;
            if (a.lse_out) a.lse_out[x] = lse;
        }
    }
    __syncthreads();
    const uint32_t tmem = S.tmem_base;
    volatile int* abort_flag = &S.abort_flag;
    auto weight = [&](int t, int s) {
        if (s < kTable) return S.weight[t][s];
        const float l = lse_part[S.first[t] + s];
        return S.lse[t] == -INFINITY ? 0.f : expf(l - S.lse[t]);
    };
    const int group = threadIdx.x >> 6;
    const uint32_t leader = elect_one();
    for (int half = 0; half < 2; ++half) {
        // ---- merge of the half's columns ----
        const int col4 = 64 * half + (threadIdx.x & 63), to4 = threadIdx.x & 63;
        // the operand boxes are free once the first half's product has read them
        auto boxes_free = [&]() {
            if (half == 1 && !spin_warp(smem_u32(&S.done[0]), 0, abort_flag)) *abort_flag = 1;
        };
        if (n <= kGroups) {
            // few rows: each row's splits are shared out over kGroups / (n rounded up to a power of two)
            // groups, which add up through shared memory
            const int np = n <= 1 ? 1 : 1 << (32 - __clz(n - 1));
            const int per = kGroups / np, t = group / per, part = group % per;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            const int cnt = t < n ? S.count[t] : 0;
            for (int s = part; s < cnt; s += 4 * per) {
                float4 v[4];
                float w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int x = s + k * per;
                    w[k] = x < cnt ? weight(t, x) : 0.f;
                    v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (w[k] != 0.f) v[k] = load_state<BF16>(o_part, S.first[t] + x, col4);   // (an empty state may hold anything)
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) fma4(sum, w[k], v[k]);
            }
            S.part[group][to4] = sum;
            __syncthreads();
            if (part == 0 && t < n) {
                for (int g = 1; g < per; ++g) fma4(sum, 1.f, S.part[group + g][to4]);
                boxes_free();
                put(sHi, sLo, t, to4, sum);
            }
        } else {
            // four rows of the group at a time, two splits of each in flight
            for (int r0 = group; r0 < n; r0 += 4 * kGroups) {
                float4 sum[4];
                int most = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sum[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                    const int t = r0 + j * kGroups;
                    if (t < n) most = max(most, S.count[t]);
                }
                for (int s = 0; s < most; s += 2) {
                    float4 v[4][2];
                    float w[4][2];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int t = r0 + j * kGroups;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            w[j][k] = t < n && s + k < S.count[t] ? weight(t, s + k) : 0.f;
                            v[j][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (w[j][k] != 0.f) v[j][k] = load_state<BF16>(o_part, S.first[t] + s + k, col4);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int k = 0; k < 2; ++k) fma4(sum[j], w[j][k], v[j][k]);
                }
                if (r0 == group) boxes_free();
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r0 + j * kGroups < n) put(sHi, sLo, r0 + j * kGroups, to4, sum[j]);
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        // ---- D[v][token] of the half, box by box of 64 columns (rows past n are not written back) ----
        if (warp == 0) {
            constexpr uint32_t id = idesc_bf16(kLatV, kTok, 0);
            if (!spin_warp_drain(smem_u32(&S.w_full[half]), 0, abort_flag)) {
                if (lane == 0) {
                    if (a.err) set_error(a.err, ERR_TIMEOUT | SITE_FULL_WAIT);
                    *abort_flag = 1;
                }
            } else {
                tc_fence_after();
                const uint64_t wd0 = desc_sw128(smem_u32(sW + half * (kBoxes / 2) * kWBox), 16, 1024);
                const uint64_t hd0 = desc_sw128(smem_u32(sHi), 16, 1024), ld0 = desc_sw128(smem_u32(sLo), 16, 1024);
#pragma unroll
                for (int j = 0; j < kBoxes / 2; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint64_t wd = wd0 + (uint64_t)((j * kWBox + k * 32) >> 4), step = (uint64_t)((j * kOBox + k * 32) >> 4);
                        if (j + k == 0 && half == 0) mma_f16_if<0>(tmem, wd, hd0 + step, id, leader);
                        else mma_f16_if<1>(tmem, wd, hd0 + step, id, leader);
                        mma_f16_if<1>(tmem, wd, ld0 + step, id, leader);
                    }
            }
            __syncwarp();
            mma_commit_if(smem_u32(&S.done[half]), leader);
        }
        __syncwarp();
    }
    __syncwarp();
    if (warp < 8) {
        // warps 0..3 the first 32 tokens, 4..7 the others; a thread per value column
        const int c0 = (warp >> 2) * 32, quad = warp & 3;
        if (spin_warp(smem_u32(&S.done[1]), 0, abort_flag)) {
            tc_fence_after();
            uint32_t d[32];
            SKV_LD32(tmem + ((uint32_t)(quad * 32) << 16) + c0, d);
            tc_wait_ld();
            __nv_bfloat16* out = (__nv_bfloat16*)a.out + ((size_t)(t0 + c0) * a.heads + head) * kLatV + 32 * quad + lane;
            if (!*abort_flag) {
#pragma unroll
                for (int t = 0; t < 32; ++t)
                    if (c0 + t < n) out[(size_t)t * a.heads * kLatV] = __float2bfloat16_rn(__uint_as_float(d[t]));
            }
        } else if (lane == 0 && a.err) {
            set_error(a.err, ERR_TIMEOUT | SITE_DRAIN);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTok) : "memory");
}

}  // namespace

cudaError_t launch_latent_project(const LatentArgs& a, const void* o_part, int part_bf16, const float* lse_part,
                                  const int32_t* indptr, cudaStream_t s) {
    if (a.total_q <= 0) return cudaSuccess;
    auto enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    CUtensorMap mw;
    cuuint64_t dims[2] = {(cuuint64_t)kLatC, (cuuint64_t)a.heads * kLatW};
    cuuint64_t strides[1] = {(cuuint64_t)kLatC * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)kLatV}, es[2] = {1, 1};
    if (enc(&mw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(a.w), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> allowed[2];
    const void* kernel = part_bf16 ? (const void*)latent_project_kernel<true> : (const void*)latent_project_kernel<false>;
    cudaError_t e = allow_smem(kernel, kSmemBytes, allowed[part_bf16 ? 1 : 0]);
    if (e != cudaSuccess) return e;
    const int ctas = a.heads * ((a.total_q + kTok - 1) / kTok);
    ProfileScope ps(SPLITKV_KERNEL_LATENT_PROJECT, s);
    if (part_bf16) latent_project_kernel<true><<<ctas, kThreads, kSmemBytes, s>>>(mw, a, o_part, lse_part, indptr);
    else latent_project_kernel<false><<<ctas, kThreads, kSmemBytes, s>>>(mw, a, o_part, lse_part, indptr);
    return cudaGetLastError();
}

}  // namespace skv
