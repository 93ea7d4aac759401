// The start of absorbed latent attention: q_lat = q_nope W_uk per head (SPLASH
// Section 2 Eq. 1), the rotary columns passed through.
//
// What bounds it: bytes, 16.8 MB of weights for 128 heads and 1.5 KB of query and
// result per token and head; for few tokens the latency of one load, product and
// store.  So a CTA takes 128 tokens by 256 of a head's 512 latent columns with nothing
// to iterate over: all its operands (96 KB) are requested at once, two CTAs share an SM, and
// a single decoding token keeps 256 CTAs, the whole GPU, reading weights.
//
// M = 128 tokens, N = 256, K = 128 on tcgen05; W_uk is read as stored (latent columns
// innermost), an MN-major operand, so no transposed copy of the weights is kept.  The
// result is rounded once to bf16, the type that the attention kernel takes.
#include <algorithm>

#include "latent.h"
#include "tc_issue.cuh"

namespace skv {
namespace {

constexpr int kM = 128;
constexpr int kN = 256;
constexpr int kThreads = 128;
constexpr int kKB = kLatNope / 64;               // k-blocks of 64 query columns
constexpr int kABox = kM * 128;                  // 128 tokens x 64 query columns
constexpr int kBBox = 64 * 128;                  // 64 weight rows x 64 latent columns
constexpr int kBBytes = kN / 64 * kBBox;         // a k-block of the weights

struct Bars {
    unsigned long long full[kKB], done;
    uint32_t tmem_base;
    int abort_flag;
};

constexpr size_t kSmemBytes = 1024 + (size_t)kKB * (kABox + kBBytes) + sizeof(Bars);

__global__ void __launch_bounds__(kThreads, 2)
latent_absorb_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mw, LatentArgs a, void* q_abs) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sA = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char* sB = sA + kKB * kABox;
    Bars& B = *(Bars*)(sB + kKB * kBBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = 2 * a.heads;
    const int m0 = (int)(blockIdx.x / per) * kM, head = (int)(blockIdx.x % per) / 2, half = (int)(blockIdx.x % per) % 2;
    volatile int* abort_flag = &B.abort_flag;
    if (threadIdx.x == 0) {
        for (int k = 0; k < kKB; ++k) mbar_init(smem_u32(&B.full[k]), 1);
        mbar_init(smem_u32(&B.done), 1);
        B.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (a.inject != 1) {   // (test hook: load nothing)
            for (int k = 0; k < kKB; ++k) {
                const uint32_t full = smem_u32(&B.full[k]);
                mbar_expect_tx(full, kABox + kBBytes);
                for (int j = 0; j < kN / 64; ++j)
                    tma_2d(smem_u32(sB + k * kBBytes + j * kBBox), &mw, half * kN + 64 * j, head * kLatW + 64 * k, full);
                tma_2d(smem_u32(sA + k * kABox), &mq, head * kLatQ + 64 * k, m0, full);
            }
        }
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B.tmem_base)), "r"(kN)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B.tmem_base;
    if (warp == 0) {
        constexpr uint32_t id = idesc_bf16(kM, kN, 1);
        const uint32_t leader = elect_one();
        const uint64_t ad0 = desc_sw128(smem_u32(sA), 16, 1024), bd0 = desc_sw128(smem_u32(sB), kBBox, 1024);
#pragma unroll
        for (int k = 0; k < kKB; ++k) {
            if (!spin_warp_drain(smem_u32(&B.full[k]), 0, abort_flag)) {
                if (lane == 0) {
                    if (a.err) set_error(a.err, ERR_TIMEOUT | SITE_FULL_WAIT);
                    *abort_flag = 1;
                }
                __syncwarp();
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 4; ++j) {   // 16 k: 32 bytes of A's rows, 16 rows of B's boxes
                const uint64_t ad = ad0 + (uint64_t)((k * kABox + j * 32) >> 4), bd = bd0 + (uint64_t)((k * kBBytes + j * 2048) >> 4);
                if (k + j == 0) mma_f16_if<0>(tmem, ad, bd, id, leader);
                else mma_f16_if<1>(tmem, ad, bd, id, leader);
            }
        }
        mma_commit_if(smem_u32(&B.done), leader);
    }
    if (half == 0) {
        // under the product, the rotary columns pass through: 128 bytes of each token, eight loads in
        // flight per lane
        const int y = m0 + 32 * warp;
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = y + 4 * k + (lane >> 3);
            if (r < a.total_q)
                v[k] = *((const uint4*)((const __nv_bfloat16*)a.q + (size_t)r * a.q_stride + head * kLatQ + kLatNope) + (lane & 7));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = y + 4 * k + (lane >> 3);
            if (r < a.total_q)
                *((uint4*)((__nv_bfloat16*)q_abs + ((size_t)r * a.heads + head) * kLatRow + kLatC) + (lane & 7)) = v[k];
        }
    }
    __syncwarp();
    const int row = m0 + 32 * warp + lane;
    if (!spin_warp(smem_u32(&B.done), 0, abort_flag)) {
        if (lane == 0 && a.err) set_error(a.err, ERR_TIMEOUT | SITE_DRAIN);
    } else if (m0 + 32 * warp < a.total_q && !*abort_flag) {
        tc_fence_after();
        __nv_bfloat16* out = (__nv_bfloat16*)q_abs + ((size_t)row * a.heads + head) * kLatRow + half * kN;
#pragma unroll 2
        for (int c = 0; c < kN; c += 32) {
            uint32_t v[32];
            SKV_LD32(tmem + ((uint32_t)(warp * 32) << 16) + c, v);
            tc_wait_ld();
            if (row < a.total_q) {
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(v[k + 2 * e]), __uint_as_float(v[k + 2 * e + 1]));
                        w[e] = *reinterpret_cast<const uint32_t*>(&p);
                    }
                    *(uint4*)(out + c + k) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            __syncwarp();   // (the tensor-memory loads are warp-collective)
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kN) : "memory");
}

cudaError_t make_map(CUtensorMap* m, const void* base, long long cols, long long rows, long long stride_elems, int box_rows) {
    auto enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)stride_elems * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_latent_absorb(const LatentArgs& a, void* q_abs, cudaStream_t s) {
    if (a.total_q <= 0) return cudaSuccess;
    CUtensorMap mq, mw;
    cudaError_t e;
    if ((e = make_map(&mq, a.q, (long long)a.heads * kLatQ, a.total_q, a.q_stride, kM)) != cudaSuccess) return e;
    if ((e = make_map(&mw, a.w, kLatC, (long long)a.heads * kLatW, kLatC, 64)) != cudaSuccess) return e;
    static std::atomic<uint64_t> allowed{0};
    if ((e = allow_smem((const void*)latent_absorb_kernel, kSmemBytes, allowed)) != cudaSuccess) return e;
    const long long ctas = (long long)((a.total_q + kM - 1) / kM) * a.heads * 2;
    {
        ProfileScope ps(SPLITKV_KERNEL_LATENT_ABSORB, s);
        latent_absorb_kernel<<<(unsigned)ctas, kThreads, kSmemBytes, s>>>(mq, mw, a, q_abs);
    }
    return cudaGetLastError();
}

}  // namespace skv
