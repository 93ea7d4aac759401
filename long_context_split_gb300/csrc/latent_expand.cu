// The expanded form's keys and values: a bf16 copy of the batch's latent rows, and
// from it k = c W_uk^T (bf16) and v = c W_uv^T (f16) of every head, on tcgen05 tensor
// cores.
//
// What bounds the product: 2 * 512 * 256 operations per token and head.  Streaming both
// operands of 128 x 256 tiles from L2 takes 384 KB a tile, and L2 gave 13 TB/s of it at
// 57 % of the tensor rate (218 us for 7.3k tokens and 128 heads).  So
// a CTA keeps its 128 latent rows (128 KB) in shared memory while it walks over
// heads, and a cluster of two CTAs (two row tiles, the same heads) shares each 64-column
// box of the head's weights: each loads half of its 256 rows and multicasts it to both
// (128 KB a tile and CTA from L2; XX us).
//
// Roles: warp 0 TMA producer, warp 1 MMA thread (M = 128 rows, N = 256 weight rows,
// K = 512 in eight boxes; two accumulators in tensor memory), warps 2..5 the epilogue,
// which rounds the accumulator once and stores 32 bytes of a row per thread and
// instruction while the next tile accumulates.  Values get f16's three more bits: they meet the
// probabilities in an f16 product.
//
// A box may be overwritten once both CTAs' products have read it: each CTA's MMA
// thread commits to both CTAs' barriers, and neither CTA leaves before the other.
// Waits are bounded; on expiry a CTA records the error, and its partner's waits run out too.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "latent.h"
#include "tc_common.cuh"

namespace skv {
namespace {

constexpr int kM = 128;
constexpr int kEpiWarps = 4;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kCluster = 2;
constexpr int kBoxes = kLatC / 64;
constexpr int kABox = kM * 128;                    // 128 latent rows x 64 columns
constexpr int kBBox = kLatW * 128;                 // a head's 256 weight rows x 64 columns
constexpr int NS = 3;                              // weight boxes in shared memory
constexpr int kTmem = 2 * kLatW;

struct Bars {
    unsigned long long a_full, a_empty;
    unsigned long long b_full[NS], b_empty[NS];
    unsigned long long acc_full[2], acc_empty[2];
    unsigned long long drain;
    uint32_t tmem_base;
    int abort_flag;
};

constexpr size_t kSmemBytes = 1024 + (size_t)kBoxes * kABox + (size_t)NS * kBBox + sizeof(Bars);
static_assert(kSmemBytes <= 232448, "shared memory budget");

__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// to the same address in both CTAs of the cluster, each counting the bytes on its own barrier
__device__ __forceinline__ void tma_2d_both(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.multicast::cluster [%0], [%1, {%2, %3}], "
        "[%4], %5;" ::"r"(dst),
        "l"((uint64_t)map), "r"(x), "r"(y), "r"(bar), "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ void commit_both(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Tiles (row pair, head), heads innermost; cluster c takes [c n / clusters, (c + 1) n / clusters).
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
latent_expand_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb, LatentArgs a,
                     int num_tiles) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sA = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char* sB = sA + kBoxes * kABox;
    Bars& B = *(Bars*)(sB + NS * kBBox);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank(), cluster = blockIdx.x / kCluster, clusters = gridDim.x / kCluster;
    const int t0 = (int)((long long)cluster * num_tiles / clusters), t1 = (int)((long long)(cluster + 1) * num_tiles / clusters);
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&B.a_full), 1);
        mbar_init(smem_u32(&B.a_empty), 1);
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&B.b_full[s]), 1);
            mbar_init(smem_u32(&B.b_empty[s]), kCluster);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&B.acc_full[b]), 1);
            mbar_init(smem_u32(&B.acc_empty[b]), kEpiWarps);
        }
        mbar_init(smem_u32(&B.drain), 1);
        B.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B.tmem_base)), "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();          // both CTAs' barriers are initialised before either's copies or commits reach them
    tc_fence_after();
    const uint32_t tmem = B.tmem_base;
    volatile int* abort_flag = &B.abort_flag;
    auto give_up = [&](int site) {
        if (!*abort_flag) {
            set_error(a.err, ERR_TIMEOUT | site);
            *abort_flag = 1;
        }
    };

    if (warp == 0) {
        // ===================== TMA producer (lane 0) =====================
        if (lane == 0) {
            uint32_t it = 0, an = 0;
            int pair = -1;
            bool ok = a.inject != 1;   // (test hook: load nothing)
            for (int t = t0; t < t1 && ok; ++t) {
                if (t / a.heads != pair) {
                    pair = t / a.heads;
                    if (!spin_bar(smem_u32(&B.a_empty), (an & 1) ^ 1, abort_flag, true)) { give_up(SITE_EMPTY_WAIT); break; }
                    // (an odd last row tile: its partner's rows are the zero fill past the tensor)
                    mbar_expect_tx(smem_u32(&B.a_full), kBoxes * kABox);
                    for (int j = 0; j < kBoxes; ++j)
                        tma_2d(smem_u32(sA + j * kABox), &ma, 64 * j, (pair * kCluster + rank) * kM, smem_u32(&B.a_full));
                    ++an;
                }
                const int y = (t % a.heads) * kLatW + rank * (kLatW / kCluster);
                for (int j = 0; j < kBoxes; ++j, ++it) {
                    const int s = (int)(it % NS);
                    if (!spin_bar(smem_u32(&B.b_empty[s]), ((it / NS) & 1) ^ 1, abort_flag, true)) {
                        give_up(SITE_EMPTY_WAIT);
                        ok = false;
                        break;
                    }
                    mbar_expect_tx(smem_u32(&B.b_full[s]), kBBox);
                    tma_2d_both(smem_u32(sB + s * kBBox + rank * (kBBox / kCluster)), &mb, 64 * j, y, smem_u32(&B.b_full[s]));
                }
            }
            // no copy may still be landing when the CTA leaves
            bool landed = true;
            for (uint32_t k = 0; k < (uint32_t)NS && k < it; ++k) {
                const uint32_t last = it - 1 - k;
                landed = spin_bar(smem_u32(&B.b_full[last % NS]), (last / NS) & 1, abort_flag, false) && landed;
            }
            if (an) landed = spin_bar(smem_u32(&B.a_full), (an - 1) & 1, abort_flag, false) && landed;
            if (!landed) set_error(a.err, ERR_TIMEOUT | SITE_DRAIN);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ===================== MMA issuer (lane 0) =====================
        if (lane == 0) {
            constexpr uint32_t id = idesc_bf16(kM, kLatW, 0);
            uint32_t it = 0, an = 0, n = 0;
            int pair = -1;
            bool ok = true;
            for (int t = t0; t < t1 && ok; ++t, ++n) {
                const uint32_t buf = n & 1, acc = tmem + buf * kLatW;
                if (t / a.heads != pair) {
                    pair = t / a.heads;
                    if (!spin_bar(smem_u32(&B.a_full), an & 1, abort_flag, true)) { give_up(SITE_FULL_WAIT); break; }
                    ++an;
                }
                if (!spin_bar(smem_u32(&B.acc_empty[buf]), ((n >> 1) & 1) ^ 1, abort_flag, true)) { give_up(SITE_EMPTY_WAIT); break; }
                for (int j = 0; j < kBoxes; ++j, ++it) {
                    const int s = (int)(it % NS);
                    if (!spin_bar(smem_u32(&B.b_full[s]), (it / NS) & 1, abort_flag, true)) {
                        give_up(SITE_FULL_WAIT);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = desc_sw128(smem_u32(sA + j * kABox), 16, 1024);
                    const uint64_t bd = desc_sw128(smem_u32(sB + s * kBBox), 16, 1024);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f16(acc, ad + (uint64_t)((k * 32) >> 4), bd + (uint64_t)((k * 32) >> 4), id, (j | k) != 0 ? 1u : 0u);
                    commit_both(smem_u32(&B.b_empty[s]));
                }
                if (!ok) break;
                mma_commit(smem_u32(&B.acc_full[buf]));
                if (t + 1 < t1 && (t + 1) / a.heads != pair) mma_commit(smem_u32(&B.a_empty));
            }
            mma_commit(smem_u32(&B.drain));
            if (!spin_bar(smem_u32(&B.drain), 0, abort_flag, false)) set_error(a.err, ERR_TIMEOUT | SITE_DRAIN);
        }
        __syncwarp();
    } else {
        // ===================== epilogue: a thread per row of the tile =====================
        const int quad = warp & 3;
        const size_t rows = (size_t)a.num_blocks * kLatPad;
        float vmax = 0.f;
        uint32_t n = 0;
        for (int t = t0; t < t1; ++t, ++n) {
            const uint32_t buf = n & 1;
            const size_t row = (size_t)(t / a.heads * kCluster + rank) * kM + 32 * quad + lane;
            const size_t at = ((size_t)(t % a.heads) * rows + row) * kLatNope;
            if (!spin_warp(smem_u32(&B.acc_full[buf]), (n >> 1) & 1, abort_flag)) {
                give_up(SITE_FULL_WAIT);
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + buf * kLatW;
#pragma unroll 1
            for (int c = 0; c < kLatW; c += 32) {
                uint32_t v[32], w[16];
                SKV_LD32(acc + c, v);
                tc_wait_ld();
                if (c + 32 == kLatW) {      // the accumulator is read: the tile after next may overwrite it
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&B.acc_empty[buf]));
                }
                if (c < kLatNope) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                        w[e] = *reinterpret_cast<const uint32_t*>(&p);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float lo = __uint_as_float(v[2 * e]), hi = __uint_as_float(v[2 * e + 1]);
                        const __half2 p = __floats2half2_rn(lo, hi);
                        w[e] = *reinterpret_cast<const uint32_t*>(&p);
                        const float m = fmaxf(fabsf(lo), fabsf(hi));
                        if (m < INFINITY) vmax = fmaxf(vmax, m);
                    }
                }
                if (row < rows) {
                    char* to = c < kLatNope ? (char*)a.keys + (at + c) * 2 : (char*)a.vals + (at + c - kLatNope) * 2;
                    store32(to, w);
                    store32(to + 32, w + 8);
                }
            }
        }
        // finite values above the f16 range became infinities
        if (vmax > 65504.f) set_error(a.err, ERR_DEVICE_CHECK | SITE_VALUE_RANGE);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
    cluster_sync();          // the partner's copies and commits into this CTA have arrived
}

// The batch's latent rows as bf16, request after request, each padded with zero rows to a
// multiple of 128: E4M3 codes are exact in bf16 (their scale is folded into the softmax and the
// output), and a row past a request's last token is zero whatever its page holds.
template <bool FP8>
__global__ void __launch_bounds__(256) latent_rows_kernel(LatentArgs a) {
    constexpr int kRowsPerCta = 16;
    constexpr int kPieces = kLatRow / 8;                  // 16-byte pieces of a copied row
    __shared__ long long src_row[kRowsPerCta];
    const int row0 = blockIdx.x * kRowsPerCta;
    const LatentBlock blk = a.blocks[row0 / kLatPad];
    if (threadIdx.x < kRowsPerCta) {
        const int tok = blk.token + (row0 + threadIdx.x) % kLatPad;
        long long w = -1;
        if (tok < a.reqs[blk.b].seq_len) {
            const int page = a.page_table[(size_t)blk.b * a.max_pages + tok / a.page_size];
            if (page >= 0 && page < a.num_pages) w = (long long)page * a.page_size + tok % a.page_size;
            else set_error(a.err, ERR_DEVICE_CHECK | SITE_PAGE_RANGE);
        }
        src_row[threadIdx.x] = w;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kRowsPerCta * kPieces; i += 256) {
        const int r = i / kPieces, p = i % kPieces;
        const long long w = src_row[r];
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (w >= 0) {
            if (FP8) {
                const uint2 c = *((const uint2*)((const uint8_t*)a.cache + w * kLatRow) + p);
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t two = ((k < 2 ? c.x : c.y) >> (16 * (k & 1))) & 0xFFFFu;
                    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3)));
                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(f.x, f.y);
                    o[k] = *reinterpret_cast<const uint32_t*>(&b2);
                }
                v = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
                v = *((const uint4*)((const __nv_bfloat16*)a.cache + w * kLatRow) + p);
            }
        }
        *((uint4*)((__nv_bfloat16*)a.rows + (size_t)(row0 + r) * kLatRow) + p) = v;
    }
}

// ---------------------------------------------------------------- host
cudaError_t make_map(CUtensorMap* m, const void* base, long long cols, long long rows, int box_rows) {
    auto enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_latent_rows(const LatentArgs& a, cudaStream_t s) {
    if (a.num_blocks <= 0) return cudaSuccess;
    const int ctas = a.num_blocks * (kLatPad / 16);
    ProfileScope ps(SPLITKV_KERNEL_LATENT_ROWS, s);
    if (a.kv_fp8) latent_rows_kernel<true><<<ctas, 256, 0, s>>>(a);
    else latent_rows_kernel<false><<<ctas, 256, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_latent_expand(const LatentArgs& a, cudaStream_t s) {
    if (a.num_blocks <= 0) return cudaSuccess;
    const long long rows = (long long)a.num_blocks * kLatPad;
    CUtensorMap ma, mb;
    cudaError_t e;
    if ((e = make_map(&ma, a.rows, kLatRow, rows, kM)) != cudaSuccess) return e;
    if ((e = make_map(&mb, a.w, kLatC, (long long)a.heads * kLatW, kLatW / kCluster)) != cudaSuccess) return e;
    static std::once_flag once;
    static cudaError_t attr_err = cudaSuccess;
    std::call_once(once, [&]() {
        attr_err = cudaFuncSetAttribute(latent_expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    });
    if (attr_err != cudaSuccess) return attr_err;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int tiles = (a.num_blocks + kCluster - 1) / kCluster * a.heads;
    {
        ProfileScope ps(SPLITKV_KERNEL_LATENT_EXPAND, s);
        latent_expand_kernel<<<kCluster * std::max(1, std::min(sms / kCluster, tiles)), kThreads, kSmemBytes, s>>>(ma, mb, a, tiles);
    }
    return cudaGetLastError();
}

}  // namespace skv
