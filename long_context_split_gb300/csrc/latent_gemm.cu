// The per-head matrix products of latent attention on tcgen05 tensor cores, and
// the copy of the batch's latent rows that the expanded form starts from.
//
// With a head's weights W = (W_uk; W_uv), 256 rows of 512 (SPLASH Section 2
// Eq. 1 writes them as the up-projections of the latent c):
//   expand   k = c W_uk^T, v = c W_uv^T      M = cached tokens, K = 512, N = 256
//   absorb   q_lat = q_nope W_uk             M = query tokens,  K = 128, N = 512
// One kernel body: tiles of 128 rows by N columns of one head, a TMA producer
// warp, an MMA thread, and four epilogue warps that empty one accumulator while
// the other fills (tensor memory holds two).  Both operands are staged in
// 64-column boxes with the 128-byte swizzle; absorb's W_uk is read as stored
// (latent columns innermost), an MN-major operand, so no transposed copy of the
// weights is kept.  Results are rounded once to bf16 (expanded values to f16,
// which has three more significant bits: they meet the probabilities in an f16
// product) and leave through shared memory by TMA stores of 32 rows x 64
// columns, one epilogue warp's part each, which clip the rows past the tensor.
//
// What bounds them: absorb moves 16.8 MB of weights for 128 heads and few query
// rows (bytes); expand is 2 * 512 * 256 operations per token and head (tensor cores).
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
constexpr int kABytes = kM * 128;                // 128 rows x 64 columns

enum Mode { kExpand, kAbsorb };

template <int MODE>
struct Cfg {
    static constexpr int N = 256;
    static constexpr int K = MODE == kAbsorb ? 128 : 512;
    static constexpr int KB = K / 64;                        // k-blocks
    static constexpr int B_BYTES = N * 128;                  // N x 64 elements
    static constexpr int STAGE = kABytes + B_BYTES;
    static constexpr int NS = 3;
    static constexpr int BOX = 32 * 128;                     // one warp's 32 rows x 64 columns
    static constexpr int OUT_BYTES = kEpiWarps * 2 * BOX;    // two boxes per warp
    static constexpr int TMEM = 2 * N;
    static constexpr int TILES_PER_HEAD = MODE == kAbsorb ? 2 : 1;
};

template <int NS>
struct Bars {
    unsigned long long full[NS], empty[NS];
    unsigned long long acc_full[2], acc_empty[2];
    unsigned long long drain;
    uint32_t tmem_base;
    int abort_flag;
};

template <int MODE>
constexpr size_t smem_bytes() {
    using C = Cfg<MODE>;
    return 1024 + (size_t)C::NS * C::STAGE + C::OUT_BYTES + sizeof(Bars<C::NS>);
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"((uint64_t)map), "r"(x),
                 "r"(y), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void store_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// tile index -> (row tile, head, column half); heads innermost: tiles that run together share
// rows of A, and the weights (33.5 MB for 128 heads) stay in L2
struct Tile {
    int m0, h, half;
};
template <int MODE>
__device__ __forceinline__ Tile tile_of(int t, int heads) {
    using C = Cfg<MODE>;
    Tile x;
    const int per = heads * C::TILES_PER_HEAD;
    x.m0 = (t / per) * kM;
    const int r = t % per;
    x.h = r / C::TILES_PER_HEAD;
    x.half = r % C::TILES_PER_HEAD;
    return x;
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
latent_gemm_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                   const __grid_constant__ CUtensorMap mo, const __grid_constant__ CUtensorMap mo2, LatentArgs a,
                   void* q_abs, int num_tiles) {
    using C = Cfg<MODE>;
    constexpr int NS = C::NS;
    static_assert(smem_bytes<MODE>() <= 232448, "shared memory budget");
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char* sStage = smem;
    unsigned char* sOut = smem + NS * C::STAGE;
    Bars<NS>& B = *(Bars<NS>*)(sOut + C::OUT_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&B.full[s]), 1);
            mbar_init(smem_u32(&B.empty[s]), 1);
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
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B.tmem_base)),
                     "r"(C::TMEM)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B.tmem_base;
    volatile int* abort_flag = &B.abort_flag;
    auto give_up = [&](int site) {
        if (!*abort_flag) {
            if (a.err) set_error(a.err, ERR_TIMEOUT | site);
            *abort_flag = 1;
        }
    };

    if (warp == 0) {
        // ===================== TMA producer (lane 0) =====================
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = a.inject != 1;   // (test hook: load nothing)
            for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
                const Tile x = tile_of<MODE>(t, a.heads);
                for (int kb = 0; kb < C::KB; ++kb, ++it) {
                    const int s = (int)(it % NS);
                    if (!wait_bar(smem_u32(&B.empty[s]), ((it / NS) & 1) ^ 1, abort_flag, true)) {
                        give_up(SITE_EMPTY_WAIT);
                        ok = false;
                        break;
                    }
                    const uint32_t full = smem_u32(&B.full[s]);
                    const uint32_t sa = smem_u32(sStage + s * C::STAGE), sb = sa + kABytes;
                    mbar_expect_tx(full, C::STAGE);
                    if (MODE == kExpand) {
                        tma_2d(sa, &ma, 64 * kb, x.m0, full);
                        tma_2d(sb, &mb, 64 * kb, x.h * kLatW, full);
                    } else {
                        // 64 key rows of W_uk by 256 latent columns: four boxes, columns innermost
                        tma_2d(sa, &ma, x.h * kLatQ + 64 * kb, x.m0, full);
                        for (int j = 0; j < 4; ++j)
                            tma_2d(sb + j * 8192, &mb, x.half * 256 + 64 * j, x.h * kLatW + 64 * kb, full);
                    }
                }
            }
            // no copy may still be landing when the CTA leaves
            for (uint32_t k = 0; k < (uint32_t)NS && k < it; ++k) {
                const uint32_t last = it - 1 - k;
                if (!wait_bar(smem_u32(&B.full[last % NS]), (last / NS) & 1, abort_flag, false) && a.err)
                    set_error(a.err, ERR_TIMEOUT | SITE_DRAIN);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ===================== MMA issuer (lane 0) =====================
        if (lane == 0) {
            constexpr uint32_t id = idesc_bf16(kM, C::N, MODE == kAbsorb ? 1 : 0);
            uint32_t it = 0, n = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x, ++n) {
                const uint32_t buf = n & 1;
                if (!wait_bar(smem_u32(&B.acc_empty[buf]), ((n >> 1) & 1) ^ 1, abort_flag, true)) {
                    give_up(SITE_EMPTY_WAIT);
                    break;
                }
                tc_fence_after();
                for (int kb = 0; kb < C::KB; ++kb, ++it) {
                    const int s = (int)(it % NS);
                    if (!wait_bar(smem_u32(&B.full[s]), (it / NS) & 1, abort_flag, true)) {
                        give_up(SITE_FULL_WAIT);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(sStage + s * C::STAGE), sb = sa + kABytes;
                    const uint64_t ad = desc_sw128(sa, 16, 1024);
                    const uint64_t bd = MODE == kAbsorb ? desc_sw128(sb, 8192, 1024) : desc_sw128(sb, 16, 1024);
                    constexpr int kStepB = MODE == kAbsorb ? 2048 : 32;   // 16 k: 16 rows of 128 B, or 32 B of a row
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f16(tmem + buf * C::N, ad + (uint64_t)((k * 32) >> 4), bd + (uint64_t)((k * kStepB) >> 4), id,
                                (kb | k) != 0 ? 1u : 0u);
                    mma_commit(smem_u32(&B.empty[s]));
                }
                if (ok) mma_commit(smem_u32(&B.acc_full[buf]));
            }
            mma_commit(smem_u32(&B.drain));
            if (!wait_bar(smem_u32(&B.drain), 0, abort_flag, false) && a.err) set_error(a.err, ERR_TIMEOUT | SITE_DRAIN);
        }
        __syncwarp();
    } else {
        // ===================== epilogue: warp = 32 rows of the tile =====================
        const int quad = warp & 3;                                   // tensor-memory lane quadrant
        unsigned char* stage = sOut + quad * 2 * C::BOX;
        const int row = lane;
        bool ok = true;
        float vmax = 0.f;
        uint32_t n = 0, boxes = 0;
        for (int t = blockIdx.x; t < num_tiles; t += gridDim.x, ++n) {
            const uint32_t buf = n & 1;
            const Tile x = tile_of<MODE>(t, a.heads);
            const int y = x.m0 + 32 * quad;
            if (MODE == kAbsorb && x.half == 0) {
                // the rotary columns pass through: 128 bytes of each of the warp's rows
                // (eight loads in flight per lane: one after the other they cost 6 us a call)
                uint4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int r = y + 4 * k + (lane >> 3);
                    if (r < a.total_q)
                        v[k] = *((const uint4*)((const __nv_bfloat16*)a.q + (size_t)r * a.q_stride + x.h * kLatQ + kLatNope) + (lane & 7));
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int r = y + 4 * k + (lane >> 3);
                    if (r < a.total_q)
                        *((uint4*)((__nv_bfloat16*)q_abs + ((size_t)r * a.heads + x.h) * kLatRow + kLatC) + (lane & 7)) = v[k];
                }
            }
            if (!warp_wait(smem_u32(&B.acc_full[buf]), (n >> 1) & 1, abort_flag, lane)) {
                give_up(SITE_FULL_WAIT);
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + buf * C::N;
#pragma unroll 1
            for (int c = 0; c < C::N; c += 64, ++boxes) {
                uint32_t v[64];
                SKV_LD32(acc + c, v);
                SKV_LD32(acc + c + 32, (v + 32));
                tc_wait_ld();
                if (c + 64 == C::N) {      // the accumulator is read: the next tile may overwrite it
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&B.acc_empty[buf]));
                }
                // the box two stores back has been read out of its half of the staging buffer
                if (lane == 0) store_wait_read<1>();
                __syncwarp();
                unsigned char* box = stage + (boxes & 1) * C::BOX;
                const bool f16 = MODE == kExpand && c >= kLatNope;
#pragma unroll
                for (int k = 0; k < 8; ++k) {                      // 16-byte piece k of the row's 128 bytes
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float lo = __uint_as_float(v[8 * k + 2 * e]), hi = __uint_as_float(v[8 * k + 2 * e + 1]);
                        if (f16) {
                            const __half2 p = __floats2half2_rn(lo, hi);
                            w[e] = *reinterpret_cast<const uint32_t*>(&p);
                            const float m = fmaxf(fabsf(lo), fabsf(hi));
                            if (m < INFINITY) vmax = fmaxf(vmax, m);
                        } else {
                            const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
                            w[e] = *reinterpret_cast<const uint32_t*>(&p);
                        }
                    }
                    *(uint4*)(box + row * 128 + ((k ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    const uint32_t src = smem_u32(box);
                    if (MODE == kExpand) {
                        const int yo = x.h * a.num_blocks * kLatPad + y;
                        if (f16) tma_store_2d(&mo2, src, c - kLatNope, yo);
                        else tma_store_2d(&mo, src, c, yo);
                    } else if (y < a.total_q) {
                        tma_store_2d(&mo, src, x.h * kLatRow + x.half * 256 + c, y);
                    }
                    store_commit();
                }
            }
        }
        (void)ok;
        if (lane == 0) store_wait_all();   // the staging buffer outlives its stores
        // finite values above the f16 range became infinities
        if (MODE == kExpand && vmax > 65504.f && a.err) set_error(a.err, ERR_DEVICE_CHECK | SITE_VALUE_RANGE);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM) : "memory");
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
cudaError_t make_map(CUtensorMap* m, const void* base, long long cols, long long rows, long long stride_elems, int box_cols,
                     int box_rows, CUtensorMapDataType dtype = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
    auto enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)stride_elems * 2};
    cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    CUresult r = enc(m, dtype, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int MODE>
cudaError_t launch_gemm(const LatentArgs& a, const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mo,
                        const CUtensorMap& mo2, void* q_abs, int m_tiles, int kernel, cudaStream_t s) {
    using C = Cfg<MODE>;
    constexpr size_t smem = smem_bytes<MODE>();
    static std::once_flag once;
    static cudaError_t attr_err = cudaSuccess;
    std::call_once(once, [&]() {
        attr_err = cudaFuncSetAttribute(latent_gemm_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (attr_err != cudaSuccess) return attr_err;
    int dev = 0, sms = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const int tiles = m_tiles * a.heads * C::TILES_PER_HEAD;
    {
        ProfileScope ps(kernel, s);
        latent_gemm_kernel<MODE><<<std::min(sms, tiles), kThreads, smem, s>>>(ma, mb, mo, mo2, a, q_abs, tiles);
    }
    return cudaGetLastError();
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
    CUtensorMap ma, mb, mk, mv;
    cudaError_t e;
    if ((e = make_map(&ma, a.rows, kLatRow, rows, kLatRow, 64, kM)) != cudaSuccess) return e;
    if ((e = make_map(&mb, a.w, kLatC, (long long)a.heads * kLatW, kLatC, 64, kLatW)) != cudaSuccess) return e;
    if ((e = make_map(&mk, a.keys, kLatNope, a.heads * rows, kLatNope, 64, 32)) != cudaSuccess) return e;
    if ((e = make_map(&mv, a.vals, kLatV, a.heads * rows, kLatV, 64, 32, CU_TENSOR_MAP_DATA_TYPE_FLOAT16)) != cudaSuccess)
        return e;
    return launch_gemm<kExpand>(a, ma, mb, mk, mv, nullptr, a.num_blocks, SPLITKV_KERNEL_LATENT_EXPAND, s);
}

cudaError_t launch_latent_absorb(const LatentArgs& a, void* q_abs, cudaStream_t s) {
    if (a.total_q <= 0) return cudaSuccess;
    CUtensorMap ma, mb, mo;
    cudaError_t e;
    if ((e = make_map(&ma, a.q, (long long)a.heads * kLatQ, a.total_q, a.q_stride, 64, kM)) != cudaSuccess) return e;
    if ((e = make_map(&mb, a.w, kLatC, (long long)a.heads * kLatW, kLatC, 64, 64)) != cudaSuccess) return e;
    if ((e = make_map(&mo, q_abs, (long long)a.heads * kLatRow, a.total_q, (long long)a.heads * kLatRow, 64, 32)) != cudaSuccess)
        return e;
    return launch_gemm<kAbsorb>(a, ma, mb, mo, mo, q_abs, (a.total_q + kM - 1) / kM, SPLITKV_KERNEL_LATENT_ABSORB, s);
}

}  // namespace skv
