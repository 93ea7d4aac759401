// The expanded form's keys and values: a bf16 copy of the batch's latent rows, and
// from it k = c W_uk^T (bf16) and v = c W_uv^T (f16) of every head, on tcgen05 tensor
// cores.
//
// What bounds the product: 2 * 512 * 256 operations per token and head.  Streaming both
// operands of 128 x 256 tiles from L2 takes 384 KB a tile, and L2 gave 13 TB/s of it at
// 57 % of the tensor rate (218 us for 7.3k tokens and 128 heads).  So a CTA keeps its 128
// latent rows while it walks over heads, as the A operand in tensor memory (256 columns),
// and loads the weights alone (256 KB a head from L2).  The weights' ring holds a whole tile, so
// that the issuing warp's code is straight-line with constant slots: with one lane's loop over
// twelve slots, issue alone took 660 cycles a box for 256 of products.  7.3k tokens and 128 heads
// take 170 us, 1.45 PFLOP/s.
//
// Roles: warp 0 TMA producer, warp 1 MMA thread (M = 128 rows, N = 128: a head's keys or
// its values, K = 512 in eight boxes; two accumulators), warps 2..5 the epilogue, which
// rounds an accumulator once and stores whole lines of the attention's operand images while
// the next tile accumulates, and which brings a new row tile into tensor memory.  Values
// get f16's three more bits: they meet the probabilities in an f16 product.  f16's range is narrow (2^-14 to
// 65504 at full precision), so the values of 64 tokens and a head are stored times a power of two that brings the
// largest to 2^14: magnitudes down to 2^-28 of it keep 11 bits, and the attention divides the power out exactly.
// (Values below 2^-14 lost bits and those below 2^-25 were zero without it; it costs 163 -> 170 us, and the attention
// 1 %.  Reading the accumulator twice instead of keeping its 128 columns in registers: 184 us.)
//
// Waits are bounded; on expiry the CTA records the error and drains its copies and products.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "latent.h"
#include "tc_issue.cuh"

namespace skv {
namespace {

constexpr int kM = 128;
constexpr int kEpiWarps = 4;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kBoxes = kLatC / 64;
constexpr int kN = 128;                            // weight rows of a tile: W_uk's or W_uv's of a head
constexpr int kABox = kM * 128;                    // 128 latent rows x 64 columns
constexpr int kBBox = kN * 128;                    // 128 weight rows x 64 columns
constexpr int NS = kBoxes;                         // weight boxes in shared memory: a tile's, so that slots are constants
constexpr int kStages = 4;                         // row boxes in flight on their way to tensor memory
constexpr int kColA = 0, kColAcc = 256;            // tensor memory: the rows (256 columns), two accumulators
constexpr int kTmem = 512;

struct Bars {
    unsigned long long as_full[kStages], as_empty[kStages];   // staging of the rows on their way to tensor memory
    unsigned long long a_ready;
    unsigned long long b_full[NS], b_empty[NS];
    unsigned long long acc_full[2], acc_empty[2];
    unsigned long long unit_max[2];            // both warps of a unit have written its maximum
    unsigned long long drain;
    uint32_t tmem_base;
    int abort_flag;
    float warp_max[2][kEpiWarps];              // largest value magnitude of a warp's 32 rows, tiles in turn
};

constexpr size_t kSmemBytes = 1024 + kStages * (size_t)kABox + (size_t)NS * kBBox + sizeof(Bars);
static_assert(kSmemBytes <= 232448, "shared memory budget");

// 16 packed columns, their 16-byte halves exchanged when `swap`
__device__ __forceinline__ void store32(void* p, const uint32_t* w, int swap) {
    uint32_t x[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[k] = swap ? w[4 + k] : w[k];
        x[4 + k] = swap ? w[k] : w[4 + k];
    }
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
                 "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

// Tiles (128 rows, head of the group, keys or values); CTA c takes [c n / ctas, (c + 1) n / ctas).
struct Tile {
    int rows, head, side;
};
__device__ __forceinline__ Tile tile_of(int t, int heads) {
    Tile x;
    x.rows = t / (2 * heads);
    x.head = t % (2 * heads) / 2;
    x.side = t % 2;
    return x;
}

__global__ void __launch_bounds__(kThreads, 1)
latent_expand_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb, LatentArgs a,
                     int num_tiles) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* sA = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char* sB = sA + kStages * kABox;
    Bars& B = *(Bars*)(sB + NS * kBBox);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = (int)((long long)blockIdx.x * num_tiles / gridDim.x), t1 = (int)((blockIdx.x + 1LL) * num_tiles / gridDim.x);
    if (threadIdx.x == 0) {
        for (int k = 0; k < kStages; ++k) {
            mbar_init(smem_u32(&B.as_full[k]), 1);
            mbar_init(smem_u32(&B.as_empty[k]), kEpiWarps);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(smem_u32(&B.acc_full[k]), 1);
            mbar_init(smem_u32(&B.acc_empty[k]), kEpiWarps);
            mbar_init(smem_u32(&B.unit_max[k]), 2);
        }
        mbar_init(smem_u32(&B.a_ready), kEpiWarps);
        for (int s = 0; s < NS; ++s) {
            mbar_init(smem_u32(&B.b_full[s]), 1);
            mbar_init(smem_u32(&B.b_empty[s]), 1);
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
            uint32_t it = 0, an = 0;   // weight boxes, row boxes so far
            int rows = -1;
            bool ok = a.inject != 1;   // (test hook: load nothing)
            for (int t = t0; t < t1 && ok; ++t) {
                const Tile x = tile_of(t, a.group);
                if (x.rows != rows) {
                    rows = x.rows;
                    for (int j = 0; j < kBoxes && ok; ++j, ++an) {
                        ok = spin_bar(smem_u32(&B.as_empty[an % kStages]), ((an / kStages) & 1) ^ 1, abort_flag, true);
                        if (!ok) break;
                        mbar_expect_tx(smem_u32(&B.as_full[an % kStages]), kABox);
                        tma_2d(smem_u32(sA + an % kStages * kABox), &ma, 64 * j, rows * kM,
                               smem_u32(&B.as_full[an % kStages]));
                    }
                }
                const int y = (a.head0 + x.head) * kLatW + x.side * kN;
                for (int j = 0; j < kBoxes && ok; ++j, ++it) {
                    const int s = (int)(it % NS);
                    ok = spin_bar(smem_u32(&B.b_empty[s]), ((it / NS) & 1) ^ 1, abort_flag, true);
                    if (!ok) break;
                    mbar_expect_tx(smem_u32(&B.b_full[s]), kBBox);
                    tma_2d(smem_u32(sB + s * kBBox), &mb, 64 * j, y, smem_u32(&B.b_full[s]));
                }
                if (!ok) give_up(SITE_EMPTY_WAIT);
            }
            // no copy may still be on its way when the CTA leaves
            bool landed = true;
            for (uint32_t k = 0; k < (uint32_t)NS && k < it; ++k) {
                const uint32_t last = it - 1 - k;
                landed = spin_bar(smem_u32(&B.b_full[last % NS]), (last / NS) & 1, abort_flag, false) && landed;
            }
            for (uint32_t k = 0; k < (uint32_t)kStages && k < an; ++k) {
                const uint32_t last = an - 1 - k;
                landed = spin_bar(smem_u32(&B.as_full[last % kStages]), (last / kStages) & 1, abort_flag, false) && landed;
            }
            if (!landed) set_error(a.err, ERR_TIMEOUT | SITE_DRAIN);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ===================== MMA issuer (the warp in step, one elected lane issues) =====================
        constexpr uint32_t id = idesc_bf16(kM, kN, 0);
        const uint32_t leader = elect_one();
        const uint64_t bd0 = desc_sw128(smem_u32(sB), 16, 1024);
        const uint32_t full0 = smem_u32(&B.b_full[0]), empty0 = smem_u32(&B.b_empty[0]);
        uint32_t an = 0, n = 0;
        int rows = -1;
        bool ok = true;
        for (int t = t0; t < t1 && ok; ++t, ++n) {
            const uint32_t buf = n & 1, acc = tmem + kColAcc + buf * kN;
            const Tile x = tile_of(t, a.group);
            if (x.rows != rows) {
                rows = x.rows;
                if (!spin_warp(smem_u32(&B.a_ready), an & 1, abort_flag)) { give_up(SITE_FULL_WAIT); break; }
                ++an;
            }
            if (!spin_warp(smem_u32(&B.acc_empty[buf]), ((n >> 1) & 1) ^ 1, abort_flag)) { give_up(SITE_EMPTY_WAIT); break; }
            // (unrolled over the slots, descriptors by constant steps: one thread issues everything,
            // and its own instructions set the pace of small products)
#pragma unroll
            for (int j = 0; j < kBoxes; ++j) {
                if (ok && !spin_warp(full0 + 8 * j, n & 1, abort_flag)) ok = false;
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4; ++k) {   // 16 columns of the rows: 8 columns of tensor memory
                    const uint64_t bd = bd0 + (uint64_t)((j * kBBox + k * 32) >> 4);
                    if (j + k == 0) mma_f16_ts_if<0>(acc, tmem + kColA, bd, id, leader);
                    else mma_f16_ts_if<1>(acc, tmem + kColA + 32 * j + 8 * k, bd, id, leader);
                }
                mma_commit_if(empty0 + 8 * j, leader);
            }
            if (!ok) { give_up(SITE_FULL_WAIT); break; }
            mma_commit_if(smem_u32(&B.acc_full[buf]), leader);
        }
        mma_commit_if(smem_u32(&B.drain), leader);
        if (!spin_warp_drain(smem_u32(&B.drain), 0, abort_flag) && lane == 0) set_error(a.err, ERR_TIMEOUT | SITE_DRAIN);
        __syncwarp();
    } else {
        // ===================== rows into tensor memory; epilogue: a thread per row =====================
        const int quad = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const int units = a.num_blocks;
        uint32_t n = 0, an = 0, vn = 0;         // tiles, row boxes, tiles of values so far
        int rows = -1;
        bool ok = true;
        for (int t = t0; t < t1 && ok; ++t, ++n) {
            const uint32_t buf = n & 1;
            const Tile x = tile_of(t, a.group);
            if (x.rows != rows) {
                // every product of the previous rows is done: this warp has seen its last tile's end
                rows = x.rows;
                for (int j = 0; j < kBoxes && ok; ++j, ++an) {
                    ok = spin_warp(smem_u32(&B.as_full[an % kStages]), (an / kStages) & 1, abort_flag);
                    if (!ok) break;
                    const unsigned char* src = sA + an % kStages * kABox + (32 * quad + lane) * 128;
                    uint32_t v[32];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint4 w = *(const uint4*)(src + ((k ^ (lane & 7)) << 4));
                        v[4 * k] = w.x;
                        v[4 * k + 1] = w.y;
                        v[4 * k + 2] = w.z;
                        v[4 * k + 3] = w.w;
                    }
                    SKV_ST32(lanes + kColA + 32 * j, v);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&B.as_empty[an % kStages]));
                }
                if (!ok) { give_up(SITE_FULL_WAIT); break; }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&B.a_ready));
            }
            const int row = x.rows * kM + 32 * quad + lane;
            const int unit = row / kLatUnit, r = row % kLatUnit, swap = (r >> 2) & 1;
            char* image = (char*)a.kv + ((size_t)x.head * units + unit) * kLatImage + x.side * kLatSide + r * 32;
            if (!spin_warp(smem_u32(&B.acc_full[buf]), (n >> 1) & 1, abort_flag)) {
                give_up(SITE_FULL_WAIT);
                break;
            }
            tc_fence_after();
            const uint32_t acc = lanes + kColAcc + buf * kN;
            uint32_t v[kN];
#pragma unroll
            for (int c = 0; c < kN; c += 32) SKV_LD32(acc + c, (v + c));
            tc_wait_ld();
            tc_fence_before();              // the accumulator is read: the tile after next may overwrite it
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&B.acc_empty[buf]));
            uint32_t w[kN / 2];
            if (x.side == 0) {
#pragma unroll
                for (int e = 0; e < kN / 2; ++e) {
                    const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                    w[e] = *reinterpret_cast<const uint32_t*>(&p);
                }
            } else {
                // the unit's largest finite magnitude: over this thread's row, the warp, the unit's two warps
                float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < kN; ++e) {
                    const float y = fabsf(__uint_as_float(v[e]));
                    m[e & 3] = fmaxf(m[e & 3], y < INFINITY ? y : 0.f);
                }
                const float own = __uint_as_float(
                    __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])))));
                const uint32_t bar = smem_u32(&B.unit_max[quad >> 1]);
                if (lane == 0) {
                    B.warp_max[vn & 1][quad] = own;
                    mbar_arrive(bar);
                }
                __syncwarp();
                if (!spin_warp(bar, vn & 1, abort_flag)) {
                    give_up(SITE_FULL_WAIT);
                    break;
                }
                const float most = fmaxf(own, ((volatile float*)B.warp_max[vn & 1])[quad ^ 1]);
                ++vn;
                // (2^14 <= most 2^up < 2^15; an unscaled finite value above the f16 range becomes infinite)
                const int up = min(kLatValueUp, max(0, kLatValueTop + 127 - (int)(__float_as_uint(most) >> 23)));
                const float scale = __uint_as_float((uint32_t)(127 + up) << 23);
                if (most > 65504.f && lane == 0) set_error(a.err, ERR_DEVICE_CHECK | SITE_VALUE_RANGE);
                if (!(quad & 1) && lane == 0 && unit < units)
                    a.v_exp[(size_t)x.head * units + unit] = LatentScale{-(float)up, scale};
#pragma unroll
                for (int e = 0; e < kN / 2; ++e) {
                    const __half2 p = __floats2half2_rn(__uint_as_float(v[2 * e]) * scale, __uint_as_float(v[2 * e + 1]) * scale);
                    w[e] = *reinterpret_cast<const uint32_t*>(&p);
                }
            }
            if (unit < units) {         // (the last 64 rows of a tile may lie past the copy)
#pragma unroll
                for (int g = 0; g < kN / 16; ++g) store32(image + g * kLatGroup, w + 8 * g, swap);
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
}

// The batch's latent rows as bf16, request after request, each padded with zero rows to a
// multiple of 64: E4M3 codes are exact in bf16 (their scale is folded into the softmax and the
// output), and a row past a request's last token is zero whatever its page holds.
template <bool FP8>
__global__ void __launch_bounds__(256) latent_rows_kernel(LatentArgs a) {
    constexpr int kRowsPerCta = 16;
    constexpr int kPieces = kLatRow / 8;                  // 16-byte pieces of a copied row
    __shared__ long long src_row[kRowsPerCta];
    const int row0 = blockIdx.x * kRowsPerCta;
    const LatentBlock blk = a.blocks[row0 / kLatUnit];
    if (threadIdx.x < kRowsPerCta) {
        const int tok = blk.token + (row0 + threadIdx.x) % kLatUnit;
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
    const int ctas = a.num_blocks * (kLatUnit / 16);
    ProfileScope ps(SPLITKV_KERNEL_LATENT_ROWS, s);
    if (a.kv_fp8) latent_rows_kernel<true><<<ctas, 256, 0, s>>>(a);
    else latent_rows_kernel<false><<<ctas, 256, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_latent_expand(const LatentArgs& a, cudaStream_t s) {
    if (a.num_blocks <= 0) return cudaSuccess;
    const long long rows = (long long)a.num_blocks * kLatUnit;
    CUtensorMap ma, mb;
    cudaError_t e;
    if ((e = make_map(&ma, a.rows, kLatRow, rows, kM)) != cudaSuccess) return e;
    if ((e = make_map(&mb, a.w, kLatC, (long long)a.heads * kLatW, kN)) != cudaSuccess) return e;
    static std::atomic<uint64_t> allowed{0};
    if ((e = allow_smem((const void*)latent_expand_kernel, kSmemBytes, allowed)) != cudaSuccess) return e;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int tiles = (int)((rows + kM - 1) / kM) * a.group * 2;
    {
        ProfileScope ps(SPLITKV_KERNEL_LATENT_EXPAND, s);
        latent_expand_kernel<<<std::min(sms, tiles), kThreads, kSmemBytes, s>>>(ma, mb, a, tiles);
    }
    return cudaGetLastError();
}

}  // namespace skv
