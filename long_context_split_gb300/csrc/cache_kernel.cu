// Rows of new tokens into a paged cache (with E4M3 quantisation), and cache
// entries back out as rows.
//
// What it computes: row r of a ragged batch belongs to the request b with
// indptr[b] <= r < indptr[b + 1] and to that request's token pos; the token's
// cache entry is in page page_table[b][pos / P], slot pos % P.  Append:
// entry = round(x) (bf16), x (float32) or E4M3(sat(x / scale)), the quotient in
// float32 and rounded to nearest even once more to 4 significant bits.  Gather:
// x = entry, or code * scale in float32, rounded once to the row type.
//
// What bounds it: bytes (each row and each entry moves once), and for a few
// rows the chain of dependent reads (indptr, length, page id).  So the row's
// data is loaded before that chain is waited for (append), a warp finds a
// row's request with one 32-way probe per factor of 32 in the batch size, and
// each thread keeps a fixed column of the token (part, head, 8 elements) and
// walks tokens with kUnroll of them in flight.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "internal.h"

namespace skv {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;        // tokens in flight per thread
constexpr int kMaxTokens = 64;    // tokens per block

struct E4M3 {
    uint8_t code;
};

// VEC consecutive elements in registers as float32
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        if constexpr (sizeof(T) == 4) x[0] = *(const float*)p;
        else if constexpr (sizeof(T) == 2) x[0] = __bfloat162float(*(const __nv_bfloat16*)p);
        else x[0] = (float)*(const __nv_fp8_e4m3*)p;
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k) {
            const float4 v = __ldcs((const float4*)p + k);
            x[4 * k] = v.x; x[4 * k + 1] = v.y; x[4 * k + 2] = v.z; x[4 * k + 3] = v.w;
        }
    } else if constexpr (sizeof(T) == 2) {
        const uint4 v = __ldcs((const uint4*)p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = __uint_as_float(w[k] << 16);
            x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
    } else {
        const uint2 v = __ldcs((const uint2*)p);
        const uint32_t w[2] = {v.x, v.y};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((w[k >> 1] >> (16 * (k & 1))) & 0xFFFFu),
                                                             __NV_E4M3);
            const float2 f = __half22float2(__half2(h));
            x[2 * k] = f.x;
            x[2 * k + 1] = f.y;
        }
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        if constexpr (sizeof(T) == 4) *(float*)p = x[0];
        else if constexpr (sizeof(T) == 2) *(__nv_bfloat16*)p = __float2bfloat16_rn(x[0]);
        else *(uint8_t*)p = __nv_cvt_float_to_fp8(x[0], __NV_SATFINITE, __NV_E4M3);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k)
            ((float4*)p)[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
    } else if constexpr (sizeof(T) == 2) {
        *(uint4*)p = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else {
        *(uint2*)p = make_uint2(pack_e4m3(x[0], x[1], x[2], x[3]), pack_e4m3(x[4], x[5], x[6], x[7]));
    }
}

// The request of row r, by a whole warp: how many of indptr[1 .. batch] are <= r
// (batch: the row is behind the last request).
__device__ __forceinline__ int warp_owner(const int32_t* indptr, int batch, int r, int lane) {
    int lo = 0, len = batch;
    while (len > 0) {
        const int step = (len + 31) / 32;
        const bool p = (long long)lane * step < len && indptr[1 + lo + lane * step] <= r;
        const int k = __popc(__ballot_sync(0xffffffffu, p));
        if (step == 1) return lo + k;
        if (k == 0) break;
        const int next = lo + (k - 1) * step + 1;   // entry next - 1 is <= r
        len = min(step - 1, lo + len - next);
        lo = next;
    }
    return lo;
}

__device__ __forceinline__ void report(int32_t* err, int32_t code) {
    if (err) atomicCAS(err, 0, code);
}

// Cache row of each of the block's tokens: page * heads * P + slot (head h at + h * P);
// -1: refused (reported), -2: behind the last request.  One warp per token.
template <bool APPEND>
__device__ __forceinline__ void locate(const CacheRowsArgs& a, int r0, int n, long long* where) {
    const int warp = (threadIdx.y * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    const int warps = (blockDim.x * blockDim.y) >> 5;
    for (int t = warp; t < n; t += warps) {
        const int r = r0 + t;
        const int b = warp_owner(a.indptr, a.batch, r, lane);
        if (lane != 0) continue;
        long long w = -2;
        if (b < a.batch) {
            const int len = a.seq_lens[b];
            const long long pos = APPEND ? (long long)len - (a.indptr[b + 1] - r)
                                         : (long long)r - a.indptr[b] + (a.kv_begin ? a.kv_begin[b] : 0);
            w = -1;
            if (pos < 0 || pos >= len || pos / a.page_size >= a.max_pages) {
                report(a.err, ERR_DEVICE_CHECK | SITE_TOKEN_RANGE);
            } else {
                const int page = a.page_table[(size_t)b * a.max_pages + pos / a.page_size];
                if (page < 0 || page >= a.num_pages) report(a.err, ERR_DEVICE_CHECK | SITE_PAGE_RANGE);
                else w = (long long)page * a.heads * a.page_size + pos % a.page_size;
            }
        }
        where[t] = w;
    }
}

// blockDim = (columns, token lanes); a thread's column is (part, head, VEC elements)
template <typename Rows, typename Cache, int VEC, bool APPEND>
__global__ void __launch_bounds__(kThreads) cache_rows_kernel(CacheRowsArgs a, int tokens_per_block) {
    __shared__ long long where[kMaxTokens];
    const int r0 = blockIdx.x * tokens_per_block;
    const int n = min(tokens_per_block, a.rows - r0);
    const int n0 = a.heads * (a.part[0].width / VEC);
    const int cols = n0 + a.heads * (a.part[1].width / VEC);
    bool located = false;
    for (int c = threadIdx.x; c < cols || !located; c += blockDim.x) {
        const bool on = c < cols;
        const CachePart& p = a.part[c >= n0 && on];
        const int per = max(1, p.width / VEC);
        const int cc = c >= n0 ? c - n0 : c;
        const int h = cc / per, e = (cc % per) * VEC;
        Rows* rows = (Rows*)p.rows + (size_t)r0 * p.token_stride + h * p.head_stride + e;
        Cache* cache = (Cache*)p.cache + (size_t)h * a.page_size * p.row_width + p.col + e;
        for (int t0 = threadIdx.y; t0 < n || !located; t0 += kUnroll * blockDim.y) {
            float x[kUnroll][VEC];
            if (APPEND) {
#pragma unroll
                for (int k = 0; k < kUnroll; ++k)
                    if (on && t0 + k * (int)blockDim.y < n) load_vec<Rows, VEC>(rows + (t0 + k * blockDim.y) * p.token_stride, x[k]);
            }
            if (!located) {   // once per block, on every thread's first pass
                locate<APPEND>(a, r0, n, where);
                __syncthreads();
                located = true;
            }
            if (!on) break;
            long long w[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) w[k] = t0 + k * (int)blockDim.y < n ? where[t0 + k * blockDim.y] : -2;
            if (APPEND) {
#pragma unroll
                for (int k = 0; k < kUnroll; ++k) {
                    if (w[k] < 0) continue;
                    if constexpr (sizeof(Cache) == 1) {
#pragma unroll
                        for (int j = 0; j < VEC; ++j) x[k][j] = x[k][j] / p.scale;
                    }
                    store_vec<Cache, VEC>(cache + w[k] * p.row_width, x[k]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < kUnroll; ++k) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) x[k][j] = 0.f;   // a refused row reads as zeros
                    if (w[k] >= 0) load_vec<Cache, VEC>(cache + w[k] * p.row_width, x[k]);
                }
#pragma unroll
                for (int k = 0; k < kUnroll; ++k) {
                    if (w[k] == -2) continue;
                    if constexpr (sizeof(Cache) == 1) {
#pragma unroll
                        for (int j = 0; j < VEC; ++j) x[k][j] *= p.scale;
                    }
                    store_vec<Rows, VEC>(rows + (t0 + k * blockDim.y) * p.token_stride, x[k]);
                }
            }
        }
    }
}

// 8 elements per access where every row and entry address is a multiple of 16 bytes (8 for
// E4M3 entries); one element otherwise
bool vectors_fit(const CacheRowsArgs& a, int rows_size, int cache_size) {
    for (const CachePart& p : a.part) {
        if (p.width == 0) continue;
        const int ra = 16 / rows_size, ca = cache_size == 1 ? 8 : 16 / cache_size;
        if (p.width % 8 || p.token_stride % ra || p.head_stride % ra || ((uintptr_t)p.rows & 15)) return false;
        if (p.row_width % ca || p.col % ca || ((uintptr_t)p.cache & (cache_size == 1 ? 7 : 15))) return false;
    }
    return true;
}

template <typename Rows, typename Cache, bool APPEND>
cudaError_t launch_rows(const CacheRowsArgs& a, cudaStream_t s) {
    int dev = 0, sms = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const bool vec = vectors_fit(a, sizeof(Rows), sizeof(Cache));
    const int v = vec ? 8 : 1;
    const int cols = a.heads * (a.part[0].width / v) + a.heads * (a.part[1].width / v);
    const int bx = std::min(kThreads, (cols + 31) / 32 * 32);
    const int by = std::max(1, kThreads / bx);
    // tokens per block: enough that a thread has kUnroll in flight, fewer while that leaves SMs idle
    const int per = std::min(kMaxTokens, std::max(by, std::min(by * kUnroll, a.rows / (2 * sms))));
    const int blocks = (a.rows + per - 1) / per;
    const dim3 block(bx, by);
    ProfileScope ps(APPEND ? SPLITKV_KERNEL_KV_APPEND : SPLITKV_KERNEL_KV_GATHER, s);
    if (vec) cache_rows_kernel<Rows, Cache, 8, APPEND><<<blocks, block, 0, s>>>(a, per);
    else cache_rows_kernel<Rows, Cache, 1, APPEND><<<blocks, block, 0, s>>>(a, per);
    return cudaGetLastError();
}

template <bool APPEND>
cudaError_t launch_any(const CacheRowsArgs& a, int cache_kind, int rows_f32, cudaStream_t s) {
    if (a.rows <= 0) return cudaSuccess;
    if (rows_f32) {
        if (cache_kind == 0) return launch_rows<float, float, APPEND>(a, s);
        if (cache_kind == 1) return launch_rows<float, __nv_bfloat16, APPEND>(a, s);
        return launch_rows<float, E4M3, APPEND>(a, s);
    }
    if (cache_kind == 0) return launch_rows<__nv_bfloat16, float, APPEND>(a, s);
    if (cache_kind == 1) return launch_rows<__nv_bfloat16, __nv_bfloat16, APPEND>(a, s);
    return launch_rows<__nv_bfloat16, E4M3, APPEND>(a, s);
}

}  // namespace

cudaError_t launch_kv_append(const CacheRowsArgs& a, int cache_kind, int rows_f32, cudaStream_t s) {
    return launch_any<true>(a, cache_kind, rows_f32, s);
}

cudaError_t launch_kv_gather(const CacheRowsArgs& a, int cache_kind, int rows_f32, cudaStream_t s) {
    return launch_any<false>(a, cache_kind, rows_f32, s);
}

}  // namespace skv
