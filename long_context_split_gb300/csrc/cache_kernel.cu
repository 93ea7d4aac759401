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
// each thread keeps a fixed column of the token (part, head, 8 or 16 elements) and
// walks tokens with several of them in flight.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "operators.h"

namespace skv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 64;    // tokens per block

struct E4M3 {
    uint8_t code;
};

// BYTES consecutive bytes in registers
template <int BYTES>
struct Raw {
    uint32_t w[(BYTES + 3) / 4];
};

// streaming loads and stores of a piece in accesses of at most 32 bytes
template <int BYTES>
__device__ __forceinline__ void load_raw(Raw<BYTES>& r, const void* p) {
    if constexpr (BYTES >= 32) {
#pragma unroll
        for (int k = 0; k < BYTES / 32; ++k) {
            uint32_t* w = r.w + 8 * k;
            asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                         : "l"((const char*)p + 32 * k));
        }
    } else if constexpr (BYTES == 16) {
        const uint4 v = __ldcs((const uint4*)p);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else if constexpr (BYTES == 8) {
        const uint2 v = __ldcs((const uint2*)p);
        r.w[0] = v.x; r.w[1] = v.y;
    } else if constexpr (BYTES == 4) {
        r.w[0] = *(const uint32_t*)p;
    } else if constexpr (BYTES == 2) {
        r.w[0] = *(const uint16_t*)p;
    } else {
        r.w[0] = *(const uint8_t*)p;
    }
}

template <int BYTES>
__device__ __forceinline__ void store_raw(void* p, const Raw<BYTES>& r) {
    if constexpr (BYTES >= 32) {
#pragma unroll
        for (int k = 0; k < BYTES / 32; ++k) {
            const uint32_t* w = r.w + 8 * k;
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"((char*)p + 32 * k), "r"(w[0]), "r"(w[1]),
                         "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
        }
    } else if constexpr (BYTES == 16) {
        *(uint4*)p = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    } else if constexpr (BYTES == 8) {
        *(uint2*)p = make_uint2(r.w[0], r.w[1]);
    } else if constexpr (BYTES == 4) {
        *(uint32_t*)p = r.w[0];
    } else if constexpr (BYTES == 2) {
        *(uint16_t*)p = (uint16_t)r.w[0];
    } else {
        *(uint8_t*)p = (uint8_t)r.w[0];
    }
}

// the VEC elements of type T in a piece, as float32
template <typename T, int VEC>
__device__ __forceinline__ void decode(const Raw<VEC * (int)sizeof(T)>& r, float (&x)[VEC]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) x[k] = __uint_as_float(r.w[k]);
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) x[k] = __uint_as_float((k & 1) ? r.w[k / 2] & 0xFFFF0000u : r.w[k / 2] << 16);
    } else {
#pragma unroll
        for (int k = 0; k < (VEC + 1) / 2; ++k) {
            const uint32_t two = (r.w[k / 2] >> (16 * (k & 1))) & 0xFFFFu;
            const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3)));
            x[2 * k] = f.x;
            if (2 * k + 1 < VEC) x[2 * k + 1] = f.y;
        }
    }
}

// float32 values rounded to type T (E4M3: saturated), packed
template <typename T, int VEC>
__device__ __forceinline__ void encode(Raw<VEC * (int)sizeof(T)>& r, const float (&x)[VEC]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) r.w[k] = __float_as_uint(x[k]);
    } else if constexpr (VEC == 1) {
        if constexpr (sizeof(T) == 2) r.w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(x[0]));
        else r.w[0] = __nv_cvt_float_to_fp8(x[0], __NV_SATFINITE, __NV_E4M3);
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int k = 0; k < VEC / 2; ++k) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
            r.w[k] = *reinterpret_cast<const uint32_t*>(&v);
        }
    } else {
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * k], x[4 * k + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * k + 2], x[4 * k + 3]), __NV_SATFINITE, __NV_E4M3);
            r.w[k] = lo | (hi << 16);
        }
    }
}

// x / scale for scales whose reciprocal and remainders stay normal numbers (plain_scale): with inv the
// rounded reciprocal, the remainder x - y scale of y = x inv in a fused multiply-add, and one correction
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", IBM J. Res. Dev.
// 34, 1990; there y starts within a unit of the quotient, here it may be a little further off).  What is needed is the
// E4M3 code of the correctly rounded quotient, and that holds: for all 2^23 mantissas of the scale and every x
// within four units of a border between two codes, the result lies on the right side of the border.
// y itself serves where E4M3 saturates, for infinities and NaN, and where E4M3 is zero (of y's
// sign: the correction would lose that of -0).
__device__ __forceinline__ float quotient(float x, float scale, float inv) {
    const float y = x * inv;
    const float q = fmaf(fmaf(-scale, y, x), inv, y);
    return fabsf(y) < 1024.f && fabsf(y) > 0x1p-20f ? q : y;
}

__device__ __forceinline__ bool plain_scale(float scale) { return scale >= 0x1p-60f && scale <= 0x1p60f; }

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

// blockDim = (columns, token lanes); a thread's column is (part, head, VEC elements).  Pieces
// stay in registers as they were read (kUnroll tokens of them) until they are converted and
// stored.  Append converts more per byte read and wants warps: 64 bytes in flight a thread and
// five blocks an SM (22.6k tokens into E4M3: 29.2 us; 37.5 with 128 bytes and three blocks);
// gather wants loads: 128 bytes and four blocks (651 MB: 107.5 us; 123 with five blocks).
template <typename Rows, typename Cache, int VEC, bool APPEND>
__global__ void __launch_bounds__(kThreads, APPEND ? 5 : 4) cache_rows_kernel(CacheRowsArgs a, int tokens_per_block) {
    using Src = std::conditional_t<APPEND, Rows, Cache>;
    using Dst = std::conditional_t<APPEND, Cache, Rows>;
    constexpr int kSrc = VEC * (int)sizeof(Src), kDst = VEC * (int)sizeof(Dst);
    constexpr int kUnroll = VEC == 1 ? 4 : std::min(8, std::max(2, (APPEND ? 64 : 128) / kSrc));
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
        const float scale = p.scale, inv = 1.f / scale;
        const bool plain = plain_scale(scale);
        for (int t0 = threadIdx.y; t0 < n || !located; t0 += kUnroll * blockDim.y) {
            Raw<kSrc> src[kUnroll];
            if (APPEND) {
#pragma unroll
                for (int k = 0; k < kUnroll; ++k)
                    if (on && t0 + k * (int)blockDim.y < n) load_raw<kSrc>(src[k], rows + (t0 + k * blockDim.y) * p.token_stride);
            }
            if (!located) {   // once per block, on every thread's first pass
                locate<APPEND>(a, r0, n, where);
                __syncthreads();
                located = true;
            }
            if (!on) break;
            if (!APPEND) {
#pragma unroll
                for (int k = 0; k < kUnroll; ++k) {
                    const long long w = t0 + k * (int)blockDim.y < n ? where[t0 + k * blockDim.y] : -2;
#pragma unroll
                    for (int j = 0; j < (kSrc + 3) / 4; ++j) src[k].w[j] = 0u;   // a refused row reads as zeros
                    if (w >= 0) load_raw<kSrc>(src[k], cache + w * p.row_width);
                }
            }
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int t = t0 + k * (int)blockDim.y;
                if (t >= n) break;
                const long long w = where[t];
                if (APPEND ? w < 0 : w == -2) continue;
                Dst* to = APPEND ? (Dst*)(cache + w * p.row_width) : (Dst*)(rows + t * p.token_stride);
                if constexpr (std::is_same_v<Src, Dst>) {
                    store_raw<kSrc>(to, src[k]);
                } else {
                    float x[VEC];
                    decode<Src, VEC>(src[k], x);
                    if constexpr (sizeof(Cache) == 1) {
                        if (!APPEND) {
#pragma unroll
                            for (int j = 0; j < VEC; ++j) x[j] *= scale;
                        } else if (plain) {
#pragma unroll
                            for (int j = 0; j < VEC; ++j) x[j] = quotient(x[j], scale, inv);
                        } else {
#pragma unroll
                            for (int j = 0; j < VEC; ++j) x[j] = x[j] / scale;
                        }
                    }
                    Raw<kDst> dst;
                    encode<Dst, VEC>(dst, x);
                    store_raw<kDst>(to, dst);
                }
            }
        }
    }
}

// Whether every row and entry address is a multiple of a piece's access (VEC elements, at most 32 bytes)
bool vectors_fit(const CacheRowsArgs& a, int vec, int rows_size, int cache_size) {
    const int rb = std::min(32, vec * rows_size), cb = std::min(32, vec * cache_size);
    for (const CachePart& p : a.part) {
        if (p.width == 0) continue;
        if (p.width % vec || p.token_stride * rows_size % rb || p.head_stride * rows_size % rb || (uintptr_t)p.rows % rb) return false;
        if (p.row_width * cache_size % cb || p.col * cache_size % cb || (uintptr_t)p.cache % cb) return false;
    }
    return true;
}

template <typename Rows, typename Cache, int VEC, bool APPEND>
cudaError_t launch_vec(const CacheRowsArgs& a, cudaStream_t s) {
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int cols = a.heads * (a.part[0].width / VEC) + a.heads * (a.part[1].width / VEC);
    const int bx = std::min(kThreads, (cols + 31) / 32 * 32);
    const int by = std::max(1, kThreads / bx);
    // tokens per block: about 8 blocks per SM (as many as fit), so that a block waits for its chain of
    // dependent reads once for many tokens; few rows get a block per `by` tokens
    const int per = std::min(kMaxTokens, std::max(by, a.rows / (8 * sms)));
    const int blocks = (int)(((long long)a.rows + per - 1) / per);
    ProfileScope ps(APPEND ? SPLITKV_KERNEL_KV_APPEND : SPLITKV_KERNEL_KV_GATHER, s);
    cache_rows_kernel<Rows, Cache, VEC, APPEND><<<blocks, dim3(bx, by), 0, s>>>(a, per);
    return cudaGetLastError();
}

// The widest piece that every address allows: 16 elements for E4M3 caches (16 bytes of codes), 8 for
// others, 4 where float32 is on 16-byte boundaries only, element by element for odd widths and offsets
template <typename Rows, typename Cache, bool APPEND>
cudaError_t launch_rows(const CacheRowsArgs& a, cudaStream_t s) {
    if constexpr (sizeof(Cache) == 1)
        if (vectors_fit(a, 16, sizeof(Rows), 1)) return launch_vec<Rows, Cache, 16, APPEND>(a, s);
    if (vectors_fit(a, 8, sizeof(Rows), sizeof(Cache))) return launch_vec<Rows, Cache, 8, APPEND>(a, s);
    if constexpr (sizeof(Rows) == 4 || sizeof(Cache) == 4)
        if (vectors_fit(a, 4, sizeof(Rows), sizeof(Cache))) return launch_vec<Rows, Cache, 4, APPEND>(a, s);
    return launch_vec<Rows, Cache, 1, APPEND>(a, s);
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
