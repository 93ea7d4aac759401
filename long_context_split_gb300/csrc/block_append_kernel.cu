// Rows of new tokens into a paged E4M3 cache that has a scale for each block of S
// tokens and KV head.
//
// What it computes, for one block and head (keys and values alike): with a = the
// largest finite |x| of the block's new tokens, and s the block's scale where
// it holds older tokens,  s' = s where there is such an s with a <= 448 s, otherwise the
// smallest power of two with a <= 448 s';  new codes E4M3(sat(x / s')), older codes
// E4M3(code s / s') where s' differs from s.
//
// What bounds it: bytes (rows read once, codes written once) for prompts, and for
// a few rows the chain row -> request -> length -> page id -> scale.  A unit (block,
// head, keys or values) is taken by 1, 2, 4 or 8 warps, as many as hold its rows in
// registers between the maximum and the quantisation (128 bytes a lane, so that four CTAs fit an SM; 256 for the
// largest), so that rows are read once; a CTA works on 8 warps' worth of units at a time, on as many rows as leave
// one round of CTAs, so that the chain is waited for once for many rows.  18,524 rows of 8 heads of 128
// (bf16, blocks of 16): 20 us, 5.7 TB/s, the rest the ramp of a short launch (61.6 with 256 bytes a lane throughout,
// 44 with magnitudes compared as floats, 24 with five CTAs an SM); blocks of 64 22, of 128 24, float32 rows 36; 64 rows,
// one a request, 5.9.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cfloat>

#include "operators.h"

namespace skv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxUnits = 128;     // rows, so at most as many blocks, of a CTA

// One block with new tokens: its first new row, how many, and where they go
struct Unit {
    long long slot;     // page * heads * P + slot of the first new token (head h at + h * P)
    int row;            // relative to the CTA's first row
    int rows;
    int old;            // older tokens of the block, the slots just before
};

// VEC elements of a row
template <typename T, int VEC>
struct Piece {
    uint32_t w[(VEC * (int)sizeof(T) + 3) / 4];
};

template <typename T, int VEC>
__device__ __forceinline__ void load_piece(Piece<T, VEC>& r, const T* p) {
    if constexpr (VEC * sizeof(T) == 16) {
        const uint4 v = __ldcs((const uint4*)p);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else if constexpr (sizeof(T) == 4) {
        r.w[0] = *(const uint32_t*)p;
    } else {
        r.w[0] = *(const uint16_t*)p;
    }
}

template <typename T, int VEC>
__device__ __forceinline__ float element(const Piece<T, VEC>& r, int k) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(r.w[k]);
    return __uint_as_float((k & 1) ? r.w[k / 2] & 0xFFFF0000u : r.w[k / 2] << 16);
}

// |x|, 0 for infinities and NaN (they leave the scale alone: a saturated code or the NaN code)
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= FLT_MAX ? a : 0.f;
}

// The largest magnitude of pieces, as bits: magnitudes order as integers do (those of infinities and NaN above
// all), two bf16 in a word.
template <typename T, int VEC>
struct Largest {
    uint32_t bits = 0;
    __device__ __forceinline__ void add(const Piece<T, VEC>& r) {
#pragma unroll
        for (int j = 0; j < (VEC * (int)sizeof(T) + 3) / 4; ++j) {
            if constexpr (sizeof(T) == 4) bits = max(bits, r.w[j] & 0x7FFFFFFFu);
            else bits = __vmaxu2(bits, r.w[j] & 0x7FFF7FFFu);
        }
    }
    __device__ __forceinline__ float value() const {
        return __uint_as_float(sizeof(T) == 4 ? bits : max(bits >> 16, bits & 0xFFFFu) << 16);
    }
};

// The smallest power of two, from 2^-126 on, whose 448-fold is not below a.  448 = 1.75 * 2^8.
__device__ __forceinline__ float pow2_scale(float a) {
    const uint32_t bits = __float_as_uint(a);
    const int e = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // biased
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

__device__ __forceinline__ bool is_pow2(float s) { return (__float_as_uint(s) & 0x807FFFFFu) == 0; }

__device__ __forceinline__ uint8_t encode1(float x) { return (uint8_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3); }

__device__ __forceinline__ uint32_t encode4(float x0, float x1, float x2, float x3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x2, x3), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// x / s in float32, correctly rounded: a power of two's reciprocal is exact
template <bool POW2>
struct Quotient {
    float s;             // its reciprocal for a power of two
    __device__ explicit Quotient(float scale) : s(POW2 ? 1.f / scale : scale) {}
    __device__ __forceinline__ float operator()(float x) const { return POW2 ? x * s : __fdiv_rn(x, s); }
};

template <typename T, int VEC, bool POW2>
__device__ __forceinline__ void store_codes(uint8_t* to, const Piece<T, VEC>& r, const Quotient<POW2>& q) {
    if constexpr (VEC == 8) {
        uint2 v;
        v.x = encode4(q(element<T, VEC>(r, 0)), q(element<T, VEC>(r, 1)), q(element<T, VEC>(r, 2)), q(element<T, VEC>(r, 3)));
        v.y = encode4(q(element<T, VEC>(r, 4 % VEC)), q(element<T, VEC>(r, 5 % VEC)), q(element<T, VEC>(r, 6 % VEC)),
                      q(element<T, VEC>(r, 7 % VEC)));
        *(uint2*)to = v;
    } else if constexpr (VEC == 4) {
        *(uint32_t*)to = encode4(q(element<T, VEC>(r, 0)), q(element<T, VEC>(r, 1)), q(element<T, VEC>(r, 2)),
                                 q(element<T, VEC>(r, 3)));
    } else {
        *to = encode1(q(element<T, VEC>(r, 0)));
    }
}

__device__ __forceinline__ void report(int32_t* err, int32_t code) {
    if (err) atomicCAS(err, 0, code);
}

// The blocks that begin among the CTA's rows (a block begins at its first new token), a thread
// per row.  Returns their number.
__device__ __forceinline__ int find_units(const CacheRowsArgs& a, int r0, int n, Unit* units, int* count) {
    const int S = 1 << a.scale_shift, P = a.page_size;
    if (threadIdx.x == 0) *count = 0;
    __syncthreads();
    if (threadIdx.x < n) {
        const int r = r0 + threadIdx.x;
        int lo = 0, hi = a.batch;             // how many of indptr[1 .. batch] are <= r
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.indptr[1 + mid] <= r) lo = mid + 1; else hi = mid;
        }
        if (lo < a.batch) {                   // (rows behind the last request are left alone)
            const int b = lo, end = a.indptr[b + 1], first = max(0, a.indptr[b]), len = a.seq_lens[b];
            const long long pos = (long long)len - (end - r);
            if (pos < 0) {
                report(a.err, ERR_DEVICE_CHECK | SITE_TOKEN_RANGE);
            } else if (r == first || pos % S == 0) {
                const long long before = (long long)len - (end - first);   // the request's first new token
                if (pos / P >= a.max_pages) {
                    report(a.err, ERR_DEVICE_CHECK | SITE_TOKEN_RANGE);
                } else {
                    const int page = a.page_table[(size_t)b * a.max_pages + pos / P];
                    if (page < 0 || page >= a.num_pages) {
                        report(a.err, ERR_DEVICE_CHECK | SITE_PAGE_RANGE);
                    } else {
                        Unit u;
                        u.slot = (long long)page * a.heads * P + pos % P;
                        u.row = threadIdx.x;
                        u.rows = min(S - (int)(pos % S), min(end, a.rows) - r);
                        u.old = before == pos ? (int)(pos % S) : 0;
                        units[atomicAdd(count, 1)] = u;   // (any order: a block is one unit's alone)
                    }
                }
            }
        }
    }
    __syncthreads();
    return *count;
}

// W warps per unit, of which a lane holds kHold pieces; gridDim.y shares the (keys or values, head) pairs out.
// per_shift: log2 of a row's pieces, -1 where that is not whole.
template <typename T, int VEC, int W, int kHold>
__global__ void __launch_bounds__(kThreads, kHold <= 8 ? 4 : 2) block_append_kernel(CacheRowsArgs a, int rows_per_cta, int per_shift) {
    __shared__ Unit units[kMaxUnits];
    __shared__ int count;
    __shared__ float warp_max[kWarps];
    const int r0 = blockIdx.x * rows_per_cta;
    const int n = find_units(a, r0, min(rows_per_cta, a.rows - r0), units, &count);
    constexpr int kLanes = 32 * W, kGroups = kWarps / W;
    const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const int pairs = 2 * a.heads, width = a.part[0].width, per = width / VEC;
    const int mine = (pairs - (int)blockIdx.y + (int)gridDim.y - 1) / (int)gridDim.y;   // pairs of this CTA
    for (int i0 = 0; i0 < n * mine; i0 += kGroups) {
        const int i = i0 + group;
        const bool on = i < n * mine;
        const Unit u = units[on ? i / mine : 0];
        const int pair = (int)blockIdx.y + (on ? i % mine : 0) * (int)gridDim.y;
        const int h = pair >> 1;
        const CachePart& p = a.part[pair & 1];
        const T* rows = (const T*)p.rows + (size_t)(r0 + u.row) * p.token_stride + h * p.head_stride;
        uint8_t* codes = (uint8_t*)p.cache + (size_t)(u.slot + (long long)h * a.page_size) * width;
        float* scale_at = p.scales + ((u.slot + (long long)h * a.page_size) >> a.scale_shift);
        const int pieces = on ? u.rows * per : 0;
        const bool held = pieces <= kHold * kLanes;
        const float was = on && u.old > 0 ? *scale_at : 0.f;
        // ---- the largest magnitude, the rows kept in registers ----
        Piece<T, VEC> x[kHold];
        float top = 0.f;
        auto at = [&](int k) {
            const int r = per_shift >= 0 ? k >> per_shift : k / per;
            return rows + (size_t)r * p.token_stride + (k - r * per) * VEC;
        };
        if (held) {
#pragma unroll
            for (int k = 0; k < kHold; ++k)
                if (lane + k * kLanes < pieces) load_piece<T, VEC>(x[k], at(lane + k * kLanes));
            Largest<T, VEC> all;
#pragma unroll
            for (int k = 0; k < kHold; ++k)
                if (lane + k * kLanes < pieces) all.add(x[k]);
            top = all.value();
            if (!(top <= FLT_MAX)) {       // an infinity or NaN among them
                top = 0.f;
#pragma unroll
                for (int k = 0; k < kHold; ++k)
                    if (lane + k * kLanes < pieces)
#pragma unroll
                        for (int j = 0; j < VEC; ++j) top = fmaxf(top, finite_abs(element<T, VEC>(x[k], j)));
            }
        } else {
            for (int k = lane; k < pieces; k += kLanes) {
                load_piece<T, VEC>(x[0], at(k));
#pragma unroll
                for (int j = 0; j < VEC; ++j) top = fmaxf(top, finite_abs(element<T, VEC>(x[0], j)));
            }
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        if constexpr (W > 1) {
            const int w0 = group * W;
            __syncthreads();
            if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = top;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < W; ++k) top = fmaxf(top, warp_max[w0 + k]);
        }
        // (also orders the read of the old scale before its update below)
        __syncwarp();
        if (!on) continue;
        const bool keep = was > 0.f && top <= 448.f * was;
        const float now = keep ? was : pow2_scale(top);
        auto quantise = [&](auto q) {
            if (u.old > 0 && !keep) {
                // ---- older codes under the new scale ----
                uint8_t* old = codes - (size_t)u.old * width;
                for (int k = lane; k < u.old * per; k += kLanes) {
                    uint8_t* c = old + (size_t)k * VEC;
                    if constexpr (VEC == 1) {
                        const float v = __half2float(__half(__nv_cvt_fp8_to_halfraw(*c, __NV_E4M3)));
                        *c = encode1(q(v * was));
                    } else {
#pragma unroll
                        for (int g = 0; g < VEC / 4; ++g) {
                            const uint32_t w = ((uint32_t*)c)[g];
                            const float2 lo = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3)));
                            const float2 hi = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3)));
                            ((uint32_t*)c)[g] = encode4(q(lo.x * was), q(lo.y * was), q(hi.x * was), q(hi.y * was));
                        }
                    }
                }
            }
            if (held) {
#pragma unroll
                for (int k = 0; k < kHold; ++k) {
                    const int e = lane + k * kLanes;
                    if (e < pieces) store_codes<T, VEC>(codes + (size_t)e * VEC, x[k], q);
                }
            } else {
                for (int k = lane; k < pieces; k += kLanes) {
                    load_piece<T, VEC>(x[0], at(k));
                    store_codes<T, VEC>(codes + (size_t)k * VEC, x[0], q);
                }
            }
        };
        if (is_pow2(now)) quantise(Quotient<true>(now));
        else quantise(Quotient<false>(now));
        if (lane == 0 && !(u.old > 0 && keep)) *scale_at = now;
    }
}

template <typename T, int VEC, int W, int kHold>
cudaError_t launch_w(const CacheRowsArgs& a, cudaStream_t s) {
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int y = std::max(1, std::min(2 * a.heads, 2 * a.heads * W / kWarps));   // one unit per group of warps
    // all CTAs at once, as many as fit (18,524 rows: 20.3 us; with five an SM 24.2, the fifth after the others)
    constexpr int kCtas = kHold <= 8 ? 4 : 2;
    const long long want = ((long long)a.rows * y + kCtas * sms - 1) / (kCtas * sms);
    const int per = (int)std::max(1ll, std::min<long long>(kMaxUnits, want));
    const long long x = ((long long)a.rows + per - 1) / per;
    if (x > 0x7fffffff) return cudaErrorInvalidValue;
    const int pieces = a.part[0].width / VEC;
    int shift = 0;
    while ((1 << shift) < pieces) ++shift;
    ProfileScope ps(SPLITKV_KERNEL_KV_APPEND, s);
    block_append_kernel<T, VEC, W, kHold><<<dim3((unsigned)x, (unsigned)y), kThreads, 0, s>>>(a, per, (1 << shift) == pieces ? shift : -1);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const CacheRowsArgs& a, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    bool vec = true;
    for (const CachePart& p : a.part)
        vec = vec && p.width % V == 0 && (a.rows == 1 || p.token_stride * sizeof(T) % 16 == 0) &&
              (a.heads == 1 || p.head_stride * sizeof(T) % 16 == 0) && !((uintptr_t)p.rows & 15) && !((uintptr_t)p.cache % V);
    if (!vec) return launch_w<T, 1, 8, 8>(a, s);
    const size_t bytes = ((size_t)a.part[0].width * sizeof(T)) << a.scale_shift;   // of a unit
    if (bytes <= 4096) return launch_w<T, V, 1, 8>(a, s);
    if (bytes <= 8192) return launch_w<T, V, 2, 8>(a, s);
    if (bytes <= 16384) return launch_w<T, V, 4, 8>(a, s);
    if (bytes <= 32768) return launch_w<T, V, 8, 8>(a, s);
    return launch_w<T, V, 8, 16>(a, s);
}

}  // namespace

cudaError_t launch_block_append(const CacheRowsArgs& a, int rows_f32, cudaStream_t s) {
    if (a.rows <= 0) return cudaSuccess;
    return rows_f32 ? launch_t<float>(a, s) : launch_t<__nv_bfloat16>(a, s);
}

}  // namespace skv
