// The next token of each row of logits, and the distribution it is drawn from.
//
// What it computes, with m the row's largest logit and T its temperature: weights exp((x_i - m) / T);
// tokens ordered by (x descending, index ascending), the order of the 64-bit number "rank" = (monotone
// image of x's bits, inverted index).  Every filter keeps the tokens from some rank up, so that what
// is kept is one `cut`: min_p's follows from m, top_k's is the k-th largest rank, top_p's the rank at
// which the weights summed in descending order reach top_p of what is left.  The draw inverts the
// distribution function over the kept tokens in index order.
//
// Arithmetic: which token a border falls on must not depend on the order of a sum, so a weight is an
// integer, its value in units of 2^-44 of a power of two just above the largest, and sums are
// integers.  Float64 runs at 1/64 of the float32 rate here, so exp is evaluated on pairs of float32
// with a table of 2^(j/128) (P. T. P. Tang, "Table-driven implementation of the exponential function
// in IEEE floating-point arithmetic", ACM Trans. Math. Softw. 15, 1989): an error below 2^-40 of the
// weight (2^-38 where |m| / T is some hundreds), in about 40 instructions.
//
// What bounds it: one pass over the logits from memory; the rest are passes over the same row from L2,
// their instructions, and latency.  128 rows of 128,000 bf16 logits: the largest alone 11 us, a draw
// without filters 46 (40 instructions a token for its weight: issue slots), top_k 50 29, top_p 0.9 77,
// over flat rows 243; one such row 5, 13, 10, 19 and 53 (a chain of passes and barriers).  A cluster
// of CTAs takes a row, a warp a contiguous segment of the vocabulary.  The first pass takes the
// maximum, and that of every lane: the r-th largest of a CTA's thread maxima has at least r tokens
// from it up, and usually not many more, so that one pass with one comparison a token collects the
// candidates of top_k, or of top_p where it also sums all weights; CTA 0 has them (at most 2048) in
// shared memory, and all else follows from them: a few are each compared with all others, more go
// through histograms of their ranks.  Where they do not reach top_p (a flat distribution) or top_k is
// large, the cut is found in a histogram of the tokens and weights over 2048 bins of x, whose bin with
// the cut is divided again while it holds more than 2048 tokens, down to equal logits told apart by
// index; the draw then takes the segments' sums of what is kept, and the one segment of the draw, as
// the verification of drafts does.
#include <cuda_bf16.h>

#include <algorithm>
#include <array>
#include <cfloat>
#include <climits>

#include "operators.h"

namespace skv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 4 * kThreads;
// Bins of 1/80 of a factor of two in weight (of exp(x) for counts) below the largest, so fine that a warp's tokens
// seldom meet in one, and after half of them of 1/16
constexpr float kFine = 80.f, kCoarse = 0.2f;
constexpr int kList = 2048;          // tokens that CTA 0 selects from in shared memory
constexpr int kOne = 44;             // weights are in units of 2^-44
constexpr int kTable = 128;
constexpr int kLimb = 15;            // a histogram's weights in three parts, each summed in 32 bits over 2^17 tokens

typedef unsigned long long u64;

// 2^(j / 128) as a sum of two floats, from the series of exp
struct Two {
    float hi, lo;
};
constexpr std::array<Two, kTable> make_table() {
    std::array<Two, kTable> t{};
    for (int j = 0; j < kTable; ++j) {
        const double x = 0.69314718055994530942 * j / kTable;
        double term = 1.0, sum = 1.0;
        for (int k = 1; k < 30; ++k) {
            term *= x / k;
            sum += term;
        }
        t[j].hi = (float)sum;
        t[j].lo = (float)(sum - (double)t[j].hi);
    }
    return t;
}
__device__ const std::array<Two, kTable> g_table = make_table();

// ---- ranks -----------------------------------------------------------------------
// larger x, larger key; both zeros alike
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.f));
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ ((key & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ u64 rank_of(float x, int v) { return ((u64)key_of(x) << 32) | (uint32_t)~v; }
__device__ __forceinline__ int token_of(u64 rank) { return (int)~(uint32_t)rank; }

// What is kept: the tokens of larger logits than x, and of x itself those up to v.  (NaN and, since x is
// finite or +infinity, -infinity are not.)
struct Cut {
    float x;
    int v;
    __device__ __forceinline__ bool keeps(float f, int token) const { return f > x || (f == x && token <= v); }
};
__device__ __forceinline__ Cut cut_at(u64 rank) { return Cut{value_of((uint32_t)(rank >> 32)), token_of(rank)}; }

// ---- weights ---------------------------------------------------------------------
struct Scale {
    float top;       // subtracted from the logits first (0 where |m| / T is small enough without)
    float hi, lo;    // log2(e) / T as a pair
    float least;     // products below it are taken as this: a weight of 2^-127 or so
    int ref;         // weights are 2^(x log2(e) / T - ref)
    int diff;        // 1: subtract top
};

struct Weight {
    float hi, lo;    // (hi + lo) 2^n, hi about 1 .. 2
    int n;           // -1 for the largest, at most, and -130 at least; below -126: nothing
};

__device__ __forceinline__ Weight weight_of(const Two* table, const Scale& s, float x) {
    float extra = 0.f;
    if (s.diff) {    // x - top exactly
        const float d = __fsub_rn(x, s.top), bb = __fsub_rn(d, x);
        extra = __fmul_rn(__fadd_rn(__fsub_rn(x, __fsub_rn(d, bb)), __fsub_rn(-s.top, bb)), s.hi);
        x = d;
    }
    // u + ue = x log2(e) / T = i / 128 + (f + ue), |f| <= 1 / 256
    // (no branch, so that several evaluations run beside one another; NaN and what is far below end at `least`)
    const float u = fmaxf(__fmul_rn(x, s.hi), s.least);
    float ue = __fmaf_rn(x, s.lo, __fadd_rn(__fmaf_rn(x, s.hi, -u), extra));
    ue = u > s.least ? ue : 0.f;
    const float magic = 12582912.f;   // 1.5 * 2^23
    const float r = __fmaf_rn(u, 128.f, magic);
    const int i = __float_as_int(r) - __float_as_int(magic);
    const float f = __fmaf_rn(__fsub_rn(r, magic), -1.f / 128.f, u);
    // y = (f + ue) ln 2 = yh + yl; exp(y) - 1 = yh + rest
    constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = (float)(0.69314718055994530942 - 0.693147182464599609375);
    const float yh = __fmul_rn(f, kLn2Hi);
    const float yl = __fmaf_rn(ue, kLn2Hi, __fmaf_rn(f, kLn2Lo, __fmaf_rn(f, kLn2Hi, -yh)));
    const float poly = __fmaf_rn(yh, __fmaf_rn(yh, 1.f / 24.f, 1.f / 6.f), 0.5f);
    const float rest = __fmaf_rn(yh, __fmaf_rn(yh, poly, yl), yl);
    const Two t = table[i & (kTable - 1)];
    Weight w;
    w.hi = __fmaf_rn(t.hi, yh, t.hi);
    const float e = __fmaf_rn(t.hi, yh, __fsub_rn(t.hi, w.hi));
    w.lo = __fmaf_rn(t.hi, rest, __fadd_rn(__fmaf_rn(t.lo, yh, e), t.lo));
    w.n = (i >> 7) - s.ref;
    return w;
}

// the weight in units of 2^-44
__device__ __forceinline__ u64 units_of(const Weight& w) {
    const int s = min(-w.n, 63);
    const long long a = ((long long)__float2int_rn(w.hi * 16777216.f) << (kOne - 24)) + __float2int_rn(w.lo * 17592186044416.f);
    return (u64)((a + (1ll << (s - 1))) >> s);
}

// floor(total f) for 0 <= f < 1 (`left`: whether something is cut off)
__device__ __forceinline__ u64 part_of(u64 total, float f, bool& left) {
    const uint32_t b = __float_as_uint(f), e = b >> 23;
    const u64 m = e ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu;
    const int s = e ? 150 - (int)e : 149;               // f = m 2^-s, s >= 24
    const u64 lo = m * total, hi = __umul64hi(m, total);
    if (s < 64) {
        left = (lo & ((1ull << s) - 1)) != 0;
        return (lo >> s) | (hi << (64 - s));
    }
    if (s >= 128) {
        left = (lo | hi) != 0;
        return 0;
    }
    left = lo != 0 || (hi & ((1ull << (s - 64)) - 1)) != 0;
    return hi >> (s - 64);
}

// The sum that top_p asks for, at least one unit
__device__ __forceinline__ u64 needed_of(u64 total, float p) {
    bool left;
    const u64 n = part_of(total, p, left);
    return max(n + (left ? 1 : 0), 1ull);
}

// The draw: the first running sum above it is the token's.  1 and more draw the last token with weight,
// negative numbers and NaN the first.
__device__ __forceinline__ u64 drawn_at(u64 total, float u) {
    bool left;
    return u >= 1.f ? total - 1 : part_of(total, u > 0.f ? u : 0.f, left);
}

// ---- clusters ----------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* local, uint32_t rank) {
    uint32_t addr;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"((uint32_t)__cvta_generic_to_shared(local)), "r"(rank));
    return addr;
}
__device__ __forceinline__ u64 load_u64(uint32_t addr) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t load_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ u64 warp_sum(u64 x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}
__device__ __forceinline__ u64 warp_max(u64 x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
}
__device__ __forceinline__ u64 warp_scan(u64 x, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    return x;
}

struct Found {       // the bin where a running sum reaches its target
    int bin;         // -1: nowhere
    u64 above;       // the sum before the bin
};

struct Shared {
    Two table[kTable];
    uint32_t part[3][kBins];         // sums of weights, 15 bits apart; counts in the first
    u64 list[kList];
    u64 warp_a[kWarps], warp_b[kWarps];
    u64 seg_sum[kWarps], sums[2][kWarps];
    u64 best, low;                   // reduced over the cluster
    u64 few_key[32], few_weight[32]; // select_key: the entries of the bin it looks for
    uint32_t few;
    uint32_t warp_top[kWarps], warp_low[kWarps];   // keys of the largest lane maximum and of the r-th largest
    uint32_t tops[kMaxCluster * kWarps], lows[kMaxCluster * kWarps];   // the whole cluster's
    uint32_t pivot;
    uint32_t listed;
    Found found;
    u64 cut, total;                  // the result of the list (CTA 0)
    int ok, token;
    Scale scale;
    Cut first_cut;
};

// the sum over the threads up to this one, and in all
__device__ __forceinline__ u64 block_scan(Shared& S, u64 a, u64& all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    a = warp_scan(a, lane);
    __syncthreads();
    if (lane == 31) S.warp_a[warp] = a;
    __syncthreads();
    const u64 x = warp_scan(lane < kWarps ? S.warp_a[lane] : 0, lane);
    all = __shfl_sync(0xffffffffu, x, kWarps - 1);
    const u64 before = __shfl_sync(0xffffffffu, x, max(warp - 1, 0));
    return warp > 0 ? a + before : a;
}

// A row of logits, in a warp's segment [v0, v1) of the vocabulary
template <typename T, int VEC>
struct Row {
    const T* x;
    int v0, v1;

    __device__ __forceinline__ void load(float (&f)[VEC], int v, int end) const {
        if (VEC > 1 && v + VEC <= end) {
            const uint4 w = *(const uint4*)(x + v);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                f[k] = sizeof(T) == 4 ? __uint_as_float(u[k % 4])
                                      : __uint_as_float((k & 1) ? u[(k / 2) % 4] & 0xFFFF0000u : u[(k / 2) % 4] << 16);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) f[k] = v + k < end ? (float)x[v + k] : -INFINITY;
        }
    }
    static constexpr int kStep = 32 * VEC, kLoads = VEC == 8 ? 2 : 4;    // vectors in flight per lane
    static constexpr int kBatch = kLoads * VEC;
    // token of entry j of the batch from v on
    static __device__ __forceinline__ int token(int v, int j) { return v + j / VEC * kStep + j % VEC; }
    // f(values, v) for the lane's batches of kBatch tokens of [a, b) (-infinity past its end)
    template <typename F>
    __device__ __forceinline__ void batches(int a, int b, int lane, F f) const {
        for (int base = a; base < b; base += kLoads * kStep) {
            const int v = base + lane * VEC;
            float t[kLoads][VEC], flat[kBatch];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) load(t[k], v + k * kStep, b);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) flat[j] = t[j / VEC][j % VEC];
            f(flat, v);
            __syncwarp();                  // (a warp that f has split would go on in parts: up to three times slower)
        }
    }
    // f(value, token) for the tokens that `keep` (value, token) holds for (never for -infinity): few
    template <typename K, typename F>
    __device__ __forceinline__ void some(int lane, K keep, F f) const {
        batches(v0, v1, lane, [&](const float (&t)[kBatch], int v) {
            uint32_t mask = 0;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) mask |= keep(t[j], token(v, j)) ? 1u << j : 0u;
            while (mask) {                 // (read again: an index into registers is none)
                const int at = token(v, __ffs(mask) - 1);
                mask &= mask - 1;
                if (at < v1) f((float)x[at], at);
            }
        });
    }
    // the sum of f over the tokens of [a, b) that `keep` holds for; a vector without any is passed over
    template <typename K, typename F>
    __device__ __forceinline__ u64 sum(int a, int b, int lane, K keep, F f) const {
        u64 s = 0;
        batches(a, b, lane, [&](const float (&t)[kBatch], int v) {
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                bool any = false;
#pragma unroll
                for (int j = k * VEC; j < (k + 1) * VEC; ++j) any = any || keep(t[j], token(v, j));
                if (!any) continue;
#pragma unroll
                for (int j = k * VEC; j < (k + 1) * VEC; ++j) {
                    const u64 e = f(t[j]);
                    s += keep(t[j], token(v, j)) ? e : 0ull;
                }
            }
        });
        return s;
    }
    // the largest (NaN aside), read from memory with more loads in flight
    __device__ __forceinline__ float largest(int lane) const {
        constexpr int kLoads = 4;
        float top = -INFINITY;
        if constexpr (VEC == 8) {
            __nv_bfloat162 m = __floats2bfloat162_rn(-INFINITY, -INFINITY);
            int v = v0 + lane * VEC;
            for (; v + (kLoads - 1) * kStep + VEC <= v1; v += kLoads * kStep) {
                uint4 w[kLoads];
#pragma unroll
                for (int k = 0; k < kLoads; ++k) w[k] = *(const uint4*)(x + v + k * kStep);
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    const __nv_bfloat162* h = (const __nv_bfloat162*)&w[k];
                    m = __hmax2(m, __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
                }
            }
            const float2 f = __bfloat1622float2(m);
            top = fmaxf(f.x, f.y);
            for (; v < v1; v += kStep) {
                float t[VEC];
                load(t, v, v1);
#pragma unroll
                for (int j = 0; j < VEC; ++j) top = fmaxf(top, t[j]);
            }
        } else {
            for (int v = v0 + lane * VEC; v < v1; v += kLoads * kStep) {
                float t[kLoads][VEC];
#pragma unroll
                for (int k = 0; k < kLoads; ++k) load(t[k], v + k * kStep, v1);
#pragma unroll
                for (int k = 0; k < kLoads; ++k)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) top = fmaxf(top, t[k][j]);
            }
        }
        return top;
    }
};

// A pivot: of the 16 C warps' r-th largest lane maxima the m-th largest, so that at least r m tokens reach
// it.  top_k takes m of at most 10 C and r = ceil(k / m), top_p the r below and m = 8 C, for about
// 1100 candidates where tokens fall on lanes at random (512 C ln(32 / (32 - r))).  top_k takes candidates while its r is no
// larger (k up to 280 with one CTA a row, 440, 510, 560, 600, 600, 560 and 640 with more): top_k of 512 over 128 rows of
// 128,000 bf16 logits 43 us, by histograms 113; of 280 over 768 rows of 32,000 65 to 72, 156; of 640 over one row 16, 37.
__device__ __forceinline__ int pivot_rank(int cluster) {
    return cluster == 1 ? 28 : cluster == 2 ? 22 : cluster == 3 ? 17 : cluster == 4 ? 14 : cluster == 5 ? 12 : cluster == 6 ? 10 : 8;
}

__device__ __forceinline__ void clear_bins(Shared& S) {
    static_assert(offsetof(Shared, part) % 16 == 0 && sizeof S.part % (16 * kThreads) == 0, "cleared 16 bytes at a time");
#pragma unroll
    for (int i = 0; i < (int)(sizeof S.part / (16 * kThreads)); ++i) ((uint4*)S.part)[i * kThreads + threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
}

// The key at which the weights, summed over the CTA's entries in descending order of their keys from `above` on,
// reach `need` (they do; keys differ, but for weights of 0).  kList / kThreads entries per thread.  The range of the
// keys is spread over the bins; of the bin of the crossing up to 32 entries are compared with one another, where it
// holds more (11 bits a round: 6 rounds at most) its range is spread again.
constexpr int kOwn = kList / kThreads;
__device__ __forceinline__ u64 select_key(Shared& S, const u64 (&key)[kOwn], const u64 (&weight)[kOwn], u64 above, u64 need) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    u64 lo = 0, hi = ~0ull;
    for (int round = 0; round < 8; ++round) {
        u64 most = 0, low = 0;            // (low: of inverted keys)
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            if (weight[j] && key[j] >= lo && key[j] <= hi) {
                most = max(most, key[j]);
                low = max(low, ~key[j]);
            }
        most = warp_max(most);
        low = warp_max(low);
        __syncthreads();
        if (lane == 0) {
            S.warp_a[warp] = most;
            S.warp_b[warp] = low;
        }
        clear_bins(S);
        if (threadIdx.x == 0) S.few = 0;
        __syncthreads();
        hi = warp_max(lane < kWarps ? S.warp_a[lane] : 0);
        lo = ~warp_max(lane < kWarps ? S.warp_b[lane] : 0);
        const int shift = max(0, 64 - __clzll((long long)(hi - lo)) - 11);
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            if (weight[j] && key[j] >= lo && key[j] <= hi) {
                const int b = (int)((hi - key[j]) >> shift);
                const uint32_t w0 = (uint32_t)weight[j] & 0x7FFFu, w1 = (uint32_t)(weight[j] >> kLimb) & 0x7FFFu, w2 = (uint32_t)(weight[j] >> (2 * kLimb));
                if (w0) atomicAdd(&S.part[0][b], w0);
                if (w1) atomicAdd(&S.part[1][b], w1);
                if (w2) atomicAdd(&S.part[2][b], w2);
            }
        __syncthreads();
        constexpr int kPer = kBins / kThreads;
        u64 sum[kPer], own = 0, all;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int i = kPer * threadIdx.x + j;
            sum[j] = S.part[0][i] + ((u64)S.part[1][i] << kLimb) + ((u64)S.part[2][i] << (2 * kLimb));
            own += sum[j];
        }
        u64 c = above + block_scan(S, own, all) - own;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (c < need && c + sum[j] >= need) S.found = Found{kPer * (int)threadIdx.x + j, c};
            c += sum[j];
        }
        __syncthreads();
        const Found f = S.found;
        above = f.above;
        const u64 h = hi - ((u64)f.bin << shift);
        lo = h - lo >= (1ull << shift) ? h - (1ull << shift) + 1 : lo;
        hi = h;
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            if (weight[j] && key[j] >= lo && key[j] <= hi) {
                const uint32_t i = atomicAdd(&S.few, 1u);
                if (i < 32) {
                    S.few_key[i] = key[j];
                    S.few_weight[i] = weight[j];
                }
            }
        __syncthreads();
        const int n = (int)S.few;
        if (n <= 32) {
            const u64 mine = lane < n ? S.few_key[lane] : 0ull, w = lane < n ? S.few_weight[lane] : 0ull;
            u64 before = above;
            for (int j = 0; j < n; ++j) before += S.few_key[j] > mine ? S.few_weight[j] : 0ull;
            const unsigned at = __ballot_sync(0xffffffffu, lane < n && before < need && before + w >= need);
            return __shfl_sync(0xffffffffu, mine, max(__ffs(at) - 1, 0));
        }
    }
    return hi;
}

// x of the lanes in descending order
__device__ __forceinline__ uint32_t warp_sort(uint32_t x, int lane) {
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) {
            const uint32_t y = __shfl_xor_sync(0xffffffffu, x, j);
            x = ((lane & j) == 0) == ((lane & k) == 0) ? max(x, y) : min(x, y);
        }
    return x;
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, 2) sample_tokens_kernel(SampleArgs a, int cluster) {
    __shared__ __align__(16) Shared S;
    const int row = blockIdx.x / cluster, rank = (int)cluster_ctarank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int V = a.vocab;
    for (int i = threadIdx.x; i < kTable; i += kThreads) S.table[i] = g_table[i];
    if (threadIdx.x == 0) S.listed = 0;
    constexpr int kStep = 32 * VEC;
    const int warps = cluster * kWarps;
    const int seg = ((V + warps - 1) / warps + kStep - 1) / kStep * kStep;
    const int w = rank * kWarps + warp;
    Row<T, VEC> x;
    x.x = (const T*)a.logits + (size_t)row * a.logits_stride;
    x.v0 = (int)min((long long)w * seg, (long long)V);
    x.v1 = min(x.v0 + seg, V);
    // ---- the row's settings ----
    const float temp = a.temperature ? a.temperature[row] : 1.f;
    const int k = a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.f;
    const float mp = a.min_p ? a.min_p[row] : 0.f;
    const bool invalid = !(temp >= 0.f);
    if (invalid && a.err && rank == 0 && threadIdx.x == 0) atomicCAS(a.err, 0, ERR_DEVICE_CHECK | SITE_TOKEN_RANGE);
    const bool greedy = temp == 0.f || p <= 0.f;
    bool want_k = !greedy && k > 0 && k < V, want_p = !greedy && p < 1.f;
    // candidates from the lanes' maxima, where r is no more than top_p's and their number as far from the list's end
    const bool fast = want_k ? k <= 10 * cluster * pivot_rank(cluster) : want_p;
    // ---- the largest logit, and logits that enough candidates reach ----
    float top, pivot = -INFINITY;
    {
        const float mine = x.largest(lane);
        const uint32_t key = key_of(mine);
        const int most = 10 * cluster, r = want_k ? (k + most - 1) / most : pivot_rank(cluster);
        const uint32_t best = __reduce_max_sync(0xffffffffu, key);
        if (fast) {
            const uint32_t low = __shfl_sync(0xffffffffu, warp_sort(key, lane), r - 1);
            if (lane == 0) S.warp_low[warp] = low;
        }
        if (lane == 0) S.warp_top[warp] = best;
        cluster_sync();
        if (threadIdx.x < warps) {
            S.tops[threadIdx.x] = load_u32(remote(&S.warp_top[threadIdx.x % kWarps], threadIdx.x / kWarps));
            if (fast) S.lows[threadIdx.x] = load_u32(remote(&S.warp_low[threadIdx.x % kWarps], threadIdx.x / kWarps));
        }
        __syncthreads();
        uint32_t all = 0;
        for (int i = lane; i < warps; i += 32) all = max(all, S.tops[i]);
        top = value_of(__reduce_max_sync(0xffffffffu, all));
        if (fast) {
            // the m-th largest: more than m - 1 are not below it, fewer than m above; four threads a value
            static_assert(4 * kMaxCluster * kWarps <= kThreads, "four threads a value");
            const int m = want_k ? (k + r - 1) / r : 8 * cluster, i = threadIdx.x >> 2;
            const uint32_t mine = i < warps ? S.lows[i] : 0u;
            int above = 0, reach = 0;
            for (int j = threadIdx.x & 3; j < warps; j += 4) {
                const uint32_t y = S.lows[j];
                above += y > mine;
                reach += y >= mine;
            }
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
                above += __shfl_xor_sync(0xffffffffu, above, d);
                reach += __shfl_xor_sync(0xffffffffu, reach, d);
            }
            if (i < warps && above < m && reach >= m) S.pivot = mine;
            __syncthreads();
            pivot = value_of(S.pivot);
        }
    }
    const bool none = invalid || top == -INFINITY;
    const bool inf = top == INFINITY;     // infinite logits share all the weight
    // ---- the scale of the weights, and what min_p leaves ----
    if (threadIdx.x == 0) {
        Scale s{0.f, 0.f, 0.f, -130.f, 1, 0};
        if (!inf && !none && temp > 0.f) {
            // log2(e) / T as a pair: the quotient and its remainder's
            constexpr float kHi = 1.44269502162933349609375f, kLo = (float)(1.44269504088896340736 - 1.44269502162933349609375);
            const float q = fminf(__fdiv_rn(kHi, temp), FLT_MAX);
            s.hi = q;
            s.lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-q, temp, kHi), kLo), temp);
            if (!(fabsf(s.lo) <= q)) s.lo = 0.f;         // (temperatures near the ends of float32)
            const float u = __fmul_rn(top, q);
            if (fabsf(u) <= 1000.f) {
                s.ref = (__float2int_rn(u * 128.f) >> 7) + 1;
                s.least = (float)(s.ref - 128);
            } else {
                s.top = top;
                s.diff = 1;
                s.least = -127.f;
            }
        }
        S.scale = s;
        Cut c{inf ? INFINITY : -FLT_MAX, INT_MAX};
        if (mp > 0.f && !greedy && !inf && !none) {
            // the smallest logit f with f - top >= T log(min_p), in float64 (top's has), among all keys
            const double lim = mp < 1.f ? (double)temp * log((double)mp) : 0.0;
            uint32_t least = key_of(-FLT_MAX), last = key_of(top);
            while (least < last) {
                const uint32_t mid = least + (last - least) / 2;
                if ((double)value_of(mid) - (double)top >= lim) last = mid; else least = mid + 1;
            }
            c.x = value_of(least);
        }
        S.first_cut = c;
    }
    __syncthreads();
    const Scale sc = S.scale;
    Cut cut = S.first_cut;
    auto weight = [&](float f) { return weight_of(S.table, sc, inf ? 0.f : f); };
    auto units = [&](float f) { return units_of(weight(f)); };
    // a token into the CTA's list
    auto take = [&](float f, int v) {
        const uint32_t i = atomicAdd(&S.listed, 1u);
        if (i < kList) S.list[i] = rank_of(f, v);
    };
    // CTA 0: the other CTAs' lists behind its own; the number of tokens in all (more than kList: not all are there).
    // (All of them adding to one list and counter cost 40 cycles a token.)
    auto collect = [&]() {
        const int mine = lane < cluster ? (int)load_u32(remote(&S.listed, lane)) : 0;
        int at = mine;
#pragma unroll
        for (int d = 1; d < kMaxCluster; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, at, d);
            if (lane >= d) at += y;
        }
        const int n = __shfl_sync(0xffffffffu, at, kMaxCluster - 1);
        if (n <= kList && warp >= 1 && warp < cluster) {
            const int count = __shfl_sync(0xffffffffu, mine, warp), to = __shfl_sync(0xffffffffu, at, warp) - count;
            for (int i = lane; i < count; i += 32) S.list[to + i] = load_u64(remote(&S.list[i], warp));
        }
        __syncthreads();
        return n;
    };
    bool done = false;                    // the token has been given, cut and total are known
    // Few tokens are kept: the CTA's part of the distribution is cleared while the list is being worked on, and what
    // the list keeps is written into it at the end (768 rows of 32,000 float32 logits: top_k of 50 79 -> 67 us, greedy 58 -> 49).
    int own = 0;                          // the CTA's entries of the list
    auto clear = [&]() {
        if (!a.probs) return;
        float* out = a.probs + (size_t)row * a.probs_stride;
        if (VEC > 1 && !((uintptr_t)out & 15)) {
            const int end = x.v1 & ~3;    // (segments start at multiples of a vector)
            for (int v = x.v0 + 4 * lane; v < end; v += 128) *(float4*)(out + v) = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int v = max(x.v0, end) + lane; v < x.v1; v += 32) out[v] = 0.f;
        } else {
            for (int v = x.v0 + lane; v < x.v1; v += 32) out[v] = 0.f;
        }
    };
    bool listed = false;                  // the distribution is to be written from the list
    u64 total = 0;
    if (none) {
        if (a.tokens && rank == 0 && threadIdx.x == 0) a.tokens[row] = -1;
        done = true;
    } else if (greedy) {
        // ---- the lowest token that has the largest logit ----
        uint32_t at = INT_MAX;
        x.some(lane, [&](float f, int) { return f == top; }, [&](float, int v) { at = min(at, (uint32_t)v); });
        clear();
        at = __reduce_min_sync(0xffffffffu, at);
        if (lane == 0) S.warp_a[warp] = at;
        __syncthreads();
        at = __reduce_min_sync(0xffffffffu, lane < kWarps ? (uint32_t)S.warp_a[lane] : INT_MAX);
        if (threadIdx.x == 0) S.low = at;
        cluster_sync();
        at = __reduce_min_sync(0xffffffffu, lane < cluster ? (uint32_t)load_u64(remote(&S.low, lane)) : INT_MAX);
        if (a.tokens && rank == 0 && threadIdx.x == 0) a.tokens[row] = (int)at;
        cut = Cut{top, (int)at};
        total = units_of(weight(top));
        if (rank == 0 && threadIdx.x == 0) S.list[0] = rank_of(top, (int)at);
        own = rank == 0;
        done = listed = true;
    } else if (fast) {
        // ---- candidates; where top_p is first to cut, the sum of all weights too ----
        const float least = fmaxf(cut.x, pivot);
        const bool whole = least == cut.x;               // nothing else is left
        const bool sum_all = !want_k && !whole;
        x.some(lane, [&](float f, int) { return f >= least; }, take);
        if (sum_all) {
            const u64 sum = warp_sum(x.sum(x.v0, x.v1, lane, [&](float f, int) { return f >= cut.x; }, units));
            if (lane == 0) S.seg_sum[warp] = sum;
        }
        clear();
        cluster_sync();
        own = (int)S.listed;
        if (rank == 0) {
            const int n = collect();
            bool ok = n <= kList;
            u64 sum = 0, last = 0;
            if (ok) {
                u64 all = 0;                             // what top_p is a part of, where that is more than the list
                if (sum_all) {
                    for (int i = lane; i < warps; i += 32) all += load_u64(remote(&S.seg_sum[i % kWarps], i / kWarps));
                    all = warp_sum(all);
                }
                // the sum over the CTA, and how many threads' `on` holds (each array of its own: no thread is behind)
                int kept = 0;
                auto total_of = [&](u64 (&part)[kWarps], u64 y, bool on) {
                    y = warp_sum(y);
                    if (lane == 0) part[warp] = y;
                    kept = __syncthreads_count(on);
                    return warp_sum(lane < kWarps ? part[lane] : 0);
                };
                if (n <= kThreads / 2) {
                    // ---- few: each entry counts what is before it, two threads an entry ----
                    u64* weights = (u64*)&S.part[0][0];
                    static_assert(sizeof S.part >= kThreads / 2 * sizeof(u64), "scratch of the list");
                    const int e = threadIdx.x >> 1, half = threadIdx.x & 1;
                    const u64 mine = e < n ? S.list[e] : 0ull;
                    u64 w0 = e < n ? units(value_of((uint32_t)(mine >> 32))) : 0ull;
                    if (e < n && half == 0) weights[e] = w0;
                    __syncthreads();
                    int place = 0;
                    u64 before = 0;
                    for (int j = half; j < n; j += 2)
                        if (S.list[j] > mine) {
                            ++place;
                            before += weights[j];
                        }
                    place += __shfl_xor_sync(0xffffffffu, place, 1);
                    before += __shfl_xor_sync(0xffffffffu, before, 1);
                    bool stay = e < n && (!want_k || place < k);
                    sum = total_of(S.sums[0], stay && half == 0 ? w0 : 0ull, stay && half == 0);
                    if (want_p) {
                        const u64 need = needed_of(sum_all ? all : sum, p);
                        ok = sum >= need;
                        stay = stay && before < need;
                        sum = total_of(S.sums[1], stay && half == 0 ? w0 : 0ull, stay && half == 0);
                    }
                    if (e < n && half == 0 && !stay) weights[e] = 0;
                    if (stay && half == 0 && place == kept - 1) S.cut = mine;
                    if (threadIdx.x == 0) S.token = INT_MAX;
                    __syncthreads();
                    last = S.cut;
                    if (ok && a.u) {
                        // the draw: the lowest token whose running sum in index order exceeds the number
                        const u64 at = drawn_at(sum, a.u[row]);
                        u64 c = 0;
                        for (int j = half; j < n; j += 2)
                            if ((uint32_t)S.list[j] >= (uint32_t)mine) c += weights[j];
                        c += __shfl_xor_sync(0xffffffffu, c, 1);
                        if (stay && c > at) atomicMin(&S.token, token_of(mine));
                        __syncthreads();
                        if (threadIdx.x == 0) a.tokens[row] = S.token;
                    }
                } else {
                    // ---- many: histograms of the list ----
                    u64 key[kOwn], wt[kOwn];
#pragma unroll
                    for (int j = 0; j < kOwn; ++j) {
                        const int e = threadIdx.x + j * kThreads;
                        key[j] = e < n ? S.list[e] : 0ull;
                        wt[j] = e < n ? units(value_of((uint32_t)(key[j] >> 32))) : 0ull;
                    }
                    auto keep_from = [&](u64 (&part)[kWarps], u64 least) {    // and their sum
                        u64 y = 0;
#pragma unroll
                        for (int j = 0; j < kOwn; ++j) {
                            wt[j] = key[j] >= least ? wt[j] : 0ull;
                            y += wt[j];
                        }
                        return total_of(part, y, false);
                    };
                    if (want_k && n > k) {
                        u64 one[kOwn];
#pragma unroll
                        for (int j = 0; j < kOwn; ++j) one[j] = threadIdx.x + j * kThreads < n ? 1ull : 0ull;
                        last = select_key(S, key, one, 0, (u64)k);
                    }
                    sum = keep_from(S.sums[0], last);
                    if (want_p) {
                        const u64 need = needed_of(sum_all ? all : sum, p);
                        ok = sum >= need;
                        if (ok) {
                            last = select_key(S, key, wt, 0, need);
                            sum = keep_from(S.sums[1], last);
                        }
                    }
                    if (last == 0) {                     // everything in the list: the least rank
                        u64 low = 0;
#pragma unroll
                        for (int j = 0; j < kOwn; ++j)
                            if (threadIdx.x + j * kThreads < n) low = max(low, ~key[j]);
                        low = warp_max(low);
                        __syncthreads();
                        if (lane == 0) S.warp_a[warp] = low;
                        __syncthreads();
                        last = ~warp_max(lane < kWarps ? S.warp_a[lane] : 0);
                    }
                    if (ok && a.u) {
                        // (inverted indices first, so the lowest token has the largest key)
#pragma unroll
                        for (int j = 0; j < kOwn; ++j) key[j] = (key[j] << 32) | (key[j] >> 32);
                        const u64 drawn = select_key(S, key, wt, 0, drawn_at(sum, a.u[row]) + 1);
                        if (threadIdx.x == 0) a.tokens[row] = (int)~(uint32_t)(drawn >> 32);
                    }
                }
                if (threadIdx.x == 0) {
                    S.cut = last;
                    S.total = sum;
                }
            }
            if (threadIdx.x == 0) S.ok = ok;
        }
        cluster_sync();
        if (threadIdx.x == 0) S.listed = 0;
        done = load_u32(remote(&S.ok, 0)) != 0;
        if (done) {
            cut = cut_at(load_u64(remote(&S.cut, 0)));
            total = load_u64(remote(&S.total, 0));
            listed = true;
        }
    }
    // ---- otherwise: top_k, then top_p, each the rank where a sum over descending ranks reaches its target ----
    while (!done && (want_k || want_p)) {
        const bool by_count = want_k;
        const float bins = (by_count ? 1.442695f : sc.hi) * kFine;
        auto bin_of = [&](float f) {
            const float d = __fmul_rn(__fsub_rn(top, f), bins);
            return inf ? 0 : (int)fminf(d < kBins / 2 ? d : __fmaf_rn(d, kCoarse, kBins / 2 * (1.f - kCoarse)), (float)(kBins - 1));
        };
        // levels of refinement: 0, bins of x; then equal parts of the ranks lo .. hi
        int level = 0, shift = 0, bin = 0;
        u64 lo = 0, hi = ~0ull, above = 0, need = 0;
        float x_lo = 0.f, x_hi = 0.f;     // values of those ranks
        constexpr int kPer = kBins / kThreads;
        while (level < 8) {               // (11 bits of the ranks each)
            clear_bins(S);
            if (threadIdx.x == 0) S.listed = 0;
            __syncthreads();
            auto add = [&](int b, u64 u) {
                atomicAdd(&S.part[0][b], by_count ? 1u : (uint32_t)u & 0x7FFFu);
                if (!by_count) {
                    atomicAdd(&S.part[1][b], (uint32_t)(u >> kLimb) & 0x7FFFu);
                    atomicAdd(&S.part[2][b], (uint32_t)(u >> (2 * kLimb)));
                }
            };
            if (level == 0) {
                x.batches(x.v0, x.v1, lane, [&](const float (&t)[Row<T, VEC>::kBatch], int v) {
#pragma unroll
                    for (int j = 0; j < Row<T, VEC>::kBatch; ++j) {
                        const u64 u = by_count ? 0ull : units(t[j]);
                        if (cut.keeps(t[j], x.token(v, j))) add(bin_of(t[j]), u);
                    }
                });
            } else {
                x.some(lane, [&](float f, int) { return f >= x_lo && f <= x_hi; }, [&](float f, int v) {
                    const u64 r = rank_of(f, v);
                    if (r >= lo && r <= hi && cut.keeps(f, v)) add((int)((hi - r) >> shift), by_count ? 0ull : units(f));
                });
            }
            cluster_sync();
            // each CTA sums a slice of the bins over the cluster (into its list, empty yet), then all read the slices
            const int slice = (kBins + cluster - 1) / cluster;
            for (int i = threadIdx.x; i < slice && rank * slice + i < kBins; i += kThreads) {
                const int b = rank * slice + i;
                u64 s = 0;
                for (int c = 0; c < cluster; ++c)
                    s += (u64)load_u32(remote(&S.part[0][b], c)) + ((u64)load_u32(remote(&S.part[1][b], c)) << kLimb) +
                         ((u64)load_u32(remote(&S.part[2][b], c)) << (2 * kLimb));
                S.list[i] = s;
            }
            cluster_sync();
            u64 sum[kPer], own = 0;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int b = kPer * threadIdx.x + j;
                sum[j] = load_u64(remote(&S.list[b % slice], b / slice));
                own += sum[j];
            }
            u64 all_s;
            const u64 incl = block_scan(S, own, all_s);
            if (level == 0) need = by_count ? (u64)k : needed_of(all_s, p);
            if (threadIdx.x == 0) S.found = Found{-1, 0};
            __syncthreads();
            u64 s0 = above + incl - own;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                if (s0 < need && s0 + sum[j] >= need) S.found = Found{kPer * (int)threadIdx.x + j, s0};
                s0 += sum[j];
            }
            cluster_sync();               // and no histogram is cleared before all have read it
            const Found fd = S.found;
            bin = fd.bin;
            if (bin < 0) break;           // fewer than top_k tokens are left
            above = fd.above;
            if (level > 0) {
                const u64 h = hi - ((u64)bin << shift);
                lo = h - lo >= (1ull << shift) ? h - (1ull << shift) + 1 : lo;
                hi = h;
            } else {
                // the keys of the bin, by bisection: lane 0 the first of bin `bin` or above it, lane 1 the first of bin - 1
                uint32_t least = key_of(-INFINITY), last = key_of(inf ? INFINITY : top) + 1;
                while (least < last) {
                    const uint32_t mid = least + (last - least) / 2;
                    if (bin_of(value_of(mid)) <= bin - (lane & 1)) last = mid; else least = mid + 1;
                }
                lo = (u64)__shfl_sync(0xffffffffu, least, 0) << 32;
                hi = ((u64)__shfl_sync(0xffffffffu, least, 1) << 32) - 1;
            }
            x_lo = fmaxf(value_of((uint32_t)(lo >> 32)), -FLT_MAX);      // (what lies past a segment's end is -infinity)
            x_hi = value_of((uint32_t)(hi >> 32));
            // ---- the tokens of the bin: to be listed, if they are few enough ----
            u64 most = 0, low = 0;        // (low: of inverted ranks)
            x.some(lane, [&](float f, int) { return f >= x_lo && f <= x_hi; }, [&](float f, int v) {
                const u64 r = rank_of(f, v);
                if (r < lo || r > hi || !cut.keeps(f, v)) return;
                most = max(most, r);
                low = max(low, ~r);
                take(f, v);
            });
            most = warp_max(most);
            low = warp_max(low);
            if (lane == 0) {
                S.warp_a[warp] = most;
                S.warp_b[warp] = low;
            }
            __syncthreads();
            most = warp_max(lane < kWarps ? S.warp_a[lane] : 0);
            low = warp_max(lane < kWarps ? S.warp_b[lane] : 0);
            if (threadIdx.x == 0) {
                S.best = most;
                S.low = low;
            }
            cluster_sync();
            const uint32_t n = __reduce_add_sync(0xffffffffu, lane < cluster ? load_u32(remote(&S.listed, lane)) : 0u);
            hi = warp_max(lane < cluster ? load_u64(remote(&S.best, lane)) : 0);
            lo = ~warp_max(lane < cluster ? load_u64(remote(&S.low, lane)) : 0);
            if (n <= kList) break;
            ++level;
            shift = max(0, 64 - __clzll((long long)(hi - lo)) - 11);
            cluster_sync();               // all have read the counts and ranks
        }
        (by_count ? want_k : want_p) = false;
        if (bin < 0) continue;
        if (rank == 0) {
            const int n = min(collect(), kList);
            u64 key[kOwn], wt[kOwn];
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
                const int e = threadIdx.x + j * kThreads;
                key[j] = e < n ? S.list[e] : 0ull;
                wt[j] = e >= n ? 0ull : by_count ? 1ull : units(value_of((uint32_t)(key[j] >> 32)));
            }
            const u64 last = select_key(S, key, wt, above, need);
            if (threadIdx.x == 0) S.cut = last;
        }
        cluster_sync();
        if (threadIdx.x == 0) S.listed = 0;
        cut = cut_at(load_u64(remote(&S.cut, 0)));
    }
    // ---- the draw, over the segments ----
    if (!done) {
        auto keep = [&](float f, int v) { return cut.keeps(f, v); };
        const u64 s = warp_sum(x.sum(x.v0, x.v1, lane, keep, units));
        if (lane == 0) S.seg_sum[warp] = s;
        cluster_sync();
        constexpr int kPer = kMaxCluster * kWarps / 32;          // consecutive segments per lane
        u64 part[kPer], own = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int i = kPer * lane + j;
            part[j] = i < warps ? load_u64(remote(&S.seg_sum[i % kWarps], i / kWarps)) : 0;
            own += part[j];
        }
        const u64 incl = warp_scan(own, lane);
        total = __shfl_sync(0xffffffffu, incl, 31);
        if (a.u) {
            const u64 at = drawn_at(total, a.u[row]);
            // the first segment whose running sum exceeds `at`
            u64 c = incl - own, before = 0;
            int hit = -1;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                if (hit < 0 && c + part[j] > at) {
                    hit = kPer * lane + j;
                    before = c;
                }
                c += part[j];
            }
            const int from = __ffs(__ballot_sync(0xffffffffu, hit >= 0)) - 1;
            const int segment = __shfl_sync(0xffffffffu, hit, from);
            before = __shfl_sync(0xffffffffu, before, from);
            if (segment / kWarps == rank) {
                // its parts, one per warp, then the token in the one of the draw
                const int g0 = segment * seg, g1 = min(g0 + seg, V);
                const int sub = (seg / kStep + kWarps - 1) / kWarps * kStep;
                const int h0 = min(g0 + warp * sub, g1), h1 = min(h0 + sub, g1);
                const u64 q = warp_sum(x.sum(h0, h1, lane, keep, units));
                if (lane == 0) S.warp_a[warp] = q;
                __syncthreads();
                const u64 mine = lane < kWarps ? S.warp_a[lane] : 0;
                const u64 run = warp_scan(mine, lane);
                const int pick = __ffs(__ballot_sync(0xffffffffu, before + run > at)) - 1;
                if (pick == warp) {
                    u64 base = before + __shfl_sync(0xffffffffu, run - mine, pick);
                    for (int v = h0; v < h1; v += kStep) {
                        float f[VEC];
                        x.load(f, v + lane * VEC, h1);
                        u64 e[VEC], sum = 0;
#pragma unroll
                        for (int j = 0; j < VEC; ++j) {
                            const u64 y = units(f[j]);
                            sum += e[j] = keep(f[j], v + lane * VEC + j) ? y : 0ull;
                        }
                        const u64 r = warp_scan(sum, lane);
                        const unsigned over = __ballot_sync(0xffffffffu, base + r > at);
                        if (over) {
                            if (lane == __ffs(over) - 1) {
                                u64 run2 = base + r - sum;
                                int t = -1;
#pragma unroll
                                for (int j = 0; j < VEC; ++j) {
                                    run2 += e[j];
                                    if (t < 0 && run2 > at) t = v + lane * VEC + j;
                                }
                                a.tokens[row] = t;
                            }
                            break;
                        }
                        base += __shfl_sync(0xffffffffu, r, 31);
                    }
                }
            }
        }
    }
    // ---- the distribution ----
    if (a.probs) {
        float* out = a.probs + (size_t)row * a.probs_stride;
        // 2^44 / total as a pair
        const float th = (float)total, tl = none ? 0.f : (float)(long long)(total - (u64)th);
        const float q = __fdiv_rn(17592186044416.f, none ? 1.f : th);
        const float ql = __fdiv_rn(__fmaf_rn(-q, tl, __fmaf_rn(-q, th, 17592186044416.f)), none ? 1.f : th);
        auto share = [&](float f) {
            const Weight y = weight(f);
            return y.n < -126 ? 0.f : __fmaf_rn(y.hi, q, __fmaf_rn(y.hi, ql, y.lo * q)) * __uint_as_float((uint32_t)(y.n + 127) << 23);
        };
        if (listed) {
            __syncthreads();                 // behind the zeros
            for (int i = threadIdx.x; i < own; i += kThreads) {
                const u64 r = S.list[i];
                const float f = value_of((uint32_t)(r >> 32));
                if (cut.keeps(f, token_of(r))) out[token_of(r)] = share(f);
            }
        }
        const bool vec = VEC > 1 && !((uintptr_t)out & 15);
        for (int v = listed ? x.v1 : x.v0 + lane * VEC; v < x.v1; v += kStep) {
            float f[VEC];
            x.load(f, v, x.v1);
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[j] = !none && cut.keeps(f[j], v + j) ? share(f[j]) : 0.f;
            if (vec && v + VEC <= x.v1) {
#pragma unroll
                for (int j = 0; j < VEC; j += 4) *(float4*)(out + v + j) = make_float4(f[j], f[(j + 1) % VEC], f[(j + 2) % VEC], f[(j + 3) % VEC]);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    if (v + j < x.v1) out[v + j] = f[j];
            }
        }
    }
    cluster_sync();   // no CTA leaves while another may still read its shared memory
}

template <typename T, int VEC>
cudaError_t launch(const SampleArgs& a, int cluster, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.rows * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    ProfileScope ps(SPLITKV_KERNEL_SAMPLE, s);
    return cudaLaunchKernelEx(&cfg, sample_tokens_kernel<T, VEC>, a, cluster);
}

}  // namespace

cudaError_t launch_sample_tokens(const SampleArgs& a, int logits_bf16, cudaStream_t s) {
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // CTAs per row: as many as leave each 4096 tokens and run at once, or twice that where top_k or top_p are given, for
    // rows that are unequal.  128 rows of 128,000 bf16 logits with 4 CTAs a row, and with 2: settings of their own 36 us, 42; top_p of
    // 0.9 with one flat row among them 96, 120; but equal rows wait for the second round of CTAs: top_k of 50 29, 19, top_p of 0.9
    // 76, 61.  Of 32,000 float32: 31, 23; 48, 51; 25, 15; 46, 29.  (Without filters 54, 46: those keep to the fewer.)  And enough for
    // the histogram's sums.
    int cluster = std::min({kMaxCluster, (a.vocab + 4095) / 4096, std::max(1, (a.top_k || a.top_p ? 4 : 2) * sms / a.rows)});
    cluster = std::max(cluster, (a.vocab + (1 << 17) - 1) >> 17);
    // Rows that do not all begin on 16 bytes are read by elements: a vocabulary of 50,257 and of 50,256, 128 rows of bf16: no
    // filter 28 us, 26, top_k of 50 29, 26, top_p of 0.9 58, 55; 768 rows of float32: 137, 120, 73, 65, 177, 161, with
    // distributions 252, 209; one row 10, 10.
    const bool vec = a.logits_stride * (logits_bf16 ? 2 : 4) % 16 == 0 && !((uintptr_t)a.logits & 15);
    if (logits_bf16) return vec ? launch<__nv_bfloat16, 8>(a, cluster, s) : launch<__nv_bfloat16, 1>(a, cluster, s);
    return vec ? launch<float, 4>(a, cluster, s) : launch<float, 1>(a, cluster, s);
}

}  // namespace skv
