// The next token of each row of logits, and the distribution it is drawn from.
//
// What it computes, with m the row's largest logit and T its temperature: weights
// exp((x_i - m) / T); tokens ordered by (x descending, index ascending), the order of the
// 64-bit number "rank" = (monotone image of x's bits, inverted index).  Every filter
// keeps the tokens from some rank up, so that what is kept is one 64-bit `cut`: min_p's follows
// from m, top_k's is the k-th largest rank, top_p's the rank at which the
// weights summed in descending order reach top_p of what is left.  The draw inverts the
// distribution function over the kept tokens in index order.
//
// Arithmetic: which token a border falls on must not depend on the order of a sum, so a
// weight is an integer, round(2^44 exp(..)), and sums are integers.  Float64 runs at
// 1/64 of the float32 rate here, so exp is evaluated on pairs of float32 with a table
// of 2^(j/128) (P. T. P. Tang, "Table-driven implementation of the exponential function in
// IEEE floating-point arithmetic", ACM Trans. Math. Softw. 15, 1989): an error below 2^-40 of the
// weight, in about 40 instructions.
//
// What bounds it: one pass over the logits from memory; the rest are passes over the
// same row from L2, and their latency.  A cluster of CTAs takes a row, a warp a
// contiguous segment of the vocabulary.  Passes: the maximum; a histogram of the tokens (and
// their weights) over 1024 bins of x, which shows the bin that the cut of top_k or top_p lies in; if no more
// than 2048 tokens lie from that bin up, they are collected in shared memory, sorted, and
// everything else follows from them; otherwise those of the bin alone are (the bin is divided again
// while it holds too many, down to equal logits told apart by index), and the segments' sums
// of what is kept, then the one segment of the draw, as in the verification of drafts.
#include <cuda_bf16.h>

#include <algorithm>
#include <array>
#include <cfloat>

#include "operators.h"

namespace skv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2 * kThreads;
constexpr int kList = 2048;          // tokens that are sorted in shared memory
constexpr int kOne = 44;             // weights are in units of 2^-44 of the largest
constexpr int kTable = 128;

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

// ---- weights ---------------------------------------------------------------------
struct Scale {
    float top;       // the largest logit
    float hi, lo;    // log2(e) / T as a pair
};

struct Weight {
    float hi, lo;    // (hi + lo) 2^n, hi about 1 .. 2; n < -kOne - 1: nothing
    int n;
};

__device__ __forceinline__ Weight weight_of(const Two* table, const Scale& s, float x) {
    // d = x - top exactly, t = d log2(e) / T as a pair
    const float dh = __fsub_rn(x, s.top), bb = __fsub_rn(dh, x);
    const float dl = __fadd_rn(__fsub_rn(x, __fsub_rn(dh, bb)), __fsub_rn(-s.top, bb));
    const float th = __fmul_rn(dh, s.hi);
    const float te = __fmaf_rn(dl, s.hi, __fmaf_rn(dh, s.lo, __fmaf_rn(dh, s.hi, -th)));
    Weight w{0.f, 0.f, -1000};
    if (!(th > -126.f)) return w;     // (float32 has no smaller normal numbers)
    // th = i / 128 + f, |f| <= 1 / 256
    const float magic = 12582912.f;   // 1.5 * 2^23
    const float r = __fadd_rn(__fmul_rn(th, 128.f), magic);
    const int i = __float_as_int(r) - __float_as_int(magic);
    const float f = __fmaf_rn(__fsub_rn(r, magic), -1.f / 128.f, th);
    // y = (f + te) ln 2 = yh + yl; exp(y) - 1 = yh + rest
    constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = (float)(0.69314718055994530942 - 0.693147182464599609375);
    const float yh = __fmul_rn(f, kLn2Hi);
    const float yl = __fmaf_rn(te, kLn2Hi, __fmaf_rn(f, kLn2Lo, __fmaf_rn(f, kLn2Hi, -yh)));
    const float poly = __fmaf_rn(yh, __fmaf_rn(yh, 1.f / 24.f, 1.f / 6.f), 0.5f);
    const float rest = __fadd_rn(yl, __fmaf_rn(__fmul_rn(yh, yh), poly, __fmul_rn(yh, yl)));
    const Two t = table[i & (kTable - 1)];
    const float p = __fmul_rn(t.hi, yh), pe = __fmaf_rn(t.hi, yh, -p);
    w.hi = __fadd_rn(t.hi, p);
    const float e = __fsub_rn(p, __fsub_rn(w.hi, t.hi));
    w.lo = __fadd_rn(__fmaf_rn(t.hi, rest, __fmaf_rn(t.lo, yh, t.lo)), __fadd_rn(e, pe));
    w.n = i >> 7;
    return w;
}

// the weight in units of 2^-44
__device__ __forceinline__ u64 units_of(const Weight& w) {
    const int s = -w.n;
    if (s > kOne + 1) return 0;
    const long long a = ((long long)__float2int_rn(w.hi * 16777216.f) << (kOne - 24)) + __float2int_rn(w.lo * 17592186044416.f);
    return (u64)(s > 0 ? (a + (1ll << (s - 1))) >> s : a);
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
    u64 count;       // tokens before the bin
    u64 in;          // tokens in the bin
    u64 total;       // the sum over all bins
};

struct Shared {
    Two table[kTable];
    uint32_t count[kBins];
    uint32_t lo[kBins], hi[kBins];   // 64-bit sums of weights, halves apart
    u64 list[kList];
    u64 warp_a[kWarps], warp_b[kWarps];
    u64 seg_sum[kWarps];
    u64 best, low;                   // largest rank; range of a refinement
    uint32_t listed;
    Found found;
    u64 cut, total;                  // the result of the list (CTA 0)
    int token;
    Scale scale;                     // by thread 0: float64 is slow
    u64 first_cut;
    float inv_hi, inv_lo;
};

// sums of two values over the threads up to this one, and in all
__device__ __forceinline__ void block_scan(Shared& S, u64& a, u64& b, u64& all_a, u64& all_b) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    a = warp_scan(a, lane);
    b = warp_scan(b, lane);
    __syncthreads();
    if (lane == 31) {
        S.warp_a[warp] = a;
        S.warp_b[warp] = b;
    }
    __syncthreads();
    u64 xa = lane < kWarps ? S.warp_a[lane] : 0, xb = lane < kWarps ? S.warp_b[lane] : 0;
    xa = warp_scan(xa, lane);
    xb = warp_scan(xb, lane);
    all_a = __shfl_sync(0xffffffffu, xa, kWarps - 1);
    all_b = __shfl_sync(0xffffffffu, xb, kWarps - 1);
    const u64 ea = __shfl_sync(0xffffffffu, xa, max(warp - 1, 0)), eb = __shfl_sync(0xffffffffu, xb, max(warp - 1, 0));
    if (warp > 0) {
        a += ea;
        b += eb;
    }
}

// list[0 .. n) in descending order (a bitonic network; the rest up to a power of two is filled with 0)
__device__ __forceinline__ void sort_list(u64* list, int n) {
    int size = 2;
    while (size < n) size <<= 1;
    for (int i = n + threadIdx.x; i < size; i += kThreads) list[i] = 0;
    __syncthreads();
    for (int k = 2; k <= size; k <<= 1) {
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int i = threadIdx.x; i < size / 2; i += kThreads) {
                const int a = 2 * i - (i & (j - 1)), b = a + j;      // a has bit j clear
                const u64 x = list[a], y = list[b];
                if ((x < y) == ((a & k) == 0)) {
                    list[a] = y;
                    list[b] = x;
                }
            }
            __syncthreads();
        }
    }
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
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[k] = f[k] == f[k] ? f[k] : -INFINITY;    // NaN has no weight
    }
    // f(x, token) of every token of [a, b), a whole warp's steps at a time
    template <typename F>
    __device__ __forceinline__ void each(int a, int b, int lane, F f) const {
        constexpr int kStep = 32 * VEC, kLoads = VEC == 8 ? 2 : 4;   // vectors in flight per lane
        for (int v = a + lane * VEC; v < b; v += kLoads * kStep) {
            float t[kLoads][VEC];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) load(t[k], v + k * kStep, b);
#pragma unroll
            for (int k = 0; k < kLoads; ++k)
#pragma unroll
                for (int j = 0; j < VEC; ++j) f(t[k][j], v + k * kStep + j);
        }
    }
    template <typename F>
    __device__ __forceinline__ void each(int lane, F f) const {
        each(v0, v1, lane, f);
    }
};

// (tokens past a segment's end come as -infinity, which no cut keeps)

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
    int k = a.top_k ? a.top_k[row] : 0;
    float p = a.top_p ? a.top_p[row] : 1.f;
    const float mp = a.min_p ? a.min_p[row] : 0.f;
    const bool invalid = !(temp >= 0.f);
    if (invalid && a.err && rank == 0 && threadIdx.x == 0) atomicCAS(a.err, 0, ERR_DEVICE_CHECK | SITE_TOKEN_RANGE);
    // ---- the largest logit, the lowest token that has it ----
    u64 best = 0;
    {
        float top = -INFINITY;
        int at = -1;
        x.each(lane, [&](float f, int v) {
            if (f > top) {
                top = f;
                at = v;
            }
        });
        if (at >= 0) best = rank_of(top, at);
        best = warp_max(best);
        if (lane == 0) S.warp_a[warp] = best;
        __syncthreads();
        best = warp_max(lane < kWarps ? S.warp_a[lane] : 0);
        if (threadIdx.x == 0) S.best = best;
        cluster_sync();
        best = warp_max(lane < cluster ? load_u64(remote(&S.best, lane)) : 0);
    }
    const bool none = best == 0 || invalid;
    const float top = none ? 0.f : value_of((uint32_t)(best >> 32));
    const bool inf = isinf(top);          // infinite logits share all the weight
    // ---- the scale of the weights, and what min_p leaves ----
    if (threadIdx.x == 0) {
        Scale s{inf ? 0.f : top, 0.f, 0.f};
        if (!inf && temp > 0.f) {
            const double c = fmin(1.4426950408889634 / (double)temp, (double)FLT_MAX);
            s.hi = (float)c;
            s.lo = (float)(c - (double)s.hi);
        }
        S.scale = s;
        uint32_t least = key_of(inf ? INFINITY : -FLT_MAX);
        if (mp > 0.f && !inf && !none) {
            // the smallest key whose value f has f - top >= T log(min_p), in float64 (the top's has)
            const double lim = mp < 1.f ? (double)temp * log((double)mp) : 0.0;
            uint32_t last = key_of(top);
            while (least < last) {
                const uint32_t mid = least + (last - least) / 2;
                if ((double)value_of(mid) - (double)top >= lim) last = mid; else least = mid + 1;
            }
        }
        S.first_cut = temp == 0.f || p <= 0.f ? best : (u64)least << 32;
    }
    __syncthreads();
    const Scale sc = S.scale;
    u64 cut = S.first_cut;
    auto weight = [&](float f) { return weight_of(S.table, sc, inf ? 0.f : f); };
    bool want_k = !none && cut != best && k > 0 && k < V, want_p = !none && cut != best && p < 1.f;
    bool done = false;                    // the list has given the token, and cut and total
    u64 total = 0;
    // ---- top_k, then top_p: the rank where a sum over descending ranks reaches its target ----
    while (want_k || want_p) {
        const bool by_count = want_k;
        const float bins = sc.hi * 20.f;  // bins of 1/20 of a factor of two in weight
        auto bin_of = [&](float f) { return (int)fminf(__fmul_rn(__fsub_rn(sc.top, f), bins), (float)(kBins - 1)); };
        // levels of refinement: 0, bins of x; then equal parts of the ranks lo .. hi
        int level = 0, shift = 0, bin = 0;
        u64 lo = 0, hi = ~0ull, above = 0, need = 0, n_above = 0;
        Found fd;
        bool all = false;                 // the list holds everything from the bin up
        while (true) {
            for (int i = threadIdx.x; i < kBins; i += kThreads) S.count[i] = S.lo[i] = S.hi[i] = 0;
            __syncthreads();
            x.each(lane, [&](float f, int v) {
                const u64 r = rank_of(f, v);
                if (r < cut || r < lo || r > hi) return;
                const int b = level == 0 ? (inf ? 0 : bin_of(f)) : (int)((hi - r) >> shift);
                atomicAdd(&S.count[b], 1u);
                if (!by_count) {
                    const u64 u = units_of(weight(f));
                    if (u) {
                        const uint32_t ul = (uint32_t)u, old = atomicAdd(&S.lo[b], ul);
                        atomicAdd(&S.hi[b], (uint32_t)(u >> 32) + (old + ul < old ? 1u : 0u));
                    }
                }
            });
            cluster_sync();
            u64 cnt[2] = {0, 0}, sum[2] = {0, 0};
            for (int c = 0; c < cluster; ++c)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int i = 2 * threadIdx.x + j;
                    const u64 n = load_u32(remote(&S.count[i], c));
                    cnt[j] += n;
                    sum[j] += by_count ? n : (u64)load_u32(remote(&S.lo[i], c)) + ((u64)load_u32(remote(&S.hi[i], c)) << 32);
                }
            u64 ca = cnt[0] + cnt[1], sa = sum[0] + sum[1], all_c, all_s;
            block_scan(S, ca, sa, all_c, all_s);
            if (level == 0) {
                if (by_count) {
                    need = (u64)k;
                } else {
                    bool left;
                    need = part_of(all_s, p, left);
                    need = max(need + (left ? 1 : 0), 1ull);
                }
            }
            if (threadIdx.x == 0) S.found = Found{-1, 0, 0, 0, all_s};
            __syncthreads();
            {
                u64 s0 = above + sa - sum[0] - sum[1], c0 = n_above + ca - cnt[0] - cnt[1];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (s0 < need && s0 + sum[j] >= need) S.found = Found{2 * (int)threadIdx.x + j, s0, c0, cnt[j], all_s};
                    s0 += sum[j];
                    c0 += cnt[j];
                }
            }
            cluster_sync();               // and no histogram is cleared before all have read it
            fd = S.found;
            if (fd.bin < 0) break;        // fewer than top_k tokens are left
            above = fd.above;
            n_above = fd.count;
            if (level == 0) {
                bin = fd.bin;
                all = fd.count + fd.in <= kList;
                if (all || fd.in <= kList) break;
                // the range of the bin's ranks
                u64 top = 0, low = 0;     // (low: of inverted ranks)
                x.each(lane, [&](float f, int v) {
                    const u64 r = rank_of(f, v);
                    if (r >= cut && (inf ? 0 : bin_of(f)) == bin) {
                        top = max(top, r);
                        low = max(low, ~r);
                    }
                });
                top = warp_max(top);
                low = warp_max(low);
                if (lane == 0) {
                    S.warp_a[warp] = top;
                    S.warp_b[warp] = low;
                }
                __syncthreads();
                top = warp_max(lane < kWarps ? S.warp_a[lane] : 0);
                low = warp_max(lane < kWarps ? S.warp_b[lane] : 0);
                if (threadIdx.x == 0) {
                    S.best = top;
                    S.low = low;
                }
                cluster_sync();
                hi = warp_max(lane < cluster ? load_u64(remote(&S.best, lane)) : 0);
                lo = ~warp_max(lane < cluster ? load_u64(remote(&S.low, lane)) : 0);
            } else {
                const u64 h = hi - ((u64)fd.bin << shift);
                lo = h - lo >= (1ull << shift) ? h - (1ull << shift) + 1 : lo;
                hi = h;
                if (fd.in <= kList) break;
            }
            ++level;
            shift = max(0, 64 - __clzll((long long)(hi - lo)) - 10);
        }
        if (fd.bin < 0) {
            want_k = false;
            continue;
        }
        // ---- the tokens concerned, in CTA 0 ----
        x.each(lane, [&](float f, int v) {
            const u64 r = rank_of(f, v);
            if (r < cut || r < lo || r > hi) return;
            if (level == 0) {
                const int b = inf ? 0 : bin_of(f);
                if (all ? b > bin : b != bin) return;
            }
            uint32_t i;
            asm volatile("atom.shared::cluster.add.u32 %0, [%1], 1;" : "=r"(i) : "r"(remote(&S.listed, 0)) : "memory");
            if (i < kList)
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(&S.list[i], 0)), "l"(r) : "memory");
        });
        cluster_sync();
        if (rank == 0) {
            int n = (int)min(S.listed, (uint32_t)kList);
            sort_list(S.list, n);
            const u64 start = all ? 0 : above;    // of the sum before the list
            // entry e's weight, 4 consecutive entries per thread
            auto entry = [&](int e) { return e < n ? units_of(weight(value_of((uint32_t)(S.list[e] >> 32)))) : 0ull; };
            auto reach = [&](u64 from, u64 to) {  // entries up to the one at which the weights reach `to`
                u64 part[kList / kThreads], own = 0, zero = 0, t0, t1;
#pragma unroll
                for (int j = 0; j < kList / kThreads; ++j) own += part[j] = entry(threadIdx.x * (kList / kThreads) + j);
                u64 incl = own;
                if (threadIdx.x == 0) S.token = n;
                block_scan(S, incl, zero, t0, t1);
                u64 c = from + incl - own;
#pragma unroll
                for (int j = 0; j < kList / kThreads; ++j) {
                    if (c < to && c + part[j] >= to) S.token = threadIdx.x * (kList / kThreads) + j + 1;
                    c += part[j];
                }
                __syncthreads();
                const int r = S.token;
                __syncthreads();
                return r;
            };
            auto sum_all = [&]() {
                u64 own = 0, zero = 0, t0, t1;
#pragma unroll
                for (int j = 0; j < kList / kThreads; ++j) own += entry(threadIdx.x * (kList / kThreads) + j);
                block_scan(S, own, zero, t0, t1);
                return t0;
            };
            if (by_count) n = (int)(need - start);
            else n = reach(start, need);
            if (all && by_count && want_p) {
                bool left;
                u64 to = part_of(sum_all(), p, left);
                n = reach(0, max(to + (left ? 1 : 0), 1ull));
            }
            u64 end = S.list[n - 1], sum = 0;
            if (all) {
                sum = sum_all();
                __syncthreads();
                if (a.u) {
                    // ---- the draw, over the kept tokens in index order ----
                    for (int i = threadIdx.x; i < n; i += kThreads) S.list[i] = (S.list[i] << 32) | (S.list[i] >> 32);
                    __syncthreads();
                    sort_list(S.list, n);         // (inverted indices, so the lowest token first)
                    for (int i = threadIdx.x; i < n; i += kThreads) S.list[i] = (S.list[i] << 32) | (S.list[i] >> 32);
                    __syncthreads();
                    const float u = a.u[row];
                    const int e = reach(0, drawn_at(sum, u) + 1);
                    if (threadIdx.x == 0) a.tokens[row] = token_of(S.list[e - 1]);
                }
            }
            if (threadIdx.x == 0) {
                S.cut = end;
                S.total = sum;
                S.listed = 0;
            }
        }
        cluster_sync();
        cut = load_u64(remote(&S.cut, 0));
        total = load_u64(remote(&S.total, 0));
        if (all) {
            done = true;
            break;
        }
        if (by_count) want_k = false;
        else want_p = false;
    }
    // ---- the draw, over the segments ----
    if (none) {
        if (a.tokens && rank == 0 && threadIdx.x == 0) a.tokens[row] = -1;
    } else if (cut == best) {
        total = 1ull << kOne;
        if (a.tokens && rank == 0 && threadIdx.x == 0) a.tokens[row] = token_of(best);
    } else if (!done) {
        auto kept = [&](float f, int v) { return rank_of(f, v) >= cut ? units_of(weight(f)) : 0ull; };
        u64 s = 0;
        x.each(lane, [&](float f, int v) { s += kept(f, v); });
        s = warp_sum(s);
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
            const float u = a.u[row];
            const u64 at = drawn_at(total, u);
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
                u64 q = 0;
                x.each(h0, h1, lane, [&](float f, int v) { q += kept(f, v); });
                q = warp_sum(q);
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
                        for (int j = 0; j < VEC; ++j) sum += e[j] = kept(f[j], v + lane * VEC + j);
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
        if (threadIdx.x == 0 && !none) {
            const double d = (double)(1ull << kOne) / (double)total;
            S.inv_hi = (float)d;
            S.inv_lo = (float)(d - (double)S.inv_hi);
        }
        __syncthreads();
        const float ih = S.inv_hi, il = S.inv_lo;
        const bool vec = VEC > 1 && !((uintptr_t)out & 15);
        for (int v = x.v0 + lane * VEC; v < x.v1; v += kStep) {
            float f[VEC];
            x.load(f, v, x.v1);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float q = 0.f;
                if (!none && rank_of(f[j], v + j) >= cut) {
                    const Weight y = weight(f[j]);
                    if (y.n >= -126) q = __fmaf_rn(y.hi, ih, __fmaf_rn(y.hi, il, y.lo * ih)) * __uint_as_float((uint32_t)(y.n + 127) << 23);
                }
                f[j] = q;
            }
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
    // CTAs per row: as many as leave each 4096 tokens and run at once (1.6 an SM fit in clusters)
    const int cluster = std::min({kMaxCluster, (a.vocab + 4095) / 4096, std::max(1, 8 * sms / 5 / a.rows)});
    const bool vec = a.logits_stride * (logits_bf16 ? 2 : 4) % 16 == 0 && !((uintptr_t)a.logits & 15);
    if (logits_bf16) return vec ? launch<__nv_bfloat16, 8>(a, cluster, s) : launch<__nv_bfloat16, 1>(a, cluster, s);
    return vec ? launch<float, 4>(a, cluster, s) : launch<float, 1>(a, cluster, s);
}

}  // namespace skv
