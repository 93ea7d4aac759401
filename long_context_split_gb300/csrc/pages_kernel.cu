// Pages and slots of a batch from its lengths.
//
// What it computes: need_b = ceil(len_b / P); a request that holds more pages gives
// back_b = held_b - need_b of them to the free list, one that holds fewer takes
// grow_b = need_b - held_b from its end.  With the exclusive sums over requests
// B_b of back and G_b of grow, n free pages before the call and f given back:
// page j of b's surplus becomes list entry n + B_b + j, and b's j-th new page is list entry
// n + f - 1 - (G_b + j) -- itself a page just given back where that is n or more.  So every id
// is found from the two sums alone, without an order among threads.
//
// What bounds it: latency (a batch's lengths -> sums -> ids -> table), and for prompts
// the slots, 8 bytes a token.  One cluster of up to 8 CTAs does the call in one
// launch (many slots take another, on all SMs): each CTA sums the whole batch for itself (a few thousand requests at most), a
// cluster barrier stands between the last read of held / free_count and their
// update in place, then all threads share out ids and slots.  256 requests, 250 slots: 6.9 us; 192 prompts,
// 213k slots: 12.0.
#include <algorithm>
#include <climits>

#include "operators.h"

namespace skv {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// how many of at[0 .. n - 1] (non-decreasing) are <= x
__device__ __forceinline__ int upper(const int* at, int n, int x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x) lo = mid + 1; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int clip(long long x) { return (int)min(x, (long long)INT_MAX); }

// The slot of row r of request b's rows lo .. hi - 1, `page_of(j)` the request's page j or -1
template <typename F>
__device__ __forceinline__ long long slot_of(const PagesArgs& a, int lo, int hi, int len, int r, int& page_j, int& page, F page_of) {
    if (lo < 0 || lo > r || hi > a.num_slots || hi - lo > len) return -1;
    const int pos = len - (hi - r), j = pos / a.page_size;
    if (j != page_j) {
        page_j = j;
        page = page_of(j);
    }
    return page < 0 ? -1 : (long long)page * a.page_size + (pos - j * a.page_size);
}

// Many slots, from the tables that assign_pages_kernel has just written: kSlots consecutive ones per thread, one
// search of the rows' bounds for all of them.
constexpr int kSlots = 8, kSlotThreads = 256;
__global__ void __launch_bounds__(kSlotThreads) slots_kernel(PagesArgs a) {
    extern __shared__ int qo[];
    for (int i = threadIdx.x; i <= a.batch; i += kSlotThreads) qo[i] = a.qo_indptr[i];
    __syncthreads();
    const int rows = min(a.num_slots, qo[a.batch]);
    const long long r0 = ((long long)blockIdx.x * kSlotThreads + threadIdx.x) * kSlots;
    if (r0 >= rows) return;
    int b = upper(qo + 1, a.batch, (int)r0), page_j = -1, page = -1, len = 0, held = 0, known = -1;
#pragma unroll
    for (int c = 0; c < kSlots; ++c) {
        const int r = (int)r0 + c;
        if (r >= rows) break;
        while (b < a.batch && qo[b + 1] <= r) ++b;
        if (b < a.batch && b != known) {
            known = b;
            page_j = -1;
            len = max(0, a.seq_lens[b]);
            held = a.held_out[b];
        }
        a.slots[r] = b < a.batch ? slot_of(a, qo[b], qo[b + 1], len, r, page_j, page, [&](int j) {
            return j < held ? a.page_table[(size_t)b * a.max_pages + j] : -1;
        }) : -1;
    }
}

// With few slots those too, one per thread and step
__global__ void __launch_bounds__(kThreads, 1) assign_pages_kernel(PagesArgs a, int cluster, int with_slots) {
    extern __shared__ int smem[];
    __shared__ long long warp_sum[2][kWarps];
    const int B = a.batch, P = a.page_size;
    int* grow_at = smem;               // inclusive sums: entry b covers requests 0 .. b
    int* back_at = smem + B;
    int* held = smem + 2 * B;          // before the call
    int* qo = smem + 3 * B;            // [B + 1]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x;
    int bad = 0;                       // what this thread found out of range
    auto tokens = [&](int b) { return max(0, a.seq_lens[b]); };
    auto pages = [&](int len) { return (int)(((long long)len + P - 1) / P); };
    // ---- both sums over the batch, every CTA for itself ----
    long long grow_base = 0, back_base = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        long long grow = 0, back = 0;
        if (b < B) {
            const int len = a.seq_lens[b], h = a.held[b];
            const int have = min(max(h, 0), a.max_pages), need = pages(max(0, len));
            if (len < 0 || have != h) bad = SITE_TOKEN_RANGE;
            held[b] = have;
            if (need > a.max_pages) bad = SITE_TOKEN_RANGE;   // keeps what it holds
            else if (need > have) grow = need - have;
            else back = have - need;
            if (a.qo_indptr) qo[b] = a.qo_indptr[b];
        }
        long long gs = grow, bs = back;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, gs, d), y = __shfl_up_sync(0xffffffffu, bs, d);
            if (lane >= d) { gs += x; bs += y; }
        }
        if (lane == 31) { warp_sum[0][warp] = gs; warp_sum[1][warp] = bs; }
        __syncthreads();
        if (warp == 0) {
            long long x = warp_sum[0][lane], y = warp_sum[1][lane];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, x, d), v = __shfl_up_sync(0xffffffffu, y, d);
                if (lane >= d) { x += u; y += v; }
            }
            warp_sum[0][lane] = x;
            warp_sum[1][lane] = y;
        }
        __syncthreads();
        if (b < B) {
            grow_at[b] = clip(grow_base + gs + (warp ? warp_sum[0][warp - 1] : 0));
            back_at[b] = clip(back_base + bs + (warp ? warp_sum[1][warp - 1] : 0));
        }
        grow_base += warp_sum[0][kWarps - 1];
        back_base += warp_sum[1][kWarps - 1];
        __syncthreads();
    }
    const int n0 = *a.free_count, n = min(max(n0, 0), a.capacity);
    if (n != n0) bad = SITE_TOKEN_RANGE;
    const int given = (int)min(back_base, (long long)(a.capacity - n));
    if (given < back_base) bad = SITE_TOKEN_RANGE;
    const int avail = n + given;
    if (a.qo_indptr && threadIdx.x == 0) qo[B] = a.qo_indptr[B];
    // every read of held and free_count, and every CTA's arrays, are done
    cluster_sync();
    // a growing request is served while the sum up to it is available: the served ones come first
    const int served = upper(grow_at, B, avail);            // requests 0 .. served - 1 (growing or not)
    const int taken = served > 0 ? grow_at[served - 1] : 0;
    auto given_page = [&](int i) {                          // i-th page given back
        const int b = upper(back_at, B, i);
        const int surplus = back_at[b] - (b ? back_at[b - 1] : 0);
        return a.page_table[(size_t)b * a.max_pages + (held[b] - surplus) + (i - (back_at[b] - surplus))];
    };
    auto taken_page = [&](int k) {                          // k-th page taken
        const int at = avail - 1 - k;
        return at >= n ? given_page(at - n) : a.free_pages[at];
    };
    const int t = rank * kThreads + threadIdx.x, step = cluster * kThreads;
    for (int b = t; b < B; b += step) {
        const int len = tokens(b), need = pages(len);
        const bool grows = need > held[b] && need <= a.max_pages;
        const bool refused = need > a.max_pages || (grows && b >= served);
        if (refused) bad = SITE_TOKEN_RANGE;
        a.held_out[b] = refused ? held[b] : need;
        if (a.qo_indptr) {
            const int lo = qo[b], hi = qo[b + 1];
            if (lo < 0 || hi < lo || hi > a.num_slots || hi - lo > len) bad = SITE_TOKEN_RANGE;
        }
    }
    if (t == 0) *a.free_count_out = avail - taken;
    for (int i = t; i < given; i += step) a.free_pages[n + i] = given_page(i);
    for (int k = t; k < taken; k += step) {
        const int b = upper(grow_at, B, k), k0 = b ? grow_at[b - 1] : 0;
        a.page_table[(size_t)b * a.max_pages + held[b] + (k - k0)] = taken_page(k);
    }
    // ---- slots: a token's page is one that its request held, or one just taken ----
    if (with_slots) {
        const int rows = min(a.num_slots, qo[B]);
        for (int r = t; r < rows; r += step) {
            const int b = upper(qo + 1, B, r);
            int page_j = -1, page = -1;
            a.slots[r] = b < B ? slot_of(a, qo[b], qo[b + 1], tokens(b), r, page_j, page, [&](int j) {
                const int need = pages(tokens(b));
                if (j < held[b]) return a.page_table[(size_t)b * a.max_pages + j];
                return need <= a.max_pages && b < served ? taken_page((b ? grow_at[b - 1] : 0) + j - held[b]) : -1;
            }) : -1;
        }
    }
    if (bad && a.err) atomicCAS(a.err, 0, ERR_DEVICE_CHECK | bad);
}

}  // namespace

cudaError_t launch_assign_pages(const PagesArgs& a, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem((const void*)assign_pages_kernel, ((size_t)4 * kMaxPagesBatch + 1) * sizeof(int), done);
    if (e != cudaSuccess) return e;
    // up to 4096 slots within the call's one launch, more on all SMs behind it (239k slots: 34 us in one launch of 8 CTAs)
    const bool apart = a.num_slots > 4096;
    const int cluster = std::min(kMaxCluster, std::max(1, (apart ? a.num_slots / 16 : a.num_slots) / kThreads));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = ((size_t)4 * a.batch + 1) * sizeof(int);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    ProfileScope ps(SPLITKV_KERNEL_ASSIGN_PAGES, s);
    e = cudaLaunchKernelEx(&cfg, assign_pages_kernel, a, cluster, apart ? 0 : 1);
    if (e != cudaSuccess || !apart) return e;
    const int per = kSlots * kSlotThreads;
    slots_kernel<<<(unsigned)(((long long)a.num_slots + per - 1) / per), kSlotThreads, ((size_t)a.batch + 1) * sizeof(int), s>>>(a);
    return cudaGetLastError();
}

}  // namespace skv
