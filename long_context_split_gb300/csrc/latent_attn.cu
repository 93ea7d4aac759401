// Expanded latent attention on sm_103a with tcgen05 tensor cores: each head's
// own keys (128 columns from the latent, 64 rotary columns shared by all heads)
// and values (128 columns), causal over the appended tokens.
//
// What it computes, for up to 256 query tokens of one (request, head) over one
// split of the request's history: s = scale (q_nope . k_nope + q_rope . k_rope),
// the softmax of each token's visible keys, o = sum p v -- the final row, or a
// split's partial state (normalised output, natural-log LSE) for the merge.
//
// What bounds it: the tensor pipe (2 * 320 operations per visible pair and head).  S with
// N = 64 keys reads both operands from shared memory at that memory's rate, 48 cycles a
// k-step for 32 of arithmetic, so a unit of 64 keys takes 832 cycles per 128-row tile
// instead of 640 (1 k + 2 k tokens after 14 k + 19 k at 32 heads: 686 us, 1.52
// PFLOP/s; leaving the softmax out took 692 to 681 when it was tried).  The keys and values of a
// (request, head) are read by all of its query tiles, which run together, so they come
// from L2.
//
// How: two 128-token tiles per CTA share each 64-key unit (K 64 x 192, V 64 x 128) under
// 96 KB of queries, in rings of three slots each: keys are released when both tiles' S is
// done, values when their P V is (released together, unit u + 3 waits for the softmax of
// unit u).  A tile's MMA thread issues S = Q K^T of unit u + 1 into one of two
// tensor-memory buffers before O += P V of unit u; the tile's four softmax warps (a thread
// per token) take the row maximum, keep a running maximum and sum (base 2; O is rescaled
// only when a maximum grows by more than 2^8), and write P over S as
// f16, the maximum at 2^7 to 2^15.  Each unit's values carry a power of two, which the maximum takes in and the sum takes back.  Two threads per token (eight warps a tile, maxima exchanged through shared
// memory) measured slower on two 3.6k-token prompts (944 us against 849, before the
// products were issued from a warp in step: 757 now).
// P and V are f16 because their product takes one type and f16's 11 significant
// bits keep both roundings below the output's own; Q and K stay bf16, as given.
// Sums, maxima and O are float32.  Products run in issue order, so S of unit u + 2
// replaces P of unit u only after P V of unit u has read it.
//
// A request of up to 128 new tokens fills one tile, and one tile's chain of product and softmax does not fill
// the SM: where there are enough of them (the plan's rule), a task is two heads of such a request, a
// tile per head, and the rings' units alternate between the two.
//
// Warp roles: warp 0 TMA producer and task claimer, warps 1 and 10 the tiles' MMA
// threads, warps 2..5 and 6..9 their softmax and epilogue.  Waits are bounded; on
// expiry the CTA records the error word and drains its copies and products.
#include <cuda_fp16.h>

#include <algorithm>

#include "latent.h"
#include "tc_issue.cuh"

#define SKV_LD8(taddr, r)                                                                                            \
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"                            \
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])    \
                 : "r"(taddr))

namespace skv {
namespace {

constexpr int kRows = 128;                          // query tokens per tile (tensor-memory lanes)
constexpr int kTiles = 2;
constexpr int kKeys = kLatUnit;                     // keys per unit
constexpr int kTR = 4;                              // task ring slots
constexpr int kSoftWarps = 4 * kTiles;
constexpr int kTaskConsumers = kTiles + kSoftWarps; // per tile an MMA thread and 4 softmax warps
constexpr int kThreads = (1 + kTiles + kSoftWarps) * 32;
constexpr int kIssuerWarp1 = 2 + kSoftWarps;
// P of a row's largest score lies in [2^kTop, 2^(kTop + kRescaleThreshold)], below f16's largest number: a weight
// under 2^-14 is subnormal there, with an absolute error of 2^-25, so each weight is off by at most 2^-(25 + kTop) of
// the row's largest.  The sum keeps what the product rounds away: of 2^20 keys that together hold
// 2 % beside one that holds the rest, P at 1 lost all of that share.  (With a threshold of 4 and kTop 11 rescaling took
// 1.5 % of the time of two 3.6k-token prompts, with 2 and 13 15 %; 8 and 7 cost what 8 and 0 do.)
constexpr float kRescaleThreshold = 8.0f, kTop = 7.0f;   // log2 units
static_assert(kRescaleThreshold + kTop <= 15.0f, "P within f16");
constexpr int kTmemTile = 256;                      // tensor-memory columns per tile: O (128) | S/P | S/P
constexpr int kColS = 128;
constexpr int kTmemCols = kTiles * kTmemTile;

constexpr int kQBoxes = kLatQ / 64;
constexpr int kQBox = kRows * 128;
constexpr int kRBox = kKeys * 128;                  // the unit's rotary columns
constexpr int kQTile = kQBoxes * kQBox;
constexpr int kQBytes = kTiles * kQTile;
constexpr int kKBytes = kLatSide + kRBox;            // a unit's keys: 24 KB
constexpr int kVBytes = kLatSide;                    // a unit's values: 16 KB
constexpr int NS = 3;                                // slots of the key ring, and of the value ring
// Loads arrive on two barriers per slot in turn.  A tile passes by units that it does not attend, and a parity
// cannot tell "the unit before is loading" from "this one has landed": with one barrier per slot, a value load
// passed by that took until the tile's next unit of that slot would have let it read the slot early.  With two,
// the latest phase of the barrier that a tile waits on is over when it starts to wait.
constexpr int NB = 2 * NS;

struct Bars {
    unsigned long long task_full[kTR], task_empty[kTR];
    int task_slot[kTR];
    unsigned long long k_full[NB], v_full[NB];
    unsigned long long s_full[kTiles][NS];        // per tile and key slot: S of the slot's unit is done (for its
                                                  // softmax, and the tile's release of the keys)
    unsigned long long pv_done[kTiles][NS];       // per tile and value slot: P V of the slot's unit is done (the
                                                  // tile's release of the values; O is up to date)
    unsigned long long q_full, q_empty;
    unsigned long long p_full[kTiles][2];
    unsigned long long o_full[kTiles], o_empty[kTiles];
    unsigned long long drain[kTiles];
    uint32_t tmem_base;
    int abort_flag;
};

constexpr size_t kSmemBytes = 1024 + kQBytes + (size_t)NS * (kKBytes + kVBytes) + sizeof(Bars);
static_assert(kSmemBytes <= 232448, "shared memory budget");

// what every role derives from a task
struct Task {
    int head, row0, kb, kend;
    int pair;             // 1: a tile per head; units alternate between the two
    int n_units;          // units that pass through the rings
    int rows[kTiles];     // valid tokens of each tile
    int nu[kTiles];       // units each tile attends
    LatentReq r;
};

template <bool PAIRS>
__device__ __forceinline__ Task read_task(const LatentArgs& a, int id) {
    Task t;
    const LatentTask d = a.tasks[id];
    t.r = a.reqs[d.b];
    t.head = d.head;
    t.row0 = d.row_begin;
    t.pair = PAIRS ? d.heads - 1 : 0;
    t.kb = t.kend = d.key_begin;
    t.n_units = 0;
#pragma unroll
    for (int x = 0; x < kTiles; ++x) {
        const int r0 = d.row_begin + (t.pair ? 0 : x * kRows);
        t.rows[x] = max(0, min(kRows, d.row_end - r0));
        t.nu[x] = 0;
        if (t.rows[x] > 0) {
            // keys the tile's last token may see, within the split
            const int ke = min(d.key_end, t.r.seq_len - t.r.q_len + r0 + t.rows[x]);
            if (ke > t.kb) {
                t.nu[x] = (ke - t.kb + kKeys - 1) / kKeys;
                t.kend = max(t.kend, ke);
                t.n_units = max(t.n_units, t.nu[x]);
            }
        }
    }
    t.n_units <<= t.pair;
    return t;
}

// ---- the softmax of an unmasked unit, in the fewest instructions: a thread's serial work per unit
// sets this kernel's pace (two softmax warps per scheduler), so maxima take three operands and
// scaling and sums two values per instruction ----
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpack2(uint64_t d, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float unit_max(const uint32_t (&s)[64]) {
    float m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = fmaxf(__uint_as_float(s[k]), __uint_as_float(s[4 + k]));
#pragma unroll
    for (int j = 8; j < 64; j += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = max3(m[k], __uint_as_float(s[j + k]), __uint_as_float(s[j + 4 + k]));
    return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}

// P = 2^(s c2 - base) as f16 pairs over the unit's S (key 2k in the low half of column k); the sum of P
__device__ __forceinline__ float unit_p(const uint32_t (&s)[64], float c2, float base, uint32_t pcol) {
    const uint64_t scale = pack2(c2, c2), shift = pack2(-base, -base);
    uint64_t sum[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        uint32_t pk[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int j = 16 * h + 2 * e;
            float x0, x1;
            unpack2(fma2(pack2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), scale, shift), x0, x1);
            x0 = ex2_ftz(x0);
            x1 = ex2_ftz(x1);
            sum[h] = e == 0 ? pack2(x0, x1) : add2(sum[h], pack2(x0, x1));
            const __half2 p2 = __floats2half2_rn(x0, x1);
            pk[e] = *reinterpret_cast<const uint32_t*>(&p2);
        }
        SKV_ST8(pcol + 8 * h, pk);
    }
    float a, b;
    unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a, b);
    return a + b;
}

struct Ring {
    uint32_t n = 0;
    // next task id (-1: no more); -2 when the wait gave up
    __device__ __forceinline__ int next(Bars& B, volatile int* abort_flag, int lane, bool whole_warp) {
        const int slot = (int)(n % kTR);
        const uint32_t par = (n / kTR) & 1;
        int ok = 1;
        if (lane == 0) ok = spin_bar(smem_u32(&B.task_full[slot]), par, abort_flag, true) ? 1 : 0;
        if (whole_warp) ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) return -2;
        (void)mbar_try(smem_u32(&B.task_full[slot]), par);
        const int id = ((volatile int*)B.task_slot)[slot];
        if (whole_warp) __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&B.task_empty[slot]));
        ++n;
        return id;
    }
};

// shared-memory operand of 32-byte rows in the 32-byte swizzle
__device__ __forceinline__ uint64_t desc_sw32(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (desc_sw128(addr, lbo, sbo) & ~((uint64_t)7 << 61)) | ((uint64_t)6 << 61);
}

// `bytes` contiguous bytes (a multiple of 16, both ends 16-byte aligned) into shared memory
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

// The producer's view of one ring: which tiles attend each slot's unit (only those release it),
// and the phase parities of the tiles' releases and of the slot's loads.
struct SlotUse {
    uint32_t occ = 0, par = 0, next = 0;   // bit 8 x + s: tile x attends slot s; its release's parity; the next one's
    uint32_t used = 0, loads = 0;          // bit b: a load has used the barrier; parity of its latest one

    __device__ __forceinline__ bool wait_free(unsigned long long (&done)[kTiles][NS], int s, volatile int* abort_flag) {
        for (int x = 0; x < kTiles; ++x) {
            const uint32_t bit = 1u << (8 * x + s);
            if ((occ & bit) && !spin_bar(smem_u32(&done[x][s]), (par & bit) ? 1u : 0u, abort_flag, true)) return false;
        }
        return true;
    }
    __device__ __forceinline__ void use(int b, bool tile0, bool tile1) {
        const int s = b % NS;
        for (int x = 0; x < kTiles; ++x) {
            const uint32_t bit = 1u << (8 * x + s);
            if (x ? tile1 : tile0) {
                occ |= bit;
                par = (par & ~bit) | (next & bit);
                next ^= bit;
            } else {
                occ &= ~bit;
            }
        }
        loads = (used >> b) & 1u ? loads ^ (1u << b) : loads;
        used |= 1u << b;
    }
    __device__ __forceinline__ bool drain(unsigned long long (&full)[NB], volatile int* abort_flag) {
        bool ok = true;
        for (int b = 0; b < NB; ++b)
            if ((used >> b) & 1u) ok = spin_bar(smem_u32(&full[b]), (loads >> b) & 1u, abort_flag, false) && ok;
        return ok;
    }
};

// PAIRS: some tasks are of two heads (without them, 1 to 3 % of the time of long prompts and histories)
template <bool PAIRS>
__global__ void __launch_bounds__(kThreads, 1)
latent_attention_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_r,
                        LatentArgs a) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char* sQ = smem;                              // tile x at x * kQTile
    unsigned char* sK = sQ + kQBytes;                      // slot: the keys' image, the rotary box
    unsigned char* sV = sK + NS * kKBytes;                 // slot: the values' image
    Bars& B = *(Bars*)(sV + NS * kVBytes);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kTR; ++s) {
            mbar_init(smem_u32(&B.task_full[s]), 1);
            mbar_init(smem_u32(&B.task_empty[s]), kTaskConsumers);
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(smem_u32(&B.k_full[b]), 1);
            mbar_init(smem_u32(&B.v_full[b]), 1);
        }
        for (int s = 0; s < NS; ++s) {
            for (int x = 0; x < kTiles; ++x) {
                mbar_init(smem_u32(&B.s_full[x][s]), 1);
                mbar_init(smem_u32(&B.pv_done[x][s]), 1);
            }
        }
        mbar_init(smem_u32(&B.q_full), 1);
        mbar_init(smem_u32(&B.q_empty), kTiles);
        for (int x = 0; x < kTiles; ++x) {
            for (int b = 0; b < 2; ++b) mbar_init(smem_u32(&B.p_full[x][b]), 4);
            mbar_init(smem_u32(&B.o_full[x]), 1);
            mbar_init(smem_u32(&B.o_empty[x]), 4);
            mbar_init(smem_u32(&B.drain[x]), 1);
        }
        B.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B.tmem_base)),
                     "r"(kTmemCols)
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
        // ===================== producer and task claimer (lane 0) =====================
        if (lane == 0) {
            uint32_t items = 0, qn = 0, claimed = 0;   // items: units of the tasks so far
            SlotUse ku, vu;
            bool ok = a.inject != 1;               // (test hook: publish nothing)
            while (ok) {
                const int slot = (int)(claimed % kTR);
                if (!spin_bar(smem_u32(&B.task_empty[slot]), ((claimed / kTR) & 1) ^ 1, abort_flag, true)) {
                    give_up(SITE_EMPTY_WAIT);
                    break;
                }
                int id = atomicAdd(&a.ctrl->chunk_head, 1);
                if (id >= a.num_tasks) id = -1;
                ((volatile int*)B.task_slot)[slot] = id;
                mbar_arrive(smem_u32(&B.task_full[slot]));
                ++claimed;
                if (id < 0) break;
                const Task t = read_task<PAIRS>(a, id);
                if (t.n_units == 0) continue;
                // the tiles' queries (rows past the request are other tokens, or the zero fill past
                // the tensor; they are never written back)
                if (!spin_bar(smem_u32(&B.q_empty), (qn & 1) ^ 1, abort_flag, true)) {
                    give_up(SITE_EMPTY_WAIT);
                    break;
                }
                const int tiles = t.rows[1] > 0 ? kTiles : 1;
                mbar_expect_tx(smem_u32(&B.q_full), tiles * kQTile);
                for (int x = 0; x < tiles; ++x)
                    for (int j = 0; j < kQBoxes; ++j)
                        tma_2d(smem_u32(sQ + x * kQTile + j * kQBox), &tmap_q, (t.head + (t.pair ? x : 0)) * kLatQ + 64 * j,
                               t.r.q_start + t.row0 + (t.pair ? 0 : x * kRows), smem_u32(&B.q_full));
                ++qn;
                // unit u of the rings: its first row of the copies, its image
                auto row_of = [&](int u) { return t.r.row_base + t.kb + (u >> t.pair) * kKeys; };
                auto image = [&](int u) {
                    return (const char*)a.kv + ((size_t)(t.head - a.head0 + (u & t.pair)) * a.num_blocks + row_of(u) / kKeys) * kLatImage;
                };
                auto use = [&](SlotUse& slots, int b, int u) {
                    if (t.pair) slots.use(b, (u & 1) == 0, (u & 1) == 1);
                    else slots.use(b, u < t.nu[0], u < t.nu[1]);
                };
                // Keys two units ahead of values, the order in which the tiles release them: P V of unit
                // u - 3 (the values' slot) is issued before S of unit u - 1 (the keys' slot of u + 2)
                auto load_keys = [&](int u) -> bool {
                    const int b = (int)((items + u) % NB), s = b % NS;
                    if (!ku.wait_free(B.s_full, s, abort_flag)) return false;
                    use(ku, b, u);
                    const uint32_t full = smem_u32(&B.k_full[b]), to = smem_u32(sK + s * kKBytes);
                    mbar_expect_tx(full, kKBytes);
                    bulk_copy(to, image(u), kLatSide, full);
                    tma_2d(to + kLatSide, &tmap_r, kLatC, row_of(u), full);
                    return true;
                };
                auto load_values = [&](int u) -> bool {
                    const int b = (int)((items + u) % NB), s = b % NS;
                    if (!vu.wait_free(B.pv_done, s, abort_flag)) return false;
                    use(vu, b, u);
                    const uint32_t full = smem_u32(&B.v_full[b]), to = smem_u32(sV + s * kVBytes);
                    mbar_expect_tx(full, kVBytes);
                    bulk_copy(to, image(u) + kLatSide, kLatSide, full);
                    return true;
                };
                ok = load_keys(0) && (t.n_units < 2 || load_keys(1));
                for (int u = 0; ok && u < t.n_units; ++u) ok = load_values(u) && (u + 2 >= t.n_units || load_keys(u + 2));
                if (!ok) {
                    give_up(SITE_EMPTY_WAIT);
                    break;
                }
                items += t.n_units;
            }
            // no copy may still be landing when the CTA leaves
            if (!ku.drain(B.k_full, abort_flag) || !vu.drain(B.v_full, abort_flag)) set_error(a.err, ERR_TIMEOUT | SITE_DRAIN);
            if (qn && !spin_bar(smem_u32(&B.q_full), (qn - 1) & 1, abort_flag, false)) set_error(a.err, ERR_TIMEOUT | SITE_DRAIN);
        }
        __syncwarp();
    } else if (warp == 1 || warp == kIssuerWarp1) {
        // ===================== MMA issuer of tile x (the warp in step, one elected lane issues) ==========
        const int x = warp == 1 ? 0 : 1;
        const uint32_t leader = elect_one();
        constexpr uint32_t id_s = idesc_bf16(kRows, kKeys, 0);
        constexpr uint32_t id_o = idesc_f16(kRows, kLatV, 1);     // P and V both f16
        const uint64_t qd = desc_sw128(smem_u32(sQ + x * kQTile), 16, 1024);
        const uint64_t kd0 = desc_sw32(smem_u32(sK), 16, 256), rd0 = desc_sw128(smem_u32(sK + kLatSide), 16, 1024);
        const uint64_t vd0 = desc_sw32(smem_u32(sV), kLatGroup, 256);
        const uint32_t ocol = tmem + x * kTmemTile, bufcol = ocol + kColS;
        const uint32_t k_full = smem_u32(&B.k_full[0]), v_full = smem_u32(&B.v_full[0]), s_full = smem_u32(&B.s_full[x][0]),
                       pv_done = smem_u32(&B.pv_done[x][0]), p_full = smem_u32(&B.p_full[x][0]);
        uint32_t qn = 0;
        uint32_t pc = 0;      // units this tile attended so far
        uint32_t tn = 0;      // tasks this tile finished
        // ring positions of the next S and of the next P V: barrier and parity of its loads
        uint32_t s_at = 0, s_par = 0, v_at = 0, v_par = 0;
        auto slot_of = [](uint32_t at) { return at < NS ? at : at - NS; };
        auto advance = [](uint32_t& at, uint32_t& par, uint32_t step) {   // step < NB
            at += step;
            if (at >= NB) {
                at -= NB;
                par ^= 1;
            }
        };
        bool ok = true;
        Ring ring;
        while (ok) {
            const int id = ring.next(B, abort_flag, lane, true);
            if (id == -2) { give_up(SITE_FULL_WAIT); break; }
            if (id < 0) break;
            const Task t = read_task<PAIRS>(a, id);
            if (t.n_units == 0) continue;
            const int nu = x ? t.nu[1] : t.nu[0];
            if (!spin_warp(smem_u32(&B.q_full), qn & 1, abort_flag)) { give_up(SITE_FULL_WAIT); break; }
            ++qn;
            if (nu == 0 && lane == 0) mbar_arrive(smem_u32(&B.q_empty));   // nothing to attend: release the queries
            tc_fence_after();
            // with two heads every second unit is this tile's: the first from the first, the second from the second
            const uint32_t step = 1 + t.pair, own = t.pair & x;
            advance(s_at, s_par, own);
            advance(v_at, v_par, own);
            auto issue_s = [&](uint32_t n) -> bool {       // n: the tile's unit count, which picks the S buffer
                if (!spin_warp(k_full + 8 * s_at, s_par, abort_flag)) return false;
                tc_fence_after();
                const uint32_t scol = bufcol + kKeys * (n & 1), s_slot = slot_of(s_at);
                const uint64_t kd = kd0 + (uint64_t)(s_slot * (kKBytes >> 4)), rd = rd0 + (uint64_t)(s_slot * (kKBytes >> 4));
#pragma unroll
                for (int kk = 0; kk < kLatQ / 16; ++kk) {
                    const uint64_t ad = qd + (uint64_t)((((kk >> 2) * kQBox) + (kk & 3) * 32) >> 4);
                    const uint64_t bd = kk < kLatNope / 16 ? kd + (uint64_t)((kk * kLatGroup) >> 4)
                                                           : rd + (uint64_t)(((kk & 3) * 32) >> 4);
                    if (kk == 0) mma_f16_if<0>(scol, ad, bd, id_s, leader);
                    else mma_f16_if<1>(scol, ad, bd, id_s, leader);
                }
                mma_commit_if(s_full + 8 * s_slot, leader);
                advance(s_at, s_par, step);
                return true;
            };
            auto issue_pv = [&](uint32_t n, bool first) -> bool {
                if (first && !spin_warp(smem_u32(&B.o_empty[x]), (tn & 1) ^ 1, abort_flag)) return false;
                if (!spin_warp(v_full + 8 * v_at, v_par, abort_flag)) return false;
                if (!spin_warp(p_full + 8 * (n & 1), (n >> 1) & 1, abort_flag)) return false;
                tc_fence_after();
                const uint32_t pcol = bufcol + kKeys * (n & 1), v_slot = slot_of(v_at);
                const uint64_t vd = vd0 + (uint64_t)(v_slot * (kVBytes >> 4));
                if (first) mma_f16_ts_if<0>(ocol, pcol, vd, id_o, leader);
                else mma_f16_ts_if<1>(ocol, pcol, vd, id_o, leader);
#pragma unroll
                for (int kk = 1; kk < 4; ++kk)     // 16 keys: 8 columns of P, 512 bytes of V
                    mma_f16_ts_if<1>(ocol, pcol + kk * 8, vd + (uint64_t)((kk * 512) >> 4), id_o, leader);
                mma_commit_if(pv_done + 8 * v_slot, leader);
                advance(v_at, v_par, step);
                return true;
            };
            if (nu > 0) {
                ok = issue_s(pc);
                for (int u = 0; ok && u + 1 < nu; ++u) ok = issue_s(pc + u + 1) && issue_pv(pc + u, u == 0);
                if (ok) mma_commit_if(smem_u32(&B.q_empty), leader);   // every S of the task is issued
                if (ok) ok = issue_pv(pc + nu - 1, nu == 1);
                if (!ok) { give_up(SITE_FULL_WAIT); break; }
                mma_commit_if(smem_u32(&B.o_full[x]), leader);
                pc += nu;
                ++tn;
            }
            if (own) {
                // with two heads, the second tile is one unit too far: the next task's first
                s_par ^= s_at == 0;
                v_par ^= v_at == 0;
                s_at = (s_at + NB - 1) % NB;
                v_at = (v_at + NB - 1) % NB;
            }
            // units that only the other tile attends pass by in the rings
            for (int u = nu; !t.pair && u < t.n_units; ++u) {
                advance(s_at, s_par, 1);
                advance(v_at, v_par, 1);
            }
        }
        // every product issued here completes before tensor memory is released
        mma_commit_if(smem_u32(&B.drain[x]), leader);
        if (!spin_warp_drain(smem_u32(&B.drain[x]), 0, abort_flag) && lane == 0) set_error(a.err, ERR_TIMEOUT | SITE_DRAIN);
        __syncwarp();
    } else {
        // ===================== softmax + epilogue (thread = query token of tile x) =====================
        const int x = (warp - 2) >> 2;
        const int row = ((warp & 3) << 5) + lane;                 // tensor-memory lane
        const uint32_t lane_addr = tmem + ((uint32_t)((warp & 3) << 5) << 16) + x * kTmemTile;
        const float c2 = a.scale_log2;
        uint32_t sn = 0, on = 0, item = 0;
        uint32_t ph = 0;                     // per slot: parity of this tile's next S (and of its next release)
        bool ok = true;
        Ring ring;
        while (ok) {
            const int id = ring.next(B, abort_flag, lane, true);
            if (id == -2) { give_up(SITE_FULL_WAIT); break; }
            if (id < 0) break;
            int nu, kb, i, limit, n_units, pair;
            bool valid;
            {
                const Task t = read_task<PAIRS>(a, id);
                const int trows = x ? t.rows[1] : t.rows[0];
                nu = x ? t.nu[1] : t.nu[0];
                kb = t.kb;
                n_units = t.n_units;
                pair = PAIRS ? t.pair : 0;
                valid = row < trows;
                i = t.row0 + (pair ? 0 : x * kRows) + (valid ? row : 0);        // token of the request
                // last key this token sees in the split
                limit = valid ? min(t.kend - 1, t.r.seq_len - t.r.q_len + i) : -1;
                if (trows == 0) nu = -1;
            }
            // the powers of two of the units' values, read a unit ahead (one load for the whole warp)
            const LatentScale* v_exp;
            {
                const LatentTask d = a.tasks[id];
                v_exp = a.v_exp + (size_t)(d.head - a.head0 + (pair & x)) * a.num_blocks + (a.reqs[d.b].row_base + kb) / kKeys;
            }
            const uint32_t item0 = item + (pair & x);              // its units in the rings: with two heads every second one
            item += n_units;
            if (nu < 0) continue;                                  // no token of the task in this tile
            float m = -INFINITY, l = 0.f;
            for (int u = 0; u < nu; ++u) {
                const LatentScale ve = v_exp[u];
                const int b2 = (int)(sn & 1), slot = (int)((item0 + (u << pair)) % NS);
                if (!spin_warp(smem_u32(&B.s_full[x][slot]), (ph >> slot) & 1u, abort_flag)) { give_up(SITE_FULL_WAIT); ok = false; break; }
                tc_fence_after();
                uint32_t sr[64];
                SKV_LD32(lane_addr + kColS + kKeys * b2, sr);
                SKV_LD32(lane_addr + kColS + kKeys * b2 + 32, (sr + 32));
                tc_wait_ld();
                ++sn;
                const int key0 = kb + u * kKeys;
                // warp-uniform: the tensor-memory instructions below are warp-collective
                const bool unmasked = __all_sync(0xffffffffu, key0 + kKeys - 1 <= limit);
                // The unit's values are stored times 2^-e (e = ve.exp2), so its weights enter the product as
                // 2^(s + e + kTop - m) and the sum as 2^-e of that: O and l stay sums over one reference.  m is the
                // maximum of s + e, by which the largest weighted value, not the largest weight, is
                // at the top of P's range.  (The scale is positive: the maximum is taken before it.)
                const float mx = fmaf(unmasked ? unit_max(sr) : row_max64<true>(sr, limit - key0 + 1), c2, ve.exp2);
                float scale_o = 1.f;
                bool need = false;
                if (m == -INFINITY) {
                    m = mx;
                } else if (mx > m + kRescaleThreshold) {
                    scale_o = exp2f(m - mx);
                    m = mx;
                    need = true;
                }
                if (__any_sync(0xffffffffu, need)) {
                    if (u >= 1) {
                        // P V of unit u - 1 has updated O once this tile released that unit's values; that
                        // barrier moves on only with this softmax's next P
                        const int rs = (int)((item0 + ((u - 1) << pair)) % NS);
                        if (!spin_warp(smem_u32(&B.pv_done[x][rs]), ((ph >> rs) & 1u) ^ 1u, abort_flag)) {
                            give_up(SITE_EMPTY_WAIT);
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                    }
                    l *= scale_o;
                    // (eight columns at a time: the unit's 64 scores stay in registers meanwhile)
#pragma unroll 1
                    for (int c = 0; c < kLatV; c += 8) {
                        uint32_t o[8];
                        SKV_LD8(lane_addr + c, o);
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * scale_o);
                        SKV_ST8(lane_addr + c, o);
                    }
                }
                const float base = (m == -INFINITY) ? 0.f : m - (ve.exp2 + kTop);
                const uint32_t pcol = lane_addr + kColS + kKeys * b2;
                l = fmaf(unmasked ? unit_p(sr, c2, base, pcol) : write_p16<true>(sr, c2, base, key0, limit, pcol), ve.back, l);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&B.p_full[x][b2]));
                ph ^= 1u << slot;
            }
            if (!ok) break;
            if (nu > 0) {
                if (!spin_warp(smem_u32(&B.o_full[x]), on & 1, abort_flag)) { give_up(SITE_FULL_WAIT); ok = false; break; }
                ++on;
                tc_fence_after();
            }
            // a token that sees no key of the split has an empty state; a sum that is not positive
            // over visible keys (NaN, or every score -inf) goes through, as in the formula
            const bool empty_row = limit < kb;
            const float inv = empty_row ? 0.f : a.v_scale / l;
            const float lse = empty_row ? -INFINITY : ((m - kTop) + log2f(l)) * 0.69314718055994531f;
            const LatentTask d = a.tasks[id];                      // (read again: few registers across the loop)
            const LatentReq r = a.reqs[d.b];
            const int head = d.head + (pair & x);
            const size_t orow = (size_t)(r.q_start + i) * a.heads + head;
            const size_t st = (size_t)r.state_base + ((size_t)i * a.heads + head) * r.n_splits + d.split;
            const bool direct = a.o_part == nullptr;
            for (int c = 0; c < kLatV; c += 32) {
                uint32_t o[32];
                if (nu > 0) {
                    SKV_LD32(lane_addr + c, o);
                    tc_wait_ld();
                }
                if (valid) {
                    if (nu == 0 || empty_row) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = 0u;
                    }
                    if (direct) {
                        uint4* op = (uint4*)((__nv_bfloat16*)a.out + orow * kLatV + c);
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __nv_bfloat162 p2 = __floats2bfloat162_rn(__uint_as_float(o[j + 2 * e]) * inv,
                                                                                __uint_as_float(o[j + 2 * e + 1]) * inv);
                                w[e] = *reinterpret_cast<const uint32_t*>(&p2);
                            }
                            op[j / 8] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            *(float4*)(a.o_part + st * kLatV + c + j) =
                                make_float4(__uint_as_float(o[j]) * inv, __uint_as_float(o[j + 1]) * inv,
                                            __uint_as_float(o[j + 2]) * inv, __uint_as_float(o[j + 3]) * inv);
                    }
                }
                __syncwarp();   // (the tensor-memory loads are warp-collective)
            }
            if (valid) {
                if (!direct) a.lse_part[st] = lse;
                else if (a.lse_out) a.lse_out[orow] = lse;
            }
            if (nu > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&B.o_empty[x]));
            }
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    if (threadIdx.x == 0) {
        // the last CTA resets the queue for the next call on this workspace
        __threadfence();
        if (atomicAdd(&a.ctrl->chunk_exit, 1) == (int)gridDim.x - 1) {
            atomicExch(&a.ctrl->chunk_head, 0);
            atomicExch(&a.ctrl->chunk_exit, 0);
        }
    }
}

// ---------------------------------------------------------------- host
cudaError_t make_map(CUtensorMap* m, const void* base, long long cols, long long rows, long long stride_elems, int box_rows) {
    auto enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)stride_elems * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_latent_attention(const LatentArgs& a, cudaStream_t s) {
    if (a.num_tasks <= 0) return cudaSuccess;
    const long long rows = (long long)a.num_blocks * kLatUnit;
    CUtensorMap mq, mr;
    cudaError_t e;
    if ((e = make_map(&mq, a.q, (long long)a.heads * kLatQ, a.total_q, a.q_stride, kRows)) != cudaSuccess) return e;
    if ((e = make_map(&mr, a.rows, kLatRow, rows, kLatRow, kKeys)) != cudaSuccess) return e;
    static std::atomic<uint64_t> allowed[2];
    const void* kernel = a.pairs ? (const void*)latent_attention_kernel<true> : (const void*)latent_attention_kernel<false>;
    if ((e = allow_smem(kernel, kSmemBytes, allowed[a.pairs ? 1 : 0])) != cudaSuccess) return e;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int ctas = std::min(sms, a.num_tasks);
    ProfileScope ps(SPLITKV_KERNEL_LATENT_ATTENTION, s);
    if (a.pairs) latent_attention_kernel<true><<<ctas, kThreads, kSmemBytes, s>>>(mq, mr, a);
    else latent_attention_kernel<false><<<ctas, kThreads, kSmemBytes, s>>>(mq, mr, a);
    return cudaGetLastError();
}

}  // namespace skv
