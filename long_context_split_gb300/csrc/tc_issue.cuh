// tcgen05 products issued from a warp in step, and bounded waits that stay
// inline.  Each including translation unit gets its own copies.
#pragma once

#include "tc_common.cuh"

namespace skv {
namespace {

// Bounded waits without a call: wait_bar_slow's call makes every waiter save and reload
// its live registers around it, on the critical path after each wait that is not over at once
// (expanded latent attention of two 3.6k-token prompts: 925 us with these, 975 with calls).
__device__ __forceinline__ bool spin_over(uint32_t it, unsigned long long& t0, volatile int* abort_flag, bool watch) {
    if ((it & 255) != 255) return false;
    const unsigned long long now = gtimer();
    if (t0 == 0) t0 = now;
    return (watch && *abort_flag) || now - t0 > kWaitLimitNs;
}

__device__ __forceinline__ bool spin_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, bool watch) {
    unsigned long long t0 = 0;
    for (uint32_t it = 0; !mbar_try(bar, parity); ++it)
        if (spin_over(it, t0, abort_flag, watch)) return false;
    return true;
}

// by a whole warp, converged before and after
__device__ __forceinline__ bool spin_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    unsigned long long t0 = 0;
    for (uint32_t it = 0; !__all_sync(0xffffffffu, mbar_try(bar, parity)); ++it)
        if (__any_sync(0xffffffffu, spin_over(it, t0, abort_flag, true))) return false;
    return true;
}

// the same without watching the abort flag (for draining what this CTA has in flight)
__device__ __forceinline__ bool spin_warp_drain(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    unsigned long long t0 = 0;
    for (uint32_t it = 0; !__all_sync(0xffffffffu, mbar_try(bar, parity)); ++it)
        if (__any_sync(0xffffffffu, spin_over(it, t0, abort_flag, false))) return false;
    return true;
}

// 1 in one lane of the (converged) warp, the same at every call.  Issuing from a warp in step
// with the instruction predicated on its leader keeps descriptors and addresses in uniform
// registers; in a branch of one lane each product first moves them there.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one;
}

template <int ACC>
__device__ __forceinline__ void mma_f16_if(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t cond) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "n"(ACC), "r"(cond));
}
template <int ACC>
__device__ __forceinline__ void mma_f16_ts_if(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t cond) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "l"(b), "r"(idesc), "n"(ACC), "r"(cond));
}

}  // namespace
}  // namespace skv
