// What the attention kernels of the 4-bit cache share: barriers and copies in
// shared memory, and the last step of a row.
#pragma once

#include <cmath>

#include "fp4_device.cuh"

namespace fp8q {

constexpr int32_t kWaitTries = 1 << 23;   // polls of a barrier before giving up
constexpr uint32_t kSleepNs = 2000;     // of one poll, at most
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// The log2 of a weight is c * raw score - maximum + shift, with raw scores below
// 2^9 * 2688 * D.  One multiply-add for it takes the roundings of the maximum,
// with the shift and without it, into the exponent whole: half a bit where
// c * raw is 2^22 and any number of bits beyond, past what fp16 holds or down to
// no weight at all.  Rows whose c allows 2^21 have the maximum subtracted first,
// from the rounded product, which leaves the largest score at the shift exactly.
// That goes by the row alone: rows beside it are what they are beside any other.
template <int D>
__device__ __forceinline__ bool in_steps(float c) { return !(c <= 0x1p21f / (512.0f * 2688.0f * D)); }
__device__ __forceinline__ float below_most(float raw, float c, float most) {
    return __fsub_rn(__fmul_rn(raw, c), most);
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void barrier_init(uint32_t bar, uint32_t arrivals) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(arrivals) : "memory");
}

__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                 :: "r"(bar), "r"(bytes) : "memory");
}

// Sleeps until the phase ends or a while has passed; a warp that polls takes
// issue slots from those that compute.
__device__ __forceinline__ bool barrier_done(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity), "r"(kSleepNs) : "memory");
    return ok != 0;
}

__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, uint32_t bytes,
                                           uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1], %2, [%3];" :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

__device__ __forceinline__ void barrier_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}

// Waits for a phase of a barrier.  Gives up after a bounded number of polls, and
// after one when the block already has: its output is not valid then.  Behind a
// wait for data a warp goes on with what there is, in the rows and for the tokens
// of its item, to the item's end; behind one for another warp's word it asks
// told() before it uses that.  (Leaving from every wait took 1 to 3 us a call.)
__device__ __forceinline__ void barrier_wait(uint32_t bar, uint32_t parity, volatile uint32_t *gave_up,
                                             uint32_t *error, int32_t tries = kWaitTries) {
    for (int32_t left = tries; !barrier_done(bar, parity); --left)
        if (left == 0 || *gave_up) {
            *gave_up = 1;
            atomicOr(error, kFp4ErrWait);
            break;
        }
}

// Whether a whole warp may use what it has waited for: no wait of the block has
// been given up.
__device__ __forceinline__ bool told(volatile uint32_t *gave_up) {
    return __all_sync(0xFFFFFFFFu, *gave_up == 0);
}

// All threads of the warps that share barrier `id` meet; true if all say so.
// Warps that meet later on leave together, or one would wait for the others.
__device__ __forceinline__ bool agree(uint32_t id, uint32_t threads, bool ok) {
    uint32_t all;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
                 "bar.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(all) : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(ok)) : "memory");
    return all != 0;
}

// What a block that gave up has under way is given a while to land: two million
// cycles, a millisecond, before it returns its shared and tensor memory.
__device__ __forceinline__ void let_land(volatile uint32_t *gave_up) {
    if (*gave_up)
        for (const long long from = clock64(); clock64() - from < 2000000;) __nanosleep(1000);
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void load_scales(const Fp4Attention &a, float *ks, float *vs) {
    *ks = a.pools.scale_dev ? a.pools.scale_dev[0] : a.pools.k_scale;
    *vs = a.pools.scale_dev ? a.pools.scale_dev[1] : a.pools.v_scale;
}

// The fp32 output of a row from its joined sums: nothing seen gives 0, a NaN
// among the scores stays one.
__device__ __forceinline__ float row_factor(float l, float v_scale) { return l == 0.0f ? 0.0f : v_scale / l; }
__device__ __forceinline__ float row_lse(float most, float l, float shift) {
    return l == 0.0f ? -INFINITY : kLn2 * (most + (log2f(l) - shift));
}

// The place of a row of an item in `out` and `lse`.
struct RowPlace {
    int32_t token, q_head;
};
__device__ __forceinline__ RowPlace row_place(int32_t token0, int32_t row, int32_t head, int32_t group) {
    const int32_t qi = row / group;
    return {token0 + qi, head * group + (row - qi * group)};
}

}  // namespace fp8q
