// nq_mbar.cuh -- mbarriers with bounded waits and bulk copies into shared
// memory, for the kernels whose warps are fed by them.
#pragma once

#include "nq_internal.cuh"

namespace nq {

constexpr unsigned long long kWaitNs = 2000000000ull;   // 2 s per wait

__device__ __forceinline__ uint32_t smem_u32(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// try_wait with a suspend-time hint: a waiting warp sleeps (up to 10 ms) until
// the phase completes instead of spinning and taking issue slots from the
// warps that do the work.
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(bar), "r"(parity), "r"(10000000u) : "memory");
    return ok != 0;
}
__device__ __forceinline__ unsigned long long global_ns()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// Wait for the phase of `bar` with the given parity.  Gives up after
// limit_ns (sets the CTA's abort flag and NQ_DEV_TIMEOUT) or when another
// role of the CTA has given up; returns false then.
static __device__ __noinline__ bool mbar_wait_until(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                             unsigned int *status, unsigned long long limit_ns)
{
    const unsigned long long t0 = global_ns();
    for (;;) {
        if (mbar_try(bar, parity)) return true;
        if (*abort_flag) return false;
        if (global_ns() - t0 > limit_ns) {
            *abort_flag = 1;
            set_status(status, NQ_DEV_TIMEOUT);
            return false;
        }
    }
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                          unsigned int *status, unsigned long long limit_ns = kWaitNs)
{
    return mbar_test(bar, parity) || mbar_wait_until(bar, parity, abort_flag, status, limit_ns);
}
// The same for hand-overs inside a step, where the sleep's wake-up would be most
// of the wait: try_wait without a time hint for some microseconds, then as above.
__device__ __forceinline__ bool mbar_wait_fast(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                               unsigned int *status, unsigned long long limit_ns = kWaitNs)
{
#pragma unroll 1
    for (int i = 0; i < 256; ++i) {
        uint32_t ok;
        asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                     : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        if (ok) return true;
    }
    return mbar_wait_until(bar, parity, abort_flag, status, limit_ns);
}
// A warp's wait for stage st of a ring of bulk copies of which it has the n from st on
// in flight: true on every lane once the stage is there.  Where that wait gives up, or
// one of the CTA has, false once the n copies have landed (or waits for them have run
// out too).
__device__ __forceinline__ bool ring_wait(uint32_t bar, int st, uint32_t parity, int n, int stages, volatile int *abort_flag,
                                          unsigned int *status, unsigned long long limit_ns)
{
    if (__all_sync(0xffffffffu, mbar_test(bar + 8 * st, parity))) return true;
    unsigned long long t0 = global_ns();
    bool ok = true;
#pragma unroll 1
    for (bool mine = *abort_flag == 0; mine && !mbar_try(bar + 8 * st, parity);)
        if (*abort_flag || global_ns() - t0 > limit_ns) mine = ok = false;
    ok = __all_sync(0xffffffffu, ok && *abort_flag == 0);
    if (ok) return true;
    if (*abort_flag == 0) {                   // the first to give up
        *abort_flag = 1;
        set_status(status, NQ_DEV_TIMEOUT);
    }
#pragma unroll 1
    for (t0 = global_ns(); n > 0 && global_ns() - t0 <= limit_ns;)
        if (mbar_try(bar + 8 * st, parity)) {
            --n;
            if (++st == stages) {
                st = 0;
                parity ^= 1u;
            }
        }
    __syncwarp();
    return false;
}
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

}  // namespace nq
