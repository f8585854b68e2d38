// ptx.cuh -- barriers, asynchronous copies and programmatic launch: the PTX
// helpers that every kernel family of the library uses.
#pragma once

#include <stdint.h>

namespace sqz {
namespace tc {

constexpr uint32_t kSuspendNs = 1000000u;  // 1 ms per poll
constexpr uint32_t kWaitLimit = 2000u;

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
// Arrive (release at CTA scope: the thread's earlier shared-memory writes are
// visible to a thread whose wait on this phase succeeds).
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
}
// One bounded poll: the thread is suspended until the phase completes or
// kSuspendNs nanoseconds pass, whichever comes first (no busy spinning that
// would take issue slots from the warps doing the arithmetic).
__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendNs)
        : "memory");
    return ok != 0;
}
// Bounded wait: false if the phase did not complete within kWaitLimit polls
// (at most kWaitLimit * kSuspendNs, about two seconds).
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity) {
    for (uint32_t i = 0; i < kWaitLimit; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return false;
}
__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}
// Asynchronous 16-byte global -> shared copy (L2 only), its commit group and
// the wait for all but the newest n groups of this thread.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_wait_newest(int n) {
    switch (n) {
#define SQZ_WAIT_CASE(k) \
    case k: cp_async_wait<k>(); break;
        SQZ_WAIT_CASE(0) SQZ_WAIT_CASE(1) SQZ_WAIT_CASE(2) SQZ_WAIT_CASE(3) SQZ_WAIT_CASE(4) SQZ_WAIT_CASE(5)
        SQZ_WAIT_CASE(6) SQZ_WAIT_CASE(7) SQZ_WAIT_CASE(8) SQZ_WAIT_CASE(9) SQZ_WAIT_CASE(10) SQZ_WAIT_CASE(11)
        SQZ_WAIT_CASE(12) SQZ_WAIT_CASE(13)
#undef SQZ_WAIT_CASE
        default: cp_async_wait<14>(); break;
    }
}
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_mbar_init() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
// Programmatic dependent launch: let the next kernel of the stream start
// (its CTAs may begin on SMs this grid leaves), and wait until the previous
// kernel of the stream has finished and its writes are visible.
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace tc
}  // namespace sqz
