// fp8_common.cuh -- device helpers shared by the block-scaled 8-bit kernels:
// tensor maps' tile loads, tcgen05 matrix instructions on 8-bit operands and
// their accumulators in tensor memory, bounded waits, cluster barriers.
//
// Operand tiles.  A tile is 128 bytes (128 codes, one scale block) of K by R
// rows, brought in by TMA with the 128-byte swizzle: row r at byte 128 r, its
// 16-byte chunk c at chunk c ^ (r % 8).  The matrix descriptor below says so:
// K-major, groups of 8 rows 1024 bytes apart, tiles 1024-byte aligned.  One
// tcgen05.mma takes 32 codes of K; the next 32 start 32 bytes further into
// the swizzle atom.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"
#include "ptx.cuh"

namespace sqz {
namespace f8 {

using tc::cp_async_commit;
using tc::cp_async_wait;
using tc::fence_mbar_init;
using tc::mbar_arrive;
using tc::mbar_expect_tx;
using tc::mbar_init;
using tc::pdl_launch_dependents;
using tc::pdl_wait_previous;
using tc::smem_u32;

constexpr int kBlockK = 128;          // codes of K per scale block = bytes of a tile row
constexpr int kTileBytes = 128 * 128; // a tile of 128 rows

enum OutType : int { kF16 = 0, kBF16 = 1, kF32 = 2 };

// Waits are bounded (kWaitCycles, about two seconds).  A wait that gives up
// sets `*dead` (shared memory), which ends the other waits of the CTA too; the
// kernel then leaves in order.  The polls carry no suspend-time hint: these
// barriers complete every few hundred cycles, and a hinted wait wakes later.
constexpr long long kWaitCycles = 4000000000ll;

__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// The same without suspending the thread (try_wait holds it for microseconds
// when the phase is not complete).
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* dead) {
    const long long t0 = clock64();
    while (!mbar_poll(bar, parity)) {
        if (*dead) return false;
        if (clock64() - t0 > kWaitCycles) {
            *dead = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait_alive(uint64_t* bar, uint32_t parity, volatile int* dead) {
    return mbar_poll(bar, parity) || wait_long(bar, parity, dead);
}

// A whole warp's wait; the answer is the same in every lane, and the compiler
// sees that it is.  The roles that issue copies and matrix instructions run
// their loops with all lanes and elect one for the instruction itself: their
// operands then stay in uniform registers.  (Under `if (lane == 0)` each operand
// is moved there first: four matrix instructions took over 300 cycles to issue.)
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* dead) {
    return __all_sync(0xffffffffu, wait_alive(bar, parity, dead));
}
// Two barriers that one step waits for, asked one step ahead: the answer to a
// poll takes about as long as issuing a block's matrix instructions, so the
// polls for the next step go out before the instructions of this one, and the
// step only waits where they came back empty.
struct Ahead {
    bool a_there, b_there;
    __device__ __forceinline__ void ask(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb) {
        a_there = mbar_test(a, pa);
        b_there = mbar_test(b, pb);
    }
    __device__ __forceinline__ bool wait(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, volatile int* dead) {
        bool ok = true;
        if (!__all_sync(0xffffffffu, a_there)) ok = wait_warp(a, pa, dead);
        if (ok && !__all_sync(0xffffffffu, b_there)) ok = wait_warp(b, pb, dead);
        return ok;
    }
};
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one != 0;
}

// After a wait gave up: time (100 ms) for the thread's own copies and matrix
// instructions in flight to end before the CTA frees its memory and leaves.
__device__ __forceinline__ void let_copies_land() {
    for (int i = 0; i < 100; ++i) __nanosleep(1000000);
}

// Loads of what the previous kernel of the stream may have written (a kernel that
// is launched early is there before that one has ended), or of what this one
// writes later: plain loads (the non-coherent path is for memory that stays as
// it is as long as the kernel lives), and volatile, so that they stay behind
// waits and before barriers.
__device__ __forceinline__ uint16_t ld_u16(const void* p) {
    uint16_t v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ld_u32(const void* p) {
    uint32_t v;
    asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ld_u64(const void* p) {
    uint2 v;
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 ld_u128(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 ld_once_u128(const void* p) {  // read once: kept out of L1
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// ------------------------------------------------------------------- TMA
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// Asynchronous 4-byte copy to shared memory.  (Lanes that have nothing to copy
// stay out: lanes copying from one address, even zero bytes, go one by one.)
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// The thread's arrival on `bar`, posted when its copies so far have landed (it
// counts as one of the barrier's expected arrivals).
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// --------------------------------------------------------------- tcgen05
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Descriptor of a swizzled K-major operand tile at a shared-memory address
// (bits 0-13 address / 16, 32-45 byte distance of 8-row groups / 16 = 64,
// 46-47 version 1, 61-63 layout 2 = 128-byte swizzle).
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor of kind::f8f6f4, fp32 accumulators, both operands
// K-major: bits 4-5 accumulator type 1, 7-9 / 10-12 operand formats (0 e4m3,
// 1 e5m2), 17-22 N / 8, 24-28 M / 16.
__host__ __device__ inline uint32_t instr_desc(int a_format, int b_format, int m, int n) {
    return (1u << 4) | ((uint32_t)a_format << 7) | ((uint32_t)b_format << 10) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1 : 0)
        : "memory");
}
// A whole 128-code block of K: four instructions, the first one overwriting.
__device__ __forceinline__ void mma_block(uint32_t d, uint32_t a_addr, uint32_t b_addr, uint32_t idesc) {
    const uint64_t a = operand_desc(a_addr), b = operand_desc(b_addr);
#pragma unroll
    for (int k = 0; k < 4; ++k) mma_f8(d, a + 2 * k, b + 2 * k, idesc, k > 0);
}
// The same across a pair of CTAs (cta_group::2), issued by one thread of the
// even one: M = 256, each CTA's tensor memory gets the 128 rows of its A tile;
// the tiles lie at the same shared-memory addresses in both CTAs, each with
// half of B's rows.
__device__ __forceinline__ void mma_block_pair(uint32_t d, uint32_t a_addr, uint32_t b_addr, uint32_t idesc) {
    const uint64_t a = operand_desc(a_addr), b = operand_desc(b_addr);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a + 2 * k), "l"(b + 2 * k), "r"(idesc), "r"(k > 0 ? 1 : 0)
            : "memory");
}
// One arrival on `bar` of both CTAs of the pair.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
// One arrival on `bar` when the thread's matrix instructions so far are done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// 16 consecutive columns of the warp's 32 lanes (lane = row).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// Wait for this thread's tcgen05.ld; the registers pass through so that no
// use of them is scheduled before it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                     "+r"(r[15])
                 :
                 : "memory");
}

// The same columns written, and the wait for such writes.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 bytes to a row of 32- or 16-byte alignment.
__device__ __forceinline__ void st_global_32b(void* p, const uint32_t (&w)[8], int align) {
    if (align == 32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        uint4* q = static_cast<uint4*>(p);
        q[0] = make_uint4(w[0], w[1], w[2], w[3]);
        q[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// -------------------------------------------------------------- clusters
// The address in the cluster's window of a shared-memory address of CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
// A tile load whose bytes are counted on a barrier of the pair's even CTA.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
// An arrival on another CTA's barrier.  What it tells about (tensor memory is
// read, a stage is free) is ordered by tcgen05 fences and copies' own
// completion: no fence at cluster scope, which costs over a thousand cycles.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Four values at the same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_cluster4(const float* p, uint32_t rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_addr(p, rank))
                 : "memory");
    return v;
}

// ---------------------------------------------------------------- scales
// A block's sum is scaled by the product of two scales.  Each of them may be
// anything fp32 holds, so the product may lie outside fp32's normal numbers where
// the scaled sum does not (sums are 2^-32 to 2^39, or 0).
__device__ __forceinline__ bool in_range(float product) {
    return fabsf(product) >= 0x1p-126f && fabsf(product) < __int_as_float(0x7F800000);
}
// Then sum a b = (sum * first) * s: `first` a power of two whose product with a
// sum that matters is exact, s rounded once, as a b is elsewhere.
struct ScalePair {
    float s, first;
};
__device__ __forceinline__ ScalePair split_scales(float a, float b) {
    const float inf = __int_as_float(0x7F800000), p = a * b;
    const bool swap = fabsf(a) > fabsf(b);
    const float lo = swap ? b : a, hi = swap ? a : b;
    ScalePair r = {p, 1.f};
    if (in_range(p) || lo == 0.f || p != p || fabsf(hi) == inf) return r;  // zeros, infinities and NaN: as they are
    if (fabsf(p) < 1.f) {  // |lo| < 2^-63
        r.first = 0x1p-64f;
        r.s = lo * 0x1p64f * hi;
    } else {  // |hi| >= 2^64; s stays finite, so that a sum of 0 gives 0
        r.first = 0x1p126f;
        r.s = fminf(fmaxf(hi * 0x1p-126f * lo, -0x1.fffffep127f), 0x1.fffffep127f);
    }
    return r;
}

__device__ __forceinline__ void store_out(void* y, int64_t at, int type, float v) {
    if (type == kF16)
        static_cast<__half*>(y)[at] = __float2half_rn(v);
    else if (type == kBF16)
        static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(y)[at] = v;
}

}  // namespace f8
}  // namespace sqz
