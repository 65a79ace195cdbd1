// cluster.cuh -- what the CTAs of a cluster do to each other's shared memory: remote stores that complete
// on the receiver's mbarrier, remote arrivals, and waits that see them.
#pragma once

#include "pipeline.cuh"

namespace csa {

// True in one lane of a converged warp, always the same one.  The compiler then knows that one thread issues what
// stands behind it: sixteen tcgen05.mma of 32 cycles each go out in 512 cycles (825 behind lane == 0).
__device__ __forceinline__ bool elect_lane()
{
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Shared-memory address of the same variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote_addr(uint32_t saddr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Store to another CTA's shared memory; the bytes complete on an mbarrier of that CTA.
__device__ __forceinline__ void st_async16(uint32_t raddr, uint4 v, uint32_t rbar)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1,%2,%3,%4}, [%5];" ::"r"(raddr),
                 "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(rbar)
                 : "memory");
}

__device__ __forceinline__ void st_async4(uint32_t raddr, uint32_t v, uint32_t rbar)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(raddr), "r"(v), "r"(rbar)
                 : "memory");
}

// Copy of shared memory to another CTA's (addresses and size multiples of 16), completing on an mbarrier there.
__device__ __forceinline__ void bulk_to_cta(uint32_t raddr, uint32_t saddr, uint32_t bytes, uint32_t rbar)
{
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(raddr),
                 "r"(saddr), "r"(bytes), "r"(rbar)
                 : "memory");
}

// Arrivals of lane 0 for its warp, predicated instead of branched around: the warp stays converged.
__device__ __forceinline__ void lane0_arrive(uint64_t *bar, int lane)
{
    asm volatile(
        "{\n.reg .pred p;\n.reg .b64 st;\n"
        "setp.eq.s32 p, %1, 0;\n"
        "@p mbarrier.arrive.shared::cta.b64 st, [%0];\n}" ::"r"(smem_addr(bar)),
        "r"(lane)
        : "memory");
}

__device__ __forceinline__ void lane0_arrive_expect_tx(uint64_t *bar, uint32_t bytes, int lane)
{
    asm volatile(
        "{\n.reg .pred p;\n.reg .b64 st;\n"
        "setp.eq.s32 p, %2, 0;\n"
        "@p mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n}" ::"r"(smem_addr(bar)),
        "r"(bytes), "r"(lane)
        : "memory");
}

// On an mbarrier of another CTA, which may then overwrite what this warp has read.
__device__ __forceinline__ void lane0_arrive_remote(uint32_t rbar, int lane)
{
    asm volatile(
        "{\n.reg .pred p;\n"
        "setp.eq.s32 p, %1, 0;\n"
        "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n}" ::"r"(rbar),
        "r"(lane)
        : "memory");
}

// Waits of kernels whose warps run many different loops.  The code of all of them together has to fit the
// SM's instruction cache, so a wait is a few instructions, with the hardware's suspension instead of polling, and no
// call, around which the compiler would spill.  Remote stores and arrivals are waited for like local ones: what
// they bring lies in this SM's shared memory when the barrier completes.  (Release and acquire at cluster
// scope would also order global memory: a fence of some thousand cycles and an invalidated L1 per tile.)
constexpr uint32_t kWaitHintNs = 4000;   // longest suspension of one try_wait

__device__ __forceinline__ bool mbar_try_wait_hint(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        "selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kWaitHintNs)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint32_t global_ns_lo()
{
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}

// Shared-memory address of the CTA's abort flag (int): 0, or which wait ran past kWaitLimitNs.
struct WaitCtx {
    uint32_t abort_flag;
};

// Wait of a whole warp, every lane in the same instructions (a wait of one lane whose outcome is then
// broadcast leaves the warp split, and the code behind it runs once for each part: measured at half of all
// instructions).  A phase that is already over costs one test (40 cycles; with a suspension time 70).  False, with the
// abort flag set to `where`, when the wait runs past kWaitLimitNs, or when another warp's has.
__device__ __forceinline__ bool warp_wait_hint(uint64_t *bar, uint32_t parity, const WaitCtx &cx, int where)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint32_t b = smem_addr(bar), t0 = global_ns_lo();
#pragma unroll 1
    do {
        if (mbar_try_wait_hint(b, parity)) return true;
        int aborted;
        asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(aborted) : "r"(cx.abort_flag) : "memory");
        if (aborted) return false;
    } while (global_ns_lo() - t0 < (uint32_t)kWaitLimitNs);
    asm volatile("st.volatile.shared.s32 [%0], %1;" ::"r"(cx.abort_flag), "r"(where) : "memory");
    return false;
}

}  // namespace csa
