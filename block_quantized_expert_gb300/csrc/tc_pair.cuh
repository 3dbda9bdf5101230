// tc_pair.cuh -- building blocks of the products that run on one CTA or on a pair of
// CTAs (a cluster of two on one tcgen05 MMA, cta_group::2): arrivals, waits and
// tensor memory of either form.
#pragma once

#include "tc_ptx.cuh"

namespace moe {
namespace tc {

// One lane of the warp, the same one each time: 1 there, 0 elsewhere.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r;
}

// Arrives on the barrier (of both CTAs of a pair) when the MMAs so far are done.
template <bool kPair>
__device__ __forceinline__ void mma_commit_by(uint32_t on, uint32_t bar) {
    if (kPair)
        asm volatile(
            "{\n.reg .pred q;\n.reg .b16 m;\nmov.b16 m, 3;\nsetp.ne.b32 q, %1, 0;\n"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}"
            ::"r"(bar), "r"(on)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar), "r"(on)
            : "memory");
}

// Arrives on the pair's first CTA's barrier at the same place as `bar` here.  What
// it orders (this CTA's shared and tensor memory, read by the pair's MMA) is local
// and fenced for the MMA before; with release.cluster instead every arrival waits
// for a fence over the cluster, about 2000 cycles a unit (measured, all else equal:
// 2260 us for the 49152 rows of 256 experts at K = N = 4096, and 1570 without).
__device__ __forceinline__ void mbar_arrive_first(uint32_t bar) {
    asm volatile(
        "{\n.reg .b32 r;\nmapa.shared::cluster.u32 r, %0, 0;\n"
        "mbarrier.arrive.shared::cluster.b64 _, [r];\n}" ::"r"(bar) : "memory");
}

// mbar_wait for phases that come late as a rule (and, in a pair, from threads of
// the other CTA as well): the thread is suspended for up to 100 us at a time, so
// that polling leaves the issue slots to the others (677 us for 684 at 3000 rows).
template <bool kPair>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if (kPair)
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
            "selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok) : "r"(bar), "r"(parity), "r"(100000u) : "memory");
    else
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
            "selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok) : "r"(bar), "r"(parity), "r"(100000u) : "memory");
    return ok != 0;
}

// One look, without suspension.
template <bool kPair>
__device__ __forceinline__ bool test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if (kPair)
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
            "selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    else
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
            "selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

template <bool kPair>
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    if (try_wait<kPair>(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    while (!try_wait<kPair>(bar, parity))
        if (*abort || globaltimer() - t0 > limit_ns) return false;
    return true;
}

__device__ __forceinline__ void pair_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <bool kPair>
__device__ __forceinline__ void tmem_alloc_all(uint32_t slot) {
    if (!kPair) return tmem_alloc(slot, 512);
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(slot) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

template <bool kPair>
__device__ __forceinline__ void tmem_free_all(uint32_t taddr) {
    if (!kPair) return tmem_dealloc(taddr, 512);
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
}

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

}  // namespace tc
}  // namespace moe
