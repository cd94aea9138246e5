// pair.cuh — what the products by pairs of SMs share: warp-uniform control, bounded waits by whole warps, the
// signals between a cluster's two CTAs, and epilogue pieces.
#pragma once

#include "common.cuh"

namespace gptq {

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// One lane of a converged warp: unlike a test of the lane number, the branch on it leaves the values
// it uses warp-uniform, so the tensor instructions take their operands from uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// The bounded wait, by a whole converged warp. Only the time is looked at while it waits: what a wait
// that gave up has to record is done after the loops, because a global atomic (or the load of its
// limit) in them cost the warps that feed the tensor core more than the waiting itself
// (8192 x 8192 x 8192 MX: 225 us with mbar_wait, 155 us with this).
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, uint64_t limit) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (__any_sync(0xffffffffu, globaltimer_ns() - t0 >= limit)) return false;
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    }
}

// ------------------------------------ the pair of CTAs ------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// the even CTA's copy of a shared-memory address
__device__ __forceinline__ uint32_t in_even_cta(uint32_t addr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}

// What these arrivals order is TMEM and copies by TMA, neither written by this thread, so the default
// (CTA) scope of the release is enough; .release.cluster would wait for the thread's own earlier
// stores of Y to be acknowledged (8192 x 8192 x 8192 MX took 408 us with it and 269 without).
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// arrive once on `bar` of both CTAs when the MMAs and scale copies issued before have completed
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// Waits for the phase of a barrier that counts copies or MMAs in flight, before the CTA leaves. They land
// within microseconds; the limit is for an unwinding pair, whose even CTA's stages may also be
// waiting for a word from the odd one that is not coming.
constexpr uint64_t kDrainNs = 20000000ull;
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < kDrainNs) {
    }
}

// max(x, 0) that keeps a NaN
__device__ __forceinline__ float relu_of(float x) {
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
    return y;
}

// 16 lanes x 32 columns of TMEM: of each 8 columns thread i gets lane i / 4, columns 2 (i % 4) and the
// next, then the same of lane 8 + i / 4 (the layout that stmatrix takes)
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

}  // namespace gptq
