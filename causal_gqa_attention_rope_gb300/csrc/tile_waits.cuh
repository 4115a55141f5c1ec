// tile_waits.cuh -- what the tile kernels' warps share: bounded waits that end the
// CTA's work together, and the softmax's maximum and exponential.
#pragma once

#include "na_internal.cuh"

__device__ __forceinline__ bool aborted(const int *flag) { return *(volatile const int *)flag != 0; }

__device__ __forceinline__ void set_abort(int *flag, int32_t *status)
{
    *(volatile int *)flag = 1;
    na_report(status, NA_ERR_DEVICE_TIMEOUT);
}

// A bounded wait whose outcome is only reported: the drains before exit (copies
// in flight, MMAs before tensor memory is released), where there is nothing
// left to skip.  A wait that gives up writes NA_ERR_DEVICE_TIMEOUT.
__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity, int32_t *status)
{
    if (!mbar_wait_bounded(bar, parity))
        na_report(status, NA_ERR_DEVICE_TIMEOUT);
}

// A bounded wait whose result every lane of the warp shares: the softmax warps
// follow it with warp-collective tensor-memory loads and stores, which no lane
// may skip while others execute them.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const int *abort_flag)
{
    const bool done = mbar_wait_bounded(bar, parity) && !aborted(abort_flag);
    return __all_sync(0xffffffffu, done);
}

__device__ __forceinline__ float max3f(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 2^x on the MUFU unit (approximate, flushes subnormal results to zero).
__device__ __forceinline__ float ex2_mufu(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// One lane of a converged warp.  (A branch on it is known to be taken by one thread, so
// that the descriptors of the matrix instructions inside stay in uniform registers.)
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// All threads of all CTAs of the cluster; what was written before is seen after.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One arrival on the barrier at `bar`'s offset in CTA `rank` of the cluster; a thread there that
// waits with mbar_wait_cluster sees what was written before.
__device__ __forceinline__ void mbar_arrive_cluster(uint64_t *bar, int rank)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(bar)), "r"(rank));
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(a) : "memory");
}

__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity)
{
    const long long start = clock64();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; i++) {
            uint32_t done;
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(done)
                : "r"(smem_addr(bar)), "r"(parity)
                : "memory");
            if (done)
                return true;
        }
        if (clock64() - start > NA_WAIT_LIMIT_CYCLES)
            return false;
    }
}
