// Sums across the CTAs of a thread-block cluster: asynchronous stores into the
// other CTAs' shared memory, counted in bytes on the receiver's mbarrier.
#pragma once

#include "common.cuh"

namespace argb {

__device__ __forceinline__ uint32_t cluster_ctarank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t to_cluster(const void* local, uint32_t cta)
{
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(remote)
                 : "r"((uint32_t)__cvta_generic_to_shared(local)), "r"(cta));
    return remote;
}

// Write v to CTA `cta`'s shared memory, at the offset of `local` in ours, and
// count its 4 bytes on that CTA's barrier at the offset of `bar` in ours.
__device__ __forceinline__ void st_async_cluster_f32(float* local, const uint64_t* bar, uint32_t cta, float v)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(to_cluster(local, cta)),
                 "r"(__float_as_uint(v)), "r"(to_cluster(bar, cta))
                 : "memory");
}

// A barrier that completes its first phase when `bytes` have landed.
__device__ __forceinline__ void cluster_bar_init(uint64_t* bar, uint32_t bytes)
{
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(bar);
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(at) : "memory");
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(at), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cluster_bar_init_fence()
{
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Bounded wait (0.1 s) for the first phase.  A CTA that has waited for all
// its barriers has nothing still landing in its shared memory.
__device__ __forceinline__ bool cluster_bar_wait(uint64_t* bar)
{
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(bar);
    uint32_t done = 0;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 0; it < (1u << 22) && !done; ++it) {
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done)
                     : "r"(at)
                     : "memory");
        if (!done && (it & 255) == 255 && globaltimer_ns() - t0 > 100000000ull) break;
    }
    return done != 0;
}

}  // namespace argb
