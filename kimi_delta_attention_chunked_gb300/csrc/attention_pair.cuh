// attention_pair.cuh -- what the attention kernels of CTA pairs (clusters of two whose tensor
// cores work on one product, cta_group::2) share.
#pragma once

#include "attention_tc.cuh"

namespace kda_tc {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// A shared-memory address of CTA `rank` of the cluster, at the place that p has here.
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(kda::smem_u32(p)), "r"(rank));
    return r;
}
// Both CTAs' threads meet: what was written before cluster_arrive is seen behind cluster_wait.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// The same without an order of memory (and so without waiting for stores to global memory): at the end, where
// only shared memory and TMEM are given up.
__device__ __forceinline__ void cluster_leave() {
    asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}
// 16 values to 32 bytes of a row, as bf16: a whole sector, on a 32-byte boundary.
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float* y) {
    uint32_t x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = kda::pack_bf16x2(y[2 * e], y[2 * e + 1]);
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
                 "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}
// Arrives on a barrier of either CTA.  What it has to order is in this SM: stores to shared memory
// (made visible to the tensor cores by fence.proxy.async) and TMEM (by tcgen05.wait and fence); release at cluster
// scope would also wait for this thread's stores to global memory, half a microsecond each time.
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Tile load into this CTA's shared memory whose bytes are counted on CTA 0's barrier.
__device__ __forceinline__ void load_pair(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
        "%3, %4}], [%5];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// D[tmem] (+)= A[smem] * B[smem] of both CTAs; issued by one thread of CTA 0.
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// The same with A in TMEM (each CTA's rows in its own).
__device__ __forceinline__ void mma_pair_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive once on the barrier at this place in both CTAs (or those of `mask`) when the products issued so far are done.
// Nothing may arrive at a CTA that has left: each one waits for, or for something behind, every arrival that it gets.
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint16_t mask = 3) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            kda::smem_u32(bar)),
        "h"(mask)
        : "memory");
}
// All of TMEM, in both CTAs: one warp of each calls these.
__device__ __forceinline__ void alloc_pair(uint32_t* dst) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(kda::smem_u32(dst)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc_pair(uint32_t tmem) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Takes the elements that are not finite out of 16 bytes of bf16; true if there were any.
__device__ __forceinline__ bool take_odd(uint4& x) {
    uint32_t* y = reinterpret_cast<uint32_t*>(&x);
    bool found = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((y[i] & 0x7f80u) == 0x7f80u) { y[i] &= 0xffff0000u; found = true; }
        if ((y[i] & 0x7f800000u) == 0x7f800000u) { y[i] &= 0x0000ffffu; found = true; }
    }
    return found;
}
// Sets an int of the shared memory of both CTAs to 1, before whatever this thread does next.
__device__ __forceinline__ void flag_pair(int* flag) {
    for (uint32_t r = 0; r < 2; ++r)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at_rank(flag, r)), "r"(1) : "memory");
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
}

}  // namespace kda_tc
