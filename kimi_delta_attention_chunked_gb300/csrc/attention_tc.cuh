// attention_tc.cuh -- what the tensor-core attention kernels share: instructions, waits
// that give up, packed arithmetic, and which keys the rows of a unit see.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <mutex>

#include "paged.cuh"
#include "umma.cuh"

namespace kda_tc {

using kda_paged::Unit;

constexpr float kGrow = 8.f;                           // octaves that a score may exceed the reference
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int x, int y, int z, int t,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(t), "r"(kda::smem_u32(bar))
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], A (M = 128) as bf16 pairs: lane = row, 8
// columns per 16 elements of K.
__device__ __forceinline__ void umma_bf16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* u) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
        "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
        "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
        "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
        : "memory");
}

// One lane of the (converged) warp.  Unlike `lane == 0`, the compiler keeps what
// is the same for the whole warp in uniform registers across this branch, where
// the operands of tcgen05.mma have to be.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// A value that is the same in all lanes, in a form the compiler knows to be so.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// What the keys of a unit mean for the rows [first, last] of its tokens.
struct Sight {
    int lo, hi;                                        // keys [lo, hi): some row sees them
    int all_lo, all_hi;                                // keys [all_lo, all_hi): every row sees them
};
__device__ __forceinline__ Sight sight(const Unit& u, int window, int first, int last) {
    Sight s;
    const int p0 = u.pos + first, p1 = u.pos + last;
    s.hi = min(max(p1 + 1, 0), u.kend);
    s.all_hi = min(max(p0 + 1, 0), u.kend);
    s.lo = kda_paged::first_key(p0, window);
    s.all_lo = kda_paged::first_key(p1, window);
    return s;
}

// The rest of a wait that did not succeed at once.  One copy of it for the whole
// kernel: its many inlined ones would be most of what a short call fetches.
static __device__ __noinline__ bool wait_longer(uint64_t* b, uint32_t parity, volatile int* abort, int* status) {
    const bool done = kda::mbar_wait_or_abort(b, parity, kda::kWaitCycles, abort);
    if (__all_sync(0xffffffffu, done)) return true;
    if (!*abort) kda::record_status(status, kda::kDevTimeout);
    *abort = 1;
    return false;
}

}  // namespace kda_tc

namespace kda_host {

// cuTensorMapEncodeTiled of the driver, or null
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

}  // namespace kda_host
