// pair_merge.cu -- joins the parts of units that were cut between pairs of CTAs (bf16):
// with M the largest of the parts' references m_i,
//     o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,   lse = (M + log2 of the divisor) ln 2.
//
// The rows of a unit are shared out over the blocks of all pairs that hold a part of it.  D / 4
// threads take a row: they form the weights of its parts first, a part a thread, and then
// read the sums of eight parts at once.  Bound: latency (description, statistics, sums).
#include <algorithm>

#include "latent.cuh"

namespace {

using kda_paged::Partials;

constexpr int kThreads = 128, kBlocks = 12, kBatch = 8;
constexpr int kMostParts = 80;                         // pairs of a call

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 8)
kda_pair_merge_kernel(Partials parts, int Gv, int Hq, __nv_bfloat16* __restrict__ o, float* __restrict__ lse) {
    constexpr int TPR = D / 4, ROWS = kThreads / TPR;  // threads of a row, rows of a pass
    __shared__ float s_w[kThreads / 32][kMostParts];   // weights of a row's parts: every warp forms its row's itself
    kda_paged::wait_for_stream();
    const int c = blockIdx.x;
    const int4 u = parts.meta[2 * c + 1 - blockIdx.z]; // z = 0: the unit that begins here, 1: the one that goes on here
    const int n = u.w & 0xffff, c0 = u.w >> 16;
    if (n == 0) return;
    const int x = threadIdx.x % TPR, lane = threadIdx.x & 31, rows = u.z * Gv;
    float* w = s_w[threadIdx.x >> 5];
    const int step = n * kBlocks * ROWS;
#pragma unroll 1
    for (int r0 = ((c - c0) * kBlocks + blockIdx.y) * ROWS; r0 < rows; r0 += step) {
        const int r = min(r0 + (int)threadIdx.x / TPR, rows - 1);
        auto stats = [&](int i) { return parts.stats(c0 + i, i == 0 ? 1 : 0)[r]; };
        auto sums = [&](int i) {
            return reinterpret_cast<const float4*>(parts.sums(c0 + i, i == 0 ? 1 : 0) + (size_t)r * D)[x];
        };
        // the first parts' sums do not wait for the weights
        float4 v[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) v[e] = e < n ? sums(e) : make_float4(0.f, 0.f, 0.f, 0.f);
        float top = -INFINITY;
        float2 st[(kMostParts + 31) / 32];
#pragma unroll
        for (int e = 0; e < (kMostParts + 31) / 32; ++e) {
            st[e] = lane + 32 * e < n ? stats(lane + 32 * e) : make_float2(-INFINITY, 0.f);
            top = fmaxf(top, st[e].x);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float ref = top == -INFINITY ? 0.f : top;
        float l = 0.f;
        __syncwarp();                                  // the row before has been read
#pragma unroll
        for (int e = 0; e < (kMostParts + 31) / 32; ++e) {
            const float f = st[e].y == 0.f ? 0.f : ex2(st[e].x - ref);       // 0: the part saw no key
            l = fmaf(f, st[e].y, l);
            if (lane + 32 * e < n) w[lane + 32 * e] = f;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        __syncwarp();
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += kBatch) {
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                const float f = i0 + e < n ? w[i0 + e] : 0.f;
                if (f != 0.f) {                        // a part that saw no key does not enter
                    acc.x = fmaf(f, v[e].x, acc.x); acc.y = fmaf(f, v[e].y, acc.y);
                    acc.z = fmaf(f, v[e].z, acc.z); acc.w = fmaf(f, v[e].w, acc.w);
                }
            }
            if (i0 + kBatch < n) {
#pragma unroll
                for (int e = 0; e < kBatch; ++e)
                    v[e] = i0 + kBatch + e < n ? sums(i0 + kBatch + e) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        if (r0 + (int)threadIdx.x / TPR >= rows || u.y + r % Gv >= Hq) continue;     // a last group of fewer heads
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const size_t at = (size_t)(u.x + r / Gv) * Hq + u.y + r % Gv;
        *reinterpret_cast<uint2*>(o + at * D + 4 * x) =
            make_uint2(kda::pack_bf16x2(acc.x * inv, acc.y * inv), kda::pack_bf16x2(acc.z * inv, acc.w * inv));
        if (lse && x == 0) lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
    }
}

template <int D>
cudaError_t merge(const kda_host::PagedArgs& a, const kda_host::PagedPlan& p, int pairs) {
    // the same split of L1 and shared memory as the attention kernel before it: an SM
    // must run dry to change it
    static kda_host::OncePerDevice once;
    const cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(kda_pair_merge_kernel<D>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                    cudaSharedmemCarveoutMaxShared);
    });
    if (e != cudaSuccess) return e;
    return kda_host::launch_overlapped(kda_pair_merge_kernel<D>, dim3(pairs, kBlocks, 2), kThreads, 0, a.stream, 1,
                                       kda_host::paged_partials(a, p), p.Gv, a.Hq, static_cast<__nv_bfloat16*>(a.o), a.lse);
}

}  // namespace

namespace kda_host {

cudaError_t launch_pair_merge(const PagedArgs& a, const PagedPlan& p, int pairs) {
    if (pairs > kMostParts) return cudaErrorInvalidValue;
    return a.d == kda_latent::kLatent ? merge<kda_latent::kLatent>(a, p, pairs) : merge<kda_latent::kValue>(a, p, pairs);
}

}  // namespace kda_host
