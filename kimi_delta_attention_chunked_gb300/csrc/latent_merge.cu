// latent_merge.cu -- joins the parts of latent attention's units that were cut between CTAs (or pairs of them):
// with M the largest of the parts' references m_i,
//     o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,   lse = (M + log2 of the divisor) ln 2.
//
// A slot's sums lie four channels wide, [D / 4][rows][4]: the threads of the tensor-core kernels hold a row
// each, so a warp's store there and a warp's load here are whole lines (by rows, 128 of 512 channels took a pair of
// CTAs 5,700 cycles to write).  A warp of the CUDA-core kernel holds four rows of 32 such columns and writes 64 bytes of
// each; by rows instead, its stores would be whole lines and the loads here not: 34 -> 41 us where 300 CTAs share a
// unit, 20.6 -> 21.7 in the absorbed fp32 case, 40.7 -> 40.3 in the expanded one.  A warp takes 16 channels of 32 rows, or, where there are more than
// four parts, of 8 rows with four lanes to a row; the warps of all CTAs that hold a part of a unit share it
// out.  Bound: latency (description, then statistics and sums: 5 us for units of a few rows) and, with 128 and
// more rows in every slot, L2 (40 MB: 8 to 10 us).
#include <algorithm>

#include "latent.cuh"

namespace {

using kda_paged::Partials;

// Blocks that a CTA's slot is shared out to; with 4, 8, 12 and 20: 128 heads 77.4, 73.3, 73.0 and 72.7 us, verification 62.6,
// 61.7, 60.9 and 61.3, few requests 14.2, 13.9, 14.2 and 14.7, 12 expanded requests 48, 44, 43 to 47 and 43.
constexpr int kThreads = 128, kBlocks = 12;
constexpr int kWide = 16;                              // channels of a warp's work
constexpr int kBatch = 4;                              // parts read at once (2, with twice the blocks on an SM: few requests
                                                       // 14.2 -> 16.2 us, verification 60.9 -> 69)

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Weighted sums of parts first, first + stride, ... of rows r (one a lane), 16 channels from 16 `wide` on.
struct Sum {
    float4 acc[kWide / 4];
    float top, l;                                      // reference; sum of the weights
    __device__ __forceinline__ void take(const Partials& parts, int c0, int n, int first, int stride, int r, int wide) {
        auto stats = [&](int i) { return i < n ? parts.stats(c0 + i, i == 0 ? 1 : 0)[r] : make_float2(-INFINITY, 0.f); };
        float4 v[kBatch][kWide / 4];
        float2 st[kBatch];
        auto load = [&](int i0) {
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                const int i = i0 + e * stride;
                st[e] = stats(i);
                if (i < n) {
                    const float4* src =
                        reinterpret_cast<const float4*>(parts.sums4(c0 + i, i == 0 ? 1 : 0, r, wide * kWide));
#pragma unroll
                    for (int x = 0; x < kWide / 4; ++x) v[e][x] = src[(size_t)x * parts.cap];
                }
            }
        };
        load(first);
        top = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int e = 0; e < kBatch; ++e) top = fmaxf(top, st[e].x);
        for (int i = first + kBatch * stride; i < n; i += stride) top = fmaxf(top, stats(i).x);
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int x = 0; x < kWide / 4; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int i0 = first;;) {
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                const float f = st[e].y == 0.f ? 0.f : ex2(st[e].x - ref);
                l = fmaf(f, st[e].y, l);
                if (i0 + e * stride < n) {             // at a weight of 0 too: 0 * NaN is NaN, wherever keys are cut
#pragma unroll
                    for (int x = 0; x < kWide / 4; ++x) add(acc[x], f, v[e][x]);
                }
            }
            i0 += kBatch * stride;
            if (i0 >= n) break;
            load(i0);
        }
    }
    static __device__ __forceinline__ void add(float4& a, float f, const float4& v) {
        a.x = fmaf(f, v.x, a.x); a.y = fmaf(f, v.y, a.y); a.z = fmaf(f, v.z, a.z); a.w = fmaf(f, v.w, a.w);
    }
};

__device__ __forceinline__ void store4(__nv_bfloat16* p, const float4& v, float f) {
    *reinterpret_cast<uint2*>(p) = make_uint2(kda::pack_bf16x2(v.x * f, v.y * f), kda::pack_bf16x2(v.z * f, v.w * f));
}
__device__ __forceinline__ void store4(float* p, const float4& v, float f) {
    *reinterpret_cast<float4*>(p) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}

// One unit: rows of q from u.x, heads from u.y, parts in slots of the CTAs c0, c0 + 1, ...
template <typename T>
struct Unit {
    int4 u;
    int n, c0, rows, Gv, Hq;
    T* o;
    float* lse;
};

// A warp's share of a unit: 32 / SHARE rows at a time, each row's parts shared by SHARE lanes.
template <int D, int SHARE, typename T>
__device__ __forceinline__ void join(const Partials& parts, const Unit<T>& j, int first, int step) {
    constexpr int ROWS = 32 / SHARE;
    const int lane = threadIdx.x & 31, blocks = (j.rows + ROWS - 1) / ROWS, items = blocks * (D / kWide);
#pragma unroll 1
    for (int item = first; item < items; item += step) {
        const int wide = item / blocks, row = (item - wide * blocks) * ROWS + lane % ROWS, r = min(row, j.rows - 1);
        Sum sum;
        sum.take(parts, j.c0, j.n, lane / ROWS, SHARE, r, wide);
        float top = sum.top, l = sum.l;
        if constexpr (SHARE > 1) {
#pragma unroll
            for (int d = ROWS; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float f = l == 0.f ? 0.f : ex2(sum.top - top);
            l *= f;
#pragma unroll
            for (int x = 0; x < kWide / 4; ++x) {
                float* y = &sum.acc[x].x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[e] *= f;
#pragma unroll
                    for (int d = ROWS; d < 32; d <<= 1) y[e] += __shfl_xor_sync(0xffffffffu, y[e], d);
                }
            }
#pragma unroll
            for (int d = ROWS; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        }
        const int head = j.u.y + r % j.Gv;
        if (row >= j.rows || head >= j.Hq) continue;   // a last group may have fewer heads
        l = kda_paged::whole_sum(top, l);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const size_t at = (size_t)(j.u.x + r / j.Gv) * j.Hq + head;
        T* dst = j.o + at * D + wide * kWide;
        if constexpr (SHARE > 1) {                     // a lane of the row stores four channels
            static_assert(SHARE == kWide / 4, "channels");
            const int x = lane / ROWS;
            float4 v = sum.acc[0];
#pragma unroll
            for (int e = 1; e < kWide / 4; ++e)
                if (x == e) v = sum.acc[e];
            store4(dst + 4 * x, v, inv);
        } else {
#pragma unroll
            for (int x = 0; x < kWide / 4; ++x) store4(dst + 4 * x, sum.acc[x], inv);
        }
        if (j.lse && wide == 0 && lane < ROWS) j.lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 4)
kda_latent_merge_kernel(Partials parts, int Gv, int Hq, T* __restrict__ o, float* __restrict__ lse) {
    constexpr int WARPS = kThreads / 32;
    kda_paged::wait_for_stream();
    const int c = blockIdx.x;
    const int4 u = parts.meta[2 * c + 1 - blockIdx.z]; // z = 0: the unit that begins here, 1: the one that goes on here
    const Unit<T> j{u, u.w & 0xffff, u.w >> 16, u.z * Gv, Gv, Hq, o, lse};
    if (j.n == 0) return;
    const int first = ((c - j.c0) * kBlocks + blockIdx.y) * WARPS + (int)(threadIdx.x >> 5), step = j.n * kBlocks * WARPS;
    if (j.n <= kBatch) join<D, 1>(parts, j, first, step);
    else join<D, 4>(parts, j, first, step);
}

template <int D, typename T>
cudaError_t merge(const kda_host::PagedArgs& a, const kda_host::PagedPlan& p, int ctas) {
    // the same split of L1 and shared memory as the attention kernel before it: an SM
    // must run dry to change it
    static kda_host::OncePerDevice once;
    const cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(kda_latent_merge_kernel<D, T>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                    cudaSharedmemCarveoutMaxShared);
    });
    if (e != cudaSuccess) return e;
    return kda_host::launch_overlapped(kda_latent_merge_kernel<D, T>, dim3(ctas, kBlocks, 2), kThreads, 0, a.stream, 1,
                                       kda_host::paged_partials(a, p), p.Gv, a.Hq, static_cast<T*>(a.o), a.lse);
}

template <int D>
cudaError_t merge_of(const kda_host::PagedArgs& a, const kda_host::PagedPlan& p, int ctas) {
    return a.dtype == KDA_BF16 ? merge<D, __nv_bfloat16>(a, p, ctas) : merge<D, float>(a, p, ctas);
}

}  // namespace

namespace kda_host {

cudaError_t launch_latent_merge(const PagedArgs& a, const PagedPlan& p, int ctas) {
    return a.d == kda_latent::kLatent ? merge_of<kda_latent::kLatent>(a, p, ctas) : merge_of<kda_latent::kValue>(a, p, ctas);
}

}  // namespace kda_host
