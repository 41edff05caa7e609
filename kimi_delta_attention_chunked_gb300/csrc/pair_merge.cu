// pair_merge.cu -- joins the parts of units that were cut between pairs of CTAs (bf16):
// with M the largest of the parts' references m_i,
//     o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,   lse = (M + log2 of the divisor) ln 2.
//
// The rows of a unit are shared out over the blocks of all pairs that hold a part of it.  D / 4
// threads take a row; units of few parts, which most are, several rows at once.  A part's weight is
// formed by one lane of each warp; the sums are read beside the statistics.  Bound: latency
// (description, then statistics and sums) and, with hundreds of rows in every slot, L2.
#include <algorithm>

#include "latent.cuh"

namespace {

using kda_paged::Partials;

constexpr int kThreads = 128, kBlocks = 12;
constexpr int kMostParts = 80;                         // pairs of a call

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One unit: request rows from u.x, heads from u.y, parts in slots of the pairs c0, c0 + 1, ...
struct Join {
    int4 u;
    int n, c0, rows, Gv, Hq;
    __nv_bfloat16* o;
    float* lse;
};

// Rows first, first + step, ... in groups of R, whose parts are read PARTS at a time.
template <int D, int R, int PARTS>
__device__ __forceinline__ void join_rows(const Partials& parts, const Join& j, int first, int step, float* w) {
    constexpr int TPR = D / 4, SETS = (kMostParts + 31) / 32, LANES = PARTS < 8 ? 1 : SETS;
    const int x = threadIdx.x % TPR, lane = threadIdx.x & 31;
    auto sums = [&](int r, int i) {
        return reinterpret_cast<const float4*>(parts.sums(j.c0 + i, i == 0 ? 1 : 0) + (size_t)r * D)[x];
    };
#pragma unroll 1
    for (int r0 = first; r0 < j.rows; r0 += R * step) {
        float4 v[R][PARTS];
        float2 st[R][LANES];
        int r[R];
#pragma unroll
        for (int a = 0; a < R; ++a) {
            r[a] = min(r0 + a * step, j.rows - 1);
#pragma unroll
            for (int e = 0; e < LANES; ++e)
                st[a][e] = lane + 32 * e < j.n ? parts.stats(j.c0 + lane + 32 * e, lane + 32 * e == 0 ? 1 : 0)[r[a]]
                                               : make_float2(-INFINITY, 0.f);
        }
#pragma unroll
        for (int a = 0; a < R; ++a)
#pragma unroll
            for (int e = 0; e < PARTS; ++e) v[a][e] = e < j.n ? sums(r[a], e) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int a = 0; a < R; ++a) {
            float top = st[a][0].x;
#pragma unroll
            for (int e = 1; e < LANES; ++e) top = fmaxf(top, st[a][e].x);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float ref = top == -INFINITY ? 0.f : top;
            float l = 0.f, f[LANES];
#pragma unroll
            for (int e = 0; e < LANES; ++e) {
                f[e] = st[a][e].y == 0.f ? 0.f : ex2(st[a][e].x - ref);       // 0: the part saw no key
                l = fmaf(f[e], st[a][e].y, l);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            auto add = [&](float g, const float4& y) {
                if (g != 0.f) {                        // a part that saw no key does not enter
                    acc.x = fmaf(g, y.x, acc.x); acc.y = fmaf(g, y.y, acc.y);
                    acc.z = fmaf(g, y.z, acc.z); acc.w = fmaf(g, y.w, acc.w);
                }
            };
            if constexpr (LANES == 1) {
#pragma unroll
                for (int e = 0; e < PARTS; ++e) add(__shfl_sync(0xffffffffu, f[0], e), v[a][e]);
            } else {
                __syncwarp();                          // the row before has been read
#pragma unroll
                for (int e = 0; e < LANES; ++e)
                    if (lane + 32 * e < j.n) w[lane + 32 * e] = f[e];
                __syncwarp();
#pragma unroll 1
                for (int i0 = 0; i0 < j.n; i0 += PARTS) {
#pragma unroll
                    for (int e = 0; e < PARTS; ++e) add(i0 + e < j.n ? w[i0 + e] : 0.f, v[a][e]);
                    if (i0 + PARTS < j.n) {
#pragma unroll
                        for (int e = 0; e < PARTS; ++e)
                            v[a][e] = i0 + PARTS + e < j.n ? sums(r[a], i0 + PARTS + e) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                }
            }
            const int head = j.u.y + r[a] % j.Gv;
            if (r0 + a * step >= j.rows || head >= j.Hq) continue;            // a last group of fewer heads
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const size_t at = (size_t)(j.u.x + r[a] / j.Gv) * j.Hq + head;
            *reinterpret_cast<uint2*>(j.o + at * D + 4 * x) =
                make_uint2(kda::pack_bf16x2(acc.x * inv, acc.y * inv), kda::pack_bf16x2(acc.z * inv, acc.w * inv));
            if (j.lse && x == 0) j.lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 8)
kda_pair_merge_kernel(Partials parts, int Gv, int Hq, __nv_bfloat16* __restrict__ o, float* __restrict__ lse) {
    constexpr int ROWS = kThreads / (D / 4);           // rows of a pass
    __shared__ float s_w[kThreads / 32][kMostParts];   // weights of a row's parts: every warp forms its row's itself
    kda_paged::wait_for_stream();
    const int c = blockIdx.x;
    const int4 u = parts.meta[2 * c + 1 - blockIdx.z]; // z = 0: the unit that begins here, 1: the one that goes on here
    const Join j{u, u.w & 0xffff, u.w >> 16, u.z * Gv, Gv, Hq, o, lse};
    if (j.n == 0) return;
    const int first = ((c - j.c0) * kBlocks + blockIdx.y) * ROWS + (int)threadIdx.x / (D / 4), step = j.n * kBlocks * ROWS;
    if (j.n <= 2) join_rows<D, 2, 2>(parts, j, first, step, nullptr);
    else if (j.n <= 4) join_rows<D, 2, 4>(parts, j, first, step, nullptr);
    else join_rows<D, 1, 8>(parts, j, first, step, s_w[threadIdx.x >> 5]);
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
