// latent_merge.cu -- joins the parts of latent attention's units that were cut between CTAs (or pairs of them):
// with M the largest of the parts' references m_i,
//     o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,   lse = (M + log2 of the divisor) ln 2.
//
// The rows of a unit are shared out over the blocks of all CTAs that hold a part of it.  D / 4
// threads take a row; units of few parts, which most are, several rows at once.  A part's weight is
// formed by one lane of each warp; the sums are read beside the statistics.  Bound: latency
// (description, then statistics and sums) and, with hundreds of rows in every slot, L2.
#include <algorithm>

#include "latent.cuh"

namespace {

using kda_paged::Partials;

constexpr int kThreads = 128, kBlocks = 12;
constexpr int kMostParts = 304;                        // CTAs or pairs of a call

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One unit: rows of q from u.x, heads from u.y, parts in slots of the CTAs c0, c0 + 1, ...
template <typename T>
struct Join {
    int4 u;
    int n, c0, rows, Gv, Hq;
    T* o;
    float* lse;
};

// Rows first, first + step, ... in groups of R, whose parts are read PARTS at a time.  ALL: PARTS are all that a unit has.
template <int D, int R, int PARTS, bool ALL, typename T>
__device__ __forceinline__ void join_rows(const Partials& parts, const Join<T>& j, int first, int step, float* w) {
    constexpr int TPR = D / 4;
    const int x = threadIdx.x % TPR, lane = threadIdx.x & 31;
    auto sums = [&](int r, int i) {
        return i < j.n ? reinterpret_cast<const float4*>(parts.sums(j.c0 + i, i == 0 ? 1 : 0) + (size_t)r * D)[x]
                       : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    auto stats = [&](int r, int i) {
        return i < j.n ? parts.stats(j.c0 + i, i == 0 ? 1 : 0)[r] : make_float2(-INFINITY, 0.f);
    };
    auto weight = [](const float2& st, float ref) { return st.y == 0.f ? 0.f : ex2(st.x - ref); };    // 0: the part saw no key
#pragma unroll 1
    for (int r0 = first; r0 < j.rows; r0 += R * step) {
        float4 v[R][PARTS];
        float2 st[R];
        int r[R];
#pragma unroll
        for (int a = 0; a < R; ++a) {
            r[a] = min(r0 + a * step, j.rows - 1);
            st[a] = stats(r[a], lane);
#pragma unroll
            for (int e = 0; e < PARTS; ++e) v[a][e] = sums(r[a], e);
        }
#pragma unroll
        for (int a = 0; a < R; ++a) {
            float top = st[a].x;
            if (!ALL)
                for (int i = lane + 32; i < j.n; i += 32) top = fmaxf(top, stats(r[a], i).x);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float ref = top == -INFINITY ? 0.f : top, f = weight(st[a], ref);
            float l = f * st[a].y;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            auto add = [&](float g, const float4& y) {
                if (g != 0.f) {                        // a part that saw no key does not enter
                    acc.x = fmaf(g, y.x, acc.x); acc.y = fmaf(g, y.y, acc.y);
                    acc.z = fmaf(g, y.z, acc.z); acc.w = fmaf(g, y.w, acc.w);
                }
            };
            if constexpr (ALL) {
#pragma unroll
                for (int e = 0; e < PARTS; ++e) add(__shfl_sync(0xffffffffu, f, e), v[a][e]);
            } else {
                __syncwarp();                          // the row before has been read
                w[lane] = f;
                for (int i = lane + 32; i < j.n; i += 32) {
                    const float2 more = stats(r[a], i);
                    w[i] = weight(more, ref);
                    l = fmaf(w[i], more.y, l);
                }
                __syncwarp();
#pragma unroll 1
                for (int i0 = 0; i0 < j.n; i0 += PARTS) {
#pragma unroll
                    for (int e = 0; e < PARTS; ++e) add(i0 + e < j.n ? w[i0 + e] : 0.f, v[a][e]);
#pragma unroll
                    for (int e = 0; e < PARTS; ++e) v[a][e] = sums(r[a], i0 + PARTS + e);
                }
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
            const int head = j.u.y + r[a] % j.Gv;
            if (r0 + a * step >= j.rows || head >= j.Hq) continue;            // a last group of fewer heads
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const size_t at = (size_t)(j.u.x + r[a] / j.Gv) * j.Hq + head;
            T* dst = j.o + at * D + 4 * x;
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<uint2*>(dst) =
                    make_uint2(kda::pack_bf16x2(acc.x * inv, acc.y * inv), kda::pack_bf16x2(acc.z * inv, acc.w * inv));
            else
                *reinterpret_cast<float4*>(dst) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            if (j.lse && x == 0) j.lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
        }
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 8)
kda_latent_merge_kernel(Partials parts, int Gv, int Hq, T* __restrict__ o, float* __restrict__ lse) {
    constexpr int ROWS = kThreads / (D / 4);           // rows of a pass
    __shared__ float s_w[kThreads / 32][kMostParts];   // weights of a row's parts: every warp forms its row's itself
    kda_paged::wait_for_stream();
    const int c = blockIdx.x;
    const int4 u = parts.meta[2 * c + 1 - blockIdx.z]; // z = 0: the unit that begins here, 1: the one that goes on here
    const Join<T> j{u, u.w & 0xffff, u.w >> 16, u.z * Gv, Gv, Hq, o, lse};
    if (j.n == 0) return;
    const int first = ((c - j.c0) * kBlocks + blockIdx.y) * ROWS + (int)threadIdx.x / (D / 4), step = j.n * kBlocks * ROWS;
    if (j.n <= 2) join_rows<D, 2, 2, true>(parts, j, first, step, nullptr);
    else if (j.n <= 4) join_rows<D, 2, 4, true>(parts, j, first, step, nullptr);
    else join_rows<D, 1, 8, false>(parts, j, first, step, s_w[threadIdx.x >> 5]);
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
    if (ctas > kMostParts) return cudaErrorInvalidValue;
    return a.d == kda_latent::kLatent ? merge_of<kda_latent::kLatent>(a, p, ctas) : merge_of<kda_latent::kValue>(a, p, ctas);
}

}  // namespace kda_host
