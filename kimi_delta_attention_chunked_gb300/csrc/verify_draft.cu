// verify_draft.cu -- acceptance of drafted tokens and the draw of the next one.
//
// Per request: draft i stands while u_i q_i(x_i) < p_i(x_i) (the product of two
// fp32 numbers is exact in fp64, so the comparison is exact), a is the number
// that stand, and one token is drawn from r = max(p_a - q_a, 0) (r = p_a when
// all stand): the first v with sum_{v' <= v} r_v' > u_K sum r.
//
// The drawn index is a whole number that must not depend on how the sum was
// cut up, and in fp32 the running sum of 10^5 probabilities is off by more than
// many of them.  So probabilities become integers, p -> floor(p 2^60), and
// every sum is exact in 64 bits.  The conversion is a shift of the mantissa (the
// fp64 units and 64-bit conversions of this GPU are far slower than its memory).
//
// A cluster of CTAs takes one request: each sums its part of the row (16 bytes
// of p and q of it per thread and step where the row is aligned), the parts are
// exchanged through distributed shared memory, and the CTA that holds the
// crossing finds the warp's part, then the element, by scanning again what is
// by then in L2.  Only row a is read: bound by HBM, 2 V numbers a request.
#include <algorithm>
#include <cooperative_groups.h>

#include "paged.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPerSm = 6;                              // CTAs of an SM

// floor(min(max(p, 0), 1) 2^60); NaN counts as 0
__device__ __forceinline__ unsigned long long fixed60(float p) {
    const unsigned b = __float_as_uint(__saturatef(p));    // 0 ... 1, NaN becomes 0
    const unsigned long long m = (unsigned long long)((b & 0x7fffffu) | 0x800000u) << 37;
    return m >> min(127u - (b >> 23), 63u);                // p = 1.m 2^(e - 127), e <= 127; below 2^-60: 0
}

template <typename T>
struct Row {
    const T* p;
    const T* q;                                            // nullptr: no draft row
    int masked;                                            // index with q = 1 (a token drafted with certainty), or -1
    __device__ __forceinline__ long long at(int v) const {
        const long long a = (long long)fixed60(kda::io<T>::ld(p + v));
        if (q) return max(a - (long long)fixed60(kda::io<T>::ld(q + v)), 0ll);
        return v == masked ? 0ll : a;
    }
};

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Sum over [lo, hi), a warp's part, lanes side by side.
template <typename T>
__device__ __forceinline__ long long part_sum(const Row<T>& row, int lo, int hi) {
    const int lane = threadIdx.x & 31;
    long long s = 0;
    constexpr int kU = 4, kStep = 32 * kU;
    float a[kU], b[kU];
    // four numbers of either row in registers while the four behind them are on their way
    auto load = [&](int v, float* x, float* y) {
#pragma unroll
        for (int e = 0; e < kU; ++e) x[e] = v + 32 * e < hi ? kda::io<T>::ld(row.p + v + 32 * e) : 0.f;
        if (row.q) {
#pragma unroll
            for (int e = 0; e < kU; ++e) y[e] = v + 32 * e < hi ? kda::io<T>::ld(row.q + v + 32 * e) : 0.f;
        }
    };
    load(lo + lane, a, b);
    for (int v = lo + lane; v < hi; v += kStep) {
        float an[kU], bn[kU];
        load(v + kStep, an, bn);
#pragma unroll
        for (int e = 0; e < kU; ++e) {
            const long long x = (long long)fixed60(a[e]);
            if (row.q) s += max(x - (long long)fixed60(b[e]), 0ll);
            else s += v + 32 * e == row.masked ? 0ll : x;
            a[e] = an[e];
            b[e] = bn[e];
        }
    }
    return warp_sum(s);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kPerSm)
kda_verify_draft_kernel(const T* __restrict__ target, const T* __restrict__ draft,
                        const int32_t* __restrict__ draft_tokens, const float* __restrict__ uniforms,
                        const int32_t* __restrict__ draft_len, int K, int V, int32_t* __restrict__ tokens,
                        int32_t* __restrict__ commit_len) {
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int n = blockIdx.x / ranks;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    kda_paged::wait_for_stream();
    cluster.barrier_arrive();                              // waited for before the first remote store: by then all CTAs run
    __shared__ int s_count, s_len;
    __shared__ long long s_cta[2][8];                      // each CTA's sum, pushed by it; one row per attempt
    __shared__ long long s_warp[kWarps];
    __shared__ long long s_scan[kWarps];

    // ---- how many drafts stand: lane i tests draft i, every CTA for itself
    if (w == 0) {
        int len = K;
        if (draft_len) len = min(max(draft_len[n], 0), K);
        bool stands = false;
        if (lane < len) {
            const int x = draft_tokens[(size_t)n * K + lane];
            if (x >= 0 && x < V) {
                const float p = kda::io<T>::ld(target + ((size_t)n * (K + 1) + lane) * V + x);
                const float q = draft ? kda::io<T>::ld(draft + ((size_t)n * K + lane) * V + x) : 1.f;
                const float u = uniforms[(size_t)n * (K + 1) + lane];
                stands = (double)u * (double)q < (double)p;
            }
        }
        const unsigned fail = ~__ballot_sync(0xffffffffu, stands);
        if (lane == 0) {
            s_count = min(__ffs((int)fail) - 1, len);      // bits at and past len are set in `fail`
            s_len = len;
        }
    }
    __syncthreads();
    const int a = s_count;
    Row<T> row{target + ((size_t)n * (K + 1) + a) * V, nullptr, -1};
    if (a < s_len) {
        if (draft) row.q = draft + ((size_t)n * K + a) * V;
        else row.masked = draft_tokens[(size_t)n * K + a];
    }

    // ---- sums: CTA `rank` has [c0, c1), its warps equal parts of that
    const int c0 = (int)((long long)V * rank / ranks), c1 = (int)((long long)V * (rank + 1) / ranks);
    auto warp_lo = [&](int i) { return c0 + (int)((long long)(c1 - c0) * i / kWarps); };
    long long total = 0, before = 0, own = 0;
    for (int attempt = 0; attempt < 2; ++attempt) {
        const long long ws = part_sum(row, warp_lo(w), warp_lo(w + 1));
        if (lane == 0) s_warp[w] = ws;
        __syncthreads();
        if (attempt == 0) cluster.barrier_wait();
        if (w == 0) {
            long long c = lane < kWarps ? s_warp[lane] : 0;
            c = warp_sum(c);
            if (lane < ranks) *cluster.map_shared_rank(&s_cta[attempt][rank], lane) = c;
        }
        cluster.sync();
        total = before = 0;
        for (int r = 0; r < ranks; ++r) {
            const long long c = s_cta[attempt][r];
            if (r < rank) before += c;
            if (r == rank) own = c;
            total += c;
        }
        if (total > 0 || (!row.q && row.masked < 0)) break;
        row.q = nullptr;                                   // nothing is left of the row: draw from the target itself
        row.masked = -1;
        __syncthreads();
    }
    // no CTA touches another's shared memory past this point

    int32_t* out = tokens + (size_t)n * (K + 1);
    if (rank == 0) {
        if (tid <= K && tid != a) out[tid] = tid < a ? draft_tokens[(size_t)n * K + tid] : -1;
        if (tid == 0) {
            commit_len[n] = a + 1;
            if (total <= 0) out[a] = V - 1;
        }
    }
    if (total <= 0) return;
    // ---- the first element whose running sum exceeds thr = floor(u total); u at
    // or above 1 takes the last positive one, u below 0 or NaN the first
    const float u = uniforms[(size_t)n * (K + 1) + K];
    const double want = (double)u * (double)total;
    long long thr = want > 0.0 ? (want < 9.0e18 ? (long long)want : total) : 0;
    thr = min(thr, total - 1);
    if (thr < before || thr >= before + own) return;
    thr -= before;
    int part = 0;
    for (; part < kWarps - 1; ++part) {
        const long long c = s_warp[part];
        if (thr < c) break;
        thr -= c;
    }
    // every thread takes `per` consecutive elements of that warp's part
    const int lo = warp_lo(part), hi = warp_lo(part + 1), per = (hi - lo + kThreads - 1) / kThreads;
    const int v0 = min(lo + tid * per, hi), v1 = min(v0 + per, hi);
    long long mine = 0;
    for (int v = v0; v < v1; ++v) mine += row.at(v);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) s_scan[w] = incl;
    __syncthreads();
    for (int i = 0; i < w; ++i) incl += s_scan[i];
    if (thr >= incl - mine && thr < incl) {
        long long at = incl - mine;
        for (int v = v0; v < v1; ++v) {
            at += row.at(v);
            if (thr < at) {
                out[a] = v;
                break;
            }
        }
    }
}

template <typename T>
cudaError_t verify(const kda_host::VerifyArgs& a) {
    // CTAs per request: as many as the GPU holds at once, but no part of a row below 4096 numbers
    const long long fit = (long long)kPerSm * kda_host::sm_count() / a.N;
    const int ranks = (int)std::max<long long>(1, std::min<long long>({8, fit, a.V / 4096}));
    return kda_host::launch_overlapped(kda_verify_draft_kernel<T>, dim3((unsigned)a.N * ranks), kThreads, 0, a.stream,
                                       ranks, static_cast<const T*>(a.target), static_cast<const T*>(a.draft),
                                       a.draft_tokens, a.uniforms, a.draft_len, a.K, a.V, a.tokens, a.commit_len);
}

}  // namespace

namespace kda_host {

cudaError_t launch_verify_draft(const VerifyArgs& a) {
    return a.dtype == KDA_BF16 ? verify<__nv_bfloat16>(a) : verify<float>(a);
}

}  // namespace kda_host
