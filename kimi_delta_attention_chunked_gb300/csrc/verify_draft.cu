// verify_draft.cu -- acceptance of drafted tokens and the draw of the next one.
//
// Per request: draft i stands while u_i q_i(x_i) < p_i(x_i) (the product of two
// fp32 numbers is exact in fp64, so the comparison is exact), a is the number
// that stand, and one token is drawn from r = max(p_a - q_a, 0) (r = p_a when
// all stand): the first v with sum_{v' <= v} r_v' > u_K sum r.
//
// The drawn index is a whole number that must not depend on how the sum was
// cut up, and in fp32 the running sum of 10^5 probabilities is off by more than
// many of them.  So the sums are in integers, which no order of summation
// changes, in two forms:
//   exact  p -> floor(p 2^60), the mantissa shifted in 64 bits: 12 integer
//          instructions a number, more than the memory gives time for;
//   quick  p -> round(p 2^46), from the bits of two fp32 sums: with x = fl(p + 1),
//          bits(x) - bits(1) = round(p 2^23), and with l = p - (x - 1) (exact),
//          bits(l 2^23 + 1.5) - bits(1.5) = round(l 2^46): 5 fp32 instructions.
// A quick sum is off by at most one unit a term.  Where that could decide the index
// (the threshold that near a border of the element found, or next to no sum; about once
// in 3000 draws at V = 160,000) one CTA does the row again in the exact form, which adds
// 42 us there: 240 us with one read in flight a thread in place of 16.
//
// A cluster of CTAs takes one request: each sums its part of the row, the parts
// are exchanged through distributed shared memory, and the CTA that holds the
// crossing finds the warp's part, then the element, by scanning again what is
// by then in L2.  Only row a is read: bound by HBM, 2 V numbers a request.
// 128 requests, V = 160,001, fp32 (164 MB, floor 24.5 us), GPU time: 47 us with
// the exact form throughout (issue bound), 37 us with the quick one.  Then three
// CTAs of 512 threads an SM, 8 numbers of each row in flight a thread: 43 us with six of 256 (more,
// smaller clusters wait longer for each other), 39 us with 4 numbers, 47 us with two of 1024,
// 49 us with clusters of four, 39 to 44 us with the row's start fetched into L2 ahead.
// bf16 rows 32 us (floor 12.2: half the bytes, the same sums, 2-byte loads); without draft rows
// 22 us in fp32 and 21 us in bf16.
// What is left of it: the chain before the row (length, token, two probabilities: three
// dependent reads) and behind it (cluster barrier, second scan), in which nothing streams.
#include <algorithm>
#include <cooperative_groups.h>

#include "paged.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPerSm = 3;                              // CTAs of an SM

// A probability as it counts: 0 ... 1, NaN as 0.
__device__ __forceinline__ float clean(float p) { return __saturatef(p); }

// floor(p 2^60) of a clean p
__device__ __forceinline__ unsigned long long fixed60(float p) {
    const unsigned b = __float_as_uint(p);
    const unsigned long long m = (unsigned long long)((b & 0x7fffffu) | 0x800000u) << 37;
    return m >> min(127u - (b >> 23), 63u);                // p = 1.m 2^(e - 127), e <= 127; below 2^-60: 0
}

// The two words of a clean p in the quick form, each with the bits of its constant added.
__device__ __forceinline__ void quick_words(float p, int& hi, int& lo) {
    const float x = __fadd_rn(p, 1.f);
    hi = __float_as_int(x);
    lo = __float_as_int(__fmaf_rn(__fadd_rn(p, -__fadd_rn(x, -1.f)), 8388608.f, 1.5f));
}
constexpr int kHiBits = 0x3f800000, kLoBits = 0x3fc00000;  // of 1 and 1.5

template <typename T>
struct Row {
    const T* p;
    const T* q;                                            // nullptr: no draft row
    int masked;                                            // index with q = 1 (a token drafted with certainty), or -1
    // element v, in units of 2^-60 (exact) or 2^-46
    template <bool kExact>
    __device__ __forceinline__ long long at(int v) const {
        const float a = clean(kda::io<T>::ld(p + v));
        if (!q && v == masked) return 0;
        const float b = q ? clean(kda::io<T>::ld(q + v)) : 0.f;
        if (!(a > b)) return 0;
        if constexpr (kExact) {
            return (long long)(fixed60(a) - fixed60(b));
        } else {
            int ah, al, bh, bl;
            quick_words(a, ah, al);
            quick_words(b, bh, bl);
            return ((long long)(ah - bh) << 23) + (al - bl);
        }
    }
};

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Quick sum over [lo, hi), a warp's part, lanes side by side.
template <typename T>
__device__ __forceinline__ long long quick_sum(const Row<T>& row, int lo, int hi) {
    const int lane = threadIdx.x & 31;
    constexpr int kU = 8;
    long long s = 0;
    int v = lo + lane;
    for (; v + 32 * (kU - 1) < hi; v += 32 * kU) {
        float a[kU], b[kU];
#pragma unroll
        for (int e = 0; e < kU; ++e) a[e] = kda::io<T>::ld(row.p + v + 32 * e);
        int h = 0, l = 0;                                  // of 8 numbers: |h| <= 2^26, |l| <= 2^26
        if (row.q) {
#pragma unroll
            for (int e = 0; e < kU; ++e) b[e] = kda::io<T>::ld(row.q + v + 32 * e);
#pragma unroll
            for (int e = 0; e < kU; ++e) {
                const float x = clean(a[e]), y = clean(b[e]);
                int xh, xl, yh, yl;
                quick_words(x, xh, xl);
                quick_words(y, yh, yl);
                if (x > y) {
                    h += xh - yh;
                    l += xl - yl;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < kU; ++e) {
                int xh, xl;
                quick_words(clean(a[e]), xh, xl);
                if (v + 32 * e != row.masked) {
                    h += xh - kHiBits;
                    l += xl - kLoBits;
                }
            }
        }
        s += ((long long)h << 23) + l;
    }
#pragma unroll 4
    for (; v < hi; v += 32) s += row.template at<false>(v);
    return warp_sum(s);
}

// floor(u total), inside [0, total - 1]: u at or above 1 takes the last positive
// element, u below 0 or NaN the first.  In whole numbers: u is m 2^-shift, the product
// has up to 87 bits, and fp64 would round it.
__device__ __forceinline__ long long threshold(float u, long long total) {
    if (!(u > 0.f)) return 0;
    if (u >= 1.f) return total - 1;
    const int b = __float_as_int(u), ex = max(b >> 23, 1), shift = 150 - ex;   // 24 ... 149
    const unsigned long long m = (b & 0x7fffff) | (b >> 23 ? 0x800000 : 0);
    const unsigned long long lo = m * (unsigned long long)total, hi = __umul64hi(m, total);
    if (shift < 64) return (long long)(hi << (64 - shift) | lo >> shift);
    return shift < 128 ? (long long)(hi >> (shift - 64)) : 0;
}

// The element of [c0, c1) at which the running sum passes `thr`, given its warps'
// parts in s_warp; the sum before it in `before`, its own value in `value`.  All threads of the
// block call it; the one that finds it gets the index, the others -1.
template <bool kExact, typename T, typename F>
__device__ __forceinline__ int locate(const Row<T>& row, F part_lo, long long thr, const long long* s_warp,
                                      long long* s_scan, long long& before, long long& value) {
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    long long base = 0;
    int part = 0;
    for (; part < kWarps - 1 && thr >= base + s_warp[part]; ++part) base += s_warp[part];
    // every thread takes `per` consecutive elements of that warp's part
    const int lo = part_lo(part), hi = part_lo(part + 1), per = (hi - lo + kThreads - 1) / kThreads;
    const int v0 = min(lo + tid * per, hi), v1 = min(v0 + per, hi);
    long long mine = 0;
    for (int v = v0; v < v1; ++v) mine += row.template at<kExact>(v);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) s_scan[w] = incl;
    __syncthreads();
    incl += base;
    for (int i = 0; i < w; ++i) incl += s_scan[i];
    before = incl - mine;
    if (thr < before || thr >= incl) return -1;
    for (int v = v0; v < v1; ++v) {
        value = row.template at<kExact>(v);
        if (thr < before + value) return v;
        before += value;
    }
    return -1;
}

// Exact sum over [lo, hi), a warp's part, lanes side by side.
template <typename T>
__device__ __forceinline__ long long exact_sum(const Row<T>& row, int lo, int hi) {
    const int lane = threadIdx.x & 31;
    constexpr int kU = 8;
    long long s = 0;
    int v = lo + lane;
    for (; v + 32 * (kU - 1) < hi; v += 32 * kU) {         // all reads ahead of the first use
        float a[kU], b[kU];
#pragma unroll
        for (int e = 0; e < kU; ++e) a[e] = kda::io<T>::ld(row.p + v + 32 * e);
#pragma unroll
        for (int e = 0; e < kU; ++e) b[e] = row.q ? kda::io<T>::ld(row.q + v + 32 * e) : v + 32 * e == row.masked ? 1.f : 0.f;
#pragma unroll
        for (int e = 0; e < kU; ++e) {
            const float x = clean(a[e]), y = clean(b[e]);
            if (x > y) s += (long long)(fixed60(x) - fixed60(y));
        }
    }
#pragma unroll 4
    for (; v < hi; v += 32) s += row.template at<true>(v);
    return warp_sum(s);
}

// The whole draw in the exact form, by one CTA.
template <typename T>
__device__ __noinline__ void draw_exact(Row<T> row, int V, float u, int32_t* out, long long* s_warp, long long* s_scan) {
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    auto part_lo = [&](int i) { return (int)((long long)V * i / kWarps); };
    long long total = 0;
    for (int attempt = 0; attempt < 2; ++attempt) {
        const long long s = exact_sum(row, part_lo(w), part_lo(w + 1));
        __syncthreads();
        if (lane == 0) s_warp[w] = s;
        __syncthreads();
        total = 0;
        for (int i = 0; i < kWarps; ++i) total += s_warp[i];
        if (total > 0 || (!row.q && row.masked < 0)) break;
        row.q = nullptr;                                   // nothing is left of the row: draw from the target itself
        row.masked = -1;
    }
    if (total <= 0) {
        if (tid == 0) *out = V - 1;
        return;
    }
    long long before, value;
    const int v = locate<true>(row, part_lo, threshold(u, total), s_warp, s_scan, before, value);
    if (v >= 0) *out = v;
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
    __shared__ int s_count, s_len, s_unsure;
    __shared__ long long s_cta[8];                         // each CTA's sum, pushed by it
    __shared__ long long s_warp[kWarps];
    __shared__ long long s_scan[kWarps];

    // ---- how many drafts stand: lane i tests draft i, every CTA for itself
    if (w == 0) {
        int len = K;
        if (draft_len) len = min(max(draft_len[n], 0), K);
        bool stands = false;
        if (lane < K) {                                    // not `len`: the two reads go out together
            const int x = draft_tokens[(size_t)n * K + lane];
            if (x >= 0 && x < V) {
                const float p = kda::io<T>::ld(target + ((size_t)n * (K + 1) + lane) * V + x);
                float q = draft ? kda::io<T>::ld(draft + ((size_t)n * K + lane) * V + x) : 1.f;
                if (q < 0.f) q = 0.f;                      // or a token with p = 0 would stand; a NaN fails the test below
                const float u = uniforms[(size_t)n * (K + 1) + lane];
                stands = lane < len && (double)u * (double)q < (double)p;
            }
        }
        const unsigned fail = ~__ballot_sync(0xffffffffu, stands);
        if (lane == 0) {
            s_count = min(__ffs((int)fail) - 1, len);      // bits at and past len are set in `fail`
            s_len = len;
            s_unsure = 0;
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
    auto part_lo = [&](int i) { return c0 + (int)((long long)(c1 - c0) * i / kWarps); };
    const long long ws = quick_sum(row, part_lo(w), part_lo(w + 1));
    if (lane == 0) s_warp[w] = ws;
    __syncthreads();
    cluster.barrier_wait();
    if (w == 0) {
        const long long c = warp_sum(lane < kWarps ? s_warp[lane] : 0);
        if (lane < ranks) *cluster.map_shared_rank(&s_cta[rank], lane) = c;
    }
    cluster.sync();
    // no CTA touches another's shared memory past this point
    long long total = 0, before = 0;
    for (int r = 0; r < ranks; ++r) {
        if (r < rank) before += s_cta[r];
        total += s_cta[r];
    }
    int32_t* out = tokens + (size_t)n * (K + 1);
    if (rank == 0) {
        if (tid <= K && tid != a) out[tid] = tid < a ? draft_tokens[(size_t)n * K + tid] : -1;
        if (tid == 0) commit_len[n] = a + 1;
    }
    const float u = uniforms[(size_t)n * (K + 1) + K];
    if (total <= 2ll * V + 2) {                            // next to nothing is left of the row
        if (rank == 0) draw_exact(row, V, u, out + a, s_warp, s_scan);
        return;
    }
    const long long thr = threshold(u, total) - before;
    if (thr < 0 || thr >= s_cta[rank]) return;
    long long sum, value;
    const int v = locate<false>(row, part_lo, thr, s_warp, s_scan, sum, value);
    if (v >= 0) {
        // by how much sum - u total can be off here: (1 - u) times the v elements before, u times
        // those behind, a unit each (half of one without a draft row); 2^-10 more for the exact
        // form's own floor (2^-14) and for the fp32 of this line
        const float f = __saturatef(u), unit = row.q ? 1.f + 0x1p-10f : 0.5f + 0x1p-10f;
        const long long margin = (long long)(unit * ((1.f - f) * v + f * (V - v))) + 4;
        if (thr - sum >= margin && sum + value - thr > margin) out[a] = v;
        else s_unsure = 1;
    }
    __syncthreads();
    if (s_unsure) draw_exact(row, V, u, out + a, s_warp, s_scan);
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
