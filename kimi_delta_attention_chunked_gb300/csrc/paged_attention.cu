// paged_attention.cu -- attention over a paged cache on CUDA cores in fp32, and
// the merge of units that were cut between CTAs (paged.cuh).
//
// Per row (a new token and query head), over the keys it sees, in one pass:
//     m' = max(m, max_j s_j),  l' = l 2^(c (m - m')) + sum_j 2^(c (s_j - m')),
//     o' = o 2^(c (m - m')) + sum_j 2^(c (s_j - m')) v_j,   s_j = q.k_j,  c = scale log2(e)
// and o / l at the end; lse = (c m + log2 l) ln 2.  The factor comes last, so that no product of a query is out of
// fp32's range where the scores are not.
//
// This path is for fp32 (whose accuracy the tensor cores' 16-bit operands do
// not reach) and for rows of q that TMA cannot fetch.  A unit
// has up to 32 rows; a tile of 64 keys and values is brought to shared memory
// as fp32 and each of 256 threads forms 2 x 4 scores, then 4 rows x d / 32
// columns of the weighted sum.  Bound: fp32 issue (one shared-memory load per
// 2 to 4 multiply-adds) for many rows, the latency of a tile's loads for few: 6
// requests of 1 to 65 tokens over 17 to 2,100 keys, 8/2 heads of 64, 15.3 us with
// the merge (29 us before a tile's pages were looked up a tile ahead and the merge
// took several parts at once); one tile a CTA there.  1000 tokens over 3000 keys, 8/2 heads:
// 233 us with d = 64 and 390 us with 128, 22 and 26 TFLOP/s; bf16 rows of q off their
// 16-byte boundaries 396 us with d = 128 (41 us on the tensor cores).
#include <algorithm>

#include "paged.cuh"

namespace {

using kda_paged::Partials;
using kda_paged::Piece;
using kda_paged::Shape;
using kda_paged::Unit;
using kda_paged::Walker;

constexpr int kThreads = 256;
constexpr int kRows = 32;                              // rows of a unit
constexpr int kTileLog2 = 6;
constexpr int kTile = 1 << kTileLog2;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.44269504088896341f;

template <int D>
struct SimtSmem {
    float q[kRows][D];
    float k[kTile][D + 4];
    float v[kTile][D];
    float p[kRows][kTile + 4];                         // weights; -1 where the row does not see the key
    float scale[kRows];                                // factor of the earlier sums
};

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 2)
kda_paged_attention_simt_kernel(const T* __restrict__ q, const T* __restrict__ kc, const T* __restrict__ vc,
                                const int32_t* __restrict__ table, const int32_t* __restrict__ cu,
                                const int32_t* __restrict__ seq_len, long long q_stride, Shape s, float scale_log2,
                                T* __restrict__ o, float* __restrict__ lse, Partials parts) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    SimtSmem<D>& sm = *reinterpret_cast<SimtSmem<D>*>(smem_raw);
    __shared__ unsigned long long s_red[kThreads / 32];
    __shared__ Piece s_piece;
    __shared__ Unit s_unit;
    __shared__ int s_more;
    __shared__ int s_page[2][kTile / 16];              // pages of a tile, 16 keys each; -1: none
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    kda_paged::wait_for_stream();

    const Piece piece = kda_paged::find_piece<kThreads>(s, cu, seq_len, blockIdx.x, gridDim.x,
                                                        reinterpret_cast<unsigned long long*>(smem_raw), s_red,
                                                        &s_piece);
    Walker walk;
    if (w == 0) walk.start(s, cu, seq_len, piece, blockIdx.x);
    if (tid == 0) parts.clear(blockIdx.x);

    constexpr int VC = D / 32;                         // value columns per thread
    for (;;) {
        __syncthreads();                               // the unit before is done with shared memory
        if (w == 0) {
            Unit nu;
            const bool more = walk.next(s, cu, seq_len, nu);
            if (lane == 0) {
                s_unit = nu;
                s_more = more;
            }
        }
        __syncthreads();
        if (!s_more) break;
        const Unit u = s_unit;
        const int rows = u.ntok * s.Gv;
        for (int e = tid; e < kRows * D; e += kThreads) {
            const int r = e / D, c = e % D;
            float x = 0.f;
            if (r < rows)
                x = kda::io<T>::ld(q + (long long)(u.tok0 + r / s.Gv) * q_stride + (long long)(u.qh0 + r % s.Gv) * D + c);
            sm.q[r][c] = x;
        }
        // softmax state: 8 threads share a row
        const int sr = tid >> 3, sx = tid & 7;
        const int my_pos = u.pos + sr / s.Gv;
        const int my_hi = sr < rows ? min(my_pos + 1, u.kend) : 0;
        const int my_lo = kda_paged::first_key(my_pos, s.window);
        float m = -INFINITY, l = 0.f;
        float acc[4][VC];
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int c = 0; c < VC; ++c) acc[a][c] = 0.f;

        // the pages of a tile are looked up a tile ahead, so that its loads wait for one read, not two
        auto page_of = [&](int t) {
            const int key = (t << kTileLog2) + 16 * tid;
            int page = -1;
            if (key < u.kend) page = table[(size_t)u.n * s.blocks + (key >> s.page_log2)];
            return page < s.n_pages ? page : -1;
        };
        if (tid < kTile / 16) s_page[u.tb & 1][tid] = page_of(u.tb);
        for (int t = u.tb; t < u.te; ++t) {
            const int key0 = t << kTileLog2;
            __syncthreads();                           // q and the pages stored; the tile before is consumed
            const int* pages = s_page[t & 1];
            int next_page = -1;
            if (tid < kTile / 16 && t + 1 < u.te) next_page = page_of(t + 1);
            // keys and values of the tile; places without a key become zero
            constexpr int VEC = 16 / sizeof(T), CH = D / VEC;        // the cache is 16-byte aligned
            constexpr int kIter = kTile * CH / kThreads, kBatch = kIter < 4 ? kIter : 4;
            static_assert(kIter >= 1 && kIter % kBatch == 0, "tile");
#pragma unroll
            for (int i0 = 0; i0 < kIter; i0 += kBatch) {
                uint4 ka[kBatch], va[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int e = tid + (i0 + i) * kThreads, j = e / CH, c = (e % CH) * VEC, key = key0 + j;
                    const int page = pages[j >> 4];
                    ka[i] = va[i] = make_uint4(0, 0, 0, 0);
                    if (page >= 0 && key < u.kend) {
                        const size_t off =
                            ((((size_t)page * s.Hkv + u.kvh) << s.page_log2) + (key & ((1 << s.page_log2) - 1))) * D + c;
                        ka[i] = *reinterpret_cast<const uint4*>(kc + off);
                        va[i] = *reinterpret_cast<const uint4*>(vc + off);
                    }
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int e = tid + (i0 + i) * kThreads, j = e / CH, c = (e % CH) * VEC;
                    const T* kt = reinterpret_cast<const T*>(&ka[i]);
                    const T* vt = reinterpret_cast<const T*>(&va[i]);
#pragma unroll
                    for (int x = 0; x < VEC; x += 4) {
                        *reinterpret_cast<float4*>(&sm.k[j][c + x]) =
                            make_float4(kda::io<T>::ld(kt + x), kda::io<T>::ld(kt + x + 1), kda::io<T>::ld(kt + x + 2),
                                        kda::io<T>::ld(kt + x + 3));
                        *reinterpret_cast<float4*>(&sm.v[j][c + x]) =
                            make_float4(kda::io<T>::ld(vt + x), kda::io<T>::ld(vt + x + 1), kda::io<T>::ld(vt + x + 2),
                                        kda::io<T>::ld(vt + x + 3));
                    }
                }
            }
            if (tid < kTile / 16 && t + 1 < u.te) s_page[(t + 1) & 1][tid] = next_page;
            // which of the keys this thread judges below (sx + 8 i) exist
            unsigned exists = 0;
#pragma unroll
            for (int i = 0; i < kTile / 8; ++i)
                if (key0 + sx + 8 * i < u.kend && pages[i >> 1] >= 0) exists |= 1u << i;
            __syncthreads();
            // scores: rows 2 ty, 2 ty + 1, keys tx + 16 i
            {
                const int ty = tid >> 4, tx = tid & 15;
                float a[2][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[0][i] = a[1][i] = 0.f;
                for (int c = 0; c < D; c += 4) {
                    const float4 q0 = *reinterpret_cast<const float4*>(&sm.q[2 * ty][c]);
                    const float4 q1 = *reinterpret_cast<const float4*>(&sm.q[2 * ty + 1][c]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 kk = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * i][c]);
                        a[0][i] = fmaf(q0.x, kk.x, fmaf(q0.y, kk.y, fmaf(q0.z, kk.z, fmaf(q0.w, kk.w, a[0][i]))));
                        a[1][i] = fmaf(q1.x, kk.x, fmaf(q1.y, kk.y, fmaf(q1.z, kk.z, fmaf(q1.w, kk.w, a[1][i]))));
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sm.p[2 * ty][tx + 16 * i] = a[0][i];
                    sm.p[2 * ty + 1][tx + 16 * i] = a[1][i];
                }
            }
            __syncthreads();
            // softmax statistics of row sr
            {
                float x[kTile / 8];
                float top = -INFINITY;
                unsigned seen = 0;
#pragma unroll
                for (int i = 0; i < kTile / 8; ++i) {
                    const int key = key0 + sx + 8 * i;
                    x[i] = sm.p[sr][sx + 8 * i];
                    if (((exists >> i) & 1) && key >= my_lo && key < my_hi) {
                        seen |= 1u << i;
                        top = fmaxf(top, x[i]);
                    }
                }
#pragma unroll
                for (int d = 4; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn;
                const float f = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : exp2f((m - ref) * scale_log2);
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < kTile / 8; ++i) {
                    const float p = (seen >> i) & 1 ? exp2f((x[i] - ref) * scale_log2) : -1.f;
                    if ((seen >> i) & 1) sum += p;
                    sm.p[sr][sx + 8 * i] = p;
                }
#pragma unroll
                for (int d = 4; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                l = fmaf(l, f, sum);
                m = mn;
                if (sx == 0) sm.scale[sr] = f;
            }
            __syncthreads();
            // weighted sums: rows 4 w .. 4 w + 3, columns lane + 32 c; a masked key is
            // passed over, not multiplied by zero, so that what stands there stays out
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const float f = sm.scale[4 * w + a];
#pragma unroll
                for (int c = 0; c < VC; ++c) acc[a][c] *= f;
            }
            if (4 * w < rows) {
                for (int j = 0; j < kTile; j += 4) {
                    float4 p[4];
#pragma unroll
                    for (int a = 0; a < 4; ++a) p[a] = *reinterpret_cast<const float4*>(&sm.p[4 * w + a][j]);
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj) {
                        float vv[VC];
#pragma unroll
                        for (int c = 0; c < VC; ++c) vv[c] = sm.v[j + jj][lane + 32 * c];
#pragma unroll
                        for (int a = 0; a < 4; ++a) {
                            const float pj = jj == 0 ? p[a].x : jj == 1 ? p[a].y : jj == 2 ? p[a].z : p[a].w;
                            if (pj != -1.f) {
#pragma unroll
                                for (int c = 0; c < VC; ++c) acc[a][c] = fmaf(pj, vv[c], acc[a][c]);
                            }
                        }
                    }
                }
            }
        }
        // the row's statistics to the threads that hold its sums
        __syncthreads();
        if (sx == 0) {
            const float2 st = kda_paged::row_stats(m, l, scale_log2, INFINITY);
            sm.p[sr][0] = st.x;
            sm.p[sr][1] = st.y;
        }
        __syncthreads();
        const bool whole = u.first && u.last;
        const int which = u.first ? 1 : 0;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const int r = 4 * w + a;
            if (r >= rows) continue;
            const float rm = sm.p[r][0];
            float rl = sm.p[r][1];
            if (whole) {
                rl = kda_paged::whole_sum(rm, rl);
                const float inv = rl == 0.f ? 0.f : 1.f / rl;
                const size_t at = (size_t)(u.tok0 + r / s.Gv) * s.Hq + u.qh0 + r % s.Gv;
#pragma unroll
                for (int c = 0; c < VC; ++c) kda::io<T>::st(o + at * D + lane + 32 * c, acc[a][c] * inv);
                if (lse && lane == 0) lse[at] = rl == 0.f ? -INFINITY : (rm + log2f(rl)) * kLn2;
            } else {
                float* dst = parts.sums(blockIdx.x, which) + (size_t)r * D;
#pragma unroll
                for (int c = 0; c < VC; ++c) dst[lane + 32 * c] = acc[a][c];
                if (lane == 0) parts.stats(blockIdx.x, which)[r] = make_float2(rm, rl);
            }
        }
        if (tid == 0) parts.describe(blockIdx.x, u);
    }
}

// Joins the parts of each cut unit: with M = max of the parts' references,
//     o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i.
// The blocks of the CTA in which a unit begins take its rows; of one of kSpread parts
// and more than kSpreadRows rows the blocks of all its CTAs do (few units, cut many times:
// 8 units of 252 rows in 19 parts: the whole call 74 us without, 42 with).  D / 4 threads
// take the columns of a row and four parts at once; where a unit has more, up to eight
// such groups share out a row's parts.  Reads each partial row once.  Bound:
// latency (description, parts, the first fetch of its instructions, so it is kept
// short): 3 us for a few cut units, 4 to 6 us for a cut in each of 152 CTAs of 64 to 256 rows.
constexpr int kMergeThreads = 256, kSpread = 6;
__device__ __forceinline__ float merge_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int D, typename T>
__global__ void __launch_bounds__(kMergeThreads, 5)
kda_paged_merge_kernel(Partials parts, int Gv, int Hq, T* __restrict__ o, float* __restrict__ lse) {
    constexpr int TPR = D / 4, GROUPS = kMergeThreads / TPR, kU = 4;
    __shared__ float4 s_acc[kMergeThreads];
    __shared__ float2 s_st[GROUPS];
    kda_paged::wait_for_stream();
    const int c = blockIdx.x;
    const int4 mine = parts.meta[2 * c + 1 - blockIdx.z];     // z = 0: the unit that begins here, 1: the one that goes on here
    const int c0 = blockIdx.z == 0 ? c : mine.x;
    if (blockIdx.z == 1 && (c0 < 0 || c0 >= c || mine.y < kSpread)) return;
    const int4 me = blockIdx.z == 0 ? mine : parts.meta[2 * c0 + 1];
    if (me.w == 0) return;
    const int x = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int rows = me.z * Gv, n = me.w;
    int share = 1;                                     // groups that share a row
    while (share * kU < n && share < 8 && share < GROUPS) share <<= 1;
    const int y = grp % share, per_pass = GROUPS / share;
    const bool spread = n >= kSpread && rows > kda_paged::kSpreadRows;
    const int step = (spread ? n : 1) * gridDim.y * per_pass;
#pragma unroll 1
    for (int r0 = ((c - c0) * gridDim.y + blockIdx.y) * per_pass; r0 < rows; r0 += step) {
        const int r = min(r0 + grp / share, rows - 1);
        float top = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        // kU more weighted sums into (top, l, acc); st.y = 0 marks a part that saw no key
        auto add = [&](const float2* st, const float4* v) {
            float m = top;
#pragma unroll
            for (int e = 0; e < kU; ++e) m = fmaxf(m, st[e].x);
            const float ref = m == -INFINITY ? 0.f : m, f = merge_ex2(top - ref);
            top = m;
            l *= f;
            acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
#pragma unroll
            for (int e = 0; e < kU; ++e) {
                const float g = st[e].y == 0.f ? 0.f : merge_ex2(st[e].x - ref);
                l = fmaf(g, st[e].y, l);
                acc.x = fmaf(g, v[e].x, acc.x); acc.y = fmaf(g, v[e].y, acc.y);
                acc.z = fmaf(g, v[e].z, acc.z); acc.w = fmaf(g, v[e].w, acc.w);
            }
        };
        float2 st[kU];
        float4 v[kU];
#pragma unroll 1
        for (int i0 = y; i0 < n; i0 += kU * share) {
#pragma unroll
            for (int e = 0; e < kU; ++e) {
                const int i = i0 + e * share;
                st[e] = make_float2(-INFINITY, 0.f);
                v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < n) {
                    st[e] = parts.stats(c0 + i, i == 0 ? 1 : 0)[r];
                    v[e] = reinterpret_cast<const float4*>(parts.sums(c0 + i, i == 0 ? 1 : 0) + (size_t)r * D)[x];
                }
            }
            add(st, v);
        }
        if (share > 1) {
            __syncthreads();                           // the pass before has been read
            s_acc[threadIdx.x] = acc;
            if (x == 0) s_st[grp] = make_float2(top, l);
            __syncthreads();
            if (y != 0) continue;
            top = -INFINITY;
            l = 0.f;
            acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int g = 0; g < share; g += kU) {      // share is 2, 4 or 8
#pragma unroll
                for (int e = 0; e < kU; ++e) {
                    const bool in = g + e < share;
                    st[e] = in ? s_st[grp + g + e] : make_float2(-INFINITY, 0.f);
                    v[e] = in ? s_acc[threadIdx.x + (g + e) * TPR] : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                add(st, v);
            }
        }
        if (r0 + grp / share >= rows) continue;
        l = kda_paged::whole_sum(top, l);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const size_t at = (size_t)(me.x + r / Gv) * Hq + me.y + r % Gv;
        T* dst = o + at * D + 4 * x;
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(kda::pack_bf16x2(acc.x * inv, acc.y * inv), kda::pack_bf16x2(acc.z * inv, acc.w * inv));
        } else {
            *reinterpret_cast<float4*>(dst) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        }
        if (lse && x == 0) lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
    }
}

template <int D, typename T>
cudaError_t launch_merge(const kda_host::PagedArgs& a, const kda_host::PagedPlan& p, int ctas) {
    // the same split of L1 and shared memory as the attention kernel before it: an SM
    // must run dry to change it
    static kda_host::OncePerDevice once;
    const cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(kda_paged_merge_kernel<D, T>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                    cudaSharedmemCarveoutMaxShared);
    });
    if (e != cudaSuccess) return e;
    return kda_host::launch_overlapped(kda_paged_merge_kernel<D, T>, dim3(ctas, std::min(10, p.rows), p.rows > kda_paged::kSpreadRows ? 2 : 1), kMergeThreads, 0,
                                       a.stream, 1, kda_host::paged_partials(a, p), p.Gv, a.Hq, static_cast<T*>(a.o),
                                       a.lse);
}

template <int D, typename T>
cudaError_t launch_simt(const kda_host::PagedArgs& a) {
    const kda_host::PagedPlan p = kda_host::paged_plan_simt(a.T, a.Hq, a.Hkv, a.d);
    const size_t smem = std::max(sizeof(SimtSmem<D>), (size_t)a.N * sizeof(unsigned long long));
    auto kern = kda_paged_attention_simt_kernel<D, T>;
    static kda_host::OncePerDevice once;
    const cudaError_t e = once.run([&] {
        constexpr size_t most = std::max(sizeof(SimtSmem<D>), (size_t)kda_paged::kMaxRequests * 8);
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    });
    if (e != cudaSuccess) return e;
    const int ctas = std::min(p.max_ctas, 2 * kda_host::sm_count());
    const cudaError_t err = kda_host::launch_overlapped(
        kern, ctas, kThreads, smem, a.stream, 1, static_cast<const T*>(a.q), static_cast<const T*>(a.k_cache), static_cast<const T*>(a.v_cache), a.block_table,
        a.cu_seqlens, a.seq_len, a.q_stride, kda_host::paged_shape(a, p), a.scale * kLog2e, static_cast<T*>(a.o), a.lse,
        kda_host::paged_partials(a, p));
    if (err != cudaSuccess) return err;
    return kda_host::launch_paged_merge(a, p, ctas);
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

namespace kda_host {

int sm_count() {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> counts[kMaxDevices] = {};  // 0: not asked yet; threads that ask at once store the same value
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        (void)cudaGetLastError();
        return 148;
    }
    int n = counts[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
            (void)cudaGetLastError();
            return 148;
        }
        counts[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

PagedPlan paged_plan_simt(int T, int Hq, int Hkv, int d) {
    PagedPlan p;
    (void)d;
    p.Gv = heads_per_unit(Hq / Hkv, kRows);
    p.U = kRows / p.Gv;
    p.rows = kda_host::paged_slot_rows(p.U, T, p.Gv);
    p.tile_log2 = kTileLog2;
    p.max_ctas = 304;
    p.extra = 0;
    return p;
}

// A multiple of 4, so that every slot and its statistics start on a 16-byte
// boundary (a row has d + 2 floats).
int paged_slot_rows(int U, int T, int Gv) { return (std::min(U, std::max(T, 1)) * Gv + 3) & ~3; }

size_t paged_plan_bytes(const PagedPlan& p, int d) {
    return up256((size_t)p.max_ctas * 2 * sizeof(int4)) + up256((size_t)p.max_ctas * 2 * p.rows * (d + 2) * sizeof(float));
}

kda_paged::Shape paged_shape(const PagedArgs& a, const PagedPlan& p) {
    Shape s;
    s.n_req = a.N;
    s.T = a.T;
    s.Hq = a.Hq;
    s.Hkv = a.Hkv;
    s.Gv = p.Gv;
    s.Hv = a.Hq / p.Gv;
    s.sub = s.Hv / a.Hkv;
    s.blocks = a.blocks;
    s.page_log2 = 0;
    while ((1 << s.page_log2) < a.page_size) ++s.page_log2;
    s.n_pages = a.n_pages;
    s.window = a.window;
    s.U = p.U;
    s.tile_log2 = p.tile_log2;
    s.extra = p.extra;
    return s;
}

kda_paged::Partials paged_partials(const PagedArgs& a, const PagedPlan& p) {
    Partials x;
    x.meta = static_cast<int4*>(a.workspace);
    x.rows = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + up256((size_t)p.max_ctas * 2 * sizeof(int4)));
    x.cap = p.rows;
    x.d = a.d;
    return x;
}

cudaError_t launch_paged_merge(const PagedArgs& a, const PagedPlan& p, int ctas) {
    const bool wide = a.dtype == KDA_BF16;
    switch (a.d) {
        case 32: return wide ? launch_merge<32, __nv_bfloat16>(a, p, ctas) : launch_merge<32, float>(a, p, ctas);
        case 64: return wide ? launch_merge<64, __nv_bfloat16>(a, p, ctas) : launch_merge<64, float>(a, p, ctas);
        case 128: return wide ? launch_merge<128, __nv_bfloat16>(a, p, ctas) : launch_merge<128, float>(a, p, ctas);
    }
    return cudaErrorNotSupported;
}

cudaError_t launch_paged_attention_simt(const PagedArgs& a) {
    const bool wide = a.dtype == KDA_BF16;
    switch (a.d) {
        case 32: return wide ? launch_simt<32, __nv_bfloat16>(a) : launch_simt<32, float>(a);
        case 64: return wide ? launch_simt<64, __nv_bfloat16>(a) : launch_simt<64, float>(a);
        case 128: return wide ? launch_simt<128, __nv_bfloat16>(a) : launch_simt<128, float>(a);
    }
    return cudaErrorNotSupported;
}

}  // namespace kda_host
