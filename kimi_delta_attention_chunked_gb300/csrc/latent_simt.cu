// latent_simt.cu -- both forms of latent attention on CUDA cores in fp32: absorbed
// over the paged latent cache, expanded over packed keys and values.
//
// Per row (a new token and a query head), over the keys it sees, in one pass:
//     m' = max(m, max_j s_j),  l' = l 2^(c (m - m')) + sum_j 2^(c (s_j - m')),
//     o' = o 2^(c (m - m')) + sum_j 2^(c (s_j - m')) v_j,   s_j = q.k_j,  c = scale log2(e)
// and o / l at the end; lse = (c m + log2 l) ln 2.  The factor comes last, so that no product of a query is out of
// fp32's range where the scores are not.  In the absorbed form k_j is a row of the
// cache and v_j its first 512 channels, so a tile is fetched once for both.
//
// This path is for fp32, whose accuracy the tensor cores' 16-bit operands do not reach, and
// for bf16 rows that TMA cannot fetch.  A tile of 32 keys lies in shared memory as fp32; the
// threads form 4 x 4 scores each (over a part of the channels: the parts are added up in the
// softmax step), then DV / 4 column groups of 4 with ROWS / RPT row groups of RPT rows each.
// Bound: latency of a tile's loads and steps, then shared memory (a 16-byte load of a warp takes four cycles,
// whatever its addresses): 6 requests of 1 to 9 tokens over 17 to 2100 keys, 5 heads, absorbed, 20.6 us with the
// merge; 5 prompts of 3 to 260 tokens over up to 860 keys, 5 heads, expanded, 34 to 37 us; 4 of 200
// over 2000, 8 heads, 360.  Long contexts are bound by shared memory, not by HBM: 64 requests of one token over 8192
// keys, 16 heads, absorbed, 683 us (bytes: 179), 16 prompts of 32 over 4032, 16 heads, expanded, 848 us (160).
#include <algorithm>
#include <type_traits>

#include "latent.cuh"

namespace {

using kda_latent::kKey;
using kda_latent::kLatent;
using kda_latent::kNope;
using kda_latent::kRope;
using kda_latent::kRow;
using kda_latent::kValue;
using kda_paged::PackedShape;
using kda_paged::Partials;
using kda_paged::Piece;
using kda_paged::Shape;
using kda_paged::Unit;
using kda_paged::Walker;

constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.44269504088896341f;

// Where the keys and values of the absorbed form lie.
template <typename T>
struct Absorbed {
    static constexpr int DK = kRow, DV = kLatent, ROWS = 16, LOG2 = 5, THREADS = 512, BLOCKS = 1;
    static constexpr bool kShared = true;              // values are the keys' first channels
    using Sh = Shape;
    const T* cache;
    const int32_t* table;
    // row of a key, or -1 where its page does not exist
    __device__ __forceinline__ long long place(const Shape& s, const Unit& u, int key) const {
        const int page = table[(size_t)u.n * s.blocks + (key >> s.page_log2)];
        if (page < 0 || page >= s.n_pages) return -1;
        return ((long long)page << s.page_log2) + (key & ((1 << s.page_log2) - 1));
    }
    // VEC channels from c on, c a multiple of VEC
    __device__ __forceinline__ const T* key(long long at, int, int c) const { return cache + at * kRow + c; }
    __device__ __forceinline__ const T* value(long long, int, int) const { return nullptr; }
};

// And of the expanded one.
template <typename T>
struct Expanded {
    static constexpr int DK = kKey, DV = kValue, ROWS = 32, LOG2 = 5, THREADS = 256, BLOCKS = 2;
    static constexpr bool kShared = false;
    using Sh = PackedShape;
    const T *k_nope, *k_rope, *v;
    long long kn_token, kn_head, kr_stride, v_token, v_head;
    const int32_t* cu_k;
    __device__ __forceinline__ long long place(const PackedShape& s, const Unit& u, int key) const {
        return (long long)min(max(cu_k[u.n], 0), s.S) + key;
    }
    __device__ __forceinline__ const T* key(long long at, int head, int c) const {
        return c < kNope ? k_nope + at * kn_token + head * kn_head + c : k_rope + at * kr_stride + (c - kNope);
    }
    __device__ __forceinline__ const T* value(long long at, int head, int c) const {
        return v + at * v_token + head * v_head + c;
    }
};

template <class Src>
struct Smem {
    static constexpr int kTile = 1 << Src::LOG2;       // keys of a tile
    float q[Src::ROWS][Src::DK + 4];                   // rows of q and k 16 bytes on in the banks from one to the next
    float k[kTile][Src::DK + 4];
    float v[Src::kShared ? 1 : kTile][Src::DV];
    static constexpr int SPLIT = Src::THREADS / (Src::ROWS / 4 * (kTile / 4));    // parts of the channels
    float part[SPLIT][Src::ROWS][kTile + 1];
    float p[kTile][Src::ROWS];                         // weights; -1 where the row does not see the key
    float scale[Src::ROWS];                            // factor of the earlier sums
    float2 stats[Src::ROWS];
};

template <typename T>
__device__ __forceinline__ void load4(const T* p, float* y) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = kda::io<T>::ld(p + i);
}

// VEC: channels a load brings (1: rows off their 16-byte boundaries)
template <class Src, typename T, int VEC>
__global__ void __launch_bounds__(Src::THREADS, Src::BLOCKS)
kda_latent_simt_kernel(const T* __restrict__ q, Src src, const int32_t* __restrict__ cu,
                       const int32_t* __restrict__ lengths, long long q_stride, bool q_wide, typename Src::Sh s, float scale_log2,
                       T* __restrict__ o, float* __restrict__ lse, Partials parts) {
    constexpr int DK = Src::DK, DV = Src::DV, ROWS = Src::ROWS, kTileLog2 = Src::LOG2, kTile = 1 << kTileLog2;
    constexpr int kThreads = Src::THREADS;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem<Src>& sm = *reinterpret_cast<Smem<Src>*>(smem_raw);
    __shared__ unsigned long long s_red[kThreads / 32];
    __shared__ Piece s_piece;
    __shared__ Unit s_unit;
    __shared__ int s_more;
    __shared__ long long s_place[2][kTile];            // rows of a tile's keys; -1: none
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    kda_paged::wait_for_stream();

    const Piece piece = kda_paged::find_piece<kThreads>(s, cu, lengths, blockIdx.x, gridDim.x,
                                                        reinterpret_cast<unsigned long long*>(smem_raw), s_red, &s_piece);
    Walker walk;
    if (w == 0) walk.start(s, cu, lengths, piece, blockIdx.x);
    if (tid == 0) parts.clear_both(blockIdx.x);

    constexpr int CG = DV / 4, RPT = ROWS * CG / kThreads;        // column groups; rows of a thread
    static_assert(RPT >= 4 && RPT % 4 == 0, "rows");
    const int cg = tid % CG, r0 = tid / CG * RPT;
    for (;;) {
        __syncthreads();                               // the unit before is done with shared memory
        if (w == 0) {
            Unit nu;
            unsigned long long from;
            const bool more = walk.step(s, cu, lengths, nu, from);
            if (more) walk.share(s, nu, from, 0);
            if (lane == 0) {
                s_unit = nu;
                s_more = more;
            }
        }
        __syncthreads();
        if (!s_more) break;
        const Unit u = s_unit;
        const int rows = u.ntok * s.Gv;
        // queries, in 16-byte pieces where their rows start on such boundaries
        auto load_q = [&](auto vec) {
            constexpr int V = decltype(vec)::value, CH = DK / V, N = (ROWS * CH + kThreads - 1) / kThreads;
            struct alignas(V * sizeof(T)) Chunk { T v[V]; };
            constexpr int B = N < 6 ? N : 6;           // loads in flight
#pragma unroll 1
            for (int e0 = tid; e0 < ROWS * CH; e0 += B * kThreads) {
                Chunk x[B];
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    const int e = e0 + i * kThreads, r = e / CH, c = e % CH * V, tok = (int)((unsigned)r / (unsigned)s.Gv);
                    const int head = u.qh0 + r - tok * s.Gv;
#pragma unroll
                    for (int y = 0; y < V; ++y) kda::io<T>::st(&x[i].v[y], 0.f);
                    if (r < rows && head < s.Hq)       // rows end before ROWS
                        x[i] = *reinterpret_cast<const Chunk*>(q + (u.tok0 + tok) * q_stride + (long long)head * DK + c);
                }
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    const int e = e0 + i * kThreads;
                    if (e >= ROWS * CH) continue;
#pragma unroll
                    for (int y = 0; y < V; ++y) sm.q[e / CH][e % CH * V + y] = kda::io<T>::ld(&x[i].v[y]);
                }
            }
        };
        if (q_wide) load_q(std::integral_constant<int, 16 / sizeof(T)>{});
        else load_q(std::integral_constant<int, 1>{});
        // softmax state: kThreads / ROWS threads share a row
        constexpr int TPR = kThreads / ROWS, KPT = kTile / TPR;
        const int sr = tid / TPR, sx = tid % TPR;
        const int my_pos = u.pos + sr / s.Gv;
        const int my_hi = sr < rows ? min(my_pos + 1, u.kend) : 0;
        float m = -INFINITY, l = 0.f;
        float acc[RPT][4];
#pragma unroll
        for (int a = 0; a < RPT; ++a)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[a][c] = 0.f;

        auto place_of = [&](int t) -> long long {
            const int key = (t << kTileLog2) + tid;
            return key < u.kend ? src.place(s, u, key) : -1;
        };
        // looked up a tile ahead, so that a tile's loads wait for one read, not two
        if (tid < kTile) s_place[u.tb & 1][tid] = place_of(u.tb);
        for (int t = u.tb; t < u.te; ++t) {
            const int key0 = t << kTileLog2;
            __syncthreads();                           // q and the places stored; the tile before is consumed
            const long long* places = s_place[t & 1];
            long long next_place = -1;
            if (tid < kTile && t + 1 < u.te) next_place = place_of(t + 1);
            // places without a key become zero
            struct alignas(VEC * sizeof(T)) Chunk { T v[VEC]; };
            constexpr int KC = DK / VEC, VC = Src::kShared ? 0 : DV / VEC, TOTAL = kTile * (KC + VC);
            constexpr int BATCH = TOTAL / kThreads < 10 ? (TOTAL + kThreads - 1) / kThreads : 10;    // loads in flight
#pragma unroll 1
            for (int e0 = tid; e0 < TOTAL; e0 += kThreads * BATCH) {
                Chunk x[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int e = e0 + i * kThreads, j = e / (KC + VC), c = e % (KC + VC);
#pragma unroll
                    for (int y = 0; y < VEC; ++y) kda::io<T>::st(&x[i].v[y], 0.f);
                    if (e >= TOTAL) continue;
                    const long long at = places[j];
                    if (at >= 0)
                        x[i] = *reinterpret_cast<const Chunk*>(c < KC ? src.key(at, u.kvh, c * VEC)
                                                                      : src.value(at, u.kvh, (c - KC) * VEC));
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    const int e = e0 + i * kThreads, j = e / (KC + VC), c = e % (KC + VC);
                    if (e >= TOTAL) continue;
                    float* dst = c < KC ? &sm.k[j][c * VEC] : &sm.v[Src::kShared ? 0 : j][(c - KC) * VEC];
                    if constexpr (VEC >= 4) {
#pragma unroll
                        for (int y = 0; y < VEC; y += 4) {
                            float z[4];
                            load4(x[i].v + y, z);
                            *reinterpret_cast<float4*>(dst + y) = make_float4(z[0], z[1], z[2], z[3]);
                        }
                    } else {
                        dst[0] = kda::io<T>::ld(x[i].v);
                    }
                }
            }
            if (tid < kTile && t + 1 < u.te) s_place[(t + 1) & 1][tid] = next_place;
            __syncthreads();
            // scores over one part of the channels: rows ty, ty + ROWS / 4, ..., keys tx, tx + KX, ...  (neighbouring
            // threads neighbouring rows of both, so that no two meet in a bank)
            {
                constexpr int SPLIT = Smem<Src>::SPLIT, CP = DK / SPLIT, KX = kTile / 4;
                static_assert(CP % 4 == 0, "channels");
                const int tx = tid % KX, ty = tid / KX % (ROWS / 4), part = tid / (KX * (ROWS / 4));
                float a[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[i][e] = 0.f;
#pragma unroll 3
                for (int c = part * CP; c < (part + 1) * CP; c += 4) {
                    float4 k[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) k[e] = *reinterpret_cast<const float4*>(&sm.k[tx + e * KX][c]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 x = *reinterpret_cast<const float4*>(&sm.q[ty + i * (ROWS / 4)][c]);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            a[i][e] = fmaf(x.x, k[e].x, fmaf(x.y, k[e].y, fmaf(x.z, k[e].z, fmaf(x.w, k[e].w, a[i][e]))));
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sm.part[part][ty + i * (ROWS / 4)][tx + e * KX] = a[i][e];
            }
            __syncthreads();
            // softmax statistics of row sr
            int hidden;                                // some row does not see some key of the tile
            {
                float x[KPT];
                float top = -INFINITY;
                unsigned seen = 0;
#pragma unroll
                for (int i = 0; i < KPT; ++i) {
                    const int j = sx + TPR * i;
                    x[i] = sm.part[0][sr][j];
#pragma unroll
                    for (int e = 1; e < Smem<Src>::SPLIT; ++e) x[i] += sm.part[e][sr][j];
                    if (places[j] >= 0 && key0 + j < my_hi) {
                        seen |= 1u << i;
                        top = fmaxf(top, x[i]);
                    }
                }
#pragma unroll
                for (int d = TPR / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn;
                const float f = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : exp2f((m - ref) * scale_log2);
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < KPT; ++i) {
                    const float p = (seen >> i) & 1 ? exp2f((x[i] - ref) * scale_log2) : sr < rows ? -1.f : 0.f;
                    if ((seen >> i) & 1) sum += p;
                    sm.p[sx + TPR * i][sr] = p;
                }
#pragma unroll
                for (int d = TPR / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                l = fmaf(l, f, sum);
                m = mn;
                if (sx == 0) sm.scale[sr] = f;
                hidden = sr < rows && seen != (1u << KPT) - 1;
            }
            hidden = __syncthreads_or(hidden);
            // weighted sums
#pragma unroll
            for (int a = 0; a < RPT; ++a) {
                const float f = sm.scale[r0 + a];
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[a][c] *= f;
            }
            // A masked key is passed over, not multiplied by zero, so that what stands there stays out.  Tiles that all
            // rows see whole do without the branches (with them everywhere: 4 prompts of 200 tokens over 2000 keys
            // 360 -> 364 us, the absorbed case 20.7 -> 20.9, the expanded one as it is)
            auto weigh = [&](auto masked) {
#pragma unroll 4
                for (int j = 0; j < kTile; ++j) {
                    const float4 v = *reinterpret_cast<const float4*>(Src::kShared ? &sm.k[j][4 * cg]
                                                                                   : &sm.v[Src::kShared ? 0 : j][4 * cg]);
#pragma unroll
                    for (int a0 = 0; a0 < RPT; a0 += 4) {
                        const float4 p4 = *reinterpret_cast<const float4*>(&sm.p[j][r0 + a0]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float p = i == 0 ? p4.x : i == 1 ? p4.y : i == 2 ? p4.z : p4.w;
                            if (!decltype(masked)::value || p != -1.f) {
                                acc[a0 + i][0] = fmaf(p, v.x, acc[a0 + i][0]);
                                acc[a0 + i][1] = fmaf(p, v.y, acc[a0 + i][1]);
                                acc[a0 + i][2] = fmaf(p, v.z, acc[a0 + i][2]);
                                acc[a0 + i][3] = fmaf(p, v.w, acc[a0 + i][3]);
                            }
                        }
                    }
                }
            };
            if (r0 < rows) {
                if (hidden) weigh(std::true_type{});
                else weigh(std::false_type{});
            }
        }
        __syncthreads();
        if (sx == 0) sm.stats[sr] = kda_paged::row_stats(m, l, scale_log2, INFINITY);
        __syncthreads();
        const bool whole = u.first && u.last;
        const int which = u.first ? 1 : 0;
#pragma unroll
        for (int a = 0; a < RPT; ++a) {
            const int r = r0 + a, head = u.qh0 + r % s.Gv;
            if (r >= rows || head >= s.Hq) continue;
            const float rm = sm.stats[r].x;
            float rl = sm.stats[r].y;
            if (whole) {
                rl = kda_paged::whole_sum(rm, rl);
                const float inv = rl == 0.f ? 0.f : 1.f / rl;
                const size_t at = (size_t)(u.tok0 + r / s.Gv) * s.Hq + head;
                T* dst = o + at * DV + 4 * cg;
                if constexpr (sizeof(T) == 2)
                    *reinterpret_cast<uint2*>(dst) = make_uint2(kda::pack_bf16x2(acc[a][0] * inv, acc[a][1] * inv),
                                                                kda::pack_bf16x2(acc[a][2] * inv, acc[a][3] * inv));
                else
                    *reinterpret_cast<float4*>(dst) =
                        make_float4(acc[a][0] * inv, acc[a][1] * inv, acc[a][2] * inv, acc[a][3] * inv);
                if (lse && cg == 0) lse[at] = rl == 0.f ? -INFINITY : (rm + log2f(rl)) * kLn2;
            } else {
                *reinterpret_cast<float4*>(parts.sums4(blockIdx.x, which, r, 4 * cg)) =
                    make_float4(acc[a][0], acc[a][1], acc[a][2], acc[a][3]);
                if (cg == 0) parts.stats(blockIdx.x, which)[r] = make_float2(rm, rl);
            }
        }
        if (tid == 0) parts.describe_both(blockIdx.x, u);
    }
}

template <class Src, typename T, int VEC>
cudaError_t launch(const Src& src, const void* q, int64_t q_stride, const int32_t* cu, const int32_t* lengths,
                   const typename Src::Sh& s, float scale, const kda_host::PagedArgs& pa, const kda_host::PagedPlan& p) {
    auto kern = kda_latent_simt_kernel<Src, T, VEC>;
    const size_t smem = std::max(sizeof(Smem<Src>), (size_t)s.n_req * sizeof(unsigned long long));
    static kda_host::OncePerDevice once;
    const cudaError_t e = once.run([&] {
        constexpr size_t most = std::max(sizeof(Smem<Src>), (size_t)kda_paged::kMaxRequests * 8);
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    });
    if (e != cudaSuccess) return e;
    const bool q_wide = reinterpret_cast<uintptr_t>(q) % 16 == 0 && q_stride * sizeof(T) % 16 == 0;
    const int ctas = std::min(p.max_ctas, Src::BLOCKS * kda_host::sm_count());
    const cudaError_t err = kda_host::launch_overlapped(kern, ctas, Src::THREADS, smem, pa.stream, 1, static_cast<const T*>(q), src,
                                                        cu, lengths, q_stride, q_wide, s, scale * kLog2e, static_cast<T*>(pa.o),
                                                        pa.lse, kda_host::paged_partials(pa, p));
    if (err != cudaSuccess) return err;
    return kda_host::launch_latent_merge(pa, p, ctas);
}

template <typename T>
cudaError_t absorbed(const kda_host::LatentArgs& a) {
    const kda_host::PagedPlan p = kda_host::latent_plan_simt(a.T, a.H);
    const kda_host::PagedArgs pa = kda_host::latent_view(a);
    const Absorbed<T> src{static_cast<const T*>(a.cache), a.block_table};
    return launch<Absorbed<T>, T, 16 / sizeof(T)>(src, a.q, a.q_stride, a.cu_seqlens, a.seq_len,
                                                  kda_host::latent_shape(a, p), a.scale, pa, p);
}

template <typename T>
cudaError_t expanded(const kda_host::ExpandedArgs& a) {
    constexpr int VEC = 16 / sizeof(T);
    const kda_host::PagedPlan p = kda_host::expanded_plan_simt(a.T);
    const kda_host::PagedArgs pa = kda_host::expanded_view(a);
    const Expanded<T> src{static_cast<const T*>(a.k_nope), static_cast<const T*>(a.k_rope), static_cast<const T*>(a.v),
                          a.kn_token, a.kn_head, a.kr_stride, a.v_token, a.v_head, a.cu_seqlens_k};
    auto on = [&](const void* ptr, int64_t s0, int64_t s1) {
        return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && s0 % VEC == 0 && s1 % VEC == 0;
    };
    const bool wide = on(a.k_nope, a.kn_token, a.kn_head) && on(a.k_rope, a.kr_stride, 0) && on(a.v, a.v_token, a.v_head);
    const kda_paged::PackedShape s = kda_host::expanded_shape(a, p);
    return wide ? launch<Expanded<T>, T, VEC>(src, a.q, a.q_stride, a.cu_seqlens, a.cu_seqlens_k, s, a.scale, pa, p)
                : launch<Expanded<T>, T, 1>(src, a.q, a.q_stride, a.cu_seqlens, a.cu_seqlens_k, s, a.scale, pa, p);
}

}  // namespace

namespace kda_host {

// Head groups of at most `most` rows, as even as can be; the last may have fewer heads.
int latent_groups(int H, int most) { return (H + most - 1) / most; }

PagedPlan latent_plan_simt(int T, int H) {
    constexpr int kRows = Absorbed<float>::ROWS;
    PagedPlan p;
    const int groups = latent_groups(H, kRows);
    p.Gv = (H + groups - 1) / groups;
    p.U = kRows / p.Gv;
    p.rows = paged_slot_rows(p.U, T, p.Gv);
    p.tile_log2 = Absorbed<float>::LOG2;
    p.max_ctas = 304;
    p.extra = 0;
    return p;
}

PagedPlan expanded_plan_simt(int T) {
    PagedPlan p;
    p.Gv = 1;
    p.U = Expanded<float>::ROWS;
    p.rows = paged_slot_rows(p.U, T, 1);
    p.tile_log2 = Expanded<float>::LOG2;
    p.max_ctas = 304;
    p.extra = 0;
    return p;
}

PagedArgs latent_view(const LatentArgs& a) {
    PagedArgs p{};
    p.N = a.N;
    p.T = a.T;
    p.Hq = a.H;
    p.Hkv = 1;
    p.d = kLatent;
    p.page_size = a.page_size;
    p.blocks = a.blocks;
    p.n_pages = a.n_pages;
    p.dtype = a.dtype;
    p.o = a.o;
    p.lse = a.lse;
    p.workspace = a.workspace;
    p.stream = a.stream;
    return p;
}

kda_paged::Shape latent_shape(const LatentArgs& a, const PagedPlan& p) {
    kda_paged::Shape s = paged_shape(latent_view(a), p);
    s.Hv = s.sub = (a.H + p.Gv - 1) / p.Gv;            // the last group may have fewer heads
    return s;
}

PagedArgs expanded_view(const ExpandedArgs& a) {
    PagedArgs p{};
    p.N = a.N;
    p.T = a.T;
    p.Hq = p.Hkv = a.H;
    p.d = kValue;
    p.page_size = 1;
    p.dtype = a.dtype;
    p.o = a.o;
    p.lse = a.lse;
    p.workspace = a.workspace;
    p.stream = a.stream;
    return p;
}

kda_paged::PackedShape expanded_shape(const ExpandedArgs& a, const PagedPlan& p) {
    kda_paged::PackedShape s;
    static_cast<kda_paged::Shape&>(s) = paged_shape(expanded_view(a), p);
    s.S = a.S;
    s.causal = a.causal;
    // In a call of at most half_unit tokens no unit has two steps a tile, and its pieces may have one place: a prompt
    // of 20 tokens over 3000 keys 12.9 -> 11.9 us, 2 of 100 over 1000 12.4 -> 11.9, 200 over 200 with 16 heads 13.5 -> 13.7.
    s.half_unit = p.half_unit > 0 && a.T > p.half_unit ? p.half_unit : p.U;
    s.extra_two = p.extra_two;
    return s;
}

cudaError_t launch_latent_attention_simt(const LatentArgs& a) {
    return a.dtype == KDA_BF16 ? absorbed<__nv_bfloat16>(a) : absorbed<float>(a);
}

cudaError_t launch_expanded_attention_simt(const ExpandedArgs& a) {
    return a.dtype == KDA_BF16 ? expanded<__nv_bfloat16>(a) : expanded<float>(a);
}

}  // namespace kda_host
