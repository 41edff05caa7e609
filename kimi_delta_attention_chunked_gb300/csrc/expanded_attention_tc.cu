// expanded_attention_tc.cu -- expanded latent attention over packed keys and values on the
// tensor cores (bf16), by pairs of CTAs.
//
// A unit (paged.cuh) is up to 512 new tokens of one request and head: two row tiles of 2 x 128
// rows, of which CTA r of a cluster of two has rows 128 r .. 128 r + 127.  Per tile of 128 keys,
// with cta_group::2 products of M = 256:
//     S = Q K^T     (256 x 128 over 192 channels: 128 of k_nope, 64 of k_rope; S in TMEM)
//     P = 2^(scale log2(e) S - m)   (registers; written back over S as bf16)
//     O += P V      (256 x 128 over 128 keys; P from TMEM, O in TMEM)
// m is a reference per row that moves, with O and the sum of weights, only when a score exceeds
// it by more than 8 octaves.
//
// Why a pair: each CTA brings half of B, 64 keys of 192 channels and 64 value channels of 128
// keys, 40 KB of a tile instead of 80.  Three tiles fit beside the queries (96 KB), which one CTA
// alone could not do with two, and a product reads 3/4 of the bytes from shared memory that
// it takes the tensor cores to multiply, where one of a CTA alone reads as many and waits for them.
//
// Work goes in steps of one row tile and one key tile; step g uses half g & 1 of TMEM (S, O) and
// of the softmax warps, so that the tensor cores run one half's products while the other half's
// weights are formed.  A unit with two row tiles takes its key tiles in two steps each; one with
// one (up to 256 tokens) sends its key tiles to the two halves in turn, which hold the sums over the
// even and the odd ones and are joined at the end.
//
// Warps of each CTA: 0-3 and 4-7 softmax and output of half 0 and 1; 8 copies; 9 issues the
// products (in CTA 0, for both); 10 walks the units; 11 cleans masked values.  Barriers of loads and of P are CTA 0's.
//
// Masked places.  A zero weight times a NaN or infinity in V is NaN.  So in a tile that not every row
// of the unit sees whole, a warp of each CTA zeroes the rows of V that no row sees (the next
// request's), and in the rows that some see and some do not takes out the elements that are not
// finite; the output adds such elements to the rows that see them.
//
// Bound, and what it measured (GPU time with the merge; cuBLAS 1888 TFLOP/s).  A prompt of 8192 tokens,
// 32 heads: 418 to 427 us, 1.61 to 1.64 PFLOP/s of the products that a causal mask leaves (floor 364): a tile of two steps
// takes 2970 cycles, 2560 of them products, and a unit's end (its last two tiles have one row tile, its
// output) 10 k cycles of 60 k to 190 k.  A chunk of 4096 tokens behind 24576 others, 16 heads: 588 us, 1.90 PFLOP/s
// (floor 592: long units, few ends).  12 requests of 1 to 700 tokens over up to 3200 keys, 16 heads: 43 to 47 us
// (floor 10.6): 2 to 6 short units a pair at 7 to 8 k cycles each; 16 prompts of 16 to 300 tokens, 16 heads: 36 us (4.5).
// What it took: arrivals at the other CTA without a fence of global memory (684 -> 528 us); the weights in two
// halves, so that the first half's products run while the second is formed, and no steps of a row tile
// behind its last key (518 -> 440); places of the division that count steps (444 -> 427); values cleaned off
// the softmax warps' path, one short output loop (431 -> 418).  Queries of lone row tiles fetched a unit
// ahead gained nothing.
// Rounding: P enters its product as bf16, the type of V; the output's error against 64 bits is 2.0e-3
// (2-norm), 1.5e-3 of it its own rounding to bf16.
#include <algorithm>

#include "attention_pair.cuh"
#include "latent.cuh"

namespace {

using namespace kda_tc;
using kda_latent::kKey;
using kda_latent::kNope;
using kda_latent::kValue;
using kda_paged::PackedShape;
using kda_paged::Partials;
using kda_paged::Piece;
using kda_paged::Walker;

constexpr int kThreads = 384;
constexpr int kCopyWarp = 8, kIssueWarp = 9, kWalkWarp = 10, kCleanWarp = 11;
constexpr int kKeys = 128, kKeysLog2 = 7;              // keys of a tile
constexpr int kRows = 128;                             // rows of a CTA's part of a row tile
constexpr int kTileTokens = 2 * kRows;                 // tokens of a row tile
constexpr int kPanels = kKey / 64;
constexpr int kQPanel = kRows * 128;                   // bytes of 128 rows x 64 channels
constexpr int kQTile = kPanels * kQPanel;
constexpr int kKPanel = kKeys / 2 * 128;               // of 64 keys x 64 channels
constexpr int kKTile = kPanels * kKPanel;
constexpr int kVTile = kKeys * 128;                    // of 128 keys x 64 channels
constexpr int kStages = 3;
constexpr int kK0 = 2 * kQTile, kV0 = kK0 + kStages * kKTile, kTail0 = kV0 + kStages * kVTile;
constexpr int kUnits = 4;                              // unit descriptions in flight
constexpr int kTailBytes = 4 * 1024;
constexpr int kSmem = kTail0 + kTailBytes;
constexpr uint32_t kTmemO = 256;                       // columns: S halves at 0 and 128, O halves from 256
static_assert(kSmem <= 227 * 1024, "shared memory");
static_assert(kStages * kKTile >= kda_paged::kMaxRequests * 8 + 512, "scratch of find_piece");

struct UnitSlot {
    Unit u;
    int more;                                          // 0: no further unit
};

struct Tail {
    uint64_t k_full[kStages], v_full[kStages], v_ready[kStages], q_full;             // CTA 0's are used
    uint64_t p_full[2][2];                             // too; P in halves of its keys
    uint64_t k_empty[kStages], v_empty[kStages], q_empty, s_full[2], o_full[2], landed[kStages];    // each CTA's own
    uint64_t join_a, join_b;
    uint64_t u_full[kUnits], u_empty[kUnits];
    uint64_t drain;
    uint32_t tmem;
    int abort;
    int odd_values[8];                                 // per unit, in turn: values that are not finite were taken out
    UnitSlot units[kUnits];
    float2 stats[2][kRows];                            // (reference in octaves, sum of weights) of each half's rows
};
static_assert(sizeof(Tail) <= kTailBytes, "tail");

// Key tiles of this part that row tile 0 of a unit of two takes: the rest hold no key that it sees.  One at
// least, so that both halves have a step in every part.
__device__ __forceinline__ int first_tiles(const Unit& u) {
    const int hi = min(max(u.pos + kTileTokens, 0), u.kend);
    return min(u.te - u.tb, max(((hi + kKeys - 1) >> kKeysLog2) - u.tb, 1));
}

// Where the values lie in global memory.
struct Values {
    const __nv_bfloat16* v;
    long long token, head;
};

// Adds to a row's output or partial sums, channels from .. to - 1, the values that are not finite, of the keys
// [first, last) among those that not all rows of the unit see: rare, and so out of the way of what every unit
// fetches.
__device__ __noinline__ void add_odd_values(__nv_bfloat16* o, float* sums, int cap, int from, int to, const __nv_bfloat16* v,
                                            long long token, int first, int last) {
    for (int key = first; key < last; ++key)
        for (int c = from; c < to; ++c) {
            const float x = __bfloat162float(v[key * token + c]);
            if ((__float_as_uint(x) & 0x7f800000u) != 0x7f800000u) continue;
            if (o) o[c] = __float2bfloat16_rn(__bfloat162float(o[c]) + x);
            else sums[(size_t)(c >> 2) * cap * 4 + (c & 3)] += x;
        }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
kda_expanded_attention_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap nmap,
                                 const __grid_constant__ CUtensorMap rmap, const __grid_constant__ CUtensorMap vmap,
                                 Values values, const int32_t* __restrict__ cu, const int32_t* __restrict__ cu_k,
                                 PackedShape s, float scale_log2, __nv_bfloat16* __restrict__ o, float* __restrict__ lse,
                                 Partials parts, int* status) {
    extern __shared__ __align__(1024) unsigned char sm[];
    Tail& tl = *reinterpret_cast<Tail*>(sm + kTail0);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank(), cluster = blockIdx.x >> 1;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the merge may be set up; it waits for this grid
    if (w == kIssueWarp) alloc_pair(&tl.tmem);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            kda::mbar_init(&tl.k_full[i], 1);
            kda::mbar_init(&tl.v_full[i], 1);
            kda::mbar_init(&tl.k_empty[i], 1);
            kda::mbar_init(&tl.v_empty[i], 1);
            kda::mbar_init(&tl.landed[i], 1);
            kda::mbar_init(&tl.v_ready[i], 2);
        }
        kda::mbar_init(&tl.q_full, 1);
        kda::mbar_init(&tl.q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            kda::mbar_init(&tl.s_full[i], 1);
            kda::mbar_init(&tl.p_full[i][0], 8);
            kda::mbar_init(&tl.p_full[i][1], 8);
            kda::mbar_init(&tl.o_full[i], 1);
        }
        kda::mbar_init(&tl.join_a, 8);
        kda::mbar_init(&tl.join_b, 8);
        for (int i = 0; i < kUnits; ++i) {
            kda::mbar_init(&tl.u_full[i], 1);
            kda::mbar_init(&tl.u_empty[i], rank == 0 ? 11 : 10);
        }
        kda::mbar_init(&tl.drain, 1);
        kda::fence_barrier_init();
        tl.abort = 0;
        for (int i = 0; i < 8; ++i) tl.odd_values[i] = 0;
    }
    if (w == kCopyWarp && lane < 4) {
        const CUtensorMap* m = lane == 0 ? &qmap : lane == 1 ? &nmap : lane == 2 ? &rmap : &vmap;
        asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    cluster_arrive();                                  // both CTAs' barriers will be there
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the kernels before this one are complete
    // this pair's piece of the work; both CTAs find the same.  Few requests: the walking warp does, below
    auto* cost = reinterpret_cast<unsigned long long*>(sm + kK0);
    Piece piece{};
    if (s.n_req > kda_paged::kWarpRequests) {
        auto* red = cost + kda_paged::kMaxRequests;
        piece = kda_paged::find_piece<kThreads>(s, cu, cu_k, cluster, gridDim.x >> 1, cost, red,
                                                reinterpret_cast<Piece*>(red + kThreads / 32));
        kda::fence_proxy_async_smem();                 // the scratch becomes the target of copies
    }
    kda::tc_fence_before();
    __syncthreads();
    cluster_wait();
    kda::tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)tl.tmem);
    volatile int* abort_f = &tl.abort;
    // true once the phase is complete; false when this CTA gives up.  Called by all
    // lanes of a warp, with one answer for all of them, so that none leaves a loop alone
    auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
        if (__all_sync(0xffffffffu, kda::mbar_try_wait(b, parity))) return true;
        return wait_longer(b, parity, &tl.abort, status);
    };
    auto read_unit = [&](int k, Unit& u) -> bool {
        if (!wait(&tl.u_full[k % kUnits], (k / kUnits) & 1)) return false;
        const UnitSlot& sl = tl.units[k % kUnits];
        u = sl.u;
        const bool more = sl.more != 0;
        __syncwarp();
        if (lane == 0) kda::mbar_arrive(&tl.u_empty[k % kUnits]);
        return more;
    };
    auto first_row = [&](const Unit& u) { return min(max(cu_k[u.n], 0), s.S); };      // of the request's keys
    int n_ld = 0, n_q = 0;                             // tiles and queries whose copies were issued

    if (w == kWalkWarp) {
        // ---------------- unit descriptions
        if (lane == 0 && rank == 0) parts.clear_both(cluster);
        if (s.n_req <= kda_paged::kWarpRequests) {
            piece = kda_paged::find_piece_warp(s, cu, cu_k, cluster, gridDim.x >> 1, cost);
            kda::fence_proxy_async_smem();
        }
        Walker walk;
        walk.start(s, cu, cu_k, piece, cluster);
        for (int k = 0;; ++k) {
            Unit u;
            unsigned long long from;
            const bool more = walk.step(s, cu, cu_k, u, from);
            if (k >= kUnits && !wait(&tl.u_empty[k % kUnits], (k / kUnits - 1) & 1)) break;
            __syncwarp();
            if (lane == 0) {
                if (more) tl.units[k % kUnits].u = u;
                tl.units[k % kUnits].more = more;
                kda::mbar_arrive(&tl.u_full[k % kUnits]);
            }
            if (!more) break;
            walk.share(s, u, from, 0);
            if (lane == 0 && rank == 0) parts.describe_both(cluster, u);
        }
    } else if (w == kCopyWarp) {
        // ---------------- copies: of each tile this CTA's keys, then its channels of the values
        bool ok = true;
        for (int k = 0; ok; ++k) {
            Unit u;
            if (!read_unit(k, u)) break;
            const int key0 = first_row(u);
            for (int tile = u.tb; tile < u.te; ++tile) {
                const int st = n_ld % kStages, at = key0 + (tile << kKeysLog2);
                const uint32_t parity = (n_ld / kStages - 1) & 1;
                if (n_ld >= kStages && !wait(&tl.k_empty[st], parity)) { ok = false; break; }
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) kda::mbar_arrive_expect_tx(&tl.k_full[st], 2 * kKTile);
                    const uint32_t dst = kda::smem_u32(sm + kK0 + st * kKTile), bar = at_rank(&tl.k_full[st], 0);
                    const int y = at + rank * (kKeys / 2);
                    load_pair(dst, &nmap, 0, u.kvh, y, bar);
                    load_pair(dst + kKPanel, &nmap, 64, u.kvh, y, bar);
                    load_pair(dst + 2 * kKPanel, &rmap, 0, 0, y, bar);
                }
                __syncwarp();
                if (tile == u.tb) {
                    const int tiles = u.ntok > kTileTokens ? 2 : 1;
                    if (k > 0 && !wait(&tl.q_empty, (k - 1) & 1)) { ok = false; break; }
                    __syncwarp();
                    if (lane == 0 && rank == 0) kda::mbar_arrive_expect_tx(&tl.q_full, 2 * tiles * kQTile);
                    __syncwarp();
                    if (lane < tiles * kPanels) {
                        const int i = lane / kPanels, c = lane % kPanels;
                        load_pair(kda::smem_u32(sm) + i * kQTile + c * kQPanel, &qmap, c * 64, u.qh0,
                                  u.tok0 + i * kTileTokens + rank * kRows, at_rank(&tl.q_full, 0));
                    }
                    ++n_q;
                }
                if (n_ld >= kStages && !wait(&tl.v_empty[st], parity)) { ok = false; break; }
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) kda::mbar_arrive_expect_tx(&tl.v_full[st], 2 * kVTile);
                    load_pair(kda::smem_u32(sm + kV0 + st * kVTile), &vmap, rank * 64, u.kvh, at, at_rank(&tl.v_full[st], 0));
                }
                __syncwarp();
                ++n_ld;
            }
        }
    } else if (w == kCleanWarp) {
        // ---------------- values that must not meet a zero weight (see the header).  CTA 1's loads count on CTA 0's
        // barriers, so it is told of them; the products wait for both CTAs
        int n_v = 0;                                   // key tiles so far
        bool ok = true;
        for (int k = 0; ok; ++k) {
            Unit u;
            if (!read_unit(k, u)) break;
            const Sight un = sight(u, 0, 0, u.ntok - 1);
            for (int tile = u.tb; tile < u.te; ++tile, ++n_v) {
                const int st = n_v % kStages, k0 = tile << kKeysLog2;
                ok = wait(rank == 0 ? &tl.v_full[st] : &tl.landed[st], (n_v / kStages) & 1);
                if (!ok) break;
                if (rank == 0 && lane == 0) arrive_remote(at_rank(&tl.landed[st], 1));
                if (k0 + kKeys > un.all_hi) {          // not every row sees it whole
                    unsigned char* v = sm + kV0 + st * kVTile;
                    const int from = max(un.all_hi - k0, 0), to = min(max(un.hi - k0, 0), kKeys);
                    bool odd = false;
#pragma unroll 4
                    for (int e = from * 8 + lane; e < to * 8; e += 32) {     // some rows see them
                        uint4* at = reinterpret_cast<uint4*>(v + e * 16);
                        uint4 x = *at;
                        if (take_odd(x)) {
                            *at = x;
                            odd = true;
                        }
                    }
                    for (int e = max(from, to) * 8 + lane; e < kKeys * 8; e += 32)            // no row sees them
                        *reinterpret_cast<uint4*>(v + e * 16) = make_uint4(0, 0, 0, 0);
                    if (odd) flag_pair(&tl.odd_values[k & 7]);
                    kda::fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) arrive_remote(at_rank(&tl.v_ready[st], 0));
            }
        }
    } else if (w == kIssueWarp) {
        // ---------------- products: CTA 0 issues for both.  All lanes wait, an elected one issues.
        // P_h lies over S_h: the scores of a half's next step are issued behind its product P_h V, which
        // waited for P_h, and the tensor cores take products in the order of issue
        const uint32_t id_s = kda::idesc_bf16(256, kKeys, 0, 0), id_o = kda::idesc_bf16(256, kValue, 0, 1);
        const uint64_t q_desc = kda::sw128_desc(kda::smem_u32(sm), 16, 1024);
        const uint64_t k_desc = kda::sw128_desc(kda::smem_u32(sm + kK0), 16, 1024);
        const uint64_t v_desc = kda::sw128_desc(kda::smem_u32(sm + kV0), kVTile, 1024);
        int g = 0, n_k = 0;                            // steps; key tiles taken
        uint32_t p_phase = 0;                          // bit h: parity of the next P_h
        bool issued = false, ok = rank == 0;
        // a step whose second product is due: flags, its tile's place in the ring
        enum { kFirstUse = 1, kLastUse = 2, kAdd = 4, kFinal = 8, kDue = 16 };
        struct Pending { int flags, at; };
        Pending older{0, 0}, newer{0, 0};              // of steps g - 2 and g - 1
        auto issue_scores = [&](int h, int tile, int at, int flags) {     // S_h = Q_tile K^T; one lane
            const uint64_t a = q_desc + kda::desc_step(tile * kQTile), b = k_desc + kda::desc_step(at % kStages * kKTile);
#pragma unroll
            for (int i = 0; i < kKey / 16; ++i)
                mma_pair(tmem + h * 128, a + kda::desc_step((i >> 2) * kQPanel + (i & 3) * 32),
                         b + kda::desc_step((i >> 2) * kKPanel + (i & 3) * 32), id_s, i > 0 ? 1u : 0u);
            commit_pair(&tl.s_full[h]);
            if (flags & kLastUse) commit_pair(&tl.k_empty[at % kStages]);
            if (flags & kFinal) commit_pair(&tl.q_empty);
        };
        // O_h += P_h V, the first half of the keys as soon as its weights are there
        auto values_step = [&](int h, const Pending& pv) -> bool {
            if ((pv.flags & kFirstUse) && !wait(&tl.v_ready[pv.at % kStages], (pv.at / kStages) & 1)) return false;
            const uint64_t b = v_desc + kda::desc_step(pv.at % kStages * kVTile);
            const uint32_t d = tmem + kTmemO + h * 128, a = tmem + h * 128;
            if (!wait(&tl.p_full[h][0], (p_phase >> h) & 1)) return false;
            kda::tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < kKeys / 32; ++i)
                    mma_pair_ta(d, a + 8 * i, b + kda::desc_step(i * 2048), id_o, (i > 0 || (pv.flags & kAdd)) ? 1u : 0u);
            }
            if (!wait(&tl.p_full[h][1], (p_phase >> h) & 1)) return false;
            p_phase ^= 1u << h;
            kda::tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int i = kKeys / 32; i < kKeys / 16; ++i) mma_pair_ta(d, a + 8 * i, b + kda::desc_step(i * 2048), id_o, 1u);
                if (pv.flags & kLastUse) commit_pair(&tl.v_empty[pv.at % kStages]);
                if (pv.flags & kFinal) commit_pair(&tl.o_full[h]);
            }
            __syncwarp();
            return true;
        };
        auto take_keys = [&](int at) -> bool {
            if (!wait(&tl.k_full[at % kStages], (at / kStages) & 1)) return false;
            kda::tc_fence_after();
            return true;
        };
        for (int k = 0; ok; ++k) {
            Unit u;
            if (!read_unit(k, u)) break;
            const int two = uniform(u.ntok > kTileTokens), tiles = uniform(u.te - u.tb), steps = tiles << two;
            const int tiles0 = two ? uniform(first_tiles(u)) : tiles;
            auto due = [&](int t, int at) {            // the second product of step t
                Pending pv;
                pv.at = at;
                const int j = t >> two;
                pv.flags = kDue | (!two || !(t & 1) || j >= tiles0 ? kFirstUse : 0) | (!two || (t & 1) ? kLastUse : 0) |
                           (t >= 2 ? kAdd : 0) | (t >= steps - 2 || (two && !(t & 1) && j == tiles0 - 1) ? kFinal : 0);
                return pv;
            };
            // a unit of two row tiles past its first key tile goes through the loop below this one
            const int slow = two ? 2 : steps;
            for (int t = 0; t < slow; ++t, ++g) {
                const int h = g & 1, first = !two || t == 0;
                if (older.flags & kDue) ok = values_step(h, older);
                if (ok && first) ok = take_keys(n_k);
                if (ok && t == 0) ok = wait(&tl.q_full, k & 1);
                if (!ok) break;
                kda::tc_fence_after();
                if (elect_one())
                    issue_scores(h, two & t, n_k, (!two || t == 1 ? kLastUse : 0) | (t == steps - 1 ? kFinal : 0));
                __syncwarp();
                issued = true;
                older = newer;
                newer = due(t, n_k);
                if (!two || t == 1) ++n_k;
            }
            if (!ok || slow == steps) continue;
            // the tensor cores' time is here: as few instructions between products as can be
            const int h0 = g & 1, h1 = h0 ^ 1;
            for (int j = 1; j < tiles; ++j, ++n_k) {
                Pending pv{kDue | kFirstUse | (j > 1 ? kAdd : 0) | (j == tiles0 ? kFinal : 0), n_k - 1};
                if (j <= tiles0) ok = values_step(h0, pv);
                ok = ok && take_keys(n_k);
                if (!ok) break;
                if (j < tiles0 && elect_one()) issue_scores(h0, 0, n_k, 0);
                pv.flags = kDue | kLastUse | (j > 1 ? kAdd : 0) | (j > tiles0 ? kFirstUse : 0);
                ok = values_step(h1, pv);
                if (!ok) break;
                if (elect_one()) issue_scores(h1, 1, n_k, kLastUse | (j == tiles - 1 ? kFinal : 0));
            }
            __syncwarp();
            g += steps - 2;
            older = due(steps - 2, n_k - 1);
            if (tiles0 < tiles) older.flags = 0;
            newer = due(steps - 1, n_k - 1);
        }
        if (ok && (older.flags & kDue)) ok = values_step(g & 1, older);
        if (ok && (newer.flags & kDue)) ok = values_step((g + 1) & 1, newer);
        if (issued) {                                  // no product in flight when TMEM is freed
            if (elect_one()) commit_pair(&tl.drain, 1);
            __syncwarp();
            (void)kda::mbar_wait(&tl.drain, 0, kda::kWaitCycles);
        }
    } else if (w < 8) {
        // ---------------- softmax and output of half h
        const int h = w >> 2, row = tid & 127;
        const uint32_t lane_off = (uint32_t)((w & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + h * 128;
        const uint32_t p_bar = at_rank(&tl.p_full[h][0], 0);
        int n_s = 0, n_j = 0, g = 0;
        uint32_t o_phase = 0;                          // bit h: parity of the next O_h
        bool ok = true;
        for (int k = 0; ok; ++k) {
            Unit u;
            if (!read_unit(k, u)) break;
            // the flag of the unit after the next three.  Nobody sets it yet: its values come into the ring when those of
            // the next unit are done with, which takes this warp's part in this one; and nobody reads it any more for
            // the unit four back
            if (tid == 0) tl.odd_values[(k + 4) & 7] = 0;
            const bool two = u.ntok > kTileTokens;
            const int tiles = u.te - u.tb, steps = tiles << (two ? 1 : 0);
            const int t0 = (h ^ g) & 1;                // this half's first step
            const int qi = two ? t0 : 0;               // its row tile
            const int first = qi * kTileTokens + rank * kRows, tok = first + row;
            const bool valid = tok < u.ntok;
            const int pos = u.pos + tok;
            const int hi = valid ? min(max(pos + 1, 0), u.kend) : 0;
            const bool busy = __any_sync(0xffffffffu, valid);
            const Sight un = sight(u, 0, 0, u.ntok - 1);
            const int mine = min(max(u.pos + first + 1, 0), u.kend);      // keys that all of this CTA's rows see,
            const int none = min(max(u.pos + first + kRows, 0), u.kend);  // and that none of them sees from here on
            const int tiles0 = two ? first_tiles(u) : tiles, last = two && qi == 0 ? 2 * tiles0 : steps;
            float m = -INFINITY, l = 0.f;
            for (int t = t0; t < last; t += 2) {
                const int j = two ? t >> 1 : t, k0 = (u.tb + j) << kKeysLog2;
                if (!wait(&tl.s_full[h], n_s & 1)) { ok = false; break; }
                ++n_s;
                kda::tc_fence_after();
                auto arrive = [&](int part) {          // weights of that half of the keys are there
                    kda::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_remote(p_bar + part * 8);
                };
                if (!busy || k0 >= none) {             // no row here sees any key of the tile
                    if (busy) {
                        const uint32_t zero[32] = {};
                        tmem_st32(tS, zero);
                        tmem_st32(tS + 32, zero);
                        kda::tmem_wait_st();
                    }
                    arrive(0);
                    arrive(1);
                    continue;
                }
                float x[128];
#pragma unroll
                for (int c = 0; c < 128; c += 32) kda::tmem_ld32(tS + c, x + c);
                kda::tmem_wait_ld();
                if (k0 + kKeys > mine) {               // keys that this row does not see
                    const int b = hi - k0;
#pragma unroll
                    for (int c = 0; c < 128; ++c) x[c] = c < b ? x[c] : -INFINITY;
                }
                float top[4] = {x[0], x[2], x[4], x[6]};
#pragma unroll
                for (int c = 0; c < 128; c += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top[e] = fmaxf(top[e], fmaxf(x[c + 2 * e], x[c + 2 * e + 1]));
                const float big = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                if (t < 2) {
                    m = big;
                } else {
                    // S complete means that this half's product before it is too, so O stands still
                    const bool grow = valid && (big - m) * scale_log2 > kGrow;
                    if (__any_sync(0xffffffffu, grow)) {
                        const float f = grow ? ex2((m - big) * scale_log2) : 1.f;
                        const uint32_t tO = tmem + lane_off + kTmemO + h * 128;
#pragma unroll 1
                        for (int c = 0; c < kValue; c += 16) {
                            float y[16];
                            kda::tmem_ld16(tO + c, y);
                            kda::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) y[e] *= f;
                            kda::tmem_st16(tO + c, y);
                        }
                        l *= f;
                        if (grow) m = big;
                    }
                }
                const float ref = kda_paged::reference(m, scale_log2);
                const uint64_t sc2 = pack2(scale_log2, scale_log2), off2 = pack2(-ref, -ref);
                uint64_t sum[2] = {0, 0};
                uint32_t p[32];
                auto weigh = [&](int from, int to) {   // weights of keys [from, to), as pairs in p
#pragma unroll
                    for (int c = from; c < to; c += 2) {
                        float a, b;
                        unpack2(fma2(pack2(x[c], x[c + 1]), sc2, off2), a, b);
                        a = ex2(a);
                        b = ex2(b);
                        sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pack2(a, b));
                        p[(c >> 1) & 31] = kda::pack_bf16x2(a, b);
                    }
                };
                weigh(0, 64);
                tmem_st32(tS, p);
                weigh(64, 96);                         // while the first half is being stored
                kda::tmem_wait_st();
                arrive(0);
                weigh(96, 128);
                tmem_st32(tS + 32, p);
                float sa, sb;
                unpack2(add2(sum[0], sum[1]), sa, sb);
                l += sa + sb;
                kda::tmem_wait_st();
                arrive(1);
            }
            if (!ok) break;
            // ---- output: one short loop for every kind of unit, since it is fetched anew each time
            const float2 mine_st = kda_paged::row_stats(m, l, scale_log2);
            const float ref = mine_st.x;
            l = mine_st.y;
            const size_t at = (size_t)(u.tok0 + tok) * s.Hq + u.qh0;
            const bool whole = u.first && u.last;
            const int which = u.first ? 1 : 0;
            // sources in TMEM and their factors, columns of this thread, statistics of the row
            uint32_t src0 = kTmemO + h * 128, src1 = src0;
            float f0 = 1.f, f1 = 0.f, top = ref, sum_l = l;
            bool use0 = true, use1 = false;            // sums that a product wrote; the others hold anything
            int from = 0, to = kValue;
            if (two) {
                ok = wait(&tl.o_full[h], (o_phase >> h) & 1);
                o_phase ^= 3;
                if (!ok) break;
            } else {
                // the halves hold the sums over every second key tile: each joins half of the columns
                const bool has[2] = {(g & 1) == 0 || steps > 1, (g & 1) == 1 || steps > 1};
                tl.stats[h][row] = make_float2(ref, l);
                __syncwarp();
                if (lane == 0) kda::mbar_arrive(&tl.join_a);
                ok = wait(&tl.join_a, n_j & 1);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (!has[e]) continue;
                    ok = ok && wait(&tl.o_full[e], (o_phase >> e) & 1);
                    o_phase ^= 1u << e;
                }
                if (!ok) break;
                const float2 st = tl.stats[h ^ 1][row];
                top = fmaxf(ref, st.x);
                const float base = top == -INFINITY ? 0.f : top;
                use0 = steps > 1 || (g & 1) == h;
                use1 = steps > 1 || (g & 1) != h;
                f0 = l == 0.f ? 0.f : ex2(ref - base);
                f1 = st.y == 0.f ? 0.f : ex2(st.x - base);
                sum_l = fmaf(f0, l, f1 * st.y);
                src1 = kTmemO + (h ^ 1) * 128;
                from = h * (kValue / 2);
                to = from + kValue / 2;
            }
            kda::tc_fence_after();
            if (busy) {
                if (whole) sum_l = kda_paged::whole_sum(top, sum_l);
                const float inv = !whole ? 1.f : sum_l == 0.f ? 0.f : 1.f / sum_l;
                f0 *= inv;
                f1 *= inv;
                __nv_bfloat16* const dst = o + at * kValue;
                float4* const part = reinterpret_cast<float4*>(parts.sums4(cluster, which, valid ? tok : 0, 0));
#pragma unroll 1
                for (int c = from; c < to; c += 16) {
                    float y[16], z[16];
                    kda::tmem_ld16(tmem + lane_off + src0 + c, y);
                    kda::tmem_ld16(tmem + lane_off + src1 + c, z);
                    kda::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e)       // a weight of 0 does not hide a sum that is not finite
                        y[e] = (use0 ? f0 * y[e] : 0.f) + (use1 ? f1 * z[e] : 0.f);
                    if (!valid) continue;
                    if (whole) {
                        store16(dst + c, y);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            part[(c / 4 + e) * parts.cap] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                    }
                }
                if (valid && (two || h == 0)) {
                    if (!whole) parts.stats(cluster, which)[tok] = make_float2(top, sum_l);
                    else if (lse) lse[at] = sum_l == 0.f ? -INFINITY : (top + log2f(sum_l)) * kLn2;
                }
                if (valid && *(volatile int*)&tl.odd_values[k & 7]) {
                    const int key0 = first_row(u);
                    add_odd_values(whole ? dst : nullptr, reinterpret_cast<float*>(part), parts.cap, from, to,
                                   values.v + key0 * values.token + u.kvh * values.head, values.token,
                                   max(un.all_hi, u.tb << kKeysLog2), min(min(un.hi, hi), u.te << kKeysLog2));
                }
            }
            if (!two) {
                kda::tc_fence_before();
                __syncwarp();
                if (lane == 0) kda::mbar_arrive(&tl.join_b);
                ok = wait(&tl.join_b, n_j & 1);
                ++n_j;
                if (!ok) break;
            }
            g += steps;
        }
    }
    kda::tc_fence_before();
    __syncthreads();
    if (*abort_f && rank == 0 && w == kCopyWarp) {     // no copy in flight into shared memory that is given up
        for (int i = max(0, n_ld - kStages); i <= n_ld; ++i) {
            (void)kda::mbar_wait(&tl.k_full[i % kStages], (i / kStages) & 1, i < n_ld ? kda::kWaitCycles : 10000000);
            (void)kda::mbar_wait(&tl.v_full[i % kStages], (i / kStages) & 1, i < n_ld ? kda::kWaitCycles : 10000000);
        }
        if (n_q > 0) (void)kda::mbar_wait(&tl.q_full, (n_q - 1) & 1, kda::kWaitCycles);
    }
    __syncthreads();
    cluster_leave();                                   // the other CTA is done with this one's memory and TMEM
    if (w == kIssueWarp) dealloc_pair(tmem);
}

// ---- host
bool make_map(CUtensorMap* m, const void* base, int channels, cuuint64_t d1, cuuint64_t d2, cuuint64_t stride1,
              cuuint64_t stride2, int box2) {
    const cuuint64_t dims[3] = {(cuuint64_t)channels, d1, d2};
    const cuuint64_t strides[2] = {stride1, stride2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)box2};
    const cuuint32_t one[3] = {1, 1, 1};
    return kda_host::tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
                                          one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

namespace kda_host {

PagedPlan expanded_plan_tc(int T) {
    PagedPlan p;
    p.Gv = 1;
    p.U = 2 * kTileTokens;
    p.rows = paged_slot_rows(p.U, T, 1);
    p.tile_log2 = kKeysLog2;
    p.max_ctas = 80;                                   // pairs
    p.half_unit = kTileTokens;
    // places for the fixed cost of a unit of one row tile and of two; with 0 and 0, 2 and 6, 5 and 5, 5 and 12, 8 and 18: a
    // prompt of 8192 tokens 445, 429, 431, 423 and 434 us, 12 requests of 1 to 700 tokens 88, 54, 45, 47 and 47
    p.extra = 5;
    p.extra_two = 12;
    return p;
}

cudaError_t launch_expanded_attention_tc(const ExpandedArgs& a) {
    const PagedPlan p = expanded_plan_tc(a.T);
    const PagedArgs pa = expanded_view(a);
    if (!tensor_map_encoder()) return cudaErrorNotSupported;
    CUtensorMap qm, nm, rm, vm;
    if (!make_map(&qm, a.q, kKey, a.H, a.T, kKey * 2, (cuuint64_t)a.q_stride * 2, kRows) ||
        !make_map(&nm, a.k_nope, kNope, a.H, a.S, (cuuint64_t)a.kn_head * 2, (cuuint64_t)a.kn_token * 2, kKeys / 2) ||
        !make_map(&rm, a.k_rope, 64, 1, a.S, 128, (cuuint64_t)a.kr_stride * 2, kKeys / 2) ||
        !make_map(&vm, a.v, kValue, a.H, a.S, (cuuint64_t)a.v_head * 2, (cuuint64_t)a.v_token * 2, kKeys))
        return cudaErrorInvalidValue;
    auto kern = kda_expanded_attention_tc_kernel;
    static OncePerDevice once;
    const cudaError_t e = once.run([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
    if (e != cudaSuccess) return e;
    const int pairs = std::min(p.max_ctas, sm_count() / 2);
    const cudaError_t err = launch_overlapped(
        kern, 2 * pairs, kThreads, kSmem, a.stream, 1, qm, nm, rm, vm,
        Values{static_cast<const __nv_bfloat16*>(a.v), a.v_token, a.v_head}, a.cu_seqlens, a.cu_seqlens_k, expanded_shape(a, p),
        a.scale * kLog2e, static_cast<__nv_bfloat16*>(a.o), a.lse, paged_partials(pa, p), a.status);
    if (err != cudaSuccess) return err;
    return launch_latent_merge(pa, p, pairs);
}

}  // namespace kda_host
