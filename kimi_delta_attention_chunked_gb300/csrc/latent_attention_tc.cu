// latent_attention_tc.cu -- absorbed attention over the paged latent cache on the tensor
// cores (bf16), by pairs of CTAs.
//
// A cache row of 576 channels is the key of every head and its first 512 channels the
// value.  A unit (paged.cuh) is up to 128 rows (a token and a query head each), up to 64 in either
// CTA of a cluster of two: half of the heads of the same tokens.  Per tile of KEYS keys, with cta_group::2
// products of M = 128:
//     S = Q K^T     (128 x KEYS over 576 channels, both operands in shared memory)
//     P = 2^(scale log2(e) S - m)   (registers; bf16 to shared memory)
//     O += P V      (128 x 512 over KEYS keys, two products of N = 256)
//
// Why a pair.  128 rows of 512 sums are the whole TMEM of an SM.  With M = 128 over two CTAs
// each holds 64 rows, and those use all 128 lanes: lanes 0-63 the first half of a product's N
// columns, lanes 64-127 the second.  So O takes 256 columns of TMEM and S KEYS / 2 (KEYS = 64), S is double
// buffered, and the tensor cores run at their full rate.  64 rows in a CTA alone would pay
// twice the tensor time for the same rows: half of the lanes stay idle there.
//
// Where the operands lie.  Of B each CTA brings half of N.  For S that is half of the tile's
// keys with all 576 channels, nine panels of 64 channels (panel 8 the rotated part).  For O it is half
// of the value channels with all keys, and a product's descriptors name the same place in both CTAs.
// So once S is complete, each CTA fetches over the four panels whose channels it does not need
// the other half's keys in its own channels, as follows (lo and hi: the tile's first and second half
// of the keys; CTA 0 loads lo, CTA 1 hi):
//     place         0,1       2,3       4,5       6,7       8
//     CTA 0, S     lo 0,1    lo 2,3    lo 4,5    lo 6,7    lo 8
//     CTA 0, O     lo 0,1    hi 0,1    lo 4,5    hi 4,5
//     CTA 1, S     hi 0,1    hi 2,3    hi 4,5    hi 6,7    hi 8
//     CTA 1, O     lo 2,3    hi 2,3    lo 6,7    hi 6,7
// Every cache row comes from HBM once; the four panels fetched again come from L2.
//
// Warps of each CTA: 0-3 softmax and output (a thread has one row and one half of the keys and
// of the channels); 4 copies tiles; 5 copies the four panels anew; 6 issues the products (in
// CTA 0, for both); 7 walks the units; 8 copies queries.  Barriers of loads and of P are CTA 0's, where the
// products are issued; a product's completion is told to both.
//
// Masked places.  A zero weight times a NaN or infinity in V is NaN.  So in a tile that not every
// row sees whole, once S is complete, the softmax warps zero the rows of V that no row of the unit
// sees, and in rows that some see and some do not take out the elements that are not finite.  They note
// if they found one (in both CTAs); the output then makes those channels NaN in the rows that see them.  NaN for an
// infinity too: the channel is one of the key's as well, so its score is NaN, or infinite and the weight NaN or 0.
//
// Bound, and what it measured (GPU time with the merge; HBM 6790 GB/s, cuBLAS 1888 TFLOP/s).  While it streams,
// HBM: a 64-key tile of a pair takes 0.85 us of the 0.83 that the copy rate allows, for any number of rows up to
// 128; with the cache in L2 (many units of a request), the tensor cores: 0.79 us of the 0.72 that cuBLAS's rate
// allows.  64 requests of 1 K to 16 K keys, 32 heads: 82 us (floor 61).  24 requests of 2 K to 32 K keys, 128
// heads: 73 us (46).  32 x 8 tokens, 32 heads, 0.7 K to 8 K keys: 60 us (29).  4 requests of 90 to 1500 keys:
// 14.2 us.  Chunks, which are all tensor cores: 512 tokens over 8192 keys, 128 heads 700 us, 1.62 PFLOP/s of what the mask
// leaves (floor 600), 16 heads 107 us, 1.33 (75: three to four units a pair), 2048 over 32768, 16 heads 1365 us, 1.66 (1199).
// Above the floors: 5 us before a pair's first product (its piece, the first unit, the page table, the
// first tile: a good part fetching instructions), 1.5 to 3 us to write a unit's sums, 5 to 10 for the merge.
// What it took, in the order of its worth: arrivals at the other CTA without a fence of global memory (136 ->
// 89 us in the first case); a merge of its own and partial sums in whole lines (verify 71 -> 61); a unit's last
// product not behind the next unit's queries; padding rows that do not move references; the heads of a token
// shared by both CTAs; the piece found by one warp.
// Rounding: P enters its product as bf16, the type of V (both operands have one type); the output's error
// against 64 bits is 2.0e-3 (2-norm), 1.7e-3 of it its own rounding to bf16.
#include <algorithm>

#include "attention_pair.cuh"
#include "latent.cuh"

namespace {

using namespace kda_tc;
using kda_latent::kLatent;
using kda_latent::kRow;
using kda_paged::Partials;
using kda_paged::Piece;
using kda_paged::Shape;
using kda_paged::Walker;

constexpr int kThreads = 288;
constexpr int kCopyWarp = 4, kSwapWarp = 5, kIssueWarp = 6, kWalkWarp = 7, kQueryWarp = 8;
constexpr int kRows = 64;                              // rows of a CTA
constexpr int kPanels = kRow / 64;                     // of a key
constexpr int kQPanel = kRows * 128;                   // bytes of 64 rows x 64 channels
constexpr int kUnits = 4;                              // unit descriptions in flight
constexpr int kTailBytes = 2 * 1024;

struct C {
    static constexpr int KEYS = 64, LOG2 = 6;          // keys of a tile: four tiles fit beside the queries
    static constexpr int HALF = KEYS / 2;              // keys that a CTA loads of a tile
    static constexpr int PANEL = HALF * 128;
    static constexpr int TILE = kPanels * PANEL;
    static constexpr int STAGES = 4;
    static constexpr int KV0 = kPanels * kQPanel;
    static constexpr int P0 = KV0 + STAGES * TILE;     // 64 rows x KEYS weights
    static constexpr int TAIL = P0 + kRows * KEYS * 2;
    static constexpr int SMEM = TAIL + kTailBytes;
    static constexpr uint32_t TMEM_S = 256;            // columns: O from 0, the two S behind it
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(STAGES * TILE >= kda_paged::kMaxRequests * 8 + 512, "scratch of find_piece");
};

// A CTA's rows of a unit: `heads` heads (the second CTA has the ones behind the first's) of `tokens` tokens.  The
// CTAs share the heads and not the tokens, so that a single token gives both of them the same work.
struct Tiling {
    int heads, tokens;
};

struct UnitSlot {
    Unit u;
    int more;                                          // 0: no further unit
};

struct Tail {
    uint64_t kv_full[4], sw_full[4], q_full, p_full;   // CTA 0's are used
    uint64_t kv_empty[4], s_full[2], q_empty, landed;  // each CTA's own
    uint64_t join[2];                                  // of the two warps that share rows
    uint64_t u_full[kUnits], u_empty[kUnits];
    uint64_t drain;
    uint32_t tmem;
    int abort;
    int odd_values[4];                                 // per unit, in turn: values that are not finite were taken out
    UnitSlot units[kUnits];
    float top[2][2][kRows];                            // per step, in turn: largest score of each half of the keys
    float sum[2][kRows];                               // sum of the weights of each half
};
static_assert(sizeof(Tail) <= kTailBytes, "tail");

// Makes NaN, in a row's output or partial sums, those of 128 channels from each of c0 and c0 + 256 on in which a key
// of [first, last), among those that not all rows of the unit see, is not finite: rare, and so out of the way of what
// every unit fetches.
__device__ __noinline__ void mark_odd_values(__nv_bfloat16* o, float* sums, int cap, int c0, const Shape& s,
                                            const __nv_bfloat16* cache, const int32_t* pages, int first, int last) {
    for (int key = first; key < last; ++key) {
        const int page = pages[key >> s.page_log2];
        if (page < 0 || page >= s.n_pages) continue;
        const __nv_bfloat16* v = cache + (((size_t)page << s.page_log2) + (key & ((1 << s.page_log2) - 1))) * kRow;
        for (int i = 0; i < 256; ++i) {
            const int c = c0 + (i & 127) + (i & 128) * 2;
            if ((__float_as_uint(__bfloat162float(v[c])) & 0x7f800000u) != 0x7f800000u) continue;
            if (o) o[c] = __float2bfloat16_rn(NAN);
            else sums[(size_t)(c >> 2) * cap * 4 + (c & 3)] = NAN;
        }
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
kda_latent_attention_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap qmap1,
                               const __grid_constant__ CUtensorMap kmap,
                               const __nv_bfloat16* __restrict__ cache, const int32_t* __restrict__ table,
                               const int32_t* __restrict__ cu, const int32_t* __restrict__ seq_len, Shape s, Tiling tiling,
                               float scale_log2, __nv_bfloat16* __restrict__ o, float* __restrict__ lse, Partials parts,
                               int* status) {
    extern __shared__ __align__(1024) unsigned char sm[];
    Tail& tl = *reinterpret_cast<Tail*>(sm + C::TAIL);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank(), cluster = blockIdx.x >> 1;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the merge may be set up; it waits for this grid
    if (w == kIssueWarp) {
        alloc_pair(&tl.tmem);
    }
    if (tid == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            kda::mbar_init(&tl.kv_full[i], 1);
            kda::mbar_init(&tl.sw_full[i], 1);
            kda::mbar_init(&tl.kv_empty[i], 1);
        }
        kda::mbar_init(&tl.q_full, 1);
        kda::mbar_init(&tl.q_empty, 1);
        kda::mbar_init(&tl.p_full, 8);
        kda::mbar_init(&tl.landed, 1);
        for (int i = 0; i < 2; ++i) {
            kda::mbar_init(&tl.s_full[i], 1);
            kda::mbar_init(&tl.join[i], 2);
        }
        for (int i = 0; i < kUnits; ++i) {
            kda::mbar_init(&tl.u_full[i], 1);
            kda::mbar_init(&tl.u_empty[i], rank == 0 ? 8 : 7);
        }
        kda::mbar_init(&tl.drain, 1);
        kda::fence_barrier_init();
        tl.abort = 0;
        for (int i = 0; i < 4; ++i) tl.odd_values[i] = 0;
    }
    if (w == kCopyWarp && lane < 3) {
        const CUtensorMap* m = lane == 0 ? &qmap : lane == 1 ? &qmap1 : &kmap;
        asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    cluster_arrive();                                  // both CTAs' barriers will be there
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the kernels before this one are complete
    // this pair's piece of the work; both CTAs find the same.  Few requests: the walking warp does, below
    auto* cost = reinterpret_cast<unsigned long long*>(sm + C::KV0);
    Piece piece{};
    if (s.n_req > kda_paged::kWarpRequests) {
        auto* red = cost + kda_paged::kMaxRequests;
        piece = kda_paged::find_piece<kThreads>(s, cu, seq_len, cluster, gridDim.x >> 1, cost, red,
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
    // pages of a half of a tile
    const int pieces = (1 << s.page_log2) >= C::HALF ? 1 : C::HALF >> s.page_log2;
    const int piece_log2 = min(s.page_log2, C::LOG2 - 1);
    // lane's page of half `which` of the tile: lane's piece is lane % pieces; n_pages reads as zeros
    auto page_of = [&](const Unit& u, int tile, int which) {
        const int key = (tile << C::LOG2) + which * C::HALF + ((lane % pieces) << piece_log2);
        int page = -1;
        if (key < u.kend) page = table[(size_t)u.n * s.blocks + (key >> s.page_log2)];
        return page < 0 || page >= s.n_pages ? s.n_pages : page;
    };
    // first place in its page of half `which` of a tile
    auto place_of = [&](int tile, int which) {
        return pieces > 1 ? 0 : ((tile << C::LOG2) + which * C::HALF) & ((1 << s.page_log2) - 1);
    };
    // the tile is not whole for every row of the unit
    auto edge = [&](const Sight& si, int tile) { return ((tile + 1) << C::LOG2) > si.all_hi; };
    int n_ld = 0, n_q = 0;                             // copies issued

    if (w == kWalkWarp) {
        // ---------------- unit descriptions
        if (lane == 0 && rank == 0) parts.clear_both(cluster);
        if (s.n_req <= kda_paged::kWarpRequests) {
            piece = kda_paged::find_piece_warp(s, cu, seq_len, cluster, gridDim.x >> 1, cost);
            kda::fence_proxy_async_smem();
        }
        Walker walk;
        walk.start(s, cu, seq_len, piece, cluster);
        for (int k = 0;; ++k) {
            Unit u;
            unsigned long long from;
            const bool more = walk.step(s, cu, seq_len, u, from);
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
        // ---------------- this CTA's half of every tile
        bool ok = true;
        for (int k = 0; ok; ++k) {
            Unit u;
            if (!read_unit(k, u)) break;
            int next_page = page_of(u, u.tb, rank);
            for (int tile = u.tb; tile < u.te; ++tile) {
                const int page = next_page, st = n_ld % C::STAGES, y = place_of(tile, rank);
                if (tile + 1 < u.te) next_page = page_of(u, tile + 1, rank);
                if (n_ld >= C::STAGES && !wait(&tl.kv_empty[st], (n_ld / C::STAGES - 1) & 1)) { ok = false; break; }
                __syncwarp();
                if (lane == 0 && rank == 0) kda::mbar_arrive_expect_tx(&tl.kv_full[st], 2 * C::TILE);
                __syncwarp();
                const uint32_t dst = kda::smem_u32(sm + C::KV0 + st * C::TILE) + ((lane % pieces) << (piece_log2 + 7));
                const uint32_t bar = at_rank(&tl.kv_full[st], 0);
                for (int c = lane / pieces; c < kPanels; c += 32 / pieces)
                    load_pair(dst + c * C::PANEL, &kmap, c * 64, y, page, bar);
                ++n_ld;
            }
        }
    } else if (w == kQueryWarp) {
        // ---------------- this CTA's rows of the queries
        const uint32_t q_bar = at_rank(&tl.q_full, 0);
        for (int k = 0;; ++k) {
            Unit u;
            if (!read_unit(k, u)) break;
            const bool one = u.ntok == 1;              // its rows alone: a fourth and less of what the box of all tokens brings
            const int bytes = kPanels * tiling.heads * (one ? 1 : tiling.tokens) * 128;
            if (k > 0 && !wait(&tl.q_empty, (k - 1) & 1)) break;
            __syncwarp();
            if (lane == 0 && rank == 0) kda::mbar_arrive_expect_tx(&tl.q_full, 2 * bytes);
            __syncwarp();
            if (lane < kPanels)
                load_pair(kda::smem_u32(sm) + lane * kQPanel, one ? &qmap1 : &qmap, lane * 64, u.qh0 + rank * tiling.heads, u.tok0,
                          q_bar);
            ++n_q;
        }
    } else if (w == kSwapWarp) {
        // ---------------- once S is complete, the other half's keys in this CTA's channels over
        // the panels whose channels it does not need: CTA 0 at places 2, 3, 6, 7, CTA 1 at 0, 1, 4, 5
        int g = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            Unit u;
            if (!read_unit(k, u)) break;
            int next_page = page_of(u, u.tb, rank ^ 1);
            for (int tile = u.tb; tile < u.te; ++tile, ++g) {
                const int page = next_page, st = g % C::STAGES, y = place_of(tile, rank ^ 1);
                if (tile + 1 < u.te) next_page = page_of(u, tile + 1, rank ^ 1);
                if (!wait(&tl.s_full[g & 1], (g >> 1) & 1)) { ok = false; break; }
                __syncwarp();
                if (lane == 0 && rank == 0) kda::mbar_arrive_expect_tx(&tl.sw_full[st], 8 * C::PANEL);
                __syncwarp();
                const uint32_t dst = kda::smem_u32(sm + C::KV0 + st * C::TILE) + ((lane % pieces) << (piece_log2 + 7));
                const uint32_t bar = at_rank(&tl.sw_full[st], 0);
                for (int i = lane / pieces; i < 4; i += 32 / pieces) {
                    const int c = 4 * (i >> 1) + (i & 1) + 2 * rank;          // channels, in panels; places: c ^ 2
                    load_pair(dst + (c ^ 2) * C::PANEL, &kmap, c * 64, y, page, bar);
                }
            }
        }
        n_ld = g;
    } else if (w == kIssueWarp) {
        // ---------------- products: CTA 0 issues for both.  All lanes wait, an elected one issues
        const uint32_t id_s = kda::idesc_bf16(128, C::KEYS, 0, 0), id_o = kda::idesc_bf16(128, 256, 0, 1);
        const uint64_t q_desc = kda::sw128_desc(kda::smem_u32(sm), 16, 1024);
        const uint64_t k_desc = kda::sw128_desc(kda::smem_u32(sm + C::KV0), 16, 1024);
        const uint64_t v_desc = kda::sw128_desc(kda::smem_u32(sm + C::KV0), C::PANEL, 1024);
        const uint64_t p_desc = kda::sw128_desc(kda::smem_u32(sm + C::P0), 16, 1024);
        int g = 0;
        bool issued = false, due = false, due_first = false, due_edge = false, ok = rank == 0;
        // O (+)= P V of step g
        auto values_step = [&](int step) -> bool {
            const int st = step % C::STAGES;
            if (!wait(&tl.sw_full[st], (step / C::STAGES) & 1)) return false;
            if (due_edge && lane < 2) arrive_remote(at_rank(&tl.landed, lane));      // both CTAs may clean
            __syncwarp();
            if (!wait(&tl.p_full, step & 1)) return false;
            kda::tc_fence_after();
            if (elect_one()) {
                const uint64_t b = v_desc + kda::desc_step(st * C::TILE);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < C::KEYS / 16; ++i) {
                        const int hi = i >= C::HALF / 16;          // second half of the keys: two places on
                        mma_pair(tmem + j * 128, p_desc + kda::desc_step(i * 32),
                                 b + kda::desc_step((4 * j + 2 * hi) * C::PANEL + (i - hi * (C::HALF / 16)) * 2048), id_o,
                                 (i > 0 || !due_first) ? 1u : 0u);
                    }
                commit_pair(&tl.kv_empty[st]);
            }
            __syncwarp();
            return true;
        };
        for (int k = 0; ok; ++k) {
            Unit u;
            if (!read_unit(k, u)) break;
            const Sight si = sight(u, 0, 0, u.ntok - 1);
            const int tb = uniform(u.tb), te = uniform(u.te);
            for (int tile = tb; tile < te; ++tile, ++g) {
                const int st = g % C::STAGES;
                // the last product of a unit does not wait for the next one's queries, which are fetched
                // when its last scores are done
                if (due && tile == tb) {
                    ok = values_step(g - 1);
                    due = false;
                }
                ok = ok && wait(&tl.kv_full[st], (g / C::STAGES) & 1);
                if (ok && tile == tb) ok = wait(&tl.q_full, k & 1);
                if (!ok) break;
                kda::tc_fence_after();
                if (elect_one()) {
                    const uint64_t b = k_desc + kda::desc_step(st * C::TILE);
                    const uint32_t d = tmem + C::TMEM_S + (g & 1) * C::HALF;
#pragma unroll
                    for (int i = 0; i < kRow / 16; ++i)
                        mma_pair(d, q_desc + kda::desc_step((i >> 2) * kQPanel + (i & 3) * 32),
                                 b + kda::desc_step((i >> 2) * C::PANEL + (i & 3) * 32), id_s, i > 0 ? 1u : 0u);
                    commit_pair(&tl.s_full[g & 1]);
                    if (tile == te - 1) commit_pair(&tl.q_empty);
                }
                __syncwarp();
                issued = true;
                if (due) ok = values_step(g - 1);
                if (!ok) break;
                due = true;
                due_first = tile == tb;
                due_edge = edge(si, tile);
            }
        }
        if (ok && due) ok = values_step(g - 1);
        if (issued) {                                  // no product in flight when TMEM is freed
            if (elect_one()) commit_pair(&tl.drain, 1);
            __syncwarp();
            (void)kda::mbar_wait(&tl.drain, 0, kda::kWaitCycles);
        }
    } else {
        // ---------------- softmax and output: row, half of the keys and of each product's channels
        const int row = tid & 63, half = tid >> 6;
        const uint32_t lane_off = (uint32_t)(w * 32) << 16;
        const int tok_in = row / tiling.heads, head_in = rank * tiling.heads + row % tiling.heads;
        const bool in_tile = row < tiling.heads * tiling.tokens;
        const uint32_t p_bar = at_rank(&tl.p_full, 0);
        int g = 0, n_landed = 0, n_join = 0;
        auto join = [&]() -> bool {                    // the two threads of a row meet: their warps do
            __syncwarp();
            if (lane == 0) kda::mbar_arrive(&tl.join[w & 1]);
            return wait(&tl.join[w & 1], n_join++ & 1);
        };
        bool ok = true;
        for (int k = 0; ok; ++k) {
            Unit u;
            if (!read_unit(k, u)) break;
            const bool valid = in_tile && tok_in < u.ntok && u.qh0 + head_in < s.Hq;
            const int hi = valid ? min(max(u.pos + tok_in + 1, 0), u.kend) : 0;
            const bool busy = __any_sync(0xffffffffu, valid);
            const Sight si = sight(u, 0, 0, u.ntok - 1);
            // lane's page of this half of the tile: 0 where there is nothing to judge
            auto judge = [&](int tile) {
                const int key = (tile << C::LOG2) + half * C::HALF + (lane << piece_log2);
                return lane < pieces && key < u.kend ? table[(size_t)u.n * s.blocks + (key >> s.page_log2)] : 0;
            };
            float m = -INFINITY, l = 0.f;
            int page = busy ? judge(u.tb) : 0;
            for (int tile = u.tb; tile < u.te; ++tile, ++g) {
                const int k0 = (tile << C::LOG2) + half * C::HALF;
                const unsigned missing = __ballot_sync(0xffffffffu, page < 0 || page >= s.n_pages);
                if (busy && tile + 1 < u.te) page = judge(tile + 1);
                const bool at_edge = edge(si, tile);
                const int before = g - 1;              // its product must be complete before P and O are touched
                auto wait_before = [&] {
                    return before < 0 || wait(&tl.kv_empty[before % C::STAGES], (before / C::STAGES) & 1);
                };
                if (!wait(&tl.s_full[g & 1], (g >> 1) & 1)) { ok = false; break; }
                kda::tc_fence_after();
                uint32_t p[C::HALF / 2];
                if (busy) {
                    float x[C::HALF];
#pragma unroll
                    for (int c = 0; c < C::HALF; c += 32)
                        kda::tmem_ld32(tmem + lane_off + C::TMEM_S + (g & 1) * C::HALF + c, x + c);
                    kda::tmem_wait_ld();
                    if (at_edge || missing) {
#pragma unroll
                        for (int c = 0; c < C::HALF; c += 16) {
                            const bool none = (missing >> (c >> piece_log2)) & 1;
#pragma unroll
                            for (int e = 0; e < 16; ++e) x[c + e] = none || k0 + c + e >= hi ? -INFINITY : x[c + e];
                        }
                    }
                    float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int c = 4; c < C::HALF; c += 4)
#pragma unroll
                        for (int e = 0; e < 4; ++e) top[e] = fmaxf(top[e], x[c + e]);
                    float big = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    tl.top[g & 1][half][row] = big;
                    if (!join()) { ok = false; break; }
                    big = fmaxf(big, tl.top[g & 1][half ^ 1][row]);
                    if (tile == u.tb) {
                        m = big;
                    } else {
                        const bool grow = valid && (big - m) * scale_log2 > kGrow;
                        if (__any_sync(0xffffffffu, grow)) {
                            if (!wait_before()) { ok = false; break; }
                            kda::tc_fence_after();
                            const float f = grow ? ex2((m - big) * scale_log2) : 1.f;
#pragma unroll 1
                            for (int c = 0; c < 256; c += 16) {
                                float y[16];
                                kda::tmem_ld16(tmem + lane_off + c, y);
                                kda::tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) y[e] *= f;
                                kda::tmem_st16(tmem + lane_off + c, y);
                            }
                            kda::tmem_wait_st();
                            l *= f;
                            if (grow) m = big;
                        }
                    }
                    const float ref = kda_paged::reference(m, scale_log2);
                    const uint64_t sc2 = pack2(scale_log2, scale_log2), off2 = pack2(-ref, -ref);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int c = 0; c < C::HALF; c += 2) {
                        float a, b;
                        unpack2(fma2(pack2(x[c], x[c + 1]), sc2, off2), a, b);
                        a = ex2(a);
                        b = ex2(b);
                        sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pack2(a, b));
                        p[c >> 1] = kda::pack_bf16x2(a, b);
                    }
                    float sa, sb;
                    unpack2(add2(sum[0], sum[1]), sa, sb);
                    l += sa + sb;
                }
                if (!wait_before()) { ok = false; break; }
                if (busy) {
                    unsigned char* dst = sm + C::P0 + row * 128;
#pragma unroll
                    for (int i = 0; i < C::HALF / 8; ++i)
                        *reinterpret_cast<uint4*>(dst + (((half * (C::HALF / 8) + i) ^ (row & 7)) << 4)) =
                            make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
                }
                if (at_edge) {
                    // values that must not meet a zero weight (see the header)
                    if (!wait(&tl.landed, n_landed & 1)) { ok = false; break; }
                    ++n_landed;
                    unsigned char* v = sm + C::KV0 + (g % C::STAGES) * C::TILE;
                    const int t0 = tile << C::LOG2;
                    int odd = 0;
#pragma unroll 1
                    for (int e = tid; e < 8 * C::HALF * 8; e += 128) {
                        const int chunk = e & 7, r = (e >> 3) & (C::HALF - 1), place = (e >> 3) / C::HALF;
                        const int key = t0 + ((place >> 1) & 1) * C::HALF + r;
                        if (key < si.all_hi) continue;
                        uint4* at = reinterpret_cast<uint4*>(v + place * C::PANEL + r * 128 + chunk * 16);
                        uint4 x = make_uint4(0, 0, 0, 0);
                        if (key < si.hi) {
                            x = *at;
                            if (!take_odd(x)) continue;
                            odd = 1;
                        }
                        *at = x;
                    }
                    if (odd) flag_pair(&tl.odd_values[k & 3]);
                }
                kda::fence_proxy_async_smem();
                kda::tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_remote(p_bar);
            }
            if (!ok) break;
            // ---- output
            const int last = g - 1;
            if (busy) {
                tl.sum[half][row] = l;
                if (!join()) break;
                l += tl.sum[half ^ 1][row];
            }
            const float2 st = kda_paged::row_stats(m, l, scale_log2);
            if (!wait(&tl.kv_empty[last % C::STAGES], (last / C::STAGES) & 1)) break;
            kda::tc_fence_after();
            if (busy) {
                const bool whole = u.first && u.last;
                const int which = u.first ? 1 : 0;
                const size_t at = (size_t)(u.tok0 + tok_in) * s.Hq + u.qh0 + head_in;
                const int prow = tok_in * 2 * tiling.heads + head_in;                // row of a partial slot
                const float sum_l = kda_paged::whole_sum(st.x, st.y), inv = sum_l == 0.f ? 0.f : 1.f / sum_l;
                __nv_bfloat16* const dst = o + at * kLatent;
                float4* const part = reinterpret_cast<float4*>(parts.sums4(cluster, which, valid ? prow : 0, 0));
#pragma unroll 1
                for (int c = 0; c < 256; c += 16) {
                    float y[16];
                    kda::tmem_ld16(tmem + lane_off + c, y);
                    kda::tmem_wait_ld();
                    if (!valid) continue;
                    const int c0 = (c & 128) * 2 + half * 128 + (c & 127);          // channel
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) y[e] *= inv;
                        store16(dst + c0, y);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            part[(c0 / 4 + e) * parts.cap] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                    }
                }
                if (valid && *(volatile int*)&tl.odd_values[k & 3])
                    mark_odd_values(whole ? dst : nullptr, reinterpret_cast<float*>(part), parts.cap, half * 128, s, cache,
                                    table + (size_t)u.n * s.blocks, max(si.all_hi, u.tb << C::LOG2),
                                    min(min(si.hi, hi), u.te << C::LOG2));
                if (valid && half == 0) {
                    if (!whole) parts.stats(cluster, which)[prow] = st;
                    else if (lse) lse[at] = sum_l == 0.f ? -INFINITY : (st.x + log2f(sum_l)) * kLn2;
                }
            }
            // no CTA is at the unit after the next before this one has arrived for the next
            if (row == 0 && half == 0) tl.odd_values[(k + 2) & 3] = 0;
            kda::tc_fence_before();
        }
    }
    kda::tc_fence_before();
    __syncthreads();
    if (*abort_f && rank == 0) {                       // no copy in flight into shared memory that is given up
        if (w == kCopyWarp) {
            for (int i = max(0, n_ld - C::STAGES); i < n_ld; ++i)
                (void)kda::mbar_wait(&tl.kv_full[i % C::STAGES], (i / C::STAGES) & 1, kda::kWaitCycles);
        }
        if (w == kQueryWarp && n_q > 0) (void)kda::mbar_wait(&tl.q_full, (n_q - 1) & 1, kda::kWaitCycles);
        if (w == kSwapWarp)
            for (int i = max(0, n_ld - C::STAGES); i < n_ld; ++i)
                (void)kda::mbar_wait(&tl.sw_full[i % C::STAGES], (i / C::STAGES) & 1, kda::kWaitCycles);
    }
    __syncthreads();
    cluster_leave();                                   // the other CTA is done with this one's memory and TMEM
    if (w == kIssueWarp) dealloc_pair(tmem);
}

// ---- host
Tiling tiling_of(int H) {
    const int groups = kda_host::latent_groups(H, 2 * kRows);        // of a unit's heads each
    Tiling t;
    t.heads = ((H + groups - 1) / groups + 1) / 2;
    t.tokens = kRows / t.heads;
    return t;
}

bool make_map(CUtensorMap* m, const void* base, cuuint64_t d1, cuuint64_t d2, cuuint64_t stride1, cuuint64_t stride2, int box1,
              int box2) {
    const cuuint64_t dims[3] = {(cuuint64_t)kRow, d1, d2};
    const cuuint64_t strides[2] = {stride1, stride2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box1, (cuuint32_t)box2};
    const cuuint32_t one[3] = {1, 1, 1};
    return kda_host::tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
                                          one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

namespace kda_host {

PagedPlan latent_plan_tc(int T, int H) {
    const Tiling t = tiling_of(H);
    PagedPlan p;
    p.Gv = 2 * t.heads;                                // heads of a unit
    p.U = t.tokens;
    p.rows = paged_slot_rows(p.U, T, p.Gv);
    p.tile_log2 = C::LOG2;
    p.max_ctas = 80;                                   // pairs
    // places for a unit's fixed cost; with 0, 2, 5, 8 and 12: 64 decode requests 87.3, 83.9, 83.2, 84.8 and 87.0 us,
    // verification 68.2, 63.7, 60.9, 62.1 and 64.1, 128 heads 75.6, 73.9, 73.0, 73.5 and 74.0
    p.extra = 5;
    return p;
}

cudaError_t launch_latent_attention_tc(const LatentArgs& a) {
    const PagedPlan p = latent_plan_tc(a.T, a.H);
    const PagedArgs pa = latent_view(a);
    const Tiling t = tiling_of(a.H);
    if (!tensor_map_encoder()) return cudaErrorNotSupported;
    CUtensorMap qm, qm1, km;
    constexpr cuuint64_t row = kRow * 2;
    if (!make_map(&qm, a.q, a.H, a.T, row, (cuuint64_t)a.q_stride * 2, t.heads, t.tokens) ||
        !make_map(&qm1, a.q, a.H, a.T, row, (cuuint64_t)a.q_stride * 2, t.heads, 1) ||
        !make_map(&km, a.cache, a.page_size, a.n_pages, row, row * a.page_size, std::min(a.page_size, C::HALF), 1))
        return cudaErrorInvalidValue;
    auto kern = kda_latent_attention_tc_kernel;
    static OncePerDevice once;
    const cudaError_t e = once.run([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (e != cudaSuccess) return e;
    const int pairs = std::min(p.max_ctas, sm_count() / 2);
    const cudaError_t err = launch_overlapped(
        kern, 2 * pairs, kThreads, C::SMEM, a.stream, 1, qm, qm1, km, static_cast<const __nv_bfloat16*>(a.cache),
        a.block_table, a.cu_seqlens, a.seq_len, latent_shape(a, p), t, a.scale * kLog2e, static_cast<__nv_bfloat16*>(a.o), a.lse,
        paged_partials(pa, p), a.status);
    if (err != cudaSuccess) return err;
    return launch_latent_merge(pa, p, pairs);
}

}  // namespace kda_host
