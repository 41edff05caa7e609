// paged_attention_tc.cu -- attention over a paged cache on the tensor cores
// (bf16).
//
// A unit (paged.cuh) is up to 2 x 128 rows: tile i of its rows holds BT = 128 /
// Gv tokens with the Gv query heads that share a cache head, row = token * Gv +
// head, which is the order in which TMA brings a [heads, tokens] box of q to
// shared memory.  Per 128-key tile:
//     S = Q K^T     (128 x 128, both operands in shared memory, S in TMEM)
//     P = 2^(scale log2(e) S - m)   (registers; written back over S as bf16)
//     O += P V      (P from TMEM, V from shared memory, O in TMEM)
// m is a reference per row, not the running maximum: it moves, and O and the sum
// of weights are scaled, only when a score exceeds it by more than 8 octaves,
// so that almost no tile pays for reading O back.  The weights then reach 2^8,
// which costs no accuracy in a floating-point format, and o / l does not change.
//
// Work goes in steps of one row tile and one key tile; step g uses half g & 1 of
// TMEM (S, O) and one of two groups of four softmax warps.  A unit with two row
// tiles takes its key tiles in two steps each, one per row tile, so that the
// tensor cores run one half's products while the other half's weights are
// formed and every key tile is loaded once.  A unit with one row tile (a few
// tokens) sends its key tiles to the two halves in turn; the halves then hold
// the sums over the even and the odd key tiles and are joined at the end.
//
// Warps: 0-3 and 4-7 softmax and output of half 0 and 1; 8 copies (TMA, one
// box of a page per lane); 9 issues the products and cleans masked values (below);
// 10 walks the CTA's units.  Rings: key and value tiles, unit descriptions.
// Every wait is bounded (kda::kWaitCycles), as in the prefill.
//
// Masked places.  K rows that a row does not see only make scores that are
// replaced; but a zero weight times a NaN or infinity in V is NaN.  So before
// the product the issuing warp zeroes the rows of V that no row of the unit
// sees (behind the last token, in a page's rest, before the window), and in
// the rows that some see and some do not (the triangle of the new tokens) takes
// out the elements that are not finite.  It notes if it found one; the output
// warps then add such elements themselves to the rows that see them.
//
// Bound, and what it measured (GPU time with the merge; HBM 6694 GB/s, 1885 TFLOP/s).
// Decode: HBM, the cache is read once: 64 requests of 1 K to 16 K keys, 32/8 heads
// of 128, 235 us, 0.93 of the copy rate.  32 requests x 8 tokens, 32/4 heads: 52 us,
// floor 31: HBM while it streams, then the last unit's latency and the merge.
// Long chunks: 2 x 4096 tokens over 12,000 and 27,001, 32/4 heads: 1.79 to 1.96 ms from run
// to run, 1.48 to 1.61 PFLOP/s (the card is at its power limit): tensor pipe 69 % active.
// With heads of 64 and 32 the same chunk takes 1.61 and 1.56 ms: the softmax warps, 3.5 to
// 3.6e12 weights a second.  Mixed lengths: uneven pieces (paged.cuh).
// What it took, in the order of its worth there: one elected lane issues (its
// operands stay in uniform registers: 2.99 -> 2.21 ms); that warp's loop over the
// key tiles in uniform control flow, with no more than waits and products (-> 1.91 ms).
// Sixteen softmax warps took issue slots from it (2.50 -> 2.39 ms against 1.91).
// Rounding: P enters its product as bf16, the type of V (both operands have one
// type); the output's error against 64 bits is 2.3e-3, 1.7e-3 of it the bf16 output.
#include <algorithm>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <mutex>

#include "paged.cuh"
#include "umma.cuh"

namespace {

using kda_paged::Partials;
using kda_paged::Piece;
using kda_paged::Shape;
using kda_paged::Unit;
using kda_paged::Walker;

constexpr int kThreads = 384;
constexpr int kCopyWarp = 8, kIssueWarp = 9, kWalkWarp = 10;
constexpr int kKeys = 128;                             // keys of a tile
constexpr int kKeysLog2 = 7;
constexpr int kPanel = 128 * 128;                      // bytes of 128 rows x 64 bf16
constexpr int kUnits = 4;                              // unit descriptions in flight
constexpr float kGrow = 8.f;                           // octaves that a score may exceed the reference
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr int kTailBytes = 3 * 1024;

template <int D>
struct Cfg {
    static constexpr int PANELS = D < 64 ? 1 : D / 64;  // d = 32: a panel whose upper half TMA fills with zeros
    static constexpr int TILE = PANELS * kPanel;       // bytes of a tile of q, keys or values
    static constexpr int STAGES = D == 128 ? 5 : 10;
    static constexpr int KV0 = 2 * TILE;
    static constexpr int TAIL = KV0 + STAGES * TILE;
    static constexpr int SMEM = TAIL + kTailBytes;
    static constexpr uint32_t TMEM_O = 256;            // columns: S halves at 0 and 128, O halves from 256
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(STAGES * TILE >= kda_paged::kMaxRequests * 8 + 512, "scratch of find_piece");
};

struct UnitSlot {
    Unit u;
    int more;                                          // 0: no further unit
};

struct Tail {
    uint64_t kv_full[10], kv_empty[10];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t join_a, join_b;
    uint64_t u_full[kUnits], u_empty[kUnits];
    uint64_t drain;
    uint32_t tmem;
    int abort;
    int odd_values[4];                                 // per unit, in turn: values that are not finite were taken out
    UnitSlot units[kUnits];
    float2 stats[2][128];                              // (reference in octaves, sum of weights) of each half's rows
};
static_assert(sizeof(Tail) <= kTailBytes, "tail");

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int x, int y, int z, int t,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(t), "r"(kda::smem_u32(bar))
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], A (M = 128) as bf16 pairs: lane = row, 8
// columns per 16 elements of K.
__device__ __forceinline__ void umma_bf16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* u) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
        "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
        "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
        "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
        : "memory");
}

// One lane of the (converged) warp.  Unlike `lane == 0`, the compiler keeps what
// is the same for the whole warp in uniform registers across this branch, where
// the operands of tcgen05.mma have to be.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// A value that is the same in all lanes, in a form the compiler knows to be so.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// What the keys of a unit mean for the rows [first, last] of its tokens.
struct Sight {
    int lo, hi;                                        // keys [lo, hi): some row sees them
    int all_lo, all_hi;                                // keys [all_lo, all_hi): every row sees them
};
__device__ __forceinline__ Sight sight(const Unit& u, int window, int first, int last) {
    Sight s;
    const int p0 = u.pos + first, p1 = u.pos + last;
    s.hi = min(max(p1 + 1, 0), u.kend);
    s.all_hi = min(max(p0 + 1, 0), u.kend);
    s.lo = kda_paged::first_key(p0, window);
    s.all_lo = kda_paged::first_key(p1, window);
    return s;
}

// Adds to o[0..31] (columns c0 ..) the values that are not finite, of the keys
// that this row sees among those that not all rows of the unit see.
template <int D>
__device__ __forceinline__ void add_odd_values(float* o, int c0, const Unit& u, const Sight& un, int lo, int hi,
                                            const Shape& s, const __nv_bfloat16* vc, const int32_t* table) {
    for (int half = 0; half < 2; ++half) {
        int a = half == 0 ? un.lo : max(un.all_hi, min(un.all_lo, un.hi));
        int b = half == 0 ? min(un.all_lo, un.hi) : un.hi;
        a = max(max(a, lo), u.tb << kKeysLog2);
        b = min(min(b, hi), u.te << kKeysLog2);
        for (int key = a; key < b; ++key) {
            const int page = table[(size_t)u.n * s.blocks + (key >> s.page_log2)];
            if (page < 0 || page >= s.n_pages) continue;
            const __nv_bfloat16* v =
                vc + ((((size_t)page * s.Hkv + u.kvh) << s.page_log2) + (key & ((1 << s.page_log2) - 1))) * D + c0;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                const float x = __bfloat162float(v[c]);
                if ((__float_as_uint(x) & 0x7f800000u) == 0x7f800000u) o[c] += x;
            }
        }
    }
}

// The rest of a wait that did not succeed at once.  One copy of it for the whole
// kernel: its many inlined ones would be most of what a short call fetches.
__device__ __noinline__ bool wait_longer(uint64_t* b, uint32_t parity, volatile int* abort, int* status) {
    const bool done = kda::mbar_wait_or_abort(b, parity, kda::kWaitCycles, abort);
    if (__all_sync(0xffffffffu, done)) return true;
    if (!*abort) kda::record_status(status, kda::kDevTimeout);
    *abort = 1;
    return false;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
kda_paged_attention_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                              const __grid_constant__ CUtensorMap vmap, const __nv_bfloat16* __restrict__ vc,
                              const int32_t* __restrict__ table, const int32_t* __restrict__ cu,
                              const int32_t* __restrict__ seq_len, Shape s, int BT, float scale_log2,
                              __nv_bfloat16* __restrict__ o, float* __restrict__ lse, Partials parts, int* status) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char sm[];
    Tail& tl = *reinterpret_cast<Tail*>(sm + C::TAIL);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the merge may be set up; it waits for this grid
    if (w == kIssueWarp) {
        kda::tmem_alloc(&tl.tmem, 512);
        kda::tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            kda::mbar_init(&tl.kv_full[i], 1);
            kda::mbar_init(&tl.kv_empty[i], 1);
        }
        kda::mbar_init(&tl.q_full, 1);
        kda::mbar_init(&tl.q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            kda::mbar_init(&tl.s_full[i], 1);
            kda::mbar_init(&tl.p_full[i], 4);
            kda::mbar_init(&tl.o_full[i], 1);
        }
        kda::mbar_init(&tl.join_a, 8);
        kda::mbar_init(&tl.join_b, 8);
        for (int i = 0; i < kUnits; ++i) {
            kda::mbar_init(&tl.u_full[i], 1);
            kda::mbar_init(&tl.u_empty[i], 10);
        }
        kda::mbar_init(&tl.drain, 1);
        kda::fence_barrier_init();
        tl.abort = 0;
    }
    if (w == kCopyWarp && lane < 3) {
        const CUtensorMap* m = lane == 0 ? &qmap : lane == 1 ? &kmap : &vmap;
        asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    // this CTA's piece of the work
    auto* cost = reinterpret_cast<unsigned long long*>(sm + C::KV0);
    auto* red = cost + kda_paged::kMaxRequests;
    const Piece piece = kda_paged::find_piece<kThreads>(s, cu, seq_len, blockIdx.x, gridDim.x, cost, red,
                                                        reinterpret_cast<Piece*>(red + kThreads / 32));
    kda::fence_proxy_async_smem();                     // the scratch becomes the target of copies
    kda::tc_fence_before();
    __syncthreads();
    kda::tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)tl.tmem);
    volatile int* abort_f = &tl.abort;
    // true once the phase is complete; false when this CTA gives up.  Called by all
    // lanes of a warp, with one answer for all of them, so that none leaves a loop alone
    auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
        if (__all_sync(0xffffffffu, kda::mbar_try_wait(b, parity))) return true;
        return wait_longer(b, parity, &tl.abort, status);
    };
    int n_ld = 0, n_q = 0;                             // copies issued (copy warp) or taken (issuing warp)
    // reads unit description k; every lane of the calling warp gets it
    auto read_unit = [&](int k, Unit& u) -> bool {
        if (!wait(&tl.u_full[k % kUnits], (k / kUnits) & 1)) return false;
        const UnitSlot& sl = tl.units[k % kUnits];
        u = sl.u;
        const bool more = sl.more != 0;
        __syncwarp();
        if (lane == 0) kda::mbar_arrive(&tl.u_empty[k % kUnits]);
        return more;
    };

    if (w == kWalkWarp) {
        // ---------------- unit descriptions
        if (lane == 0) parts.clear(blockIdx.x);
        Walker walk;
        walk.start(s, cu, seq_len, piece, blockIdx.x);
        for (int k = 0;; ++k) {
            Unit u;
            const bool more = walk.next(s, cu, seq_len, u);
            if (k >= kUnits && !wait(&tl.u_empty[k % kUnits], (k / kUnits - 1) & 1)) break;
            __syncwarp();
            if (lane == 0) {
                if (more) tl.units[k % kUnits].u = u;
                tl.units[k % kUnits].more = more;
                kda::mbar_arrive(&tl.u_full[k % kUnits]);
            }
            if (!more) break;
            if (lane == 0) parts.describe(blockIdx.x, u);
        }
    } else if (w == kCopyWarp) {
        // ---------------- copies: the keys, then the values of each tile.  (With the values two
        // steps behind, in the order of the products, a unit's last ones came behind the next unit's
        // first keys, and its output held up the ring.)
        const int pieces = s.page_log2 >= kKeysLog2 ? 1 : kKeys >> s.page_log2;   // pages of a tile
        const int box_rows = min(1 << s.page_log2, kKeys);
        auto page_of = [&](const Unit& u, int tile) {  // lane's page of the tile; n_pages reads as zeros
            const int key = (tile << kKeysLog2) + lane * box_rows;
            int page = -1;
            if (lane < pieces && key < u.kend) page = table[(size_t)u.n * s.blocks + (key >> s.page_log2)];
            return page < 0 || page >= s.n_pages ? s.n_pages : page;
        };
        auto load = [&](const CUtensorMap* map, int page, int y, int kvh) -> bool {
            const int st = n_ld % C::STAGES;
            if (n_ld >= C::STAGES && !wait(&tl.kv_empty[st], (n_ld / C::STAGES - 1) & 1)) return false;
            __syncwarp();
            if (lane == 0) kda::mbar_arrive_expect_tx(&tl.kv_full[st], C::TILE);
            __syncwarp();
            if (lane < pieces) {
                const uint32_t dst = kda::smem_u32(sm + C::KV0 + st * C::TILE) + lane * box_rows * 128;
#pragma unroll
                for (int c = 0; c < C::PANELS; ++c)
                    tma_load_4d(dst + c * kPanel, map, c * 64, y, kvh, page, &tl.kv_full[st]);
            }
            ++n_ld;
            return true;
        };
        auto load_q = [&](const Unit& u, bool two) {
            __syncwarp();
            if (lane == 0) {
                kda::mbar_arrive_expect_tx(&tl.q_full, (two ? 2 : 1) * C::PANELS * BT * s.Gv * 128);
                for (int i = 0; i < (two ? 2 : 1); ++i)
                    for (int c = 0; c < C::PANELS; ++c)
                        kda::tma_load_3d(sm + i * C::TILE + c * kPanel, &qmap, c * 64, u.qh0, u.tok0 + i * BT, &tl.q_full);
            }
            ++n_q;
        };
        bool ok = true;
        for (int k = 0; ok; ++k) {
            Unit u;
            if (!read_unit(k, u)) break;
            const bool two = u.ntok > BT;
            int next_page = page_of(u, u.tb);
            for (int tile = u.tb; ok && tile < u.te; ++tile) {
                const int page = next_page;
                if (tile + 1 < u.te) next_page = page_of(u, tile + 1);
                const int y = (tile << kKeysLog2) & ((1 << s.page_log2) - 1) & ~(box_rows - 1);
                ok = load(&kmap, page, y, u.kvh);
                if (ok && tile == u.tb) {
                    ok = k == 0 || wait(&tl.q_empty, (k - 1) & 1);
                    if (ok) load_q(u, two);
                }
                if (ok) ok = load(&vmap, page, y, u.kvh);
            }
        }
    } else if (w == kIssueWarp) {
        // ---------------- products.  All lanes wait, an elected one issues.  P_h lies over S_h: the
        // scores of a half's next step are issued behind its product P_h V, which waited for P_h, and
        // the tensor cores take products in the order of issue, so neither is overwritten in use
        const uint32_t id_s = kda::idesc_bf16(128, 128, 0, 0), id_o = kda::idesc_bf16(128, D, 0, 1);
        const uint64_t q_desc = kda::sw128_desc(kda::smem_u32(sm), 16, 1024);
        const uint64_t k_desc = kda::sw128_desc(kda::smem_u32(sm + C::KV0), 16, 1024);
        const uint64_t v_desc = kda::sw128_desc(kda::smem_u32(sm + C::KV0), kPanel, 1024);
        int g = 0, v_stage = 0, k_stage = 0;
        // the next tile's keys, and the parity of their stage; its values have the stage behind
        int stage = 0;
        uint32_t ring = 0;
        auto advance = [&](int& at, uint32_t& parity) {
            if (++at == C::STAGES) { at = 0; parity ^= 1; }
        };
        auto take_keys = [&](int& v_at, uint32_t& v_ring) -> bool {
            k_stage = stage;
            if (!wait(&tl.kv_full[stage], ring)) return false;
            advance(stage, ring);
            v_at = stage;
            v_ring = ring;
            advance(stage, ring);
            return true;
        };
        uint32_t p_phase = 0;                          // bit h: parity of the next P_h
        bool issued = false;
        // a step whose second product is due: flags, key tile, and what its unit's rows see
        enum { kFirstUse = 1, kLastUse = 2, kAdd = 4, kFinal = 8, kDue = 16 };
        struct Pending { int flags, tile, slot, kend, v_at; uint32_t v_ring; Sight si; };
        Pending older, newer;                          // of steps g - 2 and g - 1
        older.flags = newer.flags = 0;

        // takes the elements that are not finite out of rows [a, b) of a value tile; all lanes
        constexpr int CH = C::PANELS * 8, RPI = 32 / CH;   // 16-byte chunks of a row, rows a warp handles at once
        const int my_row = lane / CH, my_off = ((lane % CH) >> 3) * kPanel + (lane & 7) * 16;
        auto zero_rows = [&](unsigned char* v, int a, int b) {
            for (int r = a + my_row; r < b; r += RPI)
                *reinterpret_cast<uint4*>(v + my_off + r * 128) = make_uint4(0, 0, 0, 0);
        };
        auto finite_rows = [&](unsigned char* v, int a, int b) -> int {
            int odd = 0;
#pragma unroll 4
            for (int r = a + my_row; r < b; r += RPI) {
                uint4* p = reinterpret_cast<uint4*>(v + my_off + r * 128);
                uint4 x = *p;
                uint32_t* u = reinterpret_cast<uint32_t*>(&x);
                int found = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if ((u[i] & 0x7f80u) == 0x7f80u) { u[i] &= 0xffff0000u; found = 1; }
                    if ((u[i] & 0x7f800000u) == 0x7f800000u) { u[i] &= 0x0000ffffu; found = 1; }
                }
                if (found) { *p = x; odd = 1; }
            }
            return odd;
        };
        // values that must not meet a zero weight (see the header).  Pages that hold no
        // key below kend were filled with zeros by the copy
        auto clean = [&](unsigned char* v, const Pending& pv) {
            const int k0 = pv.tile << kKeysLog2;
            const Sight& si = pv.si;
            if (k0 >= si.all_lo && k0 + kKeys <= si.all_hi) return;
            const int page = 1 << s.page_log2;
            auto in = [&](int key) { return min(max(key - k0, 0), kKeys); };
            const int filled = in((pv.kend + page - 1) & ~(page - 1));
            zero_rows(v, 0, in(si.lo));
            zero_rows(v, in(si.hi), filled);
            const int mid = min(si.all_lo, si.hi);
            int odd = finite_rows(v, in(si.lo), in(mid));
            odd |= finite_rows(v, in(max(si.all_hi, mid)), in(si.hi));
            if (odd) tl.odd_values[pv.slot] = 1;
            kda::fence_proxy_async_smem();
            __syncwarp();
        };
        // the values of a step are there and clean
        auto take_values = [&](const Pending& pv) -> bool {
            if (!(pv.flags & kFirstUse)) return true;
            v_stage = pv.v_at;
            if (!wait(&tl.kv_full[v_stage], pv.v_ring)) return false;
            clean(sm + C::KV0 + v_stage * C::TILE, pv);
            return true;
        };
        auto take_weights = [&](int h) -> bool {
            if (!wait(&tl.p_full[h], (p_phase >> h) & 1)) return false;
            p_phase ^= 1u << h;
            return true;
        };
        auto issue_values = [&](int h, int flags) {    // O_h += P_h V; one lane
            const uint64_t b = v_desc + kda::desc_step(v_stage * C::TILE);
            const uint32_t d = tmem + C::TMEM_O + h * D, a = tmem + h * 128;
#pragma unroll
            for (int i = 0; i < kKeys / 16; ++i)
                umma_bf16_ta(d, a + 8 * i, b + kda::desc_step(i * 2048), id_o, (i > 0 || (flags & kAdd)) ? 1u : 0u);
            if (flags & kLastUse) kda::umma_commit(&tl.kv_empty[v_stage]);
            if (flags & kFinal) kda::umma_commit(&tl.o_full[h]);
        };
        auto issue_scores = [&](int h, int tile, int flags) {        // S_h = Q_tile K^T; one lane
            const uint64_t a = q_desc + kda::desc_step(tile * C::TILE), b = k_desc + kda::desc_step(k_stage * C::TILE);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const uint64_t at = kda::desc_step((i >> 2) * kPanel + (i & 3) * 32);
                kda::umma_bf16(tmem + h * 128, a + at, b + at, id_s, i > 0 ? 1u : 0u);
            }
            kda::umma_commit(&tl.s_full[h]);
            if (flags & kLastUse) kda::umma_commit(&tl.kv_empty[k_stage]);
            if (flags & kFinal) kda::umma_commit(&tl.q_empty);
        };
        auto values_step = [&](int h, const Pending& pv) -> bool {
            if (!take_values(pv) || !take_weights(h)) return false;
            kda::tc_fence_after();
            if (elect_one()) issue_values(h, pv.flags);
            __syncwarp();
            return true;
        };
        bool ok = true;
        for (int k = 0; ok; ++k) {
            Unit u;
            if (!read_unit(k, u)) break;
            const int two = uniform(u.ntok > BT), tiles = uniform(u.te - u.tb), steps = tiles << two, tb = uniform(u.tb);
            const Sight si = sight(u, s.window, 0, u.ntok - 1);
            int v_at = 0;                              // stage of the current tile's values, its parity
            uint32_t v_ring = 0;
            auto due_after = [&](int t) {              // the second product of step t
                Pending pv;
                pv.v_at = v_at;
                pv.v_ring = v_ring;
                const int lone = !two || (t & 1);
                pv.flags = kDue | (!two || !(t & 1) ? kFirstUse : 0) | (lone ? kLastUse : 0) | (t >= 2 ? kAdd : 0) |
                           (t >= steps - 2 ? kFinal : 0);
                pv.tile = tb + (t >> two);
                pv.slot = k & 3;
                pv.kend = u.kend;
                pv.si = si;
                return pv;
            };
            if (lane == 0) tl.odd_values[k & 3] = 0;
            // a unit of two row tiles past its first key tile goes through the loop below this one
            const int slow = two ? 2 : steps;
            for (int t = 0; t < slow; ++t, ++g) {
                const int h = g & 1;
                if (older.flags & kDue) ok = values_step(h, older);
                if (ok && (!two || t == 0)) ok = take_keys(v_at, v_ring);
                if (ok && t == 0) ok = wait(&tl.q_full, k & 1);
                if (!ok) break;
                kda::tc_fence_after();
                if (elect_one())
                    issue_scores(h, two & t, (!two || t == 1 ? kLastUse : 0) | (t == steps - 1 ? kFinal : 0));
                __syncwarp();
                issued = true;
                older = newer;
                newer = due_after(t);
            }
            if (!ok || slow == steps) continue;
            // the tensor cores' time is here: as few instructions between products as can be
            const int h0 = g & 1, h1 = h0 ^ 1;
            Pending pv = older;                        // values of the tile before
            for (int j = 1; j < tiles; ++j) {
                pv.tile = tb + j - 1;
                pv.flags = kDue | kFirstUse;
                pv.v_at = v_at;
                pv.v_ring = v_ring;
                ok = take_values(pv) && take_weights(h0);
                if (!ok) break;
                kda::tc_fence_after();
                const int add = j > 1 ? kAdd : 0;
                if (elect_one()) issue_values(h0, add);
                ok = take_keys(v_at, v_ring);
                if (!ok) break;
                if (elect_one()) issue_scores(h0, 0, 0);
                ok = take_weights(h1);
                if (!ok) break;
                kda::tc_fence_after();
                if (elect_one()) {
                    issue_values(h1, add | kLastUse);
                    issue_scores(h1, 1, kLastUse | (j == tiles - 1 ? kFinal : 0));
                }
            }
            __syncwarp();
            g += steps - 2;
            older = due_after(steps - 2);
            newer = due_after(steps - 1);
        }
        if (ok && (older.flags & kDue)) ok = values_step(g & 1, older);
        if (ok && (newer.flags & kDue)) ok = values_step((g + 1) & 1, newer);
        if (issued) {                                  // no product in flight when TMEM is freed
            if (elect_one()) kda::umma_commit(&tl.drain);
            __syncwarp();
            (void)kda::mbar_wait(&tl.drain, 0, kda::kWaitCycles);
        }
    } else if (w < 8) {
        // ---------------- softmax and output of half h
        const int h = w >> 2, row = tid & 127;
        const uint32_t lane_off = (uint32_t)((w & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + h * 128;
        const int rows_tile = BT * s.Gv;
        const int tok_in = row / s.Gv, head_in = row % s.Gv;
        const int pieces = s.page_log2 >= kKeysLog2 ? 1 : kKeys >> s.page_log2;
        const int piece_log2 = min(s.page_log2, kKeysLog2);
        int n_s = 0, n_j = 0, g = 0;
        uint32_t o_phase = 0;                          // bit h: parity of the next O_h
        bool ok = true;
        for (int k = 0; ok; ++k) {
            Unit u;
            if (!read_unit(k, u)) break;
            const bool two = u.ntok > BT;
            const int steps = (u.te - u.tb) << (two ? 1 : 0);
            const int t0 = (h ^ g) & 1;                // this half's first step
            const int qi = two ? t0 : 0;               // its row tile
            const int tok = qi * BT + tok_in;
            const bool valid = row < rows_tile && tok < u.ntok;
            const int pos = u.pos + tok;
            const int hi = valid ? min(max(pos + 1, 0), u.kend) : 0;
            const int lo = valid ? kda_paged::first_key(pos, s.window) : 0;
            const bool busy = __any_sync(0xffffffffu, valid);
            const Sight mine = sight(u, s.window, qi * BT, min(u.ntok, qi * BT + BT) - 1);
            auto page_of = [&](int tile) {             // lane's page of the tile: 0 where there is nothing to judge
                const int key = (tile << kKeysLog2) + (lane << piece_log2);
                return lane < pieces && key < u.kend ? table[(size_t)u.n * s.blocks + (key >> s.page_log2)] : 0;
            };
            float m = -INFINITY, l = 0.f;
            int page = busy && t0 < steps ? page_of(u.tb + (two ? 0 : t0)) : 0;
            for (int t = t0; t < steps; t += 2) {
                const int tile = u.tb + (two ? t >> 1 : t), k0 = tile << kKeysLog2;
                const unsigned missing = __ballot_sync(0xffffffffu, page < 0 || page >= s.n_pages);
                if (busy && t + 2 < steps) page = page_of(tile + (two ? 1 : 2));
                if (!wait(&tl.s_full[h], n_s & 1)) { ok = false; break; }
                ++n_s;
                kda::tc_fence_after();
                if (busy) {
                    if (k0 < mine.all_lo || k0 + kKeys > mine.all_hi || missing) {
                        // scores of keys this row does not see become -inf, in place.  Rolled: these
                        // tiles are few, and a short call's time goes into fetching instructions
#pragma unroll 1
                        for (int c = 0; c < kKeys; c += 32) {
                            const int a = max(lo - k0 - c, 0), b = hi - k0 - c;
                            uint32_t seen = a >= 32 || b <= a ? 0u : 0xffffffffu << a;
                            if (b < 32) seen &= (1u << max(b, 0)) - 1u;
                            if ((missing >> (c >> piece_log2)) & 1) seen &= piece_log2 == 4 ? 0xffff0000u : 0u;
                            if (piece_log2 == 4 && ((missing >> ((c >> 4) + 1)) & 1)) seen &= 0x0000ffffu;
                            float y[32];
                            kda::tmem_ld32(tS + c, y);
                            kda::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) y[e] = (seen >> e) & 1 ? y[e] : -INFINITY;
                            tmem_st32(tS + c, reinterpret_cast<const uint32_t*>(y));
                        }
                        kda::tmem_wait_st();
                    }
                    float x[128];
#pragma unroll
                    for (int c = 0; c < 128; c += 32) kda::tmem_ld32(tS + c, x + c);
                    kda::tmem_wait_ld();
                    float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int c = 4; c < 128; c += 4)
#pragma unroll
                        for (int e = 0; e < 4; ++e) top[e] = fmaxf(top[e], x[c + e]);
                    const float big = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    if (t < 2) {
                        m = big;
                    } else {
                        // S complete means that this half's product before it is too, so O stands still
                        const bool grow = (big - m) * scale_log2 > kGrow;
                        if (__any_sync(0xffffffffu, grow)) {
                            const float f = grow ? ex2((m - big) * scale_log2) : 1.f;
                            const uint32_t tO = tmem + lane_off + C::TMEM_O + h * D;
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
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
                    const float ref = m == -INFINITY ? 0.f : m * scale_log2;
                    const uint64_t sc2 = pack2(scale_log2, scale_log2), off2 = pack2(-ref, -ref);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int c0 = 0; c0 < 128; c0 += 64) {
                        uint32_t p[32];
#pragma unroll
                        for (int c = 0; c < 64; c += 2) {
                            float a, b;
                            unpack2(fma2(pack2(x[c0 + c], x[c0 + c + 1]), sc2, off2), a, b);
                            a = ex2(a);
                            b = ex2(b);
                            sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pack2(a, b));
                            p[c >> 1] = kda::pack_bf16x2(a, b);
                        }
                        tmem_st32(tS + c0 / 2, p);
                    }
                    float sa, sb;
                    unpack2(add2(sum[0], sum[1]), sa, sb);
                    l += sa + sb;
                    kda::tmem_wait_st();
                }
                kda::tc_fence_before();
                __syncwarp();
                if (lane == 0) kda::mbar_arrive(&tl.p_full[h]);
            }
            if (!ok) break;
            // ---- output
            const bool whole = u.first && u.last;
            const int which = u.first ? 1 : 0;
            const size_t at = (size_t)(u.tok0 + tok) * s.Hq + u.qh0 + head_in;
            const int prow = qi * rows_tile + row;     // row of a partial slot
            const Sight un = sight(u, s.window, 0, u.ntok - 1);
            float ref = m == -INFINITY ? -INFINITY : m * scale_log2;
            // writes 32 columns of this row: o, or unnormalised sums
            auto put = [&](float* y, int c0, float sum_l) {
                if (tl.odd_values[k & 3] && valid) add_odd_values<D>(y, c0, u, un, lo, hi, s, vc, table);
                if (!valid) return;
                if (whole) {
                    const float inv = sum_l == 0.f ? 0.f : 1.f / sum_l;
                    uint4* dst = reinterpret_cast<uint4*>(o + at * D + c0);
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        dst[e / 8] = make_uint4(kda::pack_bf16x2(y[e] * inv, y[e + 1] * inv),
                                                kda::pack_bf16x2(y[e + 2] * inv, y[e + 3] * inv),
                                                kda::pack_bf16x2(y[e + 4] * inv, y[e + 5] * inv),
                                                kda::pack_bf16x2(y[e + 6] * inv, y[e + 7] * inv));
                } else {
                    float4* dst = reinterpret_cast<float4*>(parts.sums(blockIdx.x, which) + (size_t)prow * D + c0);
#pragma unroll
                    for (int e = 0; e < 32; e += 4) dst[e / 4] = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                }
            };
            auto put_stats = [&](float r, float sum_l) {
                if (!valid) return;
                if (whole) {
                    if (lse) lse[at] = sum_l == 0.f ? -INFINITY : (r + log2f(sum_l)) * kLn2;
                } else {
                    parts.stats(blockIdx.x, which)[prow] = make_float2(r, sum_l);
                }
            };
            if (two) {
                ok = wait(&tl.o_full[h], (o_phase >> h) & 1);
                o_phase ^= 3;
                if (!ok) break;
                kda::tc_fence_after();
                if (busy) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float y[32];
                        kda::tmem_ld32(tmem + lane_off + C::TMEM_O + h * D + c, y);
                        kda::tmem_wait_ld();
                        put(y, c, l);
                    }
                    put_stats(ref, l);
                }
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
                kda::tc_fence_after();
                constexpr int kShare = D / 2 < 32 ? 32 : D / 2;      // columns that a half writes
                if (busy) {
                    const float2 st = tl.stats[h ^ 1][row];
                    const float top = fmaxf(ref, st.x), base = top == -INFINITY ? 0.f : top;
                    const float fm = l == 0.f ? 0.f : ex2(ref - base), fo = st.y == 0.f ? 0.f : ex2(st.x - base);
                    const float f0 = h == 0 ? fm : fo, f1 = h == 0 ? fo : fm;
                    const float sum_l = fmaf(fm, l, fo * st.y);
#pragma unroll 1
                    for (int c = h * kShare; c < min((h + 1) * kShare, D); c += 32) {
                        float y[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) y[e] = 0.f;
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            if (!has[b]) continue;
                            float z[32];
                            kda::tmem_ld32(tmem + lane_off + C::TMEM_O + b * D + c, z);
                            kda::tmem_wait_ld();
                            const float f = b == 0 ? f0 : f1;
                            if (f != 0.f) {
#pragma unroll
                                for (int e = 0; e < 32; ++e) y[e] = fmaf(f, z[e], y[e]);
                            }
                        }
                        put(y, c, sum_l);
                    }
                    if (h == 0) put_stats(top, sum_l);
                }
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
    if (*abort_f && w == kCopyWarp) {                  // no copy in flight into shared memory that is given up
        for (int i = max(0, n_ld - C::STAGES); i < n_ld; ++i)
            (void)kda::mbar_wait(&tl.kv_full[i % C::STAGES], (i / C::STAGES) & 1, kda::kWaitCycles);
        if (n_q > 0) (void)kda::mbar_wait(&tl.q_full, (n_q - 1) & 1, kda::kWaitCycles);
    }
    __syncthreads();
    if (w == kIssueWarp) kda::tmem_dealloc(tmem, 512);
}

// ---- host
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        else
            (void)cudaGetLastError();
    });
    return fn;
}

// q [T, Hq, d] with `stride` elements between tokens: boxes of 64 channels x Gv heads x BT tokens.
bool make_q_map(CUtensorMap* m, const kda_host::PagedArgs& a, int Gv, int BT) {
    const cuuint64_t dims[3] = {(cuuint64_t)a.d, (cuuint64_t)a.Hq, (cuuint64_t)a.T};
    const cuuint64_t strides[2] = {(cuuint64_t)a.d * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)Gv, (cuuint32_t)BT};
    const cuuint32_t one[3] = {1, 1, 1};
    return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, one,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A cache [n_pages, Hkv, page, d]: boxes of 64 channels x up to 128 tokens of one head and page.
bool make_cache_map(CUtensorMap* m, const void* base, const kda_host::PagedArgs& a) {
    const cuuint64_t row = (cuuint64_t)a.d * 2;
    const cuuint64_t dims[4] = {(cuuint64_t)a.d, (cuuint64_t)a.page_size, (cuuint64_t)a.Hkv, (cuuint64_t)a.n_pages};
    const cuuint64_t strides[3] = {row, row * a.page_size, row * a.page_size * a.Hkv};
    const cuuint32_t box[4] = {64, (cuuint32_t)std::min(a.page_size, kKeys), 1, 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, one,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_tc(const kda_host::PagedArgs& a) {
    const kda_host::PagedPlan p = kda_host::paged_plan_tc(a.T, a.Hq, a.Hkv);
    if (!tensor_map_encoder()) return cudaErrorNotSupported;
    CUtensorMap qm, km, vm;
    const int BT = 128 / p.Gv;
    if (!make_q_map(&qm, a, p.Gv, BT) || !make_cache_map(&km, a.k_cache, a) || !make_cache_map(&vm, a.v_cache, a))
        return cudaErrorInvalidValue;
    auto kern = kda_paged_attention_tc_kernel<D>;
    static kda_host::OncePerDevice once;
    const cudaError_t e = once.run([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
    });
    if (e != cudaSuccess) return e;
    const int ctas = std::min(p.max_ctas, kda_host::sm_count());
    kern<<<ctas, kThreads, Cfg<D>::SMEM, a.stream>>>(
        qm, km, vm, static_cast<const __nv_bfloat16*>(a.v_cache), a.block_table, a.cu_seqlens, a.seq_len,
        kda_host::paged_shape(a, p), BT, a.scale * kLog2e, static_cast<__nv_bfloat16*>(a.o), a.lse,
        kda_host::paged_partials(a, p), a.status);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    return kda_host::launch_paged_merge(a, p, ctas);
}

}  // namespace

namespace kda_host {

bool paged_tc_supported(int d, kda_dtype dt) { return dt == KDA_BF16 && (d == 32 || d == 64 || d == 128); }

PagedPlan paged_plan_tc(int T, int Hq, int Hkv) {
    PagedPlan p;
    p.Gv = heads_per_unit(Hq / Hkv, 128);
    p.U = 2 * (128 / p.Gv);
    p.rows = paged_slot_rows(p.U, T, p.Gv);
    p.tile_log2 = kKeysLog2;
    p.max_ctas = 160;
    p.extra = 3;
    return p;
}

cudaError_t launch_paged_attention_tc(const PagedArgs& a) {
    return a.d == 128 ? launch_tc<128>(a) : a.d == 64 ? launch_tc<64>(a) : launch_tc<32>(a);
}

}  // namespace kda_host
