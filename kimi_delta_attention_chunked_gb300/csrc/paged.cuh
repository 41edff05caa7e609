// paged.cuh -- what the operators of a serving step share: the checked view of
// a step's lengths, and the division of paged attention's work over the grid.
//
// Attention work comes in units: up to U new tokens of one request, with the
// Gv query heads that share a cache head, against the 128- or 64-key tiles that
// any of their rows sees.  The tiles of all units, in the order request, head,
// unit, tile, are one line, and CTA c of C takes the c-th of C equal pieces of
// it: every CTA has the same number of places whatever the lengths are.  A place is a key
// tile, though, and on the tensor cores a unit of two row tiles takes two steps for it, one of
// a single row tile one: in batches that mix the two the pieces differ in work (16 requests
// of 1 to 513 tokens under a window of 1024: 20 steps in the busiest CTA, 9.2 on average,
// 12 with no places for the fixed cost).  Before a unit's
// tiles the line has `extra` places that stand for its fixed cost (the pipeline
// drains and the output is written, 2 to 5 us).  On the tensor cores, with 0, 1, 2,
// 3, 4 and 6 of them: 64 decode requests 252, 243, 237, 235, 236 and 238 us (the CTAs of
// the short requests, with the most units, finished last), 32 x 8 tokens 57, 54, 53,
// 52, 52 and 52 us.  On the CUDA cores, whose tiles take longer, 0 is best.
// A unit that a border cuts is finished by each of its CTAs into fp32 partial
// rows, which the merge kernel joins.  A CTA finds its piece itself, from the lengths
// on the device: no plan is made on the host, and no extra launch is needed.
#pragma once

#include <float.h>

#include <atomic>

#include "common.cuh"

namespace kda_paged {

constexpr int kMaxRequests = KDA_MAX_STEP_REQUESTS;

// The kernels before this one on the stream are complete and their writes seen;
// the kernel behind it may be set up from here on.
__device__ __forceinline__ void wait_for_stream() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Sizes of one attention call.
struct Shape {
    int n_req, T;                                  // requests, rows of q
    int Hq, Hkv, Hv, Gv, sub;                      // Hv = Hkv * sub groups of Gv query heads
    int blocks, page_log2, n_pages, window;
    int U, tile_log2;                              // tokens per unit, keys per tile
    int extra;                                     // places on the line before a unit's tiles
};

// The same over packed keys: those of request n lie at rows cu_k[n] .. cu_k[n + 1] - 1 of [S, ...]
// tensors, without pages.  Where the lengths of a paged call come as cu and seq_len, those of a
// packed one come as cu and cu_k.
struct PackedShape : Shape {
    int S;                                         // rows of the keys
    int causal;                                    // 0: every row sees all keys of its request
    // Units of more than half_unit tokens take two steps a tile, and so two places, with extra_two ahead of them
    // (half_unit = U: there are none).
    int half_unit, extra_two;
};

// One request's lengths, inside the buffers whatever the device arrays hold.
struct Req {
    int tok0, len;                                 // first row of q, new tokens
    int pos0;                                      // position of the first new token (may be negative)
    int kend;                                      // keys below it exist; at most KDA_MAX_STEP_POSITIONS, so
                                                   // that the end of its tile is still a 32-bit number
};

__device__ __forceinline__ Req load_req(const Shape& s, const int32_t* __restrict__ cu,
                                        const int32_t* __restrict__ seq_len, int n) {
    Req r;
    r.tok0 = min(max(cu[n], 0), s.T);
    const int end = min(max(cu[n + 1], r.tok0), s.T);
    r.len = end - r.tok0;
    const int seq = max(seq_len[n], 0);
    r.pos0 = seq - r.len;
    const long long cap = (long long)s.blocks << s.page_log2;
    r.kend = (int)min((long long)seq, cap);
    return r;
}

__device__ __forceinline__ Req load_req(const PackedShape& s, const int32_t* __restrict__ cu,
                                        const int32_t* __restrict__ cu_k, int n) {
    Req r;
    r.tok0 = min(max(cu[n], 0), s.T);
    const int end = min(max(cu[n + 1], r.tok0), s.T);
    r.len = end - r.tok0;
    const int key0 = min(max(cu_k[n], 0), s.S);
    r.kend = min(max(cu_k[n + 1], key0), s.S) - key0;
    r.pos0 = s.causal ? r.kend - r.len : r.kend;   // at kend and behind it, a row sees every key
    return r;
}

// First key that a row at `pos` (negative: before the sequence) sees.  No difference is formed
// that could pass 32 bits: any window from 0 to 2^31 - 1 may meet any position, and a first key
// that wraps below 0 would name a place before the block table.
__host__ __device__ __forceinline__ int first_key(int pos, int window) {
    return window > 0 && pos >= window ? pos - window + 1 : 0;
}

__device__ __forceinline__ int n_units(const Shape& s, const Req& r) { return (r.len + s.U - 1) / s.U; }

// log2 of the places of a tile of unit i, and the places before its tiles.
__device__ __forceinline__ int unit_shift(const Shape&, const Req&, int) { return 0; }
__device__ __forceinline__ int unit_shift(const PackedShape& s, const Req& r, int i) {
    return min(s.U, r.len - i * s.U) > s.half_unit ? 1 : 0;
}
// CTAs that may have a piece.  Where a tile may have two places, a piece has two at least, so that one that lies
// among a unit's tiles holds the first place of one of them.
__device__ __forceinline__ unsigned long long most_pieces(const Shape&, unsigned long long total) { return total; }
__device__ __forceinline__ unsigned long long most_pieces(const PackedShape& s, unsigned long long total) {
    return total > 1 && s.half_unit < s.U ? total >> 1 : total;
}
__device__ __forceinline__ int unit_extra(const Shape& s, int) { return s.extra; }
__device__ __forceinline__ int unit_extra(const PackedShape& s, int shift) { return shift ? s.extra_two : s.extra; }

// Tiles [tb, te) of unit i: those that hold a key some row sees, and one tile
// where no row sees any (its rows are written as empty).
__device__ __forceinline__ void unit_span(const Shape& s, const Req& r, int i, int& tb, int& te) {
    const int first = i * s.U, last = min(r.len, first + s.U);
    const int hi = min(max(r.pos0 + last, 0), r.kend);
    const int lo = min(first_key(r.pos0 + first, s.window), hi);
    tb = lo >> s.tile_log2;
    te = (hi + (1 << s.tile_log2) - 1) >> s.tile_log2;
    if (te <= tb) te = tb + 1;
}

// Places of unit i.
template <class Sh>
__device__ __forceinline__ unsigned unit_places(const Sh& s, const Req& r, int i) {
    int tb, te;
    unit_span(s, r, i, tb, te);
    const int shift = unit_shift(s, r, i);
    return (unsigned)(te - tb << shift) + (unsigned)unit_extra(s, shift);
}

// Length of all units of a request, for one head.  A thread counts a request of
// few units by itself; the lanes of a warp share out one of many.
template <class Sh>
__device__ __forceinline__ unsigned long long request_places(const Sh& s, const Req& r) {
    constexpr int kAlone = 8;
    const int units = n_units(s, r);
    unsigned long long cost = 0;
    if (units <= kAlone) {
        for (int i = 0; i < units; ++i) cost += unit_places(s, r, i);
    }
    unsigned many = __ballot_sync(0xffffffffu, units > kAlone);
    while (many) {
        const int src = __ffs(many) - 1;
        many &= many - 1;
        Req q;
        q.tok0 = 0;
        q.len = __shfl_sync(0xffffffffu, r.len, src);
        q.pos0 = __shfl_sync(0xffffffffu, r.pos0, src);
        q.kend = __shfl_sync(0xffffffffu, r.kend, src);
        const int total = n_units(s, q);
        unsigned long long part = 0;
        for (int i = threadIdx.x & 31; i < total; i += 32) part += unit_places(s, q, i);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        if ((int)(threadIdx.x & 31) == src) cost = part;
    }
    return cost;
}

// Where a CTA's piece begins and ends on the line of tiles.
struct Piece {
    unsigned long long begin, end, total;          // places [begin, end) of `total`
    unsigned long long off;                        // begin - first place of request n
    unsigned long long len;                        // length of request n for one head
    int n, ctas;                                   // first request; CTAs that have a piece
    int known;                                     // its lengths are in r
    Req r;
};

// Finds the piece of CTA `c` of `C`.  Every thread of the block (NT of them)
// calls it; `cost` holds n_req words and `red` NT / 32, of 64 bits, and free again after the block's next barrier.
template <int NT, class Sh>
__device__ __forceinline__ Piece find_piece(const Sh& s, const int32_t* __restrict__ cu,
                                            const int32_t* __restrict__ seq_len, int c, int C,
                                            unsigned long long* cost,
                                            unsigned long long* red, Piece* shared) {
    constexpr int NW = NT / 32;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    Req r{0, 0, 0, 0};
    for (int base = 0; base < s.n_req; base += NT) {
        const int n = base + tid;
        r = Req{0, 0, 0, 0};
        if (n < s.n_req) r = load_req(s, cu, seq_len, n);
        const unsigned long long x = request_places(s, r);
        if (n < s.n_req) cost[n] = x;
    }
    if (tid == 0) *shared = Piece{};
    __syncthreads();
    // each thread takes `per` consecutive requests of the running sum
    const int per = (s.n_req + NT - 1) / NT, n0 = min(tid * per, s.n_req), n1 = min(n0 + per, s.n_req);
    unsigned long long mine = 0;
    for (int n = n0; n < n1; ++n) mine += cost[n];
    mine *= (unsigned)s.Hv;
    unsigned long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) red[w] = incl;
    __syncthreads();
    unsigned long long before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const unsigned long long t = red[i];
        if (i < w) before += t;
        total += t;
    }
    incl += before;
    const int ctas = (int)min((unsigned long long)C, most_pieces(s, total));
    if (c < ctas) {
        const unsigned long long begin = total * (unsigned)c / (unsigned)ctas;
        const unsigned long long excl = incl - mine;
        if (excl <= begin && begin < incl) {
            unsigned long long at = excl;
            int n = n0;
            for (; n < n1; ++n) {
                const unsigned long long x = cost[n] * (unsigned)s.Hv;
                if (begin < at + x) break;
                at += x;
            }
            shared->begin = begin;
            shared->end = total * (unsigned)(c + 1) / (unsigned)ctas;
            shared->total = total;
            shared->off = begin - at;
            shared->len = cost[n];
            shared->n = n;
            shared->ctas = ctas;
            shared->known = s.n_req <= NT;             // a thread has one request, this one this
            shared->r = r;
        }
    }
    __syncthreads();
    return *shared;
}

// The same by one warp alone, for up to kWarpRequests requests: fewer instructions and no barrier of the block,
// so the other warps go on to their parts meanwhile.  `cost` holds n_req words of shared memory.
constexpr int kWarpRequests = 512;
template <class Sh>
__device__ __forceinline__ Piece find_piece_warp(const Sh& s, const int32_t* __restrict__ cu,
                                                 const int32_t* __restrict__ seq_len, int c, int C, unsigned long long* cost) {
    const int lane = threadIdx.x & 31;
    Piece p{};
    unsigned long long total = 0;
#pragma unroll 1
    for (int base = 0; base < s.n_req; base += 32) {
        p.r = Req{0, 0, 0, 0};
        if (base + lane < s.n_req) p.r = load_req(s, cu, seq_len, base + lane);
        const unsigned long long x = request_places(s, p.r);
        if (base + lane < s.n_req) cost[base + lane] = x;
        total += x;
    }
    __syncwarp();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    p.total = total * (unsigned)s.Hv;
    p.ctas = (int)min((unsigned long long)C, most_pieces(s, p.total));
    if (c >= p.ctas) return p;
    p.begin = p.total * (unsigned)c / (unsigned)p.ctas;
    p.end = p.total * (unsigned)(c + 1) / (unsigned)p.ctas;
    p.off = p.begin;
#pragma unroll 1
    for (int base = 0; base < s.n_req; base += 32) {
        const unsigned long long x = base + lane < s.n_req ? cost[base + lane] : 0;
        unsigned long long incl = x * (unsigned)s.Hv;
        const unsigned long long mine = incl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, p.off < incl);
        if (hit) {
            const int src = __ffs((int)hit) - 1;
            p.off -= __shfl_sync(0xffffffffu, incl - mine, src);
            p.len = __shfl_sync(0xffffffffu, x, src);
            p.n = base + src;
            p.known = s.n_req <= 32;                   // a lane has one request
            p.r.tok0 = __shfl_sync(0xffffffffu, p.r.tok0, src);
            p.r.len = __shfl_sync(0xffffffffu, p.r.len, src);
            p.r.pos0 = __shfl_sync(0xffffffffu, p.r.pos0, src);
            p.r.kend = __shfl_sync(0xffffffffu, p.r.kend, src);
            return p;
        }
        p.off -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return p;
}

// Large scores.  A row's reference is its largest score m times c = scale log2(e), rounded, and on the tensor-core
// paths a weight is 2^(c x - reference) in one fused step: the reference's rounding enters all of them alike and the
// sum takes it out again, while it is no more than some octaves (|m c| < 2^29).  From there on the reference is moved up,
// so that weights end at 0 and not at infinity, and the row, or the part of it, has a reference above -inf and no sum:
// it does not pass for one that sees no key (-inf, 0), weighs nothing beside a part that is in range, and is NaN where
// it is the largest.  (2^(c (x - m)) would give such rows their values; it took the expanded prompt from 424 to 435 us.)
constexpr float kMostOctaves = 0x1p29f;
__device__ __forceinline__ float reference(float m, float c) {
    const float r = fmaxf(m * c, -FLT_MAX);
    return fabsf(r) < kMostOctaves ? r : fmaf(fabsf(r), 0x1p-22f, r);
}
// (reference, sum of weights) of a row or a part of it, from its largest score and what its weights came to.  On CUDA
// cores, where the difference of the scores is formed first, `most` is the range of fp32.
__device__ __forceinline__ float2 row_stats(float m, float l, float c, float most = kMostOctaves) {
    if (m == -INFINITY) return make_float2(-INFINITY, l);
    const float r = m * c;
    if (fabsf(r) >= most && !isinf(m) && l == l) l = 0.f;
    return make_float2(fmaxf(r, -FLT_MAX), l);
}
// The sum to divide by: 0 for a row that sees no key.
__device__ __forceinline__ float whole_sum(float top, float l) { return l == 0.f && top > -INFINITY ? NAN : l; }

// A cut unit of more rows than this is joined by the blocks of all its CTAs (if they are many).
constexpr int kSpreadRows = 64;

// One unit, or the part of it that a CTA's piece holds.
struct Unit {
    int n, kvh, qh0;                               // request, cache head, first query head
    int tok0, ntok;                                // rows of q: tokens tok0 .. tok0 + ntok - 1
    int pos, kend;                                 // position of token tok0; keys below kend exist
    int tb, te;                                    // tiles of this part
    int first, last;                               // the part holds the unit's first / last tile
    int start, parts;                              // CTA in which the unit begins (-1: not asked for), CTAs that share it
};

// Walks the units of a CTA's piece.  Used by all lanes of one warp together.
struct Walker {
    unsigned long long at, end, total;
    int ctas, c;
    int n, h, i, in;                               // next unit; places of it that lie before the piece
    int ahead, last_place;                         // of the unit whose part was handed out last: places before its
                                                   // tiles, place of its last tile
    Req r;
    int units;

    template <class Sh>
    __device__ __forceinline__ void start(const Sh& s, const int32_t* cu, const int32_t* seq_len, const Piece& p,
                                          int cta) {
        c = cta;
        at = p.begin;
        end = p.end;
        total = p.total;
        ctas = p.ctas;
        n = p.n;
        if (at >= end) return;
        r = p.known ? p.r : load_req(s, cu, seq_len, n);
        first_unit(s, p.off, p.len);
    }

    // Head, unit and place that lie `off` places behind the start of request n, whose heads have `len` each.
    template <class Sh>
    __device__ __forceinline__ void first_unit(const Sh& s, unsigned long long off, unsigned long long len) {
        units = n_units(s, r);
        h = s.Hv == 1 ? 0 : (int)(off / len);
        unsigned long long left = off - (unsigned long long)h * len;
        i = 0;
        in = (int)left;
        if (units <= 1) return;
        const int lane = threadIdx.x & 31;
#pragma unroll 1
        for (int base = 0; base < units; base += 32) {
            unsigned x = 0;
            if (base + lane < units) x = unit_places(s, r, base + lane);
            unsigned incl = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned t = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += t;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, left < incl);
            if (hit) {
                const int src = __ffs((int)hit) - 1;
                i = base + src;
                in = (int)(left - __shfl_sync(0xffffffffu, incl - x, src));
                return;
            }
            left -= __shfl_sync(0xffffffffu, incl, 31);
        }
    }

    // The next part, or false at the end of the piece.
    template <class Sh>
    __device__ __forceinline__ bool next(const Sh& s, const int32_t* cu, const int32_t* seq_len, Unit& u) {
        unsigned long long from;
        const bool more = step(s, cu, seq_len, u, from);
        if (more) share(s, u, from);
        return more;
    }

    // The same without the CTAs that share the unit (share() adds them: divisions that a kernel may put off
    // until it has handed the part on).  `from` is the unit's first place on the line.
    template <class Sh>
    __device__ __forceinline__ bool step(const Sh& s, const int32_t* cu, const int32_t* seq_len, Unit& u,
                                         unsigned long long& from) {
        while (at < end) {
            while (i >= units) {
                i = 0;
                if (units == 0 || ++h >= s.Hv) {
                    h = 0;
                    if (++n >= s.n_req) return false;
                    r = load_req(s, cu, seq_len, n);
                    units = n_units(s, r);
                }
            }
            int tb, te;
            unit_span(s, r, i, tb, te);
            const int shift = unit_shift(s, r, i);
            ahead = unit_extra(s, shift);
            last_place = ahead + (te - tb - 1 << shift);
            const int len = ahead + (te - tb << shift);
            const int take = (int)min((unsigned long long)(len - in), end - at);
            // tiles of this part: those whose first place is in it
            const int t0 = max(in - ahead, 0) + (1 << shift) - 1 >> shift;
            const int t1 = max(in + take - ahead, 0) + (1 << shift) - 1 >> shift;
            from = at - (unsigned)in;
            u.n = n;
            u.kvh = h / s.sub;
            u.qh0 = h * s.Gv;
            u.tok0 = r.tok0 + i * s.U;
            u.ntok = min(s.U, r.len - i * s.U);
            u.pos = r.pos0 + i * s.U;
            u.kend = r.kend;
            u.tb = tb + t0;
            u.te = tb + t1;
            u.first = t0 == 0;
            u.last = u.te == te;
            at += (unsigned)take;
            in = 0;
            ++i;
            if (t1 > t0) return true;
        }
        return false;
    }

    // CTA c begins at total * c / ctas, so the one that has place x is ceil((x + 1) * ctas / total) - 1.  Where a unit that goes on here begins is asked for if it has more than `spread` rows.
    template <class Sh>
    __device__ __forceinline__ void share(const Sh& s, Unit& u, unsigned long long from, int spread = kSpreadRows) const {
        u.start = c;
        u.parts = 1;
        if (!u.first) {
            u.start = -1;
            if (u.ntok * s.Gv > spread)
                u.start = (int)(((from + (unsigned)ahead + 1) * (unsigned)ctas + total - 1) / total) - 1;
        }
        if (!u.last && u.start >= 0) {
            const unsigned long long fin = from + (unsigned)last_place + 1;
            u.parts = (int)((fin * (unsigned)ctas + total - 1) / total) - u.start;
        } else if (u.start >= 0) {
            u.parts = c + 1 - u.start;
        }
    }
};

// Partial rows of cut units in the workspace: CTA c's slot 0 holds a part that
// goes on from CTA c - 1, slot 1 one that begins in CTA c and goes on in c + 1.
// A slot is rows x d unnormalised sums, then rows x (reference, sum of weights),
// the reference in units of log2.  meta[2 c + 1] describes slot 1: (first token,
// first query head, tokens, parts), parts = 0 where nothing begins and goes on;
// meta[2 c] is (CTA in which slot 0's unit begins, parts), or -1 where there is none.
struct Partials {
    int4* meta;
    float* rows;
    int cap;                                       // rows of a slot
    int d;
    __device__ __forceinline__ void clear(int c) const {
        meta[2 * c] = make_int4(-1, 0, 0, 0);
        meta[2 * c + 1] = make_int4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void describe(int c, const Unit& u) const {
        if (!u.first) meta[2 * c] = make_int4(u.start, u.parts, 0, 0);
        else if (!u.last) meta[2 * c + 1] = make_int4(u.tok0, u.qh0, u.ntok, u.parts);
    }
    // As latent attention's merge reads it: either slot's unit in full, (first token, first query head, tokens,
    // CTA in which it begins << 16 | parts), parts = 0 where there is none.
    __device__ __forceinline__ void clear_both(int c) const { meta[2 * c] = meta[2 * c + 1] = make_int4(0, 0, 0, 0); }
    __device__ __forceinline__ void describe_both(int c, const Unit& u) const {
        if (!u.first || !u.last) meta[2 * c + (u.first ? 1 : 0)] = make_int4(u.tok0, u.qh0, u.ntok, u.start << 16 | u.parts);
    }
    __device__ __forceinline__ size_t slot(int c, int which) const {
        return ((size_t)c * 2 + which) * (size_t)cap * (d + 2);
    }
    __device__ __forceinline__ float* sums(int c, int which) const { return rows + slot(c, which); }
    // Latent attention's slots hold their sums four channels wide, [d / 4][cap][4].
    __device__ __forceinline__ float* sums4(int c, int which, int row, int channel) const {
        return rows + slot(c, which) + ((size_t)(channel >> 2) * cap + row) * 4;
    }
    __device__ __forceinline__ float2* stats(int c, int which) const {
        return reinterpret_cast<float2*>(rows + slot(c, which) + (size_t)cap * d);
    }
};

}  // namespace kda_paged

namespace kda_host {

struct PagedArgs {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_table;
    const int32_t* cu_seqlens;
    const int32_t* seq_len;
    int64_t q_stride;
    int N, T, Hq, Hkv, d, page_size, blocks, n_pages;
    float scale;
    int window;
    kda_dtype dtype;
    void* o;
    float* lse;
    void* workspace;
    cudaStream_t stream;
    int* status;
};

struct TablesArgs {
    const int32_t* ctx_len;
    const int32_t* new_len;
    const int32_t* free_pages;
    int n_free, N, blocks, page_size, n_tokens;
    int32_t* block_table;
    int32_t* cu_seqlens;
    int32_t* seq_len;
    int64_t* slot_map;
    int32_t* positions;
    int32_t* n_taken;
    cudaStream_t stream;
};

struct AppendArgs {
    const void* k;
    const void* v;
    const int64_t* slot_map;
    int64_t k_stride, v_stride;
    int T, H, d, page_size, n_pages, esize;
    void* k_cache;
    void* v_cache;
    cudaStream_t stream;
};

struct VerifyArgs {
    const void* target;
    const void* draft;
    const int32_t* draft_tokens;
    const float* uniforms;
    const int32_t* draft_len;
    int N, K, V;
    kda_dtype dtype;
    int32_t* tokens;
    int32_t* commit_len;
    cudaStream_t stream;
};

// Runs a device's one-time set-up (function attributes) on its first call there.
struct OncePerDevice {
    std::atomic<unsigned long long> done{0};
    template <typename F>
    cudaError_t run(F f) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = 1ull << (dev & 63);
        if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
        e = f();                                       // twice is harmless
        if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

// Launches `kern` so that it may be set up while the kernel before it on the stream
// still runs: every thread of such a kernel calls kda_paged::wait_for_stream()
// before it touches global memory.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, int cluster,
                              A&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

int* status_word();                                // the device status word (kda_api.cu)
int sm_count();                                    // SMs of the current device

// Query heads of one unit's rows, and how many such groups share a cache head:
// the most heads that divide the group evenly and fit `most` rows.
inline int heads_per_unit(int group, int most) {
    int g = group < most ? group : most;
    while (group % g != 0) --g;
    return g;
}

// Partial-row geometry of an attention call: rows of a slot, most CTAs.
struct PagedPlan {
    int Gv, U, rows, tile_log2, max_ctas, extra;
    int half_unit = 0, extra_two = 0;                  // of packed keys (PackedShape); 0: every unit takes one step a tile
};
bool paged_tc_supported(int d, kda_dtype dt);
PagedPlan paged_plan_tc(int T, int Hq, int Hkv);
PagedPlan paged_plan_simt(int T, int Hq, int Hkv, int d);
int paged_slot_rows(int U, int T, int Gv);
size_t paged_plan_bytes(const PagedPlan& p, int d);

cudaError_t launch_build_tables(const TablesArgs& a);
cudaError_t launch_cache_append(const AppendArgs& a);
cudaError_t launch_verify_draft(const VerifyArgs& a);
cudaError_t launch_paged_attention_tc(const PagedArgs& a);
cudaError_t launch_paged_attention_simt(const PagedArgs& a);
cudaError_t launch_paged_merge(const PagedArgs& a, const PagedPlan& p, int ctas);
kda_paged::Shape paged_shape(const PagedArgs& a, const PagedPlan& p);
kda_paged::Partials paged_partials(const PagedArgs& a, const PagedPlan& p);

}  // namespace kda_host
