// paged_tables.cu -- block tables and slot map of a step, and the cache append.
//
// Tables.  With P tokens a page, request n needs
//     need_n = ceil((ctx_n + new_n) / P) - ceil(ctx_n / P)
// pages; page m of the step (m counting through the requests in order) is
// free_pages[m] and becomes entry ceil(ctx_n / P) + m - sum_{n' < n} need_n' of
// the request's row.  New token t of the step belongs to the request whose
// interval of the running sum of new_n holds t.
//
// The running sums are over at most a few thousand requests, so every CTA
// forms both at once itself (they share one 64-bit word), in shared memory,
// and then writes its share of tokens and pages: one launch, and nothing that
// one CTA waits for another for.  A token's page is looked up in the table only
// where the request held it before; a page taken in this step comes from the
// free list directly, since its table entry may be another CTA's to write.
// Bound: 12 bytes a token are written; below ~100,000 tokens the launch and the
// chain of dependent reads (lengths, running sum, free list) set the time: 24
// requests of one token 3.4 us, 320 prompts of 860,000 tokens 7.3 us (10.3 MB,
// floor 1.5 us; GPU time): the same chain, then a search a thread and a look-up a token that
// wait for each other (issue slots 32 % busy, DRAM next to idle).  Three CTAs of 256 threads an SM, four tokens a thread:
// one or two take 12.7 and 8.5 us, four of 512 threads 9.5 us (each forms the
// sums again), eight tokens a thread 8.6 us (more code to fetch than it saves).
//
// Append.  Row t of k and v moves to its slot in 16-byte pieces (single
// elements where a pointer or a stride is not a multiple of 16 bytes), four
// pieces of both in flight per thread.  Bound: HBM, 4 x the row's bytes: 40,001
// tokens x 8 heads x 128 bf16 (328 MB) 52.6 us, 0.93 of the measured copy rate.
#include <algorithm>

#include "paged.cuh"

namespace {

using kda_paged::kMaxRequests;

constexpr int kTableThreads = 256;
constexpr int kTokensPerThread = 4;

__global__ void __launch_bounds__(kTableThreads)
kda_build_tables_kernel(const int32_t* __restrict__ ctx_len, const int32_t* __restrict__ new_len,
                        const int32_t* __restrict__ free_pages, int n_free, int N, int blocks, int page_log2,
                        int n_tokens, int32_t* __restrict__ block_table, int32_t* __restrict__ cu_seqlens,
                        int32_t* __restrict__ seq_len, int64_t* __restrict__ slot_map,
                        int32_t* __restrict__ positions, int32_t* __restrict__ n_taken) {
    extern __shared__ int s_first[];                       // [N + 1] first new token of each request
    int* s_page = s_first + N + 1;                         // [N + 1] first new page of each request
    int* s_ctx = s_page + N + 1;                           // [N] cached tokens
    __shared__ unsigned long long s_red[kTableThreads / 32];
    kda_paged::wait_for_stream();

    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int page = 1 << page_log2;
    auto pages_of = [&](long long tokens) { return (int)min((tokens + page - 1) >> page_log2, (long long)blocks); };

    // running sums of new tokens (low word) and pages needed (high word), a
    // batch of kTableThreads requests at a time
    unsigned long long carry = 0;
    for (int base = 0; base < N; base += kTableThreads) {
        const int n = base + tid;
        int ctx = 0, add = 0;
        if (n < N) {
            ctx = max(ctx_len[n], 0);
            add = max(new_len[n], 0);
        }
        const int need = pages_of((long long)ctx + add) - pages_of(ctx);
        const unsigned long long mine = ((unsigned long long)(unsigned)need << 32) | (unsigned)add;
        unsigned long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        if (lane == 31) s_red[w] = incl;
        __syncthreads();
        unsigned long long before = carry;
#pragma unroll
        for (int i = 0; i < kTableThreads / 32; ++i) {
            if (i < w) before += s_red[i];
            carry += s_red[i];
        }
        if (n < N) {
            const unsigned long long excl = before + incl - mine;
            s_first[n] = (int)(unsigned)excl;
            s_page[n] = (int)(excl >> 32);
            s_ctx[n] = ctx;
            if (blockIdx.x == 0) {
                cu_seqlens[n] = (int)(unsigned)excl;
                seq_len[n] = ctx + add;
            }
        }
        __syncthreads();
    }
    const int total = (int)(unsigned)carry, taken = (int)(carry >> 32);
    if (tid == 0) {
        s_first[N] = total;
        s_page[N] = taken;
        if (blockIdx.x == 0) {
            cu_seqlens[N] = total;
            n_taken[0] = taken;
        }
    }
    __syncthreads();

    // last n with at[n] <= x (x below at[N]), so requests that add nothing are passed over
    auto find = [&](const int* at, int x) {
        int lo = 0, hi = N;                                // at[lo] <= x < at[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (at[mid] <= x) lo = mid; else hi = mid;
        }
        return lo;
    };
    const int stride = gridDim.x * kTableThreads, first = blockIdx.x * kTableThreads + tid;
    for (int m = first; m < taken; m += stride) {
        const int n = find(s_page, m);
        const int b = pages_of(s_ctx[n]) + (m - s_page[n]);
        if ((unsigned)b < (unsigned)blocks) block_table[(size_t)n * blocks + b] = m < n_free ? free_pages[m] : -1;
    }
    // four consecutive tokens a thread: one search, 16-byte stores
    for (long long t0 = (long long)first * kTokensPerThread; t0 < n_tokens; t0 += (long long)stride * kTokensPerThread) {
        long long slot[kTokensPerThread];
        int pos_out[kTokensPerThread];
        int n = t0 < total ? find(s_first, (int)t0) : N;
#pragma unroll
        for (int e = 0; e < kTokensPerThread; ++e) {
            const int t = (int)min(t0 + e, (long long)INT32_MAX);
            slot[e] = -1;
            pos_out[e] = 0;
            if (t0 + e >= total) continue;
            while (n + 1 < N && t >= s_first[n + 1]) ++n;
            const int ctx = s_ctx[n], have = pages_of(ctx);
            const long long pos = (long long)ctx + (t - s_first[n]);
            const int b = (int)min(pos >> page_log2, (long long)INT32_MAX);
            pos_out[e] = (int)pos;
            if (b < 0 || b >= blocks) continue;
            int id;
            if (b < have) {
                id = block_table[(size_t)n * blocks + b];
            } else {
                const int m = s_page[n] + b - have;
                id = (unsigned)m < (unsigned)n_free ? free_pages[m] : -1;   // sums that wrapped stay inside, too
            }
            if (id >= 0) slot[e] = ((long long)id << page_log2) + (pos & (long long)(page - 1));
        }
        if (t0 + kTokensPerThread <= n_tokens && ((uintptr_t)slot_map & 15) == 0) {
            *reinterpret_cast<longlong2*>(slot_map + t0) = make_longlong2(slot[0], slot[1]);
            *reinterpret_cast<longlong2*>(slot_map + t0 + 2) = make_longlong2(slot[2], slot[3]);
        } else {
#pragma unroll
            for (int e = 0; e < kTokensPerThread; ++e)
                if (t0 + e < n_tokens) slot_map[t0 + e] = slot[e];
        }
        if (!positions) continue;
        if (t0 + kTokensPerThread <= n_tokens && ((uintptr_t)positions & 15) == 0) {
            *reinterpret_cast<int4*>(positions + t0) = make_int4(pos_out[0], pos_out[1], pos_out[2], pos_out[3]);
        } else {
#pragma unroll
            for (int e = 0; e < kTokensPerThread; ++e)
                if (t0 + e < n_tokens) positions[t0 + e] = pos_out[e];
        }
    }
}

constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 4;

// U: the piece that moves at once.  A row of one head is `per_head` pieces, of
// all heads `per_row`; strides and cache offsets are in pieces.
template <typename U>
__global__ void __launch_bounds__(kAppendThreads)
kda_cache_append_kernel(const U* __restrict__ k, const U* __restrict__ v, const int64_t* __restrict__ slot_map,
                        long long k_stride, long long v_stride, long long total, int per_head, int per_row, int H,
                        int page_log2, long long n_slots, U* __restrict__ k_cache, U* __restrict__ v_cache) {
    kda_paged::wait_for_stream();
    const long long step = (long long)gridDim.x * kAppendThreads;
    for (long long u0 = (long long)blockIdx.x * kAppendThreads + threadIdx.x; u0 < total; u0 += step * kAppendUnroll) {
        U a[kAppendUnroll], b[kAppendUnroll];
        long long dst[kAppendUnroll];
#pragma unroll
        for (int e = 0; e < kAppendUnroll; ++e) {
            const long long u = u0 + e * step;
            dst[e] = -1;
            if (u >= total) continue;
            long long t;                                   // token, and piece of its row
            int x;
            if (total <= INT32_MAX) {
                const unsigned t32 = (unsigned)u / (unsigned)per_row;
                t = t32;
                x = (int)((unsigned)u - t32 * (unsigned)per_row);
            } else {
                t = u / per_row;
                x = (int)(u - t * per_row);
            }
            const long long slot = slot_map[t];
            if (slot < 0 || slot >= n_slots) continue;
            const int h = (unsigned)x / (unsigned)per_head, c = x - h * per_head;
            const long long page = slot >> page_log2, place = slot & ((1 << page_log2) - 1);
            dst[e] = (((page * H + h) << page_log2) + place) * per_head + c;
            a[e] = k[t * k_stride + x];
            b[e] = v[t * v_stride + x];
        }
#pragma unroll
        for (int e = 0; e < kAppendUnroll; ++e) {
            if (dst[e] < 0) continue;
            k_cache[dst[e]] = a[e];
            v_cache[dst[e]] = b[e];
        }
    }
}

int log2_of(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

template <typename U>
cudaError_t append(const kda_host::AppendArgs& a) {
    const int ratio = (int)sizeof(U) / a.esize;            // elements a piece
    const int per_head = a.d / ratio, per_row = per_head * a.H;
    const long long total = (long long)a.T * per_row;
    const long long want = (total + kAppendThreads - 1) / kAppendThreads;
    const int grid = (int)std::min<long long>(want, (long long)kda_host::sm_count() * 8);
    return kda_host::launch_overlapped(
        kda_cache_append_kernel<U>, grid, kAppendThreads, 0, a.stream, 1, static_cast<const U*>(a.k), static_cast<const U*>(a.v), a.slot_map, a.k_stride / ratio, a.v_stride / ratio,
        total, per_head, per_row, a.H, log2_of(a.page_size), (long long)a.n_pages * a.page_size,
        static_cast<U*>(a.k_cache), static_cast<U*>(a.v_cache));
}

}  // namespace

namespace kda_host {

cudaError_t launch_build_tables(const TablesArgs& a) {
    const size_t smem = ((size_t)3 * a.N + 2) * sizeof(int);
    static_assert(((size_t)3 * kMaxRequests + 2) * sizeof(int) <= 100 * 1024, "shared memory of the running sums");
    if (smem > 47 * 1024) {
        static OncePerDevice once;
        const cudaError_t e = once.run([] {
            return cudaFuncSetAttribute(kda_build_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)(((size_t)3 * kMaxRequests + 2) * sizeof(int)));
        });
        if (e != cudaSuccess) return e;
    }
    const long long work = std::max<long long>(((long long)a.n_tokens + kTokensPerThread - 1) / kTokensPerThread, 1);
    const int grid = (int)std::min<long long>((work + kTableThreads - 1) / kTableThreads, (long long)sm_count() * 3);
    return launch_overlapped(
        kda_build_tables_kernel, grid, kTableThreads, smem, a.stream, 1, a.ctx_len, a.new_len, a.free_pages, a.n_free, a.N, a.blocks, log2_of(a.page_size), a.n_tokens, a.block_table,
        a.cu_seqlens, a.seq_len, a.slot_map, a.positions, a.n_taken);
}

cudaError_t launch_cache_append(const AppendArgs& a) {
    // 16-byte pieces where every row of k and v starts on a 16-byte boundary
    // (the cache does); a head's row is always a multiple of 16 bytes long
    const bool wide = reinterpret_cast<uintptr_t>(a.k) % 16 == 0 && reinterpret_cast<uintptr_t>(a.v) % 16 == 0 &&
                      (a.k_stride * a.esize) % 16 == 0 && (a.v_stride * a.esize) % 16 == 0;
    if (wide) return append<uint4>(a);
    return a.esize == 2 ? append<uint16_t>(a) : append<uint32_t>(a);
}

}  // namespace kda_host
