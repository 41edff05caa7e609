// paged_api.cu -- C entry points of the serving-step operators: argument
// checks, path selection, launches.  See include/kda.h for their contracts.
#include <algorithm>

#include "paged.cuh"

namespace {

kda_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return KDA_OK;
    if (e == cudaErrorNotSupported) return KDA_ERR_UNSUPPORTED;
    return KDA_ERR_CUDA;
}

bool page_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128 || p == 256; }
bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }
bool dtype_ok(kda_dtype t) { return t == KDA_FP32 || t == KDA_BF16; }
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Enough for either path: which one runs also depends on the alignment of q.
size_t attention_workspace(int T, int Hq, int Hkv, int d, kda_dtype dt) {
    const size_t simt = kda_host::paged_plan_bytes(kda_host::paged_plan_simt(T, Hq, Hkv, d), d);
    if (!kda_host::paged_tc_supported(d, dt)) return simt;
    return std::max(simt, kda_host::paged_plan_bytes(kda_host::paged_plan_tc(T, Hq, Hkv), d));
}

}  // namespace

extern "C" {

kda_status kda_build_block_tables(const int32_t* ctx_len, const int32_t* new_len, const int32_t* free_pages,
                                  int n_free, int N, int max_blocks, int page_size, int n_tokens,
                                  int32_t* block_table, int32_t* cu_seqlens, int32_t* seq_len, int64_t* slot_map,
                                  int32_t* positions, int32_t* n_taken, cudaStream_t stream) {
    if (N < 0 || n_free < 0 || max_blocks < 0 || n_tokens < 0) return KDA_ERR_INVALID_ARG;
    if (!page_ok(page_size) || N > KDA_MAX_STEP_REQUESTS) return KDA_ERR_UNSUPPORTED;
    if (!cu_seqlens || !n_taken) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (!ctx_len || !new_len || !seq_len)) return KDA_ERR_INVALID_ARG;
    if (N > 0 && max_blocks > 0 && !block_table) return KDA_ERR_INVALID_ARG;
    if ((n_free > 0 && !free_pages) || (n_tokens > 0 && !slot_map)) return KDA_ERR_INVALID_ARG;
    if (!aligned(slot_map, 8)) return KDA_ERR_INVALID_ARG;
    // every CTA reads the lengths and the free list for itself, so none may write over them
    for (const void* in : {(const void*)ctx_len, (const void*)new_len, (const void*)free_pages})
        for (const void* out : {(const void*)block_table, (const void*)cu_seqlens, (const void*)seq_len,
                                (const void*)slot_map, (const void*)positions, (const void*)n_taken})
            if (in && in == out) return KDA_ERR_INVALID_ARG;
    const kda_host::TablesArgs a{ctx_len, new_len, free_pages, n_free, N, max_blocks, page_size, n_tokens,
                                 block_table, cu_seqlens, seq_len, slot_map, positions, n_taken, stream};
    return from_cuda(kda_host::launch_build_tables(a));
}

kda_status kda_cache_append(const void* k, const void* v, const int64_t* slot_map, int64_t k_stride,
                            int64_t v_stride, int T, int H_kv, int d, int page_size, int n_pages, kda_dtype dtype,
                            void* k_cache, void* v_cache, cudaStream_t stream) {
    if (T < 0 || H_kv <= 0 || n_pages < 0 || !dtype_ok(dtype)) return KDA_ERR_INVALID_ARG;
    if (!dim_ok(d) || !page_ok(page_size)) return KDA_ERR_UNSUPPORTED;
    if (H_kv > (1 << 16)) return KDA_ERR_UNSUPPORTED;
    if (k_stride < (int64_t)H_kv * d || v_stride < (int64_t)H_kv * d) return KDA_ERR_INVALID_ARG;
    if (T == 0 || n_pages == 0) return KDA_OK;
    if (!k || !v || !slot_map || !k_cache || !v_cache) return KDA_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return KDA_ERR_INVALID_ARG;
    const int esize = dtype == KDA_BF16 ? 2 : 4;
    if (!aligned(k, esize) || !aligned(v, esize) || !aligned(slot_map, 8)) return KDA_ERR_INVALID_ARG;
    if (k_cache == v_cache || k_cache == k || k_cache == v || v_cache == k || v_cache == v)
        return KDA_ERR_INVALID_ARG;
    const kda_host::AppendArgs a{k, v, slot_map, k_stride, v_stride, T, H_kv, d, page_size, n_pages, esize,
                                 k_cache, v_cache, stream};
    return from_cuda(kda_host::launch_cache_append(a));
}

size_t kda_paged_attention_workspace_size(int T, int H_q, int H_kv, int d, kda_dtype dtype) {
    if (T < 0 || H_q <= 0 || H_kv <= 0 || H_q % H_kv != 0 || !dim_ok(d) || !dtype_ok(dtype)) return 0;
    return attention_workspace(T, H_q, H_kv, d, dtype);
}

kda_status kda_paged_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                               const int32_t* cu_seqlens, const int32_t* seq_len, int64_t q_stride, int N, int T,
                               int H_q, int H_kv, int d, int page_size, int max_blocks, int n_pages, float scale,
                               int window, kda_dtype dtype, void* o, float* lse, void* workspace,
                               size_t workspace_bytes, cudaStream_t stream) {
    if (N < 0 || T < 0 || H_q <= 0 || H_kv <= 0 || H_q % H_kv != 0) return KDA_ERR_INVALID_ARG;
    if (max_blocks < 0 || n_pages < 0 || window < 0 || !dtype_ok(dtype)) return KDA_ERR_INVALID_ARG;
    if (!dim_ok(d) || !page_ok(page_size)) return KDA_ERR_UNSUPPORTED;
    if (N > KDA_MAX_STEP_REQUESTS || H_q > (1 << 16)) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)max_blocks * page_size > KDA_MAX_STEP_POSITIONS) return KDA_ERR_UNSUPPORTED;
    // at most 2^127: the kernels work with scale log2(e), which has to be finite too
    if (!(scale > 0.f) || !(scale <= 0x1p127f)) return KDA_ERR_INVALID_ARG;
    if (q_stride < (int64_t)H_q * d) return KDA_ERR_INVALID_ARG;
    if (T == 0 || N == 0) return KDA_OK;
    if (!q || !cu_seqlens || !seq_len || !o) return KDA_ERR_INVALID_ARG;
    if (n_pages > 0 && (!k_cache || !v_cache)) return KDA_ERR_INVALID_ARG;
    if (max_blocks > 0 && !block_table) return KDA_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16)) return KDA_ERR_INVALID_ARG;
    if (!aligned(q, dtype == KDA_BF16 ? 2 : 4)) return KDA_ERR_INVALID_ARG;
    if (o == q || o == k_cache || o == v_cache) return KDA_ERR_INVALID_ARG;
    const size_t need = attention_workspace(T, H_q, H_kv, d, dtype);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return KDA_ERR_WORKSPACE;
    kda_host::PagedArgs a{q, k_cache, v_cache, block_table, cu_seqlens, seq_len, q_stride, N, T, H_q, H_kv, d,
                          page_size, max_blocks, n_pages, scale, window, dtype, o, lse, workspace, stream,
                          kda_host::status_word()};
    // the tensor-core path fetches q by TMA, whose rows start on 16-byte boundaries, and
    // describes the cache to it, which an empty one cannot be
    const bool tc = kda_host::paged_tc_supported(d, dtype) && aligned(q, 16) && q_stride % 8 == 0 && n_pages > 0 &&
                    max_blocks > 0;
    return from_cuda(tc ? kda_host::launch_paged_attention_tc(a) : kda_host::launch_paged_attention_simt(a));
}

kda_status kda_verify_draft(const void* target, const void* draft, const int32_t* draft_tokens,
                            const float* uniforms, const int32_t* draft_len, int N, int K, int V, kda_dtype dtype,
                            int32_t* tokens, int32_t* commit_len, cudaStream_t stream) {
    if (N < 0 || K < 0 || V <= 0 || !dtype_ok(dtype)) return KDA_ERR_INVALID_ARG;
    if (K > 16 || N > (1 << 20)) return KDA_ERR_UNSUPPORTED;
    if (V > (1 << 30)) return KDA_ERR_UNSUPPORTED;         // the places of a row and a thread's steps past its end are 32-bit
    if (N == 0) return KDA_OK;
    if (!target || !uniforms || !tokens || !commit_len || (K > 0 && !draft_tokens)) return KDA_ERR_INVALID_ARG;
    if (tokens == draft_tokens) return KDA_ERR_INVALID_ARG;
    const size_t esize = dtype == KDA_BF16 ? 2 : 4;
    if (!aligned(target, esize) || !aligned(draft, esize)) return KDA_ERR_INVALID_ARG;
    const kda_host::VerifyArgs a{target, draft, draft_tokens, uniforms, draft_len, N, K, V, dtype, tokens,
                                 commit_len, stream};
    return from_cuda(kda_host::launch_verify_draft(a));
}

}  // extern "C"
