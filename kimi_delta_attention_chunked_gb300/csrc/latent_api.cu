// latent_api.cu -- C entry points of the latent-attention operators: argument
// checks, path selection, launches.  See include/kda.h for their contracts.
#include <algorithm>
#include <cmath>

#include "api_checks.cuh"
#include "latent.cuh"

namespace {

using kda_host::aligned;
using kda_host::dtype_ok;
using kda_host::element_size;
using kda_host::from_cuda;
using kda_host::page_ok;
using kda_host::rows_apart;
using kda_latent::kLatent;
using kda_latent::kNope;
using kda_latent::kKey;
using kda_latent::kRope;
using kda_latent::kRow;
using kda_latent::kValue;

constexpr int kMaxHeads = 1 << 16;

// Enough for either path: which one runs also depends on alignment.
size_t latent_workspace(int T, int H, kda_dtype dt) {
    const size_t simt = kda_host::paged_plan_bytes(kda_host::latent_plan_simt(T, H), kLatent);
    if (dt != KDA_BF16) return simt;
    return std::max(simt, kda_host::paged_plan_bytes(kda_host::latent_plan_tc(T, H), kLatent));
}
size_t expanded_workspace(int T, kda_dtype dt) {
    const size_t simt = kda_host::paged_plan_bytes(kda_host::expanded_plan_simt(T), kValue);
    if (dt != KDA_BF16) return simt;
    return std::max(simt, kda_host::paged_plan_bytes(kda_host::expanded_plan_tc(T), kValue));
}

// TMA fetches bf16 rows that start on 16-byte boundaries, at strides below 2^40 bytes.
bool fetchable(const void* p, int64_t s0, int64_t s1 = 8) {
    constexpr int64_t kMost = (int64_t(1) << 39) - 8;
    return aligned(p, 16) && s0 % 8 == 0 && s1 % 8 == 0 && s0 > 0 && s1 > 0 && s0 <= kMost && s1 <= kMost;
}

}  // namespace

extern "C" {

kda_status kda_rotary(const void* x, const int32_t* positions, const float* inv_freq, int64_t x_token_stride,
                      int64_t x_head_stride, int64_t out_token_stride, int64_t out_head_stride, int T, int H, int d, int rot,
                      int interleaved, float factor, kda_dtype dtype, void* out, cudaStream_t stream) {
    if (T < 0 || H <= 0 || d <= 0 || rot < 2 || rot > d || rot % 2 != 0 || !dtype_ok(dtype)) return KDA_ERR_INVALID_ARG;
    if (d > 256 || H > kMaxHeads) return KDA_ERR_UNSUPPORTED;
    if (!std::isfinite(factor)) return KDA_ERR_INVALID_ARG;
    if (x_token_stride < 0 || x_head_stride < 0 || !rows_apart(T, out_token_stride, H, out_head_stride, d))
        return KDA_ERR_INVALID_ARG;
    if (T == 0) return KDA_OK;
    if (!x || !positions || !inv_freq || !out) return KDA_ERR_INVALID_ARG;
    if (!aligned(x, element_size(dtype)) || !aligned(out, element_size(dtype))) return KDA_ERR_INVALID_ARG;
    if (x == out && ((T > 1 && x_token_stride != out_token_stride) || (H > 1 && x_head_stride != out_head_stride)))
        return KDA_ERR_INVALID_ARG;
    if (out == positions || out == inv_freq) return KDA_ERR_INVALID_ARG;
    const kda_host::RotaryArgs a{x, positions, inv_freq, x_token_stride, x_head_stride, out_token_stride, out_head_stride,
                                 T, H, d, rot, interleaved != 0, factor, dtype, out, stream};
    return from_cuda(kda_host::launch_rotary(a));
}

kda_status kda_latent_append(const void* c, const void* k_rope, const int64_t* slot_map, const int32_t* positions,
                             const float* inv_freq, int64_t c_stride, int64_t k_rope_stride, int T, int page_size,
                             int n_pages, int interleaved, float factor, kda_dtype dtype, void* cache,
                             cudaStream_t stream) {
    if (T < 0 || n_pages < 0 || !dtype_ok(dtype)) return KDA_ERR_INVALID_ARG;
    if (!page_ok(page_size)) return KDA_ERR_UNSUPPORTED;
    if (!std::isfinite(factor) || c_stride < kLatent || k_rope_stride < kRope) return KDA_ERR_INVALID_ARG;
    if ((positions == nullptr) != (inv_freq == nullptr)) return KDA_ERR_INVALID_ARG;
    if (T == 0 || n_pages == 0) return KDA_OK;
    if (!c || !k_rope || !slot_map || !cache) return KDA_ERR_INVALID_ARG;
    if (!aligned(cache, 16) || !aligned(slot_map, 8)) return KDA_ERR_INVALID_ARG;
    if (!aligned(c, element_size(dtype)) || !aligned(k_rope, element_size(dtype))) return KDA_ERR_INVALID_ARG;
    if (cache == c || cache == k_rope) return KDA_ERR_INVALID_ARG;
    const kda_host::LatentAppendArgs a{c, k_rope, slot_map, positions, inv_freq, c_stride, k_rope_stride, T, page_size,
                                       n_pages, interleaved != 0, factor, dtype, cache, stream};
    return from_cuda(kda_host::launch_latent_append(a));
}

size_t kda_latent_attention_workspace_size(int T, int H, kda_dtype dtype) {
    if (T < 0 || H <= 0 || H > kMaxHeads || !dtype_ok(dtype)) return 0;
    return latent_workspace(T, H, dtype);
}

kda_status kda_latent_attention(const void* q, const void* cache, const int32_t* block_table, const int32_t* cu_seqlens,
                                const int32_t* seq_len, int64_t q_stride, int N, int T, int H, int page_size,
                                int max_blocks, int n_pages, float scale, kda_dtype dtype, void* o, float* lse,
                                void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (N < 0 || T < 0 || H <= 0 || max_blocks < 0 || n_pages < 0 || !dtype_ok(dtype)) return KDA_ERR_INVALID_ARG;
    if (!page_ok(page_size) || N > KDA_MAX_STEP_REQUESTS || H > kMaxHeads) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)max_blocks * page_size > KDA_MAX_STEP_POSITIONS) return KDA_ERR_UNSUPPORTED;
    // at most 2^127: the kernels work with scale log2(e), which has to be finite too
    if (!(scale > 0.f) || !(scale <= 0x1p127f)) return KDA_ERR_INVALID_ARG;
    if (q_stride < (int64_t)H * kRow) return KDA_ERR_INVALID_ARG;
    if (T == 0 || N == 0) return KDA_OK;
    if (!q || !cu_seqlens || !seq_len || !o) return KDA_ERR_INVALID_ARG;
    if ((n_pages > 0 && !cache) || (max_blocks > 0 && !block_table)) return KDA_ERR_INVALID_ARG;
    if (!aligned(cache, 16) || !aligned(o, 32) || !aligned(q, element_size(dtype))) return KDA_ERR_INVALID_ARG;
    if (o == q || o == cache) return KDA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < latent_workspace(T, H, dtype) || !aligned(workspace, 256)) return KDA_ERR_WORKSPACE;
    const kda_host::LatentArgs a{q, cache, block_table, cu_seqlens, seq_len, q_stride, N, T, H, page_size, max_blocks, n_pages,
                                 scale, dtype, o, lse, workspace, stream, kda_host::status_word()};
    // the tensor-core path fetches q by TMA and describes the cache to it, which an empty one cannot be
    const bool tc = dtype == KDA_BF16 && fetchable(q, q_stride) && n_pages > 0 && max_blocks > 0;
    return from_cuda(tc ? kda_host::launch_latent_attention_tc(a) : kda_host::launch_latent_attention_simt(a));
}

size_t kda_expanded_attention_workspace_size(int T, int H, kda_dtype dtype) {
    if (T < 0 || H <= 0 || H > kMaxHeads || !dtype_ok(dtype)) return 0;
    return expanded_workspace(T, dtype);
}

kda_status kda_expanded_attention(const void* q, const void* k_nope, const void* k_rope, const void* v,
                                  const int32_t* cu_seqlens, const int32_t* cu_seqlens_k, int64_t q_stride,
                                  int64_t k_token_stride, int64_t k_head_stride, int64_t k_rope_stride,
                                  int64_t v_token_stride, int64_t v_head_stride, int N, int T, int S, int H, float scale,
                                  int causal, kda_dtype dtype, void* o, float* lse, void* workspace,
                                  size_t workspace_bytes, cudaStream_t stream) {
    if (N < 0 || T < 0 || S < 0 || H <= 0 || !dtype_ok(dtype)) return KDA_ERR_INVALID_ARG;
    if (N > KDA_MAX_STEP_REQUESTS || H > kMaxHeads) return KDA_ERR_UNSUPPORTED;
    // a row behind all of its request's keys stands at a position below S + T
    if ((int64_t)S + T > KDA_MAX_STEP_POSITIONS) return KDA_ERR_UNSUPPORTED;
    if (!(scale > 0.f) || !(scale <= 0x1p127f)) return KDA_ERR_INVALID_ARG;
    if (q_stride < (int64_t)H * kKey || k_rope_stride < kRope) return KDA_ERR_INVALID_ARG;
    // rows of their own, or at a head stride of 0 the same ones for all heads (which TMA does not fetch)
    auto rows_ok = [&](int64_t token, int64_t head, int width) { return rows_apart(S, token, head == 0 ? 1 : H, head, width); };
    if (!rows_ok(k_token_stride, k_head_stride, kNope) || !rows_ok(v_token_stride, v_head_stride, kValue)) return KDA_ERR_INVALID_ARG;
    // the stride of a dim of one has no meaning
    if (S <= 1) k_token_stride = v_token_stride = (int64_t)H * (kNope + kValue);
    if (H == 1) k_head_stride = v_head_stride = kNope;
    if (T == 0 || N == 0) return KDA_OK;
    if (!q || !cu_seqlens || !cu_seqlens_k || !o) return KDA_ERR_INVALID_ARG;
    if (S > 0 && (!k_nope || !k_rope || !v)) return KDA_ERR_INVALID_ARG;
    const int size = element_size(dtype);
    if (!aligned(q, size) || !aligned(k_nope, size) || !aligned(k_rope, size) || !aligned(v, size) || !aligned(o, 32))
        return KDA_ERR_INVALID_ARG;
    if (o == q || o == k_nope || o == k_rope || o == v) return KDA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < expanded_workspace(T, dtype) || !aligned(workspace, 256)) return KDA_ERR_WORKSPACE;
    const kda_host::ExpandedArgs a{q, k_nope, k_rope, v, cu_seqlens, cu_seqlens_k, q_stride, k_token_stride, k_head_stride,
                                   k_rope_stride, v_token_stride, v_head_stride, N, T, S, H, scale, causal != 0, dtype, o, lse,
                                   workspace, stream, kda_host::status_word()};
    const bool tc = dtype == KDA_BF16 && S > 0 && fetchable(q, q_stride) && fetchable(k_nope, k_token_stride, k_head_stride) &&
                    fetchable(k_rope, k_rope_stride) && fetchable(v, v_token_stride, v_head_stride);
    return from_cuda(tc ? kda_host::launch_expanded_attention_tc(a) : kda_host::launch_expanded_attention_simt(a));
}

}  // extern "C"
