// latent.cuh -- host interface of the latent-attention operators: rotary
// positions, latent cache append, absorbed attention over the paged latent cache,
// expanded attention over packed keys and values.
#pragma once

#include "paged.cuh"

namespace kda_latent {

// Channels: the latent (which is also every head's value in the absorbed form) and the rotated
// key part beside it; a head's own key part and value in the expanded form.
constexpr int kLatent = 512, kRope = 64, kRow = kLatent + kRope;
constexpr int kNope = 128, kKey = kNope + kRope, kValue = 128;

}  // namespace kda_latent

namespace kda_host {

struct RotaryArgs {
    const void* x;
    const int32_t* positions;
    const float* inv_freq;
    int64_t x_token, x_head, out_token, out_head;     // strides in elements
    int T, H, d, rot;
    int interleaved;
    float factor;
    kda_dtype dtype;
    void* out;
    cudaStream_t stream;
};

struct LatentAppendArgs {
    const void* c;
    const void* k_rope;
    const int64_t* slot_map;
    const int32_t* positions;                          // with inv_freq, or both null: the key part is copied
    const float* inv_freq;
    int64_t c_stride, r_stride;
    int T, page_size, n_pages;
    int interleaved;
    float factor;
    kda_dtype dtype;
    void* cache;
    cudaStream_t stream;
};

struct LatentArgs {
    const void* q;                                     // [T, H, 576]
    const void* cache;                                 // [n_pages, page_size, 576]
    const int32_t* block_table;
    const int32_t* cu_seqlens;
    const int32_t* seq_len;
    int64_t q_stride;
    int N, T, H, page_size, blocks, n_pages;
    float scale;
    kda_dtype dtype;
    void* o;                                           // [T, H, 512]
    float* lse;
    void* workspace;
    cudaStream_t stream;
    int* status;
};

struct ExpandedArgs {
    const void* q;                                     // [T, H, 192]
    const void* k_nope;                                // [S, H, 128]
    const void* k_rope;                                // [S, 64]
    const void* v;                                     // [S, H, 128]
    const int32_t* cu_seqlens;
    const int32_t* cu_seqlens_k;
    int64_t q_stride, kn_token, kn_head, kr_stride, v_token, v_head;
    int N, T, S, H;
    float scale;
    int causal;
    kda_dtype dtype;
    void* o;                                           // [T, H, 128]
    float* lse;
    void* workspace;
    cudaStream_t stream;
    int* status;
};

int latent_groups(int H, int most);
PagedArgs latent_view(const LatentArgs& a);            // what the merge and the shape need of a call
kda_paged::Shape latent_shape(const LatentArgs& a, const PagedPlan& p);
PagedArgs expanded_view(const ExpandedArgs& a);
kda_paged::PackedShape expanded_shape(const ExpandedArgs& a, const PagedPlan& p);

cudaError_t launch_latent_merge(const PagedArgs& a, const PagedPlan& p, int ctas);

cudaError_t launch_rotary(const RotaryArgs& a);
cudaError_t launch_latent_append(const LatentAppendArgs& a);
PagedPlan latent_plan_simt(int T, int H);
PagedPlan latent_plan_tc(int T, int H);
PagedPlan expanded_plan_simt(int T);
PagedPlan expanded_plan_tc(int T);
cudaError_t launch_latent_attention_simt(const LatentArgs& a);
cudaError_t launch_latent_attention_tc(const LatentArgs& a);
cudaError_t launch_expanded_attention_simt(const ExpandedArgs& a);
cudaError_t launch_expanded_attention_tc(const ExpandedArgs& a);

}  // namespace kda_host
