/*
 * kda.h -- C ABI of the GB300 (sm_103a) Kimi Delta Attention library.
 *
 * The operator.  Per head, KDA keeps a state S in R^{d_k x d_v} and, for every
 * token t, applies
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T,
 *     o_t = S_t^T q_t,
 *
 * with alpha_t in (0,1)^{d_k} a forget gate per key channel and beta_t a
 * scalar write strength ("Kimi K3" blog, section "Kimi Delta Attention"; the
 * same update in words on the "LLM architecture at trillion scale" page,
 * section "The KDA update, in plain words").  The gate is passed as
 * log_alpha = ln(alpha_t), expected in [-5, 0): the log-decay bound stated on
 * that page.  Values outside it are computed but not guaranteed to meet the
 * accuracy target.  The tightest case of the bf16 tensor-core path is the
 * no-decay end of the range (log_alpha = -1e-4 on every channel, the gate's
 * upper clamp), where the state carries each chunk's operand rounding through
 * the whole sequence: over 8192 tokens and 32 heads the output error is about
 * 4.8e-3 with beta = 1 on every token and 5.0e-3 with beta drawn by sigmoid,
 * relative to max|o|, against the 5e-3 bf16 target (in that range the chunk
 * prep feeds its Gram operands to the tensor cores as f16).  The fp32
 * CUDA-core path stays well inside it (about 3e-3).
 *
 * Two entry points compute it:
 *   kda_prefill -- many tokens at once in the chunked form ("Kimi K3: the
 *                  manos, the mythos, the legendos", section "FlashKDA
 *                  Algorithm"), returning every o_t and the final state;
 *   kda_decode  -- one token per sequence, updating an fp32 state in place
 *                  (the per-token form of the same section).
 *
 * Conventions for every call
 *   - All tensor arguments are caller-owned, contiguous, row-major DEVICE
 *     pointers (cu_seqlens_host is the one host pointer).  The library never
 *     allocates device memory and never synchronises the stream, except in
 *     kda_get_last_device_status and once per device in the first long
 *     tensor-core prefill (below).
 *   - Work is enqueued on `stream` (0 = the legacy default stream).  A call
 *     returns once the work is enqueued.  A long tensor-core prefill (the
 *     longest sequence at least 1024 chunks, its state pass on at most half
 *     of the SMs) forks part of its work onto an internal high-priority
 *     stream of the library (created once per device, kept until exit) and
 *     joins it back into `stream` with events before returning, so ordering
 *     on `stream` holds.  The first such call on a device, unless `stream`
 *     is being captured into a graph, also runs a ~10 us kernel that finds
 *     which SM ids the device has (32 bytes of the workspace) and waits for
 *     it on `stream`; later calls reuse the result.
 *   - Arguments are checked before anything is launched; a failed check
 *     returns an error and launches nothing.  A launch failure returns
 *     KDA_ERR_CUDA.  Faults detected inside a kernel (a wait that ran out of
 *     time) are recorded in a device status word read by
 *     kda_get_last_device_status.
 *   - Supported shapes: d_k, d_v in {32, 64, 128}; chunk in {16, 32, 64}.
 *     KDA_BF16 with d_k = d_v = 128 and chunk = 64 runs on the tcgen05
 *     tensor-core path; every other combination runs on the fp32 CUDA-core
 *     chunked path.  Both are GPU kernels; there is no CPU path.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#if defined(__GNUC__)
#define KDA_API __attribute__((visibility("default")))
#else
#define KDA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kda_status {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1,  /* null pointer, negative size, bad cu_seqlens, ... */
    KDA_ERR_UNSUPPORTED = 2,  /* shape / dtype / chunk combination not built     */
    KDA_ERR_WORKSPACE = 3,    /* workspace missing, too small or misaligned      */
    KDA_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed             */
    KDA_ERR_TIMEOUT = 5,      /* a kernel gave up waiting (device status only)    */
    KDA_ERR_PRECONDITION = 6, /* debug library: an input outside its stated range
                                 (device status only)                             */
    KDA_ERR_DEVICE_CHECK = 7  /* debug library: a kernel found an index outside its
                                 buffer and skipped the access (device status)    */
} kda_status;

typedef enum kda_dtype {
    KDA_FP32 = 0,             /* q, k, v and O are float                          */
    KDA_BF16 = 1              /* q, k, v and O are bfloat16 (raw 16-bit storage)  */
} kda_dtype;

/*
 * Bytes of device workspace kda_prefill needs for this problem.  0 means none
 * (the CUDA-core path).  The figure depends only on the arguments, and it
 * assumes the worst case of one partial chunk per sequence, so it is valid for
 * any cu_seqlens with these n_seq and T_total.
 */
KDA_API size_t kda_prefill_workspace_size(int n_seq, int T_total, int H, int dk, int dv,
                                  int chunk, kda_dtype dtype);

/*
 * Chunked prefill over a packed batch of variable-length sequences.
 *
 * Computes, for each sequence n and head h independently, the recurrence above
 * over the sequence's tokens, starting from S0[n,h], and returns o_t for every
 * token and the final state.  The chunked matrix form it evaluates is the one
 * of "Kimi K3: the manos, the mythos, the legendos", section "FlashKDA
 * Algorithm" (cumulative decay, Q_decay / K_decay / K_restore, the UT
 * transform U = (I + L)^{-1} Diag(beta)(V - K_decay S_in),
 * O = Q_decay S_in + M_qk U, S_out = Diag(a_last) S_in + K_restore^T U).
 *
 * q, k       [T_total, H, dk]  dtype
 * v          [T_total, H, dv]  dtype
 * log_alpha  [T_total, H, dk]  float, natural log of the gate
 * beta       [T_total, H]      float
 * S0         [n_seq, H, dk, dv] float, or NULL for zero initial states
 * cu_seqlens [n_seq + 1] int32 device array of token offsets (0 = cu[0] <=
 *            cu[1] <= ... <= cu[n_seq] = T_total), or NULL for n_seq
 *            sequences of equal length T_total / n_seq (which must divide).
 * cu_seqlens_host  optional host copy of cu_seqlens (same values).  When
 *            given it is validated and used to size the launch exactly; when
 *            NULL a device cu_seqlens is trusted (lengths are clamped on the
 *            device so that no access leaves the arrays).
 * O          [T_total, H, dv]  dtype, written for every token; must not alias
 *            an input.
 * S_final    [n_seq, H, dk, dv] float, or NULL.  May alias S0 exactly.
 * workspace  device memory of at least kda_prefill_workspace_size(...) bytes,
 *            256-byte aligned (may be NULL when that size is 0).  Its contents
 *            on entry do not matter; the call owns it until the work completes.
 * Sequences of length 0 are allowed (their S_final is S0).
 * On the tensor-core path (bf16, dk = dv = 128, chunk 64) q, k, v, log_alpha
 * and O must be 16-byte aligned; otherwise KDA_ERR_INVALID_ARG.
 */
KDA_API kda_status kda_prefill(const void* q, const void* k, const void* v,
                       const float* log_alpha, const float* beta, const float* S0,
                       const int32_t* cu_seqlens, const int32_t* cu_seqlens_host,
                       int n_seq, int T_total, int H, int dk, int dv, int chunk,
                       kda_dtype dtype, void* O, float* S_final,
                       void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * kda_prefill that also saves the recurrent state at coarse positions, for
 * prefix caching: a linear-attention layer can only resume a cached prefix
 * from a stored state, so serving stacks keep the state every so many tokens
 * ("Kimi K3: the manos, the mythos, the legendos", section "KDA Prefix Cache
 * Management"; the "LLM architecture at trillion scale" page, section "6. Deep
 * dive: what this means for serving").
 *
 * Arguments as kda_prefill, plus:
 * ckpt_every     positive multiple of chunk: a checkpoint is the state after
 *                the first m * ckpt_every tokens of a sequence (m = 1, 2, ...,
 *                as long as m * ckpt_every <= its length)
 * ckpt           [ckpt_capacity, H, dk, dv] float device array, 16-byte
 *                aligned (else KDA_ERR_INVALID_ARG); checkpoint m of
 *                sequence n goes to index sum_{n' < n} floor(len_n' /
 *                ckpt_every) + m - 1
 * ckpt_capacity  number of checkpoints ckpt holds; when the lengths are known
 *                on the host (cu_seqlens_host, or equal lengths) a smaller
 *                capacity than needed is KDA_ERR_INVALID_ARG, otherwise
 *                checkpoints past the capacity are not written.
 */
KDA_API kda_status kda_prefill_ckpt(const void* q, const void* k, const void* v,
                            const float* log_alpha, const float* beta, const float* S0,
                            const int32_t* cu_seqlens, const int32_t* cu_seqlens_host,
                            int n_seq, int T_total, int H, int dk, int dv, int chunk,
                            kda_dtype dtype, void* O, float* S_final, int ckpt_every,
                            float* ckpt, int ckpt_capacity, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream);

/*
 * Size of the fixed device array that kda_prefill_noalloc uses as its
 * workspace (bytes).  Under CUDA's lazy module loading (the default) a device
 * reserves it when the first kda_prefill_noalloc call on that device loads
 * the code that holds it, and keeps it until the process exits.
 */
#define KDA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/*
 * kda_prefill without a caller-provided workspace.  The paper has no
 * counterpart to this call; it exists for callers that cannot allocate device
 * memory -- runtimes that own all device memory through their own fixed pool
 * and do not let libraries call cudaMalloc, plugin interfaces that give a
 * library only its inputs and outputs, and deployments whose memory footprint
 * is fixed at start-up.
 *
 * Same arguments and results as kda_prefill, minus (workspace,
 * workspace_bytes).  The workspace is a file-scope device array of
 * KDA_NOALLOC_SCRATCH_BYTES; the call allocates nothing.
 *   - Returns KDA_ERR_WORKSPACE, before launching anything, when
 *     kda_prefill_workspace_size(...) for the problem exceeds
 *     KDA_NOALLOC_SCRATCH_BYTES (e.g. more than about 500 chunk-head slots
 *     on the tensor-core path: H = 32 heads of ~900 tokens).
 *   - Every call looks up the array's device address on the current device
 *     (the device of the tensors must be current).  The first call on a
 *     device also loads the code that holds the array, which reserves its
 *     64 MiB there (KDA_ERR_CUDA if that fails): make that first call at
 *     start-up, before a fixed-pool runtime takes its pool and before any
 *     stream capture.
 *   - All calls on a device share the array and it keeps the last call's
 *     contents (nothing in it needs to start at zero).  Calls that overlap
 *     on the GPU race on it: order them on one stream.
 */
KDA_API kda_status kda_prefill_noalloc(const void* q, const void* k, const void* v,
                               const float* log_alpha, const float* beta, const float* S0,
                               const int32_t* cu_seqlens, const int32_t* cu_seqlens_host,
                               int n_seq, int T_total, int H, int dk, int dv, int chunk,
                               kda_dtype dtype, void* O, float* S_final, cudaStream_t stream);

/*
 * Fused parameter-free prologue.  The Kimi Linear layer L2-normalises q and k
 * before the operator ("Kimi K3: the manos, the mythos, the legendos",
 * section "Kimi Linear") and keeps the log-decay inside (-5, 0) ("LLM
 * architecture at trillion scale", section "The KDA update, in plain words").
 * The *_fused entries take those inputs before the activations and apply, in
 * fp32 inside the kernels, per (token, head):
 *   q <- q / sqrt(sum_i q_i^2 + 1e-6),  k <- k / sqrt(sum_i k_i^2 + 1e-6)
 *   log_alpha = clamp(-softplus(gate), -5, -1e-4)      (per key channel)
 *   beta = sigmoid(beta_logit)
 * and then compute exactly what kda_prefill / kda_decode compute.
 *
 * kda_prefill_fused: arguments as kda_prefill, with
 *   q, k        [T_total, H, dk] dtype, not normalised
 *   gate        [T_total, H, dk] float, pre-activation of the log-decay
 *   beta_logit  [T_total, H] float, pre-activation of beta
 * (workspace from kda_prefill_workspace_size, as for kda_prefill).
 */
KDA_API kda_status kda_prefill_fused(const void* q, const void* k, const void* v,
                             const float* gate, const float* beta_logit, const float* S0,
                             const int32_t* cu_seqlens, const int32_t* cu_seqlens_host,
                             int n_seq, int T_total, int H, int dk, int dv, int chunk,
                             kda_dtype dtype, void* O, float* S_final, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream);

/*
 * kda_decode_fused: one decode step as kda_decode, with q, k [N, H, dk] not
 * normalised, gate [N, H, dk] and beta_logit [N, H] pre-activations (see
 * kda_prefill_fused for the prologue).
 */
KDA_API kda_status kda_decode_fused(const void* q, const void* k, const void* v,
                            const float* gate, const float* beta_logit, float* S, int N, int H,
                            int dk, int dv, kda_dtype dtype, void* o, cudaStream_t stream);

/*
 * One decode step for N independent sequences (one token each), the per-token
 * form u = beta (v - (D S)^T k), S <- D S + k u^T, o = S^T q of "Kimi K3: the
 * manos, the mythos, the legendos", section "FlashKDA Algorithm".
 *
 * q, k       [N, H, dk] dtype;  v [N, H, dv] dtype
 * log_alpha  [N, H, dk] float;  beta [N, H] float
 * S          [N, H, dk, dv] float, read and overwritten in place; 16-byte
 *            aligned (it moves as float4 vectors), else KDA_ERR_INVALID_ARG
 * o          [N, H, dv] dtype, written; must not alias an input.
 * N = 0 returns KDA_OK and launches nothing.
 */
KDA_API kda_status kda_decode(const void* q, const void* k, const void* v,
                      const float* log_alpha, const float* beta, float* S,
                      int N, int H, int dk, int dv, kda_dtype dtype, void* o,
                      cudaStream_t stream);

/*
 * Multi-token verify step for speculative decoding: the "LLM architecture at
 * trillion scale" page (section "6. Deep dive: what this means for serving")
 * has a draft model propose up to 7 tokens that the big model then checks.
 * For each of N sequences, K proposed tokens (K <= 16) are run through the
 * recurrence from the state S, every o_t is returned, and S is overwritten
 * with the state after the first commit_len[n] tokens only (0 leaves S as
 * it was; the rest of the proposal is not committed).
 *
 * q, k       [N, K, H, dk] dtype;  v [N, K, H, dv] dtype
 * log_alpha  [N, K, H, dk] float;  beta [N, K, H] float
 * S          [N, H, dk, dv] float, read, and written after commit_len tokens;
 *            16-byte aligned, else KDA_ERR_INVALID_ARG
 * commit_len [N] int32 device array, values clamped to [0, K]; NULL = K
 * K > 16 is KDA_ERR_UNSUPPORTED; N = 0 or K = 0 returns KDA_OK.
 * o          [N, K, H, dv] dtype, or NULL to skip the outputs
 * A typical use calls it twice: once with commit_len all 0 to get the
 * outputs, then, once the accepted lengths are known, with o = NULL and
 * commit_len = the accepted lengths.
 */
KDA_API kda_status kda_decode_multi(const void* q, const void* k, const void* v,
                            const float* log_alpha, const float* beta, float* S,
                            const int32_t* commit_len, int N, int K, int H, int dk, int dv,
                            kda_dtype dtype, void* o, cudaStream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Serving step of a model that mixes KDA layers with softmax-attention layers
 * of grouped query heads (keys and values of one head size, 32, 64 or 128; latent
 * attention has its own calls below).  The attention layers keep keys and values in a paged cache:
 *
 *   k_cache, v_cache  [n_pages, H_kv, page_size, d] dtype, 16-byte aligned
 *   slot              page * page_size + (place inside the page)
 *   block_table       [N, max_blocks] int32: page of every page_size tokens of
 *                     each request, in order
 *
 * page_size is 16, 32, 64, 128 or 256; N is at most KDA_MAX_STEP_REQUESTS.
 * The order of a step: kda_build_block_tables once, then per attention layer
 * kda_cache_append and kda_paged_attention; with drafted tokens,
 * kda_verify_draft at the end, whose commit_len is what kda_decode_multi takes
 * for the KDA layers.  Every length is read on the device, so a captured graph
 * serves any lengths that its buffers hold.
 */
#define KDA_MAX_STEP_REQUESTS 8192
/* Most tokens that a request's row of the block table may cover in kda_paged_attention
 * (max_blocks * page_size): positions and the ends of key tiles are 32-bit numbers. */
#define KDA_MAX_STEP_POSITIONS (INT32_MAX - 511)

/*
 * Block tables and slot map of one step.  Request n holds ctx_len[n] cached
 * tokens and adds new_len[n] (negative lengths count as 0).  Its table already
 * names the pages of the cached tokens; the pages for the new ones,
 * ceil((ctx + new) / page_size) - ceil(ctx / page_size) of them, are taken from
 * free_pages in request order and written into its row.
 *
 * ctx_len, new_len [N] int32
 * free_pages       [n_free] int32 (may be NULL when n_free is 0)
 * block_table      [N, max_blocks] int32, updated in place; only the entries
 *                  of newly taken pages are written
 * cu_seqlens       [N + 1] int32, written: offsets of each request's new tokens
 *                  (the packed batch of kda_prefill and kda_paged_attention)
 * seq_len          [N] int32, written: ctx + new
 * slot_map         [n_tokens] int64, written: slot of each new token; -1 for
 *                  the padding behind the last one, and where there is no page
 * positions        [n_tokens] int32 or NULL, written: position of each new
 *                  token in its request; 0 for the padding
 * n_taken          [1] int32, written: pages needed.  More than n_free means
 *                  that the free list ran out: the entries without a page are
 *                  -1, and the calls below leave their tokens out.
 * No output may lie over ctx_len, new_len or free_pages.
 * n_tokens is the size of slot_map; new tokens past it get no slot.  Tokens
 * past max_blocks * page_size get no page.  The new tokens of all requests
 * together must stay below 2^31, and so must the tokens (ctx + new) of each.
 */
KDA_API kda_status kda_build_block_tables(const int32_t* ctx_len, const int32_t* new_len,
                                  const int32_t* free_pages, int n_free, int N, int max_blocks,
                                  int page_size, int n_tokens, int32_t* block_table,
                                  int32_t* cu_seqlens, int32_t* seq_len, int64_t* slot_map,
                                  int32_t* positions, int32_t* n_taken, cudaStream_t stream);

/*
 * Writes the keys and values of T new tokens into the paged cache: row t goes
 * to slot_map[t]; slots below 0 or at and past n_pages * page_size are skipped.
 *
 * k, v      [T, H_kv, d] dtype; consecutive tokens are k_stride and v_stride
 *           elements apart (at least H_kv * d, so that both may be slices of a
 *           fused projection); any alignment of the elements
 * slot_map  [T] int64.  What a slot named by two tokens holds is unspecified: each
 *           piece of its row is either one's.
 */
KDA_API kda_status kda_cache_append(const void* k, const void* v, const int64_t* slot_map,
                            int64_t k_stride, int64_t v_stride, int T, int H_kv, int d, int page_size,
                            int n_pages, kda_dtype dtype, void* k_cache, void* v_cache,
                            cudaStream_t stream);

/* Bytes of device workspace kda_paged_attention needs for T new tokens. */
KDA_API size_t kda_paged_attention_workspace_size(int T, int H_q, int H_kv, int d, kda_dtype dtype);

/*
 * Attention of new tokens over a paged cache that holds their own keys and
 * values already.  Token i of the m = cu_seqlens[n + 1] - cu_seqlens[n] new
 * tokens of request n stands at position p = seq_len[n] - m + i and sees the
 * keys j <= p, with window > 0 only those with j > p - window.  Per query head
 * h, over the head h / (H_q / H_kv) of the cache:
 *
 *     o = sum_j exp(scale q.k_j - lse) v_j,   lse = ln sum_j exp(scale q.k_j)
 *
 * One call serves any mix of single tokens (decode), a few tokens (verify) and
 * long chunks (prefill).  A row that sees no key gives o = 0, lse = -inf.
 * Keys whose block_table entry names no page of the cache (below 0, n_pages or
 * more) are left out, as are keys past max_blocks * page_size.  What stands in
 * the cache at places that a row does not see, NaN among it, does not reach
 * that row.
 *
 * q           [T, H_q, d] dtype, consecutive tokens q_stride elements apart
 * cu_seqlens  [N + 1] int32 device array, 0 = cu[0] <= ... <= cu[N] <= T;
 *             rows of q at and past cu[N] are padding, their o is not written
 * seq_len     [N] int32 device array
 * scale       > 0 and at most 2^127.  A row whose largest score, times log2(e), is past the range
 *             of fp32 becomes NaN, on the tensor-core path one whose largest is 2^29 or more
 *             from 0
 * window      0: no window
 * max_blocks  at most KDA_MAX_STEP_POSITIONS / page_size
 * o           [T, H_q, d] dtype;  lse [T, H_q] float or NULL
 * workspace   kda_paged_attention_workspace_size bytes, 256-byte aligned
 * d is 32, 64 or 128; H_q a multiple of H_kv.  The scores, their statistics and
 * the sums are fp32; on the tensor-core path (bf16, q 16-byte aligned with a
 * stride that is a multiple of 8) the weights enter the second product as bf16.
 * fp32 tensors, and bf16 with other rows of q, run in fp32 on CUDA cores.
 */
KDA_API kda_status kda_paged_attention(const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_table, const int32_t* cu_seqlens,
                               const int32_t* seq_len, int64_t q_stride, int N, int T, int H_q,
                               int H_kv, int d, int page_size, int max_blocks, int n_pages,
                               float scale, int window, kda_dtype dtype, void* o, float* lse,
                               void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Latent attention.  A layer may keep, of each token, one latent vector of 512
 * channels that all heads share and a rotated key part of 64 channels beside it:
 *
 *   cache  [n_pages, page_size, 576] dtype, 16-byte aligned: the latent, then the
 *          key part; slots and block tables as above
 *
 * and has two forms.  Absorbed (kda_latent_attention): the query holds the key
 * projection already, 512 + 64 channels a head against a cache row, and the latents
 * are the values, 512 channels a head of output.  Expanded (kda_expanded_attention): keys
 * and values were projected from the latents again, 128 + 64 channels of a key (the 64
 * shared by the heads) and 128 of a value.  Single tokens and a few of them take the
 * first, prompts the second.  kda_rotary turns queries, and the key parts that go into the
 * expanded form; kda_latent_append turns the cache's on their way.
 */

/*
 * Rotary positions.  Of each head's d channels the first `rot` are turned in
 * rot / 2 pairs: pair i of a token at position p, with angle w = p * inv_freq[i],
 *     (a, b) -> factor (a cos w - b sin w, b cos w + a sin w)
 * is channels (2 i, 2 i + 1) when `interleaved`, else (i, i + rot / 2).  The other
 * channels are copied.  For every int32 position and frequency below 1 (radians a
 * position) the angle is formed to 2^-33 turns, and what is left of it beside the nearest
 * quarter turn is rounded to fp32 (2^-24 of it, 2^-28 turns at most); sine, cosine and
 * products are fp32.
 *
 * x, out     [T, H, d] dtype, strides in elements, the channels contiguous.  out may be
 *            x itself with the same strides (the other channels then stay as they
 *            are), else the two may share no element; the rows of out may not overlap
 * positions  [T] int32;  inv_freq [rot / 2] float, both device arrays
 * factor     finite; multiplies what is turned
 * rot is even; d is at most 256 (more: KDA_ERR_UNSUPPORTED).
 */
KDA_API kda_status kda_rotary(const void* x, const int32_t* positions, const float* inv_freq, int64_t x_token_stride,
                      int64_t x_head_stride, int64_t out_token_stride, int64_t out_head_stride, int T, int H, int d,
                      int rot, int interleaved, float factor, kda_dtype dtype, void* out, cudaStream_t stream);

/*
 * Writes the latents and key parts of T new tokens into the paged latent cache, the
 * key part turned by its token's position on the way (as kda_rotary does with 64 of 64
 * channels).  Row t goes to slot_map[t]; slots below 0 or at and past
 * n_pages * page_size are skipped.
 *
 * c          [T, 512] dtype, k_rope [T, 64] dtype: consecutive tokens are c_stride
 *            and k_rope_stride elements apart, at least 512 and 64 (both may be slices of
 *            one projection, but not of the cache)
 * slot_map   [T] int64.  What a slot named by two tokens holds is unspecified: each
 *            piece of its row is either one's.
 * positions  [T] int32, inv_freq [32] float; both NULL: the key part is copied
 */
KDA_API kda_status kda_latent_append(const void* c, const void* k_rope, const int64_t* slot_map, const int32_t* positions,
                             const float* inv_freq, int64_t c_stride, int64_t k_rope_stride, int T, int page_size,
                             int n_pages, int interleaved, float factor, kda_dtype dtype, void* cache,
                             cudaStream_t stream);

/* Bytes of device workspace kda_latent_attention needs for T new tokens. */
KDA_API size_t kda_latent_attention_workspace_size(int T, int H, kda_dtype dtype);

/*
 * Absorbed attention of new tokens over a paged latent cache that holds their own
 * rows already.  Token i of the m = cu_seqlens[n + 1] - cu_seqlens[n] new tokens of
 * request n stands at position p = seq_len[n] - m + i and sees the cache rows c_j,
 * j <= p, of its request.  Per head h:
 *
 *     o = sum_j exp(scale q.c_j - lse) c_j[0 .. 511],   lse = ln sum_j exp(scale q.c_j)
 *
 * One call serves any mix of single tokens (decode), a few tokens (verify) and chunks.
 * A row that sees no key gives o = 0, lse = -inf.  Keys whose block_table entry names
 * no page of the cache are left out, as are keys past max_blocks * page_size.  What
 * stands in the cache at places that a row does not see, NaN among it, does not reach
 * that row.  A latent channel that is not finite makes that channel NaN in the rows
 * that see it, and the whole row unless the key scores -inf (its weight is then 0).
 *
 * q           [T, H, 576] dtype, consecutive tokens q_stride elements apart, at least H * 576
 * cu_seqlens  [N + 1] int32 device array, 0 = cu[0] <= ... <= cu[N] <= T;
 *             rows of q at and past cu[N] are padding, their o is not written
 * seq_len     [N] int32 device array
 * scale       > 0 and at most 2^127 (of the expanded head: usually 192^-1/2).  A row whose
 *             largest score, times log2(e), is past the range of fp32 becomes NaN, on the
 *             tensor-core path one whose largest is 2^29 or more from 0
 * max_blocks  at most KDA_MAX_STEP_POSITIONS / page_size
 * o           [T, H, 512] dtype, 32-byte aligned;  lse [T, H] float or NULL
 * workspace   kda_latent_attention_workspace_size bytes, 256-byte aligned; a call has it to
 *             itself until it is complete
 * The scores, their statistics and the sums are fp32; on the tensor-core path (bf16, q
 * 16-byte aligned with a stride that is a multiple of 8) the weights enter the second product
 * as bf16.  fp32 tensors, and bf16 with other rows of q, run in fp32 on CUDA cores.
 */
KDA_API kda_status kda_latent_attention(const void* q, const void* cache, const int32_t* block_table,
                                const int32_t* cu_seqlens, const int32_t* seq_len, int64_t q_stride, int N, int T, int H,
                                int page_size, int max_blocks, int n_pages, float scale, kda_dtype dtype, void* o,
                                float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Bytes of device workspace kda_expanded_attention needs for T new tokens. */
KDA_API size_t kda_expanded_attention_workspace_size(int T, int H, kda_dtype dtype);

/*
 * Expanded attention over packed keys and values.  Request n has the rows
 * cu_seqlens[n] .. cu_seqlens[n + 1] - 1 of q (m of them) and the rows
 * cu_seqlens_k[n] .. of the keys and values (s of them).  When `causal`, token i stands
 * at position s - m + i and sees the keys j up to its own; else every token sees all
 * keys of its request (an earlier part of the context, whose result is joined to the
 * rest by the lse).  Per head h:
 *
 *     z_j = scale (q[0 .. 127].k_nope[j, h] + q[128 .. 191].k_rope[j])
 *     o = sum_j exp(z_j - lse) v[j, h],   lse = ln sum_j exp(z_j)
 *
 * A row that sees no key gives o = 0, lse = -inf.  What stands in the keys and values at
 * places that a row does not see, NaN among it, does not reach that row.  A value that is
 * not finite makes its channel infinite or NaN in the rows that see it (either, where its
 * weight is 0 in fp32).
 *
 * q             [T, H, 192] dtype, consecutive tokens q_stride elements apart, at least H * 192
 * k_nope, v     [S, H, 128] dtype, token and head strides in elements (both may be slices of
 *               one projection; tokens and heads may lie in either order).  Rows may not
 *               overlap, but a head stride of 0 gives all heads the same ones;
 *               k_rope [S, 64] dtype, tokens k_rope_stride elements apart, at least 64
 * cu_seqlens, cu_seqlens_k  [N + 1] int32 device arrays, rising from 0, at most T and S
 *               at the end; rows of q at and past cu_seqlens[N] are padding, their o is
 *               not written
 * S + T         at most KDA_MAX_STEP_POSITIONS
 * scale         > 0 and at most 2^127.  A row whose largest score, times log2(e), is past the
 *               range of fp32 becomes NaN, on the tensor-core path one whose largest is 2^29
 *               or more from 0
 * o             [T, H, 128] dtype, 32-byte aligned;  lse [T, H] float or NULL
 * workspace     kda_expanded_attention_workspace_size bytes, 256-byte aligned; a call has it
 *               to itself until it is complete
 * The scores, their statistics and the sums are fp32; on the tensor-core path (bf16, all rows
 * on 16-byte boundaries, each head its own) the weights enter the second product as bf16.  fp32
 * tensors, and bf16 with other rows, run in fp32 on CUDA cores.
 */
KDA_API kda_status kda_expanded_attention(const void* q, const void* k_nope, const void* k_rope, const void* v,
                                  const int32_t* cu_seqlens, const int32_t* cu_seqlens_k, int64_t q_stride,
                                  int64_t k_token_stride, int64_t k_head_stride, int64_t k_rope_stride,
                                  int64_t v_token_stride, int64_t v_head_stride, int N, int T, int S, int H, float scale,
                                  int causal, kda_dtype dtype, void* o, float* lse, void* workspace,
                                  size_t workspace_bytes, cudaStream_t stream);

/*
 * Verification of drafted tokens against the target's probabilities.  Request
 * n has L = draft_len[n] drafted tokens x_0 ... (at most K).  With p_i the
 * target's and q_i the draft's distribution at draft i, x_i stands while
 * u_i q_i(x_i) < p_i(x_i); with a the number of tokens that stand, one more
 * token is drawn with u_K: from max(p_a - q_a, 0) if a < L, from p_a if a = L
 * (and from p_a where max(p_a - q_a, 0) is zero everywhere).  The drawn token
 * is the first one at which the running sum exceeds u_K times the whole sum.
 *
 * target        [N, K + 1, V] dtype, probabilities in [0, 1], each row summing
 *               to about 1 (less than 4)
 * draft         [N, K, V] dtype, likewise; NULL for tokens proposed with
 *               certainty (q_i = 1 at x_i, 0 elsewhere)
 * draft_tokens  [N, K] int32; a token outside [0, V) does not stand
 * uniforms      [N, K + 1] float in [0, 1)
 * draft_len     [N] int32 clamped to [0, K], or NULL (= K)
 * tokens        [N, K + 1] int32, written: the tokens that stand, the drawn
 *               one, then -1
 * commit_len    [N] int32, written: a + 1, the number of tokens to commit when
 *               the request's last token and its drafts were run through
 *               kda_decode_multi as K + 1 tokens
 * Sums are exact to 2^-60 of a probability, in integers: no order of summation
 * enters the result.  Negative and NaN probabilities count as 0, except that a
 * token whose own p or q is NaN does not stand.  A target row
 * without a positive entry draws V - 1.  K is at most 16, V at most 2^30.
 */
KDA_API kda_status kda_verify_draft(const void* target, const void* draft, const int32_t* draft_tokens,
                            const float* uniforms, const int32_t* draft_len, int N, int K, int V,
                            kda_dtype dtype, int32_t* tokens, int32_t* commit_len,
                            cudaStream_t stream);

/*
 * Synchronises `stream`, then returns and clears the device status word:
 * KDA_OK, or KDA_ERR_TIMEOUT if a kernel since the last call gave up waiting
 * (its outputs are then incomplete), or KDA_ERR_CUDA if the synchronisation
 * itself failed.  The word is per device and shared by all streams.
 */
KDA_API kda_status kda_get_last_device_status(cudaStream_t stream);

/*
 * Check of the failure detection above (the pages have no counterpart; it
 * computes nothing of KDA): one kernel waits on an mbarrier that nothing
 * completes, with the same bounded wait the kernels use, for at most
 * `limit_cycles` SM clock cycles (0 ... ~4e9, the kernels' own limit of about
 * two seconds).  Afterwards kda_get_last_device_status returns KDA_ERR_TIMEOUT
 * and the device stays usable.  KDA_ERR_INVALID_ARG for a limit outside that
 * range, before anything is launched.
 */
KDA_API kda_status kda_check_wait_timeout(long long limit_cycles, cudaStream_t stream);

/*
 * Tracing hook.  While set, every kda_prefill / kda_decode call made from the
 * calling host thread records the given CUDA events (cudaEvent_t handles,
 * created by the caller) on its stream at the boundaries between the kernels
 * it launches, all on the caller's stream: event 0 before the first kernel;
 * for the tensor-core prefill, event 1 once every chunk-prep kernel has run
 * and event 2 when the state pass (which may run partly on an internal
 * stream, overlapped with later chunk preps, or as a segment scan of three
 * kernels for few long sequences) has finished on the caller's stream; for the
 * CUDA-core prefill and the decode, event 1 after their one kernel.  Events beyond
 * n_events are skipped.  Pass (NULL, 0) to stop.  Returns KDA_ERR_INVALID_ARG
 * for n_events < 0 or a NULL array with n_events > 0.  The array must stay
 * valid while the hook is set.  This exists so that a benchmark can time each
 * kernel with CUDA events on the stream the kernel runs on.
 */
KDA_API kda_status kda_set_trace_events(void* const* events, int n_events);

/*
 * Debug variant.  The library is also built as libkda_debug.so, compiled with
 * KDA_DEBUG: the same entry points with the same results, plus checks that the
 * release library leaves out for speed.
 *   - Precondition: before each kda_prefill, kda_prefill_ckpt,
 *     kda_prefill_noalloc, kda_decode and kda_decode_multi call, one pass over
 *     log_alpha records KDA_ERR_PRECONDITION in the device status word when a
 *     value lies outside [-5, 0] or is not a number.  That is the log-decay
 *     bound of "LLM architecture at trillion scale", section "The KDA update,
 *     in plain words", inside which the chunked form's staged decay factors
 *     stay finite and the accuracy target is stated; the call still computes.
 *     (The *_fused calls clamp the log-decay themselves and are not checked.)
 *   - Device checks: the tensor-core prefill kernels check the workspace slots
 *     and segment indices they derive from the call's lengths against the sizes
 *     they were given; an index outside records KDA_ERR_DEVICE_CHECK and the
 *     access is skipped.  Nothing traps.
 * The serving-step operators are the same in both libraries: they bring lengths,
 * slots and pages from the device into their buffers' range always.
 * kda_get_last_device_status of the same library reports either code.
 * Returns 1 in the debug library, 0 in the release library.
 */
KDA_API int kda_debug_build(void);

/* Static, NUL-terminated description of a status code (never NULL). */
KDA_API const char* kda_status_string(kda_status status);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
