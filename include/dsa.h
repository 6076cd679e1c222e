/*
 * dsa.h -- C ABI of the DSA sparse-attention step for NVIDIA B200 (sm_100a).
 *
 * The step has two parts, as the pages describe it:
 *
 *  1. Index stage ("Day0 Adaptation and Performance Optimization for Novel
 *     Long-Sequence Reasoning Models", section 3; "Large Model Inference
 *     Acceleration: Day-0 Adaptation and Performance Optimization for New
 *     Architectures", section 1.1 "Indexer Fusion: Three Kernels into One"):
 *     relevance scoring of every cached position, head-weight weighting and
 *     Top-K selection in ONE kernel that reads the paged indexer-key cache in
 *     place and writes only the final index list.  The score is the Lightning
 *     Indexer form with a ReLU gate:
 *         score(t, s) = sum_h w[t,h] * max(0, q[t,h,:] . k[s,:])
 *     Ties are broken by position (the lower position wins).
 *
 *  2. Sparse read stage ("Day0 Adaptation and Sparse Attention Optimization
 *     for Long-Sequence LLM Inference", section 4): Sparse Flash Attention
 *     gathers only the selected rows of the MLA latent cache (512 latent +
 *     64 RoPE, shared by all query heads) and computes softmax attention over
 *     them: logits = sm_scale * q . row[0:576], output = softmax . row[0:512].
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers unless stated; the caller owns
 *    every buffer (inputs, outputs and the workspace).  The library never
 *    allocates or frees memory and never synchronizes the stream, except
 *    dsa_get_status(), which synchronizes by design.
 *  - Work is enqueued asynchronously on `stream` (a cudaStream_t, passed as
 *    void*; NULL = legacy default stream).  Pointers must stay valid until
 *    that work completes.
 *  - Host-side validation failures return before anything is launched.
 *    Launch failures return DSA_ERR_CUDA.  Errors found by the kernels
 *    (out-of-range block ids, a co-scheduling wait that timed out) are
 *    recorded in a status word inside the workspace and read with
 *    dsa_get_status().
 *  - Layouts are dense, row-major, with the innermost dimension last.
 *    Query tokens are sequence-major: tokens cu_q[b] .. cu_q[b+1]-1 belong to
 *    sequence b and sit at positions seq_lens[b]-nq_b .. seq_lens[b]-1; token
 *    j of a sequence sees positions 0..its own position (causal).
 *  - Paged caches: page size 64 tokens.  block_table[b, i] is the physical
 *    page holding positions 64*i .. 64*i+63 of sequence b.  The indexer-key
 *    cache and the latent cache share the table.
 */
#ifndef DSA_H_
#define DSA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define DSA_API __attribute__((visibility("default")))
#else
#define DSA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DSA_OK = 0,
    DSA_ERR_INVALID_ARG = 1,    /* a pointer, size or shape failed validation       */
    DSA_ERR_UNSUPPORTED = 2,    /* valid request outside what the kernels implement */
    DSA_ERR_WORKSPACE = 3,      /* workspace NULL, too small or misaligned          */
    DSA_ERR_CUDA = 4,           /* a CUDA runtime / driver call failed              */
    DSA_ERR_TIMEOUT = 5,        /* device: a bounded wait expired (kernel returned) */
    DSA_ERR_DEVICE_BOUNDS = 6,  /* device: block id or index out of range (skipped) */
    DSA_ERR_CAPACITY = 7        /* device: a key chunk exceeded on-chip capacity    */
} dsa_status;

typedef enum {
    DSA_KEY_BF16 = 0,           /* indexer keys: bf16 [num_blocks, 64, D_I]                       */
    DSA_KEY_FP8_E4M3 = 1,       /* indexer keys: e4m3fn codes [num_blocks, 64, D_I] (uint8) plus  */
                                /* fp32 scales [num_blocks, 64, D_I/64], one per 64 elements      */
    DSA_KEY_MXFP8 = 2           /* indexer keys in MXFP8: e4m3fn codes [num_blocks, 64, D_I]      */
                                /* (uint8) plus one shared scale per 32 elements, [num_blocks,   */
                                /* 64, D_I/32] uint8 exponents e (scale 2^(e-127)); needs MXFP8   */
                                /* queries.  "Day0 Adaptation and Performance Optimization for   */
                                /* Novel Long-Sequence Reasoning Models", section 4: full MXFP8   */
                                /* quantization of index Q/K, every 32 elements share a scale.   */
} dsa_key_dtype;

typedef enum {
    DSA_Q_BF16 = 0,             /* indexer queries: bf16 [T, H_I, D_I]                             */
    DSA_Q_MXFP8 = 1             /* indexer queries in MXFP8: e4m3fn codes [T, H_I, D_I] (uint8) in */
                                /* q_idx plus q_scale [T, H_I, D_I/32] uint8 exponents            */
} dsa_query_dtype;

/* Batch and paging description shared by all entry points. */
typedef struct {
    int32_t batch;              /* B sequences                                            */
    int32_t num_tokens;         /* T query tokens in total                                */
    const int32_t* seq_lens;    /* device [B]: cached length INCLUDING this step's tokens */
    const int32_t* cu_q;        /* device [B+1]: query-token offsets, cu_q[0] = 0         */
    const int32_t* block_table; /* device [B, max_blocks_per_seq]                         */
    int32_t max_blocks_per_seq;
    int32_t num_blocks;         /* physical pages in each cache (bounds checks)           */
    int32_t max_seq_len;        /* host-side upper bound on every seq_lens[b]             */
    int32_t max_q_per_seq;      /* host-side upper bound on cu_q[b+1] - cu_q[b]           */
} dsa_batch;

/* Indexer inputs (Lightning Indexer + Top-K). */
typedef struct {
    const void* q_idx;          /* device [T, H_I, D_I] bf16 (or e4m3 codes, see q_dtype)      */
    const float* w;             /* device [T, H_I] fp32 head weights (any sign)                */
    const void* k_cache;        /* device indexer-key cache, layout per key_dtype              */
    const float* k_scale;       /* device key scales: [num_blocks, 64, D_I/64] fp32 (fp8 keys, */
                                /* 4-byte aligned) or [num_blocks, 64, D_I/32] uint8 exponents */
                                /* (MXFP8 keys, 16-byte aligned); NULL for bf16 keys           */
    int32_t key_dtype;          /* dsa_key_dtype                                               */
    int32_t H_I;                /* indexer heads: 8, 16, 32 or 64                              */
    int32_t D_I;                /* indexer dim: 64 or 128                                      */
    int32_t K;                  /* Top-K, 1..2048                                              */
    int32_t q_dtype;            /* dsa_query_dtype (MXFP8 exactly when key_dtype is MXFP8)     */
    const uint8_t* q_scale;     /* device [T, H_I, D_I/32] exponents of MXFP8 queries, or NULL */
} dsa_indexer_inputs;

typedef enum {
    DSA_KV_BF16 = 0,            /* latent cache rows in bf16 [num_blocks, 64, 576]                              */
    DSA_KV_FP8 = 1              /* FP8 latent cache: e4m3fn codes [num_blocks, 64, 576] (uint8, 16-byte aligned)  */
                                /* plus fp32 scales [num_blocks, 64, 5]: one per 128-element tile of a row, the  */
                                /* fifth covering the 64 RoPE elements ("Day0 Adaptation and Performance         */
                                /* Optimization ...", section 4: FP8 KV cache per token and head, tiles of 128). */
                                /* The selected rows are dequantized to bf16 (code x scale, rounded once) into   */
                                /* the workspace, 64 tokens at a time, before the attention                      */
} dsa_kv_dtype;

/* Sparse MLA attention inputs. */
typedef struct {
    const void* q;              /* device [T, H, 576] bf16 (512 latent + 64 RoPE)   */
    const void* kv_cache;       /* device latent cache, layout per kv_dtype         */
    int32_t H;                  /* query heads, 1..128                              */
    float sm_scale;             /* softmax scale applied to q . row[0:576]          */
    int32_t kv_dtype;           /* dsa_kv_dtype                                     */
    const float* kv_scale;      /* device [num_blocks, 64, 5] fp32 (FP8), else NULL */
} dsa_attn_inputs;

/*
 * Bytes of workspace needed for this batch shape by indexer_topk (ix given),
 * sparse_mla_attn (at given) or both / dsa_decode (both given).  The
 * layout is [256-byte status area][indexer group region and published-key
 * slots, a fixed size per device][attention partial slots of tokens shared
 * by several SM pairs, a fixed size per device]; one buffer sized with both
 * serves all three entry points, for any mix of shapes.  With an FP8 latent
 * cache (at->kv_dtype) a staging region follows: the selected rows of up to
 * 64 tokens as bf16 plus their per-token batch (sized for ix->K, or for
 * K = 2048 when ix is NULL); its contents are scratch.
 * The workspace must be 256-byte aligned and ZERO-FILLED before its first
 * use.  After that the library keeps it consistent by itself (a call that
 * completes without a device error leaves its histograms zero and its
 * barrier words at rest), so it can be reused by later calls on the same
 * stream; the caller must not modify it.  After a device error
 * (dsa_get_status != OK) zero-fill it again.  Calls sharing one workspace
 * must not overlap in time.
 * Status area: int32 word 0 is the device status read by dsa_get_status.
 * Words 1 and 2 are test hooks of the library's own failure tests and must
 * stay zero in normal use: word 1 shortens every bounded device wait to that
 * many microseconds (0 = the default of one second), word 2 injects a wait
 * that runs out (bit 0: an indexer group barrier waits for one CTA more than
 * its group has; bit 1: in the attention kernel the second CTA of each pair
 * never reports its first rows; bit 2: in dsa_chunk_attn the second CTA of each
 * pair never loads).
 * Returns 0 if the shape is invalid.
 */
DSA_API size_t dsa_workspace_size(const dsa_batch* batch, const dsa_indexer_inputs* ix,
                          const dsa_attn_inputs* at);

/*
 * Fused Lightning Indexer + Top-K.
 * out_idx   device [T, K] int32: the selected positions of each token in
 *           ascending order, -1 padded when fewer than K positions are
 *           visible (then every visible position is selected).
 * out_score device [T, K] fp32 score of each selected position (-inf on
 *           padding) or NULL.
 * Score rows are never written to global memory.
 */
DSA_API dsa_status indexer_topk(const dsa_batch* batch, const dsa_indexer_inputs* ix,
                        int32_t* out_idx, float* out_score,
                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * Sparse Flash Attention over the rows listed in idx (device [T, K] int32
 * logical positions; negative entries are skipped).
 * out device [T, H, 512] bf16; lse device [T, H] fp32 natural-log
 * log-sum-exp of the scaled logits (-inf if a token selects nothing) or NULL.
 * The launch is a programmatic dependent of the preceding kernel on the
 * stream: its prologue may overlap that kernel's end, and it reads nothing
 * (inputs, index list, workspace) before that kernel has completed.  When a
 * token's rows are spread over several SM pairs (few tokens), a second, small
 * kernel merges the pairs' partial results (normalised bf16 O and softmax
 * statistics, kept in the workspace) into out and lse.
 */
DSA_API dsa_status sparse_mla_attn(const dsa_batch* batch, const dsa_attn_inputs* at,
                           const int32_t* idx, int32_t K,
                           void* out, float* lse,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * sparse_mla_attn without a caller workspace (the pages have no counterpart:
 * this is a convenience of this library).  For callers that cannot provide
 * device memory for the workspace -- code that must not allocate on the
 * device, or that has no device allocator at hand.  The function itself
 * allocates nothing: it uses a fixed 20 MiB scratch array inside the library
 * module (status area and partial slots), which every GPU that loads the
 * library holds until the process exits.
 * Arguments, layouts and results are those of sparse_mla_attn.
 *  - The first call on a device (and the first after that device's context
 *    changes) looks up the scratch address with the device current; make it
 *    before any latency-critical use.
 *  - Each call first clears the scratch's status area on the stream (one
 *    memset), so a call that ended in a device error leaves nothing behind
 *    for later calls.
 *  - Shapes whose plan needs more scratch than 20 MiB are rejected with
 *    DSA_ERR_WORKSPACE (dsa_last_error() gives both sizes); on a 148-SM B200
 *    every shape fits.
 *  - All calls on a device share the one scratch: calls whose device work
 *    overlaps in time (other streams, other host threads) race and must not
 *    be issued.
 *  - Errors found by the kernels go to the scratch's status word, which this
 *    API does not expose; use sparse_mla_attn when device-side status is
 *    needed.
 */
DSA_API dsa_status sparse_mla_attn_static(const dsa_batch* batch, const dsa_attn_inputs* at,
                                          const int32_t* idx, int32_t K, void* out, float* lse,
                                          void* stream);

/*
 * The whole decode step: indexer_topk then sparse_mla_attn on one stream,
 * without a host synchronization in between.  out_idx [T, K] is required
 * (it carries the index list between the stages); out_score and lse may be
 * NULL.  The attention launch depends programmatically on the indexer
 * launch: its prologue and the first token's query load overlap the end of
 * the indexer, and it reads the index list only after the indexer completed.
 */
DSA_API dsa_status dsa_decode(const dsa_batch* batch, const dsa_indexer_inputs* ix,
                      const dsa_attn_inputs* at,
                      int32_t* out_idx, float* out_score, void* out, float* lse,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * Synchronizes `stream`, reads the device status word kept in `workspace`
 * (DSA_OK if no kernel reported an error since the last read) into
 * *device_status and clears it.  Returns DSA_ERR_CUDA if the stream itself
 * failed.
 */
DSA_API dsa_status dsa_get_status(void* workspace, void* stream, int32_t* device_status);

/*
 * Number of kernel launches dsa_decode enqueues for this shape (indexer
 * launches + the attention launch + the merge launch when tokens are shared
 * by several SM pairs), or -1 if the shape is invalid.  Useful for
 * sizing CUDA graphs and for launch accounting; performs no launch.
 */
DSA_API int32_t dsa_decode_launch_count(const dsa_batch* batch, const dsa_indexer_inputs* ix,
                                        const dsa_attn_inputs* at);

/*
 * Indexer prolog: the input preparation of the index stage ("Day0 Adaptation
 * and Performance Optimization for Novel Long-Sequence Reasoning Models",
 * section 3: query projection, key RMS normalization, query quantization and
 * head-weight projection, projections kept in bf16 (section 4); "Large Model
 * Inference Acceleration ...", section 1.2).  For each query token t with
 * hidden state x[t, :] and p = W . x[t, :] (fp32 accumulation of bf16 inputs):
 *     q[t, h, i] = p[h*D_I + i]
 *     k[t, i]    = p[HD + i] / sqrt(mean_j p[HD + j]^2 + eps) * k_gamma[i]
 *     w[t, h]    = p[HD + D_I + h]                         (HD = H_I * D_I)
 * q is written to q_out in q_dtype (bf16, round to nearest even; or MXFP8:
 * e4m3fn codes [T, H_I, D_I] plus one shared exponent per 32 elements in
 * q_scale_out [T, H_I, D_I/32], scale 2^(floor(log2 amax) - 8)); w to w_out
 * [T, H_I] fp32; k into the token's row of the paged indexer-key cache
 * (position seq_lens[b] - nq_b + j for token j of sequence b, page from the
 * block table) in key_dtype: bf16; e4m3fn codes with one fp32 scale
 * amax/448 per 64 elements in k_scale [num_blocks, 64, D_I/64]; or MXFP8
 * codes with k_scale [num_blocks, 64, D_I/32] exponents.  e4m3fn codes are
 * rounded to nearest even and saturated at +-448; a zero is stored as +0.
 * All four come out of one kernel (a tensor-core GEMM over the stacked weight
 * rows with the normalization and encoding applied to its accumulators).
 */
typedef enum {
    DSA_W_ROW_MAJOR = 0,        /* w_proj row-major [H_I*D_I + D_I + H_I, d_model]                          */
    DSA_W_TILE_PACKED = 1       /* w_proj as written by indexer_prolog_pack: each 128-row x 64-column block */
                                /* contiguous, so that the weights stream from HBM in 16 KB pieces         */
} dsa_weight_layout;

typedef struct {
    const void* x;              /* device [T, d_model] bf16 hidden states of the step's tokens, 16-byte aligned */
    const void* w_proj;         /* device [H_I*D_I + D_I + H_I, d_model] bf16, 16-byte aligned: the query    */
                                /* rows (head h, element i at row h*D_I + i), then the D_I key rows, then   */
                                /* the H_I head-weight rows                                                 */
    const float* k_gamma;       /* device [D_I] key RMS-normalization weight                                */
    float eps;                  /* RMS-normalization epsilon, >= 0                                           */
    int32_t d_model;            /* hidden size: a multiple of 8                                              */
    int32_t H_I;                /* 8, 16, 32 or 64                                                           */
    int32_t D_I;                /* 64 or 128                                                                 */
    int32_t key_dtype;          /* dsa_key_dtype of the key cache written                                    */
    int32_t q_dtype;            /* dsa_query_dtype of q_out (MXFP8 exactly when key_dtype is MXFP8)          */
    int32_t w_layout;           /* dsa_weight_layout of w_proj                                               */
} dsa_prolog_inputs;

/*
 * Bytes of the tile-packed copy of the prolog weights (0 for invalid sizes):
 * ceil(n_out/128) * ceil(d_model/64) blocks of 128 x 64 bf16, n_out =
 * H_I*D_I + D_I + H_I.  Block (i, j) holds rows 128i.. and columns 64j.. of
 * the row-major matrix (zeros past its edges), row-major, at element offset
 * (i * ceil(d_model/64) + j) * 8192.
 */
DSA_API size_t dsa_prolog_packed_bytes(int32_t H_I, int32_t D_I, int32_t d_model);

/*
 * Writes the tile-packed copy of the row-major prolog weights w_proj into
 * w_packed (dsa_prolog_packed_bytes bytes, 16-byte aligned; both device
 * pointers), enqueued on `stream`.  Done once when the weights are loaded
 * ("Day0 Adaptation and Performance Optimization ...", section 2: hardware-
 * friendly weight layouts).  Returns DSA_ERR_INVALID_ARG for bad sizes or
 * pointers, DSA_ERR_CUDA if the launch fails.
 */
DSA_API dsa_status indexer_prolog_pack(const void* w_proj, void* w_packed, int32_t H_I, int32_t D_I,
                                       int32_t d_model, void* stream);

/*
 * Bytes of workspace indexer_prolog needs for this shape (0 if the arguments
 * are invalid).  Layout: [256-byte status area][split counters][fp32 partial
 * tiles when the contraction is split along d_model].  The status area and
 * the counters must be zero-filled before the first call and stay so after
 * every successful call; the partial tiles are scratch, so a workspace that
 * indexer_prolog has used must be zero-filled again before indexer_topk,
 * sparse_mla_attn or dsa_decode use it.
 */
DSA_API size_t dsa_prolog_workspace_size(const dsa_batch* batch, const dsa_prolog_inputs* pr);

/*
 * Runs the prolog for the batch's T tokens (batch->max_seq_len and
 * max_q_per_seq are not used).  Outputs: q_out (bf16 [T, H_I, D_I], or e4m3
 * codes with q_scale_out for MXFP8), w_out [T, H_I] fp32, and the tokens'
 * rows of k_cache / k_scale (layouts of dsa_indexer_inputs); no other cache
 * row is touched.  A token whose page id is out of range is skipped and
 * recorded as DSA_ERR_DEVICE_BOUNDS in the status word.  Returns
 * DSA_ERR_INVALID_ARG / DSA_ERR_UNSUPPORTED / DSA_ERR_WORKSPACE before
 * launching anything, DSA_ERR_CUDA if the launch fails.
 */
DSA_API dsa_status indexer_prolog(const dsa_batch* batch, const dsa_prolog_inputs* pr, void* q_out,
                                  uint8_t* q_scale_out, float* w_out, void* k_cache, void* k_scale,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * Norm and rotation of queries and keys, with the write of the keys into the
 * paged cache: what stands between the projections and the attention of this
 * library (the prolog above makes indexer inputs and does not rotate).
 * For each query head x = q[t, h, :] and each token's key x = k[t, :] of D
 * elements (an MLA row: 512 latent + 64 RoPE; an indexer row: D_I):
 *     y_i = x_i * gamma_i / sqrt(mean_{j < n} x_j^2 + eps)    for i < n
 *     y_i = x_i                                               for i >= n
 * with n = q_norm or k_norm (0: no norm), then the elements
 * [rope_off, rope_off + rope_dim) are rotated in pairs by the angles
 * pos * inv_freq[i]: (a, b) -> (a cos - b sin, b cos + a sin), pairs being
 * (i, i + rope_dim/2), or (2i, 2i + 1) when interleaved.  pos is positions[t],
 * or the token's place in its sequence when positions is NULL.  The angle is
 * formed in 64 bits, statistics and products in 32; each result is rounded
 * once.
 * q_out [T, H, D] bf16, dense; it may be q itself when q is dense, and must not
 * overlap q otherwise.  k goes to the cache row of the token's place in its
 * sequence (seq_lens[b] - nq_b + j, page from the block table): bf16 rows
 * [num_blocks, 64, D], or with kv_dtype DSA_KV_FP8 (D = 576 only) e4m3fn codes
 * plus k_scale [num_blocks, 64, 5], scale amax/448 of each 128 elements (1
 * where that is zero), codes rounded to nearest even, a zero stored as +0.  No
 * other cache row is touched.  Two tokens must not share a cache row.
 * Rows of q_out behind the last sequence (t >= cu_q[B], a padded batch) are
 * left as they were.  A key whose page id or position is out of range is
 * skipped and recorded as DSA_ERR_DEVICE_BOUNDS.
 * q may be NULL (keys only), and k may be NULL (queries only; block_table is
 * not read then).  batch->max_seq_len and max_q_per_seq are not used.
 */
typedef struct {
    const void* q;              /* device [T, H, D] bf16, 16-byte aligned, or NULL                          */
    int64_t q_stride_t;         /* elements from one token (head) of q to the next: multiples of 8, >= 0    */
    int64_t q_stride_h;
    const void* k;              /* device [T, D] bf16, 16-byte aligned, or NULL                             */
    int64_t k_stride_t;         /* elements from one token of k to the next: a multiple of 8, >= 0          */
    int32_t H;                  /* query heads, >= 1                                                        */
    int32_t D;                  /* elements per row: a multiple of 8, up to 1024                            */
    const float* q_gamma;       /* device [q_norm] fp32, 16-byte aligned (NULL when q_norm is 0)            */
    const float* k_gamma;       /* device [k_norm] fp32, 16-byte aligned (NULL when k_norm is 0)            */
    int32_t q_norm;             /* leading elements that are normalized: a multiple of 8, 0..D              */
    int32_t k_norm;
    float eps;                  /* >= 0                                                                     */
    const float* inv_freq;      /* device [rope_dim / 2] fp32 angles per position (NULL when rope_dim is 0) */
    int32_t rope_dim;           /* rotated elements: a multiple of 16 (0: none)                             */
    int32_t rope_off;           /* first rotated element: a multiple of 8                                   */
    int32_t interleaved;        /* 0: pairs (i, i + rope_dim/2); 1: pairs (2i, 2i + 1)                      */
    const int32_t* positions;   /* device [T] rotation positions, or NULL                                   */
    int32_t kv_dtype;           /* dsa_kv_dtype of the cache that k is written to                           */
} dsa_rope_inputs;

/*
 * One launch.  status is a status area (256 bytes, zero-filled before its
 * first use; the start of any workspace of this library serves) that
 * dsa_get_status reads; it may be NULL when k is NULL.  No workspace is used.
 * Returns DSA_ERR_INVALID_ARG / DSA_ERR_UNSUPPORTED before launching anything,
 * DSA_ERR_CUDA if the launch fails.
 */
DSA_API dsa_status dsa_qk_norm_rope(const dsa_batch* batch, const dsa_rope_inputs* in, void* q_out, void* k_cache,
                                    float* k_scale, void* status, void* stream);

/*
 * Dense attention of new tokens over the paged latent cache: every query token
 * attends to all positions up to its own (chunks of a prompt, single tokens,
 * tokens to verify; layers and contexts that stay dense beside the sparse
 * attention above).  With p_t = seq_lens[b] - nq_b + j the position of token j
 * of sequence b (its latent row and the ones before it are in the cache):
 *     S[t,h,s] = sm_scale * q[t,h,:] . row_s[0:576]     for s = 0..p_t
 *     out[t,h,:] = sum_s softmax(S[t,h,:])_s row_s[0:512]
 *     lse[t,h] = log sum_s exp(S[t,h,s])
 * q, cache formats and block tables are those of sparse_mla_attn.  Over an FP8
 * cache the scores are fp32 sums of the codes' products, times the scales (the 64
 * RoPE elements take part as two fp16 values each: to 2^-21 of themselves or 2^-31 of the
 * scale before theirs, whichever is more; where their scale is more than 2^22 times that
 * one, the elements before them are rounded to 2^-31 of theirs), and the output's values
 * are rounded to fp16.  Where max_q_per_seq new tokens make 4096 (token, head) rows or
 * more, and batch x max_seq_len positions no more than 96 MiB of fp16 copy, the cache is copied into the scratch once (2304 bytes a
 * position: two fp16 values per element and a factor per page, to 2^-22 of a value or
 * 2^-29 of its page's largest scale, whichever is more).  Scales of a sequence that lie more
 * than 2^16 apart cost the small ones bits (a tile of zeros has the scale 1).
 * out device [T, H, 512] bf16; lse device [T, H] fp32 (natural log) or NULL.
 * Scores, softmax statistics and sums are fp32; the weights are rounded to
 * bf16 (fp16 over an FP8 cache) for the second product.
 * Rows of the cache at positions that a token does not see may hold anything,
 * and do not reach its result.  Rows of out and lse behind the last sequence
 * (t >= cu_q[B]) are left as they were.  Sequences without new tokens are
 * allowed.  A page id out of range, or lengths that do not fit the table, are
 * recorded as DSA_ERR_DEVICE_BOUNDS; the positions of such a page are not seen, and such a
 * length is taken as the table's.  A length below the sequence's count of new tokens is
 * recorded too: tokens at p_t < 0 see nothing, and their rows of out and lse are left as
 * they were.  So is a cu_q past num_tokens; the rows that are there keep their positions.
 *
 * status: a status area (256 bytes, zero-filled before its first use; the start
 * of any workspace of this library serves), read by dsa_get_status; calls may
 * share one.  scratch: dsa_chunk_scratch_size bytes, 256-byte aligned, of any
 * contents; it is in use until the call's work completes, and calls that may
 * overlap in time need one each.  Returns DSA_ERR_INVALID_ARG /
 * DSA_ERR_UNSUPPORTED / DSA_ERR_WORKSPACE before launching anything,
 * DSA_ERR_CUDA if a launch fails.
 */
DSA_API size_t dsa_chunk_scratch_size(const dsa_batch* batch, const dsa_attn_inputs* at);
DSA_API dsa_status dsa_chunk_attn(const dsa_batch* batch, const dsa_attn_inputs* at, void* out, float* lse,
                                  void* status, void* scratch, size_t scratch_bytes, void* stream);

/*
 * Attention weight of the cached positions: how much of their softmax weight the
 * step's new tokens gave to each position, summed over tokens and heads and added
 * to what the position had,
 *     weight[b, s] = decay * weight[b, s]
 *                    + sum_{j, h} exp(sm_scale * q[t,h,:] . row_s[0:576] - lse[t,h])
 * over the new tokens j of sequence b that see s (s <= p_t), for every
 * s < seq_lens[b].  lse [T, H] is what dsa_chunk_attn or sparse_mla_attn returned
 * for these queries (after sparse attention the weights of positions outside the
 * selection come out as if they had been attended to under the same lse); a row
 * whose lse is -inf adds nothing.  The sums accumulate what dsa_cache_evict
 * chooses by.
 * weight device [B, stride] fp32, stride >= max_seq_len elements; entries at
 * s >= seq_lens[b], and all of a sequence without new tokens, are left as they
 * were.  decay >= 0, finite; with 0 the old weights are not read.
 * q, cache formats, block tables, status and the bounds reported there are those
 * of dsa_chunk_attn; positions of a page whose id is out of range add nothing.  An
 * FP8 cache is copied into the scratch as fp16 (two values per element and a
 * power-of-two factor per page: 2^-22 of a value, or 2^-29 of the page's largest scale),
 * which then holds max_seq_len rows of 2304 bytes for each sequence.
 * A score is one fp32 sum of 576 products on the tensor core, which leaves weights off by
 * up to 5e-6 of themselves.
 * More than max_q_per_seq new tokens of a sequence, or a length above max_seq_len,
 * are recorded as DSA_ERR_DEVICE_BOUNDS (the surplus is not counted); so is a
 * length below the count of new tokens (tokens at p_t < 0 add nothing).
 * scratch: dsa_weight_scratch_size bytes, 256-byte aligned, of any contents, one
 * each for calls that may overlap in time.  The sums are added in a fixed order:
 * equal calls give equal bits.  Errors as for dsa_chunk_attn.
 */
DSA_API size_t dsa_weight_scratch_size(const dsa_batch* batch, const dsa_attn_inputs* at);
DSA_API dsa_status dsa_attn_weight(const dsa_batch* batch, const dsa_attn_inputs* at, const float* lse, float* weight,
                                   int64_t stride, float decay, void* status, void* scratch, size_t scratch_bytes,
                                   void* stream);

/*
 * Eviction from the paged caches: of each sequence's L = seq_lens[b] positions,
 * `keep` stay (all, when L <= keep): the first `sink`, the last `recent`, and of
 * the others those with the largest weight (dsa_attn_weight's; ties and equal
 * weights: the lower position stays; -0 equals 0; NaN goes first).
 * out_idx device [B, keep] receives the positions that stay, ascending, -1 padded;
 * out_len device [B] how many.  The rows of every array are copied, in that
 * order, to the sequence's new pages: position out_idx[b, j] becomes position j,
 * in page new_table[b, j / 64].  new_weight, if given, receives their weights in
 * the same order (entries behind out_len[b] are left as they were).  Rows keep the
 * rotation they were written with, so the tokens that follow are given their
 * rotation positions explicitly (dsa_rope_inputs.positions): the cached length is
 * no longer their place in the text.
 * The arrays may be the caches themselves (dst = src) when no new page is a page
 * that any sequence of the batch still reads from here; new pages must be
 * distinct.  batch->cu_q and max_q_per_seq are not used (but checked).
 * A page id out of range is recorded as DSA_ERR_DEVICE_BOUNDS and the row is not
 * copied (without arrays no page is looked at); a length above max_seq_len likewise,
 * and is taken as max_seq_len.
 */
typedef struct {
    const void* src;            /* device [num_blocks, 64, row_bytes]                                  */
    void* dst;                  /* device [new_num_blocks, 64, row_bytes]                              */
    int64_t row_bytes;          /* bytes per position; wider copies when rows are 16-byte aligned      */
} dsa_cache_array;

typedef struct {
    const float* weight;        /* device [B, weight_stride], weight_stride >= max_seq_len             */
    int64_t weight_stride;
    float* new_weight;          /* device [B, new_weight_stride] or NULL; apart from weight             */
    int64_t new_weight_stride;  /* >= min(keep, max_seq_len)                                           */
    int32_t keep;               /* positions that stay, >= 1                                           */
    int32_t sink;               /* first positions that stay in any case, >= 0                         */
    int32_t recent;             /* last positions that stay in any case; sink + recent <= keep         */
    const int32_t* new_table;   /* device [B, new_max_blocks]                                          */
    int32_t new_max_blocks;     /* room for min(keep, max_seq_len) positions                           */
    int32_t new_num_blocks;     /* physical pages in each dst (bounds checks)                          */
    const dsa_cache_array* arrays; /* HOST array of n_arrays (read during the call), or NULL           */
    int32_t n_arrays;           /* 0..8                                                                */
} dsa_evict_inputs;

/* status, scratch (dsa_evict_scratch_size bytes) and errors as for dsa_chunk_attn. */
DSA_API size_t dsa_evict_scratch_size(const dsa_batch* batch);
DSA_API dsa_status dsa_cache_evict(const dsa_batch* batch, const dsa_evict_inputs* in, int32_t* out_idx, int32_t* out_len,
                                   void* status, void* scratch, size_t scratch_bytes, void* stream);

/* Static description of a status code. */
DSA_API const char* dsa_status_str(int32_t status);

/*
 * Text of the last failure an entry point recorded on the calling host thread
 * (the CUDA call and its error name for DSA_ERR_CUDA), or "" if none.  The
 * string is owned by the library and stays valid until the next call on that
 * thread.
 */
DSA_API const char* dsa_last_error(void);

/* Library version string. */
DSA_API const char* dsa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DSA_H_ */
