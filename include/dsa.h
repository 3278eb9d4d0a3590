/*
 * dsa.h -- C ABI of the B200 (sm_100a) DeepSeek Sparse Attention decode path.
 *
 * The path has three steps (DSA blog by marsggbo, section 3; "DeepSeekV3.2之DSA"
 * by yuyanqi, sections 3-5):
 *   1. lightning-indexer score  I[t,s] = sum_j w[t,j] * ReLU(q^I[t,j] . k^I[s])
 *   2. per-query TopK of I[t, 0..n-1]; every position when n <= k
 *   3. MQA-mode MLA attention of all query heads over the selected latent rows,
 *      softmax(q . [c_kv; k_pe]^T) . c_kv
 *
 * Conventions shared by every call
 *   - Pointers.  Every tensor argument is a DEVICE pointer owned by the caller.
 *     The library allocates no device memory; scratch comes from the caller's
 *     `ws` buffer of at least dsa_workspace_size() bytes, 256-byte aligned and
 *     zero-filled before its first use (its first word is the status word;
 *     every call leaves the rest of ws ready for the next call).
 *     `dsa_params` and `dsa_kv` themselves are host structs (their pointer
 *     members are device pointers).
 *   - Streams.  `stream` is a cudaStream_t passed as void* (NULL = legacy
 *     default stream).  Calls only enqueue work and return; nothing
 *     synchronises implicitly.
 *   - Errors.  Every call returns a dsa_status.  Host-side validation failures
 *     launch nothing.  Problems only the device can see (an index >= n, a
 *     bounded wait that expired) are recorded in a status word inside `ws`;
 *     dsa_check_status() synchronises the stream and returns (then clears) it.
 *     dsa_last_error() gives a thread-local message for the last failure.
 *   - Threads.  Calls are stateless and re-entrant; concurrent calls must use
 *     distinct workspaces.
 *   - Layouts.  Row-major, innermost dimension last, densely packed unless a
 *     stride argument says otherwise.  FP8 is OCP E4M3 ("fn": max 448, no inf),
 *     bf16 is the upper half of binary32.
 */
#ifndef DSA_B200_H
#define DSA_B200_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DSA_OK = 0,
    DSA_ERR_INVALID_ARG = -1,  /* a pointer, size or shape is invalid; nothing launched */
    DSA_ERR_UNSUPPORTED = -2,  /* valid but outside what this build implements */
    DSA_ERR_CUDA = -3,         /* a CUDA runtime/driver call failed */
    DSA_ERR_WORKSPACE = -4,    /* ws is NULL, misaligned or smaller than required */
    DSA_ERR_TIMEOUT = -5,      /* device: a bounded wait expired (the work was abandoned) */
    DSA_ERR_DEVICE_CHECK = -6  /* device: an input failed a check (e.g. index >= n) */
} dsa_status;

/* Problem shape.
 *   nq         query tokens in the batch (>= 0)
 *   h_idx      indexer heads H_I, 1..64 ("index_n_heads", yuyanqi section 3.1)
 *   d_idx      indexer head dim d_I: 64 or 128
 *   h          attention heads, 1..128 (all share one latent row: MQA mode,
 *              marsggbo section 4)
 *   d_qk       key width: 576 (512 latent + 64 rope, yuyanqi section 5.1)
 *   d_v        value width: 512 (the first d_v columns of the same row)
 *   topk       k, 1..2048 (DeepSeek-V3.2 uses 2048, marsggbo section 3)
 *   max_n      an upper bound of every q_n (host-known; sizes the launch grid
 *              and the workspace); 0 <= q_n[i] <= max_n <= 2^27
 *   q_per_seq  queries are in blocks of q_per_seq consecutive queries that
 *              read the same sequence (1 for plain decode, 2 for next token +
 *              one speculative token, L for a prefill of L tokens); the
 *              indexer shares each k^I tile among the queries of a block
 *   scale      softmax scale applied to q . c (576^-0.5 in the workloads)
 */
typedef struct {
    int32_t nq;
    int32_t h_idx;
    int32_t d_idx;
    int32_t h;
    int32_t d_qk;
    int32_t d_v;
    int32_t topk;
    int32_t max_n;
    int32_t q_per_seq;
    float scale;
} dsa_params;

/* Where each query's history lives.  The FP8 index-K cache and the bf16
 * latent cache are indexed by the same token positions (yuyanqi section 5.2,
 * item 3): logical position s of sequence b is cache row
 *   contiguous (page_table == NULL):  seq_row0[b] + s
 *   paged      (page_table != NULL):  page_table[b * max_pages + s / page_size]
 *                                        * page_size + s % page_size
 *   q_seq      [nq] int32, device: sequence of each query
 *   q_n        [nq] int32, device: visible positions n of each query; the
 *              query sees positions 0..n-1 (s < t of marsggbo section 3 when
 *              the caller sets n = t)
 *   seq_row0   [nseq] int64, device (contiguous layout) or NULL
 *   page_table [nseq, max_pages] int32, device (paged layout) or NULL
 *   max_pages  columns of page_table
 *   page_size  tokens per page: 64 or 128 (paged layout); ignored otherwise
 *   cache_rows rows in each cache (bounds every cache access)
 */
typedef struct {
    const int32_t *q_seq;
    const int32_t *q_n;
    const int64_t *seq_row0;
    const int32_t *page_table;
    int32_t max_pages;
    int32_t page_size;
    int64_t cache_rows;
} dsa_kv;

/* Operation selector for dsa_workspace_size(). */
typedef enum {
    DSA_OP_INDEXER_SCORES = 0,
    DSA_OP_TOPK = 1,
    DSA_OP_INDEXER_TOPK = 2,
    DSA_OP_SPARSE_MLA_DECODE = 3,
    DSA_OP_SPARSE_MLA_PREFILL = 4,
    DSA_OP_FORWARD = 5,
    DSA_OP_INDEX_KL_SPARSE = 6, /* dsa_index_kl with idx (topk entries per query) */
    DSA_OP_INDEX_KL_DENSE = 7,  /* dsa_index_kl without idx (every visible position) */
    DSA_OP_MASKED_MHA = 8       /* dsa_masked_mha_prefill */
} dsa_op;

/* Bytes of scratch `ws` the given operation needs for this shape (host only,
 * no CUDA call).  `kv` may be NULL for DSA_OP_TOPK.  Returns
 * DSA_ERR_INVALID_ARG for a shape the operation rejects. */
int dsa_workspace_size(const dsa_params *p, const dsa_kv *kv, int op, size_t *bytes);

/* Step 1 alone: the lightning-indexer score of every visible position,
 * written to HBM (index-score equation, marsggbo section 3; FP8 kernel
 * comment of yuyanqi section 4.3: fp8 q.k -> fp32 logits, ReLU, * weights,
 * sum over heads, * k_s).
 *   q_idx      [nq, h_idx, d_idx] e4m3
 *   w          [nq, h_idx] bf16; every constant factor (H_I^-1/2, the q
 *              quantisation scale, d_I^-1/2; yuyanqi section 4.3) must already
 *              be folded in: the library applies none
 *   kidx_cache [cache_rows, d_idx] e4m3 index-K cache (one head shared by all
 *              indexer heads), rows 16-byte aligned
 *   k_scale    [cache_rows] fp32 per-row dequantisation scale, or NULL (= 1)
 *   scores     [nq, ld_scores] fp32 output: scores[i, s] for s < q_n[i];
 *              -inf for q_n[i] <= s < ld_scores.  ld_scores >= max_n.
 * Arithmetic: FP8 products are exact; the d_I-term dot products are
 * accumulated in fp32 by the tensor cores; ReLU, * w and the head sum in fp32. */
int dsa_indexer_scores(const dsa_params *p, const dsa_kv *kv, const void *q_idx,
                       const void *w, const void *kidx_cache, const float *k_scale,
                       float *scores, int64_t ld_scores, void *ws, size_t ws_bytes,
                       void *stream);

/* Step 2 alone: per-query TopK of scores already in HBM (marsggbo section 3;
 * indices, not values, as in yuyanqi section 4.4).  For query i with n = q_n[i]:
 * if n <= topk the result is every position 0..n-1 (yuyanqi section 3.3);
 * otherwise the topk positions with the largest score, ties broken toward
 * the lower position.  -0.0 and +0.0 are equal.  Scores must not be NaN.
 *   scores  [nq, ld_scores] fp32 (entries s >= q_n[i] are not read)
 *   q_n     [nq] int32 device
 *   idx     [nq, topk] int32 output: the min(topk, n) selected positions in
 *           ascending order, then -1 (the same output every run)
 *   nsel    [nq] int32 output min(topk, n), or NULL
 * The result is exact: identical scores give identical sets. */
int dsa_topk(const dsa_params *p, const float *scores, int64_t ld_scores,
             const int32_t *q_n, int32_t *idx, int32_t *nsel, void *ws,
             size_t ws_bytes, void *stream);

/* Steps 1 + 2 fused: the scores of a query never leave on-chip memory; only
 * the selected positions reach HBM (the fused logits + TopK path of yuyanqi
 * section 4.4).  Queries with q_n <= topk skip scoring (yuyanqi section 4.5).
 * Arguments as dsa_indexer_scores and dsa_topk.  The selected set is the one
 * dsa_topk returns on the scores dsa_indexer_scores writes, bit for bit. */
int dsa_indexer_topk(const dsa_params *p, const dsa_kv *kv, const void *q_idx,
                     const void *w, const void *kidx_cache, const float *k_scale,
                     int32_t *idx, int32_t *nsel, void *ws, size_t ws_bytes,
                     void *stream);

/* Step 3: sparse MQA-mode MLA attention (u_t = Attn(h_t, {c_s : s in I_t}),
 * marsggbo section 3; softmax(q . [c_kv; k_pe]^T) . c_kv, yuyanqi section 5.1).
 * For every query i and head h, over the valid entries s of idx[i, :]:
 *   S_s = scale * q[i,h,:] . c[s, 0:d_qk];   P = softmax(S)
 *   out[i,h,:] = sum_s P_s c[s, 0:d_v];      lse[i,h] = ln sum_s exp(S_s)
 *   q            [nq, h, d_qk] bf16
 *   kv_cache     latent cache, bf16 rows of d_qk values, row r at element
 *                offset r * kv_row_stride (kv_row_stride >= d_qk, multiple of 8)
 *   idx          [nq, topk] int32 logical positions; -1 entries are skipped;
 *                entries >= q_n[i] are skipped and flag DSA_ERR_DEVICE_CHECK;
 *                a position listed twice counts twice
 *   out          [nq, h, d_v] bf16;  lse [nq, h] fp32 (natural log)
 * A query with no valid entry gets out = 0 and lse = -inf.
 * Arithmetic: bf16 tensor-core products with fp32 accumulation; softmax in
 * fp32; P enters the P.V product as a pair of bf16 tiles (P_hi + P_lo,
 * together exact to about 2^-16).  When a query's rows are split over
 * several CTAs, each split's normalised output is kept in ws as fp16 times
 * a power-of-two scale per 256 value columns (so a finite bf16 latent of any
 * magnitude neither overflows fp16 nor falls under its normal range relative
 * to its half row's largest value) and the splits are merged by their
 * log-sum-exp. */
int dsa_sparse_mla_decode(const dsa_params *p, const dsa_kv *kv, const void *q,
                          const void *kv_cache, int64_t kv_row_stride,
                          const int32_t *idx, void *out, float *lse, void *ws,
                          size_t ws_bytes, void *stream);

/* Step 3 over an FP8 latent cache (half the bytes of every gathered row).
 * The pages give FP8 only for the indexer's keys (e4m3 with a per-row e8m0
 * scale, yuyanqi section 4.3); the latent cache here uses that same format,
 * a reading of ours: row r holds d_qk e4m3 codes and stands for
 *   c[r, d] = e4m3(kv8_cache[r * kv8_row_bytes + d]) * kv_scale[r]
 * with kv_scale[r] a power of two (then every c is exact in bf16 and the
 * result is that of dsa_sparse_mla_decode on the bf16 cache of those values).
 *   kv8_cache     [cache_rows, kv8_row_bytes] e4m3 codes, 16-byte aligned;
 *                 kv8_row_bytes >= 576 and a multiple of 16
 *   kv_scale      [cache_rows] fp32
 * Everything else (arguments, ws, errors, arithmetic) as for
 * dsa_sparse_mla_decode. */
int dsa_sparse_mla_decode_fp8(const dsa_params *p, const dsa_kv *kv, const void *q,
                              const void *kv8_cache, int64_t kv8_row_bytes,
                              const float *kv_scale, const int32_t *idx, void *out,
                              float *lse, void *ws, size_t ws_bytes, void *stream);

/* Step 3 scheduled for many queries of one sequence (causal prefill, where
 * token t sees n = t positions).  Same arguments and results as
 * dsa_sparse_mla_decode. */
int dsa_sparse_mla_prefill(const dsa_params *p, const dsa_kv *kv, const void *q,
                           const void *kv_cache, int64_t kv_row_stride,
                           const int32_t *idx, void *out, float *lse, void *ws,
                           size_t ws_bytes, void *stream);

/* Short prefill as masked MHA: dense multi-head attention over every visible
 * position with the index set applied as a mask, the form the pages give
 * DSA for short prompts (DSA blog by marsggbo, section 6; aicoding.csdn.net
 * DSA article, section 4.3: below 8K tokens).  MHA form of MLA (marsggbo,
 * section 4): every head has its own key and value rows.  For query t, head h:
 *   keep[s] = s < q_n[t] and s listed in idx[t, :]  (idx NULL: every s < q_n[t])
 *   out[t,h] = sum_{s kept} softmax(scale * q[t,h] . k[s,h]) v[s,h]
 *   lse[t,h] = ln sum_{s kept} exp(scale * q[t,h] . k[s,h])
 * A position listed twice is kept once (a mask holds membership); nothing
 * kept gives out = 0 and lse = -inf.
 *   p      d_qk = per-head q/k width (64, 128 or 192), d_v = per-head v width
 *          (64 or 128), h heads, topk = idx columns, max_n >= every q_n
 *          (<= 2^20), q_per_seq: queries come in blocks of q_per_seq
 *          consecutive queries of one sequence (a prefill of L tokens: L);
 *          h_idx / d_idx are not read
 *   kv     q_seq, q_n, seq_row0 (contiguous layout only); cache_rows = rows
 *          of k and v; position s of sequence b is row seq_row0[b] + s (rows
 *          past cache_rows read as zero)
 *   q      [nq, h, d_qk] bf16;  k [cache_rows, h, d_qk] bf16;
 *   v      [cache_rows, h, d_v] bf16 (all 16-byte aligned)
 *   idx    [nq, topk] int32 (e.g. dsa_indexer_topk's output) or NULL;
 *          entries < 0 are skipped, entries >= q_n[t] flag DSA_ERR_DEVICE_CHECK
 *   out    [nq, h, d_v] bf16;  lse [nq, h] fp32
 *   ws     dsa_workspace_size(DSA_OP_MASKED_MHA): the membership bitmap
 * Arithmetic as in dsa_sparse_mla_decode: bf16 products, fp32 accumulation,
 * softmax in fp32 with P as a bf16 pair (P_hi + P_lo). */
int dsa_masked_mha_prefill(const dsa_params *p, const dsa_kv *kv, const void *q, const void *k,
                           const void *v, const int32_t *idx, void *out, float *lse, void *ws,
                           size_t ws_bytes, void *stream);

/* The indexer's training signal, forward only: the distillation loss of each
 * query t (DSA blog by marsggbo, section 5.1 for the dense warm-up, 5.2 for
 * the sparse stage).  Over the set T_t (idx == NULL: every visible position
 * s < q_n[t]; else the valid entries of idx[t, :], a position listed twice
 * counting twice):
 *   A_h[s] = softmax over T_t of scale * q[t, h] . c[s]   (each head's
 *            attention distribution, MQA form as in dsa_sparse_mla_decode)
 *   p[s]   = sum_h A_h[s] / sum_{s' in T_t} sum_h A_h[s']  (summed over
 *            heads, L1-normalised along the sequence)
 *   kl[t]  = sum_{s in T_t} p[s] * (ln p[s] - ln softmax_{T_t}(I[t, .])[s])
 * A query whose set is empty gets kl = 0.  In the sparse stage each head is
 * normalised over T_t, the set the main model attends to (the page does not
 * say; this is the plain reading).
 *   q, kv_cache, kv_row_stride, kv  as for dsa_sparse_mla_decode
 *   index_scores [nq, ld_scores] fp32 (e.g. dsa_indexer_scores' output);
 *                max_n <= ld_scores <= 2^27
 *   idx          [nq, topk] int32 or NULL (the dense stage); entries < 0 are
 *                skipped, entries >= q_n[t] flag DSA_ERR_DEVICE_CHECK
 *   kl           [nq] fp32 output
 *   p_out        [nq, ld_scores] fp32 output or NULL: p[s] at column s,
 *                0 elsewhere (every column of the query's row is written)
 *   ws           dsa_workspace_size(DSA_OP_INDEX_KL_SPARSE, or _DENSE when
 *                idx is NULL)
 * Arithmetic: the attention scores as in dsa_sparse_mla_decode (bf16
 * products, fp32 accumulation, exp in fp32); each head's log-sum-exp is
 * merged over the splits of the set, then the scores are recomputed and
 * exp(S - lse) summed over heads in fp32; the normalisation, the index
 * scores' softmax and the KL sum in fp64. */
int dsa_index_kl(const dsa_params *p, const dsa_kv *kv, const void *q, const void *kv_cache,
                 int64_t kv_row_stride, const float *index_scores, int64_t ld_scores,
                 const int32_t *idx, float *kl, float *p_out, void *ws, size_t ws_bytes,
                 void *stream);

/* Steps 1-3 in one call: fused indexer + TopK, then sparse attention, as in
 * the decode data flow of yuyanqi section 5.1.  idx_out [nq, topk] receives
 * the selected positions (or NULL: they stay in ws).  Arguments as above;
 * page_table may be set (paged caches) or NULL (contiguous caches). */
int dsa_forward(const dsa_params *p, const dsa_kv *kv, const void *q_idx,
                const void *w, const void *kidx_cache, const float *k_scale,
                const void *q, const void *kv_cache, int64_t kv_row_stride,
                void *out, float *lse, int32_t *idx_out, void *ws,
                size_t ws_bytes, void *stream);

/* dsa_forward over paged caches (sglang's paged TopK path named in yuyanqi
 * section 4.4): kv->page_table must be non-NULL. */
int dsa_forward_paged(const dsa_params *p, const dsa_kv *kv, const void *q_idx,
                      const void *w, const void *kidx_cache, const float *k_scale,
                      const void *q, const void *kv_cache, int64_t kv_row_stride,
                      void *out, float *lse, int32_t *idx_out, void *ws,
                      size_t ws_bytes, void *stream);

/* The indexer's own inputs, produced from the hidden state and the low-rank
 * query ("DeepSeekV3.2之DSA" by yuyanqi, sections 4.1-4.3), with k^I
 * appended to the index-K cache (the decode data flow of its section 5.1).
 * For every token t:
 *   q^I[t] = W_qb . q_lora[t] as [h_idx, d_idx]             (wq_b)
 *   k^I[t] = LayerNorm(W_k . x[t]) * ln_gamma + ln_beta      (wk, k_norm;
 *            biased variance, epsilon ln_eps)
 *   RoPE on the first rope_dim dims of every q^I head and of k^I: the pair
 *            (2i, 2i+1) rotated by positions[t] * rope_theta^(-2i / rope_dim)
 *   q_scale[t, j] / k_scale = the smallest power of two s with amax / s <= 448
 *            (the e8m0 k_s of section 4.3; per (token, head) for q, per
 *            token for k), codes = e4m3(value / s) (ties to even, saturating)
 *   w[t, j] = (W_proj . x[t])_j / sqrt(h_idx) / sqrt(d_idx) * q_scale[t, j],
 *            rounded to bf16 (weights_proj with n_heads^-1/2, the softmax
 *            scale d_I^-1/2 and the q scale folded in: the form the indexer
 *            score takes, with no factor of its own)
 * Shapes: nt tokens; hidden = width of x, q_lora_rank = width of q_lora (both
 * multiples of 8); h_idx 1..64; d_idx 64 or 128; rope_dim even, <= d_idx. */
typedef struct {
    int32_t nt;
    int32_t hidden;
    int32_t q_lora_rank;
    int32_t h_idx;
    int32_t d_idx;
    int32_t rope_dim;
    float ln_eps;
    float rope_theta;
} dsa_project_params;

/* Bytes of `ws` dsa_indexer_project needs (host only). */
int dsa_project_workspace_size(const dsa_project_params *pp, size_t *bytes);

/* Produce q^I, w and k^I of nt tokens and append k^I to the cache.
 *   kv         where each token's k^I row goes: kv->q_seq [nt] is the token's
 *              sequence and positions[t] its position; the row follows
 *              kv->seq_row0 / kv->page_table as for the score (kv->q_n is not
 *              read).  A row outside [0, cache_rows) flags DSA_ERR_DEVICE_CHECK
 *              and is not written.
 *   x          [nt, hidden] bf16;  q_lora [nt, q_lora_rank] bf16
 *   w_qb       [h_idx * d_idx, q_lora_rank] bf16; w_k [d_idx, hidden] bf16;
 *   w_proj     [h_idx, hidden] bf16  (all [out, in], 16-byte aligned)
 *   ln_gamma, ln_beta [d_idx] fp32;  positions [nt] int32
 *   q_idx      [nt, h_idx, d_idx] e4m3 output (the indexer's q_idx input)
 *   q_scale    [nt, h_idx] fp32 output, or NULL
 *   w          [nt, h_idx] bf16 output (the indexer's w input)
 *   kidx_cache [cache_rows, d_idx] e4m3: row of token t overwritten
 *   k_scale    [cache_rows] fp32: entry of token t's row overwritten (pass the
 *              same array to the score as its k_scale)
 *   q_f32, k_f32, w_f32: [nt, h_idx, d_idx], [nt, d_idx], [nt, h_idx] fp32
 *              outputs of the values before rounding (after RoPE; w before
 *              folding), or NULL
 * Arithmetic: bf16 tensor-core products with fp32 accumulation (a split of
 * the K dimension is summed in a fixed order); LayerNorm and the rounding
 * decisions in fp32, RoPE angles and the weight folding in fp64. */
int dsa_indexer_project(const dsa_project_params *pp, const dsa_kv *kv, const void *x,
                        const void *q_lora, const void *w_qb, const void *w_k, const void *w_proj,
                        const float *ln_gamma, const float *ln_beta, const int32_t *positions,
                        void *q_idx, float *q_scale, void *w, void *kidx_cache, float *k_scale,
                        float *q_f32, float *k_f32, float *w_f32, void *ws, size_t ws_bytes,
                        void *stream);

/* ------------------------------------------------------------------------
 * Serving around the path: the tables a step of a paged batch needs, the
 * rotary positions of its queries and keys, the append of its latent rows,
 * and the attention of a batch that shares a long prefix.
 * ------------------------------------------------------------------------ */

/* Bytes of the status word at the start of a workspace; a workspace of this
 * size is all dsa_latent_append needs. */
#define DSA_WS_STATUS_BYTES 256

/* Page tables and slot maps of one step, from the requests' lengths.
 *   nseq       sequences, 0..16384
 *   nt         token slots of the step: entries of q_seq, positions, q_n and
 *              slots, 0..2^27; the step's tokens come first, the rest is padding
 *   page_size  tokens per page, 1..65536 (dsa_kv takes 64 and 128)
 *   max_pages  columns of page_table
 *   n_free     entries of free_pages
 *   sees_self  1: the token at position t sees t + 1 positions (its own row is
 *              appended before the attention); 0: t positions
 *   cache_rows rows in each cache; page ids are 0..cache_rows / page_size - 1 */
typedef struct {
    int32_t nseq;
    int32_t nt;
    int32_t page_size;
    int32_t max_pages;
    int32_t n_free;
    int32_t sees_self;
    int64_t cache_rows;
} dsa_table_params;

/* Bytes of `ws` dsa_build_tables needs (host only). */
int dsa_table_workspace_size(const dsa_table_params *tp, size_t *bytes);

/* Advance every sequence by its new tokens: give it the pages they need and
 * lay out the step's tokens.  For sequence b with seq_len[b] positions in the
 * cache and new_len[b] new ones (0: it waits this step):
 *   held   = ceil(seq_len[b] / page_size) entries of page_table[b, :] are set
 *   need   = ceil((seq_len[b] + new_len[b]) / page_size) - held more pages come
 *            from free_pages, in order: sequence 0's first, starting at entry
 *            free_head[0] of the list
 *   tokens = entries q_start[b] .. q_start[b + 1] - 1 of the token arrays, in
 *            sequence order
 * A sequence with fork_src[b] = a >= 0 starts as a copy of a's first
 * seq_len[b] positions: its first seq_len[b] / page_size table entries are
 * written with a's.  Only full pages are shared (seq_len[b] is a multiple of
 * page_size, at most seq_len[a]) and a must not itself be a fork in this call.
 *   seq_len, new_len [nseq] int32;  fork_src [nseq] int32 or NULL (no forks)
 *   free_pages [n_free] int32, free_head [1] int32: entries before free_head[0]
 *              are taken
 *   page_table [nseq, max_pages] int32, in and out: only the new pages' (and
 *              forks' shared) entries are written
 *   q_start    [nseq + 1] int32 output
 *   q_seq, positions, q_n, slots [nt] int32 outputs: each token's sequence, its
 *              position t, its visible positions (t or t + 1) and its cache row
 *              page * page_size + t % page_size; padding gets 0, -1, 0, -1
 *              (dsa_rope skips position -1, dsa_latent_append slot -1, and the
 *              attention gives a query of 0 positions out = 0, lse = -inf)
 *   kv_len     [nseq] int32 output seq_len + new_len; may be seq_len itself
 *   free_head_out [1] int32 output, the list's new head; may be free_head itself
 *   ws         dsa_table_workspace_size()
 * No output overlaps an input but kv_len and free_head_out as said.
 * Putting pages of finished sequences back is the owner's: write a new list.
 * A batch that cannot be laid out (a negative or too long sequence, more
 * tokens than nt, too few free pages, a bad fork) is refused as a whole: it
 * flags DSA_ERR_DEVICE_CHECK, every token entry is padding, q_start is 0,
 * kv_len = seq_len, and neither page_table nor the head changes.  A page id
 * outside the cache flags DSA_ERR_DEVICE_CHECK too; its tokens' slots are -1. */
int dsa_build_tables(const dsa_table_params *tp, const int32_t *seq_len, const int32_t *new_len,
                     const int32_t *fork_src, const int32_t *free_pages, const int32_t *free_head,
                     int32_t *page_table, int32_t *q_start, int32_t *q_seq, int32_t *positions,
                     int32_t *q_n, int32_t *slots, int32_t *kv_len, int32_t *free_head_out, void *ws,
                     size_t ws_bytes, void *stream);

/* Rotary positions (the RoPE of yuyanqi section 4.2).
 * Pair i of rope_dim / 2 turns by the angle pos * f_i:
 *   (y0, y1) = mscale * (x0 cos - x1 sin, x0 sin + x1 cos)
 * layout says which elements of the rotated range are pair i:
 *   DSA_ROPE_INTERLEAVED (2i, 2i + 1);  DSA_ROPE_HALF (i, i + rope_dim / 2)
 * scaling says how the speeds f_i = theta^(-2i / rope_dim) are stretched for
 * contexts longer than the original:
 *   DSA_ROPE_SCALE_NONE    f_i
 *   DSA_ROPE_SCALE_LINEAR  f_i / factor
 *   DSA_ROPE_SCALE_BASE    theta replaced by theta * factor^(rope_dim / (rope_dim - 2))
 *   DSA_ROPE_SCALE_YARN    f_i (1 - r_i) + f_i / factor * r_i, r_i = clamp((i - lo) / max(hi - lo, 0.001), 0, 1)
 *       with edge(b) = rope_dim ln(orig_max_pos / (2 pi b)) / (2 ln theta),
 *       lo = max(floor(edge(beta_fast)), 0), hi = min(ceil(edge(beta_slow)), rope_dim - 1)
 * mscale multiplies the rotated elements (1 for none; 0.1 ln(factor) + 1 is
 * usual with YaRN).  rope_dim is even, 0..256.  Sines and cosines are computed
 * in fp32 from angles reduced in 64 bits: they are off by about 2^-24 and by
 * at most 8 * 2^-53 of the angle pos * f_i itself (rarely a third of that).
 * For speeds up to 1 that is fp32 accuracy for positions up to 2^27, the
 * longest history any call takes; at 2^31 - 1 it is about 4e-7.  A theta and
 * factor whose speeds exceed 1e290 are refused. */
enum { DSA_ROPE_INTERLEAVED = 0, DSA_ROPE_HALF = 1 };
enum { DSA_ROPE_SCALE_NONE = 0, DSA_ROPE_SCALE_LINEAR = 1, DSA_ROPE_SCALE_BASE = 2, DSA_ROPE_SCALE_YARN = 3 };
enum { DSA_DTYPE_BF16 = 0, DSA_DTYPE_FP16 = 1, DSA_DTYPE_FP32 = 2 };
typedef struct {
    int32_t rope_dim;
    int32_t layout;
    int32_t scaling;
    int32_t orig_max_pos;
    double theta;
    double factor;
    double beta_fast;
    double beta_slow;
    double mscale;
} dsa_rope_spec;

/* What dsa_rope rotates: x [nt, x_heads, d] -> y [nt, h, d] of one type.
 *   x_heads  h, or 1: one head that every head of y receives (the rope part
 *            of a key shared by all heads, in the MHA form)
 *   begin    first rotated element of a head; [begin, begin + rope_dim) lies
 *            in [0, d); the others are copied
 *   strides  in elements between tokens and between heads of x and of y;
 *            the elements of a head are adjacent; >= 0 (0 repeats a row that is
 *            read; the rows that are written must not overlap)
 *   d        1..1024; h 1..65535; nt 0..2^27 */
typedef struct {
    int32_t nt;
    int32_t h;
    int32_t x_heads;
    int32_t d;
    int32_t begin;
    int32_t dtype;
    int64_t x_token_stride;
    int64_t x_head_stride;
    int64_t y_token_stride;
    int64_t y_head_stride;
} dsa_rope_params;

/* y = x with its rotated range turned by each token's position.
 *   positions [nt] int32; a token with a negative position is padding: its
 *             rows of y are left as they were
 *   y may be x itself with the same strides (x_heads = h): the rotated range
 *   is updated in place.  Otherwise x and y must not overlap.
 * Arithmetic: fp32 (each value is rounded to the type once). */
int dsa_rope(const dsa_rope_spec *rs, const dsa_rope_params *rp, const void *x, const int32_t *positions,
             void *y, void *stream);

/* The gradient of dsa_rope: dx [nt, x_heads, d] (x's strides) from dy
 * [nt, h, d] (y's strides): the inverse turn times mscale, summed over the
 * heads when x_heads = 1 < h (fp32, in an order that does not change from run
 * to run).  A padding token's dx is 0.  dx may be dy itself with the same
 * strides (x_heads = h). */
int dsa_rope_backward(const dsa_rope_spec *rs, const dsa_rope_params *rp, const void *dy,
                      const int32_t *positions, void *dx, void *stream);

/* Append the step's latent rows to the cache that dsa_sparse_mla_decode
 * reads: row slots[t] = [c_kv[t] | rope(k_pe[t])] (the decode data flow of
 * yuyanqi section 5.1).
 *   rs        rope_dim = 64 (the rope part of the 576-wide row)
 *   c_kv      [nt, 512] bf16, rows c_kv_stride elements apart;  k_pe [nt, 64]
 *             bf16, rows k_pe_stride apart (both 16-byte aligned, strides
 *             multiples of 8, ignored for one row: they may be the two parts
 *             of one [nt, 576] array)
 *   positions [nt] int32;  slots [nt] int32 cache rows (dsa_build_tables);
 *             -1 is padding and writes nothing; a row outside [0, cache_rows)
 *             flags DSA_ERR_DEVICE_CHECK and is not written; a row listed
 *             twice is of no use afterwards (it ends up with elements of
 *             either token, in FP8 with codes and a scale that need not belong
 *             together)
 *   kv_cache  bf16 rows kv_row_stride elements apart (as for the attention)
 *   ws        DSA_WS_STATUS_BYTES
 * The rotation is computed in fp32 and rounded to bf16 once. */
int dsa_latent_append(const dsa_rope_spec *rs, int32_t nt, const void *c_kv, int64_t c_kv_stride,
                      const void *k_pe, int64_t k_pe_stride, const int32_t *positions, const int32_t *slots,
                      void *kv_cache, int64_t kv_row_stride, int64_t cache_rows, void *ws, size_t ws_bytes,
                      void *stream);

/* The same into the FP8 latent cache of dsa_sparse_mla_decode_fp8: the row's
 * 576 values (rope part rotated in 64 bits) as e4m3 codes (ties to even) of
 * value / s, s = kv_scale[slot] the smallest power of two with amax / s <= 448
 * (at least 2^-126; 1 for a row of zeros).  Infinities and NaN do not enter
 * amax; an infinity is stored as +-448 s, NaN as NaN, and a rotated value past
 * the largest fp32 number counts as an infinity.  kv8_row_bytes and kv_scale as
 * for dsa_sparse_mla_decode_fp8. */
int dsa_latent_append_fp8(const dsa_rope_spec *rs, int32_t nt, const void *c_kv, int64_t c_kv_stride,
                          const void *k_pe, int64_t k_pe_stride, const int32_t *positions,
                          const int32_t *slots, void *kv8_cache, int64_t kv8_row_bytes, float *kv_scale,
                          int64_t cache_rows, void *ws, size_t ws_bytes, void *stream);

/* Bytes of `ws` dsa_mla_shared_prefix needs for this shape (host only): about
 * 263 KB for every 128 (query, head) rows, for every group and for every query
 * (2.2 GB for 4096 queries of 128 heads, 1.1 GB for 4096 of one head). */
int dsa_shared_prefix_workspace_size(const dsa_params *p, const dsa_kv *kv, int32_t ngroups, size_t *bytes);

/* Dense MQA-mode MLA attention of a batch whose queries share long prefixes,
 * each prefix read once for all the queries behind it (every position of the
 * history, no index list: the attention DSA falls back to and is distilled
 * from, marsggbo section 5.1; MQA form, section 4).  Queries come in ngroups
 * groups of consecutive queries:
 *   group_q0 [ngroups + 1] int32, device: group g is queries group_q0[g] ..
 *            group_q0[g + 1] - 1 (group_q0[0] = 0, group_q0[ngroups] = nq,
 *            never decreasing)
 *   group_n  [ngroups] int32, device: the first group_n[g] positions are the
 *            same for all of the group's queries (0: nothing is shared); they
 *            are read through the sequence of the group's first query, so the
 *            other sequences' tables need no entries for them
 * For query i of group g and head h, over its n = q_n[i] positions:
 *   S_s = scale * q[i,h,:] . c[s, 0:576];  out[i,h,:] = sum_s softmax(S)_s c[s, 0:512]
 *   lse[i,h] = ln sum_s exp(S_s)
 * where c[s] is the group's row for s < group_n[g] and the row of the query's
 * own sequence q_seq[i] behind it.  n may be less than group_n[g] (the query
 * then sees the first n shared positions) and 0 (out = 0, lse = -inf).  Rows
 * at or behind n are not used, whatever they hold.
 *   p      nq <= 4096 (a longer step, a prompt of 8192 tokens, goes in several
 *          calls: a query's result does not depend on the others of its call
 *          but for the order of its sums), h, max_n, scale as elsewhere; the
 *          other fields are checked, not used
 *   kv     as for dsa_sparse_mla_decode (contiguous: seq_row0[b] + s may be
 *          outside the cache for shared positions of later sequences)
 *   ngroups 1..4096 (any number when nq = 0)
 *   q, kv_cache, kv_row_stride, out, lse  as for dsa_sparse_mla_decode
 * A length out of [0, max_n], a group_q0 that is not as said, a page id or a row
 * outside the cache flags DSA_ERR_DEVICE_CHECK; nothing is read there, and the
 * queries concerned get no meaningful result.
 * Arithmetic: bf16 tensor-core products with fp32 accumulation, softmax in
 * fp32.  Every weight enters the value product rounded to bf16 once (the
 * sparse attention takes a bf16 pair: here that costs 27% of the time and
 * moves the error against 64 bits from 2.0e-3 to 1.7e-3 of the output, whose
 * own rounding is 1.7e-3). */
int dsa_mla_shared_prefix(const dsa_params *p, const dsa_kv *kv, int32_t ngroups, const int32_t *group_q0,
                          const int32_t *group_n, const void *q, const void *kv_cache,
                          int64_t kv_row_stride, void *out, float *lse, void *ws, size_t ws_bytes,
                          void *stream);

/* dsa_indexer_topk without a workspace, for callers that cannot allocate
 * device memory (their allocator owns the device, they run under a fixed
 * memory budget, or they must not enter the driver's allocator on this
 * path).  The pages have no counterpart: this is a deployment variant of
 * steps 1 + 2, same arguments and same results as dsa_indexer_topk.
 *   - Scratch lives in one fixed 8 MiB device array inside the library;
 *     every GPU that loads the library holds it until the process exits.
 *     A shape needing more scratch is rejected with DSA_ERR_UNSUPPORTED
 *     before anything is launched.  On a 148-SM B200 a decode batch of
 *     up to 78 queries at 128K context (204 at 32K) fits;
 *     dsa_workspace_size(DSA_OP_INDEXER_TOPK) gives a shape's need.
 *   - The call allocates nothing (no cudaMalloc, no allocating library
 *     call).  The first call on each device resolves the array's device
 *     address (cudaGetSymbolAddress) and keeps it for the life of the
 *     process; make that first call outside any stream capture.  Do not use
 *     this entry point after cudaDeviceReset (or anything else that tears
 *     down the device's primary context): the kept address would be stale.
 *   - All calls share the array and it keeps the last call's contents: the
 *     call clears what must start at zero itself, but calls whose work
 *     overlaps on the GPU (other streams, other threads) race; serialise them.
 *   - status (device int32, nullable) receives the device status word of
 *     this call (DSA_OK, DSA_ERR_TIMEOUT or DSA_ERR_DEVICE_CHECK) in stream
 *     order; dsa_check_status does not apply (there is no ws). */
int dsa_indexer_topk_static(const dsa_params *p, const dsa_kv *kv, const void *q_idx,
                            const void *w, const void *kidx_cache, const float *k_scale,
                            int32_t *idx, int32_t *nsel, int32_t *status, void *stream);

/* Synchronise `stream`, return the device status word stored in `ws`
 * (DSA_OK, DSA_ERR_TIMEOUT or DSA_ERR_DEVICE_CHECK) and clear it. */
int dsa_check_status(void *ws, void *stream);

/* Message describing the last failure on this thread ("" if none). */
const char *dsa_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* DSA_B200_H */
