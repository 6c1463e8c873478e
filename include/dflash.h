/*
 * dflash.h -- C ABI of a GB300 (sm_103a) library for one DFlash
 * speculative-decoding step: fuse -> inject -> draft -> verify -> accept ->
 * rollback.  Every stage runs as CUDA kernels of this library on the stream
 * the caller passes; the host only validates arguments and enqueues work.
 *
 * Sources (page titles as printed on the pages):
 *   [DD] "DFlash 深度解析：块扩散模型如何让 LLM 推理加速 6 倍——2026 投机解码完全指南"
 *        (chenxutan.com): §1.1 autoregressive decoding, §1.2 speculative
 *        decoding, §2.2 feature_fusion / kv_injection / draft_inference,
 *        §3.3 shared embedding and LM head, §5.1 one-forward block drafting,
 *        §8.2 linear verification.
 *   [LC] "从 ICML 论文到你的显卡：llama.cpp 吞下 DFlash，本地推理进入 2 倍速时代"
 *        (arex-research.com): KV injection into every drafter layer; keep the
 *        matching prefix, cut at the first error.
 *   [RD] "我在llama.cpp中测试了最新合并的DFlash在Qwen 3.6 27B本地AI上的表现"
 *        (bittide.aicompass.dev): greedy verification is lossless.
 *
 * Conventions
 *   - All pointers to tensors are DEVICE pointers owned by the caller unless
 *     stated otherwise; the library never frees them.  Row-major throughout.
 *   - Matrices are nn.Linear [out_features][in_features].
 *   - Element type of weights, KV caches, hidden states and captured states
 *     is the model's dtype (DFLASH_F32 or DFLASH_BF16); residual stream,
 *     logits and all reductions are float32.
 *   - Positions and lengths live on the device (per-sequence int32), so every
 *     call can be captured into a CUDA graph and replayed step after step.
 *   - Return values: DFLASH_OK (0) or a negative DFLASH_ERR_* code from the
 *     synchronous argument checks or from a failed CUDA launch.  Conditions
 *     detected inside kernels (capacity overflow, non-finite logits, a wait
 *     that ran out) set bits in the workspace's device status word, read with
 *     dflash_status(); kernels never trap.
 *   - Calls are asynchronous on `stream` and not thread-safe on one cache or
 *     workspace.
 */
#ifndef DFLASH_H_
#define DFLASH_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* dflash_stream_t; /* = cudaStream_t */

enum {
  DFLASH_OK = 0,
  DFLASH_ERR_INVALID_ARG = -1,
  DFLASH_ERR_UNSUPPORTED_SHAPE = -2,
  DFLASH_ERR_CUDA = -3,
  DFLASH_ERR_OOM = -4,
  DFLASH_ERR_TOO_LARGE = -5, /* a size above an entry point's fixed maximum */
};

/* device status bits (dflash_status) */
enum {
  DFLASH_STATUS_CAPACITY = 1,  /* a write beyond a cache's capacity was skipped */
  DFLASH_STATUS_NONFINITE = 2, /* a logit row held NaN/Inf */
  DFLASH_STATUS_TIMEOUT = 4,   /* a pipeline wait gave up (kernel returned early) */
  DFLASH_STATUS_BOUNDS = 8,    /* an index (token id, reference position) was out of range */
};

enum { DFLASH_F32 = 0, DFLASH_BF16 = 1 };

/* Dimensions of one decoder (target or drafter). head_dim: 64 or 128. */
typedef struct dflash_model_desc {
  int32_t n_layers, hidden, n_q_heads, n_kv_heads, head_dim, ffn, vocab;
  float rope_theta, rms_eps;
  int32_t dtype; /* DFLASH_F32 | DFLASH_BF16 */
} dflash_model_desc;

/* One pre-norm decoder layer.
 *   wqkv      [(nq + 2 nkv) * hd][H]  rows: q heads, then k heads, then v heads
 *   wo        [H][nq * hd]
 *   w_gate_up [2F][H]  row 2f is gate row f, row 2f+1 is up row f
 *   w_down    [H][F]
 *   attn_norm, ffn_norm [H] RMSNorm gains */
typedef struct dflash_layer_w {
  const void *attn_norm, *wqkv, *wo, *ffn_norm, *w_gate_up, *w_down;
} dflash_layer_w;

/* Target model.  capture[5]: 0-based layers whose output residual stream is
 * captured for feature fusion ([DD] §2.2: 5 layers from 2 to the
 * third-from-last, see dflash_capture_layers). */
typedef struct dflash_target {
  dflash_model_desc d;
  const void *embed;      /* [V][H] */
  const void *final_norm; /* [H] */
  const void *lm_head;    /* [V][H] */
  const dflash_layer_w *layers; /* HOST array of d.n_layers entries */
  int32_t capture[5];
} dflash_target;

/* Block-diffusion drafter.  It reuses the target's embedding and LM head
 * ([DD] §3.3).  w_kv_all packs, for every drafter layer l in order, that
 * layer's k rows then v rows of wqkv: [Ld * 2 * nkv * hd][H]; it holds the
 * same values as the layers' wqkv and lets one product project the fused
 * feature for all layers ([DD] §5.2 dflash_feature_injection).
 * cross_ctx: the drafter's cross-context window W ("如何使用 DFlash 试探式解码
 * 加速本地 LLM", §7, --spec-dflash-cross-ctx): W > 0 makes every drafter layer
 * attend only to the W most recent injected positions P-W..P-1 (all of them
 * when P <= W) plus the block's own rows; 0 attends to the whole context. */
typedef struct dflash_draft {
  dflash_model_desc d;
  const void *w_fc;       /* [H][5H] fusion Linear ([DD] §2.2 feature_fusion) */
  const void *fc_norm;    /* [H] fusion RMSNorm gain */
  const void *final_norm; /* [H] */
  const dflash_layer_w *layers; /* HOST array of d.n_layers entries */
  const void *w_kv_all;
  int32_t mask_id;
  int32_t cross_ctx;
} dflash_draft;

/* ------------------------------------------------------------------ caches
 * A KV cache holds, for `batch` sequences and `n_layers` layers, keys and
 * values [layer][seq][kv_head][capacity][head_dim] in the model dtype, a
 * device int32 length per sequence (starts at 0), and a float32 RoPE
 * cos/sin table for positions 0..capacity-1 (computed on the host in double
 * precision).  Library-owned device memory (cudaMalloc); free with
 * dflash_cache_free.  The target cache's length is the committed length P;
 * the drafter cache's length is the number of injected context rows.
 * Positions >= length are scratch: target_verify writes the block there and
 * dflash_draft_block writes its block's keys/values there. */
typedef struct dflash_cache dflash_cache;

int dflash_cache_alloc(const dflash_model_desc *d, int32_t n_layers, int32_t batch,
                       int32_t capacity, dflash_cache **out);

/* Storage of a cache's keys and values. */
enum { DFLASH_KV_MODEL = 0, DFLASH_KV_Q8 = 1 };
/* dflash_cache_alloc with a storage format.  DFLASH_KV_MODEL: the model dtype
 * (as dflash_cache_alloc).  DFLASH_KV_Q8 (bf16 models with head_dim 128; the
 * 8-bit K/V cache of DFlash 深度解析 §8.3 "显存优化" 方案3 and the
 * quantised cache types the datacamp tutorial runs, §5/§7, read as stated in
 * the oracle): each key or value row of 128 entries is kept as 8-bit codes
 * u = q + 128 (q in [-127, 127]) [layer][seq][kv_head][capacity][128] uint8
 * and one float32 scale s per row [layer][seq][kv_head][capacity]; the entry
 * is q * s, quantised from the float32 row x as s = max|x| / 127,
 * q = round-half-even(x / s) (a zero row keeps s = 0).  target_verify writes
 * its rows this way before attention reads them.  Attention computes in IEEE
 * half precision: the query is half, and each entry is read as the half
 * product of q and s rounded to half, half(q * half(s)).  Target caches only: the drafter's cache,
 * tree verification (target_verify_tree, dflash_accept_tree) and the fp32
 * configuration return DFLASH_ERR_UNSUPPORTED_SHAPE with a q8 cache.  A q8
 * cache's capacity is rounded up to a multiple of 8 positions. */
int dflash_cache_alloc_ex(const dflash_model_desc *d, int32_t n_layers, int32_t batch,
                          int32_t capacity, int32_t kv_format, dflash_cache **out);
/* The cache's storage format (DFLASH_KV_MODEL or DFLASH_KV_Q8), or -1. */
int32_t dflash_cache_kv_format(const dflash_cache *c);
int dflash_cache_free(dflash_cache *c);
/* A view of sequences [seq_begin, seq_begin + seq_count) sharing memory with
 * `c` (used to prefill a ragged batch one sequence at a time).  Free views
 * with dflash_cache_free before freeing their parent. */
int dflash_cache_view(dflash_cache *c, int32_t seq_begin, int32_t seq_count, dflash_cache **out);
/* Device pointer to the int32 lengths [batch] (for the caller to read). */
int32_t *dflash_cache_lengths(dflash_cache *c);
/* Synchronises `stream` and copies min(n, batch) lengths to host memory. */
int dflash_cache_get_lengths(dflash_cache *c, int32_t *host_out, int32_t n, dflash_stream_t stream);
/* Copy keys and values of positions [pos0, pos0 + n) of one layer and one
 * sequence from (write) or to (read) caller device buffers k, v laid out
 * [n_kv][n][head_dim] in the cache dtype.  Asynchronous device-to-device
 * copies; lengths are not changed.  Used to load a saved context. */
int dflash_cache_write(dflash_cache *c, int32_t layer, int32_t seq, int32_t pos0, int32_t n,
                       const void *k, const void *v, dflash_stream_t stream);
int dflash_cache_read(dflash_cache *c, int32_t layer, int32_t seq, int32_t pos0, int32_t n, void *k,
                      void *v, dflash_stream_t stream);
/* q8 caches: dflash_cache_write takes bf16 rows and quantises them on the
 * device (same rule as target_verify's writes); dflash_cache_read returns
 * DFLASH_ERR_INVALID_ARG, and dflash_cache_read_q8 copies the stored codes
 * u (uint8 [n_kv][n][128]) and scales (float32 [n_kv][n]) instead.  Either
 * output pair may be NULL. */
int dflash_cache_read_q8(dflash_cache *c, int32_t layer, int32_t seq, int32_t pos0, int32_t n,
                         void *k_codes, void *v_codes, float *k_scales, float *v_scales,
                         dflash_stream_t stream);
/* Copy every key, value (codes and scales for q8) and length of `src` into
 * `dst`, two caches (not views) of identical geometry and storage format
 * (asynchronous device-to-device copies). */
int dflash_cache_copy(dflash_cache *dst, const dflash_cache *src, dflash_stream_t stream);
/* Set the first n lengths from host memory (asynchronous). */
int dflash_cache_set_lengths(dflash_cache *c, const int32_t *host_len, int32_t n,
                             dflash_stream_t stream);
/* Set every length to 0 (asynchronous). */
int dflash_cache_reset(dflash_cache *c, dflash_stream_t stream);

/* --------------------------------------------------------------- workspace
 * Library-owned scratch for activations, split-K partial sums, attention
 * partials and the device status word.  Sized for both models, for up to
 * `max_rows` rows per call (batch x rows-per-sequence, <= 128) and contexts
 * up to `max_ctx` positions.  One workspace serves one stream at a time. */
typedef struct dflash_workspace dflash_workspace;

int dflash_workspace_alloc(const dflash_model_desc *target, const dflash_model_desc *draft,
                           int32_t max_rows, int32_t max_ctx, dflash_workspace **out);
int dflash_workspace_free(dflash_workspace *w);
/* Synchronises `stream`, returns the status bits in *status_out and clears them. */
int dflash_status(dflash_workspace *w, dflash_stream_t stream, int32_t *status_out);
/* Device pointer to one of the workspace's float32 logit buffers, row-major
 * [rows][vocab]: which = 0 the target's, written by target_verify (rows =
 * batch * n); which = 1 the drafter's, written by dflash_draft_block (rows =
 * batch * block).  Each holds the last RMSNorm'd residual times the LM head
 * ([DD] §1.1 next-token scores; §3.3 the drafter shares the head) until the
 * next such call on the workspace.  Owned by the workspace; NULL for a NULL
 * workspace or another `which`.  No synchronisation: read it on the stream. */
float *dflash_workspace_logits(dflash_workspace *w, int32_t which);
/* Failure-path testing: sets the limit, in nanoseconds, of the waits in the
 * main loop of the weight-product kernel (ring slots and accumulator), of the
 * bf16 products with 4-bit weights and of the bf16 attention over pages (of
 * 8-bit ones: with more than 32 rows n * nq / nkv a sequence, or a batch with a
 * shared length), for launches enqueued afterwards; a negative value restores
 * the default of 500 ms.  A limit of 0 expires at once, so the kernel gives up,
 * sets DFLASH_STATUS_TIMEOUT, still waits (whatever the limit) for its copies
 * and products in flight and returns; the weight product writes no result, a
 * 4-bit one at most some of it, attention over pages an unspecified one.
 * Process-wide; not an operation of the method. */
int dflash_debug_set_wait_limit(int64_t ns);
const char *dflash_strerror(int code);

/* Captured layers for a target of n_layers: 5 layers spread uniformly from
 * layer 2 to layer n_layers-3 ([DD] §2.2 feature_fusion), rounded half up. */
int dflash_capture_layers(int32_t n_layers, int32_t out[5]);

/* ------------------------------------------------------------------ stages
 * Sequence state shared by the stages (device int32 arrays, caller-owned):
 *   anchor[batch]  last emitted token; it sits at position P
 *   n_pend[batch]  captured rows not yet injected into the drafter cache;
 *                  they belong to positions P - n_pend .. P - 1
 * Invariant outside a stage: drafter length + n_pend == target length == P.
 * A step is: fuse + inject the pending rows, draft, verify, accept/rollback. */

/* Feature fusion ([DD] §2.2 feature_fusion): fused = RMSNorm(hcap · w_fcᵀ)
 * ⊙ fc_norm for `rows` rows.  hcap [rows][5H] holds the captured hidden
 * states of the 5 layers side by side (the concat); fused [rows][H]. */
int dflash_fuse_features(const dflash_draft *dr, const void *hcap, int32_t rows, void *fused,
                         dflash_workspace *ws, dflash_stream_t stream);

/* KV injection ([DD] §2.2 kv_injection, §5.2; [LC]): for every drafter layer
 * l, K = RoPE(fused · W_k,lᵀ) and V = fused · W_v,lᵀ are appended to layer
 * l's cache.  fused is [batch][rows_per_seq][H]; sequence b injects its first
 * n_pend[b] rows at positions len[b] .. len[b] + n_pend[b] - 1 of
 * draft_cache, then len[b] += n_pend[b] and n_pend[b] = 0 (the rows are
 * consumed). */
int dflash_inject_kv(const dflash_draft *dr, const void *fused, int32_t batch, int32_t rows_per_seq,
                     int32_t *n_pend, dflash_cache *draft_cache, dflash_workspace *ws,
                     dflash_stream_t stream);

/* Block drafting ([DD] §5.1, §2.2 draft_inference): one non-causal forward of
 * the block [anchor, MASK x (block-1)] at positions P .. P+block-1 (P = the
 * drafter cache length) through every drafter layer; each row attends to the
 * injected context 0..P-1 and to all block rows.  Tokens are embedded and
 * decoded with the target's embedding and LM head ([DD] §3.3).  Writes
 * draft_tokens[b][0] = anchor[b] and draft_tokens[b][j] = argmax of row j
 * (j >= 1).  block in [2, 16]. */
int dflash_draft_block(const dflash_draft *dr, const dflash_target *tg, const int32_t *anchor,
                       int32_t batch, int32_t block, dflash_cache *draft_cache,
                       int32_t *draft_tokens, dflash_workspace *ws, dflash_stream_t stream);

/* Target forward ([DD] §1.1, §1.2): tokens [batch][n] at positions
 * P .. P+n-1 (P = target cache length), causal, keys/values written into the
 * cache at those positions.  Outputs per row: argmax [batch][n] (lowest index
 * on ties), top2_gap [batch][n] (nullable; largest minus second-largest
 * logit) and hcap [batch][n][5H] (nullable), the residual stream after each
 * captured layer.  n in [1, 128], batch * n <= workspace max_rows.
 *   commit = 0  verification: lengths untouched (dflash_accept_rollback decides)
 *   commit = 1  prefill chunk: len += n, n_pend = n
 *   commit = 2  as 1, and the last row's greedy token becomes the anchor and
 *               is appended to the stream (last chunk of a prefill, or one
 *               autoregressive step) -- anchor/n_pend/stream may be NULL for
 *               commit = 0. */
int target_verify(const dflash_target *tg, const int32_t *tokens, int32_t batch, int32_t n,
                  int32_t commit, dflash_cache *target_cache, int32_t *argmax, float *top2_gap,
                  void *hcap, int32_t *anchor, int32_t *n_pend, int32_t *stream,
                  int32_t *stream_len, int32_t stream_cap, dflash_workspace *ws,
                  dflash_stream_t cuda_stream);

/* Acceptance and rollback ([DD] §1.2, §8.2; [LC]).  For each sequence b:
 *   a = the number of leading drafted tokens draft_tokens[b][i] (i >= 1) that
 *       equal the target's greedy choice argmax[b][i-1], stopping at the
 *       first mismatch (0 <= a <= block-1);
 *   emitted: argmax[b][0..a] (a drafted tokens + the target's own next token)
 *       are appended to stream[b][*] at stream_len[b] (capacity stream_cap);
 *   rollback: target len[b] = P + a + 1 (rows beyond are discarded in place,
 *       no data moves), anchor[b] = argmax[b][a], n_pend[b] = a + 1.
 * accept_len[batch] receives a (nullable). */
int dflash_accept_rollback(const int32_t *draft_tokens, const int32_t *argmax, int32_t batch,
                           int32_t block, dflash_cache *target_cache, int32_t *anchor,
                           int32_t *n_pend, int32_t *accept_len, int32_t *stream,
                           int32_t *stream_len, int32_t stream_cap, dflash_workspace *ws,
                           dflash_stream_t cuda_stream);

/* Teacher forcing (benchmark harness for random-init models, whose natural
 * acceptance is ~0).  For sequence b at step s = *step (device counter,
 * incremented by this call): k = k_draw[s][b], r = r_draw[s][b],
 * e = stream_len[b]; slots j = 1..min(k, block-1) take ref[b][e+j-1]; if
 * k+1 <= block-1, slot k+1 takes (ref[b][e+k] + 1 + r) mod vocab, which
 * differs from the reference; other slots keep the drafter's tokens.  With
 * ref the greedy stream, exactly min(k, block-1) drafts are then accepted. */
int dflash_teacher_force(int32_t *draft_tokens, int32_t batch, int32_t block, const int32_t *ref,
                         int32_t ref_stride, int32_t ref_len, const int32_t *stream_len,
                         const int32_t *k_draw, const int32_t *r_draw, int32_t max_steps,
                         int32_t *step, int32_t vocab, dflash_workspace *ws, dflash_stream_t stream);

/* ------------------------------------------------------ tree verification
 * "DFlash 深度解析" §8.2 (DDTree): one target forward explores several
 * branches of the drafter's guesses within a node budget instead of one
 * chain; the page prints no algorithm.  These calls take the following
 * reading (greedy):
 *   - candidates: per drafted slot j = 1..block-1, the drafter's top-K tokens
 *     by log-probability log q_j (softmax of the slot's logits; ties to the
 *     lower id);
 *   - the tree: the `budget` highest-scoring token prefixes, a prefix scoring
 *     the sum of its tokens' log q (best-first; every prefix's parent scores at
 *     least as high, so they form a tree rooted at the anchor); ties to the
 *     smaller depth, then the smaller rank, then the earlier parent;
 *   - verification: one target forward over the n = budget + 1 nodes (node 0
 *     the anchor), node i at position P + depth(i), attending to the context
 *     and to its own ancestors (itself included);
 *   - acceptance: from the root, move to the child whose token equals the
 *     target's greedy token after the current node while there is one; emit
 *     the path's tokens and the greedy token after its last node.
 * With K = 1 and budget = block - 1 the tree is the drafter's greedy chain and
 * the step equals linear verification.  Trees hold at most 64 nodes
 * (budget <= 63).  Per-sequence arrays are [batch][n], device memory owned by
 * the caller; tree_mask[b][i] has bit j set for every ancestor j of node i and
 * for i itself. */

/* After dflash_draft_block: build each sequence's tree from the drafter's
 * logits (workspace buffer 1).  topk in [1, 8]; budget in [1, 63] and at most
 * the number of prefixes the candidates allow, else DFLASH_ERR_INVALID_ARG. */
int dflash_draft_tree(const int32_t *anchor, int32_t batch, int32_t block, int32_t vocab, int32_t topk,
                      int32_t budget, int32_t *tree_tokens, int32_t *tree_parent, int32_t *tree_depth,
                      uint64_t *tree_mask, dflash_workspace *ws, dflash_stream_t stream);
/* Target forward of the trees (n = budget + 1 rows per sequence) at
 * positions P + depth, ancestor-masked; keys/values are written at the scratch
 * slots P .. P + n - 1 in node order; argmax [batch][n], top2_gap (nullable),
 * hcap [batch][n][5H] (nullable); lengths untouched. */
int target_verify_tree(const dflash_target *tg, const int32_t *tree_tokens, const int32_t *tree_depth,
                       const uint64_t *tree_mask, int32_t batch, int32_t n, dflash_cache *target_cache,
                       int32_t *argmax, float *top2_gap, void *hcap, dflash_workspace *ws,
                       dflash_stream_t cuda_stream);
/* The walk and the rollback: the accepted path's a drafted tokens and the
 * bonus are appended to stream; the path's keys/values (every target layer)
 * move from their node slots to positions P .. P + a and its captured rows
 * (hcap, nullable, [batch][n][5H]) to rows 0 .. a of the sequence's block;
 * len += a + 1, anchor = the bonus, n_pend = a + 1, accept_len = a
 * (nullable). */
int dflash_accept_tree(const dflash_target *tg, const int32_t *tree_tokens, const int32_t *tree_parent,
                       const int32_t *argmax, int32_t batch, int32_t n, dflash_cache *target_cache, void *hcap,
                       int32_t *anchor, int32_t *n_pend, int32_t *accept_len, int32_t *stream,
                       int32_t *stream_len, int32_t stream_cap, dflash_workspace *ws,
                       dflash_stream_t cuda_stream);

/* ------------------------------------------------------------ sampling mode
 * "DFlash 深度解析" §4.2: the speed-up holds at temperature 1 with the
 * output distribution unchanged; the page gives no rule.  These calls take
 * the standard speculative-sampling rule: with p_i = softmax(target logits of
 * row i / T) and q_j = softmax(drafter logits of slot j / T),
 *   - the drafter's slot j >= 1 is drawn from q_j;
 *   - drafted token d_i (i = 1..block-1) is accepted when u_i q_i(d_i) <
 *     p_{i-1}(d_i) (probability min(1, p/q)), stopping at the first rejection;
 *   - after a accepted drafts one more token is drawn: from the residual
 *     max(0, p_a - q_{a+1}) (renormalised; from p_a when it has no mass) when
 *     a < block-1, from p_{block-1} otherwise.
 * A draw from weights w with uniform v in [0, 1) is the smallest index whose
 * running sum exceeds v * sum(w); uniform numbers are caller-supplied device
 * float32 arrays.  Softmax statistics and running sums are float32 in a fixed
 * order.  temperature must be finite and > 0, else DFLASH_ERR_INVALID_ARG. */

/* After dflash_draft_block: draft_tokens[b][j] (j = 1..block-1) drawn from
 * the drafter's logits (workspace buffer 1) at temperature T with
 * w[b][j-1] ([batch][block-1]); slot 0 keeps the anchor. */
int dflash_draft_sample(int32_t batch, int32_t block, int32_t vocab, float temperature, const float *w,
                        int32_t *draft_tokens, dflash_workspace *ws, dflash_stream_t stream);
/* After target_verify of the drafted block (commit = 0): verification by the
 * rule above with u [batch][block-1] and v [batch], then the same rollback as
 * dflash_accept_rollback: emitted = d_1..d_a and the drawn token (a + 1
 * tokens) appended to stream; target len += a + 1; anchor = the drawn token;
 * n_pend = a + 1; accept_len[b] = a (nullable).  Reads both workspace logit
 * buffers; a drafted id outside [0, vocab) sets DFLASH_STATUS_BOUNDS and stops
 * that sequence's acceptance there. */
int dflash_accept_sample(const int32_t *draft_tokens, int32_t batch, int32_t block, int32_t vocab,
                         float temperature, const float *u, const float *v, dflash_cache *target_cache,
                         int32_t *anchor, int32_t *n_pend, int32_t *accept_len, int32_t *stream,
                         int32_t *stream_len, int32_t stream_cap, dflash_workspace *ws,
                         dflash_stream_t cuda_stream);
/* One draw per row of float32 logits [rows][vocab] at temperature T with
 * v[rows]: out[rows] (autoregressive sampling, the prefill's first token). */
int dflash_sample(const float *logits, int32_t rows, int32_t vocab, float temperature, const float *v,
                  int32_t *out, dflash_workspace *ws, dflash_stream_t stream);

/* -------------------------------------------------------- building blocks
 * The kernels behind the stages, exposed for unit parity tests. */

/* y[n][m] = sum_k x[n][k] w[m][k]; x [rows][K] (dtype), w [M][K] (dtype),
 * y [rows][M] float32.  rows <= 128. */
int dflash_linear(int32_t dtype, const void *x, const void *w, float *y, int32_t rows, int32_t M,
                  int32_t K, dflash_workspace *ws, dflash_stream_t stream);
/* y = x / sqrt(mean(x^2) + eps) * gain, x float32 [rows][H] -> y dtype. */
int dflash_rmsnorm(int32_t dtype, const float *x, const void *gain, void *y, int32_t rows,
                   int32_t H, float eps, dflash_stream_t stream);
/* Greedy token and top-2 gap of float32 logits [rows][V] ([DD] §1.1 greedy
 * choice; lowest index on ties). */
int dflash_argmax(const float *logits, int32_t rows, int32_t V, int32_t *argmax, float *gap,
                  dflash_workspace *ws, dflash_stream_t stream);
/* dflash_argmax without a workspace.  Not an operation of the method (the
 * pages have no counterpart): the same greedy token and top-2 gap of float32
 * logits [rows][V], for callers that cannot allocate device memory.  Such
 * callers hold no dflash_workspace, whose allocation needs both model
 * descriptors and reserves activation buffers sized for them, and cannot add
 * a cudaMalloc/cudaFree of their own: a sampler handed another engine's
 * logits in a serving loop whose memory is owned by a caching allocator, or
 * a loop where cudaFree's implicit device synchronisation would stall the
 * pipeline.
 *   Scratch: a fixed file-scope device array in the library (slice partials
 *   and per-row tickets, about 33 KiB per device) for at most
 *   DFLASH_ARGMAX_NOALLOC_MAX_ROWS rows; rows above it return
 *   DFLASH_ERR_TOO_LARGE before any CUDA call.  The library calls no
 *   allocator on this path.
 *   Set-up: the first call in each CUDA context (per device, with that device
 *   current) resolves the array's address (cudaGetSymbolAddress, return code
 *   checked; a failure returns DFLASH_ERR_CUDA and the next call retries).
 *   The library remembers the context's unique id and resolves again when it
 *   changes, e.g. after cudaDeviceReset.  Make the first call in a context
 *   before any stream capture begins.  Devices with an ordinal of 64 or more
 *   return DFLASH_ERR_INVALID_ARG.
 *   Each call clears the rows' tickets (an asynchronous memset on `stream`)
 *   and launches one kernel.  All calls on a device share the one array:
 *   calls that overlap in time (other streams, other host threads) race on
 *   it and must be serialised by the caller.
 *   argmax [rows] int32 and gap [rows] float32 (may be NULL) are device
 *   pointers; status (device int32, may be NULL) has DFLASH_STATUS_NONFINITE
 *   OR-ed in when a row holds NaN/Inf. */
#define DFLASH_ARGMAX_NOALLOC_MAX_ROWS 128
int dflash_argmax_noalloc(const float *logits, int32_t rows, int32_t V, int32_t *argmax,
                          float *gap, int32_t *status, dflash_stream_t stream);
/* Attention of q [batch][n][nq][hd] (dtype, RoPE applied) against layer
 * `layer` of `cache` (positions 0 .. len[b] + n - 1, the block's own keys
 * already written at len[b] ..), causal (row j sees 0..len+j) or not (every
 * row sees 0..len+n-1).  window > 0 drops the keys below len - window (the
 * drafter's cross-context window, see dflash_draft.cross_ctx); 0 keeps all.
 * out [batch][n][nq * hd] dtype.  q, out: device
 * pointers owned by the caller; q must be 16-byte aligned (the bf16 path
 * loads it by TMA), else DFLASH_ERR_INVALID_ARG before any CUDA call.  With
 * a DFLASH_KV_Q8 cache q is IEEE half precision (out stays bf16) and the
 * keys/values are the cache's codes times their row scales.
 * The scaled dot-product attention of "DFlash 深度解析" §2.2
 * draft_inference, evaluated per key group: the bf16 path splits the keys
 * into groups of a fixed number of 128-key tiles (a property of the cache),
 * keeps one running (max, sum, output) per row and group, and merges the
 * groups in order; the fp32 path does the same with 256-position chunks.
 * A row's result depends only on its own query and keys. */
int dflash_attention(const dflash_model_desc *d, const void *q, int32_t batch, int32_t n,
                     int32_t causal, int32_t window, dflash_cache *cache, int32_t layer, void *out,
                     dflash_workspace *ws, dflash_stream_t stream);

/* ----------------------------------------------------------------- KV pages
 * Keys and values of many sequences in pages of a common pool, for callers
 * that schedule more sequences than fit as whole caches or let sequences share
 * pages.  Not an operation of the method's pages ([DD] keeps one cache per
 * sequence); the same rotation and scaled dot-product attention, with another
 * place for the keys.  These calls stand beside dflash_attention: they take
 * any batch, rows of any number up to the workspace's, float32 or bf16 with
 * head_dim 64 or 128 and up to 64 query heads per KV head.
 *
 * The pool is the caller's memory: k and v, each
 * [n_layers][n_pages][n_kv][page_size][head_dim] in the model dtype, 16-byte
 * aligned, kept alive while the handle lives.  Copying, swapping or sharing
 * pages is the caller's.  page_size is 16, 32, 64 or 128.
 *
 * Every call takes, as device int32 arrays read when the kernels run:
 *   table [batch][table_stride]  page of each page_size positions: position p
 *                                of sequence b is slot p % page_size of page
 *                                table[b][p / page_size].  Only entries of
 *                                pages with a position that is written, or that
 *                                some row of the call sees, are read: pages
 *                                behind a window may have been given away;
 *   len [batch]                  positions held before this call's rows;
 *   n_rows [batch] (nullable)    rows of the sequence in this call, 0..n (values
 *                                outside are clamped); NULL: n for all.  Rows at
 *                                or past it are padding: their inputs are not
 *                                used and their outputs are left as they were.
 * len does not move: the caller adds the rows it keeps, after its last layer.
 * Device conditions set bits in the workspace's status word: a row's position
 * below 0, past the table or past max_pos sets DFLASH_STATUS_CAPACITY, a page outside
 * [0, n_pages) DFLASH_STATUS_BOUNDS; that write is skipped, that sequence's
 * attention output is unspecified, other sequences are not touched. */
typedef struct dflash_pages dflash_pages;
/* The handle: geometry, the rotation table (cos/sin of positions
 * 0..max_pos-1, angles in double precision, library-owned device memory) and
 * the pool's tensor maps.  Bound to the device current at the call; calls with
 * another device current return DFLASH_ERR_INVALID_ARG.  d supplies head
 * counts, head_dim, rope_theta and dtype. */
int dflash_pages_create(const dflash_model_desc *d, int32_t n_layers, int32_t n_pages, int32_t page_size,
                        int32_t max_pos, void *k, void *v, dflash_pages **out);
/* The same over a pool of 8-bit keys and values, half of bf16's bytes: k and v
 * [n_layers][n_pages][n_kv][page_size][head_dim] uint8 codes, k_scales and
 * v_scales [n_layers][n_pages][n_kv][page_size] float32, all 16-byte aligned and
 * apart from one another.  A row of head_dim entries is kept as dflash_cache_alloc_ex's
 * DFLASH_KV_Q8 keeps one, the entry (u - 128) s with s = max|x| / 127 and
 * u = 128 + round-half-even(x / s), x the row's float32 entries after the rotation
 * (a row of zeros: s = 0; one that holds a value that is not finite: s = NaN, so
 * it reads back as NaN).  Every call below takes such a handle, of float32 models
 * and of head_dim 64 too: dflash_paged_append quantises, the attention calls and
 * dflash_paged_read take an entry as its exact value (u - 128) s. */
int dflash_pages_create_q8(const dflash_model_desc *d, int32_t n_layers, int32_t n_pages, int32_t page_size,
                           int32_t max_pos, void *k, void *v, float *k_scales, float *v_scales, dflash_pages **out);
int dflash_pages_free(dflash_pages *p);
/* Scratch for the attention calls on handles of d's head counts and head_dim,
 * with at most max_batch sequences and batch * n <= max_rows, and a status
 * word.  Library-owned; one workspace serves one stream at a time, and so do
 * graphs captured with it: graphs that may run at once need one each.  The
 * partial results of the attention take 4 * max_rows * nq rows of hd + 2 floats,
 * 1.4 GB for 16384 rows of 40 heads of 128 (half of it for shared lengths), and
 * up to 40 MB more for the pieces; the append uses the status word alone, so any
 * workspace of the device serves it. */
typedef struct dflash_paged_workspace dflash_paged_workspace;
int dflash_paged_workspace_alloc(const dflash_model_desc *d, int32_t max_batch, int32_t max_rows,
                                 dflash_paged_workspace **out);
int dflash_paged_workspace_free(dflash_paged_workspace *w);
/* Synchronises `stream` (the one that the workspace's calls were made on),
 * returns the status bits in *status_out and clears them.  After
 * DFLASH_STATUS_TIMEOUT (a wait ran out) the results of the calls since the last
 * status are unspecified. */
int dflash_paged_status(dflash_paged_workspace *w, dflash_stream_t stream, int32_t *status_out);

/* Append with the rotation on the way: row (b, j), j < n_rows[b], of qkv
 * [batch][n] rows of q|k|v heads, ld elements apart (ld >= (nq + 2 nkv) * hd),
 * sits at position len[b] + j.  q and k are rotated at that position
 * (rotate-half pairs, float32, rounded once); q goes to q_out
 * [batch][n][nq][hd] (model dtype, 16-byte aligned), k and v into the pages.
 * q_out NULL: the rows hold k|v only (injected context).  in_dtype is the type
 * of qkv: the model dtype, or float32 (the weight product's result).  qkv may
 * have any alignment of its type; rows on 16-byte boundaries are read in wide
 * loads.  q_out, qkv and the two pools do not overlap (DFLASH_ERR_INVALID_ARG), and no
 * two rows of one call may name the same slot. */
int dflash_paged_append(dflash_pages *p, int32_t layer, int32_t in_dtype, const void *qkv, int64_t ld,
                        int32_t batch, int32_t n, const int32_t *n_rows, const int32_t *table,
                        int32_t table_stride, const int32_t *len, void *q_out, dflash_paged_workspace *ws,
                        dflash_stream_t stream);

/* Rows back out of the pages, as dflash_cache_write takes them: position
 * start[b] + j, j < n_rows[b], of sequence b goes to k_out and v_out
 * [batch][n_kv][n][head_dim] (row j of each head), of the model dtype or float32,
 * 16-byte aligned; either may be NULL.  8-bit entries are rounded once to the
 * type.  Rows at or past n_rows[b], and those whose position or page sets a status
 * bit, are left as they were.  To move a sequence to a cache or to other pages, or
 * to look at what was kept. */
int dflash_paged_read(dflash_pages *p, int32_t layer, int32_t out_dtype, int32_t batch, int32_t n,
                      const int32_t *n_rows, const int32_t *table, int32_t table_stride, const int32_t *start,
                      void *k_out, void *v_out, dflash_paged_workspace *ws, dflash_stream_t stream);

/* Attention over pages.  q [batch][n][nq][hd] (rotated, model dtype, 16-byte
 * aligned), the rows' own keys and values already appended; out likewise,
 * apart from q and from the pools (DFLASH_ERR_INVALID_ARG).
 * Row (b, i) at position p = len[b] + i sees key j of its sequence when
 *   causal      j <= p            and (j > p - window or j < sinks),
 *   not causal  j < len[b] + n_rows[b]  and (j >= len[b] - window or j < sinks);
 * window = 0 drops the second condition (sinks is then ignored).  The causal
 * window slides with each row; the other is dflash_attention's, the drafter's
 * cross-context window, with first tokens kept.  scale 1 / sqrt(hd), softmax
 * in float32; a row's result depends on the keys it sees only, whatever values
 * lie in hidden or unused slots.  In bf16 a softmax weight enters the product
 * with the values as a pair of bf16, off by 2^-16 of itself, where a sequence has
 * at most 32 rows n * nq / nkv (with a shared length: the batch at most 16), and
 * rounded to bf16 once, 2^-8 of itself, beyond: there a block's row and the same
 * row as a single token may differ by 2^-8 of the attention of |values|, besides
 * their own rounding.  Over 8-bit pages, whatever the rows, it enters, with its
 * value's scale, as a pair of halves, off by 2^-22 of itself or 2^-32 of the row's
 * largest; queries enter as halves, each row by a power of two, exact but for
 * entries 2^25 below the row's largest.  The keys are split over the GPU by all
 * lengths of the call, so the last bits of a row may depend on the batch it is
 * in (dflash_attention, which fixes the split per cache, has no such
 * dependence); equal calls give equal bits.
 * DFLASH_ERR_TOO_LARGE: a table of more than 2^30 positions, or work that could
 * outgrow the plan's 32-bit numbers, (groups of rows) * nkv * (positions of a
 * table row, max_pos at most) / 64 in bf16 and / 32 in float32 at 2^30 or more.
 * A group holds up to 256 (float32: 64; 8-bit pages of bf16 models: 128) of a sequence's n * nq / nkv rows; a
 * shared prefix adds the groups of the whole batch's. */
int dflash_paged_attention(dflash_pages *p, int32_t layer, const void *q, int32_t batch, int32_t n,
                           const int32_t *n_rows, int32_t causal, int32_t window, int32_t sinks,
                           const int32_t *table, int32_t table_stride, const int32_t *len, void *out,
                           dflash_paged_workspace *ws, dflash_stream_t stream);
/* The same for a batch whose first *shared_len positions (device int32) hold
 * the same keys and values in every sequence with rows in this call: those are
 * read once for the whole batch, from the pages that the first such sequence's
 * table names, with all sequences' rows stacked against them.  Values of
 * *shared_len outside [0, min len] are clamped to it.  Over 8-bit pages the call
 * pays where most keys are common: the whole batch's rows choose the kernel for the
 * sequences' own keys too, which can make those of single tokens three times slower. */
int dflash_paged_attention_shared(dflash_pages *p, int32_t layer, const void *q, int32_t batch, int32_t n,
                                  const int32_t *n_rows, int32_t causal, int32_t window, int32_t sinks,
                                  const int32_t *table, int32_t table_stride, const int32_t *len,
                                  const int32_t *shared_len, void *out, dflash_paged_workspace *ws,
                                  dflash_stream_t stream);

/* --------------------------------------------------------- weights in 4 bits
 * Products with weight matrices of 4-bit codes and a scale for each group of
 * columns: what the quantised targets of the pages' engines keep ("DFlash
 * 深度解析" §7; Q4 files of [RD] and the datacamp tutorial, named there, not
 * shown), read as the plain affine form
 *   w[m][k] = s[m][k / group] (code[m][k] - zero[m][k / group]),
 * codes and zero points 0..15, zero point 8 for a matrix without zeros.  A decode
 * step reads its weights once; in 4 bits they are a quarter of the bytes.  These
 * calls stand beside dflash_linear.
 *
 * A matrix lives in one buffer of the caller's, dflash_w4_bytes long and 16-byte
 * aligned, in the order in which the products read it (blocks of 128 rows by 128
 * columns, each its codes, then its scales, then its zero points; rows and
 * columns past M and K are padding).  dflash_w4_pack fills it from plain arrays,
 * dflash_w4_quantize from a matrix, dflash_w4_unpack reads it back.  group is 32,
 * 64 or 128 and divides K (else DFLASH_ERR_UNSUPPORTED_SHAPE); M is any; M K at
 * most 2^34 (else DFLASH_ERR_TOO_LARGE).  Buffers that one of these calls writes
 * overlap none that it reads (DFLASH_ERR_INVALID_ARG).  Products read a matrix
 * before they wait for the kernels ahead of them in their stream (they are launched
 * as programmatic dependents): a kernel of the caller's own that fills `packed`
 * itself must not let its dependents start early, and has to make its stores
 * visible to asynchronous copies before its end (__threadfence, fence.proxy.async);
 * copies need nothing. */
typedef struct dflash_w4 {
  int32_t M, K, group;
  int32_t scale_dtype; /* DFLASH_F32 | DFLASH_BF16 */
  int32_t zeros;       /* 0: no zero points */
  void *packed;
} dflash_w4;
/* Bytes of the buffer (w->packed is not looked at), or a negative DFLASH_ERR_*. */
int64_t dflash_w4_bytes(const dflash_w4 *w);
/* From codes [M][K / 2] (uint8: the even column's code in the low half), scales
 * [M][K / group] of the scale type and zeros [M][K / group] (uint8, values above
 * 15 count as 15; given exactly when w->zeros). */
int dflash_w4_pack(const dflash_w4 *w, const void *codes, const void *scales, const void *zeros,
                   dflash_stream_t stream);
/* The nearest codes of a finite matrix src [M][K] of type dtype, rows ld elements
 * apart.  Without zeros s = max|w| / 7 over a group and code = rhe(w / s) + 8;
 * with them, over the range [min, max] stretched to hold 0, s = (max - min) / 15,
 * zero = rhe(-min / s) and code = rhe(w / s) + zero; s is rounded to the scale
 * type first and codes are clamped to 0..15 (rhe: round half to even; a group of
 * zeros has s = 0).  Entries up to 3e38 in size have finite nearest values. */
int dflash_w4_quantize(const dflash_w4 *w, int32_t dtype, const void *src, int64_t ld, dflash_stream_t stream);
/* dst [M][K] of type dtype: the values, rounded once. */
int dflash_w4_unpack(const dflash_w4 *w, int32_t dtype, void *dst, dflash_stream_t stream);

/* Scratch of the products: partial sums for up to max_rows (<= 128) rows, whatever
 * the matrix (0.6 MB a row up to 16 rows, 10 MB up to 64, 20 MB beyond), and a
 * status word.  Library-owned; bound to the device current at the call; one
 * workspace serves one stream at a time, and so do graphs captured with it:
 * graphs that may run at once need one each. */
typedef struct dflash_w4_workspace dflash_w4_workspace;
int dflash_w4_workspace_alloc(int32_t max_rows, dflash_w4_workspace **out);
int dflash_w4_workspace_free(dflash_w4_workspace *ws);
/* Synchronises `stream` (the one that the workspace's calls were made on), returns
 * the status bits in *status_out and clears them.  After DFLASH_STATUS_TIMEOUT (a
 * wait ran out) the results of the calls since the last status are unspecified. */
int dflash_w4_status(dflash_w4_workspace *ws, dflash_stream_t stream, int32_t *status_out);

/* y[n][m] = sum_k x[n][k] w[m][k] (+ add[n][m]).  x [rows][K] of type dtype (the
 * model's), rows ldx elements apart, of any alignment of its type; rows up to the
 * workspace's.  swiglu = 0: y float32 [rows][M]; add, nullable, float32 [rows][M],
 * is y itself (a residual stream) or apart from it.  swiglu = 1, M even: y
 * [rows][M / 2] of type dtype, y[n][f] = silu(row 2f) * (row 2f + 1), the gate/up
 * order of dflash_layer_w; add comes before the activation.
 * Codes less zero points are small integers, exact in bf16; products are summed
 * in float32 and the scale is applied to a group's sum, so the only roundings are
 * float32's.  A row's result depends on its own x and the matrix only, and equal
 * calls give equal bits; in bf16 neither do the other rows' number and values change
 * its bits up to 16 rows, nor from 17 on (between the two, and in float32, sums are
 * taken in other orders). */
int dflash_linear_w4(int32_t dtype, const void *x, int64_t ldx, const dflash_w4 *w, const float *add,
                     int32_t swiglu, void *y, int32_t rows, dflash_w4_workspace *ws, dflash_stream_t stream);

/* Kernel timing for measurement passes (not for graph capture): between
 * begin and end, the library brackets each weight-GEMM launch with a CUDA
 * event pair on the launching stream, up to max_records launches.  end
 * synchronises on the last event and returns per launch the elapsed
 * milliseconds and the tags (M, K, rows); *n_out = records returned. */
int dflash_profile_begin(int32_t max_records);
int dflash_profile_end(float *ms_out, int32_t *tags_out, int32_t max, int32_t *n_out);
/* Number of kernel launches this library has enqueued (or recorded into a
 * graph under capture) since it was loaded, counted on the host. */
long long dflash_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif /* DFLASH_H_ */
