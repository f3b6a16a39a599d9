/*
 * psi_verify.h - C ABI of the Psi-Spec verify step on NVIDIA B200 (sm_100a).
 *
 * The verify step of the Psi-Spec sampler: the frozen AR path has scored a
 * block of B drafted tokens (B+1 logit rows, the last one being the bonus
 * row), the diffusion-LoRA draft supplied B logit rows and the drafted ids.
 * Per sequence the step keeps the longest prefix of drafted tokens that
 * passes speculative rejection sampling, then emits one correction token
 * (drawn from the residual at the first rejection) or one bonus token (drawn
 * from the bonus row when every draft passed).
 *
 * Sources (page title, section):
 *  [P1] "Uno / Psi-Spec - 같은 모델 안에서 초안 뽑고 AR로 도장 찍기"
 *       (lanes-ecd.pages.dev): "어디서 왔나" (the Leviathan et al. 2023
 *       draft -> verify -> correct rule), "Psi-Spec이 한 스텝에서 하는 일"
 *       (longest consecutive accepted prefix; lossless).
 *  [P3] "Uno Psi-Spec 是什麼？Diffusion-Augmented LLM 如何保留 AR 分布、
 *       一次驗證多個 Token" (alphalab.site): "Uno Psi-Spec 怎麼運作？完整走一次
 *       四個 Token" (steps 3-4: rejection rule, longest accepted prefix,
 *       residual correction; bonus token from the block-end logits; TPF
 *       bound), "Linear 與 Tree sampler" (tree verify), "想跑 Uno：先確認官方
 *       程式需要的環境" (temperature and top-p on the run card).
 *
 * Conventions shared by every entry point:
 *  - All array arguments are DEVICE pointers owned by the caller.  The
 *    library allocates nothing and keeps no data between calls (only
 *    per-device launch settings, made on a device's first call).
 *  - Calls are asynchronous on `stream` (NULL = the legacy default stream).
 *    After a device's first call, a call only launches work on `stream`, so
 *    it can be captured into a CUDA graph; its scalar arguments (seed, step,
 *    sizes) are then fixed in the graph.
 *  - Argument errors are detected on the host before any launch and
 *    returned as a psi_status; nothing is launched in that case.
 *  - Data errors found on the device (an id outside [0, V), a bad parent
 *    index, a NaN or +inf logit) are OR-ed into *dev_status (a caller-owned
 *    device uint32 that the caller zeroes; NULL = not reported).  The
 *    kernels always run to completion: they never trap, and the only waits
 *    (for bulk copies into shared memory) give up after a time limit.
 *  - Logits are bfloat16 or float32, row-major; `*_row_stride` is the
 *    distance between consecutive rows in ELEMENTS (>= V).  Sampled rows
 *    whose start is 16-byte aligned take the streaming path, others the
 *    cluster path; both give the same results.
 *  - Calls that overlap in time must not share a workspace, outputs, or a
 *    part of the cache that one of them writes; calls on one stream, and
 *    graphs replayed one after the other, may.
 *  - Randomness: the acceptance uniform of row i and the correction/bonus
 *    uniform of the emitting row are a counter-based hash of
 *    (seed, sequence id, step, row, purpose), so a step replays exactly from
 *    its counters and results do not depend on batch composition.
 */
#ifndef PSI_VERIFY_H
#define PSI_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
typedef struct CUstream_st *psi_stream_t; /* same type as cudaStream_t */

typedef enum psi_status {
  PSI_OK = 0,
  PSI_ERR_INVALID_ARG = 1, /* null pointer, size or parameter out of range */
  PSI_ERR_MISALIGNED = 2,  /* pointer not aligned to its element type */
  PSI_ERR_UNSUPPORTED = 3, /* valid but beyond this build (e.g. V too large) */
  PSI_ERR_CUDA = 4,        /* a CUDA launch or query failed */
  PSI_ERR_WORKSPACE = 5,   /* workspace NULL or smaller than the query says */
  PSI_ERR_TIMEOUT = 6      /* reserved, not returned: a kernel's wait that
                              gives up sets PSI_DEV_TIMEOUT instead */
} psi_status;

typedef enum psi_dtype { PSI_DTYPE_F32 = 0, PSI_DTYPE_BF16 = 1 } psi_dtype;

/* Bits OR-ed into *dev_status by the kernels. */
#define PSI_DEV_BAD_TOKEN_ID 1u /* drafted or node id outside [0, V): treated
                                   as rejected / unmatched */
#define PSI_DEV_BAD_PARENT 2u   /* parent index >= own index or < -1: node
                                   unmatched */
#define PSI_DEV_NONFINITE 4u    /* a NaN or +inf logit was read (-inf is a
                                   valid logit: probability zero) */
#define PSI_DEV_TIMEOUT 8u      /* a bounded wait inside a kernel gave up;
                                   never expected; outputs are then invalid */
#define PSI_DEV_BAD_PAGE 16u    /* cache: a position without a valid page (past
                                   the sequence's table, or a page index outside
                                   the pool), a page released more often than it
                                   is held, or a stack entry that is no free
                                   page: that position is left out */
#define PSI_DEV_NO_PAGES 32u    /* cache: not enough free pages, or no room in
                                   the sequence's table: it got none */
#define PSI_DEV_BAD_PATH 64u    /* cache: an accepted path that is not ascending
                                   within [0, M): cut at its first bad node */
#define PSI_DEV_BAD_SEQ 128u    /* cache: a fork whose rows are out of range,
                                   repeated or not empty: it is left out */

/* RNG purposes (the last hash input). */
#define PSI_PURPOSE_ACCEPT 0u /* u_i of the acceptance test of row i */
#define PSI_PURPOSE_RESID 1u  /* u' of the correction / bonus draw */

/* Largest supported block and vocabulary. */
#define PSI_MAX_B 32
#define PSI_MAX_V 393216
#define PSI_MAX_TREE_NODES 4096
/* Early-exit rounds of the linear verify (see psi_verify_linear): the first
 * PSI_X_SHORT_ROUNDS rounds cover PSI_X_ROUND_POSITIONS positions each, one
 * last round covers the rest of the B + 1 positions (X = SAMPLED for T > 0,
 * GREEDY for T == 0). */
#define PSI_SAMPLED_ROUND_POSITIONS 2
#define PSI_SAMPLED_SHORT_ROUNDS 2
#define PSI_GREEDY_ROUND_POSITIONS 3
#define PSI_GREEDY_SHORT_ROUNDS 3
/* Smallest batch that takes the early-exit rounds (smaller batches are
 * latency-bound: one pass over every row is faster). */
#define PSI_EARLY_EXIT_MIN_N 64

/* Workspace needed by psi_verify_linear for these sizes (bytes, a multiple
 * of 256; 0 on invalid sizes).  The workspace needs no initialisation. */
size_t psi_verify_linear_workspace_bytes(int32_t N, int32_t B, int32_t V,
                                         psi_dtype dtype, float temperature,
                                         float top_p);

/*
 * psi_verify_linear - linear (single-path) verify of N sequences.
 *
 * [P1] "Psi-Spec이 한 스텝에서 하는 일"; [P3] "完整走一次四個 Token" steps
 * 3-4 and the bonus paragraph; temperature / top-p: [P3] run card.
 *
 * For T > 0, per sequence n and row i:
 *   p_i = softmax(ar[n][i] / T), q_i = softmax(draft[n][i] / T); with
 *   top_p < 1 each is cut to its smallest descending-probability set of mass
 *   >= top_p (keeping every token tied with the last one admitted) and
 *   renormalised.  Draft x_i is accepted iff u_i * q_i(x_i) < p_i(x_i) with
 *   u_i = U(seed, seq, step, i, ACCEPT).  L = first rejected row (B if none).
 *   If L < B the correction is the inverse-CDF draw, in vocabulary order,
 *   from max(0, p_L - q_L) at u' = U(seed, seq, step, L, RESID) (from p_L
 *   itself if that residual is all zero, which needs q_L(x_L) = 0); if
 *   L == B the bonus token is drawn from p_B the same way.
 * For T == 0 (greedy): a_i = argmax of ar[n][i] (lowest index on ties);
 *   accept while x_i == a_i; emit a_L.  draft_logits may be NULL and top_p
 *   is ignored.
 *
 * ar_logits     [N][B+1] rows of V logits (row B = bonus row), stride
 *               ar_row_stride elements.
 * draft_logits  [N][B] rows, stride draft_row_stride (ignored if T == 0).
 * draft_ids     int32 [N][B].
 * seq_ids       uint64 [N] sequence ids for the RNG, or NULL (= n).
 * out_tokens    int32 [N][B+1]: x_0..x_{L-1}, then the emitted token, then -1.
 * out_n_emitted int32 [N]: L + 1, in 1..B+1.
 * out_p_draft, out_q_draft  float [N][B] or NULL: p_i(x_i), q_i(x_i) after
 *               top-p (T > 0 only; not written when T == 0).
 * Early exit (both out_p_draft and out_q_draft NULL, N >= PSI_EARLY_EXIT_MIN_N,
 *   any T): rows after a sequence's first rejection (or greedy mismatch) do
 *   not change its result, so positions are verified in rounds
 *   (PSI_SAMPLED_ROUND_POSITIONS positions each for the first
 *   PSI_SAMPLED_SHORT_ROUNDS rounds, PSI_GREEDY_ROUND_POSITIONS for the first
 *   PSI_GREEDY_SHORT_ROUNDS, then the rest), and a sequence takes
 *   part in a round only if every draft of the earlier rounds was accepted.
 *   Tokens and counts are the same as with every row read; the NONFINITE
 *   status bit then covers the rows that were read.  A caller passing p / q
 *   buffers (for T == 0 they are not written) gets every row read.
 * Limits: 1 <= N, 1 <= B <= PSI_MAX_B, 1 <= V <= PSI_MAX_V, T >= 0 and
 *   finite, 0 < top_p <= 1.
 */
psi_status psi_verify_linear(const void *ar_logits, int64_t ar_row_stride,
                             const void *draft_logits,
                             int64_t draft_row_stride, psi_dtype dtype,
                             const int32_t *draft_ids, int32_t N, int32_t B,
                             int32_t V, float temperature, float top_p,
                             uint64_t seed, const uint64_t *seq_ids,
                             uint64_t step, int32_t *out_tokens,
                             int32_t *out_n_emitted, float *out_p_draft,
                             float *out_q_draft, uint32_t *dev_status,
                             void *workspace, size_t workspace_bytes,
                             psi_stream_t stream);

/* Workspace needed by psi_verify_linear_topk (bytes; the same as
 * psi_verify_linear's for these sizes; 0 on invalid sizes). */
size_t psi_verify_linear_topk_workspace_bytes(int32_t N, int32_t B, int32_t V,
                                              psi_dtype dtype, float temperature,
                                              float top_p, int32_t top_k);

/*
 * psi_verify_linear_topk - psi_verify_linear with a top-k cut.
 *
 * Source: the run card ("想跑 Uno：先確認官方程式需要的環境") names top-k
 * beside top-p and temperature as sampler settings.  Reading of the order:
 * top-k is taken on the temperature softmax first (every token whose
 * probability is at least the k-th largest stays, ties with the k-th
 * included), the kept mass is renormalised, and top-p then cuts that
 * distribution as in psi_verify_linear.  It applies to p_i and q_i alike, so
 * the acceptance test, the residual and the bonus draw all use the cut
 * distributions.
 *
 * Arguments, results, layouts and limits as psi_verify_linear, plus
 * top_k: 0 = off; top_k >= V keeps every token (also off); negative values
 *   return PSI_ERR_INVALID_ARG.  Ignored when T == 0 (the argmax is always
 *   kept).
 * With top_k off the call is psi_verify_linear.  Rows whose set-aside
 * candidates (the elements near the maximum that the streaming scan keeps)
 * number at least k are finished from them; the other units (large k, flat
 * rows, or rows that do not start on a 16-byte boundary) go to a slower
 * whole-row path that reads their two rows a few more times.  Results do
 * not depend on which path a unit takes.
 */
psi_status psi_verify_linear_topk(const void *ar_logits, int64_t ar_row_stride,
                                  const void *draft_logits,
                                  int64_t draft_row_stride, psi_dtype dtype,
                                  const int32_t *draft_ids, int32_t N, int32_t B,
                                  int32_t V, float temperature, float top_p,
                                  int32_t top_k, uint64_t seed,
                                  const uint64_t *seq_ids, uint64_t step,
                                  int32_t *out_tokens, int32_t *out_n_emitted,
                                  float *out_p_draft, float *out_q_draft,
                                  uint32_t *dev_status, void *workspace,
                                  size_t workspace_bytes, psi_stream_t stream);

/*
 * psi_verify_linear_noalloc - psi_verify_linear for callers that cannot
 * allocate device memory (no counterpart on the pages: an integration
 * variant, same arithmetic and results as psi_verify_linear).
 *
 * Arguments and results as psi_verify_linear, without the workspace: the
 * call uses a scratch array of PSI_NOALLOC_SCRATCH_BYTES that the library
 * holds in device memory (one per device, created with the library's module;
 * nothing is allocated at run time).  Its address is looked up once per
 * device, on the first call made with that device current; make that first
 * call before capturing the stream into a graph, since it issues a
 * runtime query besides the launches.  The address is kept for the life of
 * the process: it belongs to the device's primary context, so after that
 * context is torn down (cudaDeviceReset) this entry point must not be used
 * on that device again until the library is reloaded.  The scratch needs no initialisation:
 * what the verify needs zeroed it clears itself on every call.
 * Calls that overlap in time on the same device share the scratch and race:
 * the caller serialises them (one stream, or events between streams).
 * Returns PSI_ERR_UNSUPPORTED, without launching anything, when
 * psi_verify_linear_workspace_bytes for these sizes exceeds
 * PSI_NOALLOC_SCRATCH_BYTES (the sampled path needs about 65.7 KB per logit
 * row, N * (2B + 1) rows: e.g. N <= 7 at B = 8; the greedy path far less),
 * and PSI_ERR_CUDA if the scratch address cannot be obtained.
 */
#define PSI_NOALLOC_SCRATCH_BYTES 8388608u /* 8 MiB */
psi_status psi_verify_linear_noalloc(const void *ar_logits, int64_t ar_row_stride,
                                     const void *draft_logits,
                                     int64_t draft_row_stride, psi_dtype dtype,
                                     const int32_t *draft_ids, int32_t N, int32_t B,
                                     int32_t V, float temperature, float top_p,
                                     uint64_t seed, const uint64_t *seq_ids,
                                     uint64_t step, int32_t *out_tokens,
                                     int32_t *out_n_emitted, float *out_p_draft,
                                     float *out_q_draft, uint32_t *dev_status,
                                     psi_stream_t stream);

/* Workspace needed by psi_verify_tree_greedy (bytes; 0 on invalid sizes).
 * The walk keeps its state in shared memory: 256 bytes for any valid sizes. */
size_t psi_verify_tree_greedy_workspace_bytes(int32_t N, int32_t M, int32_t V,
                                              psi_dtype dtype);

/*
 * psi_verify_tree_greedy - greedy (T = 0) verify of a draft tree per sequence.
 *
 * [P3] "Linear 與 Tree sampler": several high-probability candidates per
 * position pruned to a finite prefix tree and verified in one pass.
 *
 * ar_logits    [N][M+1] rows (row 0 = root, row k+1 = node k).
 * node_tokens  int32 [N][M]; parents int32 [N][M] (-1 = child of the root;
 *              otherwise 0 <= parent < own index).
 * Node k is matched iff node_tokens[k] == argmax(row of its parent) and its
 * parent is matched (or is the root).  The deepest matched node (lowest
 * index among equals) ends the accepted path; the bonus token is the
 * argmax of that node's own row (root row when nothing matched).
 * out_path_nodes int32 [N][M]: node indices root-side first, then -1.
 * out_path_len   int32 [N]: number of accepted nodes (0..M).
 * out_tokens     int32 [N][M+1]: accepted tokens, then the bonus, then -1.
 * Rows read: the root's and each matched node's only (level by level, one
 * cluster of CTAs per tree); the NONFINITE status bit covers those rows.
 * Invalid parents and token ids are flagged for every node.
 * Limits: 1 <= N, 1 <= M <= PSI_MAX_TREE_NODES, 1 <= V <= PSI_MAX_V.
 */
psi_status psi_verify_tree_greedy(const void *ar_logits, int64_t ar_row_stride,
                                  psi_dtype dtype, const int32_t *node_tokens,
                                  const int32_t *parents, int32_t N, int32_t M,
                                  int32_t V, int32_t *out_path_nodes,
                                  int32_t *out_path_len, int32_t *out_tokens,
                                  uint32_t *dev_status, void *workspace,
                                  size_t workspace_bytes, psi_stream_t stream);

/* Workspace needed by psi_verify_tree_sampled (bytes, a multiple of 256; 0 on
 * invalid sizes).  The workspace needs no initialisation. */
size_t psi_verify_tree_sampled_workspace_bytes(int32_t N, int32_t M, int32_t V,
                                               psi_dtype dtype, float temperature,
                                               float top_p);

/*
 * psi_verify_tree_sampled - sampled (T > 0) verify of a draft tree per
 * sequence.
 *
 * [P3] "Linear 與 Tree sampler" (a prefix tree of candidates verified in one
 * pass) with the rejection rule and residual draw of [P3] "完整走一次四個
 * Token"; the pages give no sampled tree rule, and the one taken is
 * recursive rejection over each reached node's children (SpecInfer's
 * multi-candidate speculative sampling, Miao et al., ASPLOS 2024), every
 * child being a point-mass proposal:
 *   At a node whose AR row gives the target P (softmax at temperature T,
 *   cut to its top-p set as in psi_verify_linear), the valid children are
 *   tried in ascending index.  Child k with token x is accepted iff
 *   u_k * R < w(x), where w is what remains of P after the node's rejected
 *   tokens lost their mass (a repeated token has none left), R = sum(w) and
 *   u_k = U(seed, seq, step, k + 1, ACCEPT).  An accepted child becomes the
 *   next node.  When no child is accepted (or the node is a leaf) the step
 *   ends with the inverse-CDF draw, in vocabulary order, from w (from P if
 *   nothing remains) at u' = U(seed, seq, step, j, RESID), j being that
 *   node's row (0 = root).  Every emitted token then has the law of its
 *   node's P (lossless).
 * T == 0 is the greedy tree (psi_verify_tree_greedy; top_p ignored).
 * Arguments, layouts, validity rules and outputs as psi_verify_tree_greedy,
 * plus temperature, top_p (0 < top_p <= 1), seed, seq_ids (uint64 [N] or
 * NULL = n) and step as in psi_verify_linear.  out_tokens holds the accepted
 * tokens, then the drawn one, then -1.
 * Limits: as psi_verify_tree_greedy; T >= 0 and finite.
 */
psi_status psi_verify_tree_sampled(const void *ar_logits, int64_t ar_row_stride,
                                   psi_dtype dtype, const int32_t *node_tokens,
                                   const int32_t *parents, int32_t N, int32_t M,
                                   int32_t V, float temperature, float top_p,
                                   uint64_t seed, const uint64_t *seq_ids,
                                   uint64_t step, int32_t *out_path_nodes,
                                   int32_t *out_path_len, int32_t *out_tokens,
                                   uint32_t *dev_status, void *workspace,
                                   size_t workspace_bytes, psi_stream_t stream);

/* ---------------------------------------------------------------------------
 * The key-value cache around the verify step.
 *
 * Before the verify, the frozen AR path runs over the drafted block: each of
 * its attention layers writes the block's keys and values into the cache
 * (psi_cache_append) and attends over the cache (psi_attend_block).  After
 * it, the accepted nodes stay (psi_cache_commit), and the sequences' pages
 * are fitted to their new lengths (psi_cache_resize).  psi_cache_fork
 * continues a sequence more than once.  The pages name the block and the
 * prefix tree that is verified in one pass ([P3] "Linear 與 Tree sampler");
 * the cache's form is this library's.
 *
 * Pages.  Keys and values live in two pools of num_pages pages of page_size
 * slots.  Element d of head h in slot s of page p of layer l is at
 *   l * layer_stride + p * page_stride + s * slot_stride + h * head_stride + d
 * in both pools (strides in elements, so [page][slot][head][d] and
 * [page][head][slot][d] are both cache layouts).  Both pools and every
 * stride but that of d are multiples of 16 bytes, and head_dim is a multiple
 * of 8.  Position t of sequence n is slot t % page_size of page
 * page_table[n][t / page_size]; page_table is int32 [N][max_pages].
 *
 * Blocks.  A block has R rows per sequence, as the verify's logits do: row 0
 * is the root (the last emitted token, not in the cache yet), row k + 1 is
 * drafted token or tree node k, so R = B + 1 or M + 1, and R = 1 is a step
 * of one token.  lens[n] is the number of positions in the cache before the
 * block; row r of the block takes position lens[n] + r of the cache, and its
 * rotary position is lens[n] + its depth.  parents is int32 [N][R - 1] as in
 * the tree verify, or NULL for a chain (every row continues the one before
 * it).  A row whose chain of parents holds an invalid index (>= its own or
 * < -1) is not part of the block: nothing is written for it by
 * psi_cache_append, and it attends to nothing.  lens[n] < 0 marks a sequence
 * that is not there (a padded batch): all that belongs to it is left as it
 * was.
 * ------------------------------------------------------------------------- */
#define PSI_MAX_BLOCK_ROWS 256 /* rows of a block (R) */
#define PSI_MAX_HEAD_DIM 256
#define PSI_MAX_PAGE_SIZE 1024

typedef struct psi_cache_layout {
  psi_dtype dtype;   /* of keys, values and queries */
  int32_t layers;    /* layers of the pools (commit, fork); 1 elsewhere */
  int32_t num_pages; /* pages per layer */
  int32_t page_size; /* slots per page, 1..PSI_MAX_PAGE_SIZE */
  int32_t kv_heads;
  int32_t head_dim;  /* multiple of 8, up to PSI_MAX_HEAD_DIM */
  int64_t layer_stride, page_stride, slot_stride, head_stride;
} psi_cache_layout;

/*
 * psi_cache_append - norm, rotary positions and the write of a block's keys
 * and values into one layer's pages.
 *
 * For a head x of row r (queries and keys; values are stored as they are):
 *   y = x * rsqrt(mean(x^2) + eps) * weight   (y = x where weight is NULL)
 *   each pair (a, b) of y's first rotary_dim elements is turned by the angle
 *   t = position * inv_freq[i]: rope_scale * (a cos t - b sin t,
 *   b cos t + a sin t).  Pair i is elements (i, i + rotary_dim / 2), or with
 *   `interleaved` (2i, 2i + 1).  The rest of the head keeps y.
 * The angle is taken in double precision, the rest in float, and the result
 * is rounded once.  Scaled positions (linear, by wavelength, YaRN and the
 * like) are a choice of inv_freq and rope_scale.
 *
 * q  R rows per sequence of q_heads heads, k and v of kv_heads heads: row r
 *    of sequence n, head h starts at (n * R + r) * row_stride +
 *    h * head_stride elements, so the three may be slices of one projection.
 * q_weight, k_weight  head_dim weights of the block's dtype, or NULL.
 * inv_freq   double [rotary_dim / 2] radians per position; NULL with
 *            rotary_dim 0.  rotary_dim is even and at most head_dim.
 * out_q      [N][R][q_heads][head_dim]; may be q itself when q is that.
 * The pools must not overlap the block's tensors, and two rows of a call
 * must not share a slot (pages of a sequence's block belong to it alone).
 * Limits: 1 <= N, 1 <= R <= PSI_MAX_BLOCK_ROWS, eps >= 0.
 */
psi_status psi_cache_append(const psi_cache_layout *layout, void *k_pages, void *v_pages,
                            const int32_t *page_table, int32_t max_pages, const int32_t *lens,
                            int32_t N, int32_t R, int32_t q_heads, const void *q,
                            int64_t q_row_stride, int64_t q_head_stride, const void *k,
                            int64_t k_row_stride, int64_t k_head_stride, const void *v,
                            int64_t v_row_stride, int64_t v_head_stride, const void *q_weight,
                            const void *k_weight, float eps, const double *inv_freq,
                            int32_t rotary_dim, int32_t interleaved, float rope_scale,
                            const int32_t *parents, void *out_q, uint32_t *dev_status,
                            psi_stream_t stream);

/* Workspace needed by psi_attend_block (bytes, a multiple of 256; 0 on
 * invalid sizes).  The workspace needs no initialisation. */
size_t psi_attend_block_workspace_bytes(const psi_cache_layout *layout, int32_t N, int32_t R,
                                        int32_t q_heads, int32_t max_pages);

/*
 * psi_attend_block - attention of a block over one layer's pages.
 *
 * Row r of sequence n sees positions 0..lens[n]-1 and those rows of its own
 * block that are r or lie on r's path to the root (rows 0..r of a chain):
 *   o = sum_t p_t v_t,  p = softmax over the seen t of scale * (q . k_t)
 * with kv head h / (q_heads / kv_heads) for query head h.  What a row does
 * not see has no influence on it, whatever it holds.  A row that sees
 * nothing (invalid parents; no valid page), or whose scores are all -inf,
 * gives zeros.
 *
 * q         as in psi_cache_append; the block's keys and values are in the
 *           pages already.
 * out_o     [N][R][q_heads][head_dim], not overlapping any input.
 * out_lse   float [N][R][q_heads] or NULL: log of the sum of
 *           exp(scale * q . k_t) over the seen t, -inf for none.
 * Scores, the softmax and the sums are float; bf16 weights p are rounded to
 * bf16 for the product with v.  A score's rounding, 2^-24 of its size, is an
 * error of p's exponent, so scores should stay well below 2^20; sums of
 * bf16 values are finite for |v| times the length below 2^67.
 * The same call gives the same bits, and a sequence's bits do not depend on
 * what the other sequences hold (N, R and the tables' width decide how a
 * length is divided among CTAs).
 * Limits: as psi_cache_append; q_heads a multiple of kv_heads; scale finite.
 */
psi_status psi_attend_block(const psi_cache_layout *layout, const void *k_pages,
                            const void *v_pages, const int32_t *page_table, int32_t max_pages,
                            const int32_t *lens, int32_t N, int32_t R, int32_t q_heads,
                            const void *q, int64_t q_row_stride, int64_t q_head_stride,
                            const int32_t *parents, float scale, void *out_o, float *out_lse,
                            uint32_t *dev_status, void *workspace, size_t workspace_bytes,
                            psi_stream_t stream);

/*
 * psi_cache_commit - keep the accepted path of a tree verify.
 *
 * path_nodes int32 [N][M] and path_len int32 [N] are the tree verify's
 * outputs.  In every layer, keys and values of node path_nodes[n][j]
 * (position lens[n] + 1 + path_nodes[n][j]) move to position
 * lens[n] + 1 + j, and out_lens[n] = lens[n] + 1 + path_len[n]: the root and
 * the path.  (After a linear verify the accepted rows are in place already:
 * the new length is lens + n_emitted.)
 * A path must ascend within [0, M); it is cut at its first bad node.  A
 * position without a valid page is left out.
 * out_lens int32 [N], not overlapping lens (which every CTA reads).
 * The pages that hold a sequence's block must belong to it alone.
 */
psi_status psi_cache_commit(const psi_cache_layout *layout, void *k_pages, void *v_pages,
                            const int32_t *page_table, int32_t max_pages, const int32_t *lens,
                            int32_t N, int32_t M, const int32_t *path_nodes,
                            const int32_t *path_len, int32_t *out_lens, uint32_t *dev_status,
                            psi_stream_t stream);

/* Who holds which page.  Device pointers. */
typedef struct psi_page_state {
  int32_t *page_table;  /* [N][max_pages]; -1 where no page is held */
  int32_t *page_counts; /* [N] pages held: the row's first page_counts entries */
  int32_t *refs;        /* [num_pages] sequences that hold the page */
  int32_t *free_pages;  /* [num_pages] a stack of free pages */
  int32_t *n_free;      /* [1] its height */
} psi_page_state;

/*
 * psi_cache_resize - fit each sequence's pages to lens[n] + extra positions:
 * to room for the next block (extra = R), to what is held after a commit
 * (extra = 0), or to nothing (lens = 0, extra = 0: the sequence is freed).
 *
 * Pages over ceil((lens[n] + extra) / page_size) are released: their table
 * entries become -1 and refs falls by one; pages that nobody holds any more
 * are pushed on the free stack, lowest index first.  Then missing pages are
 * popped, in the order of (sequence, position); a sequence gets all that it
 * needs or none (and so do the later ones that need any, when the stack is
 * too low; a row too short for its sequence does not count).  A popped entry
 * that is not a free page (out of range, held by a sequence, or popped before
 * in the call) is flagged, and its place in the table becomes -1.
 * lens[n] < 0: left as it is.
 * in and out may be the same state, or hold ten different arrays; table
 * entries beyond page_counts are not read.  Deterministic.
 * A forked sequence that is cut back to a length inside a page that it
 * shares must not be written to there: fork it again first.
 */
psi_status psi_cache_resize(int32_t N, int32_t max_pages, int32_t num_pages, int32_t page_size,
                            const int32_t *lens, int32_t extra, const psi_page_state *in,
                            const psi_page_state *out, uint32_t *dev_status, psi_stream_t stream);

/* Workspace needed by psi_cache_fork (bytes, a multiple of 256; 0 on invalid
 * sizes).  The workspace needs no initialisation. */
size_t psi_cache_fork_workspace_bytes(int32_t K);

/*
 * psi_cache_fork - continue sequences: row dst[k] becomes a copy of row
 * src[k] with lens[src[k]] positions.
 *
 * Whole pages are shared (refs rises by one); a page that the length ends
 * inside is copied, its filled slots in every layer, to a page popped from
 * the free stack (in the order of k; a fork gets its page or is left out,
 * and so are the later ones that need one; an entry that is not a free page
 * is flagged, and its fork left out).  out lens[dst] = lens[src].
 * A fork is left out and flagged when a row is out of [0, N), when dst holds
 * pages already, when dst is an earlier fork's dst, or any fork's src, or
 * when lens[src] < 0 or src lacks a page below its length.
 * in and out may be the same state (and out_lens the same array as lens);
 * where they differ, all else is carried over.
 * Limits: 1 <= K <= N.
 */
psi_status psi_cache_fork(const psi_cache_layout *layout, void *k_pages, void *v_pages, int32_t N,
                          int32_t max_pages, const int32_t *lens, int32_t *out_lens,
                          const psi_page_state *in, const psi_page_state *out, int32_t K,
                          const int32_t *src, const int32_t *dst, uint32_t *dev_status,
                          void *workspace, size_t workspace_bytes, psi_stream_t stream);

/*
 * psi_rng_uniforms - the uniforms the verify step draws, for inspection and
 * replay: out[s][r] = U(seed, seq_ids ? seq_ids[s] : s, step, r, purpose),
 * a float in [0, 1 - 2^-24] with 24 significant bits.
 * U is the top 24 bits of h = f(f(f(f(f(seed) ^ seq) ^ step) ^ row) ^
 * purpose), f being the SplitMix64 output function (Steele, Lea & Flood,
 * OOPSLA 2014).  out: float [n_seq][n_rows] device memory.
 */
psi_status psi_rng_uniforms(uint64_t seed, const uint64_t *seq_ids,
                            int32_t n_seq, uint64_t step, int32_t n_rows,
                            uint32_t purpose, float *out, psi_stream_t stream);

/*
 * psi_profile_main_kernel - instrumentation for roofline measurements (no
 * counterpart on the pages).  After this call, every verify call made from
 * the same host thread records `before` on its stream immediately before
 * launching its main kernel (the per-row kernel that reads the logits) and
 * `after` immediately after it, so that cudaEventElapsedTime(before, after)
 * is that kernel's duration.  The events are caller-created cudaEvent_t
 * handles, owned by the caller; psi_profile_main_kernel(NULL, NULL) stops
 * recording.  Returns PSI_ERR_INVALID_ARG if exactly one event is NULL.
 */
struct CUevent_st;
typedef struct CUevent_st *psi_event_t; /* same type as cudaEvent_t */
psi_status psi_profile_main_kernel(psi_event_t before, psi_event_t after);

/* Human-readable name of a status code (static string). */
const char *psi_status_string(psi_status status);

/* Detail of the last host-side error on this thread (static buffer). */
const char *psi_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* PSI_VERIFY_H */
