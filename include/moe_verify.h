/*
 * moe_verify.h -- C ABI of libmoeverify.so, the union-expert MoE verify layer
 * and cost-aware draft selection for MI355X (gfx950).
 *
 * Pages cited:
 *   [EcoSpec] review of "Less Experts, Faster Decoding: Cost-Aware Speculative
 *             Decoding for Mixture-of-Experts";
 *   [S2-MoE]  walkthrough of S^2-MoE (self-speculative decoding for MoE on
 *             edge devices);
 *   [W-vs-D]  summary of the width-vs-depth article (batch versus
 *             speculation for MoE on one GPU).
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers unless marked (host).  The caller owns every
 *     buffer; the library allocates nothing, keeps no per-call state and never
 *     synchronises the stream.  Work is enqueued on `stream` (a hipStream_t
 *     passed as void*; NULL = the null stream); outputs are valid once that
 *     work completes.  Calls on different streams may run concurrently if
 *     their output and workspace buffers are disjoint.
 *   - Arrays are dense, row-major, without padding.
 *   - Return codes: 0 = OK, MOE_EINVAL (null pointer, shape or range error),
 *     MOE_ENOTSUP (shape/dtype outside the built kernels), MOE_EWORKSPACE
 *     (workspace too small), MOE_EHIP (a HIP launch failed).  Arguments are
 *     validated on the host before anything is enqueued; on a non-zero return
 *     nothing has been enqueued, except after MOE_EHIP.  moe_last_error()
 *     gives a message for the calling thread's last non-zero return.
 *   - Non-finite inputs give undefined (but memory-safe) results.
 */
#ifndef MOE_VERIFY_H
#define MOE_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_OK 0
#define MOE_EINVAL (-1)
#define MOE_ENOTSUP (-2)
#define MOE_EWORKSPACE (-3)
#define MOE_EHIP (-4)

#define MOE_MAX_TOKENS 64
#define MOE_MAX_EXPERTS 512
#define MOE_MAX_TOPK 32
#define MOE_NUM_STAGES 5   /* router, route, gate-up, down, combine */
#define MOE_MAX_SEGMENTS 64 /* sequences of one call with a preferred set of their own */

/* Expert weight formats.  MOE_FP8_E4M3 is OCP FP8 E4M3FN with one float32
 * scale per 128 x 128 block (row block, column block), row-major over blocks:
 * W[i][j] = e4m3fn(q[i][j]) * scale[i / 128][j / 128]. */
typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_FP8_E4M3 = 2 } moe_dtype;

/* One MoE layer.  Routed experts use SwiGLU:
 *   FFN_e(x) = W_d,e (SiLU(W_g,e x) * (W_u,e x)),  SiLU(z) = z / (1 + e^-z).
 * Logical shapes: the gate-up matrix [2I, H] holds the I gate rows followed by
 * the I up rows; the down matrix is [H, I].
 *   Wr    [E, H]      float32 router, row-major
 *   W_gu  [E, 2I, H]  float32: row-major.  bf16 / fp8: PACKED by
 *                     moe_pack_weights(gate_up = 1), same byte size.
 *   W_d   [E, H, I]   float32: row-major.  bf16 / fp8: PACKED by
 *                     moe_pack_weights(gate_up = 0).
 *   s_gu  [E, 2I/128, H/128] float32, s_d [E, H/128, I/128] float32: fp8 block
 *         scales of the LOGICAL matrices, row-major; NULL otherwise.
 *   Wsh_gu, Wsh_d (+ ssh_gu, ssh_d for fp8): optional always-on shared expert
 *         in the same formats with E = 1, weight 1 for every token, outside the
 *         union; NULL if absent. */
typedef struct {
    int32_t H, I, E, k;
    int32_t wdtype; /* moe_dtype */
    const float *Wr;
    const void *W_gu;
    const void *W_d;
    const float *s_gu, *s_d;
    const void *Wsh_gu, *Wsh_d;
    const float *ssh_gu, *ssh_d;
} moe_layer;

/* Optional reuse-aware soft routing bias ([S2-MoE] component 2, steps 1-3,
 * Fig. 5), applied before the union is formed:
 *   g_e    = sum_b w_conf[b] * softmax(l_b)_e * [e in TopK(l_b)]
 *   P*     = the first `cap` experts by (g desc, index asc) with g_e > 0
 *   lambda_b = alpha * (l_b,(1) - l_b,(k+1))        (float32, no FMA; 0 if k == E)
 *   l'_b,e = l_b,e + lambda_b for e in P*           (float32)
 * The selection is the top-k of l'; gate weights are the softmax of the
 * ORIGINAL logits over that selection.  Requires k <= cap <= E,
 * 0 <= alpha < 1, w_conf [T] float32 (device) non-negative.
 * Sequences ([W-vs-D] section 2, ragged speculation: one call verifies the
 * drafts of several sequences): with nseg = 0 the sums run over all T tokens
 * of the call (one P*); with nseg > 0 the tokens are grouped by sequence,
 * rows seg_off[s] .. seg_off[s+1]-1 forming sequence s, and g and P* are
 * computed over each sequence's own tokens, each token biased toward its own
 * sequence's P* (so no token is pushed toward experts that only other
 * sequences chose).  seg_off (host) [nseg + 1], 0 = seg_off[0] <= ... <=
 * seg_off[nseg] = T (empty sequences allowed), read during the call only;
 * nseg <= MOE_MAX_SEGMENTS.  Errors: EINVAL. */
typedef struct {
    int32_t cap;
    float alpha;
    const float *w_conf;
    int32_t nseg;
    const int32_t *seg_off;
} moe_bias;

/* Optional outputs of moe_verify_layer (device pointers); any field may be
 * NULL, in which case the value lives only in the workspace.
 *   logits [T, E] f32          router logits
 *   topk_idx [T, k] i32        selected experts in rank order (logit desc,
 *                              index asc; biased logits when bias is on)
 *   topk_w [T, k] f32          gate weights
 *   union_size [1] i32         number of unique routed experts U
 *   union_experts [E] i32      first U entries: the union, ascending
 *   csr_ptr [E + 1] i32        first U + 1 entries: offsets into csr_tok
 *   csr_tok [T * k] i32        tokens of each union expert, ascending
 *   csr_w [T * k] f32          gate weight of each (expert, token) entry
 *   pstar [S, cap] i32, pstar_size [S] i32   preferred set of each sequence
 *                              (S = max(1, nseg); row s holds sequence s's P*
 *                              ascending in its first pstar_size[s] entries;
 *                              bias only; without the bias pstar_size[0] = 0)
 *   events: NULL or (host) array of 2 * MOE_NUM_STAGES hipEvent_t handles
 *           created by the caller with timing enabled.  Events 2i and 2i + 1
 *           mark the start and the end of the execution of stage i's kernel
 *           on `stream` (the kernel is launched with hipExtLaunchKernelGGL);
 *           a stage that runs no kernel in this call (the route stage when
 *           the gate-up kernel routes, the combine stage for bf16/fp8)
 *           records both at that point of the stream.  When the gate-up
 *           contraction is split over workgroups (the activation operand
 *           too large for one compute unit's LDS), the gate-up stage spans
 *           the gate-up kernel and the SwiGLU combine that follows it. */
typedef struct {
    float *logits;
    int32_t *topk_idx;
    float *topk_w;
    int32_t *union_size;
    int32_t *union_experts;
    int32_t *csr_ptr;
    int32_t *csr_tok;
    float *csr_w;
    int32_t *pstar;
    int32_t *pstar_size;
    void *const *events;
} moe_aux;

/* Packs row-major expert weights into the matrix-core tile layout that
 * moe_verify_layer streams (bf16 or fp8; one-time weight preparation).
 * src [E, rows, K] row-major (device), dst (device, same byte size, must not
 * overlap src).  gate_up = 1: src is the gate-up matrix, rows = 2I, K = H;
 * gate_up = 0: the down matrix, rows = H, K = I.
 * Layout of dst: per expert, 1 KB tiles of 16 rows x 32 k (bf16) or 16 rows x
 * 64 k (fp8); inside a tile, 16-byte slot l = 0..63 holds tile row l % 16 at
 * k offset (l / 16) * 8 (bf16) or (l / 16) * 16 (fp8), the operand order of
 * v_mfma_f32_16x16x32_bf16, so a wave reads 1 KB of contiguous memory per
 * load.  gate_up = 1: tiles ordered row-tile major, then K-tile; row tile rt
 * holds gate rows 8 rt .. 8 rt + 7 as tile rows 0..7 and up rows
 * I + 8 rt .. I + 8 rt + 7 as tile rows 8..15.  gate_up = 0: tiles ordered in
 * groups of 4 row tiles (64 rows): group major, then K-tile, then the row
 * tile inside the group (rows 16 (4 grp + r) .. + 15).
 * Requires K % 32 (bf16) / K % 64 (fp8) == 0, rows % 32 == 0 for gate_up = 1
 * and rows % 64 == 0 for gate_up = 0. */
int moe_pack_weights(const void *src, void *dst, int32_t E, int32_t rows, int32_t K, int32_t wdtype,
                     int32_t gate_up, void *stream);

/* Streaming-read probe (a measurement aid, not part of the verify path):
 * reads `bytes` of device memory at src with the FFN kernels' load pattern
 * (16-byte non-temporal loads, 1 KB contiguous per wave and load, one
 * workgroup of 8 waves per compute unit) and XORs the 32-bit words into
 * *checksum (device; the caller zeroes it first), so the bytes are used.
 * Its rate is the achievable streaming ceiling against which the FFN
 * kernels' HBM rates are read.  bytes: positive multiple of 16; src 16-byte
 * aligned.  Asynchronous on `stream`. */
int moe_stream_read(const void *src, size_t bytes, uint32_t *checksum, void *stream);

/* Workspace bytes that moe_verify_layer needs for this layer, T and bias
 * (host computation only; bias may be NULL).  Returns 0 for invalid input. */
size_t moe_verify_workspace_bytes(const moe_layer *layer, int32_t T, const moe_bias *bias);

/* The MoE-layer verify step ([EcoSpec] §1-§2: the verify cost at a layer is
 * the union of the experts the verified tokens route to; [S2-MoE] motivation,
 * challenge 2).  For T tokens x [T, H] float32 (device):
 *   logits = x Wr^T; per-token top-k (+ optional bias); gate weights;
 *   union U of the selected experts and the token-by-expert grouping;
 *   y[t] = sum_j w_tj FFN_{e_tj}(x_t) (+ shared expert), y [T, H] float32.
 * Each unique expert's weights are read once and applied to all of its tokens.
 * layer (host), bias (host, NULL = off), aux (host, NULL = no extra outputs).
 * ws: device workspace of at least moe_verify_workspace_bytes() bytes,
 * 256-byte aligned; its contents need no initialisation and are clobbered.
 * y may be x itself (x is read before y is first written); it must not
 * overlap the workspace, the aux outputs or the weights.
 * Limits: 1 <= T <= 64, 1 <= k <= min(E, 32), E <= 512; bf16: H a multiple of
 * 64 and I of 32; fp8: H, I multiples of 128.  Numerics: router GEMV and FFN
 * accumulate in float32; activations enter the bf16/fp8 matrix-core
 * products as a bf16 high/low pair when T <= 8 (as one bf16 otherwise). */
int moe_verify_layer(const moe_layer *layer, const float *x, int32_t T, const moe_bias *bias,
                     float *y, moe_aux *aux, void *ws, size_t ws_bytes, void *stream);

/* moe_verify_layer for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation).  Same arguments, results and errors as moe_verify_layer,
 * without the workspace: the call uses a file-scope device array of
 * MOE_NOALLOC_SCRATCH_BYTES bytes, one per GPU the library runs on, held
 * until the process ends.  It allocates nothing (no hipMalloc, no allocating
 * library routine).  Every call on a GPU shares that GPU's array and leaves
 * it holding that call's workspace; calls that overlap on one GPU (other
 * streams, other threads) race on it and give undefined results, so
 * serialise them.  A call whose workspace (moe_verify_workspace_bytes)
 * exceeds MOE_NOALLOC_SCRATCH_BYTES returns MOE_EWORKSPACE before anything
 * is enqueued.  The first call on each device looks up the array's device
 * address (hipGetSymbolAddress) and keeps it; make that call outside stream
 * capture. */
#define MOE_NOALLOC_SCRATCH_BYTES (32u << 20)
int moe_verify_layer_noalloc(const moe_layer *layer, const float *x, int32_t T, const moe_bias *bias,
                             float *y, moe_aux *aux, void *stream);

/* Per-layer union statistics ([S2-MoE] motivation, challenge 2: reuse ratio
 * = number of distinct experts over s * k).  topk_idx [nL, T, k] int32
 * (device), entries in [0, E) (entries outside are ignored);
 * counts [nL] int32 = |union of layer l|, reuse [nL] float32 =
 * counts / (T * k), correctly rounded.  Limits: 1 <= E <= 65536. */
int union_stats(const int32_t *topk_idx, int32_t nL, int32_t T, int32_t k, int32_t E,
                int32_t *counts, float *reuse, void *stream);

/* EcoSpec cost-aware greedy draft selection ([EcoSpec] §3.2 global expert
 * buffer, §3.3 score equation and greedy selection), for nt trees with the
 * same shape.
 *   parent (host) [N]: BFS order, parent[i] in [-1, i) (-1 = child of the
 *                  root); validated, so ties go to ancestors.
 *   P [nt, N] float32: path probabilities.
 *   Epred [nt, N, W] uint32: path footprints, bit b = layer * E + expert in
 *                  word b / 32, LSB first.
 * For each tree, starting from an empty buffer B, gamma times: score every
 * unchosen node t as P_t / (popcount(F_t & ~B) + eps) in float32 (add, then
 * divide, each correctly rounded), choose the highest score (ties: lowest
 * node index), B |= F_chosen.  S [nt, gamma] int32 receives node ids in
 * choice order.  P, Epred and S may be NULL when gamma == 0 or nt == 0.
 * Limits: 0 <= gamma <= N <= 4096, 1 <= W <= 4096, eps > 0.  Batches of
 * 512 or more trees with N <= 16 and W <= 512 run one wave per tree with the
 * tree in registers; otherwise one workgroup per tree, and a tree whose
 * footprints fit in 64 KB of LDS (N * W + W + N + N / 32 <= 16384 words) is
 * staged there once, a larger one read from global memory every round.
 * Every path gives the same selections. */
int select_drafts(const int32_t *parent, int32_t N, const float *P, const uint32_t *Epred,
                  int32_t W, int32_t gamma, float eps, int32_t nt, int32_t *S, void *stream);

/* Per-sequence unique experts of a ragged verify call ([W-vs-D] section 2,
 * ragged speculation: sequences verify different numbers of tokens in one
 * call).  The T tokens of the call are grouped by sequence: rows
 * offsets[s] .. offsets[s+1]-1 belong to sequence s.
 *   topk_idx [nL, T, k] int32 (device), entries outside [0, E) ignored
 *   offsets  (host) [S + 1] int32, 0 = offsets[0] <= ... <= offsets[S] = T
 *   per      [nL, S] int32 out: distinct experts of each sequence's tokens
 *   total    [nL] int32 out: distinct experts of the whole call
 * Limits: 1 <= S <= 64.  Errors: EINVAL (NULL, shapes, offsets). */
int union_stats_segments(const int32_t *topk_idx, int32_t nL, int32_t T, int32_t k, int32_t E,
                         const int32_t *offsets, int32_t S, int32_t *per, int32_t *total, void *stream);

/* Confidence-gated per-sequence depths ([W-vs-D] section 2): one batch-wide
 * depth, then greedy per-sequence truncation, maximising the expected
 * throughput
 *     sum_s (1 + c[s,1] + ... + c[s,d_s]) / (t_base + t_exp * U(d)),
 * where U(d) is the number of distinct (layer, expert) pairs over every
 * verified token (the root j = 0 and drafts 1..d_s of each sequence).  The
 * batch-wide depth is the smallest D in 0..Dmax with the largest throughput;
 * then, for s = 0..S-1 in order, d_s is lowered one step at a time while that
 * raises the throughput strictly.  Float32 as fl(total / fl(t_base +
 * fl(t_exp * U))) with A_s summed over j ascending and the total over s
 * ascending.
 *   c     [S, Dmax + 1] float32 cumulative draft confidences (column 0 unused)
 *   Epred [S, Dmax + 1, W] uint32 expert bitsets of each token
 *   d     [S] int32 out: the depths
 * Limits: S <= 64, Dmax <= 64, W <= 1024.  Errors: EINVAL. */
int gate_depths(const float *c, const uint32_t *Epred, int32_t S, int32_t Dmax, int32_t W, float t_base,
                float t_exp, int32_t *d, void *stream);

/* Static-cost ablation of the selection ([EcoSpec] section 4.3): the same
 * greedy loop and arguments as select_drafts, but every node pays the size
 * of its whole footprint, popcount(F_t), and B is never updated, so the
 * result is the top-gamma of P_t / (popcount(F_t) + eps) in float32 with
 * ties to the lower node index. */
int select_drafts_static(const int32_t *parent, int32_t N, const float *P, const uint32_t *Epred, int32_t W,
                         int32_t gamma, float eps, int32_t nt, int32_t *S, void *stream);

/* Utility-driven adaptive expansion of draft trees ([S2-MoE] component 1,
 * routing-aware adaptive speculative expansion).  Per tree, a draft token i
 * joins the expansion set S while its utility
 *     U_i = p_i * T_AR / (|E_i \ union_{j in S} E_j| * T_exp + C_i^draft)
 * is at least 1: candidates are examined in generation (BFS) order, a node
 * only once its parent is in S (or it is a child of the root), and passes
 * repeat until one adds no node.  The test is evaluated in float32 as
 * fl(p * t_ar) >= fl(fl(c * t_exp) + c_draft) with the exact count c of new
 * (layer, expert) pairs; the resulting set does not depend on the order.
 *   parent  (host) [N] int32, BFS order, -1 = child of the root, parent < child
 *   P       [nt, N] float32 acceptance probabilities (e.g. path probabilities)
 *   Epred   [nt, N, W] uint32 footprint bitsets, as for select_drafts (own or
 *           whole-path footprints give the same result, since S is
 *           prefix-closed)
 *   t_ar    saving of one accepted token (one autoregressive step), >= 0
 *   t_exp   latency of one new (layer, expert) pair, >= 0
 *   c_draft [nt, N] float32 draft-side cost of each node, or NULL (zero)
 *   S       [nt, N] int32 out: nodes in the order they join, then -1
 *   count   [nt] int32 out: size of each set
 * Limits: N <= 1024, W <= 4096.  Footprints are staged in LDS when
 * N * W + W + 3 N + N / 32 <= 16384 words, else read from global memory.
 * Errors: EINVAL (NULL, shapes, parent order, t_ar / t_exp). */
int expand_drafts(const int32_t *parent, int32_t N, const float *P, const uint32_t *Epred, int32_t W,
                  float t_ar, float t_exp, const float *c_draft, int32_t nt, int32_t *S, int32_t *count,
                  void *stream);

/* ------------------------------------------------------------------------
 * 4-bit K/V cache of the verified tokens ([EcoSpec] tree-attention verify
 * mask; [S2-MoE] component 3: draft writes are tentative, the accepted
 * tokens' K/V is committed).
 *
 * The cache is a pool of pages of `page` rows (tokens), shared by sequences
 * through a page table.  K and V are held in OCP MX style: blocks of 32
 * consecutive elements along the head dimension share a scale 2^(e - 127)
 * (one byte e), each element is an e2m1 code (0, .5, 1, 1.5, 2, 3, 4, 6 and
 * a sign in bit 3).  The scale of a block is the smallest power of two
 * 2^-100 .. 2^125 with max|x| <= 6 * 2^n, elements are rounded to nearest, ties to
 * the even code, and saturate at 6.  NaN is stored as 0, an infinity as the
 * largest value (6 * 2^125, with the block's scale): the cache holds finite
 * numbers only.
 *   data [num_pages][Hkv][page / 16] tiles of 17 D bytes (device, 16-byte
 *   aligned, kv4_cache_bytes bytes; needs no initialisation).  A tile holds
 *   16 rows i = 0..15 in matrix-core operand order:
 *     8 D bytes  K codes: element d of row i in byte i * D/2 + d/2, even d in
 *                the low half
 *     D/2        K scales: block b of row i in byte 16 b + i
 *     8 D        V codes: element d of row i, w = D / 32, in byte
 *                (64 (i/4) + 4 (d/(2w)) + i%4) w + (d%(2w))/2, even d low
 *     D/2        V scales: block b of row i in byte 16 b + i
 *   D is 64, 128 or 256; page a power of two, 16 .. 4096. */
typedef struct {
    void *data;
    int32_t num_pages, page, Hkv, D;
} moe_kv4_cache;

/* The rows of one call, grouped by sequence as in moe_bias: call row t =
 * seg_off[s] + j is row j of sequence s and has the cache position len[s] + j.
 *   table [nseq, max_pages] i32 (device): page of positions page * i ..
 *         page * (i + 1) - 1 of sequence s in table[s][i].  Entries outside
 *         [0, num_pages) hold no rows: nothing is written to them and
 *         nothing is seen in them, nor past the table's end.
 *   len   [nseq] i32 (device): rows of each sequence before this call's
 *         (negative counts as 0)
 *   seg_off (host) [nseq + 1], 0 = seg_off[0] <= ... <= seg_off[nseq] = T,
 *         read during the call only; 1 <= nseq <= MOE_MAX_SEGMENTS. */
typedef struct {
    const int32_t *table;
    int32_t max_pages;
    const int32_t *len;
    int32_t nseq;
    const int32_t *seg_off;
} moe_kv4_rows;

/* Bytes of a cache's data; 0 for invalid sizes. */
size_t kv4_cache_bytes(int32_t num_pages, int32_t page, int32_t Hkv, int32_t D);

/* Quantises K and V rows into the cache.
 *   k, v [T, Hkv, D] in dtype MOE_F32 or MOE_BF16; consecutive tokens are
 *         k_stride / v_stride elements apart (>= Hkv * D; slices of a fused
 *         projection), 16-byte aligned rows
 *   path [T], count [nseq] i32 (device), or both NULL.  NULL: row j of
 *         sequence s is written to position len[s] + j (a prompt, or the
 *         tentative rows of a draft tree).  Else the commit of an accepted
 *         path, as accept_drafts returns it: for i < count[s], row
 *         path[seg_off[s] + i] of the sequence is written to position
 *         len[s] + i (entries outside the sequence's rows are skipped).
 *   k_out, v_out [T, Hkv, D] in dtype (dense), or both NULL: the values that
 *         the codes stand for, for every row of the call; only without path.
 * Positions written twice in one call (a page listed twice) hold any mix of the
 * two rows' codes and scales: finite numbers, but neither row for certain.
 * Limits: 1 <= T <= 2^20.  Errors: EINVAL, ENOTSUP (D, dtype). */
int kv4_append(const moe_kv4_cache *cache, const moe_kv4_rows *rows, const void *k, const void *v,
               int64_t k_stride, int64_t v_stride, int32_t T, int32_t dtype, const int32_t *path,
               const int32_t *count, void *k_out, void *v_out, void *stream);

/* Workspace bytes of kv4_attend (host computation); 0 for invalid input. */
size_t kv4_attend_workspace_bytes(const moe_kv4_cache *cache, const moe_kv4_rows *rows, int32_t T, int32_t Hq,
                                  int32_t dtype);

/* Attention of the verified tokens over the cache, their own rows included
 * (append them first):
 *   out[t, h] = sum_p softmax_p(scale * q[t, h] . K[p, h / (Hq / Hkv)]) V[p, ...]
 * over the positions p that t sees: all of its sequence's rows before this
 * call, itself, and its ancestors among the call's rows.  A token that sees
 * nothing (every page outside the pool) gets zeros.  A head's query that holds
 * NaN gives NaN, and touches no other head's or token's result.
 *   q [T, Hq, D] in dtype MOE_F32 or MOE_BF16, tokens q_stride elements apart
 *         (16-byte aligned rows); out [T, Hq, D] in dtype, dense
 *   parent (host) [T], read during the call only: parent of each row inside
 *         its sequence (row j has a parent in [0, j); the first row -1), or
 *         NULL for chains (each row sees all rows before it)
 *   ws    16-byte aligned, kv4_attend_workspace_bytes bytes, no initialisation
 * Sums and softmax statistics are float32.  bf16: probabilities enter the
 * second product rounded to bf16.  float32: q and the probabilities enter
 * the products as three bf16 terms (24 bits).
 * Limits: 1 <= T <= MOE_MAX_TOKENS, Hq a multiple of Hkv. */
int kv4_attend(const moe_kv4_cache *cache, const moe_kv4_rows *rows, const void *q, int64_t q_stride, int32_t T,
               int32_t Hq, int32_t dtype, float scale, const int32_t *parent, void *out, void *ws,
               size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Rows and pages of the 4-bit cache: what prompts need of it.
 *
 * Reads rows back as dense K and V, the values that the codes stand for: call
 * row t = seg_off[s] + j is position len[s] + j of sequence s (the beginning
 * of a prompt that stands already: len 0), rows without a page are zeros.
 *   k, v [T, Hkv, D] out in dtype MOE_F32 or MOE_BF16 (exact in both), dense
 * Limits: 0 <= T <= 2^22, T * Hkv <= 2^28.  Errors: EINVAL, ENOTSUP. */
int kv4_read(const moe_kv4_cache *cache, const moe_kv4_rows *rows, void *k, void *v, int32_t T, int32_t dtype,
             void *stream);

/* The pages of a pool and who holds them.  A table entry inside [0,
 * num_pages) holds its page; refs counts the entries that hold each page, and
 * a page is free while its count is 0 or below.  Sequences may share the pages
 * of a common beginning; rows are to be written only into pages whose count is
 * 1 (kv4_append does not look).  The calls below keep counts and table in step; all
 * layers' caches share one pool and differ in their data only, so that the
 * data is moved by kv4_copy_pages, once for each layer.
 *   refs  [num_pages] i32 (device), 0 for a new pool
 *   table [nseq, max_pages] i32 (device), -1 for a new pool; the table of
 *         moe_kv4_rows for sequences 0 .. nseq - 1, or a table of which the
 *         caller gathers rows into one
 *   page  rows of a page, a power of two, 16 .. 4096
 * Limits: 1 <= num_pages <= 2^24, 1 <= nseq <= 2^16, nseq * max_pages <= 2^30,
 * max_pages * page below 2^31 - 2^22.
 * Lists name sequences by their row of the table (device, n <=
 * MOE_MAX_SEGMENTS entries); one that is outside [0, nseq) names none. */
typedef struct {
    int32_t *refs, *table;
    int32_t num_pages, page, nseq, max_pages;
} moe_kv4_pool;

/* Takes pages for the first rows[i] rows of sequence seq[i]: the entries from
 * its first one without a page on get the lowest free pages.  Entries of the
 * list are served in order, each whole or not at all.
 *   ok [n] i32 out: 1 if the sequence holds pages for its rows now; 0 if too
 *      few pages are free, or the table's row is too short, or has a page behind
 *      a gap among the entries that the rows need (these calls leave no gaps), or
 *      seq[i] names no sequence or one that an earlier entry names */
int kv4_reserve(const moe_kv4_pool *pool, const int32_t *seq, const int32_t *rows, int32_t n, int32_t *ok, void *stream);

/* Makes sequence dst[i] hold the first rows[i] rows of sequence src[i]: whole
 * pages are shared, a page that is filled in part gets the lowest free page, into
 * which its data has to be copied before either sequence writes.  What dst[i]
 * held before is let go first.
 *   pairs [n, 2] i32 out: (page, fresh page) for kv4_copy_pages; (-1, -1) where
 *         nothing is to be copied
 *   ok    [n] i32 out: 1 done.  0 if no page was free (dst[i] then holds
 *         nothing), or nothing was done and dst[i] keeps what it held: a name outside
 *         [0, nseq), rows[i] above a table's row, a source that has no page for
 *         some of the rows, a dst[i] that an earlier entry names too, or that
 *         any entry names as its source. */
int kv4_fork(const moe_kv4_pool *pool, const int32_t *src, const int32_t *dst, const int32_t *rows, int32_t n,
             int32_t *pairs, int32_t *ok, void *stream);

/* Lets go the pages of sequence seq[i] behind its first keep[i] rows (0: all
 * of them); their entries become -1.  A sequence named twice keeps the fewer.
 * A page that is kept in part stays as it is, also where other sequences hold it
 * (a fork, or its parent, cut back below the rows at which they parted): rows
 * appended behind keep[i] would then overwrite theirs.  Nothing in these calls
 * sees that.  Such a sequence is continued in a slot of its own: kv4_fork with it as
 * src, a free slot as dst and keep[i] rows, kv4_copy_pages of the pair in every
 * layer's cache, and kv4_release of the old slot. */
int kv4_release(const moe_kv4_pool *pool, const int32_t *seq, const int32_t *keep, int32_t n, void *stream);

/* Moves used pages to the pool's front: the i-th lowest free page takes the
 * i-th highest used one while it lies below it, at most max_moves of them.
 * Counts and table follow; the data has to be copied before the caches are
 * used again.  With as many moves as it takes, the used pages are 0 .. U - 1.
 *   pairs [max_moves, 2] i32 out: (from, to) for kv4_copy_pages, then (-1, -1);
 *         no page is among both
 *   ws    4-byte aligned, kv4_compact_workspace_bytes bytes, no initialisation
 * Limits: 1 <= max_moves <= 2^24. */
size_t kv4_compact_workspace_bytes(const moe_kv4_pool *pool, int32_t max_moves);
int kv4_compact(const moe_kv4_pool *pool, int32_t max_moves, int32_t *pairs, void *ws, size_t ws_bytes, void *stream);

/* Copies page pairs[i][0] of a cache to page pairs[i][1], for i < n; pairs with
 * an entry outside [0, num_pages), or of one page twice, copy nothing.  A page that is
 * written by two pairs, or read by one and written by another, holds any mix
 * of them.
 *   pairs [n, 2] i32 (device).  Limits: 0 <= n <= 2^24. */
int kv4_copy_pages(const moe_kv4_cache *cache, const int32_t *pairs, int32_t n, void *stream);

/* ------------------------------------------------------------------------
 * Prompts: any number of tokens a call, where moe_verify_layer takes 64.
 */

/* Attention of prompts: causal, over dense K and V of sequences packed one
 * behind the other.
 *   out[t, h] = sum_p softmax_p(scale * q[t, h] . k[p, h / (Hq / Hkv)]) v[p, ...]
 * Row j of a sequence with n query rows and m keys sees its first
 * j + 1 + (m - n) keys: with m = n a whole prompt, with m > n its next piece,
 * behind m - n rows that stand already (kv4_read has them); with m < n the first
 * n - m rows see nothing and get zeros.
 *   q [T, Hq, D], k, v [Tk, Hkv, D] in dtype MOE_F32 or MOE_BF16, tokens
 *         q_stride / k_stride / v_stride elements apart (slices of a fused
 *         projection), 16-byte aligned rows; out [T, Hq, D] in dtype, dense
 *   q_off, k_off (host) [nseq + 1], 0 = off[0] <= ... <= off[nseq] = T (Tk),
 *         read during the call only; 1 <= nseq <= MOE_MAX_SEGMENTS
 *   ws    256-byte aligned, prompt_attend_workspace_bytes bytes, no
 *         initialisation; may be NULL where that is 0
 * Sums and softmax statistics are float32.  bf16: probabilities enter the
 * second product rounded to bf16.  float32: all operands enter the products as
 * three bf16 terms (24 bits).  Rows of one sequence do not touch another's
 * results; a k or v that is no finite number may make any result of its
 * sequence and head NaN.  A row of a head whose query holds NaN or an infinity, or whose
 * visible scores hold NaN, +inf or nothing but -inf in float32, is NaN, and
 * touches no other row; rows that see nothing are zeros all the same.  Above
 * 2^29 in magnitude a row's scores may make it NaN.
 * Limits: 0 <= T, Tk <= 2^22, D 64, 128 or 256, Hq a multiple of Hkv, at most
 * 8192, strides of k and v up to 2^24 elements, below 2^23 blocks of 128 rows of
 * a head, float32 K below 2^33 elements.  Errors: EINVAL, ENOTSUP, EWORKSPACE. */
size_t prompt_attend_workspace_bytes(int32_t nseq, const int32_t *q_off, const int32_t *k_off, int32_t Hq, int32_t Hkv,
                                     int32_t D, int32_t dtype);
int prompt_attend(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                  int32_t nseq, const int32_t *q_off, const int32_t *k_off, int32_t Hq, int32_t Hkv, int32_t D,
                  int32_t dtype, float scale, void *out, void *ws, size_t ws_bytes, void *stream);

/* The experts of each token from its router logits [T, E] float32, rows
 * `stride` elements apart: the first k by (logit desc, index asc), NaN counts
 * as -inf and +inf as the largest float; gate weights are the softmax over
 * them (0 where even the first is -inf).
 *   topk_idx [T, k] i32, topk_w [T, k] f32 out, as moe_aux has them
 * Limits: 0 <= T <= 2^24, 1 <= E <= MOE_MAX_EXPERTS, 1 <= k <= min(E,
 * MOE_MAX_TOPK). */
int route_tokens(const float *logits, int64_t stride, int32_t T, int32_t E, int32_t k, int32_t *topk_idx,
                 float *topk_w, void *stream);

/* The experts' products over T tokens, from choices that are made already
 * (route_tokens', or any other):
 *   y[t] = sum_j topk_w[t][j] FFN_{topk_idx[t][j]}(x_t) (+ shared expert)
 * with the layer of moe_verify_layer (bf16 or fp8 weights, packed; Wr is not
 * read, but no layer is without it).  Tokens are grouped by expert, whose weights are read once for a tile of
 * up to 256 of them.
 *   x     [T, H] in dtype MOE_F32 or MOE_BF16, tokens x_stride elements apart,
 *         16-byte aligned rows
 *   topk_idx, topk_w [T, k] i32 / f32 (device); an entry outside [0, E) names
 *         no expert and counts for nothing; an expert named twice counts twice
 *   y     [T, H] out in dtype, dense; may be x itself
 *   ws    256-byte aligned, moe_experts_workspace_bytes bytes, no initialisation
 * Sums and each expert's outputs are float32.  bf16: hidden activations enter
 * the second product rounded to bf16.  float32: activations and hidden
 * activations enter the products as three bf16 terms (24 bits).  An fp8 block scale of 0 or below 2^-126 counts as
 * 2^-127.  Results do not depend on the order in which a call's workgroups run.
 * Limits: 0 <= T <= 2^20, 1 <= k <= min(E, MOE_MAX_TOPK), E <= MOE_MAX_EXPERTS; bf16: H a multiple of 64 and I of
 * 32; fp8: H, I multiples of 128; T * H below 2^33.  Errors: EINVAL, ENOTSUP
 * (float32 weights, a call too large for one grid), EWORKSPACE. */
size_t moe_experts_workspace_bytes(const moe_layer *layer, int32_t T, int32_t dtype);
int moe_experts(const moe_layer *layer, const void *x, int64_t x_stride, int32_t T, int32_t dtype,
                const int32_t *topk_idx, const float *topk_w, void *y, void *ws, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Drawing and accepting draft tokens.  Both use the filtered distribution of
 * a row of logits l [V], defined in 64 bits:
 *   the tokens with l > -inf (NaN counts as -inf, +inf as the largest float)
 *   are ranked by (l desc, index asc); w_i = exp((l_i - l_first) / temperature);
 *   the first n are kept, n the smallest (at least 1) of
 *     top_k (off when <= 0),
 *     the least number whose weights sum to >= top_p * (sum of the first
 *       top_k) (off when >= 1),
 *     the number with w_i >= min_p (off when <= 0);
 *   temperature <= 0 keeps the first only.  A temperature of NaN is 0, another
 *   filter of NaN is off.
 * p_i = w_i / (sum of the kept).  A draw with a number u in [0, 1) takes the
 * lowest kept index whose running sum in index order exceeds u * sum; a row
 * without tokens gives -1.
 * Weights are summed as integers in units of 2^-45 of the first's weight (a
 * token below 2^-46 of it is never drawn), so results do not depend on the
 * order of summation.  Rows of V > 32768 take two sums from parts joined in
 * float64 in a fixed order, off by at most V 2^-46 of the sum: the row's
 * without filters, and the one that top_p is a share of where no top_k is
 * given. */
typedef struct {
    const float *temperature; /* [T] device, or NULL: 1 */
    const int32_t *top_k;     /* [T] device, or NULL: off */
    const float *top_p;       /* [T] device, or NULL: off */
    const float *min_p;       /* [T] device, or NULL: off */
} moe_sampling;

/* Workspace bytes of sample_tokens and accept_drafts for T rows of V logits;
 * 0 for invalid input. */
size_t sample_workspace_bytes(int32_t T, int32_t V);

/* One draw per row: a draft step, or a step without drafts.
 *   logits [T, V] in dtype MOE_F32 or MOE_BF16, rows `stride` elements apart
 *   f      (host) filters, or NULL: none, temperature 1
 *   u      [T] f32 in [0, 1) (device)
 *   token  [T] i32 out;  prob [T] f32 out or NULL: the token's probability
 *          (0 with token -1; the draft confidence that select_drafts,
 *          expand_drafts and gate_depths take)
 *   probs  [T, V] f32 out (dense) or NULL: the whole distribution (the
 *          draft_probs of accept_drafts)
 *   ws     256-byte aligned, sample_workspace_bytes bytes, no initialisation
 * Limits: 0 <= T <= 65535, 1 <= V <= 2^18. */
int sample_tokens(const void *logits, int64_t stride, int32_t T, int32_t V, int32_t dtype, const moe_sampling *f,
                  const float *u, int32_t *token, float *prob, float *probs, void *ws, size_t ws_bytes,
                  void *stream);

/* Acceptance of drafts from the target's logits.  The rows of a call are
 * grouped by sequence (seg_off as in moe_kv4_rows); row 0 of a sequence is
 * its root (the last token that stands already), the others are drafts.
 * logits[t] are the target's for the token after row t.
 *   tokens [T] i32 (device): token of each row (roots' are not read)
 *   parent (host) [T] as in kv4_attend, or NULL: chains
 *   draft_probs NULL: the target draws after each row with u[t]; from the
 *          root on, a child holding the drawn token (of equal ones the
 *          first) is accepted, until none does, and that draw is the last
 *          token.
 *   draft_probs [T, V] f32 (device, dense), chains only: row t is the
 *          distribution that the draft after row t was drawn from (not read
 *          for a sequence's last row).  The draft x is accepted if
 *          u[t] * q(x) < p(x); at the first that is not, the last token is
 *          drawn with u_final[s] from max(p - q, 0) (from p if that is zero
 *          everywhere), after the last draft from p.
 *          Values of q below 0 count as 0; a draft whose q is NaN is not
 *          accepted, elsewhere NaN counts as 0.
 *   u      [T] f32, u_final [nseq] f32 in [0, 1) (device; u_final only with
 *          draft_probs, else NULL)
 *   count  [nseq] i32 out: tokens that the sequence gains, accepted drafts
 *          + 1 (0 for a sequence without rows)
 *   out    [T] i32 out: the gained tokens of sequence s from seg_off[s] on,
 *          then -1
 *   path   [T] i32 out: the rows (inside the sequence) whose K/V are to be
 *          kept, the root first: count[s] entries from seg_off[s] on, then -1
 * Limits: 1 <= T <= MOE_MAX_TOKENS, 1 <= V <= 2^18. */
int accept_drafts(const void *logits, int64_t stride, int32_t T, int32_t V, int32_t dtype, const moe_sampling *f,
                  const int32_t *tokens, int32_t nseq, const int32_t *seg_off, const int32_t *parent,
                  const float *draft_probs, const float *u, const float *u_final, int32_t *out, int32_t *path,
                  int32_t *count, void *ws, size_t ws_bytes, void *stream);

/* Message for the calling thread's last non-zero return ("" if none). */
const char *moe_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_VERIFY_H */
