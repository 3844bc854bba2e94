/*
 * kvfix.h -- C ABI of libkvfix, the repair path for reused KV-cache chunks on one
 * NVIDIA GB300 (sm_103a).
 *
 * The library re-aligns, scores, selects, corrects and stores KV caches that one
 * agent reuses from another context.  Every call enqueues hand-written CUDA kernels
 * on the caller's stream; nothing runs on the host but argument checks.
 *
 * Conventions shared by every call
 * --------------------------------
 * - bf16 tensors are passed as `kvfix_bf16*`: raw IEEE bfloat16 bit patterns.
 * - All tensor pointers are DEVICE pointers unless the name starts with `h_`.
 * - A KV plane (the keys or the values of a cache) is described by kvfix_kv_desc:
 *   element (c, l, t, h, e) -- chunk, layer, token, KV head, head dim -- lives at
 *       c*stride_chunk + l*stride_layer + t*stride_token + h*head_dim + e
 *   (strides in elements).  The heads of one token are contiguous (one token row is
 *   kv_heads*head_dim elements).  head_dim must be a multiple of 16 in [16, 256]; the
 *   base pointer must be 16-byte aligned and every stride a non-negative multiple of
 *   8 elements, so that rows move as 16-byte vectors.
 * - `stream` is a cudaStream_t cast to void* (NULL = the legacy default stream).
 * - Ownership: the caller owns every buffer.  The library keeps no per-call state
 *   and allocates no device memory; calls that need scratch take a workspace
 *   buffer whose size a companion *_workspace_bytes() query returns.
 * - Errors: arguments are checked on the host before anything is launched; a bad
 *   argument returns KVFIX_EINVAL and launches nothing.  A launch failure returns
 *   KVFIX_ECUDA.  kvfix_last_error() gives the message of the last non-OK status of
 *   the calling thread.  Conditions only the GPU can see (an index in caller data
 *   out of range, a payload overflow) set a device status word instead; the kernels
 *   then skip the offending access.  kvfix_check_status() reads and clears it.
 * - Calls are asynchronous: a KVFIX_OK return means "enqueued".
 * - Outputs never alias inputs, except where a call says so.
 *
 * Citations name the page and section that define each operation:
 *   [KVCMAS]  KVCMAS: Efficient KV cache Correction for Shared Context in Multi-Agent Systems
 *   [AKS]     AgentKVShift: Correcting Reused KV (review)
 *   [TD]      TokenDance: Scaling Multi-Agent LLM Serving via Collective KV Cache Sharing (summary)
 *   [BCR]     Budgeted Cache Repair for Cross-Context KV-Cache Reuse
 */
#ifndef KVFIX_H
#define KVFIX_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define KVFIX_API __attribute__((visibility("default")))
#else
#define KVFIX_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t kvfix_bf16;

typedef enum {
    KVFIX_OK = 0,
    KVFIX_EINVAL = 1,   /* bad argument; nothing was launched */
    KVFIX_ENOSPACE = 2, /* diff payload capacity too small (see kvfix_diff_encode), or no free page */
    KVFIX_ECUDA = 3,    /* a CUDA runtime call or launch failed */
    KVFIX_ETIMEOUT = 4, /* a bounded device-side wait gave up */
    KVFIX_EDEVICE = 5   /* the device flagged bad caller data (index out of range) */
} kvfix_status;

typedef struct {
    int32_t chunks;
    int32_t layers;
    int32_t tokens;
    int32_t kv_heads;
    int32_t head_dim;
    int64_t stride_chunk;
    int64_t stride_layer;
    int64_t stride_token;
} kvfix_kv_desc;

/* Library version, major*10000 + minor*100 + patch. */
KVFIX_API int kvfix_version(void);

/* Message of the calling thread's last non-OK status ("" if none).  The pointer
 * stays valid until the thread's next kvfix call. */
KVFIX_API const char* kvfix_last_error(void);

/* Synchronise `stream`, then read and clear the device status word.
 * Returns KVFIX_OK, KVFIX_EDEVICE (an index out of range was skipped),
 * KVFIX_ENOSPACE (a payload write was skipped, or lists wanted more pages than the pool has
 * free), KVFIX_ETIMEOUT or KVFIX_ECUDA. */
KVFIX_API kvfix_status kvfix_check_status(void* stream);

/*
 * kvfix_rerope -- re-align cached keys to new positions with rotary embeddings.
 * [KVCMAS] section 2.2 and App. A.3 (keys are re-aligned to their target positions,
 * values are not rotated); [TD] section 4.4, Algorithm 1 (RoPERecover(P_old, P_new));
 * [BCR] App. A (one scalar position shift per reused segment).
 *
 * With rotate-half RoPE, theta_i = rope_base^(-2i/D) for i < D/2 and dimension i
 * paired with i + D/2, a key encoded at position p and moved to p + delta is rotated
 * once more by the angle delta*theta_i:
 *     y_i       = x_i cos(delta theta_i) - x_{i+D/2} sin(delta theta_i)
 *     y_{i+D/2} = x_{i+D/2} cos(delta theta_i) + x_i sin(delta theta_i)
 * k_in, k_out : one KV plane each, described by in_desc / out_desc (same shape; k_out
 *               may be k_in itself with the same descriptor, for an in-place update).
 * delta       : device int32[in_desc.chunks], the shift of each chunk (any sign).
 * Arithmetic: angles reduced in double, cos/sin and the rotation in float, output
 * rounded to nearest-even bf16.  delta = 0 reproduces the input bit for bit.
 */
KVFIX_API kvfix_status kvfix_rerope(const kvfix_bf16* k_in, kvfix_kv_desc in_desc, kvfix_bf16* k_out,
                                    kvfix_kv_desc out_desc, const int32_t* delta, double rope_base,
                                    void* stream);

/*
 * kvfix_score_topk -- check-layer divergence and probe selection.
 * [AKS] "Core idea and method", steps 1-2 and the displayed b, d and w equations;
 * [TD] section 4.2 (one batched rotation and one batched check-layer comparison for
 * all requests of a round).
 *
 * Units: unit u = a*R + r pairs agent a (of `agents`) with reused chunk r (of
 * R = reuse.chunks).  For every unit and token j of the check layer:
 *     d_k[u][j] = || k_fresh[u][j] - rerope(k_reuse[r][j], delta[u]) ||_2
 *     d_v[u][j] = || v_fresh[u][j] - v_reuse[r][j] ||_2
 * where the norm runs over the whole token row (all KV heads).  Then, for each plane,
 * the b tokens with the largest d (ties to the lower index; d compared as float) are
 * the probes: idx_*[u][0..b-1] in ascending order, bit j of mask_*[u] set for each
 * (word j/32, bit j%32), w_*[u][j] = min(d[u][j], 1).  mask_union = mask_k | mask_v.
 *
 * k_reuse, v_reuse : check-layer views, `reuse` (layers == 1), R chunks.
 * k_fresh, v_fresh : check-layer views, `fresh` (layers == 1, chunks == agents*R,
 *                    same tokens/heads/head_dim as `reuse`).
 * delta            : device int32[agents*R].
 * b                : 0 <= b <= tokens (b = ceil(r n) for probe ratio r).
 * d_k, d_v, w_k, w_v : device float[agents*R][tokens], required.
 * idx_k, idx_v     : device int32[agents*R][b], required when b > 0.
 * mask_k, mask_v, mask_union : device uint32[agents*R][ceil(tokens/32)], optional.
 * Limits: tokens <= 65536.  All agents of a round are handled by one set of launches;
 * each reused check-layer row is read once for all agents.
 */
KVFIX_API kvfix_status kvfix_score_topk(const kvfix_bf16* k_reuse, const kvfix_bf16* v_reuse,
                              kvfix_kv_desc reuse, const kvfix_bf16* k_fresh,
                              const kvfix_bf16* v_fresh, kvfix_kv_desc fresh, int32_t agents,
                              const int32_t* delta, double rope_base, int32_t b, float* d_k,
                              float* d_v, float* w_k, float* w_v, int32_t* idx_k, int32_t* idx_v,
                              uint32_t* mask_k, uint32_t* mask_v, uint32_t* mask_union,
                              void* stream);

/*
 * kvfix_mean_correct -- probe-mean residual correction of every layer.
 * [AKS] "Core idea and method", steps 3-4 and the displayed mu-hat and K_corr
 * equations; [TD] section 4.2 (only the per-request refresh differs between the
 * requests of a group).
 *
 * For unit u = a*R + r, layer l, plane P in {K, V} with probe list S = idx_P[u][0..b-1]
 * and weights w_P[u]:
 *     mu_P[u][l][h*D+e] = (1/b) sum_{i<b} (fresh_P[u][l][S_i][h][e] - rot(reuse_P[r][l][S_i][h])[e])
 *     out_P[u][l][j]    = fresh_P[u][l][j]                              if j in S (bit copy)
 *                       = bf16(rot(reuse_P[r][l][j]) + w_P[u][j] * mu_P[u][l])   otherwise
 * rot is the re-rope by delta[u] for keys and the identity for values; b == 0 gives
 * mu = 0 and out = bf16(rot(reuse)).  The sum runs in a fixed order (probe i goes to
 * partial sum i mod 32; partial sums are added in order), so a round of N agents in
 * one call and N one-agent calls give the same bits.
 *
 * reuse, fresh, out : plane descriptors; reuse has R chunks, fresh and out agents*R,
 *                     all with the same layers/tokens/heads/head_dim.
 * k_* / v_*         : pass all NULL for a plane to skip it.
 * idx_k, idx_v      : device int32[agents*R][b] (ascending not required; each entry
 *                     must lie in [0, tokens) -- others are skipped and flagged).
 * w_k, w_v          : device float[agents*R][tokens].
 * mu_k, mu_v        : device float[agents*R][layers][kv_heads*head_dim], written (and
 *                     read back by the call's second kernel); must not overlap w or out.
 * Each reused row is read once for all agents of the call.
 */
KVFIX_API kvfix_status kvfix_mean_correct(const kvfix_bf16* k_reuse, const kvfix_bf16* v_reuse,
                                kvfix_kv_desc reuse, const kvfix_bf16* k_fresh,
                                const kvfix_bf16* v_fresh, kvfix_kv_desc fresh, kvfix_bf16* k_out,
                                kvfix_bf16* v_out, kvfix_kv_desc out, int32_t agents,
                                const int32_t* delta, double rope_base, const int32_t* idx_k,
                                const int32_t* idx_v, int32_t b, const float* w_k,
                                const float* w_v, float* mu_k, float* mu_v, void* stream);

/*
 * kvfix_lowrank_apply -- add a rank-r factorised delta to a KV plane.
 * [KVCMAS] Eq. 4 (corrected cache = reference + estimated delta), Eq. 7 (a delta
 * stored as A B, A of size rows x r, B of size r x D), Eq. 8 with a single anchor.
 *
 *     out[c][l][j][h][e] = bf16( x[c][l][j][h][e] + sum_{k<r} A[c][l][h][j][k] B[c][l][h][k][e] )
 * x, out : one KV plane each, described by desc / out_desc (same shape); out may be x
 *          itself with the same descriptor (in place).
 * A      : device bf16[chunks][layers][kv_heads][tokens][rank], contiguous.
 * B      : device bf16[chunks][layers][kv_heads][rank][head_dim], contiguous.
 * rank   : 16, 32 or 64.  head_dim must be 64 or 128.
 * Arithmetic: bf16 products on the tensor cores (tcgen05, accumulator in tensor memory)
 * with float accumulation, then the add in float and one rounding to bf16.
 */
KVFIX_API kvfix_status kvfix_lowrank_apply(const kvfix_bf16* x, kvfix_kv_desc desc, const kvfix_bf16* A,
                                           const kvfix_bf16* B, int32_t rank, kvfix_bf16* out,
                                           kvfix_kv_desc out_desc, void* stream);

/*
 * kvfix_draft_rank -- rank cached rows by the attention mass of draft queries, keep
 * the best k_rows, and optionally repair them.
 * [BCR] section 3 ("The repair": the row score a_j), App. B Algorithm 2 (draft
 * scoring with grouped-query keys expanded to query heads) and Algorithm 1 (the
 * selected rows' K and V overwritten with exact ones); [KVCMAS] Eq. 3.
 *
 *     scores[c][j] = sum_{l >= layer_begin} sum_{t < draft_steps} sum_{h < q_heads}
 *                    softmax_j( q[c][l][t][h] . k[c][l][j][h / (q_heads/kv_heads)] / sqrt(D) )
 * (summed over (t, h); the ranking equals the mean's).  idx[c] = the k_rows rows with
 * the largest score (ties to the lower index), ascending.
 * If k_io / v_io are non-NULL, then for every layer and KV head, rows idx[c] of k_io /
 * v_io are overwritten with the same rows of k_fresh / v_fresh.  k_io may be the
 * scored buffer `k` itself (the overwrite runs after scoring, in stream order).
 *
 * k              : the assembled keys, `desc` (heads = kv_heads).
 * q              : device bf16[chunks][layers][draft_steps][q_heads][head_dim], contiguous.
 * idx            : device int32[chunks][k_rows]; scores: device double[chunks][tokens].
 * k_fresh, v_fresh, k_io, v_io : planes described by `fresh_desc` / `desc`, or NULL.
 * workspace      : device buffer of kvfix_draft_rank_workspace_bytes(desc, layer_begin)
 *                  bytes (16-byte aligned), contents irrelevant on entry.
 * Limits: q_heads a multiple of kv_heads, q_heads/kv_heads * draft_steps <= 16,
 * head_dim 64 or 128, tokens <= 16384 per chunk, chunks * (layers - layer_begin) *
 * kv_heads <= 65535, 0 <= k_rows <= tokens.
 * Arithmetic: the logits are a bf16 tensor-core contraction (tcgen05) with float
 * accumulation kept in tensor memory; softmax statistics in float; per-unit masses in
 * float, summed over the units of a chunk in a fixed order (layer-major, then head) as
 * a compensated float pair (running sum plus its accumulated rounding errors, about 48
 * significant bits), returned as the double hi + lo.
 */
KVFIX_API size_t kvfix_draft_rank_workspace_bytes(kvfix_kv_desc desc, int32_t layer_begin);
KVFIX_API kvfix_status kvfix_draft_rank(const kvfix_bf16* k, kvfix_kv_desc desc, const kvfix_bf16* q,
                              int32_t draft_steps, int32_t q_heads, int32_t layer_begin,
                              int32_t k_rows, int32_t* idx, double* scores,
                              const kvfix_bf16* k_fresh, const kvfix_bf16* v_fresh,
                              kvfix_kv_desc fresh_desc, kvfix_bf16* k_io, kvfix_bf16* v_io,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * kvfix_lowrank_draft -- kvfix_lowrank_apply of the key plane and kvfix_draft_rank of the
 * corrected keys in one pass: each corrected key tile is scored while it is still on chip,
 * so the corrected keys are read from memory by neither step.
 * [KVCMAS] Eq. 4, 7, 8 (corrected keys = reference keys + A B); [BCR] section 3 ("The
 * repair": rows ranked by the draft queries' attention mass over the predicted keys) and
 * App. B Algorithms 1 and 2.
 *
 * Computes exactly what these calls compute, in this order:
 *     kvfix_lowrank_apply(x, desc, A, B, rank, out, out_desc)
 *     kvfix_draft_rank(out, out_desc, q, draft_steps, q_heads, layer_begin, k_rows, idx,
 *                      scores, k_fresh, v_fresh, fresh_desc, k_fresh ? out : NULL, v_io)
 * with the same bits: out, idx and scores equal the two-call sequence's.  The value
 * plane's low-rank delta is a separate kvfix_lowrank_apply (give its output as v_io to
 * repair its rows here).
 * Arguments are those of the two calls: x/out/A/B/rank as for kvfix_lowrank_apply (out may
 * be x itself, in place); q, draft_steps, q_heads, layer_begin, k_rows, idx and scores as
 * for kvfix_draft_rank.  workspace: device buffer of
 * kvfix_lowrank_draft_workspace_bytes(desc, layer_begin) bytes (16-byte aligned; the
 * draft workspace plus a fixed 132 KB exchange area), contents irrelevant on entry.  k_fresh (optional): the selected rows of out are overwritten with it;
 * v_fresh with v_io (optional): the selected rows of v_io (shaped like out) are
 * overwritten with it.  Limits: head_dim 64 or 128, rank 16/32/64, tokens <= 16384,
 * (q_heads/kv_heads)*draft_steps <= 16.
 * Runs as one persistent cooperative kernel (one CTA per SM, all of its tensor memory;
 * it fails with KVFIX_ECUDA if the device cannot hold one CTA on each SM it uses), then
 * the per-key sums, the top-k and the row repair.
 */
KVFIX_API size_t kvfix_lowrank_draft_workspace_bytes(kvfix_kv_desc desc, int32_t layer_begin);
KVFIX_API kvfix_status kvfix_lowrank_draft(const kvfix_bf16* x, kvfix_kv_desc desc, const kvfix_bf16* A,
                                           const kvfix_bf16* B, int32_t rank, kvfix_bf16* out,
                                           kvfix_kv_desc out_desc, const kvfix_bf16* q, int32_t draft_steps,
                                           int32_t q_heads, int32_t layer_begin, int32_t k_rows, int32_t* idx,
                                           double* scores, const kvfix_bf16* k_fresh, const kvfix_bf16* v_fresh,
                                           kvfix_kv_desc fresh_desc, kvfix_bf16* v_io, void* workspace,
                                           size_t workspace_bytes, void* stream);

/*
 * kvfix_draft_rank_noalloc -- kvfix_draft_rank for callers that cannot allocate device
 * memory.  The pages have no counterpart: this is a service of this library only.
 *
 * Who needs it: a serving engine that gives nearly all of HBM to its own KV-block
 * pool at start-up (a later cudaMalloc fails or fragments the pool), or a
 * latency-critical path that must not pay the device-wide synchronisation a
 * cudaMalloc/cudaFree can imply.  Same arguments and results as kvfix_draft_rank,
 * without the workspace: the scratch lives in a fixed buffer of
 * KVFIX_DRAFT_NOALLOC_SCRATCH_BYTES that the library reserves on every GPU that loads
 * it, until the process exits.  The call allocates nothing.
 * - A problem that needs more scratch than the buffer holds
 *   (kvfix_draft_rank_workspace_bytes(desc, layer_begin) > the constant) returns
 *   KVFIX_EINVAL with a message and launches nothing.
 * - All calls on a device share the buffer: calls whose kernels overlap on the GPU
 *   race.  Order them (one stream, or events).
 * - The buffer keeps the last call's contents; nothing in it needs to start at zero.
 * - The first call on a device looks up the buffer's device address with that device
 *   current; make that first call before any stream capture begins.
 */
#define KVFIX_DRAFT_NOALLOC_SCRATCH_BYTES (64u << 20)
KVFIX_API kvfix_status kvfix_draft_rank_noalloc(const kvfix_bf16* k, kvfix_kv_desc desc,
                                                const kvfix_bf16* q, int32_t draft_steps,
                                                int32_t q_heads, int32_t layer_begin,
                                                int32_t k_rows, int32_t* idx, double* scores,
                                                const kvfix_bf16* k_fresh,
                                                const kvfix_bf16* v_fresh,
                                                kvfix_kv_desc fresh_desc, kvfix_bf16* k_io,
                                                kvfix_bf16* v_io, void* stream);

/*
 * kvfix_diff_encode -- store sibling caches as block-sparse diffs against a master.
 * [TD] section 4.3 (master-mirror layout, block-sparse K/V diff) and section 5 (a
 * mirror keeps the touched block indices and those blocks' K/V contents; one index
 * list shared by K and V).
 *
 * Entry i = (s*L + l)*nblk + blk covers tokens [bt*blk, bt*blk + bt) of layer l of
 * sibling s, all heads, both planes (nblk = tokens / bt).  It is dirty iff some bf16
 * word of K or V in it differs bitwise from the master's (so -0 differs from +0).
 *     mask    : device uint32[ceil(S*L*nblk/32)], bit i%32 of word i/32 = dirty
 *     offsets : device int64[S*L*nblk + 1], offsets[i] = dirty entries before i,
 *               offsets[S*L*nblk] = total
 *     payload : device bf16[capacity_entries][2][bt][kv_heads][head_dim]; dirty entry
 *               i is stored at offsets[i]: the sibling's K block, then its V block.
 * master_* : `master` (chunks == 1); sib_* : `sib` (chunks = S siblings, same shape).
 * h_entries: optional HOST pointer.  If given, the call synchronises the stream after
 *            the mask and offsets are built, stores the total there and returns
 *            KVFIX_ENOSPACE without writing the payload if it exceeds
 *            capacity_entries.  If NULL the call stays asynchronous and the device
 *            skips (and flags) entries beyond capacity_entries.
 * bt must divide tokens.
 */
KVFIX_API kvfix_status kvfix_diff_encode(const kvfix_bf16* master_k, const kvfix_bf16* master_v,
                               kvfix_kv_desc master, const kvfix_bf16* sib_k,
                               const kvfix_bf16* sib_v, kvfix_kv_desc sib, int32_t block_tokens,
                               uint32_t* mask, int64_t* offsets, kvfix_bf16* payload,
                               int64_t capacity_entries, int64_t* h_entries, void* stream);

/*
 * kvfix_diff_gather -- restore every sibling from the master and its diff.
 * [TD] section 4.4, Algorithm 1 (load the master block, overwrite the blocks the diff
 * touches with the diff's values); section 5 (paired K/V diff kernel).
 *
 *     out_P[s][l][block blk] = payload[offsets[i]].P   if mask bit i is set
 *                            = master_P[l][block blk]   otherwise
 * Each master block is read once for all siblings.
 * mask, offsets, payload : as written by kvfix_diff_encode.
 * payload_entries        : entries the payload buffer holds; a dirty entry whose offset
 *                          lies beyond it is not read (its block gets the master's
 *                          contents) and is flagged (KVFIX_ENOSPACE in kvfix_check_status).
 * out_k, out_v           : `out` (chunks = siblings, same shape as master).
 */
KVFIX_API kvfix_status kvfix_diff_gather(const kvfix_bf16* master_k, const kvfix_bf16* master_v,
                               kvfix_kv_desc master, const uint32_t* mask,
                               const int64_t* offsets, const kvfix_bf16* payload,
                               int64_t payload_entries, int32_t siblings, int32_t block_tokens,
                               kvfix_bf16* out_k, kvfix_bf16* out_v, kvfix_kv_desc out,
                               void* stream);

/*
 * kvfix_diff_restore -- fused restore of every sibling into a paged KV pool.
 * [TD] section 4.4, Algorithm 1 (per layer: load the master block, overwrite it where
 * the sibling's block-sparse diff touches it, re-align the keys from the old to the new
 * positions with RoPERecover, write the rows to the paged cache through the slot
 * mapping); section 5 (the restore is one fused kernel, no intermediate full copy).
 *
 * Re-alignment of sibling s is one rotary shift by delta[s] = P_new - P_old (as in
 * kvfix_rerope; values are not rotated).  Token t of sibling s is written, in every
 * layer, to pool row slot_mapping[s*tokens + t]:
 *     pool_k[l][slot] = rotate(delta[s], restored K row),  pool_v[l][slot] = restored V row
 * where the restored row is the payload's if the entry is dirty, else the master's.
 * A negative slot means the token is not restored; a slot >= pool.tokens is skipped
 * and flagged (KVFIX_EDEVICE in kvfix_check_status).  Pool rows no slot names are left
 * unchanged.  Slots must be distinct (two tokens naming one row race).
 * master_*, mask, offsets, payload, payload_entries, siblings, block_tokens: as for
 *                  kvfix_diff_gather.
 * delta          : device int32[siblings].
 * rope_base      : as for kvfix_rerope.
 * slot_mapping   : device int32[siblings][tokens].
 * pool_k, pool_v : `pool` -- chunks == 1, layers and heads x head_dim as the master's,
 *                  tokens = the pool's rows per layer; neither may overlap the master.
 * delta[s] = 0 copies sibling s's keys bit for bit.
 */
KVFIX_API kvfix_status kvfix_diff_restore(const kvfix_bf16* master_k, const kvfix_bf16* master_v,
                                kvfix_kv_desc master, const uint32_t* mask,
                                const int64_t* offsets, const kvfix_bf16* payload,
                                int64_t payload_entries, int32_t siblings, int32_t block_tokens,
                                const int32_t* delta, double rope_base,
                                const int32_t* slot_mapping, kvfix_bf16* pool_k,
                                kvfix_bf16* pool_v, kvfix_kv_desc pool, void* stream);

/*
 * Anchor-pool correction.  [KVCMAS] section 3.3 (each anchor keeps its base cache and its
 * delta correction as low-rank factors, Eq. 7; the correction is the weighted sum of the
 * anchors' deltas, Eq. 8, applied to the aligned source cache, Eq. 4) and App. A.3
 * (reliability gate, Eq. 9-11; token-wise weights; keys matched in canonical positions).
 *
 * Factor layout, per plane, for C segments (src.chunks), V anchors, L layers, n tokens,
 * F = kv_heads * head_dim features and rank r:
 *     A  : device bf16 [C][V][L][n][r]        (first factor, row t of the segment)
 *     Bt : device bf16 [C][V][L][F][r]        (second factor, stored transposed)
 * so that anchor v's state of layer l is A[c][v][l] * Bt[c][v][l]^T ([n x F]).
 * anchors: 1..16; rank: 16, 32 or 64 (the first-factor tiles of all anchors stay in
 * shared memory: ranks 16 and 32 take up to 16 anchors, rank 64 up to 8; the calls return
 * KVFIX_EINVAL for shapes that do not fit); F must be a multiple of 128.
 */

/* Bytes of device workspace kvfix_anchor_gate needs for `src`, `anchors` and `prefix`. */
KVFIX_API size_t kvfix_anchor_gate_workspace_bytes(kvfix_kv_desc src, int32_t anchors,
                                                   int32_t prefix);

/*
 * kvfix_anchor_gate -- [KVCMAS] App. A.3 "Reliability Gate", Eq. 9-11, per segment c:
 *     d_v  = ( sum_l || V_src^(l)[:k] - (A_v Bt_v^T)^(l)[:k] ||_F^2 )^(1/2)
 *     g_v  = softmax_v(-d_v / T),   Hbar = -sum_v g_v log2 g_v / log2 V
 *     accept = V >= 2 && Hbar <= tau
 * v_src      : `src`, the source value plane (chunks = segments).
 * a_c, b_ct  : base-state factors of the value plane (layout above).
 * prefix k   : 1..tokens; temperature T > 0.
 * d, g       : device double [C][V];  hbar : device double [C] (NaN if V < 2);
 * accept     : device int32 [C].  Distances are summed per 128-row tile in float and
 *              across tiles and layers in double, in a fixed order.
 * workspace  : device, at least kvfix_anchor_gate_workspace_bytes(), 16-byte aligned.
 */
KVFIX_API kvfix_status kvfix_anchor_gate(const kvfix_bf16* v_src, kvfix_kv_desc src,
                                         const kvfix_bf16* a_c, const kvfix_bf16* b_ct,
                                         int32_t anchors, int32_t rank, int32_t prefix,
                                         double temperature, double tau, double* d, double* g,
                                         double* hbar, int32_t* accept, void* workspace,
                                         size_t workspace_bytes, void* stream);

/*
 * kvfix_anchor_correct -- token-weighted anchor correction of both planes:
 *     m_v[t] = (1/F) sum_f | x[t][f] - (A_c,v Bt_c,v^T)[t][f] |   (x: keys in canonical positions)
 *     w[t]   = softmax_v(-m_v[t] / T)                            (per plane, layer, token)
 *     out[t] = Align(x[t]) + sum_v w_v[t] (A_d,v Bt_d,v^T)[t]     (bf16)
 * Align rotates keys by delta[c] (as kvfix_rerope) and leaves values unchanged.
 * k_src, v_src : `src` (chunks = segments); head_dim 64 or 128.
 * a_c_*, b_ct_*: base-state factors; a_d_*, b_dt_*: delta-correction factors (layout above).
 * delta        : device int32 [C]; rope_base as for kvfix_rerope.
 * accept       : optional device int32 [C] (e.g. kvfix_anchor_gate's): segments with 0 are
 *                skipped entirely (outputs and weights untouched).  NULL corrects all.
 * w_k, w_v     : device float [C][L][n][V], written with the token weights.
 * k_out, v_out : `out`, the shape of src; may be exactly src (in place), no other overlap.
 * The delta term is formed on the tensor cores from bf16(w_v * A_d,v) (the weight is
 * folded into the first factor, rounded once to bf16) with float accumulation.
 */
KVFIX_API kvfix_status kvfix_anchor_correct(
    const kvfix_bf16* k_src, const kvfix_bf16* v_src, kvfix_kv_desc src, const kvfix_bf16* a_c_k,
    const kvfix_bf16* b_ct_k, const kvfix_bf16* a_c_v, const kvfix_bf16* b_ct_v,
    const kvfix_bf16* a_d_k, const kvfix_bf16* b_dt_k, const kvfix_bf16* a_d_v,
    const kvfix_bf16* b_dt_v, int32_t anchors, int32_t rank, double temperature,
    const int32_t* delta, double rope_base, const int32_t* accept, float* w_k, float* w_v,
    kvfix_bf16* k_out, kvfix_bf16* v_out, kvfix_kv_desc out, void* stream);

/*
 * kvfix_repair_layout -- the rows a draft-scored repair recomputes, in one of the layouts
 * of [BCR] section 3 "The layouts", App. A.2 ("The policy", Table 8) and App. B
 * (Algorithms 1 and 2).  For each unit u of scores [units][tokens]
 * (e.g. kvfix_draft_rank's), with rho = budget_num / budget_den and rounding of halves
 * to even:
 *   KVFIX_LAYOUT_SINGLE: the round(rho n) rows with the largest scores;
 *   KVFIX_LAYOUT_CHUNK : chunk_tokens-token chunks (the last may be short), each scored by
 *                        the mean of its rows' scores (summed in index order, in double);
 *                        the max(1, round(rho n / chunk_tokens)) best chunks, all their
 *                        rows.  skip_rule != 0: no rows when n < 2 chunk_tokens or
 *                        rho n < chunk_tokens (Algorithm 1's skip rule);
 *   KVFIX_LAYOUT_GROW  : round(rho n) rows: the best unselected row seeds a span, which
 *                        takes the better of its two unselected neighbours (left on a tie)
 *                        while that one scores at least tau times the seed, until neither
 *                        does or the budget is spent; then the next seed.
 * Ties go to the lower index.  Scores must be finite.
 * idx      : device int32 [units][max_rows]: the rows, ascending, then -1.
 * counts   : device int32 [units]: rows chosen (the same for every unit except when the
 *            chunk layout's last, short chunk is chosen).
 * max_rows : at least the layout's largest count (KVFIX_EINVAL otherwise): round(rho n)
 *            for single and grow, (chunks chosen) * chunk_tokens (at most n) for chunk.
 * tokens   : 1..16384.
 */
typedef enum { KVFIX_LAYOUT_SINGLE = 0, KVFIX_LAYOUT_CHUNK = 1, KVFIX_LAYOUT_GROW = 2 } kvfix_layout;
KVFIX_API kvfix_status kvfix_repair_layout(const double* scores, int32_t units, int32_t tokens,
                                           int32_t layout, int32_t chunk_tokens, int32_t budget_num,
                                           int32_t budget_den, double tau, int32_t skip_rule,
                                           int32_t* idx, int32_t max_rows, int32_t* counts,
                                           void* stream);

/*
 * kvfix_repair_rows -- overwrite the chosen rows with exact ones ([BCR] App. B Algorithm 1;
 * [KVCMAS] Eq. 3): for every chunk c of `desc`, layer and KV head, rows
 * idx[c][0 .. counts[c]) of k_io / v_io get the same rows of k_fresh / v_fresh
 * (`fresh_desc`, the shape of desc).  idx holds max_rows entries per chunk; rows out of
 * range are skipped and flagged (KVFIX_EDEVICE in kvfix_check_status).  Either plane may
 * be skipped by passing NULL for both its pointers.
 */
KVFIX_API kvfix_status kvfix_repair_rows(kvfix_bf16* k_io, kvfix_bf16* v_io, kvfix_kv_desc desc,
                                         const kvfix_bf16* k_fresh, const kvfix_bf16* v_fresh,
                                         kvfix_kv_desc fresh_desc, const int32_t* idx,
                                         int32_t max_rows, const int32_t* counts, void* stream);

/*
 * kvfix_master_select -- the master of a round's cache family.  [TD] section 4.2 ("reuse
 * plan output": the reuse pass accumulates a deviation score per request; the master is
 * the request with the lowest total deviation from the shared blocks, which keeps the
 * mirrors' diffs small) and section 4.3 (master-mirror layout).
 *     totals[a] = sum_{r < R} sum_{j < tokens} (d_k[a R + r][j] + d_v[a R + r][j])
 *     *master   = the agent with the smallest total (ties to the lower index)
 * d_k, d_v : device float [agents * R][tokens] as kvfix_score_topk writes them for a
 *            collective round (unit a R + r); either may be NULL.
 * totals   : device double [agents], summed in double in a fixed order (per agent: thread
 *            t of 256 takes every 256th value, then a tree over threads).
 * master   : device int32 [1].
 */
KVFIX_API kvfix_status kvfix_master_select(const float* d_k, const float* d_v, int32_t agents,
                                           int32_t units_per_agent, int32_t tokens, double* totals,
                                           int32_t* master, void* stream);

/*
 * kvfix_diff_encode_split -- block-sparse diffs with one block list per plane.  [TD]
 * section 5 (the K and V planes share one block index list only when they touch the same
 * blocks).  As kvfix_diff_encode, except that entry i is dirty in plane P iff some bf16
 * word of plane P in it differs from the master's, and each plane has its own list:
 *     mask_k / mask_v       : device uint32[ceil(S*L*nblk/32)]
 *     offsets_k / offsets_v : device int64[S*L*nblk + 1]
 *     payload_k / payload_v : device bf16[capacity_P][bt][kv_heads][head_dim] (one plane)
 * h_entries: optional HOST int64[2] (K, V); if given, the call synchronises and returns
 * KVFIX_ENOSPACE, writing no payload, when a plane's total exceeds its capacity.  If NULL,
 * entries beyond a capacity are skipped and flagged.
 */
KVFIX_API kvfix_status kvfix_diff_encode_split(
    const kvfix_bf16* master_k, const kvfix_bf16* master_v, kvfix_kv_desc master,
    const kvfix_bf16* sib_k, const kvfix_bf16* sib_v, kvfix_kv_desc sib, int32_t block_tokens,
    uint32_t* mask_k, uint32_t* mask_v, int64_t* offsets_k, int64_t* offsets_v,
    kvfix_bf16* payload_k, kvfix_bf16* payload_v, int64_t capacity_k, int64_t capacity_v,
    int64_t* h_entries, void* stream);

/*
 * kvfix_diff_gather_split -- restore every sibling from the master and its per-plane
 * diffs (the lists kvfix_diff_encode_split writes): K blocks from (mask_k, offsets_k,
 * payload_k), V blocks from (mask_v, offsets_v, payload_v); entries_* are the payloads'
 * sizes (an offset beyond them is not read and is flagged).  Otherwise as
 * kvfix_diff_gather.
 */
KVFIX_API kvfix_status kvfix_diff_gather_split(
    const kvfix_bf16* master_k, const kvfix_bf16* master_v, kvfix_kv_desc master,
    const uint32_t* mask_k, const uint32_t* mask_v, const int64_t* offsets_k,
    const int64_t* offsets_v, const kvfix_bf16* payload_k, const kvfix_bf16* payload_v,
    int64_t entries_k, int64_t entries_v, int32_t siblings, int32_t block_tokens,
    kvfix_bf16* out_k, kvfix_bf16* out_v, kvfix_kv_desc out, void* stream);

/*
 * kvfix_diff_restore_split -- kvfix_diff_restore from per-plane diffs (the lists
 * kvfix_diff_encode_split writes): the restored K block of a sibling comes from
 * (mask_k, offsets_k, payload_k), its V block from (mask_v, offsets_v, payload_v); a
 * plane whose block is clean is read from the master.  entries_* are the payloads' sizes
 * (an offset beyond them is not read and is flagged).  Re-alignment, slot mapping, pool
 * layout, validation and errors as for kvfix_diff_restore; the output is the same bits
 * as kvfix_diff_restore's on the joint lists of the same siblings.
 */
KVFIX_API kvfix_status kvfix_diff_restore_split(
    const kvfix_bf16* master_k, const kvfix_bf16* master_v, kvfix_kv_desc master,
    const uint32_t* mask_k, const uint32_t* mask_v, const int64_t* offsets_k,
    const int64_t* offsets_v, const kvfix_bf16* payload_k, const kvfix_bf16* payload_v,
    int64_t entries_k, int64_t entries_v, int32_t siblings, int32_t block_tokens,
    const int32_t* delta, double rope_base, const int32_t* slot_mapping, kvfix_bf16* pool_k,
    kvfix_bf16* pool_v, kvfix_kv_desc pool, void* stream);

/*
 * kvfix_anchor_gate_correct -- kvfix_anchor_gate and kvfix_anchor_correct in one pass over
 * the sources: the gate's value-plane distances (prefix k) come from the same
 * reconstructions as the value plane's token weights, the gate is decided on the device,
 * and only accepted segments are corrected (rejected ones keep their outputs; their
 * weights are still written).  Arguments as for the two calls; `accept` is an output here.
 * The gate's squares are summed per thread over the features, folded per warp by a fixed
 * tree and then over the warps in a fixed order, so d differs from kvfix_anchor_gate's in
 * the last bits (and is deterministic).
 * workspace: at least kvfix_anchor_gate_workspace_bytes(src, anchors, src.tokens).
 * head_dim 64 or 128.
 */
KVFIX_API kvfix_status kvfix_anchor_gate_correct(
    const kvfix_bf16* k_src, const kvfix_bf16* v_src, kvfix_kv_desc src, const kvfix_bf16* a_c_k,
    const kvfix_bf16* b_ct_k, const kvfix_bf16* a_c_v, const kvfix_bf16* b_ct_v,
    const kvfix_bf16* a_d_k, const kvfix_bf16* b_dt_k, const kvfix_bf16* a_d_v,
    const kvfix_bf16* b_dt_v, int32_t anchors, int32_t rank, int32_t prefix, double temperature,
    double tau, const int32_t* delta, double rope_base, double* d, double* g, double* hbar,
    int32_t* accept, float* w_k, float* w_v, kvfix_bf16* k_out, kvfix_bf16* v_out,
    kvfix_kv_desc out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Paged pools.  A pool holds `slots` rows per layer; row (layer, slot, head) stores head_dim
 * values of a key and of a value in one of three forms:
 *   KVFIX_POOL_BF16  the values, 2 head_dim bytes; no scales.
 *   KVFIX_POOL_E4M3  head_dim e4m3 codes (one byte each, in order) and one scale byte b:
 *                    value = e4m3(code) * 2^(b - 127).  With A the largest finite magnitude
 *                    of the row, 2^(b-127) is the least power of two with
 *                    A <= 448 * 2^(b-127), kept within [2^-110, 2^119]; codes are
 *                    x / 2^(b-127) rounded to nearest even; infinities saturate to the
 *                    largest code.  A row that holds a NaN gets b = 255 and codes 0, and reads
 *                    as NaN throughout (the codes 0x7f and 0xff are not written, and mean
 *                    nothing).  Bytes that are not written otherwise count as the nearest
 *                    that are: below 17 as 17, 247 to 254 as 246.  Every stored value is
 *                    exactly a bf16 value.
 *   KVFIX_POOL_INT4  head_dim/2 bytes: each 32-bit word (little endian) holds 8 codes 0..15,
 *                    value 2i in bits [4i, 4i+4) and value 2i+1 in bits [16+4i, 20+4i).
 *                    Groups of 32 values share a bf16 scale and a bf16 zero (one 32-bit
 *                    word, scale in the low half): value = bf16(scale * code + zero).  Over
 *                    the group's finite values: zero = min, scale = bf16((max - min) / 15)
 *                    (float division; 0 if below 2^-120; a range beyond the largest float
 *                    counts as that), code = rint((x - zero) * (1 / scale)) in float, kept
 *                    within 0..15 (0 if the scale is 0).  Infinities saturate, a NaN takes
 *                    code 0 (the form has no NaN); a group with no finite value is all zero.
 *
 * kvfix_pool describes a pool (or some consecutive layers of one):
 *   code bytes of (l, slot, h): k + l*stride_layer + slot*stride_slot + h*B with B = 2 D,
 *       D or D/2 (strides in BYTES, multiples of 16; stride_slot >= kv_heads*B; 16-byte
 *       aligned bases).  K and V rows may interleave, a slot's V behind its K, say;
 *   scales: contiguous [layers][kv_heads][slots] bytes (e4m3), or
 *       [layers][kv_heads][slots][D/32] 32-bit words, 4-byte aligned (int4); NULL for bf16.
 * head_dim D is 64 or 128.  The heads-major scales put the scales of one head's consecutive
 * slots side by side, as attention reads them.
 * In the calls below planes without rows (no chunks or tokens) may be NULL, and nothing is done.
 */
typedef enum { KVFIX_POOL_BF16 = 0, KVFIX_POOL_E4M3 = 1, KVFIX_POOL_INT4 = 2 } kvfix_pool_format;
typedef struct {
    int32_t format; /* kvfix_pool_format */
    int32_t layers;
    int32_t slots;
    int32_t kv_heads;
    int32_t head_dim;
    int64_t stride_layer; /* bytes */
    int64_t stride_slot;  /* bytes */
    void* k;
    void* v;
    void* k_scales;
    void* v_scales;
} kvfix_pool;

/*
 * kvfix_pool_write -- write cached rows into a pool, quantised as they are written.  [TD]
 * section 4.4, Algorithm 1 (re-aligned rows written to the paged cache through the slot
 * mapping); [AKS] combines reuse with caches kept in 2 to 4 bits, which this form serves.
 *
 * Token t of chunk c goes, in every layer, to pool row slot_mapping[c*tokens + t], in the
 * pool's format.  Keys are first rotated by delta[c] as kvfix_rerope does (the same bf16
 * bits); delta NULL, or 0, writes them as they are; values are not rotated.  A negative slot
 * means the token is not kept; a slot >= pool.slots is skipped and flagged (KVFIX_EDEVICE in
 * kvfix_check_status).  Rows no slot names are left unchanged.  Slots must be distinct (two
 * tokens naming one row race).
 * k, v         : `src` planes (any chunks and tokens, layers and heads of the pool).
 * slot_mapping : device int32[chunks][tokens].
 * delta        : device int32[chunks], or NULL.  rope_base: as for kvfix_rerope (ignored,
 *                and unchecked, without delta).
 */
KVFIX_API kvfix_status kvfix_pool_write(const kvfix_bf16* k, const kvfix_bf16* v, kvfix_kv_desc src,
                                        const int32_t* delta, double rope_base,
                                        const int32_t* slot_mapping, kvfix_pool pool, void* stream);

/*
 * kvfix_pool_read -- read pool rows back as bf16 rows, keys re-aligned on the way: the
 * inverse gather of kvfix_pool_write.  Row t of chunk c of the outputs gets the values that
 * pool row slot_mapping[c*tokens + t] stands for, keys rotated by delta[c] (as kvfix_rerope
 * of those bf16 values).  Rows with a negative slot are left unchanged; a slot >= pool.slots
 * leaves its row unchanged and is flagged.  A token may be read any number of times.
 */
KVFIX_API kvfix_status kvfix_pool_read(kvfix_pool pool, const int32_t* slot_mapping, const int32_t* delta,
                                       double rope_base, kvfix_bf16* k, kvfix_bf16* v, kvfix_kv_desc out,
                                       void* stream);

/*
 * kvfix_shared_attend -- attention of the agents of a round over the context they share and
 * their own tokens, read from one layer of a paged pool.  [TD] section 2.1 (a round's prompts
 * hold the same blocks) and section 4.4 (attention over the restored paged cache); [BCR] App.
 * B, Algorithm 2 (grouped-query keys expanded to query heads).
 *
 * The agents of group g, group_begin[g] <= a < group_begin[g+1], share the prefix of
 * prefix_len[g] keys on the pages prefix_pages[g]; agent a's own suffix_len[a] keys lie on
 * suffix_pages[a].  An agent outside every group has no prefix.  Key i of a page list is pool
 * row pages[i / page_tokens] * page_tokens + i % page_tokens.  The sequence of an agent is
 * its prefix, then its suffix; its new_tokens = q.tokens queries stand at the last new_tokens
 * places of it (their keys and values are already in the pool), so query t sees the first
 *     N_t = prefix_len + suffix_len - new_tokens + 1 + t
 * keys (none if that is not positive).  With z_j = scale * q[a][t][h] . k[j][h / (q_heads /
 * kv_heads)] over the keys it sees:
 *     out[a][t][h] = sum_j exp(z_j) v[j] / sum_j exp(z_j),   lse[a][t][h] = log sum_j exp(z_j)
 * and out = 0, lse = -inf for a query that sees no key.  A group's shared keys are read once
 * for all its agents.  One new token per agent is a decode step; more are drafts or a message
 * that every agent receives.
 * q, out       : planes with chunks = agents, layers = 1, tokens = new tokens, kv_heads =
 *                query heads (a multiple of the pool's), head_dim the pool's.
 * pool         : one layer (layers == 1), any format; slots a positive multiple of page_tokens;
 *                scales 16-byte aligned.
 * page_tokens  : 16, 32, 64 or 128.
 * prefix_pages : device int32[groups][max_prefix_pages]; prefix_len: device int32[groups];
 *                group_begin: device int32[groups + 1], ascending within 0..agents.  groups
 *                may be 0 (all three NULL).
 * suffix_pages : device int32[agents][max_suffix_pages]; suffix_len: device int32[agents].
 * scale        : > 0, with scale * log2(e) a normal float (usually head_dim^-1/2).
 * lse          : device float[agents][new tokens][q_heads], or NULL.
 * workspace    : device buffer of kvfix_shared_attend_workspace_bytes(agents, new tokens,
 *                q_heads, kv_heads, head_dim, groups) bytes, 16-byte aligned, contents
 *                irrelevant on entry.  Two float rows of head_dim per (agent, new token, query
 *                head), and whatever the call's size 131072 rows (67 MB at head_dim 128) where
 *                a block may be larger than the small ones below, 16384 or 32768 where one may
 *                be small.
 * Pages, lengths and groups are read on the device, so a captured call follows them as they
 * change.  A page out of range counts as absent (its keys are not seen), a length outside its
 * page list and a group boundary out of order are clamped; each is flagged (KVFIX_EDEVICE in
 * kvfix_check_status).  Page entries past a length are not read.
 * Limits: (max_prefix_pages + max_suffix_pages) * page_tokens < 2^30 and agents * new tokens *
 * q_heads < 2^27.
 * Arithmetic: bf16 or f16 tensor-core products with float accumulation.  Stored values are
 * exact operands; the softmax weights exp(z_j) are rounded to bf16 before their product with
 * the values (by up to 2^-8 of each).  Where a block of queries is small (at most 16 rows, a row
 * being a new token and a query head of one KV head) an e4m3 pool may go by f16 instead: the
 * products of a weight and its value row's scale are rounded, by up to 2^-11 of each, or, below
 * 2^-21 of the query's largest such product, by up to 2^-32 of that; and a query's components
 * below 2^-26 of its largest lose bits.  Maxima, sums and lse in float; one rounding of out to
 * bf16.  The same inputs give the same bits on every run; the order of sums depends on the
 * lengths.
 * A NaN or infinity in a key that a query sees reaches that query, one in a value every query
 * that sees its key; with several new tokens a value row that only the later of them see may
 * reach the earlier ones too (a weight of zero times NaN).  Rows that belong to no key, or to
 * none that a block of queries sees, may hold anything.
 */
KVFIX_API size_t kvfix_shared_attend_workspace_bytes(int32_t agents, int32_t new_tokens, int32_t q_heads,
                                                     int32_t kv_heads, int32_t head_dim, int32_t groups);
KVFIX_API kvfix_status kvfix_shared_attend(const kvfix_bf16* q, kvfix_kv_desc q_desc, kvfix_pool pool,
                                           int32_t page_tokens, const int32_t* prefix_pages,
                                           int32_t max_prefix_pages, const int32_t* prefix_len,
                                           const int32_t* group_begin, int32_t groups,
                                           const int32_t* suffix_pages, int32_t max_suffix_pages,
                                           const int32_t* suffix_len, double scale, kvfix_bf16* out,
                                           kvfix_kv_desc out_desc, float* lse, void* workspace,
                                           size_t workspace_bytes, void* stream);

/*
 * kvfix_rotary -- rotary positions of queries and keys, one position per token: what a step's
 * new rows need before they are written and attended over, and the re-alignment of cached
 * keys whose model scales its frequencies, rotates part of a head or pairs neighbours, which
 * kvfix_rerope does not cover.  [KVCMAS] section 2.2 and App. A.3; [BCR] App. A.
 *
 * With p = positions[c][t], n = rope.rotary_dim and pairs (x_a, x_b), a = i, b = i + n/2
 * (KVFIX_ROPE_HALF) or a = 2i, b = 2i + 1 (KVFIX_ROPE_INTERLEAVED), i < n/2, in every layer and head:
 *     y_a = m (x_a cos(p theta_i) - x_b sin(p theta_i)),  y_b = m (x_b cos(p theta_i) + x_a sin(p theta_i))
 * and y_d = x_d for d >= n.  m = rope.attention; theta_i = base^(-2i/n), scaled by what the pair
 * keeps of its frequency, s_i in [0, 1]: theta_i (s_i + (1 - s_i) / factor), with
 *   KVFIX_ROPE_PLAIN   s = 1 (factor, low, high and original_tokens are not read);
 *   KVFIX_ROPE_LINEAR  s = 0;
 *   KVFIX_ROPE_BANDS   s = (r_i - low) / (high - low) within [0, 1], r_i = original_tokens theta_i / 2 pi
 *                      the pair's turns over the original context;
 *   KVFIX_ROPE_YARN    s falls with the pair's number: 1 up to lo, 0 from hi, s = 1 - (i - lo) /
 *                      max(hi - lo, 0.001) between, lo = max(floor(z(high)), 0) and hi =
 *                      min(ceil(z(low)), n - 1), z(r) = n log(original_tokens / (2 pi r)) / (2 log base).
 * Rotations add up: rows at p turned by d (attention 1) are rows at p + d, so positions may be
 * shifts, of any sign; and the gradient of a rotation is the rotation of the outputs' gradient
 * by the negated positions, attention as it was.
 *
 * q, k         : planes of the same chunks, layers, tokens and head_dim, each with its heads; either
 *                may be left out (kv_heads 0 in q_desc or k_desc: its pointers and its output's
 *                descriptor are not read).
 * q_out, k_out : shaped like q and k; each exactly its input (in place) or apart from both, its rows
 *                apart from each other.  Planes may be views of one buffer whose rows
 *                interleave, as a projection leaves them.
 * positions    : device int32[chunks][tokens], any sign; apart from the outputs.
 * rope         : rotary_dim even, 2..head_dim; base > 1; attention > 0 (1: a rotation alone); scaled
 *                forms want factor >= 1, bands and yarn original_tokens >= 1 and 0 < low < high.
 * Limits: chunks * layers * tokens < 2^31, fewer than 2^30 values a token row.
 * Arithmetic: the frequencies in double on the host; angles exact modulo a turn (64-bit
 * fractions of it); cos, sin and the rotation in float; one rounding to bf16.  Position 0 with
 * attention 1 gives the input bit for bit.
 */
typedef enum { KVFIX_ROPE_HALF = 0, KVFIX_ROPE_INTERLEAVED = 1 } kvfix_rope_layout;
typedef enum {
    KVFIX_ROPE_PLAIN = 0,
    KVFIX_ROPE_LINEAR = 1,
    KVFIX_ROPE_BANDS = 2,
    KVFIX_ROPE_YARN = 3
} kvfix_rope_scaling;
typedef struct {
    int32_t layout;  /* kvfix_rope_layout */
    int32_t rotary_dim;
    int32_t scaling; /* kvfix_rope_scaling */
    int32_t original_tokens;
    double base;
    double factor;
    double low;  /* turns over the original context: at most low, the frequency is divided by factor; */
    double high; /* at least high, it is kept */
    double attention;
} kvfix_rope;
KVFIX_API kvfix_status kvfix_rotary(const kvfix_bf16* q, kvfix_kv_desc q_desc, const kvfix_bf16* k,
                                    kvfix_kv_desc k_desc, const int32_t* positions, kvfix_rope rope,
                                    kvfix_bf16* q_out, kvfix_kv_desc q_out_desc, kvfix_bf16* k_out,
                                    kvfix_kv_desc k_out_desc, void* stream);

/*
 * kvfix_tree_attend -- kvfix_shared_attend for trees of drafted tokens: each agent's drafts are
 * verified in one pass, every node seeing its own line of descent.  [TD] section 2.1; [BCR]
 * App. B, Algorithm 2 (draft queries over the cache).
 *
 * The last N = nodes[a] of agent a's suffix_len[a] own keys are its tree's nodes, in an order in
 * which a node comes after its ancestors; query t < N stands for node t.  It sees the agent's
 * whole prefix, the own keys before the tree, and node j of the tree where j <= t and bit j % 32 of
 * tree_mask[a][t][j / 32] is set (its own bit included: a mask without it hides a node from
 * itself).  A query t >= N sees nothing: out = 0, lse = -inf, as for a row that no key is left to.
 * nodes        : device int32[agents], or NULL: new_tokens each.  A number outside 0..min(q.tokens,
 *                suffix_len) is clamped and flagged (KVFIX_EDEVICE in kvfix_check_status).
 *                Apart from out, lse and the workspace, as tree_mask is.
 * tree_mask    : device uint32[agents][q.tokens][ceil(q.tokens / 32)]; rows of queries t >= N and
 *                bits past t are not read.
 * All else, the workspace (kvfix_shared_attend_workspace_bytes) and the limits are kvfix_shared_attend's,
 * with N in the place of new_tokens, and so is the arithmetic (parts may be cut elsewhere, so that
 * a chain of nodes and as many new tokens in a row may differ in their last bits).  A NaN or
 * infinity in the value row of a node may reach the agent's other nodes (a weight of zero times
 * NaN); one in a key reaches those that see it alone.
 */
KVFIX_API kvfix_status kvfix_tree_attend(const kvfix_bf16* q, kvfix_kv_desc q_desc, kvfix_pool pool,
                                         int32_t page_tokens, const int32_t* prefix_pages,
                                         int32_t max_prefix_pages, const int32_t* prefix_len,
                                         const int32_t* group_begin, int32_t groups,
                                         const int32_t* suffix_pages, int32_t max_suffix_pages,
                                         const int32_t* suffix_len, const int32_t* nodes,
                                         const uint32_t* tree_mask, double scale, kvfix_bf16* out,
                                         kvfix_kv_desc out_desc, float* lse, void* workspace,
                                         size_t workspace_bytes, void* stream);

/*
 * Page books.  A list is a sequence's page list (as kvfix_shared_attend reads them) and its length:
 * list i's token t lies in pool row pages[i][t / page_tokens] * page_tokens + t % page_tokens, for
 * t < len[i].  refs counts, for every page of the pool, the lists that hold it; a page with none
 * is free.  [TD] section 2.1 (agents of a round hold the same blocks) and section 4.3 (one master, many
 * mirrors).  Prefix and suffix lists of a round may be rows of one table.  The books lie on the device and
 * the calls below change them there, so captured graphs follow them; the same books give
 * the same pages on every run.
 * pool        : every layer of the pool (all are copied alike); any format.
 * page_tokens : 16, 32, 64 or 128; pool.slots a positive multiple of it.
 * refs        : device int32[pool.slots / page_tokens].
 * pages       : device int32[lists][max_pages]; entries at and past ceil(len / page_tokens) mean nothing.
 * len         : device int32[lists], each within 0..max_pages * page_tokens.
 * Limits: lists <= 2^24, lists * max_pages < 2^30, max_pages * page_tokens < 2^30; at most 65535 layers
 * of fewer than 2^22 values a row.
 * A list whose length, pages or arguments are out of range is left as it is and flagged
 * (KVFIX_EDEVICE in kvfix_check_status); such an entry elsewhere in its pages is skipped and flagged.
 *
 * kvfix_pages_extend -- room for extra[i] >= 0 tokens behind list i, which may begin as a fork:
 *   parent[i] = i (or parent NULL): the list grows.
 *   parent[i] = j, another list   : list i, empty until now, takes over j's tokens as they are on entry
 *                                   and shares their pages (their counts rise).
 *   parent[i] < 0                 : nothing happens to list i.
 * Tokens len .. len + extra get pages; len[i] becomes that sum.  Where extra > 0 and the last page
 * is partly full, and the list is a fork or others hold that page too (refs > 1 on entry), the
 * list gets a copy of it instead (the rows of its own tokens, all layers), and the page counts one
 * list less.  So rows behind a list's old length are its own to write.  New pages are the lowest
 * free ones: list by list, a copy's first, then the others in order; pages that become free in
 * this call are not among them.  Where the free pages do not reach, that list and every later one
 * that needs a page are left as they were and flagged (KVFIX_ENOSPACE): their len tells.  Rows of
 * new pages keep what they held.
 * workspace   : device, kvfix_pages_extend_workspace_bytes(pool pages, lists) bytes, 16-byte aligned.
 */
KVFIX_API size_t kvfix_pages_extend_workspace_bytes(int32_t pool_pages, int32_t lists);
KVFIX_API kvfix_status kvfix_pages_extend(kvfix_pool pool, int32_t page_tokens, int32_t* refs, int32_t* pages,
                                          int32_t max_pages, int32_t* len, int32_t lists, const int32_t* parent,
                                          const int32_t* extra, void* workspace, size_t workspace_bytes,
                                          void* stream);

/*
 * kvfix_pages_cut -- what a list keeps: its first base[i] tokens, then, moved up behind them, the
 * tokens base[i] + path[i][j] for j < kept[i] (a tree's accepted nodes, in ascending order); the
 * rest is dropped, and pages behind the new length lose this list (their entries become -1).
 *   base[i] = len[i] - T, path: nodes of a tree of T      accepts that path;
 *   base[i] = a shorter length, kept[i] = 0 (or max_path 0) rolls the list back;
 *   base[i] = 0, kept[i] = 0                              frees it;
 *   base[i] < 0                                           leaves it alone.
 * Rows move in all layers, codes and scales bit for bit.  The rows from base on have to be the
 * list's own (kvfix_pages_extend makes them so).  Rows that are not moved to keep what they held.
 * path        : device int32[lists][max_path], ascending from 0 or more, base + path < len.
 * kept        : device int32[lists], each within 0..max_path.  Both NULL with max_path 0.
 */
KVFIX_API kvfix_status kvfix_pages_cut(kvfix_pool pool, int32_t page_tokens, int32_t* refs, int32_t* pages,
                                       int32_t max_pages, int32_t* len, int32_t lists, const int32_t* base,
                                       const int32_t* path, int32_t max_path, const int32_t* kept, void* stream);

/*
 * kvfix_pages_compact -- pages in use move to the front of the pool, so that what lies behind can be
 * given back or handed to others: with n pages in use, the j-th lowest of those at n and behind
 * moves to the j-th lowest free page below n (all layers, codes and scales bit for bit), refs and
 * the lists' pages follow, and *live = n.  Every list that holds a page has to be among the lists.
 * live        : device int32[1].
 * workspace   : device, kvfix_pages_compact_workspace_bytes(pool pages) bytes, 16-byte aligned.
 */
KVFIX_API size_t kvfix_pages_compact_workspace_bytes(int32_t pool_pages);
KVFIX_API kvfix_status kvfix_pages_compact(kvfix_pool pool, int32_t page_tokens, int32_t* refs, int32_t* pages,
                                           int32_t max_pages, const int32_t* len, int32_t lists, int32_t* live,
                                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * kvfix_selftest_wait -- exercise the bounded wait that every pipelined kernel uses, with
 * no hang: one warp waits on a barrier phase that never completes and then on the device
 * int32 *flag (optional; 0 = not set), each for at most limit_cycles SM clocks, and records
 * a timeout in the device status word, which kvfix_check_status reports as KVFIX_ETIMEOUT
 * (and clears).  The kernel returns in about 2 * limit_cycles clocks; the context stays
 * usable.  limit_cycles in [1, 4e9].
 */
KVFIX_API kvfix_status kvfix_selftest_wait(int64_t limit_cycles, const int32_t* flag, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KVFIX_H */
