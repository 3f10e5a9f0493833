/*
 * dsa.h -- C ABI of libdsa_gb300: the DSA decode hot path of the GLM-5.3
 * sparse layers on one GB300 (sm_103a).
 *
 * Per decode row the path is
 *   S0 dsa_latent_write    RMSNorm + FP8 quantisation + paged slot write of the
 *                          row's new latent
 *   S1 dsa_index_scores    lightning-indexer score of every visible token
 *   S2 dsa_select_topk     per-row top-k of those scores
 *   S3 dsa_mla_decode_fp8  absorbed NoPE MLA gather-attend over the selection
 * issued in that order on one stream.  Around the path, for the K-token
 * verify and the indexer's write side:
 *      dsa_dense_mm_bf16   batched projection: up to 16 rows per sweep of a
 *                          bf16 weight, each row bit-identical to a one-row call
 *      dsa_indexer_write   the indexer key's LayerNorm (with bias) and its store
 *                          at the row's device-side arena position
 * and the pool-compressed form of the selection (over caller-supplied pool
 * scores):
 *      dsa_select_pools    top pools per row under (score DESC, pool ASC)
 *      dsa_expand_selection  pools to tokens, plus the visible tail
 * and, for a batch of requests each with its own number of new tokens:
 *      dsa_plan_rows       the requests' block tables grown or shrunk from a free
 *                          list, and every row's metadata, from the lengths
 *      dsa_mla_chunk_fp8   dense causal attention of the new tokens over the paged
 *                          latent cache (no selection)
 * and the projections and the indexer over 8-bit operands with a scale for each
 * block of 128, half the bytes of their bf16 forms:
 *      dsa_quantize_fp8    bf16 or FP32 values to E4M3 codes and scales
 *      dsa_dense_mm_fp8    projection of any number of rows
 *      dsa_indexer_write_fp8  the indexer key's LayerNorm, quantised and stored
 *      dsa_index_scores_fp8   S1 over those keys
 * Sources (spark_model documentation):
 * the "glm5next_dsa/layer.rs" source page (module header: decode data flow
 * and its traps; decode_k: latent write, per-row metadata, one attend for all
 * rows; attend_rows; the selection notes on a total order) and the "Struct
 * Glm5NextDsaLayer" rustdoc page (kv_scale, decode_k).
 *
 * Conventions for every entry point
 *   - Every pointer argument is a DEVICE pointer on the current CUDA device,
 *     owned by the caller and unchanged until the work on `stream` completes.
 *     The library never allocates, frees, copies host<->device or
 *     synchronises inside these calls (so the calls can be recorded into a
 *     CUDA graph by the caller).
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls
 *     are asynchronous: a DSA_OK return means the work was enqueued.
 *   - bf16 tensors are passed as uint16_t bit patterns; FP8 as uint8_t E4M3
 *     codes (OCP: bias 7, max 448, no infinities).
 *   - Argument errors detectable on the host return DSA_ERR_INVALID_ARG or
 *     DSA_ERR_UNSUPPORTED before anything is launched.  Launch failures return
 *     DSA_ERR_CUDA.  Values only visible on the device (a seq_len above
 *     max_len, a selected index outside [0, seq_len), a negative block id, a
 *     slot outside the pool, mismatched arena bases) make the kernel skip the
 *     offending access and record the first such error in a sticky device
 *     error word that dsa_get_error() reads; kernels never trap.  Every wait
 *     inside a kernel is bounded and records DSA_DEVERR_TIMEOUT when it gives
 *     up.
 */
#ifndef DSA_GB300_H
#define DSA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DSA_ABI_VERSION 7
#define DSA_LATENT_DIM 512

typedef enum dsa_status {
    DSA_OK = 0,
    DSA_ERR_INVALID_ARG = 1,
    DSA_ERR_UNSUPPORTED = 2,
    DSA_ERR_CUDA = 3,
    DSA_ERR_DEVICE = 4,      /* dsa_get_error found a recorded device-side error */
    DSA_ERR_WORKSPACE = 5    /* workspace missing or smaller than dsa_workspace_bytes() */
} dsa_status;

/* Codes recorded in the device error word. */
enum {
    DSA_DEVERR_NONE = 0,
    DSA_DEVERR_SEQ_LEN = 1,   /* seq_len < 0 or > max_len                               */
    DSA_DEVERR_SLOT = 2,      /* latent-write slot outside [0, nslots)                  */
    DSA_DEVERR_SELECT = 3,    /* selected index outside [0, seq_len) and not -1         */
    DSA_DEVERR_BLOCK = 4,     /* block-table entry missing, negative or past the pool   */
    DSA_DEVERR_ARENA = 5,     /* idx_base invalid, or rows of one group differ in base  */
    DSA_DEVERR_POSITION = 6,  /* positions[r] != seq_lens[r]-1, or slot != table slot   */
    DSA_DEVERR_TIMEOUT = 7,   /* a bounded wait inside a kernel gave up                 */
    DSA_DEVERR_BEHIND = 8,    /* a sequence's indexer keys stop short of its length:
                                 rows were never written (lockstep with the KV cache)  */
    DSA_DEVERR_ROWS = 9,      /* a sequence's rows lie outside the row buffers          */
    DSA_DEVERR_FREE = 10      /* free list too short for the blocks wanted, or too full  */
};

/*
 * Per-row metadata of one call ("glm5next_dsa/layer.rs", decode_k: the K-row
 * attn_metadata -- positions [k] u32, slot [k] i64, seq_len [k] i32,
 * block_table [k][max_blocks_per_seq] i32 -- at stable device addresses; row r
 * reads element r of each).  All pointers are device pointers.
 */
typedef struct dsa_rows {
    const uint32_t *positions;  /* [rows] token position of the row (= seq_len-1); may be
                                   NULL.  When given, dsa_latent_write checks it against
                                   seq_lens and the table and refuses inconsistent rows. */
    const int64_t *slots;       /* [rows] paged slot of the row's new latent:
                                   block_table[pos/block_size]*block_size + pos%block_size.
                                   Read only by dsa_latent_write; may be NULL otherwise.  */
    const int32_t *seq_lens;    /* [rows] the row sees tokens [0, seq_len)               */
    const int32_t *block_table; /* row r at block_table + r*bt_stride, max_blocks_per_seq
                                   entries of physical block ids; -1 = none.             */
    int32_t max_blocks_per_seq; /* entries per table row (bounds every lookup)           */
    int32_t bt_stride;          /* elements between table rows; 0 = every row uses row 0
                                   (rows of one sequence sharing one table)              */
    int32_t block_size;         /* tokens per paged block, > 0                           */
    int32_t rows;               /* R >= 1                                                */
} dsa_rows;

/*
 * S0 -- latent write ("glm5next_dsa/layer.rs", module header trap 1 and
 * decode_k "kv path: latent -> FP8 -> paged slot"; "Struct Glm5NextDsaLayer",
 * kv_scale: the write takes 1/scale).  For each row r:
 *   y = kv_a[r] * rsqrt(mean(kv_a[r]^2) + eps) * norm_w      (vanilla: w, not 1+w)
 *   pool[slots[r]][i] = E4M3_RNE_satfinite(y[i] * fl32(1/kv_scale))
 * The norm and scaling are computed in double, with one rounding to FP8.
 *   kv_a    [rows][latent_dim] bf16      norm_w [latent_dim] bf16
 *   pool    [nslots][latent_dim] FP8, written in place at the rows' slots
 * latent_dim must be 512.  A slot outside [0, nslots) (or a row inconsistent
 * with `positions`, when given) is skipped and recorded on the device; a row of
 * slot -1 and seq_len 0, an empty one of dsa_plan_rows, is skipped without that.
 */
dsa_status dsa_latent_write(const dsa_rows *rows, const uint16_t *kv_a, const uint16_t *norm_w,
                            uint8_t *pool, int64_t nslots, int32_t latent_dim, float eps,
                            float kv_scale, void *stream);

/*
 * S1 -- lightning-indexer scores ("glm5next_dsa/layer.rs", module header:
 * q_idx, k_normed, gate and the head weights feed select_tokens; trap 3:
 * weights_proj already carries index_heads^-0.5 and the score does not scale).
 * For each row r and token t in [0, seq_lens[r]):
 *   scores[r*max_len + t] = gate[b+t] * sum_h head_w[r][h] * max(0, sum_d q_idx[r][h][d]*idx_k[b+t][d])
 * with b = idx_base[r].  Entries t >= seq_lens[r] of a scores row are not written.
 *   q_idx  [rows][index_heads][index_dim] fp32   head_w [rows][index_heads] fp32
 *   idx_k  [idx_tokens][index_dim] bf16 (key arena, all sequences)
 *   idx_gate [idx_tokens] bf16 (per-token scalar gate)
 *   idx_base [rows] int64: the row's sequence start in the arena
 *   scores [rows][max_len] fp32 (output)
 * rows_per_seq: consecutive rows that share one sequence (a K-token verify);
 * they must have equal idx_base (checked on the device) and share each key
 * tile they read, up to 64 score columns (rows x index_heads) per read.
 * rows must be a multiple of rows_per_seq.
 * idx_written (optional, may be NULL): [rows / rows_per_seq] int32, the rows
 * of each sequence's keys written so far (as kept by dsa_indexer_write); a
 * row whose seq_len exceeds its sequence's count is skipped (scores not
 * written) and recorded as DSA_DEVERR_BEHIND.
 * Supported: index_dim in {64, 128}; index_heads in [1, 256]; idx_k 16-byte
 * aligned; idx_tokens < 2^31.  Each row's result does not depend on
 * rows_per_seq or on the other rows (bit for bit).
 */
dsa_status dsa_index_scores(const dsa_rows *rows, const float *q_idx, const float *head_w,
                            const uint16_t *idx_k, const uint16_t *idx_gate, int64_t idx_tokens,
                            const int64_t *idx_base, int32_t index_heads, int32_t index_dim,
                            int32_t rows_per_seq, int32_t max_len, float *scores,
                            const int32_t *idx_written, void *stream);

/*
 * S1 with flags.  dsa_index_scores is this call with flags 0.
 * DSA_INDEX_INPUTS_BEFORE_PREDECESSOR: the caller asserts that every input of
 * the call (q_idx, head_w, idx_k, idx_gate, idx_base, idx_written and the
 * rows' seq_lens) was complete before the kernel issued just before this call
 * on the stream started -- for instance a decode step whose queries and keys
 * were produced before its latent write, or steps replayed back to back over
 * resident inputs.  The indexer may then load its inputs, run its MMAs and
 * compute its scores while that kernel still runs; its stores to `scores`
 * (which a kernel before may still read) and its completion still wait for
 * that kernel.  Do not set it when the kernel before writes an input (an
 * indexer write or a projection producing q_idx).  The results are
 * bit-identical either way.  Unknown flag bits: DSA_ERR_INVALID_ARG.
 */
#define DSA_INDEX_INPUTS_BEFORE_PREDECESSOR 1u
dsa_status dsa_index_scores_ex(const dsa_rows *rows, const float *q_idx, const float *head_w,
                               const uint16_t *idx_k, const uint16_t *idx_gate, int64_t idx_tokens,
                               const int64_t *idx_base, int32_t index_heads, int32_t index_dim,
                               int32_t rows_per_seq, int32_t max_len, float *scores,
                               const int32_t *idx_written, uint32_t flags, void *stream);

/*
 * S2 -- per-row top-k ("glm5next_dsa/layer.rs", notes on batch_select_enabled
 * and select_rows_batched: the selection is taken under the total order score
 * DESC, then index ASC, so it is unique).  For each row r, the n = min(topk,
 * seq_lens[r]) tokens of [0, seq_lens[r]) that come first under that order are
 * written to sel[r*topk + 0 .. n) in ASCENDING token order; sel[r*topk + n ..
 * topk) = -1.  -0.0 and +0.0 compare equal.  Scores must not be NaN.
 *   scores [rows][max_len] fp32 (as written by dsa_index_scores)
 *   sel    [rows][topk] int32 (output)
 * topk in [1, 65536]; max_len up to about 390k tokens (a row is held in
 * shared memory by a cluster of up to 8 CTAs).  No workspace.
 */
dsa_status dsa_select_topk(const dsa_rows *rows, const float *scores, int32_t max_len,
                           int32_t topk, int32_t *sel, void *stream);

/*
 * S3 -- absorbed NoPE MLA gather-attend over the selection
 * ("glm5next_dsa/layer.rs", module header trap 4: Q arrives absorbed into the
 * 512-d latent space; attend_rows: one launch for all rows, each with its own
 * selection row, seq_len and table row, K and V the same latent pool; decode_k:
 * slot = block*block_size + pos%block_size).  For each row r and head h, over
 * the entries j of sel[r] that are not -1:
 *   Khat_j = e4m3(pool[slot(j)]) * kv_scale
 *   z_j    = sm_scale * (q[r][h] . Khat_j)
 *   out[r][h] = sum_j softmax(z)_j * Khat_j           (bf16, latent space)
 *   lse[r][h] = log sum_j exp(z_j)                     (fp32, optional)
 * A row with nothing selected gets out = 0 and lse = -inf.
 *   q   [rows][heads][latent_dim] bf16       pool [nslots][latent_dim] FP8
 *   sel [rows][topk] int32                   out  [rows][heads][latent_dim] bf16
 * out may also be page-locked host memory mapped into the device's address
 * space (cudaHostAlloc memory under unified addressing): the kernels store the
 * result there directly, with no separate device-to-host copy.
 * latent_dim must be 512; heads a multiple of 16; nslots below 2^31
 * (DSA_ERR_UNSUPPORTED otherwise).  Numerics: q enters the tensor cores as
 * two E4M3 terms per element (hi and the residual, scaled by a power of two
 * per head), which hold a bf16 q exactly except elements more than 2^10
 * below the head's largest |q|, whose last bits fall into E4M3 subnormals;
 * their products with the E4M3 latent accumulate in FP32; the softmax weights enter the weighted sum as two E4M3 terms
 * (about bf16 precision; weights 2^18 below a head's largest drop out), the
 * normalising sums and lse use the unrounded weights.  A row's selection is
 * cut into splits of at most 256 entries (2048 with more than 64 heads; 512
 * with DSA_DECODE_LONG_SPLITS, below) whose count depends only on topk, heads
 * and that flag, so each row's result is bit-identical whatever the other
 * rows of the call are.  With more than one split each
 * split's normalised partial output O/l (a convex combination of latent
 * values, kept in fp16: 2^-11 relative) and its (max, sum) pass through the
 * workspace (L2-resident, discarded after the merge), which must hold
 * dsa_workspace_bytes(rows, heads, topk) bytes, 256-byte aligned
 * (DSA_ERR_WORKSPACE otherwise).
 */
dsa_status dsa_mla_decode_fp8(const dsa_rows *rows, const uint16_t *q, const uint8_t *pool,
                              int64_t nslots, const int32_t *sel, int32_t topk, int32_t heads,
                              int32_t latent_dim, float kv_scale, float sm_scale, uint16_t *out,
                              float *lse_or_null, void *workspace, size_t workspace_bytes,
                              void *stream);

/*
 * S3 with flags.  dsa_mla_decode_fp8 is this call with flags 0.
 * DSA_DECODE_LONG_SPLITS: with at most 64 heads, splits of at most 512
 * entries instead of 256 (half the CTAs, each twice as long: for launches
 * with many rows, whose CTAs otherwise fill the GPU in more waves; a single
 * row runs faster without it).  The split count then depends on topk, heads
 * and this flag, still never on the other rows: calls whose results must
 * agree bit for bit (a K-row verify and the same rows run one at a time) use
 * the same value of the flag.  The workspace from dsa_workspace_bytes covers
 * both plans.
 * DSA_DECODE_Q_BEFORE_PREDECESSOR: the caller asserts that q was complete
 * before the kernel issued just before this call on the stream started (the
 * usual decode order: q comes from a projection before the indexer, and the
 * kernel before the attend is dsa_select_topk, which writes only sel).  The
 * attend may then load and convert q while that kernel still runs; sel, and
 * everything else a predecessor may write, is still read after the
 * dependency wait.  Without the flag q is read after the wait too.  The
 * results are bit-identical either way.  Unknown flag bits:
 * DSA_ERR_INVALID_ARG.
 */
#define DSA_DECODE_Q_BEFORE_PREDECESSOR 1u
#define DSA_DECODE_LONG_SPLITS 2u
dsa_status dsa_mla_decode_fp8_ex(const dsa_rows *rows, const uint16_t *q, const uint8_t *pool,
                                 int64_t nslots, const int32_t *sel, int32_t topk, int32_t heads,
                                 int32_t latent_dim, float kv_scale, float sm_scale, uint16_t *out,
                                 float *lse_or_null, void *workspace, size_t workspace_bytes,
                                 uint32_t flags, void *stream);

/*
 * S3 for callers that cannot allocate device memory at the point where they
 * run the attend: code that must not take cudaMalloc's implicit device
 * synchronisation on a latency-bound decode path, and code whose device
 * memory belongs to an allocator it may not call (an embedding runtime or a
 * host framework that owns every allocation).  No counterpart on the pages:
 * it is dsa_mla_decode_fp8 with the split partials kept in a device array
 * inside the library instead of a caller workspace.  It allocates nothing and
 * calls no allocating routine.
 *   - Limit: dsa_noalloc_scratch_bytes(rows, heads, topk) must not exceed
 *     DSA_NOALLOC_SCRATCH_BYTES (32 MiB), else DSA_ERR_UNSUPPORTED and
 *     nothing is launched.  Every GPU that loads the library holds that
 *     array until the process exits.
 *   - Set-up: the first call on a device looks the array's device address up
 *     (once per device, with that device current) and keeps it for the life
 *     of the process; make that first call before any stream capture.  The
 *     address belongs to the device's primary context: after
 *     cudaDeviceReset, or under another context on the same device, it is
 *     stale and this entry point must not be used.
 *   - All calls share the one array and it keeps the last call's contents
 *     (nothing in it needs to start at zero).  Calls whose work overlaps on
 *     the GPU (other streams, other threads) race on it: serialise them.
 * Other arguments, results and errors are those of dsa_mla_decode_fp8, and
 * the results are bit-identical to that entry point's.
 */
#define DSA_NOALLOC_SCRATCH_BYTES (32u << 20)
dsa_status dsa_mla_decode_fp8_noalloc(const dsa_rows *rows, const uint16_t *q, const uint8_t *pool,
                                      int64_t nslots, const int32_t *sel, int32_t topk,
                                      int32_t heads, int32_t latent_dim, float kv_scale,
                                      float sm_scale, uint16_t *out, float *lse_or_null,
                                      void *stream);

/* Bytes of the library's array that dsa_mla_decode_fp8_noalloc needs for a
 * call of this shape (0 on bad arguments). */
size_t dsa_noalloc_scratch_bytes(int32_t rows, int32_t heads, int32_t topk);

/* Device bytes of the caller-owned workspace that dsa_mla_decode_fp8 needs
 * for a call of this shape (the gather-attend's split partials; 0 when no
 * workspace is needed or on bad arguments). */
size_t dsa_workspace_bytes(int32_t rows, int32_t heads, int32_t topk);

/*
 * Pool-compressed selection, the part the pages specify
 * ("glm5next_dsa/layer.rs", the notes above batch_select_enabled and on
 * select_rows_batched).  Tokens are grouped into pools of kp; pool p holds
 * tokens [p*kp, (p+1)*kp).  For each row r, with q_pos = positions[r]:
 *   - pool p is a candidate iff pool_valid[r*valid_stride + p] != 0 (the pool
 *     is complete) and (p+1)*kp - 1 <= q_pos (its last token is visible);
 *   - row_select_k = min(select_k, (q_pos + 1) / kp);
 *   - sel_pools[r*select_k + i], i < min(row_select_k, #candidates), are the
 *     candidates in the total order (score DESC, then pool index ASC); every
 *     other entry is -1 (a non-candidate is never selected).
 * -0.0 and +0.0 compare equal; scores must not be NaN.  Only pools below
 * (q_pos+1)/kp are read, so a row's result does not depend on max_pools or
 * on the other rows.  How the pool scores are made (the pages' gate [D] and
 * ape [kp][D] compression of the pool's keys) is not on the pages: the caller
 * supplies them.
 *   pool_scores [rows][max_pools] fp32          pool_valid [rows or 1][...] u8
 *   valid_stride: elements between rows of pool_valid, 0 = one shared row
 *   sel_pools   [rows][select_k] int32 (output)
 * rows->positions is required.  kp, select_k >= 1; max_pools in
 * [1, DSA_MAX_POOLS] (DSA_ERR_UNSUPPORTED above).
 */
#define DSA_MAX_POOLS 16384
dsa_status dsa_select_pools(const dsa_rows *rows, const float *pool_scores, int32_t max_pools,
                            const uint8_t *pool_valid, int32_t valid_stride, int32_t kp,
                            int32_t select_k, int32_t *sel_pools, void *stream);

/*
 * Expansion of a pool selection to token indices (same source: the
 * expansion writes the pools' tokens, then the visible tail at
 * row_select_k * kp; the per-row row_select_k applies to both).  For each row
 * r, with q_pos = positions[r] and row_select_k as above:
 *   sel_tokens[r*out_width + i*kp + j] = sel_pools[r*select_k + i]*kp + j
 *       for i < row_select_k, j < kp (-1 where the pool entry is -1);
 *   then the tokens floor((q_pos+1)/kp)*kp .. q_pos (the part of the
 *   incomplete pool the row sees) from entry row_select_k*kp on;
 *   every other entry of the row is -1.
 * The result is a selection row for dsa_mla_decode_fp8 (which skips -1).
 * out_width >= select_k*kp + kp - 1 (room for the longest tail), else
 * DSA_ERR_INVALID_ARG.  rows->positions is required.
 */
dsa_status dsa_expand_selection(const dsa_rows *rows, const int32_t *sel_pools, int32_t kp,
                                int32_t select_k, int32_t *sel_tokens, int32_t out_width,
                                void *stream);

/*
 * Indexer write side for each row's new token ("glm5next_dsa/layer.rs",
 * module header trap 2: indexer.k_norm is an nn.LayerNorm with a bias;
 * indexer_forward: the wk projection of the token lands in the key cache row,
 * normalised in place, the row placed from a DEVICE-side position so that a
 * captured graph replays at the next position).  For each row r, at arena
 * row t = idx_base[r] + positions[r]:
 *   mu = mean_d k_raw[r][d],   var = mean_d (k_raw[r][d] - mu)^2
 *   idx_k[t][d] = bf16_rne((k_raw[r][d] - mu) / sqrt(var + eps) * ln_w[d] + ln_b[d])
 *   idx_gate[t] = gate[r]                                (when gate != NULL)
 *   k_raw [rows][index_dim] bf16 (the wk projection, e.g. from
 *         dsa_dense_mm_bf16), 8-byte aligned
 *   ln_w, ln_b [index_dim] bf16     gate [rows] bf16 or NULL
 *   idx_k [idx_tokens][index_dim] bf16, 8-byte aligned; idx_gate [idx_tokens]
 * rows->positions is required (the new token of row r is position
 * seq_lens[r]-1).  index_dim 64 or 128 (DSA_ERR_UNSUPPORTED otherwise).
 * Numerics: mean, variance and the affine map in double, one rounding to
 * bf16 (nearest, ties to even).  A row whose position is not seq_lens[r]-1
 * (DSA_DEVERR_POSITION) or whose arena row lies outside [0, idx_tokens)
 * (DSA_DEVERR_ARENA) is skipped and recorded.
 * Lockstep with the KV cache ("glm5next_dsa/layer.rs", decode_k: the indexer
 * cache must hold exactly the sequence's tokens before the step; more is the
 * leftover of a rejected verify and is rewound, fewer means rows were never
 * written and is an error), when idx_written is given ([rows / rows_per_seq]
 * int32, one count per sequence of rows_per_seq consecutive rows, which must
 * have the consecutive positions p0, p0+1, ...): a sequence whose count is
 * below p0 is not written and is recorded as DSA_DEVERR_BEHIND; otherwise
 * its rows are written and its count becomes p0 + rows_per_seq (a count
 * above p0 is rewound).  rows_per_seq in [1, 32] and dividing rows when
 * idx_written is given (ignored otherwise).
 */
dsa_status dsa_indexer_write(const dsa_rows *rows, const uint16_t *k_raw, const uint16_t *ln_w,
                             const uint16_t *ln_b, float eps, const uint16_t *gate,
                             const int64_t *idx_base, uint16_t *idx_k, uint16_t *idx_gate,
                             int64_t idx_tokens, int32_t index_dim, int32_t *idx_written,
                             int32_t rows_per_seq, void *stream);

/*
 * Batched projection for the K-token verify: the K rows of one sequence sweep
 * a BF16 weight once ("glm5next_dsa/layer.rs": the gemm helper,
 * C[M, N] = A[M, K] @ B[N, K]^T, and the decode_k notes on
 * dense_gemv_bf16_batchm -- one weight read for 2..16 rows, each row
 * bit-identical to a single-row call).
 *   c[m][n] = sum_k a[m][k] * b[n][k]          m < m_rows, n < n_out
 *   a [m_rows][k] bf16, row-major (k contiguous), 16-byte aligned
 *   b [n_out][k]  bf16 weight, row-major, 16-byte aligned
 *   c [m_rows][n_out] bf16 (c_fp32 = 0, round to nearest even) or fp32
 *     (c_fp32 = 1), 4-byte aligned
 * m_rows in [1, 16] (DSA_ERR_UNSUPPORTED above); k >= 8 and a multiple of 8
 * (16-byte row strides); n_out >= 1; DSA_ERR_INVALID_ARG otherwise.
 * Numerics: the bf16 products are exact and accumulate in FP32 on the tensor
 * cores in 64-element blocks of k, in order; when the weight has few rows the
 * k range is split (the split depends only on n_out, k and the device's SM
 * count) and the FP32 partial sums are added in order.  A row's result is a
 * function of that row of a and of b only: bit-identical whatever m_rows is
 * and whatever the other rows hold.  The split partials pass through the
 * caller's workspace of dsa_dense_mm_workspace_bytes(n_out, k) bytes (0: none
 * needed), 256-byte aligned (DSA_ERR_WORKSPACE otherwise).
 */
dsa_status dsa_dense_mm_bf16(const uint16_t *a, const uint16_t *b, void *c, int32_t m_rows,
                             int32_t n_out, int32_t k, int32_t c_fp32, void *workspace,
                             size_t workspace_bytes, void *stream);

/* The number of k ranges dsa_dense_mm_bf16 splits an n_out x k weight into on
 * a device with num_sms SMs (host arithmetic only; 0 on bad arguments).  One
 * range when the 128-row weight tiles alone reach num_sms, else enough ranges
 * to, each at least four 64-element blocks of k long. */
int32_t dsa_dense_mm_splits(int32_t n_out, int32_t k, int32_t num_sms);

/* Workspace bytes dsa_dense_mm_bf16 needs on the current device for a weight
 * of n_out x k (0 when it needs none or on bad arguments). */
size_t dsa_dense_mm_workspace_bytes(int32_t n_out, int32_t k);

/*
 * 8-bit operands with a scale for each block of 128 along k: the codes and
 * scales that dsa_dense_mm_fp8 and dsa_index_scores_fp8 take.  No counterpart on
 * the pages, whose projections and indexer keys are bf16: half the bytes.  For
 * each block of k [128 j, 128 j + 128) of one row (block_rows = 1: activations,
 * queries) or of 128 consecutive rows (block_rows = 128: weights), the last ones
 * of a row or of the tensor shorter:
 *   scale = the smallest power of two, 2^-126 at least, with max |x| <= 448 scale
 *           (the maximum over the block's finite elements)
 *   code  = E4M3_RNE(x / scale)         (x / scale is exact: one rounding)
 * An infinity becomes +-448, a NaN the code 0x7F.  A power of two costs E4M3 no
 * precision against max / 448.
 *   x      [rows][k] bf16 (x_fp32 = 0) or fp32 (1), 16-byte aligned
 *   codes  [rows][k] E4M3, 16-byte aligned, not overlapping x
 *   scales [ceil(rows / block_rows)][ceil(k / 128)] fp32
 * rows >= 1; k >= 16 and a multiple of 16; rows * ceil(k / 128) < 2^31, and with
 * block_rows = 128 rows <= 65535 * 128 (DSA_ERR_UNSUPPORTED).
 */
dsa_status dsa_quantize_fp8(const void *x, int32_t x_fp32, int32_t rows, int32_t k,
                            int32_t block_rows, uint8_t *codes, float *scales, void *stream);

/*
 * Matrix product of 8-bit operands with a scale for each block of 128, from one
 * token to a prompt's chunk (the FP8 form of dsa_dense_mm_bf16; "glm5next_dsa/
 * layer.rs", the gemm helper, C[M, N] = A[M, K] @ B[N, K]^T):
 *   c[m][n] = sum_j a_scale[m][j] * b_scale[n / 128][j]
 *                   * sum_{k in block j} e4m3(a[m][k]) * e4m3(b[n][k])
 *   a [m_rows][k] E4M3, row-major, 16-byte aligned
 *   a_scale [m_rows][ceil(k / 128)] fp32          (dsa_quantize_fp8, block_rows 1)
 *   b [n_out][k] E4M3 weight, row-major, 16-byte aligned
 *   b_scale [ceil(n_out / 128)][ceil(k / 128)] fp32  (block_rows 128, or a
 *           checkpoint's: the scales may be any fp32 values)
 *   c [m_rows][n_out] bf16 (c_fp32 = 0, round to nearest even) or fp32
 *     (c_fp32 = 1), 16-byte aligned, not overlapping an input
 * m_rows in [1, 65535] and n_out up to 65535 * 128 (DSA_ERR_UNSUPPORTED above);
 * k >= 16 and a multiple of 16 (DSA_ERR_INVALID_ARG).  No workspace.  Any
 * operand may be the output of the kernel just before (unlike dsa_dense_mm_bf16's
 * weight).
 * Numerics: a block's products are exact and accumulate in FP32 on the tensor
 * cores; each block's sum is multiplied by the product of its two scales
 * (rounded to FP32) and added in FP32, blocks in order, within each of the
 * ranges that k is split into when the output has few tiles; the ranges are then
 * added in order.  A NaN code makes the results that it enters NaN.  With
 * m_rows <= 64 a row's result is bit-identical whatever m_rows is and whatever
 * the other rows hold.  After a wait that gave up (DSA_DEVERR_TIMEOUT) c holds
 * nothing to rely on.
 */
dsa_status dsa_dense_mm_fp8(const uint8_t *a, const float *a_scale, const uint8_t *b,
                            const float *b_scale, void *c, int32_t m_rows, int32_t n_out, int32_t k,
                            int32_t c_fp32, void *stream);

/*
 * Indexer write side into an FP8 key cache (dsa_indexer_write, quantised as it is
 * written): with t = idx_base[r] + positions[r] and y the LayerNorm (with bias)
 * of k_raw[r] as there, in double and not rounded to bf16,
 *   idx_scale[t] = the smallest power of two, 2^-126 at least, with
 *                  max_d |y[d]| <= 448 idx_scale[t]  (over the finite y)
 *   idx_k[t][d]  = E4M3_RNE(y[d] / idx_scale[t])
 *   idx_gate[t]  = gate[r]                          (when gate != NULL)
 *   k_raw [rows][index_dim] bf16, ln_w, ln_b [index_dim] bf16, 8-byte aligned
 *   idx_k [idx_tokens][index_dim] E4M3, 4-byte aligned; idx_scale [idx_tokens] fp32;
 *   idx_gate [idx_tokens] bf16; gate [rows] bf16 or NULL
 * rows->positions is required; index_dim 64 or 128 (DSA_ERR_UNSUPPORTED otherwise).
 * A row whose y is not finite has codes 0x7F or +-448 there.  Rows must not share
 * an arena row.  Without idx_written each row stands for itself; with it the rows
 * of a sequence (rows_per_seq consecutive ones, at most 32) are written together
 * or not at all: not if one has not position seq_lens[r] - 1 or does not follow
 * the one before (DSA_DEVERR_POSITION), lies outside [0, idx_tokens)
 * (DSA_DEVERR_ARENA), or if the sequence's count is below its first position
 * (DSA_DEVERR_BEHIND); if written, the count becomes the last position + 1 (more
 * is the leftover of a rejected verify and is rewound).  An empty row of
 * dsa_plan_rows (position 0, seq_len 0) is skipped without a record, a sequence of
 * such rows keeps its count, and one that mixes them with others is refused
 * (DSA_DEVERR_POSITION).
 */
dsa_status dsa_indexer_write_fp8(const dsa_rows *rows, const uint16_t *k_raw, const uint16_t *ln_w,
                                 const uint16_t *ln_b, float eps, const uint16_t *gate,
                                 const int64_t *idx_base, uint8_t *idx_k, float *idx_scale,
                                 uint16_t *idx_gate, int64_t idx_tokens, int32_t index_dim,
                                 int32_t *idx_written, int32_t rows_per_seq, void *stream);

/*
 * Index scores over that cache (dsa_index_scores with 8-bit keys and queries: half
 * the bytes a key).  For each row r and token t in [0, seq_lens[r]), b = idx_base[r]:
 *   scores[r*max_len + t] = idx_gate[b+t] * idx_scale[b+t]
 *       * sum_h (head_w[r][h] * q_scale[r][h]) * max(0, sum_d e4m3(q[r][h][d]) * e4m3(idx_k[b+t][d]))
 *   q [rows][index_heads][index_dim] E4M3 and q_scale [rows][index_heads] fp32
 *     (dsa_quantize_fp8 of [rows * index_heads][index_dim] queries)
 *   idx_k [idx_tokens][index_dim] E4M3, idx_scale [idx_tokens] fp32 (any values)
 *   idx_gate [idx_tokens] bf16, or NULL: 1
 * The other arguments, the shapes supported, flags (DSA_INDEX_INPUTS_BEFORE_PREDECESSOR
 * or 0), what is checked on the device and the errors recorded are those of
 * dsa_index_scores_ex; q and idx_k are 16-byte aligned.  max(0, NaN) is 0: a NaN
 * code takes its head out of the sum.
 * Numerics: the products are exact and accumulate in FP32 on the tensor cores; the
 * heads are added in FP32, every fourth one in order into one of four sums, and
 * (s0 + s1) + (s2 + s3) is multiplied by the product of gate and scale.  Each row's
 * result does not depend on rows_per_seq or on the other rows (bit for bit).
 */
dsa_status dsa_index_scores_fp8(const dsa_rows *rows, const uint8_t *q, const float *q_scale,
                                const float *head_w, const uint8_t *idx_k, const float *idx_scale,
                                const uint16_t *idx_gate, int64_t idx_tokens, const int64_t *idx_base,
                                int32_t index_heads, int32_t index_dim, int32_t rows_per_seq,
                                int32_t max_len, float *scores, const int32_t *idx_written,
                                uint32_t flags, void *stream);

/*
 * Row plan of a batch of requests: block tables grown and shrunk from a free
 * list, and the per-row metadata of the step (dsa_rows: positions, slots,
 * seq_lens, block_table; "glm5next_dsa/layer.rs", decode_k, the K-row
 * attn_metadata), built on the device from the requests' lengths.  The pages
 * take the tables from their host scheduler; this is the same step for
 * callers whose lengths are device data.
 * Request s has L = seq_lens[s] tokens once the step's n = new_tokens[s] new
 * ones are counted, and holds h = held_in[s] blocks, the first h entries of
 * its table row.  need = ceil(L / block_size).
 *   - need < h (a finished request, L = 0, or a rejected verify's tokens): its
 *     entries need .. h-1 go back to the free list, in order, requests in
 *     order.  The table keeps the stale ids there.
 *   - need > h: entries h .. need-1 are taken from the free list.
 * The free list is a stack: free_blocks[0 .. F), F = free_in[0].  The blocks
 * given back (Rtot of them) are pushed first, then requests in order pop theirs
 * from the top.  A request is refused when the blocks wanted up to and
 * including its own exceed F + Rtot: the blocks it wanted become -1 in its
 * table, it keeps h blocks, its rows are empty, and DSA_DEVERR_FREE is recorded.
 *   held_out[s] = need (h if refused), free_out[0] = blocks left on the stack,
 *   served_lens[s] = L (0 if refused or invalid), the seq_lens to give to
 *   dsa_mla_chunk_fp8: the new tokens of a refused request have no latents, and those
 *   that fall into its last block would be read as what that block held before.
 * Rows: request s owns rows row_start[s] .. row_start[s+1]-1, n of them; its
 * row i has
 *   positions = L-n+i, seq_lens = positions+1, row_seq = s,
 *   slots = table[positions / block_size] * block_size + positions % block_size,
 *   block_table row = the request's need blocks, then -1 up to max_blocks_per_seq
 * An empty row has position 0, seq_len 0, slot -1 and a table row of -1.  Rows
 * from row_start[seqs] on are left as they were, slots of an earlier step
 * among them: calls that write by row (dsa_latent_write) are given the rows before
 * it, which whoever packs their inputs knows to be the sum of new_tokens.  With
 * DSA_PLAN_EMPTY_TAIL they are made empty rows (row_seq -1) up to `rows`, so that a
 * step captured over all rows of its buffers serves any number of new tokens:
 * dsa_latent_write skips them and dsa_mla_chunk_fp8 leaves theirs as they were.
 * A request with n outside [0, min(L, rows)], need > max_blocks_per_seq or h
 * outside [0, max_blocks_per_seq] is recorded (DSA_DEVERR_SEQ_LEN, with s as
 * the row) and changes nothing; its n rows, if 0 <= n <= rows, are empty.
 * Rows past `rows` are not written (DSA_DEVERR_ROWS).  F outside [0,
 * free_capacity] is recorded (DSA_DEVERR_FREE) and counts as 0; blocks that
 * would not fit free_capacity are dropped (DSA_DEVERR_FREE).
 * held_out may be held_in and free_out may be free_in (the state is then kept
 * in place and the call can be captured and replayed); they must not overlap
 * otherwise.  With separate buffers a repeated call gives the same result.
 * free_out[1] must be 0 before the first call and is 0 after each; calls that
 * share a state or output buffer must not overlap on the GPU.
 * Limits: seqs <= DSA_PLAN_MAX_SEQS, rows <= 65535, seqs *
 * max_blocks_per_seq, block_size * max_blocks_per_seq < 2^31
 * (DSA_ERR_UNSUPPORTED).
 */
#define DSA_PLAN_MAX_SEQS 8192
#define DSA_PLAN_EMPTY_TAIL 1u
typedef struct dsa_plan {
    const int32_t *seq_lens;     /* [seqs] tokens, the new ones included                */
    const int32_t *new_tokens;   /* [seqs] rows wanted                                   */
    const int32_t *held_in;      /* [seqs] blocks held before                            */
    int32_t *held_out;           /* [seqs] blocks held after                             */
    int32_t *block_table;        /* request s at block_table + s*bt_stride (in place)    */
    int32_t *free_blocks;        /* [free_capacity] stack of free block ids (in place)   */
    const int32_t *free_in;      /* [1] ids on the stack before                          */
    int32_t *free_out;           /* [2] ids on the stack after, and a word kept at 0     */
    int32_t *row_start;          /* [seqs + 1] out                                       */
    uint32_t *positions;         /* [rows] out                                           */
    int64_t *slots;              /* [rows] out                                           */
    int32_t *row_lens;           /* [rows] out: seq_lens of the rows                     */
    int32_t *row_table;          /* row r at row_table + r*row_bt_stride, out; may be NULL */
    int32_t *row_seq;            /* [rows] out; may be NULL                              */
    int32_t seqs;
    int32_t rows;                /* rows the row buffers hold                            */
    int32_t max_blocks_per_seq;  /* entries of a table row                               */
    int32_t bt_stride;           /* elements between the requests' table rows            */
    int32_t row_bt_stride;       /* elements between the rows' table rows                */
    int32_t block_size;
    int32_t free_capacity;
    int32_t reserved;            /* 0                                                    */
    int32_t *served_lens;        /* [seqs] out; may be NULL                              */
    uint32_t flags;              /* DSA_PLAN_*; unknown bits are DSA_ERR_INVALID_ARG     */
    int32_t reserved2;           /* 0                                                    */
} dsa_plan;
dsa_status dsa_plan_rows(const dsa_plan *plan, void *stream);

/*
 * Per-request metadata of dsa_mla_chunk_fp8, all device pointers (as written
 * by dsa_plan_rows, seq_lens its served_lens, or by the caller).  Request s has
 * seq_lens[s] tokens in the cache; its new ones, the last row_start[s+1] -
 * row_start[s] of them, are the rows row_start[s] .. row_start[s+1]-1 of q and out.
 */
typedef struct dsa_seqs {
    const int32_t *seq_lens;     /* [seqs]                                               */
    const int32_t *row_start;    /* [seqs + 1], not decreasing                           */
    const int32_t *block_table;  /* request s at block_table + s*bt_stride               */
    int32_t max_blocks_per_seq;
    int32_t bt_stride;           /* >= max_blocks_per_seq                                */
    int32_t block_size;          /* > 0                                                  */
    int32_t seqs;                /* >= 1                                                 */
} dsa_seqs;

/*
 * Attention of each request's new tokens over its paged latent cache: dense
 * and causal, absorbed NoPE MLA as in dsa_mla_decode_fp8 ("glm5next_dsa/
 * layer.rs", module header trap 4 and decode_k: K and V are the same latent
 * pool, slot = block*block_size + pos%block_size), which it equals when that
 * call's selection holds every visible token.  Row i of request s (n rows, L =
 * seq_lens[s]) and head h, over the tokens j < L - n + i + 1:
 *   Khat_j = e4m3(pool[slot(j)]) * kv_scale
 *   z_j    = sm_scale * (q[row][h] . Khat_j)
 *   out[row][h] = sum_j softmax(z)_j * Khat_j        (bf16, latent space)
 *   lse[row][h] = log sum_j exp(z_j)                  (fp32, optional)
 * The latents of the new tokens are written first (dsa_latent_write).  A token
 * whose block is missing (negative, or past the pool) is left out and recorded
 * (DSA_DEVERR_BLOCK); a row that sees no token gets out = 0 and lse = -inf.  What
 * the pool holds at tokens a row does not see, NaN codes included, never
 * reaches the row.  A request whose rows lie outside [0, rows)
 * (DSA_DEVERR_ROWS), or with rows and 0 != seq_lens[s] < n or above
 * max_blocks_per_seq * block_size (DSA_DEVERR_SEQ_LEN), is skipped, its rows
 * left as they were (the recorded row is s).  A request with rows and seq_lens[s]
 * = 0 (one that dsa_plan_rows left empty, by its served_lens) has nothing to see:
 * its rows get out = 0 and lse = -inf.  Rows of no request are left as they were.  After a wait that gave up (DSA_DEVERR_TIMEOUT, row -1) the call's
 * rows hold nothing to rely on.
 *   q   [rows][heads][latent_dim] bf16       pool [nslots][latent_dim] FP8
 *   out [rows][heads][latent_dim] bf16       lse  [rows][heads] fp32 or NULL
 * Numerics: the latents enter the FP8 tensor cores as they are; q as two E4M3
 * terms an element (as in dsa_mla_decode_fp8), a softmax weight as an E4M3 term
 * and the E5M2 term of its remainder: within 2^-7 of the weight, about 2^-9.6
 * rms, down to 2^-14 of the line's largest.  A smaller one is within 2^-21 of the
 * largest or a quarter of itself, whichever is less (but 2^-24 of the largest is
 * the smallest step), rounded up or down by the token's place: the sum over many
 * like weights is right to 2^-7 down to 2^-24 of the largest.  Logits, sums, maxima
 * and the output are FP32, lse uses the unrounded weights.  The tokens are shared out
 * among the SMs by the lengths of the whole call and partial results merged in
 * order: the same call gives the same bits, but a row's last bits may differ
 * beside other rows.
 * latent_dim must be 512; heads a multiple of 16 up to 4096; rows <= 65535;
 * seqs <= DSA_PLAN_MAX_SEQS; nslots below 2^31; block_size *
 * max_blocks_per_seq at most 2^30 (DSA_ERR_UNSUPPORTED otherwise).  q, pool and
 * out 16-byte aligned; out must not overlap q or the pool.  The workspace holds
 * dsa_chunk_workspace_bytes(rows, heads) bytes, 256-byte aligned
 * (DSA_ERR_WORKSPACE otherwise), needs no initial value, and belongs to the call
 * until its work completes: calls that may overlap on the GPU (other streams,
 * two captured graphs) need one each.
 */
dsa_status dsa_mla_chunk_fp8(const dsa_seqs *seqs, const uint16_t *q, const uint8_t *pool,
                             int64_t nslots, int32_t rows, int32_t heads, int32_t latent_dim,
                             float kv_scale, float sm_scale, uint16_t *out, float *lse_or_null,
                             void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of dsa_mla_chunk_fp8 on the current device (0 on bad
 * arguments). */
size_t dsa_chunk_workspace_bytes(int32_t rows, int32_t heads);

/*
 * Read the sticky device error word of the current device: *code_out is the
 * first DSA_DEVERR_* recorded since the last reset (0 if none), *row_out the
 * row it concerned and *count_out how many errors were recorded.  Any out
 * pointer may be NULL.  This call synchronises the device.  reset != 0 clears
 * the word.  Returns DSA_ERR_DEVICE when an error was recorded, else DSA_OK
 * (or DSA_ERR_CUDA).
 */
dsa_status dsa_get_error(int32_t *code_out, int32_t *row_out, int32_t *count_out, int32_t reset);

/* Block-table entries the paged gather can index for k rows starting at
 * seq_len, plus one of slack: (seq_len + k) / block_size + 2, a block size of
 * 0 counted as 1 ("glm5next_dsa/layer.rs", bt_entries_needed). */
int64_t dsa_bt_entries_needed(int64_t seq_len, int64_t k, int64_t block_size);

/*
 * Limit, in nanoseconds of wall time, on every pipeline wait inside the
 * kernels launched after this call (0 restores the default, 500 ms; the time that
 * the kernel before still runs does not count).  A wait
 * that runs out records DSA_DEVERR_TIMEOUT, the CTA stops its pipeline and
 * its results are zero; the CTA still waits for its own copies and MMAs in
 * flight (that drain keeps its own 500 ms limit) before it exits, so a short
 * limit never leaves work running behind the call.  Meant for tests of the
 * timeout path and for callers that prefer an early error to a long stall;
 * process-wide.  No counterpart on the pages.
 */
dsa_status dsa_set_wait_limit_ns(uint64_t limit_ns);
uint64_t dsa_get_wait_limit_ns(void);

/* Static text for a status code. */
const char *dsa_status_string(dsa_status status);

/* DSA_ABI_VERSION of the loaded library. */
int32_t dsa_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DSA_GB300_H */
