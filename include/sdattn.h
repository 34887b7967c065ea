/*
 * sdattn.h - C ABI of the GB300 (sm_103a) DSA sparse decode attention library.
 *
 * The operation is the one of the vLLM API page
 * "vllm.models.step5.nvidia.ops.sparse_decode_attention" (function
 * `sparse_decode_attention` and its module docstring): for every
 * (token, KV group) row, all query heads of that group attend over only the
 * row's selected KV regions, read in place from a paged cache through
 * block_table, with FP8 dequantised, tokens past the row's position masked,
 * split-KV partials merged through their log-sum-exp, an optional headwise
 * sigmoid gate applied with bf16 rounding (the page's `_gate`), and inactive
 * rows cleared.
 *
 * Conventions for every entry point:
 *   - Pointers inside `sda_tensor` are DEVICE pointers of the current CUDA
 *     device; shapes and strides are in elements (not bytes).
 *   - The caller owns every buffer.  The library allocates no device memory,
 *     never synchronises the stream (except sparse_decode_read_errors) and
 *     returns a status instead of aborting.  A launch is asynchronous: results
 *     are valid once the stream has reached that point.
 *   - Inputs are read only; only `output` and `workspace` are written, and
 *     neither may overlap an input.
 *   - Host threads may call at the same time.  On one stream they may also pass
 *     the same workspace: the launches of a call stay together.
 */
#ifndef SDATTN_H
#define SDATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SDA_OK = 0,
    SDA_ERR_INVALID = 1,      /* an argument breaks the documented contract            */
    SDA_ERR_UNSUPPORTED = 2,  /* well formed, but outside what the kernels handle      */
    SDA_ERR_WORKSPACE = 3,    /* workspace missing, misaligned or too small            */
    SDA_ERR_CUDA = 4,         /* a CUDA runtime or driver call failed                  */
    SDA_ERR_TIMEOUT = 5,      /* device flag: a bounded wait inside a kernel gave up   */
    SDA_ERR_BOUNDS = 6        /* device flag: an index read from the inputs was bad    */
} sda_status;

typedef enum {
    SDA_DTYPE_BF16 = 1,
    SDA_DTYPE_FP8_E4M3 = 2,   /* OCP E4M3 "fn" (finite, bias 7)                        */
    SDA_DTYPE_UINT8 = 3,      /* raw bytes; an FP8 cache may be passed as uint8        */
    SDA_DTYPE_INT32 = 4,
    SDA_DTYPE_BOOL = 5,       /* one byte, nonzero = true                              */
    SDA_DTYPE_FP32 = 6,
    SDA_DTYPE_INT64 = 7
} sda_dtype;

/* A strided view of device memory.  Unused trailing shape/stride entries are
 * ignored.  `data` may be NULL only where an argument is documented optional. */
typedef struct {
    const void *data;
    int32_t dtype;            /* sda_dtype */
    int32_t ndim;
    int64_t shape[4];
    int64_t stride[4];        /* in elements */
} sda_tensor;

/* Device error flags accumulated in the workspace header (bit values). */
#define SDA_FLAG_BOUNDS  0x1u  /* a region id < -1, a table column past the table width, or a
                                  table entry outside [0, pages) was met; that piece was skipped */
#define SDA_FLAG_TIMEOUT 0x2u  /* a pipeline wait exceeded its limit; the row's output is invalid */
#define SDA_FLAG_FULL    0x4u  /* sparse_decode_plan_step: free pages or token rows ran out, some
                                  requests got nothing this step */

/*
 * Split count per row: start at 1 and double while below 32 and
 * rows * splits * 2 <= 256, i.e. about 256 split programs per call.
 * Follows `sparse_decode_splits` on the page named above (the split cannot
 * follow context length because CUDA graphs are captured per batch size).
 * rows < 0 returns 1.
 */
int sparse_decode_splits(int rows);

/*
 * Bytes of workspace `sparse_decode_attention` needs for `rows` rows of
 * `heads` heads with `splits` splits: a 256-byte header (device error flags)
 * plus, when splits > 1, fp32 partial outputs [rows*splits*heads, 192] and
 * fp32 log-sum-exps [rows*splits*heads] (the page's `partial` and `lse`).
 * Returns 0 for arguments out of range.
 */
size_t sparse_decode_workspace_bytes(int rows, int heads, int splits);

/*
 * Sparse decode attention (page above, function `sparse_decode_attention`).
 *
 *   query        [rows, H, 192] bf16, stride[2] == 1, H in 1..16.
 *                rows = tokens * G; row r is KV group r % G of token r / G.
 *   cache        [pages, G, B, 384] bf16, FP8_E4M3 or UINT8 (E4M3 bytes);
 *                K in elements 0..191 and V in 192..383 of a token's row.
 *                stride[3] == 1; any page / group / token strides whose byte
 *                sizes are multiples of 16 (and a 16-byte aligned base).
 *   regions      [rows, R] int32, stride[1] == 1, R <= 16384 (else
 *                SDA_ERR_UNSUPPORTED).  Region ids of the row, any order; -1
 *                marks an unused slot.  Id `id` covers the request's logical
 *                tokens [id*RT, (id+1)*RT), RT = region_tokens.
 *   block_table  [requests, W] int32, stride[1] == 1.  Logical block c of
 *                request q lives in page block_table[q, c].  The G*query_len
 *                consecutive rows of one request share its table row:
 *                request = r / (G * query_len).
 *   positions    [rows] int32: the row's token position (0-based); a token t
 *                is visible iff t <= position.
 *   active       [rows] BOOL or UINT8: zero rows are not computed; with
 *                clear_inactive their output is written as +0.0.
 *   output       [rows, H, 192] bf16, stride[2] == 1 (written).
 *   scale        softmax scale applied to q.k (e.g. 1/sqrt(192)).
 *   query_len    tokens per request (>= 1).
 *   splits       split-KV programs per row, 1..64 (see sparse_decode_splits).
 *                Each split takes a contiguous chunk [s*n/S, (s+1)*n/S) of the
 *                row's live regions; splits > 1 adds the combine kernel.
 *   k_scale, v_scale  device fp32 scalars; required for an FP8 cache, ignored
 *                for bf16.  K = decode(byte) * k_scale, V = decode(byte) * v_scale.
 *   gate         NULL (or data == NULL) for no gate, else [tokens, G*H] bf16:
 *                head h of row r is multiplied by bf16(sigmoid(gate[r/G,
 *                (r%G)*H + h])) computed in fp32 (the page's `_gate`).
 *   clear_inactive  nonzero: inactive rows are written as +0.0; zero: left as is.
 *                (The adapter page's decode path passes clear_inactive || gate,
 *                so gated layers always clear; that policy is the caller's.)
 *   region_tokens   RT; 0 means RT = B.  min(RT, B, 64) must be a multiple of 8
 *                and divide both RT and B.
 *   workspace    device buffer of >= sparse_decode_workspace_bytes(rows, H,
 *                splits) bytes, 256-byte aligned; its first 4 bytes are error
 *                flags the kernels OR into (zero them once before first use;
 *                see sparse_decode_read_errors).  Calls that overlap on the
 *                GPU must not share a workspace.
 *   stream       cudaStream_t (NULL = legacy default stream).
 *
 * Returns SDA_OK after enqueueing the kernels (rows == 0 enqueues nothing),
 * SDA_ERR_INVALID / SDA_ERR_UNSUPPORTED / SDA_ERR_WORKSPACE without touching
 * the GPU, or SDA_ERR_CUDA when a launch failed.  Device-side problems are
 * reported through the workspace flags, never by a trap.
 *
 * FP8 note: the kernels convert E4M3 to fp16 exactly; the two NaN codes
 * (S.1111.111) are not meaningful cache contents and are not special-cased.
 * The FP8 path multiplies in fp16: each row's q is first scaled by a power of
 * two that puts its largest |q| in [2^14, 2^15), and the factor is undone in
 * the fp32 logit scale, so any finite bf16 query is taken at full precision
 * (values more than 2^31 below the row's largest lose low bits) as long as
 * the logits scale * q.k * k_scale fit in fp32.
 */
sda_status sparse_decode_attention(const sda_tensor *query, const sda_tensor *cache,
                                   const sda_tensor *regions, const sda_tensor *block_table,
                                   const sda_tensor *positions, const sda_tensor *active,
                                   const sda_tensor *output, float scale, int query_len,
                                   int splits, const float *k_scale, const float *v_scale,
                                   const sda_tensor *gate, int clear_inactive, int region_tokens,
                                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * Split count for the sliding-window decode below (a reading of its own: the
 * page's `swa_decode_plan` body is not shown).  Starts from
 * sparse_decode_splits(rows) and halves while a split would cover fewer than
 * 256 window tokens.
 */
int sparse_decode_swa_splits(int rows, int window);

/*
 * Gated sliding-window decode over the same packed cache: the non-DSA layers'
 * fused path of the vLLM page "vllm.models.step5.nvidia.sparse_attention"
 * (`Step5SplitKVFlashAttentionImpl.forward_with_headwise_gate`, which calls
 * `swa_decode_gated` with window = sliding_window[0] + 1, GQA packing and a
 * split window, bf16, query_len <= 4 there).
 *
 *   query, cache, block_table, output, scale, query_len, splits, k_scale,
 *   v_scale, gate, workspace, stream: as in sparse_decode_attention
 *                (rows = tokens * G; FP8 caches are accepted as well).
 *   seq_lens     [requests] int32: tokens of each request including the ones
 *                being decoded.  Token j of request q sits at position
 *                p = seq_lens[q] - query_len + j and attends over the `window`
 *                tokens [max(0, p - window + 1), p] of its request (none when
 *                p < 0: zeros).
 *   window       >= 1 (at most 2^30).
 * Every row is active.  The window is walked in pieces of min(B, 64) (FP8) or
 * min(B, 32) (bf16) tokens, which must be a multiple of 8 dividing B.  Splits
 * take contiguous chunks of the window's pieces.  Errors as for
 * sparse_decode_attention.
 */
sda_status sparse_decode_swa_attention(const sda_tensor *query, const sda_tensor *cache,
                                       const sda_tensor *block_table, const sda_tensor *seq_lens,
                                       const sda_tensor *output, float scale, int window, int query_len,
                                       int splits, const float *k_scale, const float *v_scale,
                                       const sda_tensor *gate, void *workspace, size_t workspace_bytes,
                                       void *stream);

/*
 * Region selection for decode rows: the step before sparse_decode_attention
 * on the vLLM page "vllm.models.step5.nvidia.flashinfer_sparse"
 * (`select_and_run_decode_attention` calls `select_regions(scores, current,
 * topk, topk_lengths=..., sort=False)`; its body is not on the page, so the
 * rule below is a reading).
 *
 *   scores        [rows, N] fp32, stride[1] == 1: a score per region id.
 *   current       [rows] int32: the region holding the row's own token; it is
 *                 always kept when 0 <= current < length.
 *   topk_lengths  [rows] int32 or NULL (every row has N candidates): the row
 *                 considers region ids [0, min(length, N)).
 *   topk          regions per row (>= 1).
 *   regions       [rows, topk] int32, stride[1] == 1 (written): the current
 *                 region first, then the topk - 1 best-scoring other
 *                 candidates in ascending id order, then -1 padding.  NaN
 *                 scores rank lowest; equal scores go to the lower id.
 * No workspace; returns SDA_ERR_INVALID for shapes, dtypes or strides outside
 * this contract, SDA_ERR_CUDA if the launch failed.
 */
sda_status sparse_decode_select_regions(const sda_tensor *scores, const sda_tensor *current,
                                        const sda_tensor *topk_lengths, int topk,
                                        const sda_tensor *regions, void *stream);

/*
 * Indexer decode scores: a score per 8-token region for every (token, KV
 * group) row, the input of sparse_decode_select_regions.  The adapter page
 * "vllm.models.step5.nvidia.flashinfer_sparse" computes this in
 * `decode_logits` (fast path `decode_summary_scores`, for FP8 queries of 8
 * heads x 256 and uint8 summaries [*, G, 256]) through an FP8 paged
 * MQA-logits kernel whose formula is not on the page; the reading taken is
 *     score[row, j] = sum_h weights[token, g, h] * max(0, <q_h, m_j>)
 * over the 8 index heads h, with q_h = query[token, g, h, :] and m_j the
 * summary of region j of group g, both decoded from E4M3 (no scale), the
 * product accumulated in fp32.
 *
 *   query        [tokens, G, 8, 256] FP8 E4M3 (or uint8 holding E4M3 bytes);
 *                stride[3] == 1, stride[2] == 256, stride[0] and stride[1]
 *                multiples of 16, base 16-byte aligned.  Row r = t * G + g.
 *   weights      [tokens, G, 8] fp32, stride[2] == 1.
 *   summaries    [slots, G, 256] FP8 E4M3 / uint8, stride[2] == 1,
 *                stride[1] == 256, stride[0] a multiple of 16, base 16-byte
 *                aligned.  Slot page * (block_size / 8) + k holds the summary
 *                of tokens [8k, 8k + 8) of that page.
 *   block_table  [reqs, W] int32, stride[1] == 1: the request's pages.
 *   seq_lens     [>= reqs] int32: request lengths; the query_len tokens of
 *                request q are tokens q * query_len + i at position
 *                seq_lens[q] - query_len + i.
 *   block_size   tokens per page, a multiple of 8.
 *   query_len    tokens per request, 1..4; tokens must be a multiple of it.
 *   scores       [tokens * G, N] fp32, stride[1] == 1 (written): columns
 *                j < min(pos / 8 + 1, N) hold the score of region j, the
 *                rest -inf (all -inf when pos < 0).  Region j's page is
 *                block_table[req, 8j / block_size].
 *   current      [tokens * G] int32 or NULL (written): pos / 8, -1 if pos < 0.
 *   lengths      [tokens * G] int32 or NULL (written): the number of scored
 *                columns, min(pos / 8 + 1, N) (0 if pos < 0).
 *   workspace    NULL, or >= 256 bytes, 256-byte aligned: receives
 *                SDA_FLAG_BOUNDS when a scored region's table column is past
 *                W or its page has no slots in `summaries` (that region
 *                scores -inf); read it with sparse_decode_read_errors.
 * Every summary is read from HBM once per (request, group): the query_len
 * tokens share it.  Returns SDA_ERR_INVALID for shapes, dtypes or strides
 * outside this contract, SDA_ERR_UNSUPPORTED for query_len > 4 or
 * misaligned operands, SDA_ERR_WORKSPACE for a bad workspace, SDA_ERR_CUDA if
 * the launch failed; tokens == 0 returns SDA_OK with no launch.
 */
sda_status sparse_decode_summary_scores(const sda_tensor *query, const sda_tensor *weights,
                                        const sda_tensor *summaries, const sda_tensor *block_table,
                                        const sda_tensor *seq_lens, int block_size, int query_len,
                                        const sda_tensor *scores, const sda_tensor *current,
                                        const sda_tensor *lengths, void *workspace,
                                        size_t workspace_bytes, void *stream);

/*
 * Tables of a step, built on the GPU from request lengths: which pages the new
 * tokens take, the block table with them, and each new token's slot, position
 * and request - what sparse_decode_rope_append writes by and the attention
 * entry points read by.  No counterpart on the pages, whose serving engine
 * builds these on the host.
 *
 *   context_lens  [Q] int32: tokens of each request already in the cache.
 *   new_lens      [Q] int32: tokens the step adds; 0 leaves the request out;
 *                 -1 releases it: its ceil(context / B) pages go back and its
 *                 length becomes 0 (its table entries stay as they were).
 *   block_size    B, tokens per page.
 *   rows_per_request  0: the token rows are packed, request after request.  k >
 *                 0: T == Q * k, request q has rows q k .. q k + k - 1 and its
 *                 tokens are the last of them, as sparse_decode_paged_attention
 *                 with query_len = k reads them; more than k tokens are outside
 *                 the contract.
 *   free_pages    [F] int32, a ring of free page ids (read and written).
 *   free_state    [2] int32: the ring's first free entry and how many are free.
 *   free_next     [2] int32 (written): the same after the step; may be
 *                 free_state itself.
 *   block_table   [Q, W] int32, stride[1] == 1, rows that do not overlap (read
 *                 and written): the columns of the pages taken are written.
 *   seq_lens      [Q] int32 (written): lengths after the step; may be
 *                 context_lens itself (same stride).
 *   token_starts  [Q + 1] int32 (written): the row of each request's first
 *                 token (where it would be, if there is none), and the row
 *                 after the last.
 *   slots         [T] int64 (written): page * B + offset of each token row.
 *   positions     [T] int32 (written): the token's position in its request.
 *   requests      [T] int32 (written): the token's request.
 *                 Rows without a token get -1 in all three.
 *   workspace     >= 256 bytes, 256-byte aligned, zeroed once before first use;
 *                 receives the flags below.  Calls that overlap on the GPU
 *                 must not share one.
 * Pages are taken from the ring in the order of the requests and of their
 * columns, token rows likewise, so the result is a function of the inputs
 * alone.  A request whose pages or rows do not fit gets nothing and keeps its
 * length, as do those after it that need what ran out (SDA_FLAG_FULL).
 * Pages released in a step go behind the ring's last free entry and can be
 * taken by the next step.  A request outside the contract (a negative context,
 * new_lens below -1, more pages than W, a ring with no room for what it
 * returns) is left out with SDA_FLAG_BOUNDS, as is a whole ring whose
 * free_state is out of range; a table entry below 0 under a partly filled page
 * gives slot -1 with the same flag.
 * All but the per-request vectors have stride 1.  Returns SDA_ERR_INVALID for
 * shapes, dtypes or strides outside this contract, SDA_ERR_UNSUPPORTED for
 * Q > 8192 or F or T above 2^30, SDA_ERR_WORKSPACE for a bad workspace,
 * SDA_ERR_CUDA if the launch failed.
 */
sda_status sparse_decode_plan_step(const sda_tensor *context_lens, const sda_tensor *new_lens,
                                   int block_size, int rows_per_request, const sda_tensor *free_pages,
                                   const sda_tensor *free_state, const sda_tensor *free_next,
                                   const sda_tensor *block_table, const sda_tensor *seq_lens,
                                   const sda_tensor *token_starts, const sda_tensor *slots,
                                   const sda_tensor *positions, const sda_tensor *requests,
                                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * Rotary positions with one to four axes (text; time, height and width of
 * images and video), and the new keys and values written to their slots of the
 * packed cache.  The pages' model does both before it calls the attention
 * above; they print neither.
 *
 * Frequency pair i of a head, elements (a, b), turns by the angle
 * t = positions[axis(i), token] * inv_freq[i]:
 *     a' = amplitude * (a cos t - b sin t),  b' = amplitude * (b cos t + a sin t)
 * over the first 2 * len(inv_freq) dims; the others pass through.  The angle
 * is reduced in 64-bit fixed point: at any position it is off by less than
 * max(1, |inv_freq|) * 2^-32 of a turn, beside the rounding of its fp32 sine
 * and cosine.  The products are fp32, each output is rounded once.
 *
 *   query       [T, Hq, D] bf16 or NULL; query_out (written) the same shape;
 *               query_out may be query itself, else they must not overlap.
 *   key, value  [T, G, D] bf16, or both NULL (then cache and slots may be
 *               NULL; slots, when given, still mark padding).
 *   positions   [A, T] int32, A in 1..4, any strides (0 included); or NULL: no
 *               rotation, inv_freq is ignored.  Negative positions turn
 *               backwards.
 *   inv_freq    [R] fp32, stride 1, finite; 2R a multiple of 16, 2R <= D.
 *   sections    A ints whose sum is R, or NULL with A == 1: pairs per axis.
 *   interleaved_axes  zero: the first sections[0] pairs turn by axis 0, the
 *               next sections[1] by axis 1, ...  Nonzero: pair i turns by axis
 *               a = i % A while i / A < sections[a], a > 0; the others by axis 0
 *               (sections[a] <= ceil((R - a) / A) for a > 0).
 *   adjacent_pairs    zero: pair i is dims (i, i + R); nonzero: dims (2i, 2i + 1).
 *   amplitude   factor on the turned dims (1 for plain rotary positions).
 *   slots       [T] int64, stride 1: page * B + offset; -1 marks a padding row:
 *               nothing of it is used, and its query_out row is left as it was.
 *               A slot outside the cache leaves its row out with
 *               SDA_FLAG_BOUNDS.  Two rows must not name the same slot (its
 *               contents would be a mix of the two).
 *   cache       [pages, G, B, 2D] bf16, FP8_E4M3 or UINT8, K first then V
 *               (written at the slots only): K turned, V as it is.  FP8:
 *               e4m3(x / scale), rounded to nearest even, saturated at 448.
 *   k_scale, v_scale  device fp32 scalars; required for an FP8 cache.
 *   workspace   NULL, or >= 256 bytes, 256-byte aligned: receives the flag.
 * D is a multiple of 16 up to 512.  stride[2] == 1 (cache: stride[3] == 1);
 * the bases and the other byte strides are multiples of 16, else
 * SDA_ERR_UNSUPPORTED.  Returns SDA_ERR_INVALID for shapes, dtypes or strides
 * outside this contract, SDA_ERR_WORKSPACE for a bad workspace, SDA_ERR_CUDA if
 * the launch failed; T == 0 returns SDA_OK with no launch.
 */
sda_status sparse_decode_rope_append(const sda_tensor *query, const sda_tensor *query_out,
                                     const sda_tensor *key, const sda_tensor *value,
                                     const sda_tensor *positions, const sda_tensor *inv_freq,
                                     const int32_t *sections, int interleaved_axes, int adjacent_pairs,
                                     float amplitude, const sda_tensor *slots, const sda_tensor *cache,
                                     const float *k_scale, const float *v_scale, void *workspace,
                                     size_t workspace_bytes, void *stream);

/*
 * Bytes of workspace sparse_decode_paged_attention needs for query rows of
 * `heads` heads, `query_len` tokens a request and head size `head_dim`: a
 * 256-byte header (device error flags), the join tasks, and fp32 partial
 * outputs and log-sum-exps of the pieces of requests that CTAs share.  It
 * depends on no batch size or length.  Returns 0 for arguments out of range.
 */
size_t sparse_decode_paged_workspace_bytes(int heads, int query_len, int head_dim);

/*
 * Attention of each request's newest query_len tokens over its whole paged
 * cache (the layers that neither select regions nor slide a window).
 *
 *   query        [rows, H, D] bf16, stride[2] == 1; rows = tokens * G, row r is
 *                KV group r % G of token r / G; D in {64, 128, 192, 256};
 *                H * query_len <= 64.
 *   cache        [pages, G, B, 2D] bf16, FP8_E4M3 or UINT8: K then V; as in
 *                sparse_decode_attention.  B a multiple of 8.
 *   block_table  [requests, W] int32, stride[1] == 1.
 *   seq_lens     [requests] int32: tokens of each request, the query_len being
 *                decoded included.  Token j sits at seq_lens - query_len + j and
 *                sees tokens 0..that position; a token below position 0 sees
 *                nothing: its output is +0.0 and its lse -inf.  seq_lens < 0
 *                marks a padding request: its rows are left as they were.
 *   output       [rows, H, D] bf16, stride[2] == 1 (written).
 *   lse          NULL, or [rows, H] fp32 (written): natural log-sum-exp of the
 *                row's scaled logits, for joining with attention over other keys.
 *   scale, query_len, k_scale, v_scale, gate, stream: as in
 *                sparse_decode_attention (the gate does not enter lse).
 *   workspace    >= sparse_decode_paged_workspace_bytes(H, query_len, D) bytes,
 *                256-byte aligned, its header zeroed once before first use.
 *                Calls that overlap on the GPU must not share one.
 * The cache tiles of all requests are dealt out evenly over the GPU whatever
 * the lengths, on the device, so the call can be captured in a graph; the
 * pieces of a request are joined by their log-sum-exps in a fixed order, so
 * equal inputs give equal bits.  What masked or unused cache places hold (NaN
 * included) does not reach the output.  An infinite value in V gives the rows
 * that see it an infinity of its sign, NaN where they see both signs or where
 * its weight underflows.  A length past the table counts as W * B, and the
 * piece of a table entry outside the cache is left out; both raise
 * SDA_FLAG_BOUNDS.
 * Logits, sums and outputs are fp32.  The weights that multiply V have 16 bits
 * beside a bf16 cache; beside FP8 they have 11 down to 2^-27 of the row's
 * largest, and below that are off by 2^-38 of it at most.
 * How the work is split follows the width W, which the host knows, and not the
 * lengths: where a table is wider than this step's longest request, a view of
 * its first columns is the faster call (block_table with a smaller shape[1] and
 * the same strides).
 * Errors as for sparse_decode_attention.
 */
sda_status sparse_decode_paged_attention(const sda_tensor *query, const sda_tensor *cache,
                                         const sda_tensor *block_table, const sda_tensor *seq_lens,
                                         const sda_tensor *output, const sda_tensor *lse, float scale,
                                         int query_len, const float *k_scale, const float *v_scale,
                                         const sda_tensor *gate, void *workspace, size_t workspace_bytes,
                                         void *stream);

/*
 * Reads the device error flags (SDA_FLAG_*) from a workspace into *flags,
 * optionally clearing them.  Synchronises `stream` (it must be the stream the
 * calls ran on).  Returns SDA_ERR_CUDA if a CUDA call failed.
 */
sda_status sparse_decode_read_errors(const void *workspace, uint32_t *flags, int clear, void *stream);

/*
 * Upper bound in nanoseconds for every pipeline wait inside the kernels
 * (default 1e9).  A wait that runs out sets SDA_FLAG_TIMEOUT, stops the row,
 * lets in-flight copies land and returns.  Applies to launches made after the
 * call, process-wide.  Meant for failure-detection tests.
 */
void sparse_decode_set_wait_limit_ns(uint64_t ns);

/*
 * Allocation-free variant of sparse_decode_attention.  The page has no
 * counterpart for it.
 *
 * For callers that cannot obtain device memory for a workspace: plugin or
 * FFI hosts that are handed tensor pointers by another runtime but no
 * allocator, and code that must not call cudaMalloc while other work is in
 * flight (an allocation can synchronise the device).  Arguments and results
 * are those of sparse_decode_attention without `workspace` /
 * `workspace_bytes`: the scratch (flag header, split partials and LSEs) lives
 * in an 8 MiB static device array inside the library, which every GPU that
 * loads the library holds until the process exits.
 *   - Limit: sparse_decode_workspace_bytes(rows, H, splits) must be at most
 *     8 MiB (8388608), else SDA_ERR_WORKSPACE is returned and nothing is
 *     enqueued.  splits == 1 needs 256 bytes, so any row count fits; with
 *     16 heads, rows * splits up to 679 fits.  Arguments outside the contract
 *     get the statuses of sparse_decode_attention, checked first, also with
 *     nothing enqueued.
 *   - The first call on a device (of this function or of
 *     sparse_decode_no_alloc_read_errors) looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current) and zeroes its flag
 *     header with an async memset on `stream`; make that first call before
 *     any stream capture on the device.
 *   - Every call on a device shares the one array, which keeps the previous
 *     call's contents.  Calls whose kernels overlap on the GPU (different
 *     streams, no ordering between them) race on it: serialise them.
 *   - Device flags (SDA_FLAG_*) collect in the array's header over calls, as
 *     in a caller's workspace; read and clear them with
 *     sparse_decode_no_alloc_read_errors.
 *   - Nothing is allocated: no cudaMalloc, cudaFree or allocating library call.
 */
sda_status sparse_decode_attention_no_alloc(const sda_tensor *query, const sda_tensor *cache,
                                            const sda_tensor *regions, const sda_tensor *block_table,
                                            const sda_tensor *positions, const sda_tensor *active,
                                            const sda_tensor *output, float scale, int query_len,
                                            int splits, const float *k_scale, const float *v_scale,
                                            const sda_tensor *gate, int clear_inactive,
                                            int region_tokens, void *stream);

/*
 * The device flags of sparse_decode_attention_no_alloc on the current device
 * (the page has no counterpart): as sparse_decode_read_errors on the static
 * array's header.  Synchronises `stream`, which must be ordered after the
 * calls whose flags are wanted; with `clear` the header is zeroed afterwards.
 * Returns SDA_ERR_INVALID for a NULL `flags`, SDA_ERR_CUDA if a CUDA call
 * failed.
 */
sda_status sparse_decode_no_alloc_read_errors(uint32_t *flags, int clear, void *stream);

/*
 * Diagnostic builds only (the library compiled with SDA_TIMELINE): registers a
 * device buffer of at least 83886080 bytes (10 x 2^20 uint64) into which the
 * split and combine kernels of later launches write %globaltimer stamps (ns) at
 * their phase boundaries: split CTA u at entries u * 8 + k (k = 0 start, 1 the
 * consumers released with the row's live regions, 2 first K|V stage landed, 3
 * stage loop done, 4 output writes start, 5 done), combine CTA r at entries
 * 2^23 + r * 2 + k (k = 0 start, 1 past its wait on the split kernel).  NULL
 * stops the stamps.  Not thread-safe, synchronous.  The regular library returns
 * SDA_ERR_UNSUPPORTED and does nothing; its kernels carry no stamps.  No
 * counterpart on the pages: it is a measurement aid.
 */
sda_status sparse_decode_timeline_buffer(void *buffer, size_t bytes);

/* A static description of a status code. */
const char *sparse_decode_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* SDATTN_H */
