/*
 * msa.h -- block-sparse paged decode attention for one NVIDIA GB300 (sm_103a).
 *
 * One decode step of the MiniMax-M3 sparse-attention ("MSA") path, as the
 * TensorRT-LLM pages describe it, for every query token t of the step:
 *   (a) score every cached token's index key against the token's index
 *       query and keep the maximum per 128-token block;
 *   (b) select the top-k blocks, ties going to the smaller block index,
 *       as an ascending, -1-padded table;
 *   (c) grouped-query attention (16 query heads per KV head) over only the
 *       selected 128-token pages, reached through the block table, giving
 *       the bf16 output and the log-sum-exp.
 *
 * Sources (prose only; none prints a formula or a layout):
 *   "MiniMax-M3 NVFP4 low-latency decode megakernel for modeling_v2 for
 *    Blackwell" -- sections "The TP4 decode target" (index scorer over
 *    index-K pages, long-context block selector and its smaller-block tie
 *    contract, long-context sparse decode) and "The TP8 decode target"
 *    (index scoring fused with block selection, 8-head sparse decode);
 *   "Add Rubin (sm_107) MiniMax-M3.1 low-latency decode targets" -- section
 *    "Items and numerics" (split-K merge of the long-context sparse decode:
 *    fixed order, no atomics, one divide per output), section "Disclosures
 *    and known gaps" (int32 KV offsets overflow at 1M context), and the
 *    commit messages on the selector / sparse-decode hooks (identical
 *    arguments), the long-context select (top-16 over up to 9216 blocks),
 *    the prefill select tile (per-block max-score buffer) and the q8kv4
 *    indexer (the ascending, -1-padded table contract);
 *   "MiniMax-M3: native P128 draft KV view for the NVFP4 hybrid cache" --
 *    section "Description" (128-token pages filled through one block table).
 * Where the pages are silent the library follows these definitions:
 *   - token t = r * q_per_req + j (request r, query j) sees positions
 *     0 .. seq_lens[r] + j - 1 (the causal limit);
 *   - index score = plain dot product; block score = max over the block's
 *     visible positions, -inf for a block with none;
 *   - only blocks with a visible position can be selected;
 *   - query head h uses KV head h / 16;
 *   - with one index head every KV head of a token uses one table; with
 *     Hi = num_index_heads > 1 (a multiple of Hkv), index head i belongs to
 *     KV head i / (Hi / Hkv) and each KV head g gets its own table, selected
 *     on the maximum over its index heads of their block scores
 *     ("KV-head-reduced scores", selector-hook commit of "Add Rubin (sm_107)
 *     ..."; the select op's table is [tokens, heads, topk]);
 *   - init / local forcing (prefill-select commit of "Add Rubin (sm_107)
 *     ..."): the first init_blocks and the last local_blocks blocks a token
 *     sees are always selected (init_blocks + local_blocks <= topk); the
 *     other places go to the best block scores as above;
 *   - logits are softmax_scale * q . k (FP8 keys times k_scale), the output
 *     is the softmax-weighted mean of V (FP8 values times v_scale), and
 *     lse = ln(sum exp(logit)) (natural log); NVFP4 keys and values are
 *     e2m1 x E4M3 scale x the tensor scale (k_scale, v_scale);
 *   - NVFP4 index keys: dimension 2i is the low nibble of byte i, one E4M3
 *     scale per 16 consecutive dimensions, no global scale.
 *
 * Conventions for every entry point:
 *   - Pointers are caller-owned device memory unless stated; the library
 *     allocates nothing and keeps no per-call state.
 *   - Calls are asynchronous on `stream`; only msa_check_device_status
 *     synchronises.
 *   - Arguments are validated on the host before anything is launched.  A
 *     shape the kernels do not cover returns MSA_ERR_UNSUPPORTED (never a
 *     silent fallback); bad pointers, sizes or alignment return
 *     MSA_ERR_INVALID_ARGUMENT.  Nothing is launched in either case.
 *   - Values that can only be checked on the device (page ids in the block
 *     table, seq_lens, selected block ids) are bounds-checked by the
 *     kernels before use (each of msa_index_score, msa_select_topk and
 *     msa_sparse_decode checks the ones it reads); a bad one sets a bit in
 *     the workspace's error word, the offending access is skipped, and the
 *     outputs of that call are unspecified.  msa_check_device_status
 *     reports and clears it.
 *   - Every device pointer must be 16-byte aligned.
 *
 * Layouts (row-major, element type as stored; T = num_requests * q_per_req,
 * Hi = num_index_heads, Hs = 1 if Hi == 1 else num_kv_heads (tables per
 * token), P = page_size = 128, D = head_dim = 128, Di = index_dim = 128):
 *   q_idx        bf16 [T][Hi][Di]
 *   idxk_pool    MSA_BF16:  bf16 [num_pages][Hi][P][Di]
 *                MSA_NVFP4: uint8 [num_pages][Hi][P][Di/2]  (e2m1 pairs)
 *   idxk_scales  MSA_NVFP4 only: E4M3 [num_pages][Hi][P][Di/16], else NULL
 *   q            bf16 [T][Hq][D]
 *   kv_pool      MSA_BF16 or MSA_FP8_E4M3 [num_pages][2][Hkv][P][D]: the K
 *                page of KV head g of page p, then the V pages after all K;
 *                MSA_NVFP4 [num_pages][2][Hkv] tiles of 9216 bytes: e2m1
 *                pairs [P][D/2] (dimension 2i in the low nibble) then E4M3
 *                scales [P][D/16], one per 16 dimensions; k_scale and
 *                v_scale are the tensor (second-level) scales
 *   block_table  int32 [num_requests][max_blocks_per_seq]; entry b of row r
 *                is the page of logical block b of request r.  Only blocks
 *                b < ceil((seq_lens[r] + q_per_req - 1) / P) are read.
 *   seq_lens     int32 [num_requests], each >= 1
 *   block_scores fp32 [T][Hi][max_blocks_per_seq]; entries b < the
 *                request's cached block count are written (-inf where the
 *                token sees no position of block b); the rest are untouched
 *   selected     int32 [T][Hs][topk], ascending, -1 padded
 *   out          bf16 [T][Hq][D] (round to nearest even from fp32)
 *   lse          fp32 [T][Hq]
 */
#ifndef MSA_H
#define MSA_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum msa_status {
    MSA_OK = 0,
    MSA_ERR_INVALID_ARGUMENT = 1, /* null / misaligned pointer, bad size, small workspace */
    MSA_ERR_UNSUPPORTED = 2,      /* a shape or dtype the kernels do not cover */
    MSA_ERR_CUDA = 3,             /* a CUDA runtime call failed */
    MSA_ERR_DEVICE_CHECK = 4,     /* a kernel found a bad page id, seq_len or block id */
    MSA_ERR_TIMEOUT = 5           /* a kernel's bounded wait ran out */
} msa_status;

typedef enum msa_dtype {
    MSA_BF16 = 0,
    MSA_FP8_E4M3 = 1,
    MSA_NVFP4 = 2
} msa_dtype;

/* Shape and scalars of one call.  Covered today: head_dim = index_dim =
 * page_size = 128, num_q_heads = 16 * num_kv_heads, num_index_heads = 1 or
 * a multiple of num_kv_heads up to 64, 1 <= q_per_req <= 64,
 * 1 <= topk <= 256, max_blocks_per_seq <= 16384,
 * num_requests * q_per_req <= 8192, kv_dtype in {BF16, FP8_E4M3, NVFP4},
 * index_dtype in {BF16, NVFP4}. */
typedef struct msa_shape {
    int32_t num_requests;       /* R */
    int32_t q_per_req;          /* query tokens per request (1 + draft length) */
    int32_t num_q_heads;        /* Hq */
    int32_t num_kv_heads;       /* Hkv */
    int32_t head_dim;           /* D */
    int32_t num_index_heads;    /* Hi */
    int32_t index_dim;          /* Di */
    int32_t page_size;          /* P, tokens per page */
    int32_t num_pages;          /* pages in kv_pool and idxk_pool */
    int32_t max_blocks_per_seq; /* block_table row width */
    int32_t topk;               /* blocks selected per token */
    int32_t kv_dtype;           /* msa_dtype of kv_pool */
    int32_t index_dtype;        /* msa_dtype of idxk_pool */
    int32_t decode_ctas;        /* persistent CTAs of the sparse decode; 0 = library default */
    float softmax_scale;        /* multiplies q . k (1/sqrt(128) in the workloads) */
    float k_scale;              /* FP8 K dequantisation scale (ignored for bf16) */
    float v_scale;              /* FP8 V dequantisation scale (ignored for bf16) */
    int32_t init_blocks;        /* first blocks every token keeps (0: none) */
    int32_t local_blocks;       /* most recent blocks every token keeps (0: none) */
} msa_shape;

/* Bytes of device workspace the calls below need for `shape` (0 if the
 * shape is invalid or unsupported).  Pure host function. */
size_t msa_workspace_bytes(const msa_shape *shape);

/* Zero the workspace (error word and the decode's split-arrival counters).
 * Call once after allocating it, and again after a call reported
 * MSA_ERR_TIMEOUT; every other call leaves the counters at zero. */
msa_status msa_workspace_init(void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* Stage (a): block_scores[t][i][b] = max over the visible positions of
 * block b of dot(q_idx[t][i], index key of head i).  One pass per index
 * head.  Exact in fp32 for integer-valued
 * bf16 inputs with |score| < 2^24 and for NVFP4 keys with power-of-two
 * scales.  ("MiniMax-M3 NVFP4 low-latency decode megakernel ...", "The TP4
 * decode target": the index scorer; prefill-select commit of "Add Rubin
 * (sm_107) ...": the per-block max-score buffer.) */
msa_status msa_index_score(const msa_shape *shape, const void *q_idx, const void *idxk_pool,
                           const void *idxk_scales, const int32_t *block_table,
                           const int32_t *seq_lens, float *block_scores, void *workspace,
                           size_t workspace_bytes, cudaStream_t stream);

/* Stage (b): for each token (and KV head, when Hs > 1), the topk blocks
 * with the largest block score (the maximum over the KV head's index heads)
 * among blocks 0 .. ceil((seq_lens[r] + j) / 128) - 1, ties to the smaller
 * block index, after the init_blocks first and local_blocks last of them,
 * which are always kept; written ascending and -1 padded.  Bit-exact.
 * init_blocks + local_blocks > topk, or either negative, returns
 * MSA_ERR_INVALID_ARGUMENT.
 * ("MiniMax-M3 NVFP4 low-latency decode megakernel ...", "The TP4 decode
 * target": tie contract; q8kv4 indexer commit of "Add Rubin (sm_107) ...":
 * the ascending, -1-padded table.) */
msa_status msa_select_topk(const msa_shape *shape, const float *block_scores,
                           const int32_t *seq_lens, int32_t *selected, void *workspace,
                           size_t workspace_bytes, cudaStream_t stream);

/* Stage (c): attention of each token over the visible positions of its
 * selected blocks, split over persistent CTAs and merged in a fixed order
 * with one reciprocal per output row (no atomics).  out: bf16, lse: fp32.
 * The CTAs' task ranges are cut in 32-bit arithmetic: a call with
 * T * num_kv_heads * topk * (decode CTAs + 1) >= 2^32 returns
 * MSA_ERR_UNSUPPORTED (so does msa_decode_step).
 * ("MiniMax-M3 NVFP4 low-latency decode megakernel ...", "The TP4 decode
 * target": long-context sparse decode; "Add Rubin (sm_107) ...", "Items and
 * numerics": the split-K merge.) */
msa_status msa_sparse_decode(const msa_shape *shape, const void *q, const void *kv_pool,
                             const int32_t *block_table, const int32_t *seq_lens,
                             const int32_t *selected, void *out, float *lse, void *workspace,
                             size_t workspace_bytes, cudaStream_t stream);

/* Stages (a) + (b) + (c) in one call (the fused decode step).  block_scores
 * and selected may be NULL, in which case the workspace holds them. */
msa_status msa_decode_step(const msa_shape *shape, const void *q_idx, const void *idxk_pool,
                           const void *idxk_scales, const void *q, const void *kv_pool,
                           const int32_t *block_table, const int32_t *seq_lens,
                           float *block_scores, int32_t *selected, void *out, float *lse,
                           void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* The KV / index-key update: writes this step's new tokens into their pages
 * through the block table, to run before msa_index_score / msa_decode_step
 * on the same stream.  ("MiniMax-M3 NVFP4 low-latency decode megakernel
 * ...", "The TP4 decode target": the attention megakernels carry "the KV
 * update"; q8kv4 indexer commit of "Add Rubin (sm_107) ...": the NVFP4
 * index-K copy is "refreshed from this step's slots".)
 *   k_new, v_new  bf16 [T][Hkv][D]   this step's keys and values
 *   idxk_new      bf16 [T][Hi][Di]   this step's index keys
 *   kv_pool, idxk_pool, idxk_scales  the pools of the layouts above (written)
 * New token j of request r goes to position seq_lens[r] - 1 + j (the last
 * position it sees): row (pos % 128) of page block_table[r][pos / 128].
 * Only those rows are written.  Encodings: bf16 pools take the inputs as
 * they are; MSA_FP8_E4M3 pools store E4M3(x / k_scale) for K and
 * E4M3(x / v_scale) for V; MSA_NVFP4 K / V pools store y = x / k_scale
 * (x / v_scale) by the index keys' recipe; MSA_NVFP4 index keys store, per 16 consecutive
 * dimensions, the E4M3 scale c = E4M3(max |x| / 6) and the e2m1 codes of
 * x / value(c) (0 when c is 0), dimension 2i in the low nibble.  Every
 * rounding is to nearest even and saturating, quotients in fp32, and a code
 * that rounds to zero is stored as +0.  A bad seq_len or page id is
 * reported through the workspace error word (that row is skipped). */
msa_status msa_kv_update(const msa_shape *shape, const void *k_new, const void *v_new,
                         const void *idxk_new, const int32_t *block_table,
                         const int32_t *seq_lens, void *kv_pool, void *idxk_pool,
                         void *idxk_scales, void *workspace, size_t workspace_bytes,
                         cudaStream_t stream);

/* Block tables of many query rows (a prefill's context rows) from a
 * head-major max-score buffer, one table per row and selection head, the
 * same table bit for bit as msa_select_topk gives each row (ties to the
 * smaller block, init / local forcing).  ("Add Rubin (sm_107) ...",
 * prefill-select commit: context rows take a tile select, one CTA per KV
 * head and 8 queries over a [heads, max_k_tiles, tokens] max-score block,
 * each score sector read once.)
 *   scores_hbt  fp32 [Hs][max_blocks_per_seq][T], the row index innermost:
 *               the selection heads' block scores (already reduced over
 *               index heads); entry b of row t is read for
 *               b < ceil((seq_lens[r] + j) / 128), t = r * q_per_req + j
 *   selected    int32 [T][Hs][topk], ascending, -1 padded
 * q_per_req may exceed the decode's 64 here (a prefill of C tokens is one
 * request with q_per_req = C and seq_lens = 1).  max_blocks_per_seq above
 * 2048 returns MSA_ERR_UNSUPPORTED (msa_select_topk covers longer rows in
 * the token-major layout).  Only the workspace's error word is used: a
 * workspace of 256 bytes suffices. */
msa_status msa_select_rows(const msa_shape *shape, const float *scores_hbt,
                           const int32_t *seq_lens, int32_t *selected, void *workspace,
                           size_t workspace_bytes, cudaStream_t stream);

/* ---- the whole cache: dense decode, accumulated weights, eviction --------
 * The three calls below work on every cached position instead of selected
 * blocks.  They share msa_shape, the layouts above, the conventions above and
 * one workspace; msa_workspace_init and msa_check_device_status work on it as
 * on the other.  Differences to the calls above:
 *   - num_q_heads is any multiple G of num_kv_heads with 1 <= G <= 64: query
 *     head h uses KV head h / G; num_kv_heads is at most 8192;
 *   - seq_lens[r] may be 0: an idle slot of a padded batch.  Its out rows are
 *     0, its lse -inf, its weights untouched, its new length 0; its block
 *     table row is not read.  A negative length, or one the table cannot
 *     hold, is reported through the error word;
 *   - topk, init_blocks and local_blocks are not looked at (topk is, where a
 *     `selected` table is given), nor the index fields where no index keys are
 *     given; num_requests * max_blocks_per_seq * num_kv_heads * the query rows'
 *     tiles stays below 2^31, num_pages * num_kv_heads * 288 too, else
 *     MSA_ERR_UNSUPPORTED;
 *   - decode_ctas > 0 sets the persistent CTAs of the dense decode and of the
 *     accumulation (at most 8192); 0 takes one per SM;
 *   - bytes of a page behind the last cached position may hold anything
 *     (infinities and NaN among it);
 *   - outputs overlap neither inputs nor one another, but for weights_out,
 *     which may be weights_in;
 *   - nothing is kept in the workspace between calls but the error word.  Calls
 *     on two streams that may overlap, and CUDA graphs that may, need a
 *     workspace each. */

/* Bytes of device workspace for the three calls below (0 if the shape is
 * invalid or unsupported).  Pure host function. */
size_t msa_cache_workspace_bytes(const msa_shape *shape);

/* Attention of each token over all positions it sees (0 .. seq_lens[r] + j - 1):
 * the result of msa_sparse_decode with every block selected, without its limit
 * of 256 blocks.  The pages of a request are read once for all its tokens, are
 * split over persistent CTAs and joined in a fixed order (no atomics: the same
 * inputs give the same bits).  out: bf16, lse: fp32.  Sums and the softmax are
 * fp32; probabilities meet V as a pair of bf16 (off by 2^-16 at most) over bf16
 * pages, as fp16 (2^-11) over E4M3 and NVFP4 pages; queries meet E4M3 and NVFP4
 * keys as fp16 after a power of two (elements 2^-23 below a row's largest lose
 * bits).  An infinity or NaN in V makes that dimension of the outputs that see
 * its position infinite or NaN, and no other. */
msa_status msa_dense_decode(const msa_shape *shape, const void *q, const void *kv_pool,
                            const int32_t *block_table, const int32_t *seq_lens, void *out,
                            float *lse, void *workspace, size_t workspace_bytes,
                            cudaStream_t stream);

/* The attention weight of every cached position, accumulated over steps:
 *   weights_out[r][g][p] = decay * weights_in[r][g][p]
 *                          + sum over tokens j and heads h of KV head g that see p
 *                            of exp(softmax_scale * q . k[p] - lse)
 * for p < seq_lens[r] + q_per_req - 1 (other elements stay as they are), with
 * the lse that msa_dense_decode (selected = NULL) or msa_sparse_decode
 * (selected = its table: only positions in blocks a token selected count for
 * it) returned for the same inputs.  A token with lse = -inf adds nothing.
 *   selected     int32 [T][Hs][topk] or NULL
 *   weights_in   fp32 [num_requests][Hkv][max_blocks_per_seq * 128], or NULL
 *                for zeros; positions of this step's own tokens
 *                (p >= seq_lens[r] - 1) count as 0 whatever it holds, so rows
 *                need no clearing when a token is cached (or a rejected draft
 *                token's row is written again)
 *   weights_out  the same layout; may be weights_in
 *   decay        finite; 1 keeps the plain sum, less fades older steps */
msa_status msa_weight_accumulate(const msa_shape *shape, const void *q, const void *kv_pool,
                                 const int32_t *block_table, const int32_t *seq_lens,
                                 const int32_t *selected, const float *lse, float decay,
                                 const float *weights_in, float *weights_out, void *workspace,
                                 size_t workspace_bytes, cudaStream_t stream);

/* Eviction by accumulated weight: of the n = seq_lens[r] + q_per_req - 1 cached
 * positions of request r, min(n, keep) stay -- the first `first`, the last
 * `last`, and those with the largest weights (NaN above every number), ties
 * to the lower position -- and their rows are copied, in ascending order of
 * position, to positions 0, 1, ... of new pages.  One list a request when
 * num_index_heads is 1, on the maximum over KV heads of their weights; one per
 * KV head otherwise (Hs lists, as for block tables), index head i moving with
 * KV head i / (Hi / Hkv).
 *   weights      fp32 [num_requests][Hkv][max_blocks_per_seq * 128]
 *   new_table    int32 [num_requests][ceil(keep / 128)]: pages of kv_pool (and
 *                idxk_pool) that receive the rows.  Only entries below
 *                ceil(min(n, keep) / 128) are read, only the rows copied are
 *                written.  The new pages are pages that no block table row of
 *                the call reads and no other new row names, else the copied
 *                rows are unspecified; old pages are not written and may be
 *                shared between requests
 *   kv_pool, idxk_pool, idxk_scales  the pools of the layouts above;
 *                idxk_pool may be NULL (no index keys), idxk_scales is used for
 *                MSA_NVFP4 index keys.  Stored bytes are moved as they are
 *   new_weights  fp32 [num_requests][Hkv][ceil(keep / 128) * 128] or NULL: the
 *                weights of the kept positions (elements below min(n, keep))
 *   kept         int32 [num_requests][Hs][keep], ascending, -1 padded
 *   new_lens     int32 [num_requests]: min(n, keep) - q_per_req + 1, the
 *                seq_lens of the shortened cache (0 for an idle slot)
 * keep >= max(1, q_per_req), first >= 0, last >= q_per_req - 1 and
 * first + last <= keep, else MSA_ERR_INVALID_ARGUMENT; so are
 * new_table == block_table, new_weights == weights and new_lens == seq_lens.
 * keep above 2097152 is MSA_ERR_UNSUPPORTED.  A page id outside the pool is
 * reported through the error word and its rows are skipped. */
msa_status msa_cache_evict(const msa_shape *shape, int32_t keep, int32_t first, int32_t last,
                           const float *weights, const int32_t *block_table,
                           const int32_t *seq_lens, const int32_t *new_table, void *kv_pool,
                           void *idxk_pool, void *idxk_scales, float *new_weights, int32_t *kept,
                           int32_t *new_lens, void *workspace, size_t workspace_bytes,
                           cudaStream_t stream);

/* ---- ragged batches: tokens into the cache, and their attention -----------
 * A prompt, a chunk of one, or a step: request r brings any number of tokens,
 * none among them, rows offsets[r] .. offsets[r + 1] - 1 of the inputs
 * (offsets int32 [num_requests + 1], ascending from 0, offsets[num_requests] <=
 * num_tokens); rows behind the last request's are neither read for a result nor
 * written.  seq_lens[r] is, as everywhere here, what the first of them sees:
 * token j of request r stands at position seq_lens[r] - 1 + j.  A request
 * without tokens is not looked at.  q_per_req, topk and the selection's fields
 * of msa_shape are not looked at.  num_tokens is at most 4194304; with 0 of them
 * nothing is done and pointers may be NULL.  Outputs overlap inputs and one another
 * only where a call says so. */

/* Norm and rotation of rows x of 128 elements of the token at position p:
 *   n = x / sqrt(mean x^2 + norm_eps) * (weight + norm_offset)   where a weight is given
 *   a' = scale (a cos t - b sin t), b' = scale (b cos t + a sin t)
 * for each pair (a, b) of the first rotary_dim elements of n, t = p f_i; the
 * others stay as they are.  fp32, rounded once, to bf16 or to the pool's
 * format; rows without norm and rotation are copied bit by bit to bf16.  mean x^2 is
 * fp32 too: a row whose sum of squares passes 2^128 becomes zeros. */
typedef struct msa_rope {
    int32_t rotary_dim;       /* a multiple of 16 up to 128; 0: no rotation */
    int32_t interleaved;      /* 0: element i turns with i + rotary_dim / 2; 1: 2 i with 2 i + 1 */
    int32_t per_head_weights; /* norm weights are bf16 [heads][128]; 0: [128] for all heads */
    float scale;              /* multiplies the rotated elements (1, or an attention factor) */
    float norm_eps;           /* >= 0 */
    float norm_offset;        /* added to the weights (0; 1 where they are stored as w - 1) */
    /* elements from a token's rows to the next token's, a multiple of 8 (rows that
     * are parts of a fused projection's output); 0: dense */
    int64_t q_stride, k_stride, v_stride, q_idx_stride, idxk_stride;
} msa_rope;

/* turns[i] = f_i / (2 pi) as a fraction of 2^64, for angles of f_i radians a
 * position, 0 <= |f_i| < 2 pi * 2^31: the rotation's frequencies as the calls
 * below take them (a table of rotary_dim / 2 in device memory, filled once: every
 * angle is then p * turns[i] modulo 2^64, which loses nothing at any position).  An
 * entry is off by 2^-52 of itself, from double's roundings, and 2^-64 of a turn.  Pure host
 * function on host memory; MSA_ERR_INVALID_ARGUMENT for a frequency that is
 * not finite or too large. */
msa_status msa_rope_frequencies(const double *radians, int32_t count, uint64_t *turns);

/* Norm and rotation of the query heads, and of key heads in the same pass.
 *   positions    int32 [num_tokens] (negative ones turn the other way)
 *   q            bf16 [num_tokens] x q_stride, num_q_heads * 128 elements each
 *   q_weight     bf16 norm weights, or NULL: no norm (k_weight alike)
 *   q_out        bf16 [num_tokens][num_q_heads][128]; may be q where q is dense
 *   k, k_out     the same for num_k_heads heads; both NULL with num_k_heads = 0
 * freqs may be NULL where rotary_dim is 0. */
msa_status msa_qk_norm_rope(const msa_rope *rope, const uint64_t *freqs, int32_t num_tokens,
                            const int32_t *positions, int32_t num_q_heads, const void *q,
                            const void *q_weight, void *q_out, int32_t num_k_heads, const void *k,
                            const void *k_weight, void *k_out, cudaStream_t stream);

/* Bytes of device workspace for the two calls below (0 if the shape is invalid
 * or unsupported; msa_ragged_attention has one more limit, which depends on the
 * tokens).  Pure host function. */
size_t msa_ragged_workspace_bytes(const msa_shape *shape);

/* The tokens of a ragged batch into their pages, keys and index keys with norm
 * and rotation on the way, and their queries and index queries in the same pass.
 *   k, v         bf16 [num_tokens] x k_stride (v_stride), Hkv * 128 elements each
 *   idxk         bf16, Hi * 128 elements a token, or NULL (then idxk_pool is not written)
 *   q, q_out     bf16, Hq * 128 elements a token; both NULL: no queries.  q_out is
 *                dense [num_tokens][Hq][128] and may be q where q is dense
 *   q_idx, q_idx_out  the same for Hi index queries
 *   k_weight, idxk_weight, q_weight, q_idx_weight  norm weights, each may be NULL.
 *                Values are neither normed nor rotated
 *   block_table, seq_lens, pools  as for msa_kv_update, whose encodings these are:
 *                with rotary_dim 0 and no weights the pools get the same bytes
 * Only the rows of the new tokens are written.  Two tokens of one call that share
 * a row of a page leave either's.  A bad length or page id is reported through the
 * workspace's error word and its token's rows, queries among them, are skipped.
 * Offsets that go down or past num_tokens are reported too: the tokens of a request
 * that ends past num_tokens are skipped, one that two requests have goes to either's
 * place or none.  Only the workspace's error word is used: 256 bytes suffice. */
msa_status msa_kv_append(const msa_shape *shape, const msa_rope *rope, const uint64_t *freqs,
                         int32_t num_tokens, const int32_t *offsets, const void *k,
                         const void *k_weight, const void *v, const void *idxk,
                         const void *idxk_weight, const void *q, const void *q_weight, void *q_out,
                         const void *q_idx, const void *q_idx_weight, void *q_idx_out,
                         const int32_t *block_table, const int32_t *seq_lens, void *kv_pool,
                         void *idxk_pool, void *idxk_scales, void *workspace,
                         size_t workspace_bytes, cudaStream_t stream);

/* Attention of a ragged batch's query rows over paged states: token j of request r
 * sees positions 0 .. seq_lens[r] + j - 1 (causal: a prompt, a chunk of one, or a
 * step, its own keys and values appended before), or all seq_lens[r] of them (not
 * causal: cross attention to states of another length).  What msa_dense_decode
 * computes, without its limits on tokens; probabilities are coarser over bf16 pages,
 * see below.
 *   q, out       bf16 [num_tokens][Hq][128]
 *   lse          fp32 [num_tokens][Hq]
 * num_q_heads is any multiple G of num_kv_heads with 1 <= G <= 64.  seq_lens[r] may
 * be 0: no states, outputs of 0 and lse -inf for all tokens of the request.  (Causal
 * too: seq_lens counts the first token's own position, so a prompt's first chunk has
 * 1.  msa_kv_append reports a 0.)  Offsets past num_tokens, a negative
 * length and one that the table cannot hold are reported through the error word and
 * the request is skipped; offsets that go down are reported and nothing is written;
 * a page id outside the pool is reported, and the outputs of the call are unspecified.
 * Bytes behind the last position may hold anything; an infinity or NaN in V reaches the
 * outputs that see its position, in that dimension, and no other.  One in a query makes
 * its row's outputs not finite; the rows that see a key with one are unspecified.  Sums and the softmax are fp32, in a
 * fixed order (the same inputs give the same bits).  Probabilities meet V as bf16
 * over bf16 pages, and the sum that divides is that of the rounded ones: an output
 * is a mean of values with weights that are off by 2^-8 of themselves at most, and
 * sum to 1 (msa_dense_decode has a pair of bf16: 2^-16).  Over E4M3 and NVFP4 pages they are fp16, and the sum is that of the p as
 * they are: a weight is off by 2^-11 of itself, or by 2^-32 where that is more (one
 * below 2^-33 may count as 0); queries meet the keys as fp16 after a power of two
 * (elements 2^-23 below a row's largest lose bits).
 * decode_ctas > 0 sets the persistent CTAs (at most 8192); 0 takes one per SM.
 * MSA_ERR_UNSUPPORTED also where (num_tokens / 4 + num_requests) * num_kv_heads *
 * (max_blocks_per_seq + 8) passes 2147483000 a CTA.
 * Nothing is kept in the workspace between calls but the error word: calls that may
 * overlap, and CUDA graphs that may, need a workspace each. */
msa_status msa_ragged_attention(const msa_shape *shape, int32_t num_tokens, int32_t causal,
                                const void *q, const int32_t *offsets, const void *kv_pool,
                                const int32_t *block_table, const int32_t *seq_lens, void *out,
                                float *lse, void *workspace, size_t workspace_bytes,
                                cudaStream_t stream);

/* Size of the fixed device scratch used by msa_sparse_decode_noalloc. */
#define MSA_NOALLOC_SCRATCH_BYTES (8u << 20)

/* The paper has no counterpart to this entry point; it exists for callers
 * that cannot allocate device memory: a plugin handed only its input and
 * output tensors by a runtime that owns every device allocation, or code on
 * a path where the allocator may not be called.  It computes exactly what
 * msa_sparse_decode computes, with the same kernels, but keeps the scratch
 * (split partials, their arrival counters and the error word) in a fixed
 * array of MSA_NOALLOC_SCRATCH_BYTES compiled into the library, which every
 * GPU that loads the library holds until the process exits.  It allocates
 * nothing.
 *   - Every call asks the CUDA runtime for the address of the array in the
 *     current device's context (cudaGetSymbolAddress).  The first call on a
 *     device loads the library's device code there; make that first call
 *     before any stream capture.
 *   - All calls share the one array: calls whose work overlaps on the GPU
 *     (different streams, or different host threads) race and give wrong
 *     results.  Each call clears the error word and the arrival counters it
 *     needs; the partial slots are always written before they are read.
 *   - Device-side failures are not reported (there is no workspace to read
 *     them from): neither a bounds failure (bad page id, seq_len or block id)
 *     nor a bounded wait that ran out (MSA_ERR_TIMEOUT elsewhere).  After one
 *     the call still returns MSA_OK and its outputs are unspecified; callers
 *     that need to detect them use msa_sparse_decode.
 *   - Shapes are checked as by every other entry point, with the same
 *     statuses (MSA_ERR_INVALID_ARGUMENT, MSA_ERR_UNSUPPORTED).
 *   - Returns MSA_ERR_UNSUPPORTED when the scratch it needs exceeds
 *     MSA_NOALLOC_SCRATCH_BYTES: 256 bytes of error word, a 4-byte counter per
 *     (token, KV head) pair rounded up to 256 bytes, and (decode CTAs + pairs)
 *     partial slots of 8320 bytes (with 152 decode CTAs, the default on a
 *     152-SM GPU: at most 855 (token, KV head) pairs). */
msa_status msa_sparse_decode_noalloc(const msa_shape *shape, const void *q, const void *kv_pool,
                                     const int32_t *block_table, const int32_t *seq_lens,
                                     const int32_t *selected, void *out, float *lse,
                                     cudaStream_t stream);

/* Test hook, not for production use: the SM-clock limit of the sparse
 * decode's bounded waits in the calls that follow, for the whole process
 * (clocks <= 0 restores the default, 2^31).  With a limit of a few clocks a
 * normal decode gives up at its first wait that is not already complete: its
 * CTAs stop, wait (with the default limit) for their copies and tensor-core
 * work in flight, free their tensor memory and exit, and the call reports
 * MSA_ERR_TIMEOUT through msa_check_device_status.  That is how the timeout
 * path is tested without a hang or a fault.  Always returns MSA_OK. */
msa_status msa_set_decode_wait_limit(int64_t clocks);

/* Synchronise `stream`, read the workspace's error word and clear it.
 * Returns MSA_OK, MSA_ERR_DEVICE_CHECK, MSA_ERR_TIMEOUT or MSA_ERR_CUDA. */
msa_status msa_check_device_status(void *workspace, cudaStream_t stream);

/* Static, human-readable name of a status. */
const char *msa_status_string(msa_status status);

#ifdef __cplusplus
}
#endif

#endif /* MSA_H */
