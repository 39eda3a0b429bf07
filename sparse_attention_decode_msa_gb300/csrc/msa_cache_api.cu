// msa_cache_api.cu -- the C ABI of the whole-cache operators (msa_dense_decode,
// msa_weight_accumulate, msa_cache_evict): host-side validation, workspace
// layout and launches.  No allocation, no state between calls.
#include <cmath>

#include "msa_cache.cuh"

namespace msa {
namespace {

constexpr size_t kAlign = 256;

bool aligned16(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// The shape rules of these operators: any 1 .. 64 query heads per KV head; the
// block selection's fields are looked at where a call uses them.
msa_status check_cache_shape(const msa_shape *s)
{
    if (!s)
        return MSA_ERR_INVALID_ARGUMENT;
    if (s->num_requests < 0 || s->q_per_req < 1 || s->num_kv_heads < 1 || s->num_q_heads < 1 ||
        s->num_pages < 1 || s->max_blocks_per_seq < 1 || s->decode_ctas < 0 || s->num_index_heads < 1)
        return MSA_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(s->softmax_scale) || !std::isfinite(s->k_scale) || !std::isfinite(s->v_scale))
        return MSA_ERR_INVALID_ARGUMENT;
    if (s->head_dim != kDim || s->page_size != kPage || s->num_q_heads % s->num_kv_heads != 0 ||
        s->num_q_heads / s->num_kv_heads > kMaxGroup || s->num_kv_heads > kMaxKvHeads)
        return MSA_ERR_UNSUPPORTED;
    if (s->num_index_heads > kMaxIndexHeads ||
        (s->num_index_heads > 1 && s->num_index_heads % s->num_kv_heads != 0))
        return MSA_ERR_UNSUPPORTED;
    if (s->q_per_req > kMaxQPerReq || s->num_requests > kMaxRequests ||
        (long long)s->num_requests * s->q_per_req > kMaxTokens || s->max_blocks_per_seq > kMaxBlocks)
        return MSA_ERR_UNSUPPORTED;
    if (s->kv_dtype != MSA_BF16 && s->kv_dtype != MSA_FP8_E4M3 && s->kv_dtype != MSA_NVFP4)
        return MSA_ERR_UNSUPPORTED;
    // row coordinates of the KV tensor map (144 rows a tile at most), and the
    // line of (page, KV head, row tile) tasks, fit in int32
    const int rows = s->q_per_req * (s->num_q_heads / s->num_kv_heads);
    const long long tiles = (rows + dense_tile_rows(rows) - 1) / dense_tile_rows(rows);
    if ((long long)s->num_pages * 2 * s->num_kv_heads * 144 > 0x7FFFFFFFll ||
        (double)s->num_requests * s->max_blocks_per_seq * s->num_kv_heads * (double)tiles > 2147483647.0)
        return MSA_ERR_UNSUPPORTED;
    if (s->decode_ctas > kMaxTokens)
        return MSA_ERR_UNSUPPORTED;
    return MSA_OK;
}

struct CacheLayout {
    size_t joins_off, partial_off, total;
};

CacheLayout layout_of(const msa_shape *s)
{
    const int rows = s->q_per_req * (s->num_q_heads / s->num_kv_heads);
    const size_t ctas = s->decode_ctas > 0 ? s->decode_ctas : kCacheCtaBound;
    CacheLayout w;
    w.joins_off = kAlign; // after the error word
    w.partial_off = align_to(w.joins_off + ctas * sizeof(int4), kAlign);
    w.total = align_to(w.partial_off + 2 * ctas * dense_slot_floats(dense_tile_rows(rows)) * sizeof(float), kAlign);
    return w;
}

msa_status check_workspace(const msa_shape *s, const void *ws, size_t bytes)
{
    return ws && aligned16(ws) && bytes >= layout_of(s).total ? MSA_OK : MSA_ERR_INVALID_ARGUMENT;
}

// Persistent CTAs: the shape's, else one per SM; -1 if the device cannot be read.
int cache_ctas(const msa_shape *s)
{
    if (s->decode_ctas > 0)
        return s->decode_ctas;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
        return -1;
    return sms < kCacheCtaBound ? sms : kCacheCtaBound;
}

msa_status cuda_status(cudaError_t e)
{
    return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

void fill(CacheParams &p, const msa_shape *s, const void *q, const void *kv_pool,
          const int32_t *block_table, const int32_t *seq_lens, void *ws)
{
    p.q = static_cast<const uint16_t *>(q);
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.kv = static_cast<const uint8_t *>(kv_pool);
    p.err = static_cast<uint32_t *>(ws);
    p.R = s->num_requests;
    p.nq = s->q_per_req;
    p.Hkv = s->num_kv_heads;
    p.G = s->num_q_heads / s->num_kv_heads;
    p.maxB = s->max_blocks_per_seq;
    p.num_pages = s->num_pages;
    p.scale_log2 = s->softmax_scale * 1.4426950408889634f * (s->kv_dtype != MSA_BF16 ? s->k_scale : 1.f);
    p.wait_limit = decode_wait_limit();
}

} // namespace
} // namespace msa

using namespace msa;

extern "C" {

size_t msa_cache_workspace_bytes(const msa_shape *shape)
{
    return check_cache_shape(shape) == MSA_OK ? layout_of(shape).total : 0;
}

msa_status msa_dense_decode(const msa_shape *shape, const void *q, const void *kv_pool,
                            const int32_t *block_table, const int32_t *seq_lens, void *out,
                            float *lse, void *workspace, size_t workspace_bytes,
                            cudaStream_t stream)
{
    msa_status st = check_cache_shape(shape);
    if (st != MSA_OK)
        return st;
    if ((st = check_workspace(shape, workspace, workspace_bytes)) != MSA_OK)
        return st;
    if (!q || !kv_pool || !block_table || !seq_lens || !out || !lse)
        return MSA_ERR_INVALID_ARGUMENT;
    if (!aligned16(q) || !aligned16(kv_pool) || !aligned16(block_table) || !aligned16(seq_lens) ||
        !aligned16(out) || !aligned16(lse))
        return MSA_ERR_INVALID_ARGUMENT;
    if (shape->num_requests == 0)
        return MSA_OK;
    const int ctas = cache_ctas(shape);
    if (ctas < 1)
        return MSA_ERR_CUDA;
    const CacheLayout w = layout_of(shape);
    DenseParams p;
    fill(p, shape, q, kv_pool, block_table, seq_lens, workspace);
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.joins = reinterpret_cast<int4 *>(static_cast<uint8_t *>(workspace) + w.joins_off);
    p.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + w.partial_off);
    p.v_scale = shape->kv_dtype != MSA_BF16 ? shape->v_scale : 1.f;
    p.rows = p.nq * p.G;
    p.tiles = (p.rows + dense_tile_rows(p.rows) - 1) / dense_tile_rows(p.rows);
    return cuda_status(launch_dense_decode(p, shape->kv_dtype, ctas, stream));
}

msa_status msa_weight_accumulate(const msa_shape *shape, const void *q, const void *kv_pool,
                                 const int32_t *block_table, const int32_t *seq_lens,
                                 const int32_t *selected, const float *lse, float decay,
                                 const float *weights_in, float *weights_out, void *workspace,
                                 size_t workspace_bytes, cudaStream_t stream)
{
    msa_status st = check_cache_shape(shape);
    if (st != MSA_OK)
        return st;
    if (selected && shape->topk < 1)
        return MSA_ERR_INVALID_ARGUMENT;
    if (selected && shape->topk > kMaxTopk)
        return MSA_ERR_UNSUPPORTED;
    if ((st = check_workspace(shape, workspace, workspace_bytes)) != MSA_OK)
        return st;
    if (!q || !kv_pool || !block_table || !seq_lens || !lse || !weights_out || !std::isfinite(decay))
        return MSA_ERR_INVALID_ARGUMENT;
    if (!aligned16(q) || !aligned16(kv_pool) || !aligned16(block_table) || !aligned16(seq_lens) ||
        !aligned16(selected) || !aligned16(lse) || !aligned16(weights_in) || !aligned16(weights_out))
        return MSA_ERR_INVALID_ARGUMENT;
    if (shape->num_requests == 0)
        return MSA_OK;
    const int ctas = cache_ctas(shape);
    if (ctas < 1)
        return MSA_ERR_CUDA;
    WeightParams p;
    fill(p, shape, q, kv_pool, block_table, seq_lens, workspace);
    p.lse = lse;
    p.selected = selected;
    p.weights_in = weights_in;
    p.weights_out = weights_out;
    p.decay = decay;
    p.Hs = shape->num_index_heads == 1 ? 1 : shape->num_kv_heads;
    p.k = shape->topk;
    return cuda_status(launch_weight_accumulate(p, shape->kv_dtype, ctas, stream));
}

msa_status msa_cache_evict(const msa_shape *shape, int32_t keep, int32_t first, int32_t last,
                           const float *weights, const int32_t *block_table,
                           const int32_t *seq_lens, const int32_t *new_table, void *kv_pool,
                           void *idxk_pool, void *idxk_scales, float *new_weights, int32_t *kept,
                           int32_t *new_lens, void *workspace, size_t workspace_bytes,
                           cudaStream_t stream)
{
    msa_status st = check_cache_shape(shape);
    if (st != MSA_OK)
        return st;
    const bool idx_f4 = idxk_pool && shape->index_dtype == MSA_NVFP4;
    if (idxk_pool && (shape->index_dim != kDim || (shape->index_dtype != MSA_BF16 && !idx_f4)))
        return MSA_ERR_UNSUPPORTED;
    // the step's own tokens stay (their queries see one another by position)
    if (keep < 1 || keep < shape->q_per_req || first < 0 || last < shape->q_per_req - 1 ||
        (long long)first + last > keep)
        return MSA_ERR_INVALID_ARGUMENT;
    if (keep > kMaxBlocks * kPage)
        return MSA_ERR_UNSUPPORTED;
    if ((st = check_workspace(shape, workspace, workspace_bytes)) != MSA_OK)
        return st;
    // lists are copied while others are still read: the new pages are other pages
    if (!weights || !block_table || !seq_lens || !new_table || !kv_pool || !kept || !new_lens ||
        (idx_f4 && !idxk_scales) || new_table == block_table || new_weights == weights ||
        new_lens == seq_lens)
        return MSA_ERR_INVALID_ARGUMENT;
    if (!aligned16(weights) || !aligned16(block_table) || !aligned16(seq_lens) || !aligned16(new_table) ||
        !aligned16(kv_pool) || !aligned16(idxk_pool) || !aligned16(idxk_scales) || !aligned16(new_weights) ||
        !aligned16(kept) || !aligned16(new_lens))
        return MSA_ERR_INVALID_ARGUMENT;
    if (shape->num_requests == 0)
        return MSA_OK;
    EvictParams p;
    p.weights = weights;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.new_table = new_table;
    p.kv = static_cast<uint8_t *>(kv_pool);
    p.idxk = static_cast<uint8_t *>(idxk_pool);
    p.idxk_scales = static_cast<uint8_t *>(idxk_scales);
    p.new_weights = new_weights;
    p.kept = kept;
    p.new_lens = new_lens;
    p.err = static_cast<uint32_t *>(workspace);
    p.R = shape->num_requests;
    p.nq = shape->q_per_req;
    p.Hkv = shape->num_kv_heads;
    p.Hi = shape->num_index_heads;
    p.Hs = p.Hi == 1 ? 1 : p.Hkv;
    p.maxB = shape->max_blocks_per_seq;
    p.newB = (keep + kPage - 1) / kPage;
    p.num_pages = shape->num_pages;
    p.keep = keep;
    p.first = first;
    p.last = last;
    p.kv_fmt = shape->kv_dtype == MSA_BF16 ? kFmtBf16 : shape->kv_dtype == MSA_FP8_E4M3 ? kFmtFp8 : kFmtF4;
    p.idx_f4 = idx_f4;
    return cuda_status(launch_cache_evict(p, stream));
}

} // extern "C"
