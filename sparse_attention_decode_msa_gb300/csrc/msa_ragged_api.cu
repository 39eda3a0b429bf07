// msa_ragged_api.cu -- the C ABI of the calls on ragged batches (msa_rope_frequencies,
// msa_qk_norm_rope, msa_kv_append, msa_ragged_attention): host-side validation and launches.  No
// allocation, no state between calls.
#include <cmath>

#include "msa_ragged.cuh"

namespace msa {
namespace {

constexpr size_t kAlign = 256;

bool aligned16(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

msa_status cuda_status(cudaError_t e)
{
    return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

// The shape rules of these operators: those of the whole cache, without a number
// of tokens a request.
msa_status check_ragged_shape(const msa_shape *s)
{
    if (!s)
        return MSA_ERR_INVALID_ARGUMENT;
    if (s->num_requests < 0 || s->num_kv_heads < 1 || s->num_q_heads < 1 || s->num_pages < 1 ||
        s->max_blocks_per_seq < 1 || s->decode_ctas < 0 || s->num_index_heads < 1)
        return MSA_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(s->softmax_scale) || !std::isfinite(s->k_scale) || !std::isfinite(s->v_scale))
        return MSA_ERR_INVALID_ARGUMENT;
    if (s->head_dim != kDim || s->page_size != kPage || s->num_q_heads % s->num_kv_heads != 0 ||
        s->num_q_heads / s->num_kv_heads > kMaxGroup || s->num_kv_heads > kMaxKvHeads)
        return MSA_ERR_UNSUPPORTED;
    if (s->num_index_heads > kMaxIndexHeads || s->num_requests > kMaxRequests ||
        s->max_blocks_per_seq > kMaxBlocks || s->decode_ctas > kMaxTokens)
        return MSA_ERR_UNSUPPORTED;
    if (s->kv_dtype != MSA_BF16 && s->kv_dtype != MSA_FP8_E4M3 && s->kv_dtype != MSA_NVFP4)
        return MSA_ERR_UNSUPPORTED;
    // row coordinates of the KV tensor map (144 rows a tile at most) fit in int32
    if ((long long)s->num_pages * 2 * s->num_kv_heads * 144 > 0x7FFFFFFFll)
        return MSA_ERR_UNSUPPORTED;
    return MSA_OK;
}

msa_status check_rope(const msa_rope *r, const uint64_t *freqs)
{
    if (!r || r->rotary_dim < 0 || !std::isfinite(r->scale) || !std::isfinite(r->norm_offset) ||
        !std::isfinite(r->norm_eps) || r->norm_eps < 0.f)
        return MSA_ERR_INVALID_ARGUMENT;
    if (r->rotary_dim > kDim || r->rotary_dim % 16 != 0)
        return MSA_ERR_UNSUPPORTED;
    if (r->rotary_dim > 0 && (!freqs || !aligned16(freqs)))
        return MSA_ERR_INVALID_ARGUMENT;
    return MSA_OK;
}

// One kind of rows: pointers, alignment, the stride between tokens, and rows that
// are written over their input only where they lie the same.
msa_status add_set(AppendParams &p, const void *x, int64_t stride, const void *weight, void *y, int heads, int where, bool rotated)
{
    const int64_t dense = (int64_t)heads * kDim, by = stride == 0 ? dense : stride;
    if (!x || !aligned16(x) || !aligned16(weight) || !aligned16(y) || (where == kToOut && !y) || by < dense || by % 8 != 0 ||
        (x == y && by != dense))
        return MSA_ERR_INVALID_ARGUMENT;
    RowSet &s = p.set[p.sets++];
    s.x = static_cast<const uint16_t *>(x);
    s.weight = static_cast<const uint16_t *>(weight);
    s.y = static_cast<uint8_t *>(y);
    s.scales = nullptr;
    s.stride = by;
    s.bytes = s.head_step = 2 * kDim;
    s.block_step = (long long)heads * s.head_step;
    s.scales_head_step = 0;
    s.scales_block_step = 0;
    s.scale = s.inverse = 1.f;
    s.heads = heads;
    s.group0 = p.groups;
    s.where = where;
    s.rotated = rotated;
    p.groups += (heads + 3) / 4;
    return MSA_OK;
}

void set_rope(AppendParams &p, const msa_rope *r, const uint64_t *freqs)
{
    p.freqs = reinterpret_cast<const unsigned long long *>(freqs);
    p.units = r->rotary_dim / 16;
    p.interleaved = r->interleaved != 0;
    p.per_head = r->per_head_weights != 0;
    p.scale = r->scale;
    p.eps = r->norm_eps;
    p.offset = r->norm_offset;
}

// 1 / s where a product with it is the quotient by s: s a power of two.
float exact_inverse(float s)
{
    int e;
    const float m = std::frexp(std::fabs(s), &e);
    return m == 0.5f && e > -120 && e < 120 ? 1.f / s : 0.f;
}

// The set added last goes to head tiles of kPage rows of a pool, from tile `first` of a page's `tiles` on:
// codes and scales of a tile together (scales == nullptr) or in two pools.
void to_pool(AppendParams &p, void *pool, void *scales, int dtype, int first, int tiles, float scale)
{
    RowSet &s = p.set[p.sets - 1];
    s.bytes = dtype == MSA_BF16 ? 2 * kDim : dtype == MSA_FP8_E4M3 ? kDim : kDim / 2;
    const bool f4 = dtype == MSA_NVFP4;
    s.head_step = kPage * s.bytes + (f4 && !scales ? kPage * (kDim / 16) : 0);
    s.block_step = (long long)tiles * s.head_step;
    s.y = static_cast<uint8_t *>(pool) + (long long)first * s.head_step;
    if (f4) {
        s.scales_head_step = scales ? kPage * (kDim / 16) : s.head_step;
        s.scales_block_step = (long long)tiles * s.scales_head_step;
        s.scales = scales ? static_cast<uint8_t *>(scales) + (long long)first * s.scales_head_step : s.y + kPage * s.bytes;
    }
    s.scale = scale;
    s.inverse = exact_inverse(scale);
}

struct RaggedLayout {
    size_t joins_off, partial_off, total;
};

RaggedLayout layout_of(const msa_shape *s)
{
    const size_t ctas = s->decode_ctas > 0 ? s->decode_ctas : kCacheCtaBound;
    RaggedLayout w;
    w.joins_off = kAlign; // after the error word
    w.partial_off = align_to(w.joins_off + ctas * sizeof(AttendJoin), kAlign);
    w.total = align_to(w.partial_off + 2 * ctas * attend_slot_bytes(), kAlign);
    return w;
}

// Persistent CTAs: the shape's, else one per SM; below 1 if the device cannot be read.
int attend_ctas(const msa_shape *s)
{
    if (s->decode_ctas > 0)
        return s->decode_ctas;
    const int sms = device_sms();
    return sms < kCacheCtaBound ? sms : kCacheCtaBound;
}

} // namespace

int device_sms()
{
    int dev = 0, sms = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? sms : -1;
}

} // namespace msa

using namespace msa;

extern "C" {

msa_status msa_rope_frequencies(const double *radians, int32_t count, uint64_t *turns)
{
    if (count < 0 || (count > 0 && (!radians || !turns)))
        return MSA_ERR_INVALID_ARGUMENT;
    for (int32_t i = 0; i < count; ++i) {
        const double t = std::fabs(radians[i]) * 0.15915494309189533577; // 1 / (2 pi)
        if (!(t < 2147483648.0))
            return MSA_ERR_INVALID_ARGUMENT;
        const uint64_t u = static_cast<uint64_t>(std::ldexp(t - std::floor(t), 64)); // (the difference is exact)
        turns[i] = radians[i] < 0.0 ? 0u - u : u; // a negative one modulo a turn
    }
    return MSA_OK;
}

msa_status msa_qk_norm_rope(const msa_rope *rope, const uint64_t *freqs, int32_t num_tokens,
                            const int32_t *positions, int32_t num_q_heads, const void *q,
                            const void *q_weight, void *q_out, int32_t num_k_heads, const void *k,
                            const void *k_weight, void *k_out, cudaStream_t stream)
{
    msa_status st = check_rope(rope, freqs);
    if (st != MSA_OK)
        return st;
    if (num_tokens < 0 || num_q_heads < 1 || num_k_heads < 0)
        return MSA_ERR_INVALID_ARGUMENT;
    if (num_q_heads > kMaxKvHeads || num_k_heads > kMaxKvHeads || num_tokens > kMaxRows)
        return MSA_ERR_UNSUPPORTED;
    if (num_tokens == 0) // rows without elements may have no address
        return MSA_OK;
    if (!positions || !aligned16(positions))
        return MSA_ERR_INVALID_ARGUMENT;
    AppendParams p{};
    set_rope(p, rope, freqs);
    const bool turn = p.units > 0;
    if ((st = add_set(p, q, rope->q_stride, q_weight, q_out, num_q_heads, kToOut, turn)) != MSA_OK)
        return st;
    if (num_k_heads == 0 ? k || k_out
                         : (st = add_set(p, k, rope->k_stride, k_weight, k_out, num_k_heads, kToOut, turn)) != MSA_OK)
        return MSA_ERR_INVALID_ARGUMENT;
    p.positions = positions;
    p.T = num_tokens;
    return cuda_status(launch_append(p, stream));
}

size_t msa_ragged_workspace_bytes(const msa_shape *shape)
{
    return check_ragged_shape(shape) == MSA_OK ? layout_of(shape).total : 0;
}

msa_status msa_kv_append(const msa_shape *shape, const msa_rope *rope, const uint64_t *freqs,
                         int32_t num_tokens, const int32_t *offsets, const void *k,
                         const void *k_weight, const void *v, const void *idxk,
                         const void *idxk_weight, const void *q, const void *q_weight, void *q_out,
                         const void *q_idx, const void *q_idx_weight, void *q_idx_out,
                         const int32_t *block_table, const int32_t *seq_lens, void *kv_pool,
                         void *idxk_pool, void *idxk_scales, void *workspace,
                         size_t workspace_bytes, cudaStream_t stream)
{
    msa_status st = check_ragged_shape(shape);
    if (st != MSA_OK || (st = check_rope(rope, freqs)) != MSA_OK)
        return st;
    const bool idx_f4 = idxk && shape->index_dtype == MSA_NVFP4;
    if ((idxk || q_idx) && (shape->index_dim != kDim || (shape->index_dtype != MSA_BF16 && shape->index_dtype != MSA_NVFP4)))
        return MSA_ERR_UNSUPPORTED;
    if (num_tokens > kMaxRows)
        return MSA_ERR_UNSUPPORTED;
    if (num_tokens == 0 || shape->num_requests == 0) // rows without elements may have no address
        return MSA_OK;
    if (num_tokens < 0 || !offsets || !block_table || !seq_lens || !kv_pool || !workspace || workspace_bytes < kAlign)
        return MSA_ERR_INVALID_ARGUMENT;
    if (!aligned16(offsets) || !aligned16(block_table) || !aligned16(seq_lens) || !aligned16(kv_pool) ||
        !aligned16(idxk_pool) || !aligned16(idxk_scales) || !aligned16(workspace))
        return MSA_ERR_INVALID_ARGUMENT;
    if ((idxk && !idxk_pool) || (idx_f4 && !idxk_scales) || !q != !q_out || !q_idx != !q_idx_out)
        return MSA_ERR_INVALID_ARGUMENT;
    AppendParams p{};
    set_rope(p, rope, freqs);
    const bool turn = p.units > 0;
    const int Hkv = shape->num_kv_heads, Hi = shape->num_index_heads;
    if (q && (st = add_set(p, q, rope->q_stride, q_weight, q_out, shape->num_q_heads, kToOut, turn)) != MSA_OK)
        return st;
    if (q_idx && (st = add_set(p, q_idx, rope->q_idx_stride, q_idx_weight, q_idx_out, Hi, kToOut, turn)) != MSA_OK)
        return st;
    if ((st = add_set(p, k, rope->k_stride, k_weight, nullptr, Hkv, kToK, turn)) != MSA_OK)
        return st;
    to_pool(p, kv_pool, nullptr, shape->kv_dtype, 0, 2 * Hkv, shape->kv_dtype == MSA_BF16 ? 1.f : shape->k_scale);
    if ((st = add_set(p, v, rope->v_stride, nullptr, nullptr, Hkv, kToV, false)) != MSA_OK)
        return st;
    to_pool(p, kv_pool, nullptr, shape->kv_dtype, Hkv, 2 * Hkv, shape->kv_dtype == MSA_BF16 ? 1.f : shape->v_scale);
    if (idxk) {
        if ((st = add_set(p, idxk, rope->idxk_stride, idxk_weight, nullptr, Hi, kToIndex, turn)) != MSA_OK)
            return st;
        to_pool(p, idxk_pool, idxk_scales, shape->index_dtype, 0, Hi, 1.f);
    }
    p.offsets = offsets;
    p.seq_lens = seq_lens;
    p.block_table = block_table;
    p.err = static_cast<uint32_t *>(workspace);
    p.T = num_tokens;
    p.R = shape->num_requests;
    p.maxB = shape->max_blocks_per_seq;
    p.num_pages = shape->num_pages;
    return cuda_status(launch_append(p, stream));
}

msa_status msa_ragged_attention(const msa_shape *shape, int32_t num_tokens, int32_t causal,
                                const void *q, const int32_t *offsets, const void *kv_pool,
                                const int32_t *block_table, const int32_t *seq_lens, void *out,
                                float *lse, void *workspace, size_t workspace_bytes,
                                cudaStream_t stream)
{
    msa_status st = check_ragged_shape(shape);
    if (st != MSA_OK)
        return st;
    if (num_tokens < 0)
        return MSA_ERR_INVALID_ARGUMENT;
    if (num_tokens > kMaxRows)
        return MSA_ERR_UNSUPPORTED;
    if (num_tokens == 0 || shape->num_requests == 0) // rows without elements may have no address
        return MSA_OK;
    const RaggedLayout w = layout_of(shape);
    if (!q || !offsets || !kv_pool || !block_table || !seq_lens || !out || !lse || !workspace || workspace_bytes < w.total)
        return MSA_ERR_INVALID_ARGUMENT;
    if (!aligned16(q) || !aligned16(offsets) || !aligned16(kv_pool) || !aligned16(block_table) || !aligned16(seq_lens) ||
        !aligned16(out) || !aligned16(lse) || !aligned16(workspace))
        return MSA_ERR_INVALID_ARGUMENT;
    const int ctas = attend_ctas(shape);
    if (ctas < 1)
        return MSA_ERR_CUDA;
    // a CTA counts the pages of its range in int32, each unit with a few more for its queries and outputs
    const long long units = num_tokens / 4 + shape->num_requests; // at least 4 tokens a unit, but the last of a request
    if ((double)units * shape->num_kv_heads * (shape->max_blocks_per_seq + 8.0) / ctas > 2147483000.0)
        return MSA_ERR_UNSUPPORTED;
    AttendParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.kv = static_cast<const uint8_t *>(kv_pool);
    p.err = static_cast<uint32_t *>(workspace);
    p.R = shape->num_requests;
    p.Hkv = shape->num_kv_heads;
    p.G = shape->num_q_heads / shape->num_kv_heads;
    p.maxB = shape->max_blocks_per_seq;
    p.num_pages = shape->num_pages;
    p.scale_log2 = shape->softmax_scale * 1.4426950408889634f * (shape->kv_dtype != MSA_BF16 ? shape->k_scale : 1.f);
    p.wait_limit = decode_wait_limit();
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.offsets = offsets;
    p.joins = reinterpret_cast<AttendJoin *>(static_cast<uint8_t *>(workspace) + w.joins_off);
    p.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + w.partial_off);
    p.v_scale = shape->kv_dtype != MSA_BF16 ? shape->v_scale : 1.f;
    p.T = num_tokens;
    p.causal = causal != 0;
    return cuda_status(launch_attend(p, shape->kv_dtype, ctas, stream));
}

} // extern "C"
