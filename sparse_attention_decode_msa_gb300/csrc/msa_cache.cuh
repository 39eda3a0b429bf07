// msa_cache.cuh -- shared parts of the whole-cache operators (dense decode,
// accumulated attention weights, eviction): parameters, the page ring's tile
// formats, and the loads that turn a staged K or V tile of any pool format
// into mma.sync fragments.
//
// Fragment layouts (m16n8k16, lane = 4 n + c): an S tile has 16 query rows x
// 8 positions, A = Q, B = K; an O tile has 16 query rows x 8 dimensions,
// A = P, B = V.  The order of the contraction index is free as long as A and
// B agree on it, and so is the order of an output tile's columns: 8-bit and
// 4-bit rows use the orders in which ldmatrix delivers their bytes, so that
// widening a register gives whole fragments without moving data between lanes.
//   format   K: dims of k-step ks held by lane c        O: dim of (tile, column)
//   bf16     16 ks + {2c, 2c+1, 2c+8, 2c+9}             8 nt + col
//   E4M3     16 ks + 4c + {0..3}                        16 (nt/2) + 2 col + nt%2
//   NVFP4    32 (ks/2) + 8c + 4 (ks%2) + {0..3}         32 (nt/4) + 4 col + nt%4
#pragma once

#include "msa_internal.cuh"

namespace msa {

constexpr int kMaxGroup = 64;      // query heads per KV head of the whole-cache operators
constexpr int kMaxKvHeads = 8192;  // list counts and a page's 16-byte pieces stay in int32
constexpr int kCacheCtaBound = 160; // workspace bound on the default persistent CTAs

// KV formats of the kernel instances
constexpr int kFmtBf16 = 0, kFmtFp8 = 1, kFmtF4 = 2;

struct CacheParams {
    const uint16_t *q; // bf16 bits [T][Hq][D]
    const int32_t *block_table;
    const int32_t *seq_lens;
    const uint8_t *kv; // the pool (bulk copies of NVFP4 scales)
    uint32_t *err;
    int R, nq, Hkv, G, maxB, num_pages;
    float scale_log2; // softmax_scale * log2(e) (* k_scale where keys are scaled)
    long long wait_limit;
};

struct DenseParams : CacheParams {
    uint16_t *out;   // bf16 bits [T][Hq][D]
    float *lse;      // [T][Hq]
    float *partial;  // 2 slots per CTA: o[rows][128], m[rows], l[rows]
    int4 *joins;     // one record per CTA: the split unit whose first cut is that CTA's start
    float v_scale;
    int rows, tiles; // query rows of a (request, KV head) and their row tiles
};

struct WeightParams : CacheParams {
    const float *lse;         // [T][Hq]
    const int32_t *selected;  // [T][Hs][k] or nullptr
    const float *weights_in;  // [R][Hkv][maxB * 128] or nullptr
    float *weights_out;
    float decay;
    int Hs, k;
};

struct EvictParams {
    const float *weights;      // [R][Hkv][maxB * 128]
    const int32_t *block_table;
    const int32_t *seq_lens;
    const int32_t *new_table;  // [R][newB]
    uint8_t *kv, *idxk, *idxk_scales;
    float *new_weights;        // [R][Hkv][newB * 128] or nullptr
    int32_t *kept;             // [R][Hs][keep]
    int32_t *new_lens;
    uint32_t *err;
    int R, nq, Hkv, Hi, Hs, maxB, newB, num_pages;
    int keep, first, last;
    int kv_fmt;
    bool idx_f4;
};

cudaError_t launch_dense_decode(const DenseParams &p, int kv_dtype, int ctas, cudaStream_t stream);
// Units of more than 16 query rows, on the tcgen05 tensor cores (the join is the caller's).
cudaError_t launch_dense_umma(const DenseParams &p, const CUtensorMap &map, int kv_dtype, int ctas, cudaStream_t stream);
cudaError_t launch_weight_accumulate(const WeightParams &p, int kv_dtype, int ctas,
                                     cudaStream_t stream);
cudaError_t launch_cache_evict(const EvictParams &p, cudaStream_t stream);

// Query rows of one tile of the dense decode, and the bytes of one partial slot.
int dense_tile_rows(int rows);
constexpr size_t dense_slot_floats(int tile_rows)
{
    return (size_t)tile_rows * (kDim + 2);
}

// Bytes of a K or V tile in the page ring.
__host__ __device__ constexpr int tile_bytes(int fmt)
{
    return fmt == kFmtBf16 ? 32768 : fmt == kFmtFp8 ? 16384 : 9216;
}

// Tensor map of the KV pool for tile copies: bf16 boxes of 64 dims x 128 rows
// and E4M3 boxes of 128 x 128 (128-byte swizzle); NVFP4 tiles seen as 144 rows
// of 64 bytes, 128 of codes (one box, 64-byte swizzle) and 16 of scales.
inline bool encode_pool_map(CUtensorMap *map, const void *kv, int kv_dtype, int num_pages, int Hkv)
{
    const uint64_t tiles = (uint64_t)num_pages * 2 * Hkv;
    if (kv_dtype == MSA_BF16)
        return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kv, kDim, tiles * kPage, kDim * 2,
                         64, kPage, CU_TENSOR_MAP_SWIZZLE_128B);
    if (kv_dtype == MSA_FP8_E4M3)
        return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, kv, kDim, tiles * kPage, kDim, kDim,
                         kPage, CU_TENSOR_MAP_SWIZZLE_128B);
    return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, kv, 64, tiles * 144, 64, 64, kPage,
                     CU_TENSOR_MAP_SWIZZLE_64B);
}

#ifdef __CUDACC__

// Cached blocks of request r: 0 for an idle slot (seq_len 0) and, reported in
// *bad, for a length the block table cannot hold.
__device__ __forceinline__ int cached_blocks(int seq_len, int nq, int maxB, bool *bad)
{
    *bad = false;
    if (seq_len == 0)
        return 0;
    const long long nb = ((long long)seq_len + nq - 1 + kPage - 1) / kPage;
    if (seq_len < 0 || nb > maxB) {
        *bad = true;
        return 0;
    }
    return (int)nb;
}

__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}

static __device__ __noinline__ bool ring_wait_slow(uint32_t bar, uint32_t parity, const volatile int *abort_flag, long long limit)
{
    const bool poll = limit < (1 << 16); // a test's limit: the suspending form may sleep past it
    const long long start = clock64();
    while (!(poll ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))) {
        if (*abort_flag || clock64() - start > limit)
            return false;
    }
    return true;
}

// Wait for phase `parity` of a ring barrier; false after `limit` SM clocks or
// once another thread of the CTA gave up.  The waiting itself is a call: the
// roles of these kernels share the instruction caches, and a dozen inlined wait
// loops push their inner loops out.
__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, const volatile int *abort_flag, long long limit)
{
    return mbar_test_wait(bar, parity) || ring_wait_slow(bar, parity, abort_flag, limit);
}

// Copy tile (page, kv, g) into the ring (one thread; `bytes` already expected).
template <int FMT>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, const uint8_t *kv_pool,
                                          long long tile, uint32_t bar)
{
    if (FMT == kFmtBf16) {
        tma_load_2d(dst, map, 0, (int)(tile * kPage), bar);
        tma_load_2d(dst + 16384, map, 64, (int)(tile * kPage), bar);
    } else if (FMT == kFmtFp8) {
        tma_load_2d(dst, map, 0, (int)(tile * kPage), bar);
    } else {
        tma_load_2d(dst, map, 0, (int)(tile * 144), bar);
        bulk_load(dst + 8192, kv_pool + tile * 9216 + 8192, 1024, bar);
    }
}

__device__ __forceinline__ uint64_t lds64(uint32_t a)
{
    uint64_t v;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(a));
    return v;
}

// E4M3 bytes i and j of the 8 scales in w, as an f16 pair.
__device__ __forceinline__ uint32_t scale_pair(uint32_t wi, int i, uint32_t wj, int j)
{
    return e4m3x2_to_f16x2(__byte_perm(wi, wj, (uint32_t)(i & 3) | (uint32_t)(4 + (j & 3)) << 4) & 0xFFFFu);
}

// Scales of this lane's two K rows (positions pos0 + n and pos0 + 8 + n): word
// kk of s[t] is the f16 pair (s, s) of 32-dim chunk kk, for the lane's half of it.
__device__ __forceinline__ void load_k_scales(uint32_t tile, int pos0, uint32_t (&s)[2][4])
{
    const int lane = threadIdx.x & 31, odd = (lane >> 1) & 1;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const uint64_t w = lds64(tile + 8192 + (pos0 + 8 * t + (lane >> 2)) * 8);
        const uint32_t lo = (uint32_t)w, hi = (uint32_t)(w >> 32);
        const uint32_t sel = odd ? 0x31u : 0x20u;
        const uint32_t a = e4m3x2_to_f16x2(__byte_perm(lo, 0, sel) & 0xFFFFu);
        const uint32_t b = e4m3x2_to_f16x2(__byte_perm(hi, 0, sel) & 0xFFFFu);
        s[t][0] = __byte_perm(a, a, 0x1010);
        s[t][1] = __byte_perm(a, a, 0x3232);
        s[t][2] = __byte_perm(b, b, 0x1010);
        s[t][3] = __byte_perm(b, b, 0x3232);
    }
}

// S += Q K^T for positions pos0 .. pos0 + 15 of the staged K tile: s[t] is the
// n-tile of positions pos0 + 8 t ...  Two accumulators per n-tile (even and
// odd k-steps) halve the chain of dependent MMAs.
template <int FMT>
__device__ __forceinline__ void score16(float (&s)[2][4], const uint32_t (&q)[8][4], uint32_t tile, int pos0)
{
    const int lane = threadIdx.x & 31, mi = lane >> 3;
    float e[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s[t][i] = 0.f;
    if (FMT == kFmtBf16) {
        const int row = pos0 + (lane & 7) + (mi >> 1) * 8;
        const uint32_t base = tile + row * 128;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            uint32_t b[4];
            const int chunk = 2 * (ks & 3) + (mi & 1);
            ldsm_x4(b, base + (ks >> 2) * 16384 + ((chunk ^ (row & 7)) << 4));
            mma_bf16(ks & 1 ? e[0] : s[0], q[ks], b[0], b[1]);
            mma_bf16(ks & 1 ? e[1] : s[1], q[ks], b[2], b[3]);
        }
    } else if (FMT == kFmtFp8) {
        const int row = pos0 + (lane & 7) + (mi & 1) * 8;
        const uint32_t base = tile + row * 128;
#pragma unroll
        for (int k2 = 0; k2 < 4; ++k2) {
            uint32_t b[4], x0, x1;
            const int chunk = 2 * k2 + (mi >> 1);
            ldsm_x4(b, base + ((chunk ^ (row & 7)) << 4));
            e4m3x4_to_f16x2x2(b[0], x0, x1);
            mma_f16(s[0], q[2 * k2], x0, x1);
            e4m3x4_to_f16x2x2(b[1], x0, x1);
            mma_f16(s[1], q[2 * k2], x0, x1);
            e4m3x4_to_f16x2x2(b[2], x0, x1);
            mma_f16(e[0], q[2 * k2 + 1], x0, x1);
            e4m3x4_to_f16x2x2(b[3], x0, x1);
            mma_f16(e[1], q[2 * k2 + 1], x0, x1);
        }
    } else {
        const int row = pos0 + (lane & 7) + (mi & 1) * 8;
        const uint32_t base = tile + row * 64;
        uint32_t sc[2][4];
        load_k_scales(tile, pos0, sc);
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
            uint32_t b[4];
            const int chunk = 2 * k2 + (mi >> 1);
            ldsm_x4(b, base + ((chunk ^ ((row >> 1) & 3)) << 4));
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uint32_t x[4];
                    e2m1x8_scaled_f16x2(b[2 * h + t], sc[t][2 * k2 + h], x);
                    mma_f16(s[t], q[4 * k2 + 2 * h], x[0], x[1]);
                    mma_f16(e[t], q[4 * k2 + 2 * h + 1], x[2], x[3]);
                }
        }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s[t][i] += e[t][i];
}

// Query rows (bf16) of one 16-row tile as A fragments: row0 / row1 point at the
// lane's rows n and n + 8 (nullptr: a row of zeros).  8-bit and 4-bit keys
// multiply in f16: each query row is first scaled by a power of two that
// brings its largest element to [2^8, 2^9) (exact; elements 2^-23 below it
// lose bits), and inv0 / inv1 undo it in the logits.
template <int FMT>
__device__ __forceinline__ void load_queries(uint32_t (&q)[8][4], const uint16_t *row0, const uint16_t *row1,
                                             float &inv0, float &inv1)
{
    const int c = threadIdx.x & 3;
    inv0 = inv1 = 1.f;
    if (FMT == kFmtBf16) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            q[ks][0] = row0 ? *reinterpret_cast<const uint32_t *>(row0 + 16 * ks + 2 * c) : 0u;
            q[ks][1] = row1 ? *reinterpret_cast<const uint32_t *>(row1 + 16 * ks + 2 * c) : 0u;
            q[ks][2] = row0 ? *reinterpret_cast<const uint32_t *>(row0 + 16 * ks + 2 * c + 8) : 0u;
            q[ks][3] = row1 ? *reinterpret_cast<const uint32_t *>(row1 + 16 * ks + 2 * c + 8) : 0u;
        }
        return;
    }
    float mx[2] = {0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
        const int d = FMT == kFmtFp8 ? 16 * ks + 4 * c : 32 * (ks >> 1) + 8 * c + 4 * (ks & 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint16_t *row = h ? row1 : row0;
            const uint2 v = row ? *reinterpret_cast<const uint2 *>(row + d) : make_uint2(0u, 0u);
            q[ks][h] = v.x;
            q[ks][2 + h] = v.y;
            const float m = fmaxf(fmaxf(fabsf(__uint_as_float(v.x << 16)), fabsf(__uint_as_float(v.x & 0xFFFF0000u))),
                                  fmaxf(fabsf(__uint_as_float(v.y << 16)), fabsf(__uint_as_float(v.y & 0xFFFF0000u))));
            mx[h] = fmaxf(mx[h], m);
        }
    }
    float up[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        // 2^(8 - exponent) with the exponent clamped so that neither it nor its inverse overflows
        int e = (int)(__float_as_uint(mx[h]) >> 23) - 127;
        e = e < -100 ? -100 : e > 127 ? 127 : e;
        up[h] = __uint_as_float((uint32_t)(8 - e + 127) << 23);
        (h ? inv1 : inv0) = __uint_as_float((uint32_t)(e - 8 + 127) << 23);
    }
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = q[ks][i];
            const float s = up[i & 1];
            q[ks][i] = pack_f16(__uint_as_float(v << 16) * s, __uint_as_float(v & 0xFFFF0000u) * s);
        }
}

// CTA-wide: exclusive prefix (in blocks) of this thread's share of the
// requests [lo, hi) and the total.  `tmp` holds blockDim / 32 + 1 ints.
__device__ __forceinline__ int scan_blocks(const CacheParams &p, int lo, int hi, int *tmp, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    int sum = 0;
    for (int r = lo; r < hi; ++r) {
        bool bad;
        sum += cached_blocks(p.seq_lens[r], p.nq, p.maxB, &bad);
        if (bad && blockIdx.x == 0)
            set_error(p.err, kErrSeqLen);
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += v;
    }
    if (lane == 31)
        tmp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int w = lane < nwarps ? tmp[lane] : 0;
        int wi = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, wi, o);
            if (lane >= o)
                wi += v;
        }
        if (lane < nwarps)
            tmp[lane] = wi - w;
        if (lane == nwarps - 1)
            tmp[nwarps] = wi;
    }
    __syncthreads();
    *total = tmp[nwarps];
    return tmp[warp] + incl - sum;
}

// W tasks cut into n equal ranges (the first W % n one longer): start of range c,
// and the range that holds task x.
__device__ __forceinline__ int range_start(int c, int W, int n)
{
    const int each = W / n, more = W - each * n;
    return c * each + min(c, more);
}

__device__ __forceinline__ int range_of(int x, int W, int n)
{
    const int each = W / n, more = W - each * n;
    const int cut = more * (each + 1);
    return x < cut ? x / (each + 1) : more + (x - cut) / each;
}

#endif // __CUDACC__

} // namespace msa
