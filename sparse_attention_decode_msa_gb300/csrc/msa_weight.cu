// msa_weight.cu -- the attention weight accumulated per cached position
// (msa_weight_accumulate):
//
//   w'[r][g][p] = decay w[r][g][p] + sum_{j, h in group g} exp(scale q_jh . K[p] - lse_jh)
//
// over the query rows (tokens j, heads h) that see position p, or whose
// selected blocks hold it; w[r][g][p] counts as 0 at the positions of this
// step's own tokens.  With the log-sum-exp of the step's attention the
// probabilities need no second softmax: one read of K, no V.
//
// What bounds it: the bytes of K and of the weights with few rows, the
// exponentials (16 a clock and SM) with many.  Layout: K tiles are B
// fragments, 16 positions per warp, kept in registers while the query rows
// pass by as A fragments staged once per (request, KV head) in shared memory;
// the sum over rows is then a sum over a lane's own accumulators and one
// reduction of 8 lanes per page.  Every element is written by one thread, in
// row order: no atomics.
//
// After a sparse step only pages that some token of the request selected are
// read; a bitmap of 64 token bits per page, built in shared memory, says which
// rows count.  The weights of the other pages are only faded.
#include "msa_cache.cuh"

namespace msa {
namespace {

constexpr int kConsumers = 8;
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kQTiles = 16;     // 16-row query tiles staged at a time (256 rows, 64 KiB)
constexpr int kPagesAtATime = 512; // pages whose token masks are held at a time

__host__ __device__ constexpr int ring_stages(int fmt)
{
    return fmt == kFmtBf16 ? 4 : fmt == kFmtFp8 ? 8 : 14;
}

struct Smem {
    int ring, q, rows, mask, bars, misc, total;
};

__host__ __device__ constexpr Smem smem_layout(int fmt)
{
    Smem s{};
    s.ring = 0;
    s.q = ring_stages(fmt) * tile_bytes(fmt);
    s.rows = s.q + kQTiles * 4096;           // float4 per row: logit scale, lse, token
    s.mask = s.rows + kQTiles * 16 * 16;     // uint64 per page
    s.bars = s.mask + kPagesAtATime * 8;
    s.misc = s.bars + 2 * ring_stages(fmt) * 8;
    s.total = s.misc + 64 + 1024;
    return s;
}

// K fragments of 16 positions, all 8 k-steps: {tile 0: b0, b1, tile 1: b0, b1}.
template <int FMT>
__device__ __forceinline__ void load_keys(uint32_t (&kb)[8][4], uint32_t tile, int pos0)
{
    const int lane = threadIdx.x & 31, mi = lane >> 3;
    if (FMT == kFmtBf16) {
        const int row = pos0 + (lane & 7) + (mi >> 1) * 8;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            const int chunk = 2 * (ks & 3) + (mi & 1);
            ldsm_x4(kb[ks], tile + row * 128 + (ks >> 2) * 16384 + ((chunk ^ (row & 7)) << 4));
        }
    } else if (FMT == kFmtFp8) {
        const int row = pos0 + (lane & 7) + (mi & 1) * 8;
#pragma unroll
        for (int k2 = 0; k2 < 4; ++k2) {
            uint32_t b[4];
            const int chunk = 2 * k2 + (mi >> 1);
            ldsm_x4(b, tile + row * 128 + ((chunk ^ (row & 7)) << 4));
            e4m3x4_to_f16x2x2(b[0], kb[2 * k2][0], kb[2 * k2][1]);
            e4m3x4_to_f16x2x2(b[1], kb[2 * k2][2], kb[2 * k2][3]);
            e4m3x4_to_f16x2x2(b[2], kb[2 * k2 + 1][0], kb[2 * k2 + 1][1]);
            e4m3x4_to_f16x2x2(b[3], kb[2 * k2 + 1][2], kb[2 * k2 + 1][3]);
        }
    } else {
        const int row = pos0 + (lane & 7) + (mi & 1) * 8;
        uint32_t sc[2][4];
        load_k_scales(tile, pos0, sc);
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
            uint32_t b[4];
            const int chunk = 2 * k2 + (mi >> 1);
            ldsm_x4(b, tile + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uint32_t x[4];
                    e2m1x8_scaled_f16x2(b[2 * h + t], sc[t][2 * k2 + h], x);
                    kb[4 * k2 + 2 * h][2 * t] = x[0];
                    kb[4 * k2 + 2 * h][2 * t + 1] = x[1];
                    kb[4 * k2 + 2 * h + 1][2 * t] = x[2];
                    kb[4 * k2 + 2 * h + 1][2 * t + 1] = x[3];
                }
        }
    }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    weight_kernel(const __grid_constant__ CUtensorMap map, const WeightParams p)
{
    constexpr int STAGES = ring_stages(FMT), TB = tile_bytes(FMT);
    extern __shared__ uint8_t smem_raw[];
    __shared__ int scan_tmp[kThreads / 32 + 1];
    __shared__ int start_r, start_before;
    constexpr Smem L = smem_layout(FMT);
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t full = smem + L.bars, empty = full + STAGES * 8;
    uint8_t *gsm = smem_raw + (smem - smem_u32(smem_raw));
    uint4 *qf = reinterpret_cast<uint4 *>(gsm + L.q);         // [tile][k-step][lane]
    float4 *rows4 = reinterpret_cast<float4 *>(gsm + L.rows); // [row]
    unsigned long long *mask = reinterpret_cast<unsigned long long *>(gsm + L.mask);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gsm + L.misc);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n8 = lane >> 2, c4 = lane & 3;
    const int rows = p.nq * p.G;

    if (threadIdx.x == 0) {
        prefetch_tensormap(&map);
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, kConsumers);
        }
        fence_mbar_init();
        *abort_flag = 0;
    }
    const int per = (p.R + kThreads - 1) / kThreads;
    const int lo = min(p.R, (int)threadIdx.x * per), hi = min(p.R, lo + per);
    int total;
    const int before = scan_blocks(p, lo, hi, scan_tmp, &total);
    const int W = total * p.Hkv;
    const int x0 = range_start(blockIdx.x, W, gridDim.x), x1 = range_start(blockIdx.x + 1, W, gridDim.x);
    if (x0 == x1)
        return;
    for (int r = lo, b = before; r < hi; ++r) {
        bool bad;
        const int nb = cached_blocks(p.seq_lens[r], p.nq, p.maxB, &bad);
        if (nb > 0 && b * p.Hkv <= x0 && x0 < (b + nb) * p.Hkv) {
            start_r = r;
            start_before = b;
        }
        b += nb;
    }
    __syncthreads();
    bool bad;
    int r = start_r, seq_len = p.seq_lens[r];
    int nb = cached_blocks(seq_len, p.nq, p.maxB, &bad);
    const int in = x0 - start_before * p.Hkv;
    int g = in / nb, b = in - g * nb;

    int st = 0, issued = 0;
    uint32_t ph = 0;
    bool stop = false;
    for (int x = x0; x < x1;) {
        const int n = min(nb - b, x1 - x); // pages b .. b + n - 1 of (r, g)
        const size_t first_row = (size_t)r * p.nq * p.Hkv * p.G + (size_t)g * p.G;
        const size_t pitch = (size_t)p.Hkv * p.G;
        const size_t wrow = ((size_t)r * p.Hkv + g) * p.maxB * kPage;
        for (int q0 = 0; q0 < rows; q0 += 16 * kQTiles) {
            const int tiles = min(kQTiles, (rows - q0 + 15) / 16);
            for (int s0 = 0; s0 < n; s0 += kPagesAtATime) {
                const int sn = min(kPagesAtATime, n - s0), sb = b + s0;
                __syncthreads(); // the last pages' queries and masks are done with
                if (p.selected)
                    for (int i = threadIdx.x; i < sn; i += kThreads)
                        mask[i] = 0ull;
                if (s0 == 0)
                    for (int t = warp; t < tiles; t += kThreads / 32) {
                        const int i0 = q0 + 16 * t + n8, i1 = i0 + 8;
                        const int j0 = min(i0, rows - 1) / p.G, j1 = min(i1, rows - 1) / p.G;
                        const size_t a0 = first_row + j0 * pitch + (min(i0, rows - 1) - j0 * p.G);
                        const size_t a1 = first_row + j1 * pitch + (min(i1, rows - 1) - j1 * p.G);
                        uint32_t q[8][4];
                        float inv0, inv1;
                        // padding rows repeat the last row: zeros would turn an infinite key into NaN
                        load_queries<FMT>(q, p.q + a0 * kDim, p.q + a1 * kDim, inv0, inv1);
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            qf[(t * 8 + ks) * 32 + lane] = make_uint4(q[ks][0], q[ks][1], q[ks][2], q[ks][3]);
                        if (c4 == 0) {
                            // rows that count nothing (padding, or a token that attended to nothing:
                            // lse = -inf) get lse = +inf
                            const float inf = __uint_as_float(0x7F800000u);
                            float e0 = i0 < rows ? p.lse[a0] : inf, e1 = i1 < rows ? p.lse[a1] : inf;
                            e0 = e0 == -inf ? inf : e0 * 1.4426950408889634f;
                            e1 = e1 == -inf ? inf : e1 * 1.4426950408889634f;
                            rows4[16 * t + n8] = make_float4(p.scale_log2 * inv0, e0, __int_as_float(j0), 0.f);
                            rows4[16 * t + n8 + 8] = make_float4(p.scale_log2 * inv1, e1, __int_as_float(j1), 0.f);
                        }
                    }
                if (p.selected) {
                    __syncthreads();
                    // one bit per token for every page of [sb, sb + sn) in its table
                    for (int i = threadIdx.x; i < p.nq * p.k; i += kThreads) {
                        const int j = i / p.k;
                        const int blk = p.selected[(((size_t)r * p.nq + j) * p.Hs + (p.Hs > 1 ? g : 0)) * p.k + (i - j * p.k)];
                        if (blk < -1 || (blk >= 0 && (long long)blk * kPage >= seq_len + j))
                            set_error(p.err, kErrSelection);
                        else if (blk >= sb && blk < sb + sn)
                            atomicOr(&mask[blk - sb], 1ull << j);
                    }
                }
                __syncthreads();

                if (warp == kConsumers) {
                    const int32_t *row = p.block_table + (size_t)r * p.maxB;
                    for (int i = 0; i < sn && !stop; i += 32) {
                        const bool want = i + lane < sn && (!p.selected || mask[i + lane] != 0ull);
                        const int mine = want ? row[sb + i + lane] : 0;
                        uint32_t todo = __ballot_sync(0xffffffffu, want);
                        while (todo) {
                            const int k = __ffs(todo) - 1;
                            todo &= todo - 1;
                            long long page = __shfl_sync(0xffffffffu, mine, k);
                            if (page < 0 || page >= p.num_pages) {
                                if (lane == 0)
                                    set_error(p.err, kErrPage);
                                page = 0; // in the pool: the outputs of the call are unspecified
                            }
                            const bool ok = issued < STAGES ||
                                            ring_wait(empty + 8 * st, ph ^ 1u, abort_flag, p.wait_limit);
                            if (__any_sync(0xffffffffu, !ok)) {
                                *abort_flag = 1;
                                stop = true;
                                if (lane == 0)
                                    set_error(p.err, kErrTimeout);
                                break;
                            }
                            if (lane == 0) {
                                const uint32_t bar = full + 8 * st;
                                mbar_arrive_expect_tx(bar, TB);
                                load_tile<FMT>(smem + st * TB, &map, p.kv, (page * 2) * p.Hkv + g, bar);
                            }
                            __syncwarp();
                            ++issued;
                            if (++st == STAGES) {
                                st = 0;
                                ph ^= 1u;
                            }
                        }
                    }
                } else {
                    for (int i = 0; i < sn; ++i) {
                        const int page0 = (sb + i) * kPage;
                        const unsigned long long m = p.selected ? mask[i] : ~0ull;
                        if (m == 0ull) { // no row looks at this page: its weights fade
                            if ((i & 7) == warp && q0 == 0) {
                                const size_t at = wrow + page0 + 4 * lane;
                                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                                if (p.weights_in)
                                    v = *reinterpret_cast<const float4 *>(p.weights_in + at);
                                float e[4] = {v.x * p.decay, v.y * p.decay, v.z * p.decay, v.w * p.decay};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const int pos = page0 + 4 * lane + k;
                                    if (pos < seq_len + p.nq - 1)
                                        p.weights_out[at + k] = pos < seq_len - 1 ? e[k] : 0.f;
                                }
                            }
                            continue;
                        }
                        // this warp's 16 positions: lanes of the first row write two pairs
                        const int pos = 16 * warp + 2 * c4;
                        float old[4] = {0.f, 0.f, 0.f, 0.f};
                        if (n8 == 0) {
                            const float *src = q0 > 0 ? p.weights_out : p.weights_in;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int at = page0 + pos + (k & 1) + 8 * (k >> 1);
                                if (q0 > 0 ? at < seq_len + p.nq - 1 : src && at < seq_len - 1)
                                    old[k] = src[wrow + at];
                                if (q0 == 0)
                                    old[k] *= p.decay;
                            }
                        }
                        if (!ring_wait(full + 8 * st, ph, abort_flag, p.wait_limit) && !*abort_flag) {
                            *abort_flag = 1;
                            if (lane == 0)
                                set_error(p.err, kErrTimeout);
                        }
                        uint32_t kb[8][4];
                        load_keys<FMT>(kb, smem + st * TB, 16 * warp);
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(empty + 8 * st);
                        if (++st == STAGES) {
                            st = 0;
                            ph ^= 1u;
                        }
                        const bool part = page0 + kPage > seq_len || p.selected;
                        float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                        for (int t = 0; t < tiles; ++t) {
                            float s[2][2][4];
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                s[k >> 3][(k >> 2) & 1][k & 3] = 0.f;
#pragma unroll
                            for (int ks = 0; ks < 8; ++ks) {
                                const uint4 v = qf[(t * 8 + ks) * 32 + lane];
                                const uint32_t a[4] = {v.x, v.y, v.z, v.w};
                                mma_fmt<FMT>(s[ks & 1][0], a, kb[ks][0], kb[ks][1]);
                                mma_fmt<FMT>(s[ks & 1][1], a, kb[ks][2], kb[ks][3]);
                            }
                            const float4 ra = rows4[16 * t + n8], rb = rows4[16 * t + n8 + 8];
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float4 &rr = e < 2 ? ra : rb;
                                    float v = ex2(fmaf(s[0][k][e] + s[1][k][e], rr.x, -rr.y));
                                    if (part) {
                                        const int j = __float_as_int(rr.z), at = page0 + pos + 8 * k + (e & 1);
                                        if (at >= seq_len + j || !((m >> j) & 1ull))
                                            v = 0.f;
                                    }
                                    w[2 * k + (e & 1)] += v;
                                }
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            w[k] += __shfl_xor_sync(0xffffffffu, w[k], 4);
                            w[k] += __shfl_xor_sync(0xffffffffu, w[k], 8);
                            w[k] += __shfl_xor_sync(0xffffffffu, w[k], 16);
                        }
                        if (n8 == 0) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int at = page0 + pos + (k & 1) + 8 * (k >> 1);
                                if (at < seq_len + p.nq - 1)
                                    p.weights_out[wrow + at] = old[k] + w[k];
                            }
                        }
                    }
                }
            }
        }
        x += n;
        b = 0;
        if (++g == p.Hkv) {
            g = 0;
            do {
                if (++r >= p.R)
                    break;
                seq_len = p.seq_lens[r];
                nb = cached_blocks(seq_len, p.nq, p.maxB, &bad);
            } while (nb == 0);
        }
    }
    // the CTA's memory must outlive the copies in flight, also after a wait ran out
    if (warp == kConsumers && lane == 0)
        for (int i = max(0, issued - STAGES); i < issued; ++i)
            mbar_wait_bounded(full + 8 * (i % STAGES), (uint32_t)(i / STAGES) & 1u);
}

template <int FMT>
cudaError_t launch_t(const WeightParams &p, const CUtensorMap &map, int ctas, cudaStream_t stream)
{
    constexpr int smem = smem_layout(FMT).total;
    cudaError_t e = cudaFuncSetAttribute(weight_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = launch_kernel(weight_kernel<FMT>, dim3(ctas), dim3(kThreads), smem, stream, false, map, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace

cudaError_t launch_weight_accumulate(const WeightParams &p, int kv_dtype, int ctas, cudaStream_t stream)
{
    CUtensorMap map;
    if (!encode_pool_map(&map, p.kv, kv_dtype, p.num_pages, p.Hkv))
        return cudaErrorInvalidValue;
    if (kv_dtype == MSA_BF16)
        return launch_t<kFmtBf16>(p, map, ctas, stream);
    if (kv_dtype == MSA_FP8_E4M3)
        return launch_t<kFmtFp8>(p, map, ctas, stream);
    return launch_t<kFmtF4>(p, map, ctas, stream);
}

} // namespace msa
