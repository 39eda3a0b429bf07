// msa_dense.cu -- decode attention over every cached position (msa_dense_decode).
//
// For query row h of token t (request r, KV head g), over the visible
// positions p < seq_lens[r] + j:
//   s(p) = scale q . K[p],  lse = ln sum_p exp s(p),
//   out  = sum_p exp(s(p) - lse) V[p]
// in one pass over the pages: a running maximum m (log2 units), the
// denominator l = sum 2^(s - m) and O = sum 2^(s - m) V, all fp32, rescaled
// when m rises.  The nq * G query rows of a (request, KV head) share every
// page that is read.  This file has the kernel for up to 16 rows (one token of 16
// heads, two of 8, ...), the join of cut units and the launch; more rows go to
// the tcgen05 kernel of msa_dense_umma.cu.  With 16 rows that kernel multiplies eight
// times as many and widens every E4M3 tile: 352 us for 198 here (48 E4M3 contexts,
// 1.1 GB), 41.9 for 37.5 (8 heads, 165 MB of bf16), 16.4 for 11.7 (one context of 4096
// positions); with two row tiles here, 32 rows took 121 us for 70 there (349 MB).
//
// What bounds it: the bytes of the pages (16 heads: 16 flop a byte of bf16 K/V),
// so the kernel is a ring of whole pages fed by TMA, with as much in flight as
// shared memory holds (192 KiB an SM), and mma.sync (m16n8k16: 16 rows are one
// tile, no accumulator leaves the registers), whose work hides behind the copies:
// 5.6 TB/s over 1.1 GB of E4M3 pages (48 requests, 197 us), 4.4 TB/s over 165 MB of
// bf16 pages (8 heads, 37 us with the join), 7.1 TB/s over 5.1 GB in units of 1024
// pages.  A unit costs some 4 us of each CTA besides its pages (query rows, the sum over
// warps, outputs): 6.6 TB/s with units of 128 pages.
//
// Work split: the pages of all (request, KV head, row tile) units in one line,
// cut into equal ranges, one per persistent CTA.  A unit inside one range is
// finished there; a unit that is cut leaves one partial per CTA (at most two a
// CTA: its first and its last unit), joined in CTA order by a second, small
// kernel launched as a programmatic dependent.  No atomics, nothing kept
// between calls.
//
// Inside a CTA: one producer warp and eight consumer warps with 16 positions of every
// page each.  A consumer warp keeps m, l and O of the 16 rows over its own share of
// the pages, so warps meet only at the end of a unit.
#include <type_traits>

#include "msa_cache.cuh"

namespace msa {
namespace {

constexpr int kConsumers = 8;
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kJoinBytes = 32768; // cross-warp sum of O at the end of a unit
constexpr float kPUp = 15.f;      // P of 8-bit and 4-bit values: f16 of 2^15 P

__host__ __device__ constexpr int ring_stages(int fmt)
{
    return fmt == kFmtBf16 ? 3 : fmt == kFmtFp8 ? 6 : 10;
}

struct Smem {
    int ring, join, ml, bars, misc, total;
};

__host__ __device__ constexpr Smem smem_layout(int fmt)
{
    Smem s{};
    s.ring = 0;
    s.join = ring_stages(fmt) * 2 * tile_bytes(fmt);
    s.ml = s.join + kJoinBytes;          // m then l: [position groups][rows]
    s.bars = s.ml + 2 * 128 * 4;         // full[], empty[]
    s.misc = s.bars + 2 * ring_stages(fmt) * 8;
    s.total = s.misc + 64 + 1024;        // 1024: the ring's alignment
    return s;
}

__device__ __forceinline__ void consumers_sync()
{
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumers) : "memory");
}

// O += P V for 16 positions of the staged V tile.  hi (and for bf16 values lo,
// the bf16 rounding error of hi): P as A fragments.  MASKED: the values of
// positions 2c, 2c + 1 are taken through the bit mask k0, of 2c + 8, 2c + 9
// through k1 (a probability of 0 does not hide an infinity or NaN).
template <int FMT, bool MASKED>
__device__ __forceinline__ void accumulate16(float (&o)[16][4], const uint32_t (&hi)[4],
                                             const uint32_t (&lo)[4], uint32_t tile, int pos0,
                                             uint32_t k0 = 0u, uint32_t k1 = 0u)
{
    const int lane = threadIdx.x & 31, mi = lane >> 3;
    const int row = pos0 + (lane & 7) + (mi & 1) * 8;
    if (FMT == kFmtBf16) {
        const uint32_t base = tile + row * 128;
#pragma unroll
        for (int i = 0; i < 8; ++i) { // 16 dimensions: two n-tiles
            uint32_t b[4];
            const int chunk = 2 * (i & 3) + (mi >> 1);
            ldsm_x4_t(b, base + (i >> 2) * 16384 + ((chunk ^ (row & 7)) << 4));
            if (MASKED) {
                b[0] &= k0;
                b[1] &= k1;
                b[2] &= k0;
                b[3] &= k1;
            }
            mma_bf16(o[2 * i], hi, b[0], b[1]);
            mma_bf16(o[2 * i + 1], hi, b[2], b[3]);
            mma_bf16(o[2 * i], lo, b[0], b[1]);
            mma_bf16(o[2 * i + 1], lo, b[2], b[3]);
        }
    } else if (FMT == kFmtFp8) {
        const uint32_t base = tile + row * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) { // 32 dimensions: four n-tiles
            uint32_t b[4], x0[4], x1[4];
            const int chunk = 2 * i + (mi >> 1);
            ldsm_x4_t(b, base + ((chunk ^ (row & 7)) << 4));
            // bytes (p, d) (p, d + 1) (p + 1, d) (p + 1, d + 1) -> position pairs of d, of d + 1
#pragma unroll
            for (int k = 0; k < 4; ++k)
                e4m3x4_to_f16x2x2(__byte_perm(b[k], 0, 0x3120), x0[k], x1[k]);
            if (MASKED)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x0[k] &= k & 1 ? k1 : k0;
                    x1[k] &= k & 1 ? k1 : k0;
                }
            mma_f16(o[4 * i], hi, x0[0], x0[1]);
            mma_f16(o[4 * i + 1], hi, x1[0], x1[1]);
            mma_f16(o[4 * i + 2], hi, x0[2], x0[3]);
            mma_f16(o[4 * i + 3], hi, x1[2], x1[3]);
        }
    } else {
        const uint32_t base = tile + row * 64;
        const int n = lane >> 2, c = lane & 3;
        uint64_t w[4]; // the 8 scales of positions 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = lds64(tile + 8192 + (pos0 + 2 * c + (k & 1) + (k >> 1) * 8) * 8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t b[4];
            const int chunk = 2 * i + (mi >> 1);
            ldsm_x4_t(b, base + ((chunk ^ ((row >> 1) & 3)) << 4));
#pragma unroll
            for (int h = 0; h < 2; ++h) { // 32-dim chunk 2 i + h: four n-tiles
                const int grp = 2 * h + (n >> 2); // of the four scale bytes of this 64-dim half
                uint32_t x[2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k) { // positions 2c, 2c + 1, then + 8
                    const uint32_t wa = (uint32_t)(w[2 * k] >> (32 * i)), wb = (uint32_t)(w[2 * k + 1] >> (32 * i));
                    const uint32_t s2 = scale_pair(wa, grp, wb, grp);
                    const uint32_t v = b[2 * h + k];
                    // nibbles: p dims d..d+3, then p + 1 dims d..d+3 -> position pairs of each dim
                    const uint32_t even = v & 0x0F0F0F0Fu, odd = (v >> 4) & 0x0F0F0F0Fu;
                    const uint32_t e2 = even | (even >> 12), o2 = odd | (odd >> 12);
                    x[k][0] = hmul2_u32(e2m1x2_to_f16x2(e2 & 0xFFu), s2);
                    x[k][1] = hmul2_u32(e2m1x2_to_f16x2(o2 & 0xFFu), s2);
                    x[k][2] = hmul2_u32(e2m1x2_to_f16x2((e2 >> 8) & 0xFFu), s2);
                    x[k][3] = hmul2_u32(e2m1x2_to_f16x2((o2 >> 8) & 0xFFu), s2);
                    if (MASKED)
#pragma unroll
                        for (int d = 0; d < 4; ++d)
                            x[k][d] &= k ? k1 : k0;
                }
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    mma_f16(o[8 * i + 4 * h + d], hi, x[0][d], x[1][d]);
            }
        }
    }
}

// Which of the 16 positions pos0 .. (bits 0 .. 15) hold a V row with an infinity or NaN.
template <int FMT>
__device__ __forceinline__ uint32_t nonfinite_rows(uint32_t tile, int pos0)
{
    const int lane = threadIdx.x & 31, row = pos0 + (lane >> 1), half = lane & 1;
    bool bad = false;
    if (FMT == kFmtF4) {
        const uint64_t w = lds64(tile + 8192 + row * 8);
        const uint32_t x = half ? (uint32_t)(w >> 32) : (uint32_t)w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            bad |= ((x >> (8 * i)) & 0x7Fu) == 0x7Fu;
    } else {
        // half a row: bf16 has its halves in two boxes, E4M3 in one
        const uint32_t at = FMT == kFmtBf16 ? tile + half * 16384 + row * 128 : tile + row * 128 + half * 64;
        for (int i = 0; i < (FMT == kFmtBf16 ? 16 : 8); ++i) {
            const uint64_t w = lds64(at + 8 * i);
            // all exponent bits (bf16), or all bits but the sign (E4M3), set in some element
            for (int k = 0; k < (FMT == kFmtBf16 ? 4 : 8); ++k)
                bad |= FMT == kFmtBf16 ? ((w >> (16 * k)) & 0x7F80u) == 0x7F80u : ((w >> (8 * k)) & 0x7Fu) == 0x7Fu;
        }
    }
    uint32_t m = __ballot_sync(0xffffffffu, bad);
    m |= m >> 1; // bit 2 i: row i
    uint32_t rows = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        rows |= ((m >> (2 * i)) & 1u) << i;
    return rows;
}

// One stored value of V (without the tensor scale).
template <int FMT>
__device__ __forceinline__ float value_at(const uint8_t *tile, int row, int d)
{
    if (FMT == kFmtBf16)
        return __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t *>(
                                   tile + (d >> 6) * 16384 + row * 128 + ((((d & 63) >> 3) ^ (row & 7)) << 4) + (d & 7) * 2)
                               << 16);
    float a, b;
    if (FMT == kFmtFp8) {
        f16x2_to_f32x2(e4m3x2_to_f16x2(tile[row * 128 + (((d >> 4) ^ (row & 7)) << 4) + (d & 15)]), a, b);
        return a;
    }
    const uint32_t byte = tile[row * 64 + (((d >> 5) ^ ((row >> 1) & 3)) << 4) + ((d & 31) >> 1)];
    f16x2_to_f32x2(e2m1x2_to_f16x2(d & 1 ? byte >> 4 : byte & 15u), a, b);
    const float v = a;
    f16x2_to_f32x2(e4m3x2_to_f16x2(tile[8192 + row * 8 + (d >> 4)]), a, b);
    return v * a;
}

struct Flag {
    bool value;
};

// A 16-bit output pair at dimension d of one row.
__device__ __forceinline__ void store_bf16x2(uint16_t *row, int d, float a, float b)
{
    *reinterpret_cast<uint32_t *>(row + d) = pack_bf16(a, b);
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    dense_stream_kernel(const __grid_constant__ CUtensorMap map, const DenseParams p)
{
    constexpr int STAGES = ring_stages(FMT), TB = tile_bytes(FMT);
    constexpr int ROWS = 16;
    constexpr int TG = FMT == kFmtBf16 ? 1 : FMT == kFmtFp8 ? 2 : 4; // n-tiles that interleave their dimensions
    extern __shared__ uint8_t smem_raw[];
    __shared__ int scan_tmp[kThreads / 32 + 1];
    __shared__ int start_r, start_before;
    constexpr Smem L = smem_layout(FMT);
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t full = smem + L.bars, empty = full + STAGES * 8;
    uint8_t *gsm = smem_raw + (smem - smem_u32(smem_raw));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gsm + L.misc);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int heads = p.Hkv; // units of a request

    launch_dependents();
    if (threadIdx.x == 0) {
        prefetch_tensormap(&map);
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, kConsumers);
        }
        fence_mbar_init();
        *abort_flag = 0;
    }

    // this CTA's range of tasks, and the request it starts in
    const int per = (p.R + kThreads - 1) / kThreads;
    const int lo = min(p.R, (int)threadIdx.x * per), hi = min(p.R, lo + per);
    int total;
    const int before = scan_blocks(p, lo, hi, scan_tmp, &total);
    const int W = total * heads;
    const int x0 = range_start(blockIdx.x, W, gridDim.x), x1 = range_start(blockIdx.x + 1, W, gridDim.x);
    if (x0 < x1) {
        int b = before;
        for (int r = lo; r < hi; ++r) {
            bool bad;
            const int nb = cached_blocks(p.seq_lens[r], p.nq, p.maxB, &bad);
            if (nb > 0 && b * heads <= x0 && x0 < (b + nb) * heads) {
                start_r = r;
                start_before = b;
            }
            b += nb;
        }
    }
    __syncthreads();
    if (x0 == x1) { // more CTAs than tasks
        if (threadIdx.x == 0)
            p.joins[blockIdx.x] = make_int4(0, 0, -1, -1);
    }

    int r = 0, u = 0, b = 0, nb = 1, seq_len = 0;
    if (x0 < x1) {
        bool bad;
        r = start_r;
        seq_len = p.seq_lens[r];
        nb = cached_blocks(seq_len, p.nq, p.maxB, &bad);
        const int in = x0 - start_before * heads;
        u = in / nb;
        b = in - u * nb;
        if (threadIdx.x == 0) {
            // the unit is cut here: whoever owns its first cut has it joined
            int c0 = -1, c1 = -1;
            if (b > 0) {
                c0 = range_of(x0 - b, W, gridDim.x);
                c1 = range_of(x0 - b + nb - 1, W, gridDim.x);
                if (c0 != (int)blockIdx.x - 1)
                    c0 = c1 = -1;
            }
            p.joins[blockIdx.x] = make_int4(r, u, c0, c1);
        }
    }

    if (warp == kConsumers) {
        // ---- producer: one page (K and V tiles) per stage ----
        int st = 0, issued = 0;
        uint32_t ph = 0;
        bool stop = false;
        for (int x = x0; x < x1 && !stop;) {
            const int n = min(nb - b, x1 - x);
            const int32_t *row = p.block_table + (size_t)r * p.maxB;
            const int g = u;
            for (int i = 0; i < n && !stop; i += 32) { // 32 table entries at a time, one per lane
                const int mine = i + lane < n ? row[b + i + lane] : 0;
                for (int k = 0; k < min(32, n - i); ++k) {
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
                        break;
                    }
                    if (lane == 0) {
                        const uint32_t dst = smem + st * 2 * TB, bar = full + 8 * st;
                        mbar_arrive_expect_tx(bar, 2 * TB);
                        load_tile<FMT>(dst, &map, p.kv, (page * 2) * p.Hkv + g, bar);
                        load_tile<FMT>(dst + TB, &map, p.kv, (page * 2 + 1) * p.Hkv + g, bar);
                    }
                    __syncwarp();
                    ++issued;
                    if (++st == STAGES) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            x += n;
            b = 0;
            if (++u == heads) {
                u = 0;
                bool bad;
                do {
                    if (++r >= p.R)
                        break;
                    nb = cached_blocks(p.seq_lens[r], p.nq, p.maxB, &bad);
                } while (nb == 0);
            }
        }
        if (lane == 0) {
            if (stop)
                set_error(p.err, kErrTimeout);
            // the CTA's memory must outlive the copies in flight, also when a
            // consumer's wait ran out and the consumers do not wait for them
            for (int i = max(0, issued - STAGES); i < issued; ++i)
                mbar_wait_bounded(full + 8 * (i % STAGES), (uint32_t)(i / STAGES) & 1u);
        }
        __syncwarp();
        // idle slots: outputs of requests without cached positions
        for (int q = blockIdx.x; q < p.R; q += gridDim.x) {
            bool bad;
            if (cached_blocks(p.seq_lens[q], p.nq, p.maxB, &bad) > 0)
                continue;
            const size_t rows = (size_t)p.nq * p.Hkv * p.G;
            uint4 *out = reinterpret_cast<uint4 *>(p.out + q * rows * kDim);
            for (size_t i = lane; i < rows * (kDim / 8); i += 32)
                out[i] = make_uint4(0u, 0u, 0u, 0u);
            for (size_t i = lane; i < rows; i += 32)
                p.lse[q * rows + i] = __uint_as_float(0xFF800000u);
        }
        return;
    }

    // ---- consumers ----
    const int n8 = lane >> 2, c4 = lane & 3;
    float *sm_m = reinterpret_cast<float *>(gsm + L.ml), *sm_l = sm_m + 128;
    float *join = reinterpret_cast<float *>(gsm + L.join);
    int st = 0;
    uint32_t ph = 0;
    for (int x = x0; x < x1;) {
        const int n = min(nb - b, x1 - x);
        const int g = u;
        const size_t first_row = (size_t)r * p.nq * p.Hkv * p.G + (size_t)g * p.G; // of token 0
        // query row i of the unit: token i / G, head i % G
        const int i0 = n8, i1 = i0 + 8;
        const int j0 = min(i0, p.rows - 1) / p.G, j1 = min(i1, p.rows - 1) / p.G;
        const size_t pitch = (size_t)p.Hkv * p.G;
        uint32_t q[8][4];
        float inv0, inv1;
        load_queries<FMT>(q, i0 < p.rows ? p.q + (first_row + j0 * pitch + (i0 - j0 * p.G)) * kDim : nullptr,
                          i1 < p.rows ? p.q + (first_row + j1 * pitch + (i1 - j1 * p.G)) * kDim : nullptr, inv0, inv1);
        const float sc0 = p.scale_log2 * inv0, sc1 = p.scale_log2 * inv1;
        const int lim0 = seq_len + j0, lim1 = seq_len + j1, cached = seq_len + p.nq - 1;
        float o[16][4];
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[i][k] = 0.f;
        const float ninf = __uint_as_float(0xFF800000u);
        float m0 = ninf, m1 = ninf, l0 = 0.f, l1 = 0.f;

        for (int i = 0; i < n; ++i) {
            if (!ring_wait(full + 8 * st, ph, abort_flag, p.wait_limit) && !*abort_flag) {
                *abort_flag = 1;
                if (lane == 0)
                    set_error(p.err, kErrTimeout);
            }
            const uint32_t kt = smem + st * 2 * TB, vt = kt + TB;
            const int page0 = (b + i) * kPage;
            const bool tail = page0 + kPage > seq_len;
            const int at = 16 * warp; // this warp's positions of the page
            auto use_page = [&](auto ends) { // ends: some row does not see all of the page
                float s[2][4];
                score16<FMT>(s, q, kt, at);
                float a0 = ninf, a1 = ninf;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = s[t][e] * (e < 2 ? sc0 : sc1);
                        if (ends.value && page0 + at + 8 * t + 2 * c4 + (e & 1) >= (e < 2 ? lim0 : lim1))
                            v = ninf;
                        s[t][e] = v;
                        if (e < 2)
                            a0 = fmaxf(a0, v);
                        else
                            a1 = fmaxf(a1, v);
                    }
                a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, 1));
                a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, 1));
                a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, 2));
                a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, 2));
                if (FMT != kFmtBf16) {
                    a0 -= kPUp;
                    a1 -= kPUp;
                }
                if (__any_sync(0xffffffffu, a0 > m0 || a1 > m1)) {
                    const float n0 = fmaxf(m0, a0), n1 = fmaxf(m1, a1);
                    const float f0 = n0 == ninf ? 1.f : ex2(m0 - n0), f1 = n1 == ninf ? 1.f : ex2(m1 - n1);
                    m0 = n0;
                    m1 = n1;
                    l0 *= f0;
                    l1 *= f1;
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        o[k][0] *= f0;
                        o[k][1] *= f0;
                        o[k][2] *= f1;
                        o[k][3] *= f1;
                    }
                }
                const float r0 = m0 == ninf ? 0.f : m0, r1 = m1 == ninf ? 0.f : m1;
                uint32_t hi4[4], lo4[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float e0 = ex2(s[t][0] - r0), e1 = ex2(s[t][1] - r0);
                    const float e2 = ex2(s[t][2] - r1), e3 = ex2(s[t][3] - r1);
                    l0 += e0 + e1;
                    l1 += e2 + e3;
                    s[t][0] = e0;
                    s[t][1] = e1;
                    s[t][2] = e2;
                    s[t][3] = e3;
                    if (FMT == kFmtBf16) {
                        // P = hi + lo, 16 significant bits: the rounding of P to bf16 alone
                        // (up to 2^-8 relative) would weigh as much as the rounding of the output
                        const uint32_t h0 = pack_bf16(e0, e1), h1 = pack_bf16(e2, e3);
                        hi4[2 * t] = h0;
                        hi4[2 * t + 1] = h1;
                        lo4[2 * t] = pack_bf16(e0 - __uint_as_float(h0 << 16), e1 - __uint_as_float(h0 & 0xFFFF0000u));
                        lo4[2 * t + 1] = pack_bf16(e2 - __uint_as_float(h1 << 16), e3 - __uint_as_float(h1 & 0xFFFF0000u));
                    } else { // f16 of 2^15 P: 11 significant bits down to P = 2^-29
                        hi4[2 * t] = pack_f16(e0, e1);
                        hi4[2 * t + 1] = pack_f16(e2, e3);
                    }
                }
                const int past = cached - page0 - at; // rows from `past` on are not cached
                if (ends.value && page0 + at + 16 > seq_len && (past < 16 || p.nq > 1)) {
                    uint32_t drop = past < 16 ? 0xFFFFu << max(past, 0) & 0xFFFFu : 0u;
                    // positions that only later tokens see: their infinities and NaN are added
                    // to the rows that see them, one position at a time, past the MMA
                    uint32_t later = 0xFFFFu << max(seq_len - page0 - at, 0) & 0xFFFFu & ~drop;
                    if (later)
                        later &= nonfinite_rows<FMT>(vt, at);
                    drop |= later;
                    for (; later; later &= later - 1) {
                        const int pp = __ffs(later) - 1, src = (lane & ~3) | ((pp & 7) >> 1);
                        const float c0 = pp & 8 ? (pp & 1 ? s[1][1] : s[1][0]) : (pp & 1 ? s[0][1] : s[0][0]);
                        const float c1 = pp & 8 ? (pp & 1 ? s[1][3] : s[1][2]) : (pp & 1 ? s[0][3] : s[0][2]);
                        const float p0 = __shfl_sync(0xffffffffu, c0, src), p1 = __shfl_sync(0xffffffffu, c1, src);
                        const bool see0 = page0 + at + pp < lim0, see1 = page0 + at + pp < lim1;
#pragma unroll
                        for (int t = 0; t < 16; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float v = value_at<FMT>(gsm + st * 2 * TB + TB, at + pp,
                                                              8 * TG * (t / TG) + TG * (2 * c4 + e) + t % TG);
                                if (see0)
                                    o[t][e] = fmaf(p0, v, o[t][e]);
                                if (see1)
                                    o[t][2 + e] = fmaf(p1, v, o[t][2 + e]);
                            }
                    }
                    const uint32_t d0 = drop >> (2 * c4), d1 = d0 >> 8;
                    accumulate16<FMT, true>(o, hi4, lo4, vt, at, (d0 & 1 ? 0u : 0xFFFFu) | (d0 & 2 ? 0u : 0xFFFF0000u),
                                            (d1 & 1 ? 0u : 0xFFFFu) | (d1 & 2 ? 0u : 0xFFFF0000u));
                } else {
                    accumulate16<FMT, false>(o, hi4, lo4, vt, at);
                }
            };
            // whole pages by themselves where V is widened: NVFP4 1040 -> 993 us, E4M3 714 -> 708 us
            // over 19 x 131072 positions of 8 KV heads; bf16 8 heads lost, 37.5 -> 38.8 us
            if constexpr (FMT == kFmtBf16)
                use_page(Flag{tail});
            else if (tail)
                use_page(std::true_type{});
            else
                use_page(std::false_type{});
            __syncwarp();
            if (lane == 0)
                mbar_arrive(empty + 8 * st);
            if (++st == STAGES) {
                st = 0;
                ph ^= 1u;
            }
        }

        // ---- end of the unit's share: warps of the same rows add up ----
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if (c4 == 0) {
            sm_m[ROWS * warp + n8] = m0;
            sm_m[ROWS * warp + n8 + 8] = m1;
            sm_l[ROWS * warp + n8] = l0;
            sm_l[ROWS * warp + n8 + 8] = l1;
        }
        consumers_sync();
        float M0 = ninf, M1 = ninf, L0 = 0.f, L1 = 0.f;
#pragma unroll
        for (int k = 0; k < kConsumers; ++k) {
            M0 = fmaxf(M0, sm_m[ROWS * k + n8]);
            M1 = fmaxf(M1, sm_m[ROWS * k + n8 + 8]);
        }
#pragma unroll
        for (int k = 0; k < kConsumers; ++k) {
            const float a = sm_m[ROWS * k + n8], c = sm_m[ROWS * k + n8 + 8];
            L0 += a == ninf ? 0.f : sm_l[ROWS * k + n8] * ex2(a - M0);
            L1 += c == ninf ? 0.f : sm_l[ROWS * k + n8 + 8] * ex2(c - M1);
        }
        const float f0 = m0 == ninf ? 0.f : ex2(m0 - M0), f1 = m1 == ninf ? 0.f : ex2(m1 - M1);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            o[k][0] *= f0;
            o[k][1] *= f0;
            o[k][2] *= f1;
            o[k][3] *= f1;
        }
        float *mine = join + (warp % (kConsumers / 2)) * 2048 + lane;
        if (warp >= kConsumers / 2) {
#pragma unroll
            for (int k = 0; k < 64; ++k)
                mine[k * 32] = o[k >> 2][k & 3];
        }
        consumers_sync();
        if (warp < kConsumers / 2) {
#pragma unroll
            for (int k = 0; k < 64; ++k)
                mine[k * 32] += o[k >> 2][k & 3];
        }
        consumers_sync();

        // this warp finishes two n-tiles, in groups of TG: 2 TG consecutive dimensions a lane
        const bool whole = b == 0 && n == nb; // no other CTA has a part of this unit
        const bool ends = b + n == nb;
        float *slot = p.partial + (size_t)(2 * blockIdx.x + (ends ? 0 : 1)) * (ROWS * (kDim + 2));
        const float g0 = L0 > 0.f || L0 != L0 ? p.v_scale / L0 : 0.f, g1 = L1 > 0.f || L1 != L1 ? p.v_scale / L1 : 0.f;
        const size_t out0 = first_row + j0 * pitch + (i0 - j0 * p.G), out1 = first_row + j1 * pitch + (i1 - j1 * p.G);
        for (int grp = warp; grp < 16 / TG; grp += kConsumers) {
            float v[2][2 * TG];
#pragma unroll
            for (int t = 0; t < TG; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float a = 0.f;
#pragma unroll
                    for (int k = 0; k < kConsumers / 2; ++k)
                        a += join[k * 2048 + ((grp * TG + t) * 4 + e) * 32 + lane];
                    v[e >> 1][(e & 1) * TG + t] = a;
                }
            const int d = 8 * TG * grp + 2 * TG * c4;
            if (whole) {
#pragma unroll
                for (int k = 0; k < 2 * TG; k += 2) {
                    if (i0 < p.rows)
                        store_bf16x2(p.out + out0 * kDim, d + k, v[0][k] * g0, v[0][k + 1] * g0);
                    if (i1 < p.rows)
                        store_bf16x2(p.out + out1 * kDim, d + k, v[1][k] * g1, v[1][k + 1] * g1);
                }
            } else {
                float *a = slot + (size_t)n8 * kDim + d;
#pragma unroll
                for (int k = 0; k < 2 * TG; k += 2) {
                    *reinterpret_cast<float2 *>(a + k) = make_float2(v[0][k], v[0][k + 1]);
                    *reinterpret_cast<float2 *>(a + 8 * kDim + k) = make_float2(v[1][k], v[1][k + 1]);
                }
            }
        }
        if (warp == 0 && c4 == 0) {
            if (whole) {
                if (i0 < p.rows)
                    p.lse[out0] = L0 == 0.f ? ninf : (M0 + log2f(L0)) * 0.6931471805599453f;
                if (i1 < p.rows)
                    p.lse[out1] = L1 == 0.f ? ninf : (M1 + log2f(L1)) * 0.6931471805599453f;
            } else {
                float *ml = slot + (size_t)ROWS * kDim + n8;
                ml[0] = M0;
                ml[8] = M1;
                ml[ROWS] = L0;
                ml[ROWS + 8] = L1;
            }
        }
        consumers_sync(); // the join buffers are free for the next unit

        x += n;
        b = 0;
        if (++u == heads) {
            u = 0;
            bool bad;
            do {
                if (++r >= p.R)
                    break;
                seq_len = p.seq_lens[r];
                nb = cached_blocks(seq_len, p.nq, p.maxB, &bad);
            } while (nb == 0);
        }
    }
}

// Joins the partials of the rows of one cut unit, in CTA order: blockIdx.x + 1
// is the CTA at whose start the unit was first cut.  SPLIT warps share a row
// (warp s takes every SPLIT-th partial, as many units are cut often only where
// they have few rows); lane l has dimensions 4 l .. 4 l + 3.
template <int SPLIT>
__global__ void __launch_bounds__(256) dense_join_kernel(const DenseParams p, int tile_rows)
{
    __shared__ float sm_m[8], sm_l[8];
    __shared__ float4 sm_o[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp % SPLIT;
    grid_dependency_wait();
    const int4 jn = p.joins[blockIdx.x + 1];
    if (jn.z < 0)
        return;
    const int row = blockIdx.y * (8 / SPLIT) + warp / SPLIT;
    const int g = jn.y / p.tiles, i = (jn.y - g * p.tiles) * tile_rows + row;
    const bool real = row < tile_rows && i < p.rows;
    if (SPLIT == 1 && !real)
        return;
    const float ninf = __uint_as_float(0xFF800000u);
    const size_t floats = (size_t)tile_rows * (kDim + 2);
    float M = ninf, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = jn.z + w; c <= jn.w && real; c += 4 * SPLIT) {
        float m[4], l[4];
        float4 v[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int cc = c + SPLIT * s;
            m[s] = ninf;
            l[s] = 0.f;
            v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (cc <= jn.w) {
                const float *slot = p.partial + (size_t)(2 * cc + (cc < jn.w ? 1 : 0)) * floats;
                m[s] = slot[(size_t)tile_rows * kDim + row];
                l[s] = slot[(size_t)tile_rows * (kDim + 1) + row];
                v[s] = reinterpret_cast<const float4 *>(slot + (size_t)row * kDim)[lane];
            }
        }
        const float n = fmaxf(M, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
        const float ref = n == ninf ? 0.f : n;
        const float f = ex2(M - ref);
        L *= f;
        o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const float e = ex2(m[s] - ref);
            L += l[s] * e;
            o.x += v[s].x * e, o.y += v[s].y * e, o.z += v[s].z * e, o.w += v[s].w * e;
        }
        M = n;
    }
    if (SPLIT > 1) {
        if (lane == 0) {
            sm_m[warp] = M;
            sm_l[warp] = L;
        }
        sm_o[warp][lane] = o;
        __syncthreads();
        if (w != 0 || !real)
            return;
        M = ninf;
#pragma unroll
        for (int s = 0; s < SPLIT; ++s)
            M = fmaxf(M, sm_m[warp + s]);
        const float ref = M == ninf ? 0.f : M;
        L = 0.f;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int s = 0; s < SPLIT; ++s) {
            const float e = ex2(sm_m[warp + s] - ref);
            const float4 v = sm_o[warp + s][lane];
            L += sm_l[warp + s] * e;
            o.x += v.x * e, o.y += v.y * e, o.z += v.z * e, o.w += v.w * e;
        }
    }
    const float f = L > 0.f || L != L ? p.v_scale / L : 0.f;
    const int j = i / p.G;
    const size_t out = ((size_t)jn.x * p.nq + j) * p.Hkv * p.G + (size_t)g * p.G + (i - j * p.G);
    reinterpret_cast<uint2 *>(p.out + out * kDim)[lane] = make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
    if (lane == 0)
        p.lse[out] = L == 0.f ? ninf : (M + log2f(L)) * 0.6931471805599453f;
}

cudaError_t launch_join(const DenseParams &p, int tile_rows, int ctas, cudaStream_t stream)
{
    const int rows = p.rows < tile_rows ? p.rows : tile_rows;
    if (tile_rows == 16)
        return launch_kernel(dense_join_kernel<4>, dim3(ctas - 1, (rows + 1) / 2), dim3(256), 0, stream, true, p, tile_rows);
    return launch_kernel(dense_join_kernel<1>, dim3(ctas - 1, (rows + 7) / 8), dim3(256), 0, stream, true, p, tile_rows);
}

template <int FMT>
cudaError_t launch_t(const DenseParams &p, const CUtensorMap &map, int ctas, cudaStream_t stream)
{
    constexpr int smem = smem_layout(FMT).total;
    cudaError_t e = cudaFuncSetAttribute(dense_stream_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = launch_kernel(dense_stream_kernel<FMT>, dim3(ctas), dim3(kThreads), smem, stream, false, map, p);
    return e;
}

} // namespace

int dense_tile_rows(int rows)
{
    return rows <= 16 ? 16 : rows <= 128 ? 128 : 256;
}

cudaError_t launch_dense_decode(const DenseParams &p, int kv_dtype, int ctas, cudaStream_t stream)
{
    CUtensorMap map;
    if (!encode_pool_map(&map, p.kv, kv_dtype, p.num_pages, p.Hkv))
        return cudaErrorInvalidValue;
    cudaError_t e;
    if (p.rows > 16)
        e = launch_dense_umma(p, map, kv_dtype, ctas, stream);
    else if (kv_dtype == MSA_BF16)
        e = launch_t<kFmtBf16>(p, map, ctas, stream);
    else if (kv_dtype == MSA_FP8_E4M3)
        e = launch_t<kFmtFp8>(p, map, ctas, stream);
    else
        e = launch_t<kFmtF4>(p, map, ctas, stream);
    if (e == cudaSuccess && ctas > 1)
        e = launch_join(p, dense_tile_rows(p.rows), ctas, stream);
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace msa
