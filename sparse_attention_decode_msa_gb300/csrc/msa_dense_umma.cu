// msa_dense_umma.cu -- dense decode for many query rows (speculative tokens, a
// prompt's last chunk): S = Q K^T and O += P V on the tcgen05 tensor cores.
//
// Mathematics as in msa_dense.cu: a running maximum m, l = sum 2^(s - m) and
// O = sum 2^(s - m) V per query row, fp32, one pass over the pages.  Rows are
// the M dimension, 128 of them per accumulator, one thread per row: the
// softmax needs no exchange between threads.
//
// Two streams share a CTA's pages, so that the tensor cores work for one while
// the other is in its softmax, and each stream works in steps of 64 positions
// with two S buffers, so that the S of its next step is ready when a softmax
// ends.  With more than 128 query rows a (request, KV head), stream t has rows
// 128 t .. of a 256-row tile and takes both halves of every page; with fewer,
// both have the same rows, stream t takes half t of every page, and the two
// (m, l, O) are added at the end.  With NVFP4 tiles up to 64 rows are in the operand
// tile twice (TWICE), rows 0 .. for stream 0 and 64 .. for stream 1: a softmax warp can
// read one quarter of the accumulator lanes only, and so the streams' warps with rows in
// them sit on different schedulers (32 requests of 2 tokens over 65536 positions: 456 us,
// 495 without).  E4M3 and bf16 lose more to the longer end of a unit
// than they gain: 143 us for 137, 2 tokens over 64 x 32768 E4M3 positions, 78 for 70 on 8
// requests of 4 bf16 tokens.
//
// Operands: Q in shared memory (K-major, 128-byte swizzle), K tiles as TMA
// lands them (K-major), P in tensor memory over the S it came from, V tiles as
// landed (MN-major).  bf16 P is a pair hi + lo (16 significant bits): the rounding to
// bf16 alone is up to 2^-8 of each p, and where many positions have the same logit
// (repeated keys, a scale near 0) all of them round the same way, so that an output would be
// off by 2^-8 of the largest |v| however small the single p are (48 tokens over 2 x 131072
// positions take 457 us with the pair, 394 with hi alone).  E4M3 and NVFP4 tiles are
// widened to f16 by converter warps and P is one f16: off by 2^-11 of p at most, by as much of the
// largest |v| at worst, an eighth of what the storage of the output takes.
//
// TMEM columns: S/P of step s of stream t at 128 t + 64 (s & 1) (one row tile: at
// 128 (s & 1) + 64 t), O of stream t at 256 + 128 t.
// Warps: 0 TMA producer (and outputs of idle slots), 1 issues S (and owns the TMEM),
// 2 and 3 issue P V of stream 0 and 1, 4-7 and 8-11 softmax of stream 0 and 1,
// 12-15 (and 16-19) converters (E4M3, NVFP4).
//
// What bounds it: the tensor cores when rows are many (measured: an MMA of
// 128 x 128 x 16 takes 66 clocks, one of 128 x 64 x 16 takes 50 as both read 4 KiB
// of Q from shared memory; a page of 128 rows is 16 of these for S, or 8 of those
// with one row tile, and 8, or 16 as pairs, of those for P V), HBM when they are few.
// Measured: 48 tokens over 2 x 131072 bf16 positions 432 .. 468 us, 0.88 .. 0.95 PFLOP/s (the chain
// S, maximum, exponentials, P V of a step is longer than its MMAs: tensor pipe 55% busy);
// 4 tokens, 349 MB of bf16 pages 70 us, 5.0 TB/s; 2 tokens, 1.2 GB of NVFP4 pages 456 us,
// 2.65 TB/s (no unit is full: issue slots 48%, tensor pipe 41%; the roles wait for one another).
#include <type_traits>

#include "msa_umma.cuh"

namespace msa {
namespace {

constexpr int kTile16 = 32768;   // a 16-bit K, V or Q tile
constexpr int kStaged = 4;       // widened tiles in flight
constexpr float kSlack = 8.f;    // how far (log2) a row's maximum may pass its reference before O is rescaled
constexpr float kPUp16 = 7.f;    // f16 P: 2^7 2^(s - m), at most 2^15 with the slack

// Groups of four converter warps, which take the tiles in turn.  With one row tile two of
// them (456 us for 572 on 32 requests of 2 tokens over 65536 NVFP4 positions); with two,
// whose tiles have more to multiply, the second would only take registers from the softmax
// (48 tokens over 2 x 131072: 424 us for 438, E4M3, and 412 for 433, NVFP4).
__host__ __device__ constexpr int conv_groups(int fmt, bool two)
{
    return fmt == kFmtBf16 ? 0 : two ? 1 : 2;
}

__host__ __device__ constexpr int threads_of(int fmt, bool two)
{
    return 384 + 128 * conv_groups(fmt, two);
}

// Tiles (K or V) in the ring: an even number where two converter groups widen them (a slot
// belongs to one group, which follows all of its barriers' phases).
__host__ __device__ constexpr int ring_tiles(int fmt, bool two)
{
    return fmt == kFmtBf16 ? (two ? 5 : 6) : fmt == kFmtFp8 ? (two ? 2 : 4) : (two ? 2 : 6);
}

struct Smem {
    int ring, staged, q, ml, inv, bars, misc, total;
};

__host__ __device__ constexpr Smem smem_layout(int fmt, bool two)
{
    Smem s{};
    s.ring = 0;
    s.staged = ring_tiles(fmt, two) * tile_bytes(fmt);
    s.q = s.staged + (fmt == kFmtBf16 ? 0 : kStaged * kTile16);
    s.ml = s.q + (two ? 2 : 1) * kTile16; // m[128], l[128] of stream 1 (one row tile)
    s.inv = s.ml + (two ? 0 : 2 * 128 * 4); // factors that undo the scaling of query rows
    s.bars = s.inv + (fmt == kFmtBf16 ? 0 : (two ? 2 : 1) * 128 * 4);
    s.misc = s.bars + (2 * ring_tiles(fmt, two) + 2 * kStaged + 21) * 8;
    s.total = s.misc + 64 + 1024;
    return s;
}
static_assert(smem_layout(kFmtBf16, true).total <= 232448 && smem_layout(kFmtBf16, false).total <= 232448 &&
                  smem_layout(kFmtFp8, true).total <= 232448 && smem_layout(kFmtFp8, false).total <= 232448 &&
                  smem_layout(kFmtF4, true).total <= 232448 && smem_layout(kFmtF4, false).total <= 232448,
              "shared memory");

// One stored K (0) or V (1) value in global memory, without its tensor scale.
template <int FMT>
__device__ __forceinline__ float stored_value(const uint8_t *kv, long long tile, int row, int d)
{
    float a, b;
    if (FMT == kFmtBf16)
        return __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t *>(kv + (tile * kPage + row) * 256 + 2 * d) << 16);
    if (FMT == kFmtFp8) {
        f16x2_to_f32x2(e4m3x2_to_f16x2(kv[(tile * kPage + row) * 128 + d]), a, b);
        return a;
    }
    const uint8_t *t = kv + tile * 9216;
    const uint32_t byte = t[row * 64 + (d >> 1)];
    f16x2_to_f32x2(e2m1x2_to_f16x2(d & 1 ? byte >> 4 : byte & 15u), a, b);
    const float v = a;
    f16x2_to_f32x2(e4m3x2_to_f16x2(t[8192 + row * 8 + (d >> 4)]), a, b);
    return v * a;
}

__device__ __forceinline__ bool finite(float v)
{
    return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u;
}

// Rows of 64 positions (from row0) of a staged bf16 V tile on a last page: rows from `past` on are
// not cached and become zeros, and so do infinities and NaN of rows from `seen` on, which only
// later tokens see (a probability of 0 does not hide them; those tokens get them at the
// end of the unit, told by *bad).  One warp; done twice it does no more.
__device__ __noinline__ void clear_values(uint8_t *v, int row0, int seen, int past, volatile int *bad, int mark)
{
    const int from = max(row0, seen);
    for (int k = from * 16 + (int)(threadIdx.x & 31); k < (row0 + 64) * 16; k += 32) { // 16-byte pieces
        const int row = k >> 4, piece = k & 15;
        uint4 *at = reinterpret_cast<uint4 *>(v + (piece >> 3) * 16384 + row * 128 + (piece & 7) * 16);
        if (row >= past) {
            *at = make_uint4(0u, 0u, 0u, 0u);
            continue;
        }
        uint4 d = *at;
        uint32_t *e = &d.x;
        bool any = false;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if ((e[c] & 0x7F80u) == 0x7F80u)
                e[c] &= 0xFFFF0000u, any = true;
            if ((e[c] & 0x7F800000u) == 0x7F800000u)
                e[c] &= 0x0000FFFFu, any = true;
        }
        if (any) {
            *bad = mark; // told before the value is gone
            __threadfence_block();
            *at = d;
        }
    }
    fence_async_smem();
    __syncwarp();
}

// Place of a tile in the order in which the issuer uses the tiles of n pages.
template <bool TWO>
__device__ __forceinline__ int order_of_k(int page)
{
    return TWO ? 2 * page : page < 2 ? page : 2 * page - 1;
}
template <bool TWO>
__device__ __forceinline__ int order_of_v(int page, int n)
{
    return TWO ? 2 * page + 1 : min(2 * page + 2, 2 * n - 1);
}

template <int FMT, bool TWO, bool TWICE>
__global__ void __launch_bounds__(threads_of(FMT, TWO), 1)
    dense_umma_kernel(const __grid_constant__ CUtensorMap map, const DenseParams p)
{
    constexpr int TILES = ring_tiles(FMT, TWO), TB = tile_bytes(FMT), NT = threads_of(FMT, TWO);
    constexpr bool CONV = FMT != kFmtBf16;
    constexpr int ROWS = TWO ? 256 : 128;
    constexpr Smem L = smem_layout(FMT, TWO);
    extern __shared__ uint8_t smem_raw[];
    __shared__ int scan_tmp[NT / 32 + 1];
    __shared__ int start_r, start_before;
    __shared__ uint32_t tmem_slot;
    __shared__ int later_bad[8]; // unit counter + 1 where V rows of draft tokens are not finite
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *gsm = smem_raw + (smem - smem_u32(smem_raw));
    const uint32_t full = smem + L.bars, empty = full + TILES * 8, sfull = empty + TILES * 8, sempty = sfull + kStaged * 8;
    const uint32_t q_full = sempty + kStaged * 8, q_free = q_full + 16, s_full = q_free + 8, p_full = s_full + 32,
                   pv_done = p_full + 32, o_free = pv_done + 32, drain = o_free + 16;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gsm + L.misc);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int heads = p.Hkv * p.tiles;
    const long long wl = p.wait_limit;

    launch_dependents();
    if (threadIdx.x == 0) {
        prefetch_tensormap(&map);
        for (int i = 0; i < TILES; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, CONV ? 4 : 2);
        }
        for (int i = 0; i < kStaged; ++i) {
            mbar_init(sfull + 8 * i, 4);
            mbar_init(sempty + 8 * i, 2);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(q_full + 8 * t, TWO ? 4 : 8);
            mbar_init(s_full + 16 * t, 1);
            mbar_init(s_full + 16 * t + 8, 1);
            mbar_init(p_full + 16 * t, 4);
            mbar_init(p_full + 16 * t + 8, 4);
            mbar_init(pv_done + 16 * t, 1);
            mbar_init(pv_done + 16 * t + 8, 1);
            mbar_init(o_free + 8 * t, 4);
        }
        mbar_init(q_free, 1);
        for (int i = 0; i < 3; ++i)
            mbar_init(drain + 8 * i, 1);
        fence_mbar_init();
        *abort_flag = 0;
    }
    if (threadIdx.x < 8)
        later_bad[threadIdx.x] = 0;
    if (warp == 1)
        tmem_alloc(smem_u32(&tmem_slot), 512);

    const int per = (p.R + NT - 1) / NT;
    const int lo = min(p.R, (int)threadIdx.x * per), hi = min(p.R, lo + per);
    int total;
    const int before = scan_blocks(p, lo, hi, scan_tmp, &total);
    const int W = total * heads;
    Walk w{};
    w.x = range_start(blockIdx.x, W, gridDim.x);
    w.x1 = range_start(blockIdx.x + 1, W, gridDim.x);
    w.nb = 1;
    if (w.x < w.x1) {
        int b = before;
        for (int r = lo; r < hi; ++r) {
            bool bad;
            const int nb = cached_blocks(p.seq_lens[r], p.nq, p.maxB, &bad);
            if (nb > 0 && b * heads <= w.x && w.x < (b + nb) * heads) {
                start_r = r;
                start_before = b;
            }
            b += nb;
        }
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = tmem_slot;
    if (w.x < w.x1) {
        bool bad;
        w.r = start_r;
        w.seq_len = p.seq_lens[w.r];
        w.nb = cached_blocks(w.seq_len, p.nq, p.maxB, &bad);
        const int in = w.x - start_before * heads;
        w.u = in / w.nb;
        w.b = in - w.u * w.nb;
    }
    if (threadIdx.x == 0) {
        int c0 = -1, c1 = -1;
        if (w.x < w.x1 && w.b > 0) {
            c0 = range_of(w.x - w.b, W, gridDim.x);
            c1 = range_of(w.x - w.b + w.nb - 1, W, gridDim.x);
            if (c0 != (int)blockIdx.x - 1)
                c0 = c1 = -1;
        }
        p.joins[blockIdx.x] = make_int4(w.r, w.u, c0, c1);
    }
    // a wait that ran out: the CTA's roles run on without waiting, so that all
    // reach the end; what they compute is unspecified
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!ring_wait(bar, parity, abort_flag, wl) && !*abort_flag) {
            *abort_flag = 1;
            set_error(p.err, kErrTimeout);
        }
    };

    if (warp == 0) {
        // ---- producer: K and V tiles in the order of their use ----
        int z = 0, st = 0;
        uint32_t ph = 0;
        for (; w.x < w.x1; w.next(p, heads)) {
            const int n = w.pages(), g = w.u / p.tiles;
            const int32_t *row = p.block_table + (size_t)w.r * p.maxB + w.b;
            // two windows of 32 table entries: K runs at most two pages ahead of V
            int ent = 0, ent0 = -1, prev = 0;
            int kp = 0, vp = 0;
            for (int i = 0; i < 2 * n; ++i) {
                const bool is_k = kp < n && order_of_k<TWO>(kp) == i;
                const int pg = is_k ? kp++ : vp++;
                const int win = pg >> 5;
                if (win > ent0) {
                    prev = ent;
                    ent0 = win;
                    ent = 32 * win + lane < n ? row[32 * win + lane] : 0;
                }
                long long page = __shfl_sync(0xffffffffu, win == ent0 ? ent : prev, pg & 31);
                if (page < 0 || page >= p.num_pages) {
                    if (lane == 0)
                        set_error(p.err, kErrPage);
                    page = 0; // in the pool: the outputs of the call are unspecified
                }
                if (z >= TILES)
                    wait(empty + 8 * st, ph ^ 1u);
                if (__any_sync(0xffffffffu, *abort_flag != 0))
                    break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(full + 8 * st, TB);
                    load_tile<FMT>(smem + st * TB, &map, p.kv, (page * 2 + (is_k ? 0 : 1)) * p.Hkv + g, full + 8 * st);
                }
                __syncwarp();
                ++z;
                if (++st == TILES) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (__any_sync(0xffffffffu, *abort_flag != 0))
                break;
        }
        if (lane == 0) // the CTA's memory must outlive the copies in flight
            for (int i = max(0, z - TILES); i < z; ++i)
                mbar_wait_bounded(full + 8 * (i % TILES), (uint32_t)(i / TILES) & 1u);
        __syncwarp();
        // ---- idle slots: outputs of requests without cached positions ----
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
    } else if (warp < 4) {
        // ---- MMA issuers: warp 1 issues S (one row tile: an S tile is a whole page, stream
        // t takes columns 64 t ..), warps 2 and 3 P V of stream 0 and 1.  An issuer's own
        // instructions between two MMAs take longer than an MMA, so that one issuer cannot
        // keep the tensor cores busy ----
        const uint32_t one = lane == 0, tm = uniform(tmem), base = uniform(smem);
        constexpr uint32_t kTypes = CONV ? ~((1u << 7) | (1u << 10)) : ~0u; // f16 or bf16 operands
        constexpr uint32_t idesc_s = umma_idesc_bf16(128, TWO ? 64 : 128, 0, 0) & kTypes;
        constexpr uint32_t idesc_o = umma_idesc_bf16(128, 128, 0, 1) & kTypes;
        constexpr int DEPTH = CONV ? kStaged : TILES;
        constexpr uint32_t STEP = CONV ? kTile16 : TB, RING = CONV ? L.staged : 0, HALF = 64 * 128 >> 4;
        const uint32_t tile_full = CONV ? sfull : full, tile_free = CONV ? sempty : empty;
        uint32_t fill0 = 0, fill1 = 0; // steps of either S buffer so far
        int z0 = 0;
        for (; w.x < w.x1; w.next(p, heads)) {
            const int n = w.pages();
            const int nsteps = TWO ? 2 * n : n;
            if (warp == 1) {
                wait(q_full, w.seg & 1);
                if (TWO)
                    wait(q_full + 8, w.seg & 1);
                const uint32_t q = uniform(desc_low(base + L.q, 16));
                for (int i = 0; i < nsteps; ++i) {
                    const int z = z0 + order_of_k<TWO>(TWO ? i >> 1 : i), st = z % DEPTH;
                    const uint32_t k = uniform(desc_low(base + RING + st * STEP, 16) + (TWO && (i & 1) ? HALF : 0u));
                    const uint32_t fill = i & 1 ? fill1++ : fill0++;
                    wait(tile_full + 8 * st, (uint32_t)(z / DEPTH) & 1u);
#pragma unroll
                    for (int t = 0; t < (TWO ? 2 : 1); ++t) {
                        // the buffer's last P has been multiplied
                        if (fill > 0) {
                            wait(pv_done + 16 * t + 8 * (i & 1), (fill - 1) & 1u);
                            if (!TWO)
                                wait(pv_done + 16 + 8 * (i & 1), (fill - 1) & 1u);
                        }
                        tcgen05_after_sync();
                        const uint32_t d = tm + uniform(TWO ? 128 * t + 64 * (i & 1) : 128 * (i & 1));
                        const uint32_t qt = q + t * (kTile16 >> 4);
#pragma unroll
                        for (uint32_t ks = 0; ks < 8; ++ks)
                            umma_ss(one, d, qt + (ks >> 2) * 1024 + (ks & 3) * 2, k + (ks >> 2) * 1024 + (ks & 3) * 2, idesc_s, ks > 0);
                        if (one)
                            umma_commit(s_full + 16 * t + 8 * (i & 1));
                    }
                    if (one && (!TWO || (i & 1))) { // a tile is given back twice: V by either stream
                        umma_commit(tile_free + 8 * st);
                        umma_commit(tile_free + 8 * st);
                    }
                }
                if (one)
                    umma_commit(q_free);
            } else {
                const int t = warp - 2;
                const uint32_t d = tm + uniform(256 + 128 * t);
                for (int i = 0; i < nsteps; ++i) {
                    const int page = TWO ? i >> 1 : i, z = z0 + order_of_v<TWO>(page, n), st = z % DEPTH;
                    const uint32_t v = uniform(desc_low(base + RING + st * STEP, 16384) + ((TWO ? i & 1 : t) ? HALF : 0u));
                    const uint32_t a = tm + uniform(TWO ? 128 * t + 64 * (i & 1) : 128 * (i & 1) + 64 * t);
                    const uint32_t more = uniform(i > 0);
                    wait(tile_full + 8 * st, (uint32_t)(z / DEPTH) & 1u);
                    if (!CONV && (w.b + page + 1) * kPage > w.seq_len) // (converters do it for their tiles)
                        clear_values(gsm + st * TB, (TWO ? i & 1 : t) * 64, w.seq_len - (w.b + page) * kPage,
                                     w.seq_len + p.nq - 1 - (w.b + page) * kPage, &later_bad[w.seg & 7], w.seg + 1);
                    if (i == 0 && w.seg > 0)
                        wait(o_free + 8 * t, (w.seg - 1) & 1);
                    wait(p_full + 16 * t + 8 * (i & 1), (i & 1 ? fill1++ : fill0++) & 1u);
                    tcgen05_after_sync();
                    // V, MN-major: 16 positions are 16 rows of 128 bytes
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        umma_ts(one, d, a + 8 * ks, v + ks * (2048 >> 4), idesc_o, ks > 0 ? 1u : more);
                        if (!CONV)
                            umma_ts(one, d, a + 32 + 8 * ks, v + ks * (2048 >> 4), idesc_o, 1u);
                    }
                    if (one) {
                        umma_commit(pv_done + 16 * t + 8 * (i & 1));
                        if (!TWO || (i & 1))
                            umma_commit(tile_free + 8 * st);
                    }
                }
            }
            z0 += 2 * n;
            if (__any_sync(0xffffffffu, *abort_flag != 0)) // all lanes alike
                break;
        }
        // nothing of this CTA's may be in flight when its tensor memory is freed
        if (one) {
            umma_commit(drain + 8 * (warp - 1));
            mbar_wait_bounded(drain + 8 * (warp - 1), 0);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 12) {
        // ---- softmax: thread = query row ----
        const int t = (warp - 4) >> 2, mine = threadIdx.x & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21); // this warp's lane quarter
        const uint32_t o_at = lanes + 256 + 128 * t;
        const float ninf = __uint_as_float(0xFF800000u);
        float *ml = reinterpret_cast<float *>(gsm + L.ml);
        // steps that took either S buffer so far, alike for both streams.  Every
        // barrier of a step exists once per buffer: its next phase needs a step that
        // this warp has not given yet, so a wait cannot fall two phases behind.
        uint32_t fills0 = 0, fills1 = 0;
        auto product_wait = [&](int k, int i) { // P V of step i (the last of its buffer) of stream k
            wait(pv_done + 16 * k + 8 * (i & 1), ((i & 1 ? fills1 : fills0) - 1) & 1u);
        };
        constexpr bool twice = TWICE;
        const int lane0 = twice ? 64 * t : 0; // the stream's first accumulator lane
        float *qinv = reinterpret_cast<float *>(gsm + L.inv) + (TWO ? 128 * t : 0);
        auto sync_all = [&] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
        auto sync_stream = [&] { // the warps that share a query tile
            if (TWO)
                asm volatile("bar.sync %0, 128;" ::"r"(3 + t) : "memory");
            else
                sync_all();
        };
        // Query rows of unit u into the operand tile, once the last S of the unit before is
        // done: before that unit's outputs are written, so that S goes on meanwhile.  Rows
        // beyond the unit's are left as they are: nothing is read from what they give.
        auto stage_queries = [&](const Walk &u) {
            const int g = u.u / p.tiles, base = (u.u - g * p.tiles) * ROWS + (TWO ? 128 * t : 0);
            const size_t first = (size_t)u.r * p.nq * p.Hkv * p.G + (size_t)g * p.G, pitch = (size_t)p.Hkv * p.G;
            const int rows = min(128, p.rows - base);
            sync_stream();
            if (u.seg > 0)
                wait(q_free, (u.seg - 1) & 1);
            stage_rows<CONV ? kRowsF16 : kRows16>(
                gsm + L.q + (TWO ? t * kTile16 : 0), 16384, twice ? 64 + rows : rows, TWO ? warp & 3 : warp - 4, TWO ? 4 : 8,
                [&](int i) {
                    i = twice ? min(i & 63, rows - 1) : i;
                    const int j = (base + i) / p.G;
                    return p.q + (first + j * pitch + (base + i - j * p.G)) * kDim;
                },
                [&](int i, float x) { qinv[i] = x; });
            fence_async_smem();
            if (CONV)
                sync_stream();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(q_full + (TWO ? 8 * t : 0));
        };
        if (w.x < w.x1)
            stage_queries(w);
        Walk nx = w;
        for (; w.x < w.x1; w = nx) {
            const int n = w.pages(), nsteps = TWO ? 2 * n : n;
            const int g = w.u / p.tiles, base = (w.u - g * p.tiles) * ROWS + (TWO ? 128 * t : 0);
            const int i_row = base + mine - lane0, i_read = min(max(i_row, 0), p.rows - 1), j = i_read / p.G;
            const bool real = i_row == i_read;
            const int first = (warp & 3) * 32 - lane0;
            const bool idle = first < 0 || base + first >= p.rows; // no row of this warp's is the unit's
            const size_t out_row = (size_t)w.r * p.nq * p.Hkv * p.G + (size_t)j * p.Hkv * p.G + (size_t)g * p.G + (i_read - j * p.G);
            const float sc = p.scale_log2 * (CONV && real ? qinv[mine] : 1.f);
            const int lim = w.seq_len + j;
            float m = ninf, l = 0.f; // reference maximum and denominator
            for (int i = 0; i < nsteps; ++i) {
                const int pos0 = (w.b + (TWO ? i >> 1 : i)) * kPage + 64 * (TWO ? i & 1 : t);
                const bool tail = pos0 + 64 > w.seq_len;
                const int seen = tail ? lim - pos0 : 64; // columns this row sees
                const uint32_t at_s = lanes + (TWO ? 128 * t + 64 * (i & 1) : 128 * (i & 1) + 64 * t);
                wait(s_full + (TWO ? 16 * t : 0) + 8 * (i & 1), (i & 1 ? fills1++ : fills0++) & 1u);
                if (idle) {
                    if (lane == 0)
                        mbar_arrive(p_full + 16 * t + 8 * (i & 1));
                    continue;
                }
                tcgen05_after_sync();
                // the extreme logit of the row (the scale's sign says which end).  The 64
                // columns stay in registers; with two converter groups a thread has fewer of
                // those, keeps columns 0 .. 31 and reads the others again
                constexpr int HELD = conv_groups(FMT, TWO) == 2 ? 32 : 64;
                uint32_t v[HELD];
                const bool neg = sc < 0.f;
                float mx = neg ? -ninf : ninf;
#pragma unroll
                for (int c = 64 - HELD; c >= 0; c -= HELD) {
#pragma unroll
                    for (int h = 0; h < HELD; h += 32)
                        tmem_ld32(at_s + c + h, v + h);
#pragma unroll
                    for (int h = 0; h < HELD; h += 32)
                        tmem_wait_ld(v + h);
                    if (tail || neg) {
#pragma unroll
                        for (int k = 0; k < HELD; ++k)
                            if (c + k < seen)
                                mx = neg ? fminf(mx, __uint_as_float(v[k])) : fmaxf(mx, __uint_as_float(v[k]));
                    } else {
                        float m4[4] = {ninf, ninf, ninf, ninf};
#pragma unroll
                        for (int k = 0; k < HELD; k += 2)
                            m4[(k >> 1) & 3] = fmaxf(m4[(k >> 1) & 3], fmaxf(__uint_as_float(v[k]), __uint_as_float(v[k + 1])));
                        mx = fmaxf(mx, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
                    }
                }
                mx *= sc;
                if (CONV)
                    mx -= kPUp16;
                const bool rise = mx > m + kSlack || (m == ninf && mx > ninf);
                if (__any_sync(0xffffffffu, rise)) { // rare, and so everything that it needs is in here
                    const float f = rise ? ex2(m - mx) : 1.f;
                    m = rise ? mx : m;
                    l *= f;
                    if (i > 0) {
                        product_wait(t, i - 1); // O holds every step before this one
                        tcgen05_after_sync();
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            float o[16];
                            tmem_ld16(o_at + 16 * c, o);
                            uint32_t r[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                r[k] = __float_as_uint(o[k] * f);
                            tmem_st16(o_at + 16 * c, r);
                        }
                    }
                }
                const float ref = m == ninf ? 0.f : m;
                const uint64_t sc2 = pair(sc, sc), ref2 = pair(-ref, -ref), minus = pair(-1.f, -1.f);
                uint64_t sum[2] = {0ull, 0ull};
                // the common step by itself: with the tests for a last page in its unrolled
                // loop 48 tokens over 2 x 131072 positions took 473 us, without 468
                auto to_p = [&](auto plain) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) { // 32 columns of S become P
                        if (HELD == 32 && c == 1) {
                            tmem_ld32(at_s + 32, v);
                            tmem_wait_ld(v);
                        }
                        const uint32_t *x = v + (HELD == 32 ? 0 : 32 * c);
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const int at = 32 * c + 2 * k;
                            float e0, e1;
                            unpair(fma2(pair(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), sc2, ref2), e0, e1);
                            e0 = ex2(e0);
                            e1 = ex2(e1);
                            if (!plain.value && tail) {
                                e0 = at < seen ? e0 : 0.f;
                                e1 = at + 1 < seen ? e1 : 0.f;
                            }
                            const uint64_t e = pair(e0, e1);
                            sum[k & 1] = add2(sum[k & 1], e);
                            if (CONV) {
                                hi[k] = pack_f16(e0, e1);
                            } else {
                                hi[k] = pack_bf16(e0, e1);
                                float d0, d1;
                                unpair(fma2(pair(__uint_as_float(hi[k] << 16), __uint_as_float(hi[k] & 0xFFFF0000u)), minus, e), d0, d1);
                                lo[k] = pack_bf16(d0, d1);
                            }
                        }
                        tmem_st16(at_s + 16 * c, hi);
                        if (!CONV)
                            tmem_st16(at_s + 32 + 16 * c, lo);
                    }
                };
                if (tail)
                    to_p(std::false_type{});
                else
                    to_p(std::true_type{});
                {
                    float a, b;
                    unpair(add2(sum[0], sum[1]), a, b);
                    l += a + b;
                }
                tmem_wait_st();
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(p_full + 16 * t + 8 * (i & 1));
            }

            // ---- end of the unit's share ----
            nx.next(p, heads);
            if (nx.x < nx.x1)
                stage_queries(nx);
            const bool whole = w.b == 0 && n == w.nb, ends = w.b + n == w.nb;
            float *slot = p.partial + (size_t)(2 * blockIdx.x + (ends ? 0 : 1)) * (ROWS * (kDim + 2));
            float M = m, Lsum = l, fa = 1.f, fb = 0.f;
            // stream 1's O where rows are there twice: 16-byte piece k of row i at 64 k + i, in the place
            // of rows 64 .. of the partial slot, which no output uses
            float4 *other = reinterpret_cast<float4 *>(slot + (size_t)64 * kDim) + (mine & 63);
            if (twice) {
                if (t == 1) {
                    if (w.seg > 0) // stream 0 has read the last unit's
                        asm volatile("bar.sync 2, 256;" ::: "memory");
                    product_wait(1, nsteps - 1);
                    tcgen05_after_sync();
#pragma unroll 1
                    for (int c = 0; c < 8 && !idle; ++c) {
                        float a[16];
                        tmem_ld16(o_at + 16 * c, a);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            other[64 * (4 * c + k)] = make_float4(a[4 * k], a[4 * k + 1], a[4 * k + 2], a[4 * k + 3]);
                    }
                    if (real) {
                        slot[(size_t)ROWS * kDim + mine] = m;
                        slot[(size_t)ROWS * (kDim + 1) + mine] = l;
                    }
                    tcgen05_before_sync();
                    sync_all();
                    if (lane == 0)
                        mbar_arrive(o_free + 8);
                    continue;
                }
                sync_all();
                if (real) {
                    const float mb = __ldcg(slot + (size_t)ROWS * kDim + 64 + mine), lb = __ldcg(slot + (size_t)ROWS * (kDim + 1) + 64 + mine);
                    M = fmaxf(m, mb);
                    fa = m == ninf ? 0.f : ex2(m - M);
                    fb = mb == ninf ? 0.f : ex2(mb - M);
                    Lsum = l * fa + lb * fb;
                }
            } else if (!TWO) {
                if (t == 1) {
                    ml[mine] = m;
                    ml[128 + mine] = l;
                }
                sync_all();
                const float mb = ml[mine], lb = ml[128 + mine];
                sync_all();
                if (t == 1)
                    continue; // stream 0 reads both accumulators (of as many steps)
                M = fmaxf(m, mb);
                fa = m == ninf ? 0.f : ex2(m - M);
                fb = mb == ninf ? 0.f : ex2(mb - M);
                Lsum = l * fa + lb * fb;
            }
            product_wait(t, nsteps - 1);
            if (!TWO && !twice)
                product_wait(1, nsteps - 1);
            tcgen05_after_sync();
            const int slot_row = (TWO ? 128 * t : 0) + mine;
            const float fin = Lsum > 0.f || Lsum != Lsum ? p.v_scale / Lsum : 0.f;
            const bool bad = later_bad[w.seg & 7] == w.seg + 1;
            float4 ahead[4]; // stream 1's next 16 columns
            if (twice)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    ahead[k] = __ldcg(other + 64 * k);
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
                float a[16], b2[16];
                __syncwarp();
                tmem_ld16(o_at + 16 * c, a);
                if (!TWO) {
                    if (twice) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float4 x = ahead[k];
                            b2[4 * k] = x.x, b2[4 * k + 1] = x.y, b2[4 * k + 2] = x.z, b2[4 * k + 3] = x.w;
                            if (c < 7)
                                ahead[k] = __ldcg(other + 64 * (4 * (c + 1) + k));
                        }
                    } else {
                        tmem_ld16(o_at + 128 + 16 * c, b2);
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        a[k] = a[k] * fa + b2[k] * fb;
                }
                if (bad) { // infinities and NaN of draft tokens' V, for the rows that see them
                    const float ref = M == ninf ? 0.f : M;
                    for (int pos = max(w.seq_len, w.b * kPage); pos < min(lim, (w.b + n) * kPage); ++pos) {
                        const long long page = p.block_table[(size_t)w.r * p.maxB + pos / kPage];
                        if (page < 0 || page >= p.num_pages)
                            continue;
                        float pr = 0.f;
                        bool have = false;
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float v = stored_value<FMT>(p.kv, (page * 2 + 1) * p.Hkv + g, pos % kPage, 16 * c + k);
                            if (finite(v))
                                continue;
                            if (!have) {
                                const uint16_t *qv = p.q + out_row * kDim;
                                for (int d = 0; d < kDim; ++d)
                                    pr = fmaf(__uint_as_float((uint32_t)qv[d] << 16),
                                              stored_value<FMT>(p.kv, page * 2 * p.Hkv + g, pos % kPage, d), pr);
                                pr = ex2(fmaf(pr, p.scale_log2, -ref));
                                have = true;
                            }
                            a[k] = fmaf(pr, v, a[k]);
                        }
                    }
                }
                if (real) {
                    if (whole) {
                        uint4 d[2];
                        uint32_t *e = &d[0].x;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            e[k] = pack_bf16(a[2 * k] * fin, a[2 * k + 1] * fin);
                        uint4 *dst = reinterpret_cast<uint4 *>(p.out + out_row * kDim + 16 * c);
                        dst[0] = d[0];
                        dst[1] = d[1];
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(slot + (size_t)slot_row * kDim + 16 * c);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            dst[k] = make_float4(a[4 * k], a[4 * k + 1], a[4 * k + 2], a[4 * k + 3]);
                    }
                }
            }
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(o_free + 8 * t);
                if (!TWO && !twice)
                    mbar_arrive(o_free + 8);
            }
            if (twice && nx.x < nx.x1)
                asm volatile("bar.arrive 2, 256;" ::: "memory");
            if (real) {
                if (whole) {
                    p.lse[out_row] = Lsum == 0.f ? ninf : (M + log2f(Lsum)) * 0.6931471805599453f;
                } else {
                    slot[(size_t)ROWS * kDim + slot_row] = M;
                    slot[(size_t)ROWS * (kDim + 1) + slot_row] = Lsum;
                }
            }
        }
    } else if (CONV && warp >= 12) {
        // ---- converters: a ring tile to a 16-bit tile, in the order of use ----
        const int grp = (warp - 12) >> 2, row = (warp & 3) * 32 + lane;
        int z = 0;
        for (; w.x < w.x1; w.next(p, heads)) {
            const int n = w.pages(), cached = w.seq_len + p.nq - 1;
            int kp = 0, vp = 0;
            for (int i = 0; i < 2 * n; ++i, ++z) {
                const bool is_k = kp < n && order_of_k<TWO>(kp) == i;
                const int page0 = (w.b + (is_k ? kp++ : vp++)) * kPage;
                if (conv_groups(FMT, TWO) == 2 && (z & 1) != grp)
                    continue;
                const bool tail = !is_k && page0 + kPage > w.seq_len;
                const bool drop = tail && page0 + row >= cached;              // not cached
                const bool check = tail && !drop && page0 + row >= w.seq_len; // seen by later tokens only
                wait(full + 8 * (z % TILES), (uint32_t)(z / TILES) & 1u);
                if (z >= kStaged)
                    wait(sempty + 8 * (z % kStaged), (uint32_t)(z / kStaged - 1) & 1u);
                const uint8_t *src = gsm + (z % TILES) * TB;
                uint8_t *dst = gsm + L.staged + (z % kStaged) * kTile16 + row * 128;
                bool bad = false;
                if (FMT == kFmtFp8) {
#pragma unroll 2 // (all: 426 us for 413, 48 tokens over 2 x 131072; NVFP4 loses with less, 507 for 488)
                    for (int c = 0; c < 8; ++c) { // 16 dimensions
                        const uint4 d = *reinterpret_cast<const uint4 *>(src + row * 128 + ((c ^ (row & 7)) << 4));
                        uint32_t e[4] = {d.x, d.y, d.z, d.w}, o[8];
                        if (tail) {
#pragma unroll
                            for (int q = 0; q < 16; ++q)
                                if (check && ((e[q >> 2] >> (8 * (q & 3))) & 0x7Fu) == 0x7Fu)
                                    e[q >> 2] &= ~(0xFFu << (8 * (q & 3))), bad = true;
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                e[q] = drop ? 0u : e[q];
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            e4m3x4_to_f16x2x2(e[q], o[2 * q], o[2 * q + 1]);
                        uint8_t *at = dst + (c >> 2) * 16384;
                        *reinterpret_cast<uint4 *>(at + (((2 * c) & 7) ^ (row & 7)) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4 *>(at + (((2 * c + 1) & 7) ^ (row & 7)) * 16) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                } else {
                    uint64_t sc = *reinterpret_cast<const uint64_t *>(src + 8192 + row * 8);
                    uint32_t zero = 0u; // 16-dim groups that become zeros
                    if (tail) {
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            if (check && ((sc >> (8 * q)) & 0x7Fu) == 0x7Fu)
                                zero |= 1u << q, bad = true;
                        zero = drop ? 0xFFu : zero;
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            if ((zero >> q) & 1u)
                                sc &= ~(0xFFull << (8 * q)); // a scale of 0: products of 0
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) { // 32 dimensions, two scales
                        const uint4 d = *reinterpret_cast<const uint4 *>(src + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
                        const uint32_t e[4] = {d.x, d.y, d.z, d.w};
                        const uint32_t s2 = e4m3x2_to_f16x2((uint32_t)(sc >> (16 * c)) & 0xFFFFu);
                        const uint32_t sa = __byte_perm(s2, s2, 0x1010), sb = __byte_perm(s2, s2, 0x3232);
                        uint8_t *at = dst + (c >> 1) * 16384;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t o[4];
                            e2m1x8_scaled_f16x2(e[q], q < 2 ? sa : sb, o);
                            *reinterpret_cast<uint4 *>(at + ((((c & 1) * 4 + q) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    }
                }
                if (bad)
                    later_bad[w.seg & 7] = w.seg + 1;
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(empty + 8 * (z % TILES));
                    mbar_arrive(sfull + 8 * (z % kStaged));
                }
            }
        }
    }

    tcgen05_before_sync();
    __syncthreads();
    if (warp == 1) {
        tcgen05_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

template <int FMT, bool TWO, bool TWICE = false>
cudaError_t launch_t(const DenseParams &p, const CUtensorMap &map, int ctas, cudaStream_t stream)
{
    constexpr int smem = smem_layout(FMT, TWO).total;
    cudaError_t e = cudaFuncSetAttribute(dense_umma_kernel<FMT, TWO, TWICE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    e = launch_kernel(dense_umma_kernel<FMT, TWO, TWICE>, dim3(ctas), dim3(threads_of(FMT, TWO)), smem, stream, false, map, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace

cudaError_t launch_dense_umma(const DenseParams &p, const CUtensorMap &map, int kv_dtype, int ctas, cudaStream_t stream)
{
    const bool two = p.rows > 128;
    if (kv_dtype == MSA_BF16)
        return two ? launch_t<kFmtBf16, true>(p, map, ctas, stream) : launch_t<kFmtBf16, false>(p, map, ctas, stream);
    if (kv_dtype == MSA_FP8_E4M3)
        return two ? launch_t<kFmtFp8, true>(p, map, ctas, stream) : launch_t<kFmtFp8, false>(p, map, ctas, stream);
    return two ? launch_t<kFmtF4, true>(p, map, ctas, stream)
           : p.rows <= 64 ? launch_t<kFmtF4, false, true>(p, map, ctas, stream)
                          : launch_t<kFmtF4, false>(p, map, ctas, stream);
}

} // namespace msa
