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
// S^T = K Q^T on the tcgen05 tensor cores: positions are the 128 lanes of an
// accumulator and query rows its columns, so the sum over rows is a sum over a
// thread's own columns, and a warp reads and writes 32 consecutive weights.  No
// exchange between threads, no atomics; rows are added in a fixed order.
//
// bf16 keys are operands as they land, and so are E4M3 keys: each bf16 query row then is
// two columns, an E4M3 pair hi + lo / 16 after a power of two that brings its largest
// element to (224, 448].  The pair is exact for elements of 2^-6 or more, 2^-13.8 of the
// row's largest, and off by at most 2^-14, 2^-21.8 of the largest, below.  (One token over
// 0.59 GB of E4M3 keys: 116 us, 5.1 TB/s; 153 us with keys widened to f16.  8 tokens over
// 64 x 32768 positions: 109 us for 133, 16 tokens 189 for 209.)  NVFP4 keys are widened to
// f16 by converter warps.
//
// What bounds it: the bytes of K and of the weights with few rows; with many the chain
// of MMA, load from tensor memory and exponentials of a buffer, and that few K tiles fit
// beside the query rows (32 tokens over 2 x 32768 bf16 positions: 46 us, 0.74 PFLOP/s).
// Two groups (an MMA issuer, four softmax warps and, where keys are widened, four
// converter warps each) share the work, so that one's waits pass behind the other's work:
// each takes every second page, 128 accumulator columns at a time in two buffers (both
// groups on every page, with half of the columns each, was 5 .. 25% slower).  The query
// rows of a (request, KV head), up to 512 (NVFP4: 256) at a time, stay in shared memory.
//
// After a sparse step only pages that some token of the request selected are
// read; a bitmap of 64 token bits per page, built in shared memory, says which
// rows count.  The weights of the other pages are only faded.
//
// Warps: 0 producer and bitmaps, 1 and 2 issuers, 4-7 and 8-11 softmax, 12-15
// and 16-19 converters of group 0 and 1.
#include <type_traits>

#include "msa_umma.cuh"

namespace msa {
namespace {

constexpr int kPagesAtATime = 512; // pages whose bitmaps are held at a time
constexpr int kTile16 = 32768;     // a 16-bit K tile
constexpr int kMaxRing = 16;
constexpr int kSmemMax = 232192;   // what the layouts below stay under (232448 with the static part)

__host__ __device__ constexpr int threads_of(int fmt)
{
    return fmt == kFmtF4 ? 640 : 384;
}

// Query rows in shared memory at a time (NVFP4 keys need staged tiles besides).
__host__ __device__ constexpr int query_rows(int fmt)
{
    return fmt == kFmtF4 ? 256 : 512;
}

// Rows held are padded to whole loads of 32 accumulator columns.
__host__ __device__ constexpr int padded(int fmt, int rows)
{
    return fmt == kFmtFp8 ? (rows + 15) / 16 * 16 : (rows + 31) / 32 * 32;
}

// Shared memory by the query rows held: the rest is the ring
// of K tiles.  Ring and staged tiles are even in number: a slot belongs to one
// group, which follows all of its barriers' phases.
struct Smem {
    int ring, staged, q, cols, tok, mask, bars, misc, total;
    int depth, nstaged;
};

__host__ __device__ inline Smem smem_layout(int fmt, int qpad, bool masks)
{
    Smem s{};
    const int rest = qpad * (256 + 8 + 1) + (masks ? 2 * kPagesAtATime * 8 : 0) + (2 * kMaxRing + 32) * 8 + 64 + 1024 + 256;
    int room = 232448 - rest;
    s.nstaged = fmt != kFmtF4 ? 0 : room >= 6 * kTile16 ? 4 : 2;
    room -= s.nstaged * kTile16;
    s.depth = room / tile_bytes(fmt) / 2 * 2;
    s.depth = s.depth > kMaxRing ? kMaxRing : s.depth;
    s.staged = 0;
    s.q = s.nstaged * kTile16;
    s.ring = s.q + qpad * 256;
    s.cols = s.ring + s.depth * tile_bytes(fmt);
    s.tok = s.cols + qpad * 8;
    s.mask = (s.tok + qpad + 15) / 16 * 16;
    s.bars = s.mask + (masks ? 2 * kPagesAtATime * 8 : 0);
    s.misc = s.bars + (2 * kMaxRing + 32) * 8;
    s.total = s.misc + 64 + 1024;
    return s;
}

template <int FMT>
__global__ void __launch_bounds__(threads_of(FMT), 1)
    weight_kernel(const __grid_constant__ CUtensorMap map, const WeightParams p, const Smem L)
{
    constexpr int TB = tile_bytes(FMT), NT = threads_of(FMT);
    constexpr bool CONV = FMT == kFmtF4, PAIR = FMT == kFmtFp8;
    constexpr int kQRows = query_rows(FMT);
    extern __shared__ uint8_t smem_raw[];
    __shared__ int scan_tmp[NT / 32 + 1];
    __shared__ int start_r, start_before;
    __shared__ uint32_t tmem_slot;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *gsm = smem_raw + (smem - smem_u32(smem_raw));
    const uint32_t full = smem + L.bars, empty = full + kMaxRing * 8, sfull = empty + kMaxRing * 8, sempty = sfull + 32,
                   q_full = sempty + 32, q_free = q_full + 8, s_full = q_free + 8, s_free = s_full + 32, m_full = s_free + 32,
                   m_free = m_full + 16, drain = m_free + 16;
    // bf16 keys: -lse of four query rows a word (one load for four: 137 -> 129 us at 256 rows);
    // else the scales of two rows, then their -lse
    float4 *cols = reinterpret_cast<float4 *>(gsm + L.cols);
    uint8_t *tok = gsm + L.tok;                              // token of a column
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gsm + L.misc);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rows = p.nq * p.G, heads = p.Hkv;
    const bool sparse = p.selected != nullptr;
    const long long wl = p.wait_limit;

    if (threadIdx.x == 0) {
        prefetch_tensormap(&map);
        for (int i = 0; i < L.depth; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, CONV ? 4 : 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(sfull + 8 * i, 4);
            mbar_init(sempty + 8 * i, 1);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(s_free + 8 * i, 4);
        }
        mbar_init(q_full, 8);
        mbar_init(q_free, 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(m_full + 8 * i, 1);
            mbar_init(m_free + 8 * i, CONV ? 18 : 10);
            mbar_init(drain + 8 * i, 1);
        }
        fence_mbar_init();
        *abort_flag = 0;
    }
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
    if (w.x < w.x1)
        for (int r = lo, b = before; r < hi; ++r) {
            bool bad;
            const int nb = cached_blocks(p.seq_lens[r], p.nq, p.maxB, &bad);
            if (nb > 0 && b * heads <= w.x && w.x < (b + nb) * heads) {
                start_r = r;
                start_before = b;
            }
            b += nb;
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
    // a wait that ran out: the CTA's roles run on without waiting, so that all reach the end
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!ring_wait(bar, parity, abort_flag, wl) && !*abort_flag) {
            *abort_flag = 1;
            set_error(p.err, kErrTimeout);
        }
    };
    // Every role walks units, chunks of query rows and (after a sparse step) runs of
    // pages alike: `round` counts the runs, z the pages that are read (group z & 1),
    // st / ph the ring slot of page z.
    int round = 0, z = 0, st = 0;
    uint32_t ph = 0;
    auto bits_of = [&](int i) { // token bits of page i of the run
        return sparse ? reinterpret_cast<const volatile unsigned long long *>(gsm + L.mask)[(round & 1) * kPagesAtATime + i] : ~0ull;
    };
    auto next_tile = [&] {
        ++z;
        if (++st == L.depth) {
            st = 0;
            ph ^= 1u;
        }
    };
    auto run_begins = [&] {
        if (sparse)
            wait(m_full + 8 * (round & 1), (uint32_t)(round >> 1) & 1u);
    };
    auto run_ends = [&] {
        if (sparse) {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(m_free + 8 * (round & 1));
        }
        ++round;
    };

    if (warp == 0) {
        // ---- producer ----
        for (; w.x < w.x1; w.next(p, heads)) {
            const int n = w.pages(), g = w.u;
            const int32_t *row = p.block_table + (size_t)w.r * p.maxB;
            for (int q0 = 0; q0 < rows; q0 += kQRows)
                for (int s0 = 0; s0 < n; s0 += sparse ? kPagesAtATime : n, ++round) {
                    const int sb = w.b + s0, sn = sparse ? min(kPagesAtATime, n - s0) : n;
                    unsigned long long *mask = reinterpret_cast<unsigned long long *>(gsm + L.mask) + (round & 1) * kPagesAtATime;
                    if (sparse) {
                        if (round >= 2)
                            wait(m_free + 8 * (round & 1), (uint32_t)((round >> 1) - 1) & 1u);
                        for (int i = lane; i < sn; i += 32)
                            mask[i] = 0ull;
                        __syncwarp();
                        // one bit per token for every page of [sb, sb + sn) in its table
                        for (int i0 = lane; i0 < p.nq * p.k; i0 += 256) { // eight entries a lane in flight
                            int blk[8];
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                const int i = i0 + 32 * c, j = i / p.k;
                                blk[c] = i < p.nq * p.k ? p.selected[(((size_t)w.r * p.nq + j) * p.Hs + (p.Hs > 1 ? g : 0)) * p.k + (i - j * p.k)] : -1;
                            }
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                const int j = (i0 + 32 * c) / p.k;
                                if (blk[c] < -1 || (blk[c] >= 0 && (long long)blk[c] * kPage >= w.seq_len + j))
                                    set_error(p.err, kErrSelection);
                                else if (blk[c] >= sb && blk[c] < sb + sn)
                                    atomicOr(&mask[blk[c] - sb], 1ull << j);
                            }
                        }
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(m_full + 8 * (round & 1));
                    }
                    for (int i = 0; i < sn; i += 32) {
                        const bool want = i + lane < sn && (!sparse || bits_of(i + lane) != 0ull);
                        const int mine = want ? row[sb + i + lane] : 0;
                        for (uint32_t todo = __ballot_sync(0xffffffffu, want); todo; todo &= todo - 1) {
                            long long page = __shfl_sync(0xffffffffu, mine, __ffs(todo) - 1);
                            if (page < 0 || page >= p.num_pages) {
                                if (lane == 0)
                                    set_error(p.err, kErrPage);
                                page = 0; // in the pool: the outputs of the call are unspecified
                            }
                            if (z >= L.depth)
                                wait(empty + 8 * st, ph ^ 1u);
                            if (__any_sync(0xffffffffu, *abort_flag != 0))
                                continue;
                            if (lane == 0) {
                                mbar_arrive_expect_tx(full + 8 * st, TB);
                                load_tile<FMT>(smem + L.ring + st * TB, &map, p.kv, (page * 2) * p.Hkv + g, full + 8 * st);
                            }
                            __syncwarp();
                            next_tile();
                        }
                    }
                }
        }
        if (lane == 0) // the CTA's memory must outlive the copies in flight
            for (int i = max(0, z - L.depth); i < z; ++i)
                mbar_wait_bounded(full + 8 * (i % L.depth), (uint32_t)(i / L.depth) & 1u);
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        // ---- MMA issuers: the whole warp, lane 0 issuing ----
        const int grp = warp - 1;
        const uint32_t one = lane == 0, tm = uniform(tmem + 256 * grp), base = uniform(smem), q = uniform(desc_low(base + L.q, 16));
        const uint32_t idesc = umma_idesc_bf16(128, 0, 0, 0) & (FMT != kFmtBf16 ? ~((1u << 7) | (1u << 10)) : ~0u); // f16 or E4M3, or bf16
        uint32_t item = 0, qround = 0;
        for (; w.x < w.x1; w.next(p, heads)) {
            const int n = w.pages();
            for (int q0 = 0; q0 < rows; q0 += kQRows, ++qround) {
                const int qpad = padded(FMT, min(kQRows, rows - q0));
                const int ncols = PAIR ? 2 * qpad : qpad;
                const uint32_t half = uniform(qpad * 128 >> 4);
                wait(q_full, qround & 1u);
                for (int s0 = 0; s0 < n; s0 += sparse ? kPagesAtATime : n) {
                    const int sn = sparse ? min(kPagesAtATime, n - s0) : n;
                    run_begins();
                    for (int i = 0; i < sn; ++i) {
                        if (bits_of(i) == 0ull)
                            continue;
                        if ((z & 1) == grp) {
                            const int slot = CONV ? z % L.nstaged : st;
                            const uint32_t k = uniform(desc_low(base + (CONV ? L.staged + slot * kTile16 : L.ring + slot * TB), 16));
                            wait(CONV ? sfull + 8 * slot : full + 8 * st, CONV ? (uint32_t)(z / L.nstaged) & 1u : ph);
                            for (int c = 0; c < ncols; c += 128, ++item) {
                                const uint32_t d = tm + uniform(128 * (item & 1u)), b = q + uniform(c * 128 >> 4);
                                const uint32_t id = uniform(idesc | (uint32_t)(min(128, ncols - c) >> 3) << 17);
                                if (item >= 2)
                                    wait(s_free + 16 * grp + 8 * (item & 1u), ((item >> 1) - 1) & 1u);
                                tcgen05_after_sync();
                                if (PAIR) { // 32 dimensions an MMA
#pragma unroll
                                    for (uint32_t ks = 0; ks < 4; ++ks)
                                        umma_ss8(one, d, k + ks * 2, b + ks * 2, id, ks > 0);
                                } else {
#pragma unroll
                                    for (uint32_t ks = 0; ks < 4; ++ks)
                                        umma_ss(one, d, k + ks * 2, b + ks * 2, id, ks > 0);
#pragma unroll
                                    for (uint32_t ks = 0; ks < 4; ++ks)
                                        umma_ss(one, d, k + 1024 + ks * 2, b + half + ks * 2, id, 1u);
                                }
                                if (one)
                                    umma_commit(s_full + 16 * grp + 8 * (item & 1u));
                            }
                            if (one)
                                umma_commit(CONV ? sempty + 8 * slot : empty + 8 * st);
                        }
                        next_tile();
                    }
                    run_ends();
                }
                if (one)
                    umma_commit(q_free);
            }
        }
        if (one) { // nothing of this CTA's may be in flight when its tensor memory is freed
            umma_commit(drain + 8 * grp);
            mbar_wait_bounded(drain + 8 * grp, 0);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 12) {
        // ---- softmax: thread = position ----
        const int grp = (warp - 4) >> 2, mine = (warp & 3) * 32 + lane, me = threadIdx.x - 128;
        const uint32_t s_at = tmem + 256 * grp + ((uint32_t)(warp & 3) << 21);
        const float inf = __uint_as_float(0x7F800000u);
        uint32_t item = 0, qround = 0;
        for (; w.x < w.x1; w.next(p, heads)) {
            const int n = w.pages(), g = w.u, cached = w.seq_len + p.nq - 1;
            const size_t first_row = (size_t)w.r * p.nq * p.Hkv * p.G + (size_t)g * p.G, pitch = (size_t)p.Hkv * p.G;
            const size_t wrow = ((size_t)w.r * p.Hkv + g) * p.maxB * kPage;
            for (int q0 = 0; q0 < rows; q0 += kQRows, ++qround) {
                const int qpad = padded(FMT, min(kQRows, rows - q0));
                asm volatile("bar.sync 1, 256;" ::: "memory"); // the last rows' columns are done with
                if (qround > 0)
                    wait(q_free, (qround - 1) & 1u);
                // padding columns repeat the last row (zeros would turn an infinite key into NaN)
                // and count nothing, as do tokens that attended to nothing (lse = -inf)
                auto source = [&](int i) {
                    const int at = min(q0 + i, rows - 1), j = at / p.G;
                    return first_row + j * pitch + (at - j * p.G);
                };
                for (int i = me; i < qpad; i += 256) {
                    const float e = q0 + i < rows ? p.lse[source(i)] : inf;
                    reinterpret_cast<float *>(cols)[FMT == kFmtBf16 ? i : (i >> 1) * 4 + 2 + (i & 1)] = e == -inf ? -inf : e * -1.4426950408889634f;
                    tok[i] = (uint8_t)(min(q0 + i, rows - 1) / p.G);
                }
                stage_rows<FMT == kFmtBf16 ? kRows16 : PAIR ? kRowsPair : kRowsF16>(
                    gsm + L.q, qpad * 128, qpad, warp - 4, 8, [&](int i) { return p.q + source(i) * kDim; },
                    [&](int i, float inv) { reinterpret_cast<float *>(cols + (i >> 1))[i & 1] = p.scale_log2 * inv; });
                fence_async_smem();
                asm volatile("bar.sync 1, 256;" ::: "memory");
                if (lane == 0)
                    mbar_arrive(q_full);
                const float *src = q0 > 0 ? p.weights_out : p.weights_in;
                for (int s0 = 0; s0 < n; s0 += sparse ? kPagesAtATime : n) {
                    const int sn = sparse ? min(kPagesAtATime, n - s0) : n, sb = w.b + s0;
                    run_begins();
                    // pages that no token looked at: their weights fade (four loads in flight)
                    for (int i0 = warp - 4; sparse && q0 == 0 && i0 < sn; i0 += 32) {
                        float4 v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int i = i0 + 8 * k;
                            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (src && i < sn && bits_of(i) == 0ull)
                                v[k] = *reinterpret_cast<const float4 *>(src + wrow + (size_t)(sb + i) * kPage + 4 * lane);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int i = i0 + 8 * k, at = (sb + i) * kPage + 4 * lane;
                            if (i >= sn || bits_of(i) != 0ull)
                                continue;
                            const float e[4] = {v[k].x * p.decay, v[k].y * p.decay, v[k].z * p.decay, v[k].w * p.decay};
                            if (at + 4 <= w.seq_len - 1) {
                                *reinterpret_cast<float4 *>(p.weights_out + wrow + at) = make_float4(e[0], e[1], e[2], e[3]);
                            } else {
                                for (int c = 0; c < 4; ++c)
                                    if (at + c < cached)
                                        p.weights_out[wrow + at + c] = at + c < w.seq_len - 1 ? e[c] : 0.f;
                            }
                        }
                    }
                    for (int i = 0; i < sn; ++i) {
                        const unsigned long long bits = bits_of(i);
                        if (bits == 0ull)
                            continue;
                        if ((z++ & 1) != grp)
                            continue;
                        const int at = (sb + i) * kPage + mine;
                        float old = 0.f;
                        if (q0 > 0 ? at < cached : src && at < w.seq_len - 1)
                            old = src[wrow + at];
                        const bool whole_page = (sb + i + 1) * kPage <= w.seq_len, part = sparse || !whole_page;
                        uint64_t sum[2] = {0ull, 0ull};
                        const int ncols = PAIR ? 2 * qpad : qpad;
                        // 32 accumulator columns: 32 query rows, or 16 as hi + lo
                        auto add_rows = [&](auto partly, int col, const uint32_t *v) {
                            constexpr int ROWS = PAIR ? 16 : 32;
                            const int row0 = PAIR ? col >> 1 : col;
                            const float4 *info = cols + (row0 >> (FMT == kFmtBf16 ? 2 : 1));
                            const uint64_t same = pair(p.scale_log2, p.scale_log2);
#pragma unroll
                            for (int k = 0; k < ROWS / 2; ++k) {
                                const float4 f = info[FMT == kFmtBf16 ? k >> 1 : k];
                                const uint64_t scales = FMT == kFmtBf16 ? same : pair(f.x, f.y);
                                const uint64_t minus = FMT == kFmtBf16 && k % 2 == 0 ? pair(f.x, f.y) : pair(f.z, f.w);
                                uint64_t x;
                                if (PAIR)
                                    x = fma2(pair(__uint_as_float(v[(4 * k + 1) & 31]), __uint_as_float(v[(4 * k + 3) & 31])), pair(0.0625f, 0.0625f),
                                             pair(__uint_as_float(v[(4 * k) & 31]), __uint_as_float(v[(4 * k + 2) & 31])));
                                else
                                    x = pair(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
                                float e0, e1;
                                unpair(fma2(x, scales, minus), e0, e1);
                                e0 = ex2(e0);
                                e1 = ex2(e1);
                                if (partly.value) { // a token counts where it looked at this block and sees the position
                                    const int j0 = tok[row0 + 2 * k], j1 = tok[row0 + 2 * k + 1];
                                    e0 = ((bits >> j0) & 1ull) && at < w.seq_len + j0 ? e0 : 0.f;
                                    e1 = ((bits >> j1) & 1ull) && at < w.seq_len + j1 ? e1 : 0.f;
                                }
                                sum[k & 1] = add2(sum[k & 1], pair(e0, e1));
                            }
                        };
                        auto add_page = [&](auto partly) {
                            for (int c0 = 0; c0 < ncols; c0 += 128, ++item) {
                                const int cn = min(128, ncols - c0);
                                wait(s_full + 16 * grp + 8 * (item & 1u), (item >> 1) & 1u);
                                tcgen05_after_sync();
                                const uint32_t s_buf = s_at + 128 * (item & 1u);
                                // whole buffers: the next 32 columns are loaded meanwhile (243 -> 228 us at
                                // 512 rows; the instances with converters have no registers for it)
                                if (!CONV && !partly.value && cn == 128) {
                                    uint32_t v2[2][32];
                                    tmem_ld32(s_buf, v2[0]);
                                    tmem_wait_ld(v2[0]);
#pragma unroll
                                    for (int c = 0; c < 4; ++c) {
                                        if (c < 3) {
                                            tmem_ld32(s_buf + 32 * (c + 1), v2[(c + 1) & 1]);
                                        } else {
                                            tcgen05_before_sync();
                                            __syncwarp();
                                            if (lane == 0)
                                                mbar_arrive(s_free + 16 * grp + 8 * (item & 1u));
                                        }
                                        add_rows(std::false_type{}, c0 + 32 * c, v2[c & 1]);
                                        if (c < 3)
                                            tmem_wait_ld(v2[(c + 1) & 1]);
                                    }
                                    continue;
                                }
                                uint32_t v[32];
#pragma unroll 1
                                for (int c = 0; c < cn; c += 32) {
                                    bool all = false;
                                    if (partly.value) { // the tokens of these columns: none or all of them?
                                        const int r0 = PAIR ? (c0 + c) >> 1 : c0 + c, r1 = r0 + (PAIR ? 15 : 31);
                                        const int j0 = tok[r0], j1 = tok[r1];
                                        const unsigned long long those = (~0ull >> (63 - (j1 - j0))) << j0;
                                        if ((bits & those) == 0ull)
                                            continue;
                                        all = (bits & those) == those && whole_page;
                                    }
                                    tmem_ld32(s_buf + c, v);
                                    tmem_wait_ld(v);
                                    if (partly.value && !all)
                                        add_rows(std::true_type{}, c0 + c, v);
                                    else
                                        add_rows(std::false_type{}, c0 + c, v);
                                    __syncwarp();
                                }
                                tcgen05_before_sync();
                                __syncwarp();
                                if (lane == 0)
                                    mbar_arrive(s_free + 16 * grp + 8 * (item & 1u));
                            }
                        };
                        if (part)
                            add_page(std::true_type{});
                        else
                            add_page(std::false_type{});
                        float a, b;
                        unpair(add2(sum[0], sum[1]), a, b);
                        if (at < cached)
                            p.weights_out[wrow + at] = (q0 > 0 ? old : old * p.decay) + (a + b);
                    }
                    run_ends();
                }
            }
        }
    } else if (CONV && warp >= 12) {
        // ---- converters: a ring tile to a 16-bit tile ----
        const int grp = (warp - 12) >> 2, row = (warp & 3) * 32 + lane;
        for (; w.x < w.x1; w.next(p, heads)) {
            const int n = w.pages();
            for (int q0 = 0; q0 < rows; q0 += kQRows)
                for (int s0 = 0; s0 < n; s0 += sparse ? kPagesAtATime : n) {
                    const int sn = sparse ? min(kPagesAtATime, n - s0) : n;
                    run_begins();
                    for (int i = 0; i < sn; ++i) {
                        if (bits_of(i) == 0ull)
                            continue;
                        if ((z & 1) == grp) {
                            const int slot = z % L.nstaged;
                            wait(full + 8 * st, ph);
                            if (z >= L.nstaged)
                                wait(sempty + 8 * slot, (uint32_t)(z / L.nstaged - 1) & 1u);
                            widen_row(gsm + L.ring + st * TB, gsm + L.staged + slot * kTile16, row);
                            fence_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                mbar_arrive(empty + 8 * st);
                                mbar_arrive(sfull + 8 * slot);
                            }
                        }
                        next_tile();
                    }
                    run_ends();
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

template <int FMT>
cudaError_t launch_t(const WeightParams &p, const CUtensorMap &map, int ctas, cudaStream_t stream)
{
    const int rows = p.nq * p.G, qpad = padded(FMT, rows < query_rows(FMT) ? rows : query_rows(FMT));
    const Smem L = smem_layout(FMT, qpad, p.selected != nullptr);
    // the same limit for every shape: another host thread may launch another shape meanwhile
    if (L.total > kSmemMax)
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(weight_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e == cudaSuccess)
        e = launch_kernel(weight_kernel<FMT>, dim3(ctas), dim3(threads_of(FMT)), (size_t)L.total, stream, false, map, p, L);
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
