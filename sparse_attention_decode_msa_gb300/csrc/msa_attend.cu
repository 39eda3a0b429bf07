// msa_attend.cu -- attention of ragged query rows over paged states: cross attention
// (every token of a request sees all of its states) and the attention of a prompt's
// chunk (causal).
//
// For a query row q of a token that sees n positions: s_p = scale q . K[p], m the running
// maximum, out = sum 2^(s - m) V / sum 2^(s - m), lse = m + ln sum, in one pass over the
// pages, fp32.
//
// Work.  The rows of a (request, KV head) are cut into units of T = floor(256 / G) tokens
// with their G heads, at most 256 rows; a unit's pages are those that its last token
// sees.  All units laid end to end (request, KV head, unit) are a line of pages that is
// cut into equal ranges, one a CTA, whatever the lengths are; a unit cut between CTAs is
// joined by attend_join_kernel in the order of its pages.  Pages before unit i of a causal
// request are a sum of floors, which a Euclid-like recursion gives in a few steps: no
// table, no kernel before this one.
//
// Two streams of 128 rows share a CTA's pages, so that the tensor cores work for one while
// the other is in its softmax: rows 128 t .. of the unit are stream t's, and both take
// every page; a unit of up to 128 rows goes to both streams, which take its pages in
// turn, and their (m, l, O) are added at the end.
//
// Operands: Q in shared memory (K-major, 128-byte swizzle), K tiles as TMA lands them, P in
// tensor memory over the S it came from, V tiles as landed (MN-major).  E4M3 and NVFP4 tiles
// are widened to f16 by converter warps, and P is f16: off by 2^-11 of p.  Over bf16 pages P
// is bf16 (V's type, which a product needs): each p is off by 2^-8 of itself at most, and
// the sum that divides is that of the rounded p, so that an output is a mean of values
// with weights that are off by 2^-8 of themselves and still sum to 1: off by 2^-8 of the
// weighted mean distance of the values from it at most, exact where all values or all
// logits are alike.  lse has the sum of the p as they are.  (P as a pair of bf16, as the dense decode
// has it, doubles the products of P V.)
//
// TMEM columns: S/P of stream t at 128 t, O of stream t at 256 + 128 t.
// Warps: 0 TMA producer, 1 issues all MMAs (and owns the TMEM), 2 clears what must not be
// multiplied from V tiles on last pages (bf16), 3 outputs of requests without states, 4-7
// and 8-11 softmax of stream 0 and 1, 12-15 converters (E4M3, NVFP4).
#include <type_traits>

#include "msa_ragged.cuh"
#include "msa_umma.cuh"

namespace msa {
namespace {

constexpr int kRows = 256;       // query rows of a unit
constexpr int kTile16 = 32768;   // a 16-bit K, V or Q tile
constexpr int kStaged = 4;       // widened tiles in flight
constexpr float kSlack = 8.f;    // how far (log2) a row's maximum may pass its reference before O is rescaled
constexpr float kPUp16 = 7.f;    // f16 P: 2^7 2^(s - m), at most 2^15 with the slack
constexpr int kSlotFloats = kRows * (kDim + 3); // o[rows][128], m, l, l of the rounded p
constexpr int kMinPages = 2;     // pages a CTA takes at least

__host__ __device__ constexpr int threads_of(int fmt)
{
    return fmt == kFmtBf16 ? 384 : 512;
}

// Registers a thread of warpgroup 0, of the softmax warpgroups (whose threads hold a row of 128 columns,
// or half of one) and of the converters.  The sums are what the block is launched with (168 and 128 a thread).
constexpr int kRegs0 = 72;
__host__ __device__ constexpr int regs_softmax(int fmt)
{
    return fmt == kFmtBf16 ? 216 : 176;
}
constexpr int kRegsConv = 88;
static_assert(kRegs0 + 2 * regs_softmax(kFmtBf16) <= 3 * 168 && kRegs0 + 2 * regs_softmax(kFmtFp8) + kRegsConv <= 4 * 128, "registers");

__host__ __device__ constexpr int ring_tiles(int fmt)
{
    return fmt == kFmtBf16 ? 5 : 2;
}

struct Smem {
    int staged, q, ml, inv, bars, misc, total;
};

// Tiles that the issuer takes: widened ones, or the ring's own once they have passed the clearing warp.
__host__ __device__ constexpr int ready_tiles(int fmt)
{
    return fmt == kFmtBf16 ? ring_tiles(fmt) : kStaged;
}

// Barriers: full[], empty[] of the ring, ready[], ready_free[] (widened tiles), q_full, q_free, s_full[2],
// p_full[2][2], pv_done[2], o_free[2], drain.
__host__ __device__ constexpr Smem smem_layout(int fmt)
{
    Smem s{};
    s.staged = ring_tiles(fmt) * tile_bytes(fmt);
    s.q = s.staged + (fmt == kFmtBf16 ? 0 : kStaged * kTile16);
    s.ml = s.q + 2 * kTile16;   // m[128], l[128], rounded l[128] of stream 1 (units of up to 128 rows)
    s.inv = s.ml + 3 * 128 * 4; // factors that undo the scaling of query rows
    s.bars = s.inv + (fmt == kFmtBf16 ? 0 : kRows * 4);
    s.misc = s.bars + (2 * ring_tiles(fmt) + 2 * ready_tiles(fmt) + 13) * 8;
    s.total = s.misc + 256;
    return s;
}
static_assert(smem_layout(kFmtBf16).total <= 232448 && smem_layout(kFmtFp8).total <= 232448 && smem_layout(kFmtF4).total <= 232448, "shared memory");

struct Misc {
    long long start_before;
    long long scan[17];
    int abort, start_r;
    uint32_t tmem;
    int later_bad[8]; // unit counter + 1 where V rows of later tokens are not finite
};
static_assert(sizeof(Misc) <= 256, "misc");

// sum over i < n of floor((a i + b) / m)
__device__ __forceinline__ long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b)
{
    unsigned long long s = 0;
    while (n > 0) {
        if (a >= m) {
            s += (unsigned long long)n * (n - 1) / 2 * (a / m);
            a %= m;
        }
        if (b >= m) {
            s += (unsigned long long)n * (b / m);
            b %= m;
        }
        const uint32_t y = a * n + b; // below 2^31: a < 128 here, n at most 2^22
        if (y < m)
            break;
        n = y / m;
        b = y % m;
        const uint32_t t = m;
        m = a;
        a = t;
    }
    return (long long)s;
}

// A request: its tokens, what its first token sees, its units.
struct Request {
    int first, n, L, units;
    __device__ __forceinline__ int tokens(const AttendParams &p, int u) const { return min(p.unit_tokens, n - u * p.unit_tokens); }
    // positions that the first token of unit u sees, and its pages
    __device__ __forceinline__ int seen(const AttendParams &p, int u) const { return L + (p.causal ? u * p.unit_tokens : 0); }
    __device__ __forceinline__ int pages(const AttendParams &p, int u) const
    {
        return (seen(p, u) + (p.causal ? tokens(p, u) - 1 : 0) + kPage - 1) / kPage;
    }
    // pages of units 0 .. u - 1 of one KV head
    __device__ __forceinline__ long long before(const AttendParams &p, int u) const
    {
        if (!p.causal)
            return (long long)u * pages(p, 0);
        const int k = u < units ? u : units - 1; // all units but the last have unit_tokens tokens
        return floor_sum(k, kPage, p.unit_tokens, L + p.unit_tokens + kPage - 2) + (u > k ? pages(p, k) : 0);
    }
};

// Reads request r: units = 0 where it has no tokens, no states (idle) or lengths that are refused (reported in *bad).
__device__ __forceinline__ Request read_request(const AttendParams &p, int r, bool *bad, bool *idle)
{
    Request q{};
    *bad = *idle = false;
    q.first = p.offsets[r];
    const long long n = (long long)p.offsets[r + 1] - q.first;
    if (n == 0)
        return q;
    q.L = p.seq_lens[r];
    if (n < 0 || q.first < 0 || q.first + n > p.T || q.L < 0 ||
        (q.L + (p.causal ? n - 1 : 0) + kPage - 1) / kPage > p.maxB) {
        *bad = true;
        return q;
    }
    q.n = (int)n;
    if (q.L == 0)
        *idle = true;
    else
        q.units = (q.n + p.unit_tokens - 1) / p.unit_tokens;
    return q;
}

__device__ __forceinline__ long long cut(int c, long long W, int n)
{
    const long long each = W / n, more = W - each * n;
    return c * each + min((long long)c, more);
}

__device__ __forceinline__ int cut_of(long long x, long long W, int n)
{
    const long long each = W / n, more = W - each * n, at = more * (each + 1);
    return (int)(x < at ? x / (each + 1) : more + (x - at) / each);
}

// The share of a CTA, unit by unit.  Every role walks it alike.
struct Share {
    long long x, x1;
    Request q;
    int r, head, u, b, nb, seg;
    __device__ __forceinline__ int pages() const { return (int)min((long long)(nb - b), x1 - x); }
    __device__ __forceinline__ int rows(const AttendParams &p) const { return q.tokens(p, u) * p.G; }
    __device__ __forceinline__ void next(const AttendParams &p)
    {
        x += pages();
        ++seg;
        b = 0;
        if (++u == q.units) {
            u = 0;
            if (++head == p.Hkv) {
                head = 0;
                bool bad, idle;
                do {
                    if (++r >= p.R)
                        return; // the end of the line: x = x1
                    q = read_request(p, r, &bad, &idle);
                } while (q.units == 0);
            }
        }
        nb = q.pages(p, u);
    }
};

// Place of a tile in the order in which the issuer uses the tiles of n pages.
__device__ __forceinline__ int order_of_k(bool two, int page)
{
    return two ? 2 * page : page < 2 ? page : 2 * page - 1;
}
__device__ __forceinline__ int order_of_v(bool two, int page, int n)
{
    return two ? 2 * page + 1 : min(2 * page + 2, 2 * n - 1);
}

// Rows of a staged bf16 V tile on a last page: rows from `past` on are not in the request and become
// zeros, and so do infinities and NaN of rows from `seen` on, which only later tokens of the
// unit see (a probability of 0 does not hide them; those tokens get them at the end of the
// unit, told by *bad).  One warp.
__device__ __forceinline__ void clear_rows(uint8_t *v, int seen, int past, volatile int *bad, int mark)
{
    const int lane = threadIdx.x & 31;
    bool any = false;
#pragma unroll 4
    for (int k = max(0, seen) * 16 + lane; k < kPage * 16; k += 32) { // 16-byte pieces
        const int row = k >> 4, piece = k & 15;
        uint4 *at = reinterpret_cast<uint4 *>(v + (piece >> 3) * 16384 + row * 128 + (piece & 7) * 16);
        uint4 d = *at;
        uint32_t *e = &d.x;
        uint32_t gone[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            gone[c] = __vcmpeq2(e[c] & 0x7F807F80u, 0x7F807F80u);
        if (row >= past || (gone[0] | gone[1] | gone[2] | gone[3])) {
            any = any || row < past;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                e[c] &= row >= past ? 0u : ~gone[c];
            *at = d;
        }
    }
    if (any)
        *bad = mark;
    __threadfence_block();
    fence_async_smem();
    __syncwarp();
}

template <int FMT>
__global__ void __launch_bounds__(threads_of(FMT), 1)
    attend_kernel(const __grid_constant__ CUtensorMap map, const AttendParams p)
{
    constexpr int TILES = ring_tiles(FMT), TB = tile_bytes(FMT), NT = threads_of(FMT);
    constexpr bool CONV = FMT != kFmtBf16;
    constexpr Smem L = smem_layout(FMT);
    extern __shared__ __align__(1024) uint8_t gsm[];
    const uint32_t smem = smem_u32(gsm);
    Misc &misc = *reinterpret_cast<Misc *>(gsm + L.misc);
    constexpr int DEPTH = ready_tiles(FMT);
    const uint32_t full = smem + L.bars, empty = full + TILES * 8, ready = empty + TILES * 8, ready_free = ready + DEPTH * 8;
    const uint32_t q_full = ready_free + DEPTH * 8, q_free = q_full + 8, s_full = q_free + 8, p_full = s_full + 16,
                   pv_done = p_full + 32, o_free = pv_done + 16, drain = o_free + 16;
    volatile int *abort_flag = &misc.abort;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long wl = p.wait_limit;

    launch_dependents();
    if (smem & 1023u) { // swizzled tiles need it; the declaration gives it
        if (threadIdx.x == 0) {
            set_error(p.err, kErrScratch);
            p.joins[blockIdx.x].c0 = -1;
        }
        return;
    }
    if (threadIdx.x == 0) {
        prefetch_tensormap(&map);
        for (int i = 0; i < TILES; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, CONV ? 4 : 1); // the converter warps, or the issuer
        }
        for (int i = 0; i < DEPTH; ++i) {
            mbar_init(ready + 8 * i, CONV ? 4 : 1); // the converter warps, or the clearing warp
            mbar_init(ready_free + 8 * i, 1);
        }
        mbar_init(q_full, 8);
        mbar_init(q_free, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full + 8 * t, 1);
            mbar_init(p_full + 16 * t, 4);
            mbar_init(p_full + 16 * t + 8, 4);
            mbar_init(pv_done + 8 * t, 1);
            mbar_init(o_free + 8 * t, 4);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        misc.abort = 0;
    }
    if (threadIdx.x < 8)
        misc.later_bad[threadIdx.x] = 0;
    if (warp == 1)
        tmem_alloc(smem_u32(&misc.tmem), 512);

    // ---- the line of pages and this CTA's range of it ----
    const int per = (p.R + NT - 1) / NT;
    const int lo = min(p.R, (int)threadIdx.x * per), hi = min(p.R, lo + per);
    long long mine = 0;
    for (int r = lo; r < hi; ++r) {
        bool bad, idle;
        const Request q = read_request(p, r, &bad, &idle);
        if (q.units)
            mine += q.before(p, q.units) * p.Hkv;
        if (bad && blockIdx.x == 0)
            set_error(p.err, kErrSeqLen);
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += v;
    }
    if (lane == 31)
        misc.scan[warp] = incl;
    __syncthreads();
    long long before = incl - mine, W = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        before += i < warp ? misc.scan[i] : 0;
        W += misc.scan[i];
    }
    const int ranges = (int)min((long long)gridDim.x, max(1ll, W / kMinPages));
    Share w{};
    w.x = (int)blockIdx.x < ranges ? cut(blockIdx.x, W, ranges) : W;
    w.x1 = (int)blockIdx.x < ranges ? cut(blockIdx.x + 1, W, ranges) : W;
    w.nb = 1;
    if (w.x < w.x1 && before <= w.x && w.x < before + mine) {
        long long at = before;
        for (int r = lo; r < hi; ++r) {
            bool bad, idle;
            const Request q = read_request(p, r, &bad, &idle);
            const long long some = q.units ? q.before(p, q.units) * p.Hkv : 0;
            if (at <= w.x && w.x < at + some) {
                misc.start_r = r;
                misc.start_before = at;
            }
            at += some;
        }
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = misc.tmem;
    if (w.x < w.x1) {
        bool bad, idle;
        w.r = misc.start_r;
        w.q = read_request(p, w.r, &bad, &idle);
        const long long in = w.x - misc.start_before, each = w.q.before(p, w.q.units);
        w.head = (int)(in / each);
        const long long rest = in - w.head * each;
        // the last unit with before(u) <= rest: the lanes try 32 at a time
        int n = w.q.units;
        while (n > 1) {
            const int step = (n + 31) >> 5, u = w.u + lane * step;
            const bool below = lane > 0 && u < w.u + n && w.q.before(p, u) <= rest;
            const int k = __popc(__ballot_sync(0xffffffffu, below));
            w.u += k * step;
            n = min(step, n - k * step);
        }
        w.b = (int)(rest - w.q.before(p, w.u));
        w.nb = w.q.pages(p, w.u);
    }
    if (threadIdx.x == 0) {
        AttendJoin j{};
        j.c0 = -1;
        if (w.x < w.x1 && w.b > 0) {
            const int c0 = cut_of(w.x - w.b, W, ranges);
            if (c0 == (int)blockIdx.x - 1) {
                j.token0 = w.q.first + w.u * p.unit_tokens;
                j.rows = w.rows(p);
                j.head = w.head;
                j.c0 = c0;
                j.c1 = cut_of(w.x - w.b + w.nb - 1, W, ranges);
            }
        }
        p.joins[blockIdx.x] = j;
    }
    // a wait that ran out: the CTA's roles run on without waiting, so that all
    // reach the end; what they compute is unspecified.  (Inlined: a kernel that moves registers
    // between its warpgroups can call nothing.)
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (mbar_test_wait(bar, parity))
            return;
        const bool poll = wl < (1 << 16); // a test's limit: the suspending form may sleep past it
        const long long start = clock64();
        while (!(poll ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))) {
            if (*abort_flag)
                return;
            if (clock64() - start > wl) {
                *abort_flag = 1;
                set_error(p.err, kErrTimeout);
                return;
            }
        }
    };

    if (warp < 4) {
        setmaxnreg_dec<kRegs0>();
        if (warp == 0) {
            // ---- producer: K and V tiles in the order of their use ----
            int z = 0, st = 0;
            uint32_t ph = 0;
            for (; w.x < w.x1; w.next(p)) {
                const int n = w.pages();
                const bool two = w.rows(p) > 128;
                const int32_t *row = p.block_table + (size_t)w.r * p.maxB + w.b;
                // two windows of 32 table entries: K runs at most two pages ahead of V
                int ent = 0, ent0 = -1, prev = 0;
                int kp = 0, vp = 0;
                for (int i = 0; i < 2 * n; ++i) {
                    const bool is_k = kp < n && order_of_k(two, kp) == i;
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
                        load_tile<FMT>(smem + st * TB, &map, p.kv, (page * 2 + (is_k ? 0 : 1)) * p.Hkv + w.head, full + 8 * st);
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
        } else if (warp == 1) {
            // ---- MMA issuer.  Step j is a page of one stream (t = j & 1): S(j), then P V(j) once its
            // softmax is done, then S(j + 2) behind it, while the other stream is in its softmax ----
            const uint32_t one = lane == 0, tm = uniform(tmem), base = uniform(smem);
            constexpr uint32_t kTypes = CONV ? ~((1u << 7) | (1u << 10)) : ~0u; // f16 or bf16 operands
            constexpr uint32_t idesc_s = umma_idesc_bf16(128, 128, 0, 0) & kTypes;
            constexpr uint32_t idesc_o = umma_idesc_bf16(128, 128, 0, 1) & kTypes;
            constexpr uint32_t RING = CONV ? L.staged : 0;
            const uint32_t tile_free = CONV ? ready_free : empty;
            uint32_t done0 = 0, done1 = 0; // P V of either stream so far
            int z0 = 0;
            for (; w.x < w.x1; w.next(p)) {
                const int n = w.pages();
                const bool two = w.rows(p) > 128;
                const int nsteps = two ? 2 * n : n;
                auto score = [&](int j) {
                    const int t = j & 1, z = z0 + order_of_k(two, two ? j >> 1 : j), st = z % DEPTH;
                    const uint32_t k = uniform(desc_low(base + RING + st * kTile16, 16)), q = uniform(desc_low(base + L.q + (two ? t * kTile16 : 0), 16));
                    const uint32_t d = tm + uniform(128 * t), done = t ? done1 : done0;
                    wait(ready + 8 * st, (uint32_t)(z / DEPTH) & 1u);
                    if (done > 0) // P, which S replaces, has been multiplied
                        wait(pv_done + 8 * t, (done - 1) & 1u);
                    tcgen05_after_sync();
#pragma unroll
                    for (uint32_t ks = 0; ks < 8; ++ks)
                        umma_ss(one, d, q + (ks >> 2) * 1024 + (ks & 3) * 2, k + (ks >> 2) * 1024 + (ks & 3) * 2, idesc_s, ks > 0);
                    if (one) {
                        umma_commit(s_full + 8 * t);
                        if (!two || t)
                            umma_commit(tile_free + 8 * st);
                        if (j == nsteps - 1)
                            umma_commit(q_free);
                    }
                    __syncwarp();
                };
                wait(q_full, w.seg & 1);
                score(0);
                if (nsteps > 1)
                    score(1);
                for (int j = 0; j < nsteps; ++j) {
                    const int t = j & 1, page = two ? j >> 1 : j, z = z0 + order_of_v(two, page, n), st = z % DEPTH;
                    const uint32_t v = uniform(desc_low(base + RING + st * kTile16, 16384));
                    const uint32_t a = tm + uniform(128 * t), d = tm + uniform(256 + 128 * t), more = uniform(j > 1); // a stream's first step of the unit sets O
                    wait(ready + 8 * st, (uint32_t)(z / DEPTH) & 1u);
                    if (j < 2 && w.seg > 0)
                        wait(o_free + 8 * t, (w.seg - 1) & 1);
                    const uint32_t done = t ? done1++ : done0++;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        wait(p_full + 16 * t + 8 * h, done & 1u);
                        tcgen05_after_sync();
                        // V, MN-major: 16 positions are 16 rows of 128 bytes
#pragma unroll
                        for (int ks = 4 * h; ks < 4 * h + 4; ++ks)
                            umma_ts(one, d, a + 8 * ks, v + ks * (2048 >> 4), idesc_o, ks > 0 ? 1u : more);
                    }
                    if (one) {
                        umma_commit(pv_done + 8 * t);
                        if (!two || t)
                            umma_commit(tile_free + 8 * st);
                    }
                    __syncwarp();
                    if (j + 2 < nsteps)
                        score(j + 2);
                    if (__any_sync(0xffffffffu, *abort_flag != 0)) // all lanes alike
                        break;
                }
                z0 += 2 * n;
                if (__any_sync(0xffffffffu, *abort_flag != 0))
                    break;
            }
            // nothing of this CTA's may be in flight when its tensor memory is freed
            if (one) {
                umma_commit(drain);
                mbar_wait_bounded(drain, 0);
            }
            __syncwarp();
        } else if (warp == 2 && !CONV) {
            // ---- clearing of V tiles (converters do it for theirs).  Every tile passes this warp on its way
            // to the issuer, so that no barrier gets two phases ahead of it ----
            int z = 0;
            for (; w.x < w.x1; w.next(p)) {
                const int n = w.pages(), seen = w.q.seen(p, w.u), past = seen + (p.causal ? w.q.tokens(p, w.u) - 1 : 0);
                const bool two = w.rows(p) > 128;
                int kp = 0, vp = 0;
                for (int i = 0; i < 2 * n; ++i, ++z) {
                    const bool is_k = kp < n && order_of_k(two, kp) == i;
                    const int pg = w.b + (is_k ? kp++ : vp++), st = z % TILES;
                    wait(full + 8 * st, (uint32_t)(z / TILES) & 1u);
                    if (!is_k && (pg + 1) * kPage > seen)
                        clear_rows(gsm + st * TB, seen - pg * kPage, past - pg * kPage, &misc.later_bad[w.seg & 7], w.seg + 1);
                    if (lane == 0)
                        mbar_arrive(ready + 8 * st);
                    __syncwarp();
                }
            }
        } else if (warp == 3) {
            // ---- outputs of requests without states ----
            for (int r = blockIdx.x; r < p.R; r += gridDim.x) {
                bool bad, idle;
                const Request q = read_request(p, r, &bad, &idle);
                if (!idle)
                    continue;
                const size_t rows = (size_t)p.Hkv * p.G, all = rows * q.n;
                uint4 *out = reinterpret_cast<uint4 *>(p.out + rows * q.first * kDim);
                for (size_t i = lane; i < all * (kDim / 8); i += 32)
                    out[i] = make_uint4(0u, 0u, 0u, 0u);
                for (size_t i = lane; i < all; i += 32)
                    p.lse[rows * q.first + i] = __uint_as_float(0xFF800000u);
            }
        }
    } else if (warp < 12) {
        // ---- softmax: thread = query row ----
        setmaxnreg_inc<regs_softmax(FMT)>();
        const int t = (warp - 4) >> 2, at_lane = threadIdx.x & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21); // this warp's lane quarter
        const uint32_t at_s = lanes + 128 * t, o_at = lanes + 256 + 128 * t;
        const float ninf = __uint_as_float(0xFF800000u);
        float *ml = reinterpret_cast<float *>(gsm + L.ml);
        float *qinv = reinterpret_cast<float *>(gsm + L.inv);
        const size_t Hq = (size_t)p.Hkv * p.G;
        uint32_t steps = 0, steps1 = 0; // of this stream and of stream 1 so far
        auto sync_all = [&] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
        // Query rows of unit u into the operand tiles, once the last S of the unit before is done: before
        // that unit's outputs are written, so that S goes on meanwhile.  Rows beyond the unit's
        // are left as they are: nothing is read from what they give.
        auto stage_queries = [&](const Share &u) {
            const int rows = u.rows(p);
            const bool two = rows > 128;
            const int row0 = two ? 128 * t : 0;
            const size_t first = (size_t)(u.q.first + u.u * p.unit_tokens) * Hq + (size_t)u.head * p.G;
            sync_all();
            if (u.seg > 0)
                wait(q_free, (u.seg - 1) & 1);
            stage_rows<CONV ? kRowsF16 : kRows16>(
                gsm + L.q + (two ? t * kTile16 : 0), 16384, min(128, rows - row0), two ? warp & 3 : warp - 4, two ? 4 : 8,
                [&](int i) {
                    const int j = (row0 + i) / p.G;
                    return p.q + (first + j * Hq + (row0 + i - j * p.G)) * kDim;
                },
                [&](int i, float x) { qinv[row0 + i] = x; });
            fence_async_smem();
            if (CONV)
                sync_all();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(q_full);
        };
        if (w.x < w.x1)
            stage_queries(w);
        Share nx = w;
        for (; w.x < w.x1; w = nx) {
            const int n = w.pages(), rows = w.rows(p);
            const bool two = rows > 128;
            const int nsteps = two ? n : (n + 1 - t) >> 1; // this stream's
            const int slot_row = (two ? 128 * t : 0) + at_lane, j = min(slot_row, rows - 1) / p.G;
            const bool real = slot_row < rows;
            const bool idle = (two ? 128 * t : 0) + (warp & 3) * 32 >= rows; // no row of this warp's is the unit's
            const size_t out_row = (size_t)(w.q.first + w.u * p.unit_tokens + j) * Hq + (size_t)w.head * p.G + (min(slot_row, rows - 1) - j * p.G);
            const float sc = p.scale_log2 * (CONV && real ? qinv[slot_row] : 1.f);
            const bool neg = sc < 0.f;
            const int seen0 = w.q.seen(p, w.u), lim = seen0 + (p.causal ? j : 0);
            steps1 += two ? n : n >> 1;
            float m = ninf, l = 0.f, lr = 0.f; // reference maximum, sum, sum of the rounded p
            for (int i = 0; i < nsteps; ++i, ++steps) {
                const int pos0 = (w.b + (two ? i : 2 * i + t)) * kPage;
                const bool tail = pos0 + kPage > seen0;
                const int seen = tail ? lim - pos0 : kPage; // columns this row sees
                wait(s_full + 8 * t, steps & 1u);
                if (idle) {
                    if (lane == 0) {
                        mbar_arrive(p_full + 16 * t);
                        mbar_arrive(p_full + 16 * t + 8);
                    }
                    continue;
                }
                tcgen05_after_sync();
                // the extreme logit of the row (the scale's sign says which end).  The columns stay in
                // registers; where converters need some, columns 0 .. 63 do and the others are read again
                constexpr int HELD = CONV ? 64 : 128;
                uint32_t v[HELD];
                float mx = neg ? -ninf : ninf;
#pragma unroll
                for (int c = 128 - HELD; c >= 0; c -= HELD) {
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
                if (tail && seen <= 0)
                    mx = ninf;
                if (CONV)
                    mx -= kPUp16;
                const bool rise = mx > m + kSlack || (m == ninf && mx > ninf);
                if (__any_sync(0xffffffffu, rise)) { // rare, and so everything that it needs is in here
                    const float f = rise ? ex2(m - mx) : 1.f;
                    m = rise ? mx : m;
                    l *= f;
                    lr *= f;
                    if (i > 0) {
                        wait(pv_done + 8 * t, (steps - 1) & 1u); // O holds every step before this one
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
                const uint64_t sc2 = pair(sc, sc), ref2 = pair(-ref, -ref);
                uint64_t sum[2] = {0ull, 0ull}, sumr[2] = {0ull, 0ull};
                // the common step by itself, without the tests for a last page
                auto to_p = [&](auto plain) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) { // 32 columns of S become P
                        if (HELD == 64 && c == 2) {
                            tmem_ld32(at_s + 64, v);
                            tmem_ld32(at_s + 96, v + 32);
                            tmem_wait_ld(v);
                            tmem_wait_ld(v + 32);
                        }
                        uint32_t hi[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const int at = 32 * c + 2 * k, x = at % HELD;
                            float e0, e1;
                            unpair(fma2(pair(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), sc2, ref2), e0, e1);
                            e0 = ex2(e0);
                            e1 = ex2(e1);
                            if (!plain.value) {
                                e0 = at < seen ? e0 : 0.f;
                                e1 = at + 1 < seen ? e1 : 0.f;
                            }
                            sum[k & 1] = add2(sum[k & 1], pair(e0, e1));
                            if (CONV) {
                                hi[k] = pack_f16(e0, e1);
                            } else {
                                hi[k] = pack_bf16(e0, e1);
                                sumr[k & 1] = add2(sumr[k & 1], pair(__uint_as_float(hi[k] << 16), __uint_as_float(hi[k] & 0xFFFF0000u)));
                            }
                        }
                        tmem_st16(at_s + 16 * c, hi);
                        if (c & 1) { // half of P: the issuer can begin
                            tmem_wait_st();
                            tcgen05_before_sync();
                            __syncwarp();
                            if (lane == 0)
                                mbar_arrive(p_full + 16 * t + 8 * (c >> 1));
                        }
                    }
                };
                if (tail)
                    to_p(std::false_type{});
                else
                    to_p(std::true_type{});
                float a, b;
                unpair(add2(sum[0], sum[1]), a, b);
                l += a + b;
                if (!CONV) {
                    unpair(add2(sumr[0], sumr[1]), a, b);
                    lr += a + b;
                }
            }
            if (CONV)
                lr = l;

            // ---- end of the unit's share ----
            const bool more = w.x + n < w.x1;
            nx.next(p);
            if (more)
                stage_queries(nx);
            const bool whole = w.b == 0 && n == w.nb, ends = w.b + n == w.nb;
            float *slot = p.partial + (size_t)(2 * blockIdx.x + (ends ? 0 : 1)) * kSlotFloats;
            float M = m, fa = 1.f, fb = 0.f;
            if (!two) {
                if (t == 1) {
                    ml[at_lane] = m;
                    ml[128 + at_lane] = l;
                    ml[256 + at_lane] = lr;
                }
                sync_all();
                const float mb = ml[at_lane], lb = ml[128 + at_lane], lrb = ml[256 + at_lane];
                sync_all();
                if (t == 1)
                    continue; // stream 0 reads both accumulators
                M = fmaxf(m, mb);
                fa = m == ninf ? 0.f : ex2(m - M);
                fb = mb == ninf ? 0.f : ex2(mb - M);
                l = l * fa + lb * fb;
                lr = lr * fa + lrb * fb;
            }
            if (n > 1 || two || t == 0)
                wait(pv_done + 8 * t, (steps - 1) & 1u);
            if (!two && n > 1) // stream 1 has given all its P: the last of its products is the one under way
                wait(pv_done + 8, (steps1 - 1) & 1u);
            tcgen05_after_sync();
            const float fin = lr > 0.f || lr != lr ? p.v_scale / lr : 0.f;
            const bool bad = misc.later_bad[w.seg & 7] == w.seg + 1;
#pragma unroll 1
            for (int c = 0; c < 8 && !idle; ++c) {
                float a[16];
                tmem_ld16(o_at + 16 * c, a);
                if (!two) {
                    float o[16];
                    tmem_ld16(o_at + 128 + 16 * c, o);
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        a[k] = a[k] * fa + (n > 1 ? o[k] * fb : 0.f); // (with one page stream 1 has no O)
                }
                if (bad) { // infinities and NaN of later tokens' V, for the rows that see them
                    const float ref = M == ninf ? 0.f : M;
                    for (int pos = max(seen0, w.b * kPage); pos < min(lim, (w.b + n) * kPage); ++pos) {
                        const long long page = p.block_table[(size_t)w.r * p.maxB + pos / kPage];
                        if (page < 0 || page >= p.num_pages)
                            continue;
                        float pr = 0.f;
                        bool have = false;
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float x = stored_value<FMT>(p.kv, (page * 2 + 1) * p.Hkv + w.head, pos % kPage, 16 * c + k);
                            if (finite(x))
                                continue;
                            if (!have) {
                                const uint16_t *qv = p.q + out_row * kDim;
                                for (int d = 0; d < kDim; ++d)
                                    pr = fmaf(__uint_as_float((uint32_t)qv[d] << 16),
                                              stored_value<FMT>(p.kv, page * 2 * p.Hkv + w.head, pos % kPage, d), pr);
                                pr = ex2(fmaf(pr, p.scale_log2, -ref));
                                have = true;
                            }
                            a[k] = fmaf(pr, x, a[k]);
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
                if (!two)
                    mbar_arrive(o_free + 8);
            }
            if (real) {
                if (whole) {
                    p.lse[out_row] = l == 0.f ? ninf : (M + log2f(l)) * 0.6931471805599453f;
                } else {
                    slot[(size_t)kRows * kDim + slot_row] = M;
                    slot[(size_t)kRows * (kDim + 1) + slot_row] = l;
                    slot[(size_t)kRows * (kDim + 2) + slot_row] = lr;
                }
            }
        }
    } else if constexpr (CONV) {
        // ---- converters: a ring tile to a 16-bit tile, in the order of use ----
        setmaxnreg_dec<kRegsConv>();
        const int row = threadIdx.x & 127;
        int z = 0;
        for (; w.x < w.x1; w.next(p)) {
            const int n = w.pages(), seen = w.q.seen(p, w.u), past = seen + (p.causal ? w.q.tokens(p, w.u) - 1 : 0);
            const bool two = w.rows(p) > 128;
            int kp = 0, vp = 0;
            for (int i = 0; i < 2 * n; ++i, ++z) {
                const bool is_k = kp < n && order_of_k(two, kp) == i;
                const int page0 = (w.b + (is_k ? kp++ : vp++)) * kPage;
                const bool tail = !is_k && page0 + kPage > seen;
                const bool drop = tail && page0 + row >= past;           // not in the request
                const bool check = tail && !drop && page0 + row >= seen; // seen by later tokens only
                wait(full + 8 * (z % TILES), (uint32_t)(z / TILES) & 1u);
                if (z >= DEPTH)
                    wait(ready_free + 8 * (z % DEPTH), (uint32_t)(z / DEPTH - 1) & 1u);
                const bool bad = convert_row<FMT>(gsm + (z % TILES) * TB, gsm + L.staged + (z % DEPTH) * kTile16 + row * 128, row, tail, drop, check);
                if (bad)
                    misc.later_bad[w.seg & 7] = w.seg + 1;
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(empty + 8 * (z % TILES));
                    mbar_arrive(ready + 8 * (z % DEPTH));
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

// Units cut between CTAs: block (c, y) has rows y, y + 32, ... of the unit that CTA c + 1 begins inside
// of, a warp a row, or all warps where a unit has many cuts.
__global__ void __launch_bounds__(256) attend_join_kernel(const AttendParams p)
{
    __shared__ float sm_m[8], sm_l[8], sm_r[8];
    __shared__ float4 sm_o[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    const AttendJoin jn = p.joins[blockIdx.x + 1];
    if (jn.c0 < 0)
        return;
    const bool shared = jn.c1 - jn.c0 >= 8;
    const float ninf = __uint_as_float(0xFF800000u);
    for (int k = 0; k < (shared ? 8 : 1); ++k) {
        const int row = blockIdx.y + 32 * (shared ? k : warp), step = shared ? 8 : 1;
        if (row >= jn.rows)
            return; // with shared rows, all threads
        float M = ninf, l = 0.f, lr = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float m, float a, float r, float4 v) {
            const float n = fmaxf(M, m), ref = n == ninf ? 0.f : n, f = ex2(M - ref), e = ex2(m - ref);
            l = l * f + a * e;
            lr = lr * f + r * e;
            o = make_float4(o.x * f + v.x * e, o.y * f + v.y * e, o.z * f + v.z * e, o.w * f + v.w * e);
            M = n;
        };
        for (int c = jn.c0 + (shared ? warp : 0); c <= jn.c1; c += 4 * step) {
            float m[4], a[4], r[4];
            float4 v[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) { // four slots on their way at once
                const int cc = c + step * s;
                m[s] = ninf;
                a[s] = r[s] = 0.f;
                v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (cc <= jn.c1) {
                    const float *slot = p.partial + (size_t)(2 * cc + (cc < jn.c1 ? 1 : 0)) * kSlotFloats;
                    m[s] = slot[(size_t)kRows * kDim + row];
                    a[s] = slot[(size_t)kRows * (kDim + 1) + row];
                    r[s] = slot[(size_t)kRows * (kDim + 2) + row];
                    v[s] = reinterpret_cast<const float4 *>(slot + (size_t)row * kDim)[lane];
                }
            }
#pragma unroll
            for (int s = 0; s < 4; ++s)
                add(m[s], a[s], r[s], v[s]);
        }
        if (shared) {
            if (lane == 0) {
                sm_m[warp] = M;
                sm_l[warp] = l;
                sm_r[warp] = lr;
            }
            sm_o[warp][lane] = o;
            __syncthreads();
            if (warp == 0)
                for (int s = 1; s < 8; ++s)
                    add(sm_m[s], sm_l[s], sm_r[s], sm_o[s][lane]);
            __syncthreads();
        }
        if (shared && warp > 0)
            continue;
        const float f = lr > 0.f || lr != lr ? p.v_scale / lr : 0.f;
        const int j = row / p.G;
        const size_t out = ((size_t)(jn.token0 + j) * p.Hkv + jn.head) * p.G + (row - j * p.G);
        reinterpret_cast<uint2 *>(p.out + out * kDim)[lane] = make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
        if (lane == 0)
            p.lse[out] = l == 0.f ? ninf : (M + log2f(l)) * 0.6931471805599453f;
    }
}

template <int FMT>
cudaError_t launch_t(const AttendParams &p, const CUtensorMap &map, int ctas, cudaStream_t stream)
{
    constexpr int smem = smem_layout(FMT).total;
    cudaError_t e = cudaFuncSetAttribute(attend_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    cudaFuncAttributes fa;
    if (e == cudaSuccess)
        e = cudaFuncGetAttributes(&fa, attend_kernel<FMT>);
    if (e != cudaSuccess)
        return e;
    // a raise waits until the lowerings have freed enough of the launch's registers: never launch
    // an instance built with fewer than the split needs
    if (fa.numRegs * threads_of(FMT) < 128 * (kRegs0 + 2 * regs_softmax(FMT) + (FMT == kFmtBf16 ? 0 : kRegsConv)))
        return cudaErrorInvalidConfiguration;
    e = launch_kernel(attend_kernel<FMT>, dim3(ctas), dim3(threads_of(FMT)), smem, stream, false, map, p);
    if (e == cudaSuccess && ctas > 1)
        e = launch_kernel(attend_join_kernel, dim3(ctas - 1, 32), dim3(256), 0, stream, true, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace

size_t attend_slot_bytes()
{
    return kSlotFloats * sizeof(float);
}

cudaError_t launch_attend(const AttendParams &params, int kv_dtype, int ctas, cudaStream_t stream)
{
    AttendParams p = params;
    p.unit_tokens = kRows / p.G;
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
