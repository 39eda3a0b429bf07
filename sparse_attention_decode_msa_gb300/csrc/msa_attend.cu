// msa_attend.cu -- attention of ragged query rows over paged states: cross attention
// (every token of a request sees all of its states) and the attention of a prompt's
// chunk (causal).
//
// For a query row q of a token that sees n positions: s_p = scale q . K[p], m the running
// maximum, out = sum 2^(s - m) V / sum 2^(s - m), lse = m + ln sum, in one pass over the
// pages, fp32.
//
// Work.  The rows of a (request, KV head) are cut into units of T = 2 floor(128 / G)
// tokens with their G heads, at most 256 rows; a unit's pages are those that its last token
// sees.  All units laid end to end (request, KV head, unit), each with a few pages' time for its
// queries and outputs in front (kUnitCost), are a line that is cut into equal ranges, one a CTA,
// whatever the lengths are; a unit cut between CTAs is
// joined by attend_join_kernel in the order of its pages.  Pages before unit i of a causal
// request are a sum of floors, lattice points under a line, which are counted in a few steps: no
// table, no kernel before this one.
//
// Two streams of up to 128 rows share a CTA's pages, so that the tensor cores work for one
// while the other is in its softmax: tokens t floor(128 / G) .. of the unit are stream t's, and
// both take every page; a unit whose tokens fit in one stream goes to both, which take its pages
// in turn, and their (m, l, O) are added at the end.
//
// Operands: Q in shared memory (K-major, 128-byte swizzle), K tiles as TMA lands them, P in
// tensor memory over the S it came from, V tiles as landed (MN-major).  E4M3 and NVFP4 tiles
// are widened to f16 by converter warps, and P is f16, 2^7 for the heaviest position of a row's first page: off by
// 2^-11 of p, or by 2^-32 of that position's below 2^-21 of it (a subnormal's half step).  Over bf16 pages P
// is bf16 (V's type, which a product needs): each p is off by 2^-8 of itself at most, and
// the sum that divides is that of the rounded p, so that an output is a mean of values
// with weights that are off by 2^-8 of themselves and still sum to 1: off by 2^-8 of the
// weighted mean distance of the values from it at most, exact where all values or all
// logits are alike.  lse has the sum of the p as they are.  (P as a pair of bf16, as the dense decode
// has it, doubles the products of P V.  Only for units that fit one stream, in place of their S, it took
// 96 us for 82 of single tokens over 1500 states and 14.3 for 12.3 of 7 tokens: a page's tiles are held longer.)
//
// What bounds it, and what it measured (one GB300).  A page and both streams are 2060 clocks of
// products; the chain S -> exponentials -> P -> P V, with tensor memory full, and the ends of units
// keep the tensor cores waiting for the rest: ragged prompts over bf16 pages (4 of 1500 to 4096 tokens, 0.54 PFLOP)
// 422 us, 1.29 PFLOP/s.  Over E4M3 pages shared memory carries 320 KB a page, 2500 clocks: 512 tokens
// over 65536 positions (1.10 PFLOP) 665 us, 1.66 PFLOP/s, what power sustains; NVFP4, chunks of 33 to 100 tokens, 120 us, 1.19 PFLOP/s.
// 64 single tokens over 1500 bf16 states (394 MB) 82 us, 4.8 TB/s: start, joins, and what the ring does not
// cover when a unit ends.  Spilled registers do not stay in the L1 that the shared memory leaves, the code of all
// roles has to share the instruction caches, and the way out of a wait is in every link of the chain: most
// of the choices below that look small are about one of the three.
//
// TMEM columns: S/P of stream t at 128 t, O of stream t at 256 + 128 t.
// Warps: 0 TMA producer, 1 and 2 issue the MMAs of stream 0 and 1 (1 owns the TMEM), 3 clears what
// must not be multiplied from V tiles on last pages (bf16), 4-11 and 12-19 softmax of stream 0 and 1, two
// warps a row quarter: columns 0 .. 63 and 64 .. of a page, 20-23 converters (E4M3, NVFP4).
#include <type_traits>

#include "msa_ragged.cuh"
#include "msa_umma.cuh"

namespace msa {
namespace {

constexpr int kRows = 256;       // query rows of a unit
constexpr int kTile16 = 32768;   // a 16-bit K, V or Q tile
constexpr int kStaged = 4;       // widened tiles in flight
constexpr float kMost = 0x1p16f;   // what the p of a page may add up to before the row's reference rises
constexpr float kMost16 = 0x1p15f; // the same where P is f16
constexpr float kPUp16 = 7.f;      // f16 P: 2^7 2^(s - m)
constexpr int kSlotFloats = kRows * (kDim + 2); // o[rows][128], m, l
constexpr int kUnitCost = 3;     // a unit's queries and outputs in pages (ragged prompts 422 us; 2: 432, 4: 431)
constexpr int kMinRange = 4;     // what a CTA takes at least

__host__ __device__ constexpr int threads_of(int fmt)
{
    return fmt == kFmtBf16 ? 640 : 768;
}

__host__ __device__ constexpr int ring_tiles(int fmt)
{
    return fmt == kFmtBf16 ? 5 : 2;
}

struct Smem {
    int staged, q, xch, inv, bars, misc, total;
};

// Tiles that the issuer takes: widened ones, or the ring's own once they have passed the clearing warp.
__host__ __device__ constexpr int ready_tiles(int fmt)
{
    return fmt == kFmtBf16 ? ring_tiles(fmt) : kStaged;
}

// Barriers: full[], empty[] of the ring, ready[], ready_free[] (widened tiles), and for each stream
// q_raw (their copy), q_full, s_full, p_full, pv_done, o_free, turn, drain.
__host__ __device__ constexpr Smem smem_layout(int fmt)
{
    Smem s{};
    s.staged = ring_tiles(fmt) * tile_bytes(fmt);
    s.q = s.staged + (fmt == kFmtBf16 ? 0 : kStaged * kTile16);
    s.xch = s.q + 2 * kTile16;      // a float for each softmax thread: what the warps of a row tell one another
    s.inv = s.xch + 4 * 128 * 4; // exponents that undo the scaling of query rows, of two units
    s.bars = s.inv + (fmt == kFmtBf16 ? 0 : 2 * kRows);
    s.misc = s.bars + (2 * ring_tiles(fmt) + 2 * ready_tiles(fmt) + 16) * 8;
    s.total = s.misc + 288;
    return s;
}
static_assert(smem_layout(kFmtBf16).total <= 232448 && smem_layout(kFmtFp8).total <= 232448 && smem_layout(kFmtF4).total <= 232448, "shared memory");

// sum over i < n of floor((a i + b) / m), the lattice points under a line by columns.  What a and b have of whole m
// is a sum at once.  Of the rest, y = floor((a (n - 1) + b) / m) rows of points, row j + 1 lacks the columns before
// ceil(((j + 1) m - b) / a): n y less the same sum over y rows with a and m changed over, as in Euclid's algorithm.
__device__ __noinline__ long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b)
{
    long long s = 0;
    for (bool plus = true; n > 0; plus = !plus) {
        long long t = (long long)((unsigned long long)n * (n - 1) / 2 * (a / m) + (unsigned long long)n * (b / m));
        a %= m;
        b %= m;
        const uint32_t y = (a * (n - 1) + b) / m; // below 2^30: a < 128, n at most 2^22, and both fall
        t += (long long)n * y;
        s = plus ? s + t : s - t;
        b = m - b + a - 1;
        n = y;
        const uint32_t old = m;
        m = a;
        a = old;
    }
    return s;
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
    // the line's length up to unit u of one KV head
    __device__ __forceinline__ long long before(const AttendParams &p, int u) const
    {
        if (!p.causal)
            return (long long)u * (kUnitCost + pages(p, 0));
        const int k = u < units ? u : units - 1; // all units but the last have unit_tokens tokens
        return floor_sum(k, kPage, p.unit_tokens, L + p.unit_tokens + kPage - 2) + (long long)u * kUnitCost + (u > k ? pages(p, k) : 0);
    }
};

struct Misc {
    long long start_before;
    long long scan[24];
    Request start;
    long long wait_limit;
    uint32_t *err;
    int abort, start_r;
    uint32_t tmem;
    int later_bad[8]; // unit counter + 1 where V rows of later tokens are not finite
    int idle;         // there are requests without states
};
static_assert(sizeof(Misc) <= 288, "misc");

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
        (q.L > 0 && (q.L + (p.causal ? n - 1 : 0) + kPage - 1) / kPage > p.maxB)) {
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

// x / y, in 32 bits where both fit (a 64-bit division takes as long as the rest of a CTA's start)
__device__ __forceinline__ long long quotient(long long x, long long y)
{
    if (((unsigned long long)(x | y) >> 32) == 0)
        return (unsigned)x / (unsigned)y;
    return x / y;
}

// The line of length W cut into n ranges (the first W % n one longer): where range c begins, and the range that
// holds place x.
__device__ __forceinline__ long long cut(int c, long long W, int n)
{
    const long long each = quotient(W, n), more = W - each * n;
    return c * each + min((long long)c, more);
}

__device__ __forceinline__ int cut_of(long long x, long long W, int n)
{
    const long long each = quotient(W, n), more = W - each * n, at = more * (each + 1);
    return (int)(x < at ? quotient(x, each + 1) : more + quotient(x - at, each));
}

// The share of a CTA, unit by unit.  Every role walks it alike.
struct Share {
    Request q;
    int left; // of the line, from this unit's beginning to the range's end; 0: no pages any more
    int r, head, u, b, nb, seg;
    __device__ __forceinline__ int pages() const { return min(nb, left - kUnitCost) - b; }
    __device__ __forceinline__ int token0(const AttendParams &p) const { return q.first + u * p.unit_tokens; }
    __device__ __forceinline__ bool two(const AttendParams &p) const { return 2 * q.tokens(p, u) > p.unit_tokens; }
    __device__ __forceinline__ bool last() const { return left - (kUnitCost + nb) <= kUnitCost; }
    __device__ __forceinline__ void next(const AttendParams &p)
    {
        left = last() ? 0 : left - (kUnitCost + nb);
        ++seg;
        b = 0;
        if (left == 0)
            return;
        if (++u == q.units) {
            u = 0;
            if (++head == p.Hkv) {
                head = 0;
                bool bad, idle;
                do {
                    if (++r >= p.R) { // (the line is as long as the ranges say)
                        left = 0;
                        return;
                    }
                    q = read_request(p, r, &bad, &idle);
                } while (q.units == 0);
            }
        }
        nb = q.pages(p, u);
    }
};

// A share in one register of a warp, a word a lane: the softmax warps keep it so over their pages, where every
// register counts.
__device__ __forceinline__ int fold(const Share &w)
{
    const int words[11] = {w.q.first, w.q.n, w.q.L, w.q.units, w.left, w.r, w.head, w.u, w.b, w.nb, w.seg};
    int v = 0;
#pragma unroll
    for (int k = 0; k < 11; ++k)
        v = (int)(threadIdx.x & 31) == k ? words[k] : v;
    return v;
}

__device__ __forceinline__ Share unfold(int v)
{
    auto word = [&](int k) { return __shfl_sync(0xffffffffu, v, k); };
    Share w;
    w.q.first = word(0);
    w.q.n = word(1);
    w.q.L = word(2);
    w.q.units = word(3);
    w.left = word(4);
    w.r = word(5);
    w.head = word(6);
    w.u = word(7);
    w.b = word(8);
    w.nb = word(9);
    w.seg = word(10);
    return w;
}

// The order in which the issuers use the tiles of n pages: K and V of each page, or, where the streams take
// pages in turn, both K and both V of each pair of pages.
__device__ __forceinline__ bool tile_of(bool two, int n, int i, int *page)
{
    if (two) {
        *page = i >> 1;
        return !(i & 1);
    }
    const int first = i >> 2 << 1, pair = min(2, n - first), in = i & 3;
    *page = first + (in & (pair - 1));
    return in < pair;
}

// Rows of a staged bf16 V tile on a last page: rows from `past` on are not in the request and become
// zeros, and so do infinities and NaN of rows from `seen` on, which only later tokens of the
// unit see (a probability of 0 does not hide them; those tokens get them at the end of the
// unit, told by *bad).  One warp.
__device__ __forceinline__ void clear_rows(uint8_t *v, int seen, int past, volatile int *bad, int mark)
{
    const int lane = threadIdx.x & 31;
    auto at = [&](int k) { return reinterpret_cast<uint4 *>(v + (k >> 3 & 1) * 16384 + (k >> 4) * 128 + (k & 7) * 16); }; // 16-byte piece k
    const int stop = 16 * min(past, kPage);
#pragma unroll 4
    for (int k = max(stop, 0) + lane; k < 16 * kPage; k += 32)
        *at(k) = make_uint4(0u, 0u, 0u, 0u);
    bool any = false;
    for (int k0 = max(0, seen) * 16; k0 < stop; k0 += 128) {
        uint4 d[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (k0 + 32 * u + lane < stop)
                d[u] = *at(k0 + 32 * u + lane);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (k0 + 32 * u + lane >= stop)
                continue;
            uint32_t *e = &d[u].x, gone = 0u;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t g = __vcmpeq2(e[c] & 0x7F807F80u, 0x7F807F80u);
                e[c] &= ~g;
                gone |= g;
            }
            if (gone) {
                any = true;
                *at(k0 + 32 * u + lane) = d[u];
            }
        }
    }
    if (any)
        *bad = mark;
    __threadfence_block();
    fence_async_smem();
    __syncwarp();
}

// The largest sc s over the first `seen` of 64 columns of this thread's row of S, -inf for none.
__device__ __noinline__ float row_maximum(uint32_t at_s, float sc, int seen)
{
    const float inf = __uint_as_float(0x7F800000u);
    float top[2] = {-inf, -inf}, low[2] = {inf, inf};
#pragma unroll 1
    for (int c = 0; c < 64; c += 32) {
        uint32_t v[32];
        tmem_ld32(at_s + c, v);
        tmem_wait_ld(v);
        if (__any_sync(0xffffffffu, seen < c + 32)) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
                if (c + k < seen) {
                    top[0] = fmaxf(top[0], __uint_as_float(v[k]));
                    low[0] = fminf(low[0], __uint_as_float(v[k]));
                }
        } else {
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
                top[k >> 1 & 1] = fmaxf(top[k >> 1 & 1], fmaxf(__uint_as_float(v[k]), __uint_as_float(v[k + 1])));
                low[k >> 1 & 1] = fminf(low[k >> 1 & 1], fminf(__uint_as_float(v[k]), __uint_as_float(v[k + 1])));
            }
        }
    }
    // which end of the row is the largest goes by the scale's sign
    return seen <= 0 ? -inf : sc < 0.f ? fminf(low[0], low[1]) * sc : fmaxf(top[0], top[1]) * sc;
}

// 64 columns of this thread's row of S to p = 2^(sc s - ref), as pairs of bf16 (f16) in pr; their
// sum, and that of the bf16 they become.  TAIL: columns from `seen` on are 0.
template <bool F16, bool TAIL>
__device__ __forceinline__ float row_to_p(uint32_t at_s, float sc, float ref, int seen, uint32_t (&pr)[32], float &rounded)
{
    const uint64_t sc2 = pair(sc, sc), ref2 = pair(-ref, -ref);
    uint64_t sum[2] = {0ull, 0ull}, sumr[2] = {0ull, 0ull};
    // 16 columns at a time, none on their way meanwhile: the other warps of a scheduler fill the gap.  Beside
    // converters a thread has 80 registers, and what it spills does not stay in the L1 that 227 KB of shared
    // memory leave (8 columns ahead and 24 bytes on the stack: a 512-token chunk over 65536 E4M3 positions
    // 745 us, nothing spilled 725; over bf16 pages 16 ahead: ragged prompts 422, none ahead 419).
    constexpr int N = 16;
#pragma unroll
    for (int c = 0; c < 64 / N; ++c) {
        uint32_t x[N];
        tmem_ld_async(at_s + N * c, x);
        tmem_wait_async(x);
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            float e0, e1;
            unpair(fma2(pair(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), sc2, ref2), e0, e1);
            e0 = ex2(e0);
            e1 = ex2(e1);
            if (TAIL) {
                e0 = N * c + k < seen ? e0 : 0.f;
                e1 = N * c + k + 1 < seen ? e1 : 0.f;
            }
            sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pair(e0, e1));
            const uint32_t both = pr[N / 2 * c + (k >> 1)] = F16 ? pack_f16(e0, e1) : pack_bf16(e0, e1);
            if (!F16)
                sumr[(k >> 1) & 1] = add2(sumr[(k >> 1) & 1], pair(__uint_as_float(both << 16), __uint_as_float(both & 0xFFFF0000u)));
        }
    }
    float a, b;
    unpair(add2(sumr[0], sumr[1]), a, b);
    rounded = a + b;
    unpair(add2(sum[0], sum[1]), a, b);
    return a + b;
}

__device__ __forceinline__ float lds32(uint32_t a)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ void sts32(uint32_t a, float v)
{
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// Whether any thread of the two warps that meet at a barrier says so.  What either warp stores to tensor memory
// behind it comes after what both have read before it.
__device__ __forceinline__ bool any_of_two_warps(int barrier, bool v)
{
    uint32_t any;
    tcgen05_before_sync();
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 64, p;\n selp.b32 %0, 1, 0, q;\n}\n"
                 : "=r"(any)
                 : "r"((uint32_t)v), "r"(barrier)
                 : "memory");
    tcgen05_after_sync();
    return any != 0;
}

// Infinities and NaN of V at positions from .. to - 1, which were kept out of the products, for a row that
// sees them: into dimensions d0 .. d0 + 63 of its output, or of its partial one in a slot.
template <int FMT>
__device__ __noinline__ void add_late_values(const AttendParams &p, int r, int head, long long row, int from, int to, float ref, float *slot, int d0)
{
    for (int pos = from; pos < to; ++pos) {
        const long long page = p.block_table[(size_t)r * p.maxB + pos / kPage];
        if (page < 0 || page >= p.num_pages)
            continue;
        float pr = 0.f;
        bool have = false;
        for (int d = d0; d < d0 + 64; ++d) {
            const float x = stored_value<FMT>(p.kv, (page * 2 + 1) * p.Hkv + head, pos % kPage, d);
            if (finite(x))
                continue;
            if (!have) {
                const uint16_t *q = p.q + row * kDim;
                for (int e = 0; e < kDim; ++e)
                    pr = fmaf(__uint_as_float((uint32_t)q[e] << 16), stored_value<FMT>(p.kv, page * 2 * p.Hkv + head, pos % kPage, e), pr);
                pr = ex2(fmaf(pr, p.scale_log2, -ref));
                have = true;
            }
            if (slot) {
                slot[(d >> 2) * (4 * kRows) + (d & 3)] += pr * x;
            } else {
                uint16_t *o = p.out + row * kDim + d;
                *o = (uint16_t)pack_bf16(__uint_as_float((uint32_t)*o << 16) + pr * x, 0.f);
            }
        }
    }
}

// Two pieces of N words of each of two neighbouring lanes: d[k] becomes piece lane % 2 of lane k of the two.
template <int N>
__device__ __forceinline__ void transpose2(uint32_t (&d)[2][N])
{
    const bool high = threadIdx.x & 1;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? d[0][k] : d[1][k], 1);
        d[0][k] = high ? got : d[0][k];
        d[1][k] = high ? d[1][k] : got;
    }
}

__device__ __forceinline__ void store(void *a, const uint32_t (&d)[4])
{
    *reinterpret_cast<uint4 *>(a) = make_uint4(d[0], d[1], d[2], d[3]);
}

// 32 bytes in one store, or two of 16 where the tensor begins at an odd multiple of 16.
__device__ __forceinline__ void store(void *a, const uint32_t (&d)[8])
{
    if (reinterpret_cast<uintptr_t>(a) & 16) {
        reinterpret_cast<uint4 *>(a)[0] = make_uint4(d[0], d[1], d[2], d[3]);
        reinterpret_cast<uint4 *>(a)[1] = make_uint4(d[4], d[5], d[6], d[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a), "r"(d[0]), "r"(d[1]), "r"(d[2]), "r"(d[3]), "r"(d[4]), "r"(d[5]),
                 "r"(d[6]), "r"(d[7])
                 : "memory");
}

// The query rows of an operand tile from bf16 to f16, in place, by four warps: each row after a power of two
// that brings its largest element to [2^8, 2^9) (exact; elements 2^-23 below it lose bits), whose
// exponent is told with the sign turned.
__device__ __forceinline__ void widen_queries(uint8_t *tile, int8_t *exps)
{
    const int lane = threadIdx.x & 31, c = lane & 15, first = 2 * ((threadIdx.x >> 5) & 3) + (lane >> 4);
#pragma unroll 1
    for (int i0 = 0; i0 < 128; i0 += 32) {
        uint4 d[4];
        float mx[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + 8 * u + first;
            d[u] = *reinterpret_cast<const uint4 *>(tile + (c >> 3) * 16384 + 128 * i + (((c & 7) ^ (i & 7)) << 4));
            const uint32_t *e = &d[u].x;
            mx[u] = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mx[u] = fmaxf(mx[u], fmaxf(fabsf(__uint_as_float(e[k] << 16)), fabsf(__uint_as_float(e[k] & 0xFFFF0000u))));
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1)
#pragma unroll
            for (int u = 0; u < 4; ++u)
                mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], o));
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + 8 * u + first;
            int x = (int)(__float_as_uint(mx[u]) >> 23) - 127; // clamped so that neither factor overflows
            x = x < -100 ? -100 : x > 127 ? 127 : x;
            const float up = __uint_as_float((uint32_t)(8 - x + 127) << 23);
            uint32_t *e = &d[u].x;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                e[k] = pack_f16(__uint_as_float(e[k] << 16) * up, __uint_as_float(e[k] & 0xFFFF0000u) * up);
            *reinterpret_cast<uint4 *>(tile + (c >> 3) * 16384 + 128 * i + (((c & 7) ^ (i & 7)) << 4)) = d[u];
            if (c == 0)
                exps[i] = (int8_t)(x - 8);
        }
    }
}

// A wait that was not over at once (out of line: two dozen places wait, and the code of all roles shares the
// instruction caches).  One that runs out: the CTA's roles run on without waiting, so that all reach the end;
// what they compute is unspecified.
__device__ __noinline__ void long_wait(uint32_t bar, uint32_t parity, Misc *misc)
{
    volatile int *abort_flag = &misc->abort;
    const long long limit = misc->wait_limit, start = clock64();
    const bool poll = limit < (1 << 16); // a test's limit: the suspending form may sleep past it
    while (!(poll ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))) {
        if (*abort_flag)
            return;
        if (clock64() - start > limit) {
            *abort_flag = 1;
            set_error(misc->err, kErrTimeout);
            return;
        }
    }
}

// Rows from .. to - 1 (of all heads) of the outputs, of requests without states: one warp.
__device__ __forceinline__ void write_idle(const AttendParams &p, size_t from, size_t to)
{
    const int lane = threadIdx.x & 31;
    uint4 *out = reinterpret_cast<uint4 *>(p.out + from * kDim);
    for (size_t i = lane; i < (to - from) * (kDim / 8); i += 32)
        out[i] = make_uint4(0u, 0u, 0u, 0u);
    for (size_t i = from + lane; i < to; i += 32)
        p.lse[i] = __uint_as_float(0xFF800000u);
}

template <int FMT>
__global__ void __launch_bounds__(threads_of(FMT), 1)
    attend_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap q_map, const AttendParams p)
{
    constexpr int TILES = ring_tiles(FMT), TB = tile_bytes(FMT), NT = threads_of(FMT);
    constexpr bool CONV = FMT != kFmtBf16;
    constexpr Smem L = smem_layout(FMT);
    extern __shared__ __align__(1024) uint8_t gsm[];
    const uint32_t smem = smem_u32(gsm);
    Misc &misc = *reinterpret_cast<Misc *>(gsm + L.misc);
    constexpr int DEPTH = ready_tiles(FMT);
    const uint32_t full = smem + L.bars, empty = full + TILES * 8, ready = empty + TILES * 8, ready_free = ready + DEPTH * 8;
    const uint32_t q_full = ready_free + DEPTH * 8, s_full = q_full + 16, p_full = s_full + 16, pv_done = p_full + 16,
                   o_free = pv_done + 16, turn = o_free + 16, drain = turn + 16, q_raw = CONV ? drain + 16 : q_full;
    volatile int *abort_flag = &misc.abort;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    launch_dependents();
    if (smem & 1023u) { // swizzled tiles need it; the declaration gives it
        if (threadIdx.x == 0) {
            set_error(p.err, kErrScratch);
            p.joins[blockIdx.x].c0 = -1, p.joins[blockIdx.x].idle = 0;
        }
        return;
    }
    if (threadIdx.x == 0) {
        prefetch_tensormap(&map);
        prefetch_tensormap(&q_map);
        for (int i = 0; i < TILES; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, CONV ? 4 : 2); // the converter warps, or the issuers
        }
        for (int i = 0; i < DEPTH; ++i) {
            mbar_init(ready + 8 * i, CONV ? 4 : 1); // the converter warps, or the clearing warp
            mbar_init(ready_free + 8 * i, 2);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(q_full + 8 * t, CONV ? 4 : 1); // the converter warps, or the copy itself
            if (CONV)
                mbar_init(q_raw + 8 * t, 1);
            mbar_init(turn + 8 * t, 1);
            mbar_init(drain + 8 * t, 1);
            mbar_init(s_full + 8 * t, 1);
            mbar_init(p_full + 8 * t, 8);
            mbar_init(pv_done + 8 * t, 1);
            mbar_init(o_free + 8 * t, 8);
        }
        fence_mbar_init();
        misc.abort = 0;
        misc.idle = 0;
        misc.wait_limit = p.wait_limit;
        misc.err = p.err;
    }
    if (threadIdx.x < 8)
        misc.later_bad[threadIdx.x] = 0;
    if (warp == 1)
        tmem_alloc(smem_u32(&misc.tmem), 512);

    // ---- the line of pages and this CTA's range of it ----
    const int per = (p.R + NT - 1) / NT;
    const int lo = min(p.R, (int)threadIdx.x * per), hi = min(p.R, lo + per);
    long long mine = 0;
    Request q{};
    bool idle_here = false; // requests without states
    bool down = false;      // offsets that go down: requests that share rows, in sum more of them than the batch has
    for (int r = lo; r < hi; ++r) {
        bool bad, idle;
        q = read_request(p, r, &bad, &idle);
        down |= p.offsets[r + 1] < q.first;
        idle_here |= idle;
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
    down = __syncthreads_or(down);
    long long before = incl - mine, W = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        before += i < warp ? misc.scan[i] : 0;
        W += misc.scan[i];
    }
    if (down) // reported: no line, and no outputs
        W = 0;
    if (idle_here && !down)
        misc.idle = 1;
    const int ranges = (int)min((long long)gridDim.x, max(1ll, W / kMinRange));
    Share w{};
    const long long x0 = (int)blockIdx.x < ranges ? cut(blockIdx.x, W, ranges) : W;
    const long long x1 = (int)blockIdx.x < ranges ? cut(blockIdx.x + 1, W, ranges) : W;
    if (x0 < x1 && before <= x0 && x0 < before + mine) {
        long long at = before;
        int r = lo;
        if (per > 1)
            for (;; ++r) {
                bool bad, idle;
                q = read_request(p, r, &bad, &idle);
                const long long some = q.units ? q.before(p, q.units) * p.Hkv : 0;
                if (x0 < at + some)
                    break;
                at += some;
            }
        misc.start = q;
        misc.start_r = r;
        misc.start_before = at;
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = misc.tmem;
    if (x0 < x1) {
        w.r = misc.start_r;
        w.q = misc.start;
        const long long in = x0 - misc.start_before, each = w.q.before(p, w.q.units);
        w.head = (int)quotient(in, each);
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
        const int in_unit = (int)(rest - w.q.before(p, w.u));
        w.b = max(0, in_unit - kUnitCost);
        w.nb = w.q.pages(p, w.u);
        w.left = (int)(x1 - x0) + in_unit; // (the host has seen that it fits)
        if (w.left <= kUnitCost + w.b)     // the range ends before the unit's first page
            w.left = 0;
    }
    if (threadIdx.x == 0) {
        AttendJoin j{};
        j.c0 = -1;
        j.idle = misc.idle;
        if (w.left > 0 && w.b > 0) {
            const int c0 = cut_of(x0 - w.b, W, ranges); // (x0 is page b)
            if (c0 == (int)blockIdx.x - 1) {
                j.token0 = w.token0(p);
                j.tokens = w.q.tokens(p, w.u);
                j.head = w.head;
                j.c0 = c0;
                j.c1 = cut_of(x0 - w.b + w.nb - 1, W, ranges);
            }
        }
        p.joins[blockIdx.x] = j;
    }
    auto wait = [&](uint32_t bar, uint32_t parity) {
        // (the suspending form at once: asking first costs more than it saves wherever the wait is a real one:
        // ragged prompts 432 us so, 422 without)
        if (p.wait_limit < (1 << 16) || !mbar_try_wait(bar, parity))
            long_wait(bar, parity, &misc);
    };

    if (warp == 0) {
        // ---- producer: K and V tiles in the order of their use ----
        int z = 0, st = 0;
        uint32_t ph = 0;
        for (; w.left > 0; w.next(p)) {
            const int n = w.pages();
            const bool two = w.two(p);
            const int32_t *row = p.block_table + (size_t)w.r * p.maxB + w.b;
            int ent = 0, ent0 = -1;
            for (int i = 0; i < 2 * n; ++i) {
                int pg;
                const bool is_k = tile_of(two, n, i, &pg);
                const int win = pg >> 5; // (a pair of pages lies in one window)
                if (win > ent0) {
                    ent0 = win;
                    ent = 32 * win + lane < n ? row[32 * win + lane] : 0;
                }
                long long page = __shfl_sync(0xffffffffu, ent, pg & 31);
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
    } else if (warp < 3) {
        // ---- MMA issuer of stream t.  The issuers take turns: P V of a page and S of the stream's next page,
        // which waits for P V (it replaces P), and then the other stream's, whose softmax that time
        // was for.  Left to themselves the streams fall into step, both in their softmax and then both at
        // the tensor cores (a page of two streams 3500 clocks).  (One issuer for both spends longer on its
        // own instructions between two MMAs than an MMA takes.) ----
        const int t = warp - 1;
        const uint32_t one = elect_one(), tm = uniform(tmem), base = uniform(smem);
        constexpr uint32_t kTypes = CONV ? ~((1u << 7) | (1u << 10)) : ~0u; // f16 or bf16 operands
        constexpr uint32_t idesc_s = umma_idesc_bf16(128, 128, 0, 0) & kTypes;
        constexpr uint32_t idesc_o = umma_idesc_bf16(128, 128, 0, 1) & kTypes;
        constexpr uint32_t RING = CONV ? L.staged : 0;
        const uint32_t tile_free = CONV ? ready_free : empty;
        const uint32_t q = uniform(desc_low(base + L.q + t * kTile16, 16)), d_s = tm + uniform(128 * t), d_o = tm + uniform(256 + 128 * t);
        const uint32_t ring = uniform((base + RING) >> 4);
        uint32_t done = 0, turns_taken = 0; // steps and turns of this stream so far
        auto take_turn = [&] {
            if (t == 1 || turns_taken > 0)
                wait(turn + 8 * t, (t == 1 ? turns_taken : turns_taken - 1) & 1u);
            ++turns_taken;
        };
        auto end_turn = [&] {
            if (lane == 0)
                mbar_arrive(turn + 8 * (t ^ 1));
        };
        int st0 = 0;       // the unit's first tile: its slot and the slot's phase
        uint32_t ph0 = 0;
        for (; w.left > 0; w.next(p)) {
            const int n = w.pages();
            const bool two = w.two(p);
            // (both streams take as many steps: stream 1 one without a page behind an odd number of them)
            const int nsteps = two ? n : (n + 1) >> 1, stride = two ? 2 : 4, pages = two || t == 0 ? nsteps : n >> 1;
            // slot and phase of the tile i places behind the unit's first
            auto slot_of = [&](int i, uint32_t &ph) {
                const int z = st0 + i, turns = z / DEPTH;
                ph = (ph0 + turns) & 1u;
                return uniform(z - turns * DEPTH);
            };
            // a tile is given back, once its products are done, by both streams, or twice by the one that uses it
            auto give_back = [&](uint32_t st) {
                umma_commit(tile_free + 8 * st);
                if (!two)
                    umma_commit(tile_free + 8 * st);
            };
            wait(q_full + 8 * t, w.seg & 1);
            // S of a step into the S buffer (its K tile has been waited for).  The turn ends half way: the other
            // issuer's waits end as these products do (behind the last: ragged prompts 466 us, half way 459)
            auto score = [&](uint32_t st, bool page) {
                const uint32_t k = (ring + st * (kTile16 >> 4) & 0x3FFFu) | (16u >> 4) << 16;
                if (page) {
#pragma unroll
                    for (uint32_t ks = 0; ks < 8; ++ks) {
                        umma_ss(one, d_s, q + (ks >> 2) * 1024 + (ks & 3) * 2, k + (ks >> 2) * 1024 + (ks & 3) * 2, idesc_s, ks > 0);
                        if (ks == 3)
                            end_turn();
                    }
                } else {
                    end_turn();
                }
                if (elect_one())
                    umma_commit(s_full + 8 * t);
                __syncwarp();
            };
            uint32_t k_ph, k_st = slot_of(two ? 0 : t, k_ph);
            if (pages > 0)
                wait(ready + 8 * k_st, k_ph);
            take_turn();
            tcgen05_after_sync();
            score(k_st, pages > 0); // (P V of the unit before, which reads what S replaces, was waited for at its end)
            if (pages > 0 && elect_one())
                give_back(k_st);
            __syncwarp();
            for (int i = 0; i < nsteps; ++i, ++done) {
                // everything that can be known and waited for before P is there
                uint32_t v_ph; // (V lies behind both K of the pair, or the only one)
                const uint32_t v_st = slot_of(i * stride + (two ? 1 : min(2, n - 2 * i) + t), v_ph);
                const uint32_t v = (ring + v_st * (kTile16 >> 4) & 0x3FFFu) | (16384u >> 4) << 16, more = uniform(i > 0);
                const bool page = i < pages, again = i + 1 < nsteps, next_page = i + 1 < pages;
                if (page)
                    wait(ready + 8 * v_st, v_ph);
                if (next_page) {
                    k_st = slot_of((i + 1) * stride + (two ? 0 : t), k_ph);
                    wait(ready + 8 * k_st, k_ph);
                }
                if (i == 0 && w.seg > 0) // the last unit's O has been read
                    wait(o_free + 8 * t, (w.seg - 1) & 1);
                take_turn(); // (before the wait for P, which is the longer one: a wait that need not wait takes 150 clocks)
                wait(p_full + 8 * t, done & 1u);
                tcgen05_after_sync();
                if (page) {
                    // V, MN-major: 16 positions are 16 rows of 128 bytes
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        umma_ts(one, d_o, d_s + 8 * ks, v + ks * (2048 >> 4), idesc_o, ks > 0 ? 1u : more);
                }
                if (elect_one())
                    umma_commit(pv_done + 8 * t);
                __syncwarp();
                if (again) // S replaces P: products of one thread run in the order of their issue
                    score(k_st, next_page);
                else
                    end_turn();
                if (elect_one()) {
                    if (page)
                        give_back(v_st);
                    if (next_page)
                        give_back(k_st);
                }
                __syncwarp();
            }
            const int turns = (st0 + 2 * n) / DEPTH;
            st0 += 2 * n - turns * DEPTH;
            ph0 ^= turns & 1u;
            if (__any_sync(0xffffffffu, *abort_flag != 0)) // all lanes alike
                break;
        }
        // nothing of this CTA's may be in flight when its tensor memory is freed
        if (one) {
            umma_commit(drain + 8 * t);
            mbar_wait_bounded(drain + 8 * t, 0);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ---- clearing of V tiles (converters do it for theirs).  Every tile passes this warp on its way
        // to the issuers, so that no barrier gets two phases ahead of it ----
        int z = 0;
        for (; !CONV && w.left > 0; w.next(p)) {
            const int n = w.pages(), seen = w.q.seen(p, w.u), past = seen + (p.causal ? w.q.tokens(p, w.u) - 1 : 0);
            const bool two = w.two(p);
            for (int i = 0; i < 2 * n; ++i, ++z) {
                int pg;
                const bool is_k = tile_of(two, n, i, &pg);
                const int st = z % TILES;
                pg += w.b;
                wait(full + 8 * st, (uint32_t)(z / TILES) & 1u);
                if (!is_k && (pg + 1) * kPage > seen)
                    clear_rows(gsm + st * TB, seen - pg * kPage, past - pg * kPage, &misc.later_bad[w.seg & 7], w.seg + 1);
                if (lane == 0)
                    mbar_arrive(ready + 8 * st);
                __syncwarp();
            }
        }
        // ---- outputs of requests without states, where no kernel follows ----
        for (int r = 0; r < p.R && gridDim.x == 1 && misc.idle; ++r) {
            bool bad, idle;
            const Request q = read_request(p, r, &bad, &idle);
            const size_t heads = (size_t)p.Hkv * p.G;
            if (idle)
                write_idle(p, heads * q.first, heads * (q.first + q.n));
        }
    } else if (warp < 20) {
        // ---- softmax: a thread has 64 columns of a page of a query row ----
        const int t = (warp - 4) >> 3, half = (warp >> 2) + 1 & 1, at_lane = threadIdx.x & 127;
        const bool leads = warp == 4 + 8 * t; // the stream's warp that copies queries
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21); // this warp's lane quarter
        const uint32_t at_s = lanes + 128 * t + 64 * half, at_p = lanes + 128 * t + 32 * half, o_at = lanes + 256 + 128 * t + 64 * half;
        const float ninf = __uint_as_float(0xFF800000u);
        const uint32_t xch = smem + L.xch + 4 * at_lane; // float [stream][half][row]
        const uint32_t mine = xch + 1024 * t + 512 * half, others = xch + 1024 * t + 512 * (half ^ 1);
        const int Hq = p.Hkv * p.G, each = p.unit_tokens >> 1; // tokens of a stream
        uint32_t steps = 0; // so far, alike for both streams
        const int pair_bar = 1 + 4 * t + (warp & 3);
        auto sync_pair = [&] { asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory"); };
        auto sync_all = [&] { asm volatile("bar.sync 9, 512;" ::: "memory"); };
        // Query rows of a unit into the stream's operand tile, once the stream's last S of the unit
        // before is done.  Rows beyond the unit's hold anything: nothing is read from what they give.
        uint32_t copies = 0;
        auto copy_queries = [&](const Share &u) {
            if (*abort_flag) // (the last copy may still be on its way)
                return;
            ++copies;
            if (elect_one()) {
                const int token = u.token0(p) + (u.two(p) ? each * t : 0);
                const uint32_t dst = smem + L.q + t * kTile16, bar = q_raw + 8 * t;
                mbar_arrive_expect_tx(bar, 2 * 128 * p.G * each);
                tma_load_3d(dst, &q_map, 0, u.head * p.G, token, bar);
                tma_load_3d(dst + 16384, &q_map, 64, u.head * p.G, token, bar);
            }
            __syncwarp();
        };
        auto rows_of = [&](const Share &w) { return (w.two(p) && t ? w.q.tokens(p, w.u) - each : min(each, w.q.tokens(p, w.u))) * p.G; }; // the stream's
        const int token_in = at_lane / p.G, head_in = at_lane - token_in * p.G; // the row's in its stream (beyond the unit's rows: some)
        auto token_of = [&](const Share &w) { return (w.two(p) ? each * t : 0) + token_in; };
        auto sees = [&](const Share &w) { return w.q.seen(p, w.u) + (p.causal ? token_of(w) : 0); };                                    // and its positions
        if (w.left > 0 && leads)
            copy_queries(w);
        while (w.left > 0) {
            float m = 0.f, l = 0.f, lr = 0.f; // reference, sum, sum of the rounded p
            const int kept = fold(w);
            {
                const int n = w.pages();
                const bool two = w.two(p);
                const int nsteps = two ? n : (n + 1) >> 1, npages = two || t == 0 ? nsteps : n >> 1; // (see the issuers)
                const bool real = at_lane < rows_of(w), idle = (warp & 3) * 32 >= rows_of(w); // idle: no row of this warp's is the unit's
                float sc = p.scale_log2;
                const int parity = w.seg & 1;
                // A row's reference is its maximum over the first page.  Later pages are not searched for theirs:
                // p may pass 1 as long as it stays a number that P and the sums can hold, which the sum of half a
                // page tells; where a row's passes kMost its warps' rows get new references before P is written.
                auto new_reference = [&](int i, int seen) {
                    if (CONV && i == 0 && real) // (the exponents are there once S is)
                        sc *= __uint_as_float((uint32_t)(reinterpret_cast<const int8_t *>(gsm + L.inv)[kRows * parity + 128 * t + at_lane] + 127) << 23);
                    float mx = row_maximum(at_s, sc, seen);
                    sts32(mine, mx);
                    sync_pair();
                    mx = fmaxf(mx, lds32(others)) - (CONV ? kPUp16 : 0.f);
                    const float ref = mx == ninf ? 0.f : mx, f = i > 0 && mx > m ? ex2(m - ref) : 1.f;
                    m = i == 0 || mx > m ? ref : m;
                    l *= f;
                    lr *= f;
                    if (i > 0) {
                        wait(pv_done + 8 * t, (steps - 1) & 1u); // O holds every step before this one
                        tcgen05_after_sync();
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            float o[16];
                            tmem_ld16(o_at + 16 * c, o);
                            uint32_t r[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                r[k] = __float_as_uint(o[k] * f);
                            tmem_st16(o_at + 16 * c, r);
                        }
                    }
                };
                auto page_done = [&](const uint32_t *pr) {
                    tmem_st32(at_p, pr);
                    tmem_wait_st();
                    tcgen05_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(p_full + 8 * t);
                };
                // all pages but the last of the share and those that some row does not see to their end
                const int step = two ? kPage : 2 * kPage, pos1 = (w.b + (two ? 0 : t)) * kPage;
                const int to_end = w.q.seen(p, w.u) - kPage - pos1;
                const int whole_pages = idle ? 0 : max(0, min(npages - 1, to_end >= 0 ? to_end / step + 1 : 0));
                int seen = sees(w) - pos1 - whole_pages * step - 64 * half; // columns that this row sees behind those
                int i = 0;
#pragma unroll 1
                for (; i < whole_pages; ++i, ++steps) {
                    wait(s_full + 8 * t, steps & 1u);
                    tcgen05_after_sync();
                    if (i == 0)
                        new_reference(0, 64);
                    uint32_t pr[32];
                    float rounded, sum;
                    bool again = false;
                    do {
                        if (again)
                            new_reference(i, 64);
                        sum = row_to_p<CONV, false>(at_s, sc, m, 64, pr, rounded);
                        // (both warps have read S, which P replaces)
                        again = any_of_two_warps(pair_bar, !again && real && i > 0 && sum > (CONV ? kMost16 : kMost));
                    } while (again);
                    l += sum;
                    lr += rounded;
                    page_done(pr);
                }
#pragma unroll 1
                for (; i < nsteps; ++i, ++steps, seen -= step) {
                    wait(s_full + 8 * t, steps & 1u);
                    if (i == nsteps - 1 && leads) {
                        Share nx = unfold(kept); // S was the last to read this unit's
                        if (!nx.last()) {
                            nx.next(p);
                            copy_queries(nx);
                        }
                    }
                    if (idle || i >= npages) {
                        if (lane == 0)
                            mbar_arrive(p_full + 8 * t);
                        continue;
                    }
                    tcgen05_after_sync();
                    if (i == 0)
                        new_reference(0, min(64, seen));
                    uint32_t pr[32];
                    float rounded, sum;
                    bool again = false;
                    do {
                        if (again)
                            new_reference(i, min(64, seen));
                        sum = row_to_p<CONV, true>(at_s, sc, m, seen, pr, rounded);
                        again = any_of_two_warps(pair_bar, !again && real && i > 0 && sum > (CONV ? kMost16 : kMost));
                    } while (again);
                    l += sum;
                    lr += rounded;
                    page_done(pr);
                }
            }

            // ---- end of the unit's share ----
            w = unfold(kept);
            const int n = w.pages(), rows = rows_of(w);
            const bool two = w.two(p), real = at_lane < rows, idle = (warp & 3) * 32 >= rows;
            const bool whole = w.b == 0 && n == w.nb, ends = w.b + n == w.nb;
            // both warps of a row get the same sums: l goes by a thread's own place, lr back by the other's
            sts32(mine, l);
            sync_pair();
            l += lds32(others);
            if (!CONV)
                sts32(others, lr);
            sync_pair();
            if (!CONV)
                lr += lds32(mine);
            // O is divided by the sum of the rounded p, here as a factor: the sums that go on are those of the p
            float M = m, fa = CONV || l == 0.f ? 1.f : l / lr, fb = 0.f;
            if (!two) {
                sync_all(); // (every pair has read its sums)
                if (t == 1) {
                    sts32(mine, half ? l : m);
                    if (half)
                        sts32(xch, fa);
                }
                sync_all();
                const float mb = lds32(xch + 1024), lb = lds32(xch + 1536), cb = lds32(xch);
                sync_all();
                if (t == 1) { // stream 0 reads both accumulators
                    w.next(p);
                    continue;
                }
                // (a sum of 0: no column, and any reference)
                M = l == 0.f ? mb : lb == 0.f ? m : fmaxf(m, mb);
                const float ea = l == 0.f ? 0.f : ex2(m - M), eb = lb == 0.f ? 0.f : ex2(mb - M);
                l = l * ea + lb * eb;
                fa *= ea;
                fb = cb * eb;
            }
            // (what does not need O comes before the wait for its last products)
            // this row among the batch's: behind the unit's first token's first head by so many
            const int in_unit = token_of(w) * Hq + w.head * p.G + head_in;
            const long long unit_row = (long long)w.token0(p) * Hq;
            const int slot_row = (two ? 128 * t : 0) + at_lane;
            float *slot = p.partial + (size_t)(2 * blockIdx.x + (ends ? 0 : 1)) * kSlotFloats;
            const float fin = whole ? (l > 0.f || l != l ? p.v_scale / l : 0.f) : 1.f;
            const float ga = fa * fin, gb = n > 1 ? fb * fin : 0.f; // (with one page stream 1 has no O)
            const int neighbours = __shfl_xor_sync(0xffffffffu, in_unit, 1);
            if (real && half == 0) {
                if (whole) {
                    p.lse[unit_row + in_unit] = l == 0.f ? ninf : (M + log2f(l)) * 0.6931471805599453f;
                } else {
                    slot[(size_t)kRows * kDim + slot_row] = l == 0.f ? ninf : M;
                    slot[(size_t)kRows * (kDim + 1) + slot_row] = l;
                }
            }
            const bool zeros = __any_sync(0xffffffffu, fa == 0.f || (!two && gb == 0.f));
            wait(pv_done + 8 * t, (steps - 1) & 1u);
            if (!two) // stream 1 has given all its P: the last of its products is the one under way
                wait(pv_done + 8, (steps - 1) & 1u);
            tcgen05_after_sync();
            constexpr int C = CONV ? 16 : 32; // columns at a time (registers, as above)
#pragma unroll 1
            for (int c = 0; c < 64 && !idle; c += C) {
                uint32_t a[C];
                auto load = [&](uint32_t at, uint32_t *v) { // 16 columns
                    uint32_t(&w16)[16] = *reinterpret_cast<uint32_t(*)[16]>(v);
                    tmem_ld_async(at, w16);
                    tmem_wait_async(w16);
                };
#pragma unroll
                for (int h = 0; h < C; h += 16)
                    load(o_at + c + h, a + h);
                if (zeros) { // a row of zeros, whatever V has
#pragma unroll
                    for (int k = 0; k < C; ++k)
                        a[k] = fa != 0.f ? a[k] : 0u;
                }
#pragma unroll
                for (int k = 0; k < C; k += 2) {
                    float e0, e1;
                    unpair(mul2(pair(__uint_as_float(a[k]), __uint_as_float(a[k + 1])), pair(ga, ga)), e0, e1);
                    a[k] = __float_as_uint(e0);
                    a[k + 1] = __float_as_uint(e1);
                }
                if (!two)
#pragma unroll
                    for (int h = 0; h < C; h += 16) {
                        uint32_t o[16];
                        load(o_at + 128 + c + h, o);
                        if (zeros) {
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[k] = gb != 0.f ? o[k] : 0u;
                        }
#pragma unroll
                        for (int k = 0; k < 16; k += 2) {
                            float e0, e1;
                            unpair(fma2(pair(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), pair(gb, gb), pair(__uint_as_float(a[h + k]), __uint_as_float(a[h + k + 1]))), e0, e1);
                            a[h + k] = __float_as_uint(e0);
                            a[h + k + 1] = __float_as_uint(e1);
                        }
                    }
                if (whole) { // C values a row by two lanes
                    uint32_t d[2][C / 4];
#pragma unroll
                    for (int k = 0; k < C / 2; ++k)
                        d[k / (C / 4)][k % (C / 4)] = pack_bf16(__uint_as_float(a[2 * k]), __uint_as_float(a[2 * k + 1]));
                    transpose2(d); // d[k]: piece lane % 2 of row k of the two
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if ((at_lane & ~1) + k < rows)
                            store(p.out + (unit_row + ((lane & 1) == k ? in_unit : neighbours)) * kDim + 64 * half + c + C / 2 * (lane & 1), d[k]);
                } else if (real) {
#pragma unroll
                    for (int k = 0; k < C / 4; ++k) // 16-byte piece i of row r of a slot lies at i kRows + r
                        reinterpret_cast<uint4 *>(slot)[(16 * half + c / 4 + k) * kRows + slot_row] =
                            make_uint4(a[4 * k], a[4 * k + 1], a[4 * k + 2], a[4 * k + 3]);
                }
            }
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(o_free + 8 * t);
                if (!two)
                    mbar_arrive(o_free + 8);
            }
            if (real && misc.later_bad[w.seg & 7] == w.seg + 1)
                add_late_values<FMT>(p, w.r, w.head, unit_row + in_unit, max(w.q.seen(p, w.u), w.b * kPage), min(sees(w), (w.b + w.pages()) * kPage), M,
                                     whole ? nullptr : slot + 4 * slot_row, 64 * half);
            w.next(p);
        }
        if (copies > 0) // the CTA's memory must outlive them (they have long landed unless a wait ran out)
            mbar_wait_bounded(q_raw + 8 * t, (copies - 1) & 1u);
    } else if constexpr (CONV) {
        // ---- converters: a ring tile to a 16-bit tile, in the order of use ----
        const int row = threadIdx.x & 127;
        int z = 0;
        for (; w.left > 0; w.next(p)) {
            const int n = w.pages(), seen = w.q.seen(p, w.u), past = seen + (p.causal ? w.q.tokens(p, w.u) - 1 : 0);
            const bool two = w.two(p);
            for (int t = 0; t < 2; ++t) {
                wait(q_raw + 8 * t, w.seg & 1);
                widen_queries(gsm + L.q + t * kTile16, reinterpret_cast<int8_t *>(gsm + L.inv) + kRows * (w.seg & 1) + 128 * t);
                fence_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(q_full + 8 * t);
            }
            for (int i = 0; i < 2 * n; ++i, ++z) {
                int page0;
                const bool is_k = tile_of(two, n, i, &page0);
                page0 = (w.b + page0) * kPage;
                const bool tail = !is_k && page0 + kPage > seen;
                const bool drop = tail && page0 + row >= past;           // not in the request
                const bool check = tail && !drop && page0 + row >= seen; // seen by later tokens only
                // (mostly over already: both are asked before either answer is waited for)
                const bool here = mbar_test_wait(full + 8 * (z % TILES), (uint32_t)(z / TILES) & 1u);
                const bool room = z < DEPTH || mbar_test_wait(ready_free + 8 * (z % DEPTH), (uint32_t)(z / DEPTH - 1) & 1u);
                if (!here)
                    wait(full + 8 * (z % TILES), (uint32_t)(z / TILES) & 1u);
                if (!room)
                    wait(ready_free + 8 * (z % DEPTH), (uint32_t)(z / DEPTH - 1) & 1u);
                // (E4M3: four pieces ahead; two: the 512-token chunk 748 us for 675, eight: 681)
                const bool bad = convert_row<FMT, 2, 4>(gsm + (z % TILES) * TB, gsm + L.staged + (z % DEPTH) * kTile16 + row * 128, row, tail, drop, check);
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

// Units cut between CTAs: block (c, y, z) has rows 32 y .. and columns 32 z .. of the unit that CTA c + 1
// begins inside of; a warp has a 16-byte piece of each row, a lane a row.  Beside that the outputs of requests
// without states, a share of each one's rows by each block: 4096 tokens of 64 heads (67 MB) 29 us, a fill of them 20 (one
// warp a request: 1070; all warps of the kernel above, at its end: 28, but ragged cross attention 68 -> 71).
__global__ void __launch_bounds__(256) attend_join_kernel(const AttendParams p)
{
    constexpr int U = 4; // slots on their way at once
    __shared__ float4 sm_o[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    const AttendJoin jn = p.joins[blockIdx.x + 1];
    if (jn.idle && blockIdx.y == 0)
        for (int r0 = 32 * warp; r0 < p.R; r0 += 32 * 8) {
            bool bad, idle = false;
            Request q{};
            if (r0 + lane < p.R)
                q = read_request(p, r0 + lane, &bad, &idle);
            for (uint32_t some = __ballot_sync(0xffffffffu, idle); some; some &= some - 1) {
                const size_t heads = (size_t)p.Hkv * p.G, first = heads * __shfl_sync(0xffffffffu, q.first, __ffs(some) - 1);
                const size_t rows = heads * __shfl_sync(0xffffffffu, q.n, __ffs(some) - 1);
                const int part = 4 * blockIdx.x + blockIdx.z, parts = 4 * gridDim.x;
                write_idle(p, first + rows * part / parts, first + rows * (part + 1) / parts);
            }
        }
    const int each = p.unit_tokens >> 1, t = blockIdx.y >> 2, row = 32 * blockIdx.y + lane;
    const int rows = min(each, jn.tokens - t * each) * p.G; // of stream t, from row 128 t on
    if (jn.c0 < 0 || 32 * (int)(blockIdx.y & 3) >= rows)
        return;
    const float ninf = __uint_as_float(0xFF800000u);
    const bool real = 32 * (int)(blockIdx.y & 3) + lane < rows;
    const int piece = 8 * blockIdx.z + warp;
    float M = ninf, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = jn.c0; c <= jn.c1 && real; c += U) {
        float m[U], a[U];
        float4 v[U];
#pragma unroll
        for (int s = 0; s < U; ++s) {
            const int cc = c + s;
            m[s] = ninf;
            a[s] = 0.f;
            v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (cc <= jn.c1) {
                const float *slot = p.partial + (size_t)(2 * cc + (cc < jn.c1 ? 1 : 0)) * kSlotFloats;
                m[s] = slot[(size_t)kRows * kDim + row];
                a[s] = slot[(size_t)kRows * (kDim + 1) + row];
                v[s] = reinterpret_cast<const float4 *>(slot)[piece * kRows + row];
            }
        }
        float n = M;
#pragma unroll
        for (int s = 0; s < U; ++s)
            n = fmaxf(n, m[s]);
        const float ref = n == ninf ? 0.f : n, f = ex2(M - ref);
        l *= f;
        o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
        for (int s = 0; s < U; ++s) {
            const float e = ex2(m[s] - ref);
            l += a[s] * e;
            if (m[s] != ninf) // (a slot's row without columns holds anything)
                o.x += v[s].x * e, o.y += v[s].y * e, o.z += v[s].z * e, o.w += v[s].w * e;
        }
        M = n;
    }
    const float f = l > 0.f || l != l ? p.v_scale / l : 0.f;
    const int i = 32 * (blockIdx.y & 3) + lane, j = t * each + i / p.G;
    if (real && piece == 0)
        p.lse[((size_t)(jn.token0 + j) * p.Hkv + jn.head) * p.G + i % p.G] = l == 0.f ? ninf : (M + log2f(l)) * 0.6931471805599453f;
    sm_o[warp][lane] = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    __syncthreads();
    // 64 bytes a row
    const int k = threadIdx.x >> 3, ik = 32 * (blockIdx.y & 3) + k;
    if (ik < rows) {
        const float4 x = sm_o[threadIdx.x & 7][k];
        const size_t out = ((size_t)(jn.token0 + t * each + ik / p.G) * p.Hkv + jn.head) * p.G + ik % p.G;
        reinterpret_cast<uint2 *>(p.out + out * kDim + 32 * blockIdx.z)[threadIdx.x & 7] = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
    }
}

template <int FMT>
cudaError_t launch_t(const AttendParams &p, const CUtensorMap &map, const CUtensorMap &q_map, int ctas, cudaStream_t stream)
{
    constexpr int smem = smem_layout(FMT).total;
    cudaError_t e = cudaFuncSetAttribute(attend_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess)
        return e;
    // no more CTAs than the line can have ranges, whatever the lengths in device memory are
    const double units = (double)(p.T / p.unit_tokens + p.R) * p.Hkv, most = units * (kUnitCost + p.maxB) / kMinRange;
    if (most < ctas)
        ctas = most < 1 ? 1 : (int)most;
    e = launch_kernel(attend_kernel<FMT>, dim3(ctas), dim3(threads_of(FMT)), smem, stream, false, map, q_map, p);
    // a unit has no more rows than the batch
    const int rows = (p.T < p.unit_tokens / 2 ? p.T : p.unit_tokens / 2) * p.G, blocks = p.T > p.unit_tokens / 2 ? 8 : (rows + 31) / 32;
    if (e == cudaSuccess && ctas > 1)
        e = launch_kernel(attend_join_kernel, dim3(ctas - 1, blocks, 4), dim3(256), 0, stream, true, p);
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
    p.unit_tokens = 2 * (kRows / 2 / p.G);
    CUtensorMap map, q_map;
    if (!encode_pool_map(&map, p.kv, kv_dtype, p.num_pages, p.Hkv) || !encode_token_rows(&q_map, p.q, p.T, p.Hkv * p.G, p.G, p.unit_tokens / 2))
        return cudaErrorInvalidValue;
    if (kv_dtype == MSA_BF16)
        return launch_t<kFmtBf16>(p, map, q_map, ctas, stream);
    if (kv_dtype == MSA_FP8_E4M3)
        return launch_t<kFmtFp8>(p, map, q_map, ctas, stream);
    return launch_t<kFmtF4>(p, map, q_map, ctas, stream);
}

} // namespace msa
