// msa_append.cu -- norm and rotation of query and key rows, and new keys, values
// and index keys written into their pages, one pass over the rows.
//
// For a row x of 128 elements of the token at position p:
//   n = x rsqrt(mean x^2 + eps) (w + offset)            (rows with norm weights)
//   a' = s (a cos t - b sin t), b' = s (b cos t + a sin t)   for each pair (a, b) of
//   the first rotary_dim elements of n, t = p f_i; the others stay.
// Everything is fp32 and rounded once, to bf16 or to the pool's format.  Angles
// are fixed point: the table has f_i as a fraction of 2^64 of a turn, and p times that
// wraps around by itself at any position (in fp32 p f_i loses 2^-24 of itself, 0.06 rad
// at a million).  What is left is a turn in [-1/2, 1/2), as a float: off by 2^-26 of a
// turn and 2^-32, beside p times what the table is off by (2^-52 of f_i and 2^-64 of a turn).
//
// Memory-bound: 256 bytes read and 256 (E4M3 128, NVFP4 72) written a row, latency
// where tokens are few.  A warp takes four heads of one token at a time, eight lanes
// a row; a lane holds two 16-byte pieces that rotate with one another, so that the
// rotation needs no exchange and the norm three shuffles.  The lane's eight angles
// are the same for all heads: computed once a token, two by each row's lanes.
//
// Measured (one GB300): 8192 tokens of 68 rows (285 MB) 54.5 us, 5.2 TB/s; ragged bf16 prompts with their queries
// (659 MB) 111 us, 5.9 TB/s; E4M3 keys and values of 8 heads alone (146 MB) 40 us, 3.7 TB/s, bound by fixed latencies
// (16 warps an SM, issue slots 58 % busy) and by the instructions of a token beside those of its few groups of rows;
// 48 single tokens 5.8 us.
//
// Counted in instructions, 1 KB in and out are 90 clocks of an SM's share of HBM, and so every
// instruction of a group of rows counts: arithmetic on pairs of fp32, weights kept in
// registers from one head to the next, four codes rid of their -0 at a time.
#include "msa_quant.cuh"
#include "msa_ragged.cuh"
#include "msa_umma.cuh"

namespace msa {
namespace {

constexpr int kWarps = 4, kCtas = 4; // warps a CTA, CTAs an SM (5, of 96 registers that spill: ragged prompts 111 -> 131 us)
constexpr int kSlots = 4;            // groups of four rows that a warp has room for: all but one on their way

// Eight bf16 as four pairs of fp32, and back.
__device__ __forceinline__ void widen(uint4 d, uint64_t *v)
{
    const uint32_t e[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        v[k] = pair(__uint_as_float(e[k] << 16), __uint_as_float(e[k] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 narrow(const uint64_t *v)
{
    uint32_t e[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float a, b;
        unpair(v[k], a, b);
        e[k] = pack_bf16(a, b);
    }
    return make_uint4(e[0], e[1], e[2], e[3]);
}

// The request whose tokens token t is among, -1 if none: the last r with
// offsets[r] <= t.  The warp's lanes try 32 places at a time.
__device__ __forceinline__ int request_of(const int32_t *offsets, int R, int t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = R;
    while (n > 1) {
        const int step = (n + 31) >> 5, at = lo + lane * step;
        const bool below = lane > 0 && at < lo + n && offsets[at] <= t;
        const int k = __popc(__ballot_sync(0xffffffffu, below));
        lo += k * step;
        n = min(step, n - k * step);
    }
    return offsets[lo] <= t && t < offsets[lo + 1] ? lo : -1;
}

// Where a lane's two pieces of 8 elements lie: piece i < m turns with piece i + m
// (m = rotary_dim / 16, interleaved pairs: 8), and of those behind them piece 2 m + i is
// with 8 + m + i.  Neighbouring lanes have neighbouring pieces: with a lane's two
// next to one another each load and store asks for halves of sectors, twice (a plain copy of
// 8192 x 68 rows 67 us, 44 so).
__device__ __forceinline__ int piece(int l, int slot, int m)
{
    return slot == 0 ? (l < m ? l : l + m) : (l < m ? l + m : l + 8);
}

// Eight floats by the scale s (inv: its reciprocal where that is exact).
__device__ __forceinline__ void unscale(const uint64_t *v, float s, float inv, float *out)
{
    if (inv != 0.f) {
        const uint64_t by = pair(inv, inv);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            unpair(mul2(v[k], by), out[2 * k], out[2 * k + 1]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            unpair(v[k], out[2 * k], out[2 * k + 1]);
            out[2 * k] = __fdiv_rn(out[2 * k], s);
            out[2 * k + 1] = __fdiv_rn(out[2 * k + 1], s);
        }
    }
}

// Four floats to E4M3 codes (round to nearest even, saturating), a zero as +0.
__device__ __forceinline__ uint32_t e4m3x4(const float *v)
{
    const uint32_t low = 0x7F7F7F7Fu;
    uint32_t w;
    asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n mov.b32 %0, {a, b};\n}\n"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]));
    return w & (((w & low) + low) | low); // a byte's sign stays where its other bits are not 0
}

// A row as NVFP4: v[0], v[1] are this lane's pieces (already divided by the tensor
// scale); 16 elements share a scale, and the other half of them is another lane's
// or this lane's other piece.
__device__ __forceinline__ void store_nvfp4(const float (&v)[2][8], int m, bool real, uint8_t *codes, uint8_t *scales)
{
    const int lane = threadIdx.x & 31, l = lane & 7;
    float amax[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        amax[s] = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            amax[s] = fmaxf(amax[s], fabsf(v[s][k]));
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int c = piece(l, s, m), o = c ^ 1;
        const int owner = o < m ? o : o < m + 8 ? o - m : o - 8, slot = o < m || (o >= 2 * m && o < m + 8) ? 0 : 1;
        const float a = __shfl_sync(0xffffffffu, amax[0], (lane & 24) + owner);
        const float b = __shfl_sync(0xffffffffu, amax[1], (lane & 24) + owner);
        const float top = fmaxf(amax[s], slot ? b : a);
        const uint32_t sc = e4m3x2_rn_sat(0.f, __fdiv_rn(top, 6.f)) & 0xFFu;
        float S, unused;
        f16x2_to_f32x2(e4m3x2_to_f16x2(sc), S, unused);
        uint32_t w = 0;
        if (S > 0.f) {
            float q[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                q[k] = __fdiv_rn(v[s][k], S);
            w = e2m1x4_rn_sat(q[0], q[1], q[2], q[3]) | e2m1x4_rn_sat(q[4], q[5], q[6], q[7]) << 16;
        }
        if (real) {
            *reinterpret_cast<uint32_t *>(codes + 4 * c) = w;
            if ((c & 1) == 0)
                scales[c >> 1] = (uint8_t)sc;
        }
    }
}

// A place in the line of groups: token, set, group of the set, and where this lane's row begins.
struct Cursor {
    const uint16_t *src;
    int t, s, g, n; // n: groups of the set
    __device__ __forceinline__ void enter(const AppendParams &p, int sub)
    {
        const RowSet &set = p.set[s];
        n = (set.heads + 3) >> 2;
        src = set.x + t * set.stride + (g * 4 + sub) * kDim;
    }
    __device__ __forceinline__ void next(const AppendParams &p, int sub)
    {
        src += 4 * kDim;
        if (++g < n)
            return;
        g = 0;
        if (++s == p.sets) {
            s = 0;
            ++t;
        }
        enter(p, sub);
    }
};

// CACHE: tokens of requests, rows to their pages and to outputs; else outputs alone, at the given positions.
template <bool CACHE>
__global__ void __launch_bounds__(32 * kWarps, kCtas) append_kernel(const AppendParams p)
{
    __shared__ uint4 ring[kWarps][kSlots][2][32]; // a lane reads what it copied itself
    const int lane = threadIdx.x & 31, l = lane & 7, sub = lane >> 3;
    const long long all = (long long)p.T * p.groups, wi = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const long long x0 = wi * p.per_warp;
    int left = (int)min((long long)p.per_warp, all - x0);
    // offsets that go down, or past the tokens: a request a thread (there are as many)
    auto check_offsets = [&] {
        const int i = blockIdx.x * (32 * kWarps) + threadIdx.x;
        if (CACHE && i < p.R) {
            const int at = p.offsets[i], next = p.offsets[i + 1];
            if ((at < 0) | (next < at) | (next > p.T))
                set_error(p.err, kErrSeqLen);
        }
    };
    if (left <= 0) {
        check_offsets();
        return;
    }
    const int m = p.interleaved ? 8 : p.units;
    const int at0 = 8 * piece(l, 0, m), at1 = 8 * piece(l, 1, m);
    const uint32_t mine = smem_u32(&ring[threadIdx.x >> 5][0][0][lane]);

    Cursor at{};
    at.t = (int)(x0 / p.groups);
    at.g = (int)(x0 - (long long)at.t * p.groups);
    while (at.s + 1 < p.sets && at.g >= p.set[at.s + 1].group0)
        ++at.s;
    at.g -= p.set[at.s].group0;
    at.enter(p, sub);
    // rows on their way, into the slot that was read before the one to be read next
    Cursor to = at;
    int asked = 0;
    auto ask = [&] {
        if (asked < left && to.g * 4 + sub < p.set[to.s].heads) {
            const uint32_t slot = mine + (asked & (kSlots - 1)) * 1024;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot), "l"(to.src + at0) : "memory");
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + 512), "l"(to.src + at1) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (++asked < left)
            to.next(p, sub);
    };
#pragma unroll 1
    for (int k = 0; k < kSlots - 1; ++k)
        ask();

    int r = -1, first = 0, behind = 0, len = 0; // the token's request, its first token and the first behind it
    const int turned = 2 * p.units; // rotated pieces of 8 elements (interleaved)
    const bool turn0 = p.interleaved ? l < turned : l < m, turn1 = p.interleaved ? l + 8 < turned : turn0;
    // the lane's frequencies: two of the eight pairs that its row's lanes share
    unsigned long long freq[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int e = 2 * sub + k, i = p.interleaved ? (e < 4 ? 4 * l + e : 28 + 4 * l + e) : 8 * l + e;
        freq[k] = i < 8 * p.units ? p.freqs[i] : 0ull;
    }
    long long page = -1; // -1: outside the pool, its tokens are skipped
    int row = 0, token = -1, entry = -1; // entry: the block of the table that `page` is from
    bool skip = false;                 // nothing of this token is written
    uint64_t cs[4], sn[4], ns[4];      // cosines, sines and the sines' negatives, in pairs
    uint64_t weight[2][4] = {};
    int done = 0;

    while (done < left) {
        // ---- the token: position, page, angles ----
        if (at.t != token) {
            const int t = token = at.t;
            int pos = 0;
            skip = false;
            if constexpr (!CACHE) {
                pos = p.positions[t];
            } else {
                if (r < 0 || t >= behind) {
                    r = request_of(p.offsets, p.R, t);
                    entry = -1;
                    if (r >= 0) {
                        first = p.offsets[r];
                        behind = p.offsets[r + 1];
                        len = first < 0 || behind > p.T ? 0 : p.seq_lens[r]; // (no length: its tokens are skipped)
                    }
                }
                const int room = p.maxB * kPage; // at most 2^21
                skip = r < 0;                    // behind the last request's tokens: left as it is
                pos = (int)((unsigned)(len - 1) + ((unsigned)t - (unsigned)first));
                if (!skip && (len < 1 || len > room || pos >= room)) { // (nothing overflows behind the first two)
                    if (lane == 0)
                        set_error(p.err, kErrSeqLen);
                    skip = true;
                }
                if (!skip) {
                    row = pos % kPage;
                    if (pos / kPage != entry) { // (not the page of the token before)
                        entry = pos / kPage;
                        page = p.block_table[(size_t)r * p.maxB + entry];
                        if (page < 0 || page >= p.num_pages) {
                            if (lane == 0)
                                set_error(p.err, kErrPage);
                            page = -1;
                        }
                    }
                    skip = page < 0;
                }
            }
            if (p.units > 0) {
                float c2[2], s2[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int turn = (int)(unsigned)((freq[k] * (unsigned long long)(long long)pos) >> 32);
                    sincospif((float)turn * 4.656612873077393e-10f, &s2[k], &c2[k]); // 2^-31: half turns
                    s2[k] *= p.scale;
                    c2[k] *= p.scale;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float s0 = __shfl_sync(0xffffffffu, s2[0], 8 * e + l), s1 = __shfl_sync(0xffffffffu, s2[1], 8 * e + l);
                    cs[e] = pair(__shfl_sync(0xffffffffu, c2[0], 8 * e + l), __shfl_sync(0xffffffffu, c2[1], 8 * e + l));
                    sn[e] = pair(s0, s1);
                    ns[e] = pair(-s0, -s1);
                }
            }
        }

        // ---- the set's rows: where the lane's goes, and how far the next one is ----
        const RowSet &set = p.set[at.s];
        const int where = CACHE ? set.where : kToOut, heads = set.heads, end = done + min(at.n - at.g, left - done);
        const bool normed = set.weight != nullptr, rotated = set.rotated;
        const bool f4 = CACHE && set.bytes == kDim / 2, f8 = CACHE && set.bytes == kDim;
        int h = at.g * 4 + sub;
        const int stop = skip ? 0 : heads; // rows from here on are not written
        const long long block = where == kToOut ? at.t : page;
        const int in = where == kToOut ? 0 : row;
        uint8_t *dst = set.y + block * set.block_step + (unsigned)(h * set.head_step + in * set.bytes);
        uint8_t *dst_scales = set.scales + block * set.scales_block_step + (unsigned)(h * set.scales_head_step + in * (kDim / 16));
        const int step = 4 * set.head_step, step_scales = 4 * set.scales_head_step;
        const float scale = set.scale, inverse = set.inverse;
        const uint16_t *weights = set.weight;
        uint4 raw[2]; // the lane's norm weights: the set's, or of the head at hand, asked for before its row is
        auto ask_weights = [&](const uint16_t *w) {
            raw[0] = __ldg(reinterpret_cast<const uint4 *>(w + at0));
            raw[1] = __ldg(reinterpret_cast<const uint4 *>(w + at1));
        };
        auto take_weights = [&] {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                widen(raw[q], weight[q]);
                if (p.offset != 0.f)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        weight[q][k] = add2(weight[q][k], pair(p.offset, p.offset));
            }
        };
        const bool each_head = normed && p.per_head;
        if (normed && !each_head) {
            ask_weights(weights);
            take_weights();
        }

#pragma unroll 1
        for (; done < end; ++done, h += 4, dst += step, dst_scales += step_scales) {
            uint4 d[2];
            if (each_head)
                ask_weights(weights + (h < heads ? h * kDim : 0));
            ask();
            asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
            const uint32_t slot = mine + (done & (kSlots - 1)) * 1024;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(d[0].x), "=r"(d[0].y), "=r"(d[0].z), "=r"(d[0].w) : "r"(slot) : "memory");
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(d[1].x), "=r"(d[1].y), "=r"(d[1].z), "=r"(d[1].w) : "r"(slot + 512) : "memory");
            const bool real = h < stop;
            // rows without norm and rotation are copied bit by bit where they stay bf16
            if (!normed && !rotated && !f4 && !f8) {
                if (real) {
                    *reinterpret_cast<uint4 *>(dst + 2 * at0) = d[0];
                    *reinterpret_cast<uint4 *>(dst + 2 * at1) = d[1];
                }
                continue;
            }
            uint64_t v[2][4];
            widen(d[0], v[0]);
            widen(d[1], v[1]);
            if (normed) {
                if (each_head)
                    take_weights();
                uint64_t s2[2] = {0ull, 0ull};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s2[0] = fma2(v[0][k], v[0][k], s2[0]);
                    s2[1] = fma2(v[1][k], v[1][k], s2[1]);
                }
                float ss, s_odd;
                unpair(add2(s2[0], s2[1]), ss, s_odd);
                ss += s_odd;
#pragma unroll
                for (int o = 1; o < 8; o <<= 1)
                    ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float f = rsqrtf(fmaf(ss, 1.f / kDim, p.eps));
                const uint64_t f2 = pair(f, f);
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[q][k] = mul2(mul2(v[q][k], f2), weight[q][k]);
            }
            if (rotated) {
                if (!p.interleaved) {
                    if (turn0)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint64_t a = v[0][k], b = v[1][k];
                            v[0][k] = fma2(b, ns[k], mul2(a, cs[k]));
                            v[1][k] = fma2(a, sn[k], mul2(b, cs[k]));
                        }
                } else {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        if (q ? turn1 : turn0)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float a, b, c[2], z[2];
                                unpair(v[q][k], a, b);
                                unpair(cs[2 * q + (k >> 1)], c[0], c[1]);
                                unpair(sn[2 * q + (k >> 1)], z[0], z[1]);
                                v[q][k] = pair(a * c[k & 1] - b * z[k & 1], b * c[k & 1] + a * z[k & 1]);
                            }
                }
            }
            if (f4) {
                float y[2][8];
                unscale(v[0], scale, inverse, y[0]);
                unscale(v[1], scale, inverse, y[1]);
                store_nvfp4(y, m, real, dst, dst_scales);
            } else if (f8) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float y[8];
                    unscale(v[q], scale, inverse, y);
                    if (real)
                        *reinterpret_cast<uint2 *>(dst + (q ? at1 : at0)) = make_uint2(e4m3x4(y), e4m3x4(y + 4));
                }
            } else if (real) {
                *reinterpret_cast<uint4 *>(dst + 2 * at0) = narrow(v[0]);
                *reinterpret_cast<uint4 *>(dst + 2 * at1) = narrow(v[1]);
            }
        }
        // ---- the next set, or the next token ----
        at.g = 0;
        if (++at.s == p.sets) {
            at.s = 0;
            ++at.t;
        }
        at.n = (p.set[at.s].heads + 3) >> 2;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    check_offsets();
}

} // namespace

cudaError_t launch_append(const AppendParams &params, cudaStream_t stream)
{
    AppendParams p = params;
    if (p.T == 0 || p.groups == 0)
        return cudaSuccess;
    // Few groups: a warp for each, the latency of one.  Many: as many warps as the GPU holds at a time, with
    // runs of neighbouring groups, which share angles and places.
    const int sms = device_sms();
    if (sms < 1)
        return cudaErrorInvalidDevice;
    const long long all = (long long)p.T * p.groups, warps = (long long)sms * kCtas * kWarps;
    p.per_warp = (int)((all + warps - 1) / warps);
    long long blocks = (all + (long long)p.per_warp * kWarps - 1) / ((long long)p.per_warp * kWarps);
    const int checking = p.positions ? 0 : (p.R + 32 * kWarps - 1) / (32 * kWarps); // a thread looks at each request's offsets
    blocks = blocks < checking ? checking : blocks;
    const cudaError_t e = launch_kernel(p.positions ? append_kernel<false> : append_kernel<true>, dim3((unsigned)blocks), dim3(32 * kWarps), 0, stream, false, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace msa
