// msa_umma.cuh -- tcgen05 issue helpers, tensor-memory loads and stores, packed
// fp32 arithmetic and the per-CTA walk shared by the whole-cache kernels.
#pragma once

#include "msa_cache.cuh"

#ifdef __CUDACC__

namespace msa {

// The MMAs below are executed by a whole warp and issued by the lane with `one`
// set.  Their operands live in uniform registers: a value the compiler cannot
// prove uniform costs moves before every MMA (about 100 clocks an MMA, where the
// tensor cores need 64).  A reduction over the warp gives a value that it can.
__device__ __forceinline__ uint32_t uniform(uint32_t v)
{
    return __reduce_or_sync(0xffffffffu, v);
}

// 1 in one lane of the warp, the same at every call.  (A commit in a branch on it takes 22 clocks,
// 52 in a branch on lane == 0.)
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one;
}

// A box of a 3-D tensor map into shared memory.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// Shared-memory operand descriptor (128-byte swizzle, version 1) from its low
// word: address / 16 and the leading offset / 16 in bits 16 ..; stride 1024.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;

__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lead)
{
    return ((addr >> 4) & 0x3FFFu) | (lead >> 4) << 16;
}

// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void umma_ss(uint32_t one, uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n .reg .pred p, q;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
                 " mov.b64 a, {%1, %6};\n mov.b64 b, {%2, %6};\n"
                 " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
                 "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(one), "r"(kDescHigh)
                 : "memory");
}

// The same with 8-bit operands.
__device__ __forceinline__ void umma_ss8(uint32_t one, uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n .reg .pred p, q;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
                 " mov.b64 a, {%1, %6};\n mov.b64 b, {%2, %6};\n"
                 " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n}\n" ::"r"(d),
                 "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(one), "r"(kDescHigh)
                 : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void umma_ts(uint32_t one, uint32_t d, uint32_t a, uint32_t b_low, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n .reg .pred p, q;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
                 " mov.b64 b, {%2, %6};\n"
                 " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
                 "r"(a), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(one), "r"(kDescHigh)
                 : "memory");
}

// 32 consecutive TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
          "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a));
}

// Wait for the loads issued so far; r (the registers of one of them) is read
// and written here so that no use of its values can move before the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t *r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// 16 columns, and the wait for them, in the same way.
__device__ __forceinline__ void tmem_ld_async(uint32_t a, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(a));
}

__device__ __forceinline__ void tmem_wait_async(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(a)
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
        "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(a)
        : "memory");
}

// Two fp32 at a time (the packed forms issue once for both).
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ void unpair(uint64_t v, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Two floats to E4M3 (round to nearest, saturating): a -> low byte, b -> high byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b)
{
    uint32_t out;
    asm("{\n .reg .b16 t;\n cvt.rn.satfinite.e4m3x2.f32 t, %2, %1;\n cvt.u32.u16 %0, t;\n}\n"
        : "=r"(out)
        : "f"(a), "f"(b));
    return out;
}

// Query rows 0 .. n - 1 (bf16, `row(i)` in global memory) into an operand tile in
// shared memory, K-major with the 128-byte swizzle, by warp `wi` of `nw`: half a
// warp takes a row, 16 bytes a lane, so that loads are whole lines and several rows
// are in flight.
//   kRows16   bf16 as they are (half of the dimensions `half` bytes after the other)
//   kRowsF16  f16: each row scaled by a power of two that brings its largest element to
//             [2^8, 2^9) (exact; elements 2^-23 below it lose bits)
//   kRowsPair E4M3 pairs hi, 16 lo in rows 2 i, 2 i + 1 (lo = what rounding to hi left, at
//             most 16 itself), after a power of two that brings the row's largest element
//             to (224, 448]
// inverse(i, x) is told the factor that undoes the scaling (one lane of the row).
constexpr int kRows16 = 0, kRowsF16 = 1, kRowsPair = 2;

template <int MODE, typename Row, typename Inverse>
__device__ __forceinline__ void stage_rows(uint8_t *dst, int half, int n, int wi, int nw, Row &&row, Inverse &&inverse)
{
    constexpr int U = 4;
    const int lane = threadIdx.x & 31, c = lane & 15;
    if constexpr (MODE == kRows16) { // nothing passes through registers: all rows in flight at once
        for (int i = 2 * wi + (lane >> 4); i < n; i += 2 * nw)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst + (c >> 3) * half + 128 * i + (((c & 7) ^ (i & 7)) << 4))),
                         "l"(reinterpret_cast<const uint4 *>(row(i)) + c)
                         : "memory");
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        for (int i0 = 2 * wi; i0 < n; i0 += 2 * U * nw) {
            uint4 d[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + 2 * u * nw + (lane >> 4);
                d[u] = make_uint4(0u, 0u, 0u, 0u);
                if (i < n)
                    d[u] = reinterpret_cast<const uint4 *>(row(i))[c];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + 2 * u * nw + (lane >> 4);
                uint32_t *e = &d[u].x;
                float mx = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(e[k] << 16)), fabsf(__uint_as_float(e[k] & 0xFFFF0000u))));
#pragma unroll
                for (int o = 1; o < 16; o <<= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                // the exponent clamped so that neither factor overflows
                int x = (int)(__float_as_uint(mx) >> 23) - 127;
                x = x < -100 ? -100 : x > 127 ? 127 : x;
                float up = __uint_as_float((uint32_t)(8 - x + 127) << 23), inv = __uint_as_float((uint32_t)(x - 8 + 127) << 23);
                if (MODE == kRowsPair && mx * up > 448.f) // E4M3's largest
                    up *= 0.5f, inv *= 2.f;
                if (c == 0 && i < n)
                    inverse(i, inv);
                if (MODE == kRowsPair) {
                    uint32_t hi[2] = {0u, 0u}, lo[2] = {0u, 0u};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float a = __uint_as_float(e[k] << 16) * up, b = __uint_as_float(e[k] & 0xFFFF0000u) * up;
                        const uint32_t h = to_e4m3x2(a, b);
                        float ha, hb;
                        f16x2_to_f32x2(e4m3x2_to_f16x2(h), ha, hb);
                        hi[k >> 1] |= h << (16 * (k & 1));
                        lo[k >> 1] |= to_e4m3x2(16.f * (a - ha), 16.f * (b - hb)) << (16 * (k & 1));
                    }
                    if (i < n) {
                        uint8_t *at = dst + 256 * i + (c & 1) * 8;
                        *reinterpret_cast<uint2 *>(at + (((c >> 1) ^ ((2 * i) & 7)) << 4)) = make_uint2(hi[0], hi[1]);
                        *reinterpret_cast<uint2 *>(at + 128 + (((c >> 1) ^ ((2 * i + 1) & 7)) << 4)) = make_uint2(lo[0], lo[1]);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        e[k] = pack_f16(__uint_as_float(e[k] << 16) * up, __uint_as_float(e[k] & 0xFFFF0000u) * up);
                }
                if (MODE != kRowsPair && i < n)
                    *reinterpret_cast<uint4 *>(dst + (c >> 3) * half + 128 * i + (((c & 7) ^ (i & 7)) << 4)) = d[u];
            }
        }
    }
}

// One row of an NVFP4 tile as the TMA lands it, widened to f16 in the layout of a
// 16-bit tile (two halves of 64 dimensions, 128-byte swizzle).
__device__ __forceinline__ void widen_row(const uint8_t *src, uint8_t *tile, int row)
{
    uint8_t *dst = tile + row * 128;
    const uint64_t sc = *reinterpret_cast<const uint64_t *>(src + 8192 + row * 8);
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

// Row `row` of a ring tile (E4M3, NVFP4) to f16 in the layout of a 16-bit tile; dst is the row's place in its
// first half.  On a last page (tail) a row that is not cached becomes zeros (drop), and infinities
// and NaN of a row that only later tokens see (check) do too: true is returned for those.
// AHEAD: 16-byte pieces that are loaded before any of them is stored (the compiler moves no load past a store).
template <int FMT, int UNROLL = 2, int AHEAD = 1>
__device__ __forceinline__ bool convert_row(const uint8_t *src, uint8_t *dst, int row, bool tail, bool drop, bool check)
{
    bool bad = false;
    if (FMT == kFmtFp8) {
#pragma unroll UNROLL // (dense decode, all: 426 us for 413, 48 tokens over 2 x 131072; NVFP4 loses with less, 507 for 488)
        for (int c0 = 0; c0 < 8; c0 += AHEAD) { // 16 dimensions each
            uint4 d[AHEAD];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                d[u] = *reinterpret_cast<const uint4 *>(src + row * 128 + (((c0 + u) ^ (row & 7)) << 4));
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int c = c0 + u;
                uint32_t e[4] = {d[u].x, d[u].y, d[u].z, d[u].w}, o[8];
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
        uint4 d[4];
#pragma unroll
        for (int c = 0; AHEAD > 1 && c < 4; ++c)
            d[c] = *reinterpret_cast<const uint4 *>(src + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
#pragma unroll
        for (int c = 0; c < 4; ++c) { // 32 dimensions, two scales
            if (AHEAD == 1)
                d[c] = *reinterpret_cast<const uint4 *>(src + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
            const uint32_t e[4] = {d[c].x, d[c].y, d[c].z, d[c].w};
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
    return bad;
}

// The share of a CTA, unit by unit.  Every role walks it alike.
struct Walk {
    int x, x1, r, u, b, nb, seq_len, seg;
    __device__ __forceinline__ int pages() const { return min(nb - b, x1 - x); }
    __device__ __forceinline__ void next(const CacheParams &p, int heads)
    {
        x += pages();
        ++seg;
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
};

} // namespace msa

#endif // __CUDACC__
