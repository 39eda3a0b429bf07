// msa_append.cu -- norm and rotation of query and key rows, and new keys, values
// and index keys written into their pages, one pass over the rows.
//
// For a row x of 128 elements of the token at position p:
//   n = x rsqrt(mean x^2 + eps) (w + offset)            (rows with norm weights)
//   a' = s (a cos t - b sin t), b' = s (b cos t + a sin t)   for each pair (a, b) of
//   the first rotary_dim elements of n, t = 2 pi p f_i; the others stay.
// Everything is fp32 and rounded once, to bf16 or to the pool's format.  Angles
// are exact in 64-bit fixed point: f_i is a fraction of 2^64 of a turn, p f_i wraps
// around by itself, and what is left is a turn in [-1/2, 1/2) of 32 bits, off by
// 2^-32 of a turn and p 2^-65 whatever the position (in fp32 p f_i loses 2^-24 of
// itself, 0.06 rad at a million).
//
// Memory-bound: 256 bytes read and 256 (E4M3 128, NVFP4 72) written a row, latency
// where tokens are few.  A warp takes four heads of one token at a time, eight lanes
// a row; a lane holds two 16-byte pieces that rotate with one another, so that the
// rotation needs no exchange and the norm three shuffles.  The lane's eight angles
// are the same for all heads: computed once a warp, two by each row's lanes.
#include "msa_quant.cuh"
#include "msa_ragged.cuh"

namespace msa {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ void widen(uint4 d, float *v)
{
    const uint32_t e[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(e[k] << 16);
        v[2 * k + 1] = __uint_as_float(e[k] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 narrow(const float *v)
{
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
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
// (m = rotary_dim / 16, interleaved pairs: 8), the pieces behind them in twos.
__device__ __forceinline__ int piece(int l, int slot, int m)
{
    return l < m ? l + slot * m : 2 * l + slot;
}

// Eight floats by the scale s (inv: its reciprocal where that is exact).
__device__ __forceinline__ void unscale(float *v, float s, float inv)
{
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = inv != 0.f ? v[k] * inv : __fdiv_rn(v[k], s);
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
        const int owner = o < m ? o : o < 2 * m ? o - m : o >> 1, slot = o < m ? 0 : o < 2 * m ? 1 : o & 1;
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

__global__ void __launch_bounds__(32 * kWarps) append_kernel(const AppendParams p)
{
    const int lane = threadIdx.x & 31, l = lane & 7, sub = lane >> 3;
    const long long wi = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int t = (int)(wi / p.chunks), g0 = (int)(wi - (long long)t * p.chunks) * p.per_warp;
    if (t >= p.T)
        return;
    const int g1 = min(p.groups, g0 + p.per_warp);
    const int m = p.interleaved ? 8 : p.units;
    const int at0 = 8 * piece(l, 0, m), at1 = 8 * piece(l, 1, m);

    // a group of four rows: its set, this lane's head and the row's two pieces
    auto fetch = [&](int g, int &s, int &h, uint4 (&d)[2]) {
        s = 0;
#pragma unroll
        for (int k = 1; k < kMaxSets; ++k)
            s += k < p.sets && g >= p.set[k].group0;
        h = (g - p.set[s].group0) * 4 + sub;
        d[0] = d[1] = make_uint4(0u, 0u, 0u, 0u);
        if (h < p.set[s].heads) {
            const uint16_t *x = p.set[s].x + t * p.set[s].stride + (long long)h * kDim;
            d[0] = *reinterpret_cast<const uint4 *>(x + at0);
            d[1] = *reinterpret_cast<const uint4 *>(x + at1);
        }
    };
    int s, h;
    uint4 d[2];
    fetch(g0, s, h, d); // on its way while the token's place and angles are found

    // ---- the token: position, page, angles ----
    int pos;
    long long page = -1; // -1: nothing of this token goes to the cache
    int row = 0;
    if (p.positions) {
        pos = p.positions[t];
    } else {
        const int r = request_of(p.offsets, p.R, t);
        if (r < 0)
            return; // behind the last request's tokens: left as it is
        const int len = p.seq_lens[r];
        const long long at = (long long)len - 1 + (t - p.offsets[r]);
        if (len < 1 || at / kPage >= p.maxB) {
            if (lane == 0)
                set_error(p.err, kErrSeqLen);
            return;
        }
        pos = (int)at;
        row = pos % kPage;
        page = p.block_table[(size_t)r * p.maxB + pos / kPage];
        if (page < 0 || page >= p.num_pages) {
            if (lane == 0)
                set_error(p.err, kErrPage);
            page = -1;
        }
    }
    const int turned = 2 * p.units; // rotated pieces (interleaved), 2 units of 8 elements
    const bool turn0 = p.interleaved ? l < turned : l < m, turn1 = p.interleaved ? l + 8 < turned : turn0;
    float cs[8], sn[8];
    {
        float c2[2], s2[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int e = 2 * sub + k, i = p.interleaved ? (e < 4 ? 4 * l + e : 28 + 4 * l + e) : 8 * l + e;
            const unsigned long long f = i < 8 * p.units ? p.freqs[i] : 0ull;
            const int turn = (int)(unsigned)((f * (unsigned long long)(long long)pos) >> 32);
            sincospif((float)turn * 4.656612873077393e-10f, &s2[k], &c2[k]); // 2^-31: half turns
            s2[k] *= p.scale;
            c2[k] *= p.scale;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            cs[e] = __shfl_sync(0xffffffffu, c2[e & 1], (e >> 1) * 8 + l);
            sn[e] = __shfl_sync(0xffffffffu, s2[e & 1], (e >> 1) * 8 + l);
        }
    }

    for (int g = g0; g < g1; ++g) {
        int s_next = 0, h_next = 0;
        uint4 d_next[2] = {};
        if (g + 1 < g1)
            fetch(g + 1, s_next, h_next, d_next);
        const RowSet &set = p.set[s];
        const bool real = h < set.heads;
        float v[2][8];
        widen(d[0], v[0]);
        widen(d[1], v[1]);
        if (set.weight) {
            float ss = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                ss = fmaf(v[0][k], v[0][k], fmaf(v[1][k], v[1][k], ss));
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float f = rsqrtf(fmaf(ss, 1.f / kDim, p.eps));
            const uint16_t *w = set.weight + (p.per_head && real ? h * kDim : 0);
            float wv[8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                widen(*reinterpret_cast<const uint4 *>(w + (q ? at1 : at0)), wv);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[q][k] = v[q][k] * f * (wv[k] + p.offset);
            }
        }
        if (set.rotated) {
            if (!p.interleaved) {
                if (turn0)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float a = v[0][k], b = v[1][k];
                        v[0][k] = a * cs[k] - b * sn[k];
                        v[1][k] = b * cs[k] + a * sn[k];
                    }
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (q ? turn1 : turn0)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float a = v[q][2 * k], b = v[q][2 * k + 1], c = cs[4 * q + k], z = sn[4 * q + k];
                            v[q][2 * k] = a * c - b * z;
                            v[q][2 * k + 1] = b * c + a * z;
                        }
            }
        }
        // rows without norm and rotation are copied bit by bit where they stay bf16
        const bool plain = !set.weight && !set.rotated;
        const uint4 b0 = plain ? d[0] : narrow(v[0]), b1 = plain ? d[1] : narrow(v[1]);
        if (set.where == kToOut) {
            if (real) {
                uint16_t *y = set.y + ((size_t)t * set.heads + h) * kDim;
                *reinterpret_cast<uint4 *>(y + at0) = b0;
                *reinterpret_cast<uint4 *>(y + at1) = b1;
            }
        } else if (page >= 0) {
            const bool index = set.where == kToIndex;
            const size_t head = index ? (size_t)page * p.Hi + h : ((size_t)page * 2 + (set.where == kToV)) * p.Hkv + h;
            const size_t prow = head * kPage + row;
            if (index ? p.idx_f4 : p.kv_fmt == kFmtF4) {
                if (index) {
                    store_nvfp4(v, m, real, p.idxk + prow * (kDim / 2), p.idxk_scales + prow * (kDim / 16));
                } else {
                    const float sc = set.where == kToV ? p.v_scale : p.k_scale, inv = set.where == kToV ? p.v_inv : p.k_inv;
                    unscale(v[0], sc, inv);
                    unscale(v[1], sc, inv);
                    uint8_t *tile = p.kv + head * kF4KvTile;
                    store_nvfp4(v, m, real, tile + row * (kDim / 2), tile + kPage * (kDim / 2) + row * (kDim / 16));
                }
            } else if (!index && p.kv_fmt == kFmtFp8) {
                const float sc = set.where == kToV ? p.v_scale : p.k_scale, inv = set.where == kToV ? p.v_inv : p.k_inv;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    unscale(v[q], sc, inv);
                    const uint2 c = make_uint2(e4m3x2_rn_sat(v[q][1], v[q][0]) | e4m3x2_rn_sat(v[q][3], v[q][2]) << 16,
                                               e4m3x2_rn_sat(v[q][5], v[q][4]) | e4m3x2_rn_sat(v[q][7], v[q][6]) << 16);
                    if (real)
                        *reinterpret_cast<uint2 *>(p.kv + prow * kDim + (q ? at1 : at0)) = c;
                }
            } else if (real) {
                uint8_t *at = (index ? p.idxk : p.kv) + prow * (2 * kDim);
                *reinterpret_cast<uint4 *>(at + 2 * at0) = b0;
                *reinterpret_cast<uint4 *>(at + 2 * at1) = b1;
            }
        }
        s = s_next, h = h_next;
        d[0] = d_next[0], d[1] = d_next[1];
    }
}

} // namespace

cudaError_t launch_append(const AppendParams &params, cudaStream_t stream)
{
    AppendParams p = params;
    if (p.T == 0 || p.groups == 0)
        return cudaSuccess;
    // Few tokens: a warp for each group, the latency of one.  Many: up to eight groups
    // a warp, which share its angles and its place.
    const long long all = (long long)p.T * p.groups;
    const int per = (int)(all / (152 * 48) < 1 ? 1 : all / (152 * 48) > 8 ? 8 : all / (152 * 48));
    p.chunks = (p.groups + per - 1) / per;
    p.per_warp = (p.groups + p.chunks - 1) / p.chunks;
    const long long blocks = ((long long)p.T * p.chunks + kWarps - 1) / kWarps;
    if (blocks > 0x7FFFFFFFll)
        return cudaErrorInvalidValue;
    const cudaError_t e = launch_kernel(append_kernel, dim3((unsigned)blocks), dim3(32 * kWarps), 0, stream, false, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace msa
