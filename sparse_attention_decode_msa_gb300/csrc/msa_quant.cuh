// msa_quant.cuh -- the roundings with which new rows enter E4M3 and NVFP4 pools,
// shared by the calls that write them.
#pragma once

#include "msa_internal.cuh"

#ifdef __CUDACC__

namespace msa {

// Two floats to E4M3 codes (round to nearest even, saturating): a -> high
// byte, b -> low byte; a zero result is +0.
__device__ __forceinline__ uint32_t e4m3x2_rn_sat(float a, float b)
{
    uint32_t out;
    asm("{\n .reg .b16 t;\n cvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n cvt.u32.u16 %0, t;\n}\n"
        : "=r"(out)
        : "f"(a), "f"(b));
    if ((out & 0x7Fu) == 0)
        out &= ~0x80u;
    if ((out & 0x7F00u) == 0)
        out &= ~0x8000u;
    return out;
}

// Four floats to e2m1 codes (round to nearest even, saturating) packed in 16
// bits, x0 in the lowest nibble; a zero result is +0.
__device__ __forceinline__ uint32_t e2m1x4_rn_sat(float x0, float x1, float x2, float x3)
{
    uint32_t out;
    asm("{\n .reg .b8 b0, b1, b2, b3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b2, 0f00000000, 0f00000000;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b3, 0f00000000, 0f00000000;\n"
        " mov.b32 %0, {b0, b1, b2, b3};\n}\n"
        : "=r"(out)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (((out >> (4 * i)) & 7u) == 0)
            out &= ~(8u << (4 * i));
    return out;
}

constexpr int kF4KvTile = kPage * kDim / 2 + kPage * kDim / 16; // NVFP4 K or V tile

} // namespace msa

#endif // __CUDACC__
