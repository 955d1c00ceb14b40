// gq_fp8.cuh -- 8-bit floating point in blocks of 128 (include/gq.h, gq_fp8_layout): exponents, codes, values.
//
// A block's scale is the power of two 2^(E - 127), E the smallest with which its largest value passes no code:
// 1.75 * 2^8 (E4M3) or 1.75 * 2^15 (E5M2) is the largest.  A power of two costs up to a bit of a block's range
// against max / 448, and in return scaling rounds nothing: c * 2^(E - 127) is exact in bf16 and binary32 (E >= 10
// keeps the smallest code above bf16's smallest value), products of two values are exact in binary32's
// exponent range, and the tensor cores take such scales as they are (their ue8m0 is this byte).
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "gq.h"

namespace gq {

constexpr int kBlock = 128;
constexpr uint32_t kInfBits = 0x7f800000u;

// Two values at a time: each operation rounds its two results alone.
typedef unsigned long long Two;
__device__ __forceinline__ Two two(float a, float b)
{
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void apart(Two x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ Two mul2(Two a, Two b)
{
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// E of a block whose largest |x| has these bits (a NaN's or infinity's bits give 255).
template <int FMT>
__device__ __forceinline__ uint32_t fp8_exp(uint32_t abs_bits)
{
    constexpr int top = FMT == GQ_FP8_E4M3 ? 8 : 15;
    // the exponent, one more above 1.75 of its power of two
    const int e = (int)((abs_bits + 0x1fffffu) >> 23) - top;
    return abs_bits >= kInfBits ? 255u : (uint32_t)max(e, 10);
}
// 2^(127 - E), the factor of a block's values before rounding (E = 255: anything finite).
__device__ __forceinline__ float fp8_inverse(uint32_t E) { return __uint_as_float((254u - min(E, 253u)) << 23); }
// 2^(E - 127) of a block that packing or a step wrote: infinity for E = 255, whose codes are NaN, and 0 for E = 0, whose
// codes are 0.
__device__ __forceinline__ float fp8_scale(uint32_t E) { return __uint_as_float(E << 23); }
// 2^(E - 127) of any block, whatever its codes; NaN for E = 255.  (AdamW's step takes the other one: with this one 64 tensors
// of 1e6, bf16 with masters, take 201 us, not 186.)
__device__ __forceinline__ float fp8_scale_any(uint32_t E)
{
    return __uint_as_float(E - 1u < 254u ? E << 23 : E == 0u ? 0x400000u : 0x7fffffffu);
}

// The codes of two values already scaled, a in the low byte: nearest, ties to even.
template <int FMT>
__device__ __forceinline__ uint32_t fp8_pair(float a, float b)
{
    uint16_t r;
    if constexpr (FMT == GQ_FP8_E4M3) asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    else asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// The codes of 8 values under E; a block with E = 255 has codes 0x7f.
template <int FMT>
__device__ __forceinline__ uint2 fp8_codes8(const float (&v)[8], uint32_t E)
{
    const float inv = fp8_inverse(E);
    const Two scale = two(inv, inv);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        apart(mul2(two(v[2 * i], v[2 * i + 1]), scale), a, b);
        q[i] = fp8_pair<FMT>(a, b);
    }
    if (E == 255u) return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}
// The values of two codes (low byte first), before the scale.
template <int FMT>
__device__ __forceinline__ float2 fp8_values(uint32_t two)
{
    uint32_t h;
    if constexpr (FMT == GQ_FP8_E4M3) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    else asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// 8 codes (two words) to values.
template <int FMT>
__device__ __forceinline__ void fp8_decode8(uint2 q, float scale, float (&v)[8])
{
    const uint32_t w[4] = {q.x & 0xffffu, q.x >> 16, q.y & 0xffffu, q.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = fp8_values<FMT>(w[i]);
        v[2 * i] = __fmul_rn(f.x, scale);
        v[2 * i + 1] = __fmul_rn(f.y, scale);
    }
}

}  // namespace gq
