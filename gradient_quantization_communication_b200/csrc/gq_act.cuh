// gq_act.cuh -- the 8-bit activation checkpoint's format, and the chunks of 256 columns that a warp
// loads, stores, encodes and decodes.
//
// Format (include/gq.h, gq_act_layout).  A group is 32 consecutive columns of a row.  With
// m = max |x| of the group, e is the smallest integer that keeps |rint(x * 2^-e)| <= 127 for all of
// its values, so m * 2^-e lies in [63.75, 127.5): between 6 and 7 bits and a sign are kept of the
// largest value.  The exponent byte is E = e + 133: m's biased binary32 exponent after m's mantissa
// was rounded up from 127.5/128.  Because the scale is a power of two, q * 2^e has at most 7
// significant bits: bf16 and binary32 hold every decoded value exactly, down to E = 0 (2^-133 is
// bf16's smallest subnormal), and the products that read a checkpoint round nothing of it.
// E = 255 marks a group with a NaN or an infinity; it decodes to NaN.  The largest finite groups
// (E would be 255) keep E = 254 and saturate their codes at 127.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace gq {

constexpr int kChunk = 256;  // columns of a row that one warp handles at a time: 8 per lane

// ---------------------------------------------------------------------------------------------
// A lane's 8 elements, as loaded.
// VEC: columns base + 8 * lane + j, 16-byte accesses (row starts 16-byte aligned).
// else: columns base + 32 * j + lane, one element per access (any row start).
// ---------------------------------------------------------------------------------------------
template <typename T>
struct Raw {
    uint32_t w[2 * sizeof(T)];
};

__device__ __forceinline__ uint32_t elem_bits(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t elem_bits(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }
__device__ __forceinline__ uint32_t elem_bits(__half x) { return __half_as_ushort(x); }

template <typename T>
__device__ __forceinline__ void raw_set(Raw<T> &r, int j, uint32_t bits)
{
    if constexpr (sizeof(T) == 4) {
        r.w[j] = bits;
    } else {
        if (j & 1) r.w[j >> 1] |= bits << 16;
        else r.w[j >> 1] = bits;
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void chunk_load(Raw<T> &r, const T *row, int base, int lane, int cols)
{
    if constexpr (VEC) {
        const int c0 = base + lane * 8;
        if (c0 + 8 <= cols) {
            const uint4 *p = reinterpret_cast<const uint4 *>(row + c0);
            const uint4 a = __ldg(p);
            r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
            if constexpr (sizeof(T) == 4) {
                const uint4 b = __ldg(p + 1);
                r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) raw_set(r, j, c0 + j < cols ? elem_bits(row[c0 + j]) : 0u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = base + j * 32 + lane;
            raw_set(r, j, c < cols ? elem_bits(row[c]) : 0u);
        }
    }
}

__device__ __forceinline__ void to_floats(const Raw<float> &r, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r.w[j]);
}
__device__ __forceinline__ void to_floats(const Raw<__nv_bfloat16> &r, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(r.w[j] << 16);
        v[2 * j + 1] = __uint_as_float(r.w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void to_floats(const Raw<__half> &r, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2 h = *reinterpret_cast<const __half2 *>(&r.w[j]);
        const float2 f = __half22float2(h);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
    }
}

__device__ __forceinline__ void from_floats(Raw<float> &r, const float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) r.w[j] = __float_as_uint(v[j]);
}
__device__ __forceinline__ void from_floats(Raw<__nv_bfloat16> &r, const float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        r.w[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
}
__device__ __forceinline__ void from_floats(Raw<__half> &r, const float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        r.w[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <typename T>
__device__ __forceinline__ T raw_get(const Raw<T> &r, int j)
{
    if constexpr (sizeof(T) == 4) {
        return __uint_as_float(r.w[j]);
    } else {
        const unsigned short h = (unsigned short)((j & 1) ? r.w[j >> 1] >> 16 : r.w[j >> 1] & 0xffffu);
        if constexpr (sizeof(T) == 2 && __is_same(T, __half)) return __ushort_as_half(h);
        else return __ushort_as_bfloat16(h);
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void chunk_store(const Raw<T> &r, T *row, int base, int lane, int cols)
{
    if constexpr (VEC) {
        const int c0 = base + lane * 8;
        if (c0 + 8 <= cols) {
            uint4 *p = reinterpret_cast<uint4 *>(row + c0);
            p[0] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
            if constexpr (sizeof(T) == 4) p[1] = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + j < cols) row[c0 + j] = raw_get(r, j);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = base + j * 32 + lane;
            if (c < cols) row[c] = raw_get(r, j);
        }
    }
}

// Column of a lane's element j.
template <bool VEC>
__device__ __forceinline__ int chunk_col(int base, int lane, int j)
{
    return VEC ? base + lane * 8 + j : base + j * 32 + lane;
}

// ---------------------------------------------------------------------------------------------
// The checkpoint
// ---------------------------------------------------------------------------------------------
struct Ckpt {
    uint8_t *codes;      // rows of code_pitch bytes
    uint8_t *exps;       // rows of exp_pitch bytes
    int code_pitch;      // columns rounded up to whole groups
    int exp_pitch;       // groups rounded up to four
};

// E of a group whose largest |x| has these bits (a NaN's or infinity's bits give 255).
__device__ __forceinline__ uint32_t group_exp(uint32_t abs_bits)
{
    const uint32_t e = min((abs_bits + 0x10000u) >> 23, 254u);
    return abs_bits >= 0x7f800000u ? 255u : e;
}

// The code of v as a byte in a word's low 8 bits (other bits undefined).  fma(v, 2^-e, 1.5 * 2^23)
// leaves rint(v * 2^-e), ties to even, in two's complement in the low mantissa bits; v * 2^-e is exact.
// Outside 6 <= E <= 253 the scale leaves binary32's range or the code may pass 127: see group_code_slow.
__device__ __forceinline__ uint32_t group_code(float v, float inv)
{
    return __float_as_uint(__fmaf_rn(v, inv, 12582912.0f));
}
__device__ __forceinline__ bool group_is_slow(uint32_t E) { return E - 6u > 247u; }
__device__ __forceinline__ float group_inv(uint32_t E) { return __uint_as_float((260u - E) << 23); }
static __device__ __noinline__ uint32_t group_code_slow(float v, uint32_t E)
{
    if (E == 255u) return 0u;
    float t;
    if (E >= 6u) t = __fmul_rn(v, __uint_as_float((260u - E) << 23));
    else t = __fmul_rn(__fmul_rn(v, __uint_as_float(254u << 23)), __uint_as_float((133u - E) << 23));
    t = fminf(fmaxf(t, -127.0f), 127.0f);
    return __float_as_uint(__fadd_rn(t, 12582912.0f));
}

// 2^(E - 133), NaN for E = 255.
__device__ __forceinline__ float group_scale(uint32_t E)
{
    const uint32_t b = E > 6u ? (E - 6u) << 23 : 0x00400000u >> (6u - E);
    return __uint_as_float(E == 255u ? 0x7fffffffu : b);
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Encode a lane's 8 values (0 past the last column) of a chunk; every lane of the warp calls it.
template <bool VEC>
__device__ __forceinline__ void ckpt_store(const float (&v)[8], const Ckpt &k, int64_t row, int base, int lane)
{
    uint8_t *codes = k.codes + row * k.code_pitch;
    uint8_t *exps = k.exps + row * k.exp_pitch;
    if constexpr (VEC) {
        float m = fabsf(v[0]);
#pragma unroll
        for (int j = 1; j < 8; ++j) m = max_nan(m, fabsf(v[j]));
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t E = group_exp(__float_as_uint(m) & 0x7fffffffu);
        uint32_t q[8];
        if (!group_is_slow(E)) {
            const float inv = group_inv(E);
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = group_code(v[j], inv);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = group_code_slow(v[j], E);
        }
        const int c0 = base + lane * 8;
        if (c0 < k.code_pitch)
            *reinterpret_cast<uint2 *>(codes + c0) =
                make_uint2(pack_bytes(q[0], q[1], q[2], q[3]), pack_bytes(q[4], q[5], q[6], q[7]));
        if ((lane & 3) == 0 && (c0 >> 5) < k.exp_pitch) exps[c0 >> 5] = (uint8_t)E;
    } else {
        uint32_t mine = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(v[j]) & 0x7fffffffu);
            const uint32_t E = group_exp(m);
            const uint32_t q = group_is_slow(E) ? group_code_slow(v[j], E) : group_code(v[j], group_inv(E));
            const int c = base + j * 32 + lane;
            if (c < k.code_pitch) codes[c] = (uint8_t)q;
            if (lane == j) mine = E;
        }
        if (lane < 8 && (base >> 5) + lane < k.exp_pitch) exps[(base >> 5) + lane] = (uint8_t)mine;
    }
}

// A lane's codes and exponents of a chunk, as loaded.
template <bool VEC>
struct RawCkpt {
    uint32_t q[2];
    uint32_t e[VEC ? 1 : 8];
};

template <bool VEC>
__device__ __forceinline__ void ckpt_load(RawCkpt<VEC> &r, const Ckpt &k, int64_t row, int base, int lane)
{
    const uint8_t *codes = k.codes + row * k.code_pitch;
    const uint8_t *exps = k.exps + row * k.exp_pitch;
    if constexpr (VEC) {
        const int c0 = base + lane * 8;
        r.q[0] = r.q[1] = r.e[0] = 0;
        if (c0 < k.code_pitch) {
            const uint2 a = __ldg(reinterpret_cast<const uint2 *>(codes + c0));
            r.q[0] = a.x;
            r.q[1] = a.y;
            r.e[0] = __ldg(exps + (c0 >> 5));
        }
    } else {
        r.q[0] = r.q[1] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = base + j * 32 + lane;
            const bool in = c < k.code_pitch;
            r.q[j >> 2] |= (in ? (uint32_t)__ldg(codes + c) : 0u) << (8 * (j & 3));
            r.e[j] = in ? __ldg(exps + (c >> 5)) : 0u;
        }
    }
}

template <bool VEC>
__device__ __forceinline__ void ckpt_floats(const RawCkpt<VEC> &r, float (&v)[8])
{
    const uint32_t a = r.q[0] ^ 0x80808080u, b = r.q[1] ^ 0x80808080u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        // 2^23 + (q + 128), then the exact integer q, then its exact product with the scale
        const float f = __uint_as_float(__byte_perm(j < 4 ? a : b, 0x4B000000u, 0x7440 | (j & 3)));
        v[j] = __fmul_rn(__fsub_rn(f, 8388736.0f), group_scale(r.e[VEC ? 0 : j]));
    }
}

// Largest finite binary16: decoded values saturate there (a group's largest value may round up to 65536).
template <typename T>
__device__ __forceinline__ void saturate(float (&v)[8])
{
    if constexpr (__is_same(T, __half)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // NaN stays NaN
            v[j] = v[j] > 65504.0f ? 65504.0f : v[j] < -65504.0f ? -65504.0f : v[j];
        }
    }
}

}  // namespace gq
