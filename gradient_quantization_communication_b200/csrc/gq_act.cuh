// gq_act.cuh -- the 8-bit activation checkpoint's format, and the chunks of 256 columns that a warp
// loads, stores, encodes and decodes.
//
// Format (include/gq.h, gq_act_layout).  A group is 32 consecutive columns of a row.  With
// m = max |x| of the group, e is the smallest integer that keeps |rint(x * 2^-e)| <= 127 for all of
// its values, so m * 2^-e lies in [63.75, 127.5): between 6 and 7 bits and a sign are kept of the
// largest value.  The exponent byte is E = e + 133: m's biased binary32 exponent, one more where m is
// at least 127.5/128 of the next power of two, and at least 0.  Because the scale is a power of two,
// q * 2^e has at most 7 significant bits: bf16 and binary32 hold every decoded value exactly, down to
// E = 0 (2^-133 is bf16's smallest subnormal), and the products that read a checkpoint round nothing
// of it.
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
// A lane's 8 elements, columns base + 8 * lane + j of a row, as loaded.
// AL: every row starts on 16 bytes, and the 8 elements are one or two 16-byte accesses.
// else: rows start anywhere (on their element size).  A lane loads the aligned 16-byte pieces its elements
// lie in and shifts them into place when it uses them; a store shifts its elements, with the next lane's
// first ones behind them, onto aligned pieces.  Loading element by element took twice as long.
// ---------------------------------------------------------------------------------------------
template <typename T>
struct Words {
    uint32_t w[2 * sizeof(T)];  // the 8 elements
};
template <typename T, bool AL>
struct Raw {
    uint32_t w[2 * sizeof(T) + (AL ? 0 : 4)];
};

__device__ __forceinline__ uint32_t elem_bits(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t elem_bits(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }
__device__ __forceinline__ uint32_t elem_bits(__half x) { return __half_as_ushort(x); }

// Element j of an array of words.
template <typename T>
__device__ __forceinline__ void elem_set(uint32_t *w, int j, uint32_t bits)
{
    if constexpr (sizeof(T) == 4) {
        w[j] = bits;
    } else {
        if (j & 1) w[j >> 1] |= bits << 16;
        else w[j >> 1] = bits;
    }
}
template <typename T>
__device__ __forceinline__ T elem_get(const uint32_t *w, int j)
{
    if constexpr (sizeof(T) == 4) {
        return __uint_as_float(w[j]);
    } else {
        const unsigned short h = (unsigned short)((j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu);
        if constexpr (__is_same(T, __half)) return __ushort_as_half(h);
        else return __ushort_as_bfloat16(h);
    }
}

// Bytes by which a row's start lies past a 16-byte boundary.
template <typename T>
__device__ __forceinline__ uint32_t row_shift(const T *row)
{
    return (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
}

// The 16-byte pieces from `from` bytes past the start of w: out[i] = w[i + from / 4], shifted by from % 4.
template <int N>
__device__ __forceinline__ void shift_words(const uint32_t (&in)[N + 4], uint32_t from, uint32_t (&out)[N])
{
    uint32_t t[N + 4];
#pragma unroll
    for (int i = 0; i < N + 4; ++i) t[i] = in[i];
    if (from & 8u) {
#pragma unroll
        for (int i = 0; i < N + 2; ++i) t[i] = t[i + 2];
    }
    if (from & 4u) {
#pragma unroll
        for (int i = 0; i < N + 1; ++i) t[i] = t[i + 1];
    }
    const uint32_t bits = (from & 3u) * 8u;
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = __funnelshift_r(t[i], t[i + 1], bits);
}

// Eight words at once, to a 32-byte boundary: two stores of 16 bytes write each sector in halves (unpacking
// 8192 x 4096 to float32 took 44 us with them, 33 us so).
template <typename W>
__device__ __forceinline__ void store32(void *p, const W &w)
{
    if constexpr (sizeof(w) >= 32)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
}

// KEPT: nothing writes the memory while the kernel runs, so that the read-only path may be taken.
template <bool KEPT>
__device__ __forceinline__ uint4 load16(const void *p)
{
    if constexpr (KEPT) return __ldg(reinterpret_cast<const uint4 *>(p));
    else return *reinterpret_cast<const uint4 *>(p);
}

// FULL: all lanes' 16-byte pieces lie inside the row (inner_chunk).
template <typename T, bool AL, bool FULL = false, bool KEPT = true>
__device__ __forceinline__ void chunk_load(Raw<T, AL> &r, const T *row, int base, int lane, int cols)
{
    const int c0 = base + lane * 8;
    if constexpr (AL) {
        if (FULL || c0 + 8 <= cols) {
            const uint4 a = load16<KEPT>(row + c0);
            r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
            if constexpr (sizeof(T) == 4) {
                const uint4 b = load16<KEPT>(row + c0 + 4);
                r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) elem_set<T>(r.w, j, c0 + j < cols ? elem_bits(row[c0 + j]) : 0u);
        }
    } else {
        // only bytes of the row are read: a piece that reaches over its start or end is put together
        constexpr int P = sizeof(T) == 4 ? 3 : 2, E = 16 / sizeof(T);
        const int first = c0 - (int)(row_shift(row) / sizeof(T));  // column of the first piece's first element
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = first + i * E;
            if (FULL || (c >= 0 && c + E <= cols)) {
                const uint4 a = load16<KEPT>(row + c);
                r.w[4 * i] = a.x; r.w[4 * i + 1] = a.y; r.w[4 * i + 2] = a.z; r.w[4 * i + 3] = a.w;
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j)
                    elem_set<T>(r.w + 4 * i, j, c + j >= 0 && c + j < cols ? elem_bits(row[c + j]) : 0u);
            }
        }
    }
}

// Whether all pieces of the chunk at column base lie inside the row: then nothing is checked lane by lane.
// Unaligned rows need up to 8 columns more on either side.
template <typename T, bool AL>
__device__ __forceinline__ bool inner_chunk(int base, int cols)
{
    return AL ? base + kChunk <= cols : base > 0 && base + kChunk + 8 <= cols;
}

// The loaded elements in place.
template <typename T, bool AL>
__device__ __forceinline__ Words<T> in_place(const Raw<T, AL> &r, const T *row)
{
    Words<T> o;
    if constexpr (AL) {
#pragma unroll
        for (int i = 0; i < (int)(2 * sizeof(T)); ++i) o.w[i] = r.w[i];
    } else {
        shift_words<2 * sizeof(T)>(r.w, row_shift(row), o.w);
    }
    return o;
}

__device__ __forceinline__ void to_floats(const Words<float> &r, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r.w[j]);
}
__device__ __forceinline__ void to_floats(const Words<__nv_bfloat16> &r, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(r.w[j] << 16);
        v[2 * j + 1] = __uint_as_float(r.w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void to_floats(const Words<__half> &r, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2 h = *reinterpret_cast<const __half2 *>(&r.w[j]);
        const float2 f = __half22float2(h);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
    }
}

__device__ __forceinline__ void from_floats(Words<float> &r, const float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) r.w[j] = __float_as_uint(v[j]);
}
__device__ __forceinline__ void from_floats(Words<__nv_bfloat16> &r, const float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        r.w[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
}
__device__ __forceinline__ void from_floats(Words<__half> &r, const float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        r.w[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Every lane of the warp calls it.
template <typename T, bool AL, bool FULL = false>
__device__ __forceinline__ void chunk_store(const Words<T> &r, T *row, int base, int lane, int cols)
{
    constexpr int W = 2 * sizeof(T);
    const int c0 = base + lane * 8;
    const uint32_t shift = AL ? 0u : row_shift(row);
    if (AL || shift == 0u) {
        if (FULL || c0 + 8 <= cols) {
            uint4 *p = reinterpret_cast<uint4 *>(row + c0);
            if (sizeof(T) == 4 && (reinterpret_cast<uintptr_t>(row) & 31u) == 0) {
                store32(p, r.w);
            } else {
                p[0] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
                if constexpr (sizeof(T) == 4) p[1] = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + j < cols) row[c0 + j] = elem_get<T>(r.w, j);
        }
        return;
    }
    // a lane's pieces start `head` elements into its own and end `head` elements into the next lane's
    const int head = (int)((16u - shift) / sizeof(T));
    uint32_t w[W + 4], o[W];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = r.w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[W + i] = __shfl_down_sync(0xffffffffu, r.w[i], 1);
    shift_words<W>(w, 16u - shift, o);
    const bool whole = lane < 31 && (FULL || c0 + head + 8 <= cols);
    if (whole) {
        uint4 *p = reinterpret_cast<uint4 *>(row + c0 + head);
        p[0] = make_uint4(o[0], o[1], o[2], o[3]);
        if constexpr (sizeof(T) == 4) p[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
    // elements no piece covers: the first lane's head, and the last lanes' rest
    const bool own_head = lane == 0 || (!FULL && c0 + head > cols);
    if (own_head || !whole) {
        const uint32_t heads = (1u << head) - 1u;
        uint32_t mine = (own_head ? heads : 0u) | (whole ? 0u : ~heads);
        if (!FULL) mine &= (1u << min(max(cols - c0, 0), 8)) - 1u;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (mine & 1u << j) row[c0 + j] = elem_get<T>(r.w, j);
    }
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
    // the border is 127.5 of the scale: of a subnormal's last place 2^-149, 127.5 * 2^16
    const uint32_t up = abs_bits < 0x00800000u ? 0x8000u : 0x10000u;
    const uint32_t e = min((abs_bits + up) >> 23, 254u);
    return abs_bits >= 0x7f800000u ? 255u : e;
}

// The code of v as a byte in a word's low 8 bits (other bits undefined): fma(v, 2^-e, 1.5 * 2^23) leaves
// rint(v * 2^-e), ties to even, in two's complement in the low mantissa bits; v * 2^-e is exact.
__device__ __forceinline__ uint32_t group_code(float v, float inv)
{
    return __float_as_uint(__fmaf_rn(v, inv, 12582912.0f));
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

// The codes of a lane's 8 values of a group, as two words: with the scale 1 / inv, and under E.
__device__ __forceinline__ uint2 codes_of(const float (&v)[8], float inv)
{
    uint32_t q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = group_code(v[j], inv);
    return make_uint2(pack_bytes(q[0], q[1], q[2], q[3]), pack_bytes(q[4], q[5], q[6], q[7]));
}
__device__ __forceinline__ uint2 group_codes(const float (&v)[8], uint32_t E)
{
    if (E - 6u <= 247u) return codes_of(v, __uint_as_float((260u - E) << 23));
    // The scale leaves binary32's range (E < 6: in two steps), a code may pass 127 (E = 254), or the group has
    // no codes (E = 255: all 0; the bounds swallow NaN).
    const float bound = E < 6u ? __uint_as_float(0x7f800000u) : E == 254u ? 127.0f * 0x1p121f : 0.0f;
    const float pre = E < 6u ? 0x1p64f : 1.0f;
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = __fmul_rn(fminf(fmaxf(v[j], -bound), bound), pre);
    return codes_of(w, E < 6u ? __uint_as_float((196u - E) << 23) : 0x1p-121f);
}

// E of the group that a lane's 8 elements belong to (4 lanes hold it); every lane of the warp calls it.
__device__ __forceinline__ uint32_t group_of(const Words<float> &r)
{
    uint32_t m = r.w[0] & 0x7fffffffu;  // as integers, NaNs and infinities are the largest
#pragma unroll
    for (int j = 1; j < 8; ++j) m = max(m, r.w[j] & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return group_exp(m);
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <typename W>
__device__ __forceinline__ uint32_t max16x2(const W &r)
{
    uint32_t m = r.w[0] & 0x7fff7fffu;
#pragma unroll
    for (int j = 1; j < 4; ++j) m = max_u16x2(m, r.w[j] & 0x7fff7fffu);
    m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return max(m & 0xffffu, m >> 16);
}
__device__ __forceinline__ uint32_t group_of(const Words<__nv_bfloat16> &r) { return group_exp(max16x2(r) << 16); }
__device__ __forceinline__ uint32_t group_of(const Words<__half> &r)
{
    return group_exp(__float_as_uint(__half2float(__ushort_as_half((unsigned short)max16x2(r)))));
}

// Encode a lane's 8 elements (0 past the last column; r and v hold the same) of a chunk; every lane of the
// warp calls it.
template <typename T, bool FULL = false>
__device__ __forceinline__ void ckpt_store(const Words<T> &r, const float (&v)[8], const Ckpt &k, int64_t row, int base, int lane)
{
    const uint32_t E = group_of(r);
    const uint2 q = group_codes(v, E);
    const int c0 = base + lane * 8;
    if (FULL || c0 < k.code_pitch) *reinterpret_cast<uint2 *>(k.codes + row * k.code_pitch + c0) = q;
    if ((lane & 3) == 0 && (FULL || (c0 >> 5) < k.exp_pitch)) k.exps[row * k.exp_pitch + (c0 >> 5)] = (uint8_t)E;
}

// A lane's codes and their exponent, as loaded.
struct RawCkpt {
    uint32_t q[2], e;
};

template <bool FULL = false>
__device__ __forceinline__ void ckpt_load(RawCkpt &r, const Ckpt &k, int64_t row, int base, int lane)
{
    const int c0 = base + lane * 8;
    if (!FULL) r.q[0] = r.q[1] = r.e = 0;
    if (FULL || c0 < k.code_pitch) {
        const uint2 a = __ldg(reinterpret_cast<const uint2 *>(k.codes + row * k.code_pitch + c0));
        r.q[0] = a.x;
        r.q[1] = a.y;
        r.e = __ldg(k.exps + row * k.exp_pitch + (c0 >> 5));
    }
}

// Code j (0 .. 7) as a binary32 integer.
__device__ __forceinline__ float code_float(const RawCkpt &r, int j)
{
    // 2^23 + (q + 128), less 2^23 + 128
    return __fsub_rn(__uint_as_float(__byte_perm(r.q[j >> 2] ^ 0x80808080u, 0x4B000000u, 0x7440 | (j & 3))), 8388736.0f);
}

__device__ __forceinline__ void ckpt_floats(const RawCkpt &r, float (&v)[8])
{
    const float s = group_scale(r.e);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(code_float(r, j), s);
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
