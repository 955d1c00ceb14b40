// gq_act.cu -- pack and unpack of the 8-bit activation checkpoint, and activation functions whose
// forward pass writes the checkpoint of its input and whose backward pass reads it.
//
// All are one pass over their tensors: a warp takes chunks of 256 columns of a row, two at a time.
#include "gq_act.cuh"
#include "gq_act.h"
#include "gq_internal.h"

namespace gq {
namespace {

constexpr int kThreads = 256;

// f(x) and f'(x), in binary32.
//   GELU       x Phi(x);  Phi(x) + x phi(x).  Phi = erfc(-x / sqrt 2) / 2, which keeps the negative
//              tail's digits, where 1 + erf would cancel.
//   GELU tanh  x s(2u), u = sqrt(2/pi) (x + 0.044715 x^3)  [= x (1 + tanh u) / 2], s the logistic function;
//   SiLU       x s(x);  s (1 + x (1 - s)).
template <int KIND>
struct Fn;

// s(t) = 1 / (1 + exp(-t)) and 1 - s, through exp(-|t|) <= 1: neither overflows nor cancels.
__device__ __forceinline__ void logistic(float t, float &s, float &one_minus)
{
    const float e = expf(-fabsf(t));
    const float a = __fdividef(1.0f, 1.0f + e), b = e * a;
    s = t >= 0.0f ? a : b;
    one_minus = t >= 0.0f ? b : a;
}

template <>
struct Fn<GQ_FN_GELU> {
    static __device__ __forceinline__ float f(float x) { return 0.5f * x * erfcf(-x * 0.70710678f); }
    static __device__ __forceinline__ float df(float x)
    {
        return __fmaf_rn(x * 0.39894228f, expf(-0.5f * x * x), 0.5f * erfcf(-x * 0.70710678f));
    }
};
template <>
struct Fn<GQ_FN_GELU_TANH> {
    static constexpr float c = 1.5957691f;  // 2 sqrt(2/pi)
    // s is 0 or 1 in binary32 beyond |x| = 30; there x^3 need not be formed, which could overflow
    static __device__ __forceinline__ float bounded(float x) { return max_nan(min_nan(x, 30.0f), -30.0f); }
    static __device__ __forceinline__ float f(float x)
    {
        const float b = bounded(x);
        float s, r;
        logistic(c * __fmaf_rn(0.044715f * b, b * b, b), s, r);
        return x * s;
    }
    static __device__ __forceinline__ float df(float x)
    {
        const float b = bounded(x);
        float s, r;
        logistic(c * __fmaf_rn(0.044715f * b, b * b, b), s, r);
        return __fmaf_rn(b * s * r, c * __fmaf_rn(0.134145f * b, b, 1.0f), s);
    }
};
template <>
struct Fn<GQ_FN_SILU> {
    static __device__ __forceinline__ float f(float x)
    {
        float s, r;
        logistic(x, s, r);
        return x * s;
    }
    static __device__ __forceinline__ float df(float x)
    {
        float s, r;
        logistic(x, s, r);
        return s * __fmaf_rn(x, r, 1.0f);
    }
};

struct Params {
    int64_t rows, chunks;  // chunks: rows * chunks per row
    int cols, per_row;
    const void *a;
    void *b;
    int64_t sa, sb;
    Ckpt k;
};

template <typename T, int OP, int KIND, bool VEC>
__global__ void __launch_bounds__(kThreads) k_act(const __grid_constant__ Params p)
{
    constexpr int U = 2;
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t id0 = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); id0 < p.chunks; id0 += U * warps) {
        Raw<T> raw[U];
        RawCkpt<VEC> rk[U];
        int64_t row[U];
        int base[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t id = id0 + u * warps;
            if (id >= p.chunks) break;
            row[u] = id / p.per_row;
            base[u] = (int)(id - row[u] * p.per_row) * kChunk;
            if constexpr (OP != kUnpack)
                chunk_load<T, VEC>(raw[u], static_cast<const T *>(p.a) + row[u] * p.sa, base[u], lane, p.cols);
            if constexpr (OP == kUnpack || OP == kBackward) ckpt_load<VEC>(rk[u], p.k, row[u], base[u], lane);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (id0 + u * warps >= p.chunks) break;
            float v[8], o[8];
            if constexpr (OP == kPack || OP == kForward || OP == kForwardKeep) to_floats(raw[u], v);
            else ckpt_floats<VEC>(rk[u], v);
            if constexpr (OP == kPack || OP == kForwardKeep) ckpt_store<VEC>(v, p.k, row[u], base[u], lane);
            if constexpr (OP == kPack) continue;
            if constexpr (OP == kUnpack) {
                saturate<T>(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = v[j];
            } else if constexpr (OP == kBackward) {
                float d[8];
                to_floats(raw[u], d);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = d[j] * Fn<KIND>::df(v[j]);
            } else if constexpr (OP != kPack) {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = Fn<KIND>::f(v[j]);
            }
            if constexpr (OP != kPack) {
                Raw<T> out;
                from_floats(out, o);
                chunk_store<T, VEC>(out, static_cast<T *>(p.b) + row[u] * p.sb, base[u], lane, p.cols);
            }
        }
    }
}

template <typename T, int OP, int KIND>
cudaError_t launch(const ActArgs &a, cudaStream_t stream)
{
    const CkptLayout l = ckpt_layout(a.rows, a.cols);
    Params p;
    p.rows = a.rows;
    p.cols = (int)a.cols;
    p.per_row = (int)((a.cols + kChunk - 1) / kChunk);
    p.chunks = a.rows * p.per_row;
    p.a = a.a.p;
    p.sa = a.a.stride;
    p.b = const_cast<void *>(a.b.p);
    p.sb = a.b.stride;
    p.k = Ckpt{static_cast<uint8_t *>(a.ckpt), static_cast<uint8_t *>(a.ckpt) + l.exps_off, (int)l.code_pitch,
               (int)l.exp_pitch};
    // 16-byte accesses need every row to start on 16 bytes (the bases do)
    const int per16 = 16 / (int)sizeof(T);
    const bool vec = (OP == kUnpack || a.rows == 1 || p.sa % per16 == 0) && (OP == kPack || a.rows == 1 || p.sb % per16 == 0);
    auto kern = vec ? k_act<T, OP, KIND, true> : k_act<T, OP, KIND, false>;
    int per_sm = 0, sms = 0;
    const cudaError_t e = kernel_occupancy(reinterpret_cast<const void *>(kern), kThreads, 0, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    const int64_t need = (p.chunks + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t grid = need < (int64_t)per_sm * sms ? need : (int64_t)per_sm * sms;
    kern<<<(unsigned)grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T, int OP>
cudaError_t by_kind(const ActArgs &a, cudaStream_t s)
{
    switch (a.kind) {
    case GQ_FN_GELU: return launch<T, OP, GQ_FN_GELU>(a, s);
    case GQ_FN_GELU_TANH: return launch<T, OP, GQ_FN_GELU_TANH>(a, s);
    default: return launch<T, OP, GQ_FN_SILU>(a, s);
    }
}

template <typename T>
cudaError_t by_op(ActOp op, const ActArgs &a, cudaStream_t s)
{
    switch (op) {
    case kPack: return launch<T, kPack, 0>(a, s);
    case kUnpack: return launch<T, kUnpack, 0>(a, s);
    case kForward: return by_kind<T, kForward>(a, s);
    case kForwardKeep: return by_kind<T, kForwardKeep>(a, s);
    default: return by_kind<T, kBackward>(a, s);
    }
}

}  // namespace

cudaError_t launch_act(ActOp op, const ActArgs &a, cudaStream_t stream)
{
    if (a.dtype == GQ_FLOAT32) return by_op<float>(op, a, stream);
    if (a.dtype == GQ_BFLOAT16) return by_op<__nv_bfloat16>(op, a, stream);
    return by_op<__half>(op, a, stream);
}

}  // namespace gq
