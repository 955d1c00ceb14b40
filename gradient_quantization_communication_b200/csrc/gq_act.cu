// gq_act.cu -- pack and unpack of the 8-bit activation checkpoint, and activation functions whose
// forward pass writes the checkpoint of its input and whose backward pass reads it.
//
// All are one pass over their tensors: a warp takes 512 or 1024 columns of a row at a time.  At
// full bandwidth 16-bit types leave some 27 instruction slots an element: pack (10) and unpack (8) are bound by
// the bytes.  GELU (28 an element forward with the checkpoint, 29 backward) would take 51 and 53 us by issue alone at
// 1.965 GHz; issue is 75 and 71 % active, and the rest is latency, in the backward pass that of its loads.  Measured in a graph at 16384 x 4096 bf16, of 6554 GB/s: pack 34 us (92 %), unpack 36 us (86 %), GELU forward
// with the checkpoint 72 us (72 %), backward 79 us (65 %), SiLU 60 and 76 us (86 and 68 %), GELU tanh 71 and 91 us.
#include "gq_act.cuh"
#include "gq_act.h"
#include "gq_internal.h"

namespace gq {
namespace {

constexpr int kThreads = 256;
constexpr int kWide = 4 * kChunk;
// Chunks of a row that a warp takes at a time.  Four spread an item's addresses over the most elements; where a
// chunk is two loads, or is shifted into place, their registers cost more.  At 16384 x 4096, two against four: SiLU
// backward bf16 76 and 102 us, forward with the checkpoint 59 and 60 us, GELU's 74 and 72 us, SiLU's of float32 112
// and 100 us; at 16384 x 4095 bf16 (shifted) SiLU forward with the checkpoint 106 and 140 us.
__host__ __device__ constexpr int chunks_of(int op, bool al) { return op == kBackward || !al ? 2 : 4; }

// f(x) and f'(x), in binary32.
//   GELU       x Phi(x);  Phi(x) + x phi(x).  Phi = erfc(-x / sqrt 2) / 2, which keeps the negative
//              tail's digits, where 1 + erf would cancel.
//   GELU tanh  x s(2u), u = sqrt(2/pi) (x + 0.044715 x^3)  [= x (1 + tanh u) / 2], s the logistic function;
//   SiLU       x s(x);  s (1 + x (1 - s)).
// In 16-bit types, whose own step hides it, the exponential is the hardware's (2^-22 of its result, besides what
// its argument's roundings make of it: 2^-17 where the result nears 2^-126), and Phi's tail comes from a
// polynomial; binary32 calls expf and erfcf.
// exp(t) for t <= 0, subnormal results included.
template <bool FAST>
__device__ __forceinline__ float exp_neg(float t)
{
    if constexpr (!FAST) return expf(t);
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(t * 1.4426950f));
    return r;
}
// 1 / x for 1 <= x.
template <bool FAST>
__device__ __forceinline__ float inverse(float x)
{
    if constexpr (!FAST) return __fdividef(1.0f, x);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// s(t) = 1 / (1 + exp(-t)) and 1 - s, through exp(-|t|) <= 1: neither overflows nor cancels.
template <bool FAST>
__device__ __forceinline__ void logistic(float t, float &s, float &one_minus)
{
    const float e = exp_neg<FAST>(-fabsf(t));
    const float a = inverse<FAST>(1.0f + e), b = e * a;
    s = t >= 0.0f ? a : b;
    one_minus = t >= 0.0f ? b : a;
}

// Phi(x) and exp(-x^2 / 2) * kUp<FAST>.  The fast exponential flushes results below 2^-126 to 0, where bf16 and
// binary32 still have values: it is formed 2^24 times as large, down to 2^-150, and the factors after it are that
// much smaller, for no more instructions (the offset joins the product with log2 e).
template <bool FAST>
constexpr float kUp = FAST ? 0x1p24f : 1.0f;

template <bool FAST>
__device__ __forceinline__ void normal(float x, float &Phi, float &e)
{
    if constexpr (FAST) {
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmaf_rn(-0.72134752f * x, x, 24.0f)));
        // Phi(-z) exp(z^2 / 2) = t P(t) with t = 1 / (1 + 0.31 z), z = |x|: the smoothest of such maps of
        // [0, inf) to (0, 1].  P has degree 7, fitted on z <= 14.5 (beyond, the tail is below binary32's
        // range) by Lawson's weighted least squares to the smallest largest relative error: 1.9e-7 with the
        // coefficients as rounded here, 5e-7 in binary32 arithmetic.
        constexpr float d = 1.0f / kUp<true>;
        const float t = inverse<true>(__fmaf_rn(0.31f, fabsf(x), 1.0f));
        float h = 0.035870399326086044f * d;
        h = __fmaf_rn(h, t, -0.1417304277420044f * d);
        h = __fmaf_rn(h, t, 0.15529736876487732f * d);
        h = __fmaf_rn(h, t, -0.015128081664443016f * d);
        h = __fmaf_rn(h, t, 0.11023717373609543f * d);
        h = __fmaf_rn(h, t, 0.10772977769374847f * d);
        h = __fmaf_rn(h, t, 0.12406746298074722f * d);
        h = __fmaf_rn(h, t, 0.12365640699863434f * d);
        const float tail = h * t * e;
        Phi = x >= 0.0f ? 1.0f - tail : tail;
    } else {
        e = expf(-0.5f * x * x);
        Phi = 0.5f * erfcf(-x * 0.70710678f);
    }
}

template <int KIND, bool FAST>
struct Fn;

template <bool FAST>
struct Fn<GQ_FN_GELU, FAST> {
    static __device__ __forceinline__ float f(float x)
    {
        float P, e;
        normal<FAST>(x, P, e);
        return x * P;
    }
    static __device__ __forceinline__ float df(float x)
    {
        float P, e;
        normal<FAST>(x, P, e);
        return __fmaf_rn(x * (0.39894228f / kUp<FAST>), e, P);
    }
};
template <bool FAST>
struct Fn<GQ_FN_GELU_TANH, FAST> {
    static constexpr float c = 1.5957691f;  // 2 sqrt(2/pi)
    // s is 0 or 1 in binary32 beyond |x| = 30; there x^3 need not be formed, which could overflow
    static __device__ __forceinline__ float bounded(float x) { return max_nan(min_nan(x, 30.0f), -30.0f); }
    static __device__ __forceinline__ float f(float x)
    {
        const float b = bounded(x);
        float s, r;
        logistic<FAST>(c * __fmaf_rn(0.044715f * b, b * b, b), s, r);
        return x * s;
    }
    static __device__ __forceinline__ float df(float x)
    {
        const float b = bounded(x);
        float s, r;
        logistic<FAST>(c * __fmaf_rn(0.044715f * b, b * b, b), s, r);
        return __fmaf_rn(b * s * r, c * __fmaf_rn(0.134145f * b, b, 1.0f), s);
    }
};
template <bool FAST>
struct Fn<GQ_FN_SILU, FAST> {
    static __device__ __forceinline__ float f(float x)
    {
        float s, r;
        logistic<FAST>(x, s, r);
        return x * s;
    }
    static __device__ __forceinline__ float df(float x)
    {
        float s, r;
        logistic<FAST>(x, s, r);
        return s * __fmaf_rn(x, r, 1.0f);
    }
};

struct Params {
    int64_t items;         // rows * items per row
    int cols, per_row;
    int64_t drow;          // warps of the grid = drow rows of items and dplace items
    int dplace;
    const void *a;
    void *b;
    int64_t sa, sb;
    Ckpt k;
};

// One item: up to chunks_of() chunks from column `base` of a row.  FULL: all of them are inner chunks.
template <typename T, int OP, int KIND, bool AL, bool FULL>
__device__ __forceinline__ void act_item(const Params &p, int64_t row, int base, int lane)
{
    constexpr bool READS = OP != kUnpack, WRITES = OP != kPack, DECODES = OP == kUnpack || OP == kBackward;
    constexpr int U = chunks_of(OP, AL);
    using F = Fn<KIND, sizeof(T) == 2>;
    const T *a = static_cast<const T *>(p.a) + row * p.sa;
    Raw<T, AL> raw[U];
    RawCkpt rk[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (!FULL && u > 0 && base + u * kChunk >= p.cols) break;
        if constexpr (READS) chunk_load<T, AL, FULL>(raw[u], a, base + u * kChunk, lane, p.cols);
        if constexpr (DECODES) ckpt_load<FULL>(rk[u], p.k, row, base + u * kChunk, lane);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int at = base + u * kChunk;
        if (!FULL && u > 0 && at >= p.cols) break;
        float in[8], v[8], o[8];
        if constexpr (READS) {
            const Words<T> w = in_place<T, AL>(raw[u], a);
            to_floats(w, in);
            if constexpr (OP == kPack || OP == kForwardKeep) ckpt_store<T, FULL>(w, in, p.k, row, at, lane);
        }
        if constexpr (DECODES) ckpt_floats(rk[u], v);
        if constexpr (OP == kUnpack) saturate<T>(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (OP == kUnpack) o[j] = v[j];
            else if constexpr (OP == kBackward) o[j] = in[j] * F::df(v[j]);
            else if constexpr (WRITES) o[j] = F::f(in[j]);
        }
        if constexpr (WRITES) {
            Words<T> out;
            from_floats(out, o);
            chunk_store<T, AL, FULL>(out, static_cast<T *>(p.b) + row * p.sb, at, lane, p.cols);
        }
    }
}

template <typename T, int OP, int KIND, bool AL>
__global__ void __launch_bounds__(kThreads) k_act(const __grid_constant__ Params p)
{
    constexpr int kItem = chunks_of(OP, AL) * kChunk;
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    int64_t id = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    // (row, place in the row) of id; a step of `warps` is (drow, dplace), without divisions
    int64_t row = id / p.per_row;
    int place = (int)(id - row * p.per_row);
    for (; id < p.items; id += warps) {
        const int base = place * kItem;
        if (inner_chunk<T, AL>(base, p.cols) && inner_chunk<T, AL>(base + kItem - kChunk, p.cols))
            act_item<T, OP, KIND, AL, true>(p, row, base, lane);
        else act_item<T, OP, KIND, AL, false>(p, row, base, lane);
        row += p.drow;
        place += p.dplace;
        if (place >= p.per_row) {
            place -= p.per_row;
            ++row;
        }
    }
}

template <typename T, int OP, int KIND>
cudaError_t launch(ActArgs a, cudaStream_t stream)
{
    // Rows without gaps, in the tensors and in the checkpoint, are one long row: cut it into rows of whole items.
    const int64_t n = a.rows * a.cols;
    if (a.cols % 128 == 0 && n % kWide == 0 && (OP == kUnpack || a.a.stride == a.cols) && (OP == kPack || a.b.stride == a.cols)) {
        a.cols = a.a.stride = a.b.stride = kWide;
        a.rows = n / kWide;
    }
    const CkptLayout l = ckpt_layout(a.rows, a.cols);
    Params p;
    p.cols = (int)a.cols;
    p.a = a.a.p;
    p.sa = a.a.stride;
    p.b = const_cast<void *>(a.b.p);
    p.sb = a.b.stride;
    p.k = Ckpt{static_cast<uint8_t *>(a.ckpt), static_cast<uint8_t *>(a.ckpt) + l.exps_off, (int)l.code_pitch,
               (int)l.exp_pitch};
    // whether every row starts on 16 bytes (the bases do)
    const int per16 = 16 / (int)sizeof(T);
    const bool al = (OP == kUnpack || a.rows == 1 || p.sa % per16 == 0) && (OP == kPack || a.rows == 1 || p.sb % per16 == 0);
    const int item = chunks_of(OP, al) * kChunk;
    p.per_row = (int)((a.cols + item - 1) / item);
    p.items = a.rows * p.per_row;
    auto kern = al ? k_act<T, OP, KIND, true> : k_act<T, OP, KIND, false>;
    int per_sm = 0, sms = 0;
    const cudaError_t e = kernel_occupancy(reinterpret_cast<const void *>(kern), kThreads, 0, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    const int64_t need = (p.items + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t grid = need < (int64_t)per_sm * sms ? need : (int64_t)per_sm * sms;
    const int64_t warps = grid * (kThreads / 32);
    p.drow = warps / p.per_row;
    p.dplace = (int)(warps - p.drow * p.per_row);
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
