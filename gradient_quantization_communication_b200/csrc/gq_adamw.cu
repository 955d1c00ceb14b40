// gq_adamw.cu -- AdamW over many tensors in one launch, the gradients' global norm, and the moments' values.
//
// A block takes 4096 elements of one tensor, found in a table that the optimizer keeps on the device; a lane takes
// 8 consecutive ones, a warp 256 at a time: two blocks of 128 where the moments are in 8 bits, so that a block's
// largest value is found by shuffles within 16 lanes and every state is read and written once.
// Every operation rounds on its own (the formula's order, IEEE division and square root).
#include <type_traits>

#include "gq_act.cuh"
#include "gq_adamw.h"
#include "gq_device.cuh"
#include "gq_fp8.cuh"

namespace gq {
namespace {

constexpr int kThreads = 256;

struct Params {
    AdamStep s;
    const AdamTensor *tensors;
    const AdamChunk *table;
    uint32_t rk0[10], rk1[10];  // Philox round keys
};

// Largest of 8 values' absolute bits over a block of 128 (NaN above infinity).
__device__ __forceinline__ uint32_t block_max(const float (&x)[8])
{
    uint32_t b = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) b = max(b, __float_as_uint(x[j]) & 0x7fffffffu);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) b = max(b, __shfl_xor_sync(kFull, b, o));
    return b;
}

// The second moment's format (include/gq.h): 5 exponent and 3 mantissa bits of binary32, counted from 31 below E.
__device__ __forceinline__ uint32_t square_exp(uint32_t bits)
{
    return bits >= kInfBits ? 255u : min(max((bits + 0xfffffu) >> 23, 32u), 254u);
}
__device__ __forceinline__ uint32_t square_code(float v, uint32_t noise16, uint32_t E)
{
    const uint32_t bits = __float_as_uint(v);
    const int c = (int)((bits + (noise16 << 4)) >> 20) - (int)((E - 31u) << 3);
    return E == 255u || bits == 0u ? 0u : (uint32_t)min(max(c, 1), 255);
}
__device__ __forceinline__ float square_value(uint32_t c, uint32_t E)
{
    const float v = __uint_as_float((c + ((E - 31u) << 3)) << 20);
    return E == 255u ? __uint_as_float(0x7fffffffu) : c == 0u ? 0.0f : v;
}

__device__ __forceinline__ uint2 load8(const uint8_t *p) { return *reinterpret_cast<const uint2 *>(p); }
__device__ __forceinline__ uint32_t byte_of(uint2 q, int j) { return ((j < 4 ? q.x : q.y) >> (8 * (j & 3))) & 0xffu; }

// One warp's 256 elements from `base` of a chunk of n elements that starts at element `first` of its tensor.
template <typename P, typename G, bool MASTER, bool EIGHT, bool AL>
__device__ __forceinline__ void update(const Params &p, const AdamTensor &t, const gq_adamw_scalars_t &now, float scale,
                                       int64_t first, int n, int base, int lane)
{
    using S = typename std::conditional<MASTER, float, P>::type;  // what is updated
    S *const param = MASTER ? reinterpret_cast<S *>(t.master) + first : static_cast<S *>(t.param) + first;
    const G *const grad = static_cast<const G *>(t.grad) + first;
    // Unaligned loads take whole 16-byte pieces, with bytes that other warps may be writing: those are dropped.
    Raw<S, AL> rp;
    Raw<G, AL> rg;
    float m[8], v[8];
    chunk_load<S, AL, false, false>(rp, param, base, lane, n);
    chunk_load<G, AL, false>(rg, grad, base, lane, n);
    const int64_t at = first + base + lane * 8;  // of the tensor
    uint8_t *const m8 = static_cast<uint8_t *>(t.m), *const v8 = static_cast<uint8_t *>(t.v);
    const size_t exps = adam_exps_off(t.n);
    const bool in = base + lane * 8 < n;
    if constexpr (EIGHT) {
        uint2 qm = make_uint2(0u, 0u), qv = qm;
        uint32_t em = 0, ev = 32;
        if (in) {
            qm = load8(m8 + at);
            qv = load8(v8 + at);
            em = m8[exps + (at >> 7)];
            ev = v8[exps + (at >> 7)];
        }
        fp8_decode8<GQ_FP8_E4M3>(qm, fp8_scale(em), m);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = square_value(byte_of(qv, j), ev);
    } else {
        Raw<float, AL> r;
        chunk_load<float, AL, false, false>(r, static_cast<float *>(t.m) + first, base, lane, n);
        to_floats(in_place<float, AL>(r, static_cast<float *>(t.m) + first), m);
        chunk_load<float, AL, false, false>(r, static_cast<float *>(t.v) + first, base, lane, n);
        to_floats(in_place<float, AL>(r, static_cast<float *>(t.v) + first), v);
    }
    float x[8], g[8];
    to_floats(in_place<S, AL>(rp, param), x);
    to_floats(in_place<G, AL>(rg, grad), g);
    const float lr = __fmul_rn(now.lr, t.lr_scale);
    const float keep = __fsub_rn(1.0f, __fmul_rn(lr, t.decay)), size = __fmul_rn(lr, now.inv1);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float gj = __fmul_rn(g[j], scale);
        m[j] = __fadd_rn(__fmul_rn(m[j], p.s.beta1), __fmul_rn(gj, p.s.rest1));
        v[j] = __fadd_rn(__fmul_rn(v[j], p.s.beta2), __fmul_rn(__fmul_rn(gj, gj), p.s.rest2));
        const float below = __fadd_rn(__fmul_rn(__fsqrt_rn(v[j]), now.inv2), p.s.eps);
        x[j] = __fsub_rn(__fmul_rn(x[j], keep), __fmul_rn(size, __fdiv_rn(m[j], below)));
    }
    Words<S> ws;
    from_floats(ws, x);
    chunk_store<S, AL>(ws, param, base, lane, n);
    if constexpr (MASTER) {
        P *const out = static_cast<P *>(t.param) + first;
        Words<P> wp;
        from_floats(wp, x);
        chunk_store<P, AL>(wp, out, base, lane, n);
    }
    if constexpr (EIGHT) {
        // elements past the tensor's last are zeros
        if (base + lane * 8 + 8 > n) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (base + lane * 8 + j >= n) m[j] = v[j] = 0.0f;
        }
        const uint32_t em = fp8_exp<GQ_FP8_E4M3>(block_max(m)), ev = square_exp(block_max(v));
        const float inv = fp8_inverse(em);
        const uint2 qm = make_uint2(fp8_codes4<GQ_FP8_E4M3>(m[0], m[1], m[2], m[3], inv, em),
                                    fp8_codes4<GQ_FP8_E4M3>(m[4], m[5], m[6], m[7], inv, em));
        // Philox's counter (element / 8, step, tensor + 2^31)
        const uint64_t group = (uint64_t)at >> 3;
        const uint32_t c0 = (uint32_t)group, c2 = now.step;
        const unsigned long long p0 = (unsigned long long)0xD2511F53u * c0, p1 = (unsigned long long)0xCD9E8D57u * c2;
        const uint4 d = philox_rounds_2_to_10((uint32_t)(p1 >> 32) ^ (uint32_t)(group >> 32) ^ p.rk0[0], (uint32_t)p1,
                                              (uint32_t)(p0 >> 32) ^ (t.number | 0x80000000u) ^ p.rk1[0], (uint32_t)p0,
                                              p.rk0 + 1, p.rk1 + 1);
        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
        uint32_t q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = square_code(v[j], (j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu, ev);
        const uint2 qv = make_uint2(pack_bytes(q[0], q[1], q[2], q[3]), pack_bytes(q[4], q[5], q[6], q[7]));
        // whole blocks are written, the last one's codes past the tensor as 0
        if (first + base + (lane & 16) * 8 < t.n) {
            *reinterpret_cast<uint2 *>(m8 + at) = qm;
            *reinterpret_cast<uint2 *>(v8 + at) = qv;
            if ((lane & 15) == 0) {
                m8[exps + (at >> 7)] = (uint8_t)em;
                v8[exps + (at >> 7)] = (uint8_t)ev;
            }
        }
    } else {
        Words<float> w;
        from_floats(w, m);
        chunk_store<float, AL>(w, static_cast<float *>(t.m) + first, base, lane, n);
        from_floats(w, v);
        chunk_store<float, AL>(w, static_cast<float *>(t.v) + first, base, lane, n);
    }
}

template <typename P, typename G, bool MASTER, bool EIGHT>
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ Params p)
{
    const AdamChunk c = p.table[blockIdx.x];
    const float scale = p.s.scale ? *p.s.scale : 1.0f;
    if (scale != scale) return;
    gq_adamw_scalars_t now = p.s.now;
    if (p.s.scalars) now = *p.s.scalars;
    const AdamTensor t = p.tensors[c.tensor];
    const int64_t first = (int64_t)c.part * kAdamChunk;
    const int n = (int)min((int64_t)kAdamChunk, t.n - first), lane = threadIdx.x & 31;
    for (int base = (int)(threadIdx.x >> 5) * kChunk; base < n; base += kThreads / 32 * kChunk) {
        if (t.aligned) update<P, G, MASTER, EIGHT, true>(p, t, now, scale, first, n, base, lane);
        else update<P, G, MASTER, EIGHT, false>(p, t, now, scale, first, n, base, lane);
    }
}

// ---------------------------------------------------------------------------------------------
// The moments' values.
// ---------------------------------------------------------------------------------------------
template <typename T, bool AL>
__device__ __forceinline__ void put_values(float (&x)[8], void *out, int64_t at, int n, int base, int lane)
{
    saturate<T>(x);
    Words<T> w;
    from_floats(w, x);
    chunk_store<T, AL>(w, static_cast<T *>(out) + at, base, lane, n);
}

template <typename T, bool EIGHT, bool AL>
__device__ __forceinline__ void moments(const AdamTensor &t, int64_t first, int n, int base, int lane, void *m, void *v)
{
    const int64_t at = first + base + lane * 8, to = t.start + first;
    const bool in = base + lane * 8 < n;
    float x[8];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        void *const out = which ? v : m;
        if (!out) continue;
        if constexpr (EIGHT) {
            const uint8_t *const src = static_cast<const uint8_t *>(which ? t.v : t.m);
            uint2 q = make_uint2(0u, 0u);
            uint32_t E = 32;
            if (in) {
                q = __ldg(reinterpret_cast<const uint2 *>(src + at));
                E = __ldg(src + adam_exps_off(t.n) + (at >> 7));
            }
            if (which == 0) {
                fp8_decode8<GQ_FP8_E4M3>(q, fp8_scale(E), x);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = square_value(byte_of(q, j), E);
            }
        } else {
            // the tensor's slices may start elsewhere than the output's
            const float *const src = static_cast<const float *>(which ? t.v : t.m) + first;
            Raw<float, false> r;
            chunk_load<float, false>(r, src, base, lane, n);
            to_floats(in_place<float, false>(r, src), x);
        }
        put_values<T, AL>(x, out, to, n, base, lane);
    }
}

template <typename T, bool EIGHT>
__global__ void __launch_bounds__(kThreads) k_moments(const __grid_constant__ Params p, void *m, void *v)
{
    const AdamChunk c = p.table[blockIdx.x];
    const AdamTensor t = p.tensors[c.tensor];
    const int64_t first = (int64_t)c.part * kAdamChunk;
    const int n = (int)min((int64_t)kAdamChunk, t.n - first), lane = threadIdx.x & 31;
    const bool al = t.start % (16 / (int)sizeof(T)) == 0;
    for (int base = (int)(threadIdx.x >> 5) * kChunk; base < n; base += kThreads / 32 * kChunk) {
        if (al) moments<T, EIGHT, true>(t, first, n, base, lane, m, v);
        else moments<T, EIGHT, false>(t, first, n, base, lane, m, v);
    }
}

// ---------------------------------------------------------------------------------------------
// The gradients' norm, in binary64 throughout: squares neither overflow nor vanish, and a sum of 2^40 of them keeps
// more bits than the result has.  Blocks walk the table in strides of the grid; a second kernel adds their sums.
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ double block_sum(double s, double *shared)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    if (lane == 0) shared[warp] = s;
    __syncthreads();
    s = 0.0;
    if (threadIdx.x == 0)
        for (int i = 0; i < kThreads / 32; ++i) s += shared[i];
    return s;
}

template <typename G, bool AL>
__device__ __forceinline__ double squares(const G *grad, int n, int base, int lane)
{
    Raw<G, AL> r;
    chunk_load<G, AL>(r, grad, base, lane, n);
    float g[8];
    to_floats(in_place<G, AL>(r, grad), g);
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = __fma_rn((double)g[j], (double)g[j], s);
    return s;
}

template <typename G>
__global__ void __launch_bounds__(kThreads) k_norm(const AdamTensor *tensors, const AdamChunk *table, int64_t chunks, double *parts)
{
    __shared__ double shared[kThreads / 32];
    const int lane = threadIdx.x & 31;
    double s = 0.0;
    for (int64_t i = blockIdx.x; i < chunks; i += gridDim.x) {
        const AdamChunk c = table[i];
        const AdamTensor &t = tensors[c.tensor];
        const int64_t first = (int64_t)c.part * kAdamChunk;
        const G *const grad = static_cast<const G *>(t.grad) + first;
        const int n = (int)min((int64_t)kAdamChunk, t.n - first);
        const bool al = t.aligned != 0;
        for (int base = (int)(threadIdx.x >> 5) * kChunk; base < n; base += kThreads / 32 * kChunk)
            s += al ? squares<G, true>(grad, n, base, lane) : squares<G, false>(grad, n, base, lane);
    }
    s = block_sum(s, shared);
    if (threadIdx.x == 0) parts[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads) k_norm_join(const double *parts, int n, double max_norm, float *out)
{
    __shared__ double shared[kThreads / 32];
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) s += parts[i];
    s = block_sum(s, shared);
    if (threadIdx.x == 0) {
        const double norm = sqrt(s), f = norm > max_norm ? max_norm / norm : 1.0;
        out[0] = (float)norm;
        out[1] = norm <= 1.7e308 ? (float)f : __uint_as_float(0x7fffffffu);
    }
}

template <typename P, typename G, bool MASTER>
cudaError_t launch_state(const AdamArgs &a, const Params &p, cudaStream_t s)
{
    if (a.state_bits == 8) k_adamw<P, G, MASTER, true><<<(unsigned)a.chunks, kThreads, 0, s>>>(p);
    else k_adamw<P, G, MASTER, false><<<(unsigned)a.chunks, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}
template <typename P, typename G>
cudaError_t launch_master(const AdamArgs &a, const Params &p, cudaStream_t s)
{
    if constexpr (sizeof(P) == 2) {
        if (a.master) return launch_state<P, G, true>(a, p, s);
    }
    return launch_state<P, G, false>(a, p, s);
}
template <typename P>
cudaError_t launch_grad(const AdamArgs &a, const Params &p, cudaStream_t s)
{
    if (a.grad_dtype == GQ_FLOAT32) return launch_master<P, float>(a, p, s);
    if (a.grad_dtype == GQ_BFLOAT16) return launch_master<P, __nv_bfloat16>(a, p, s);
    return launch_master<P, __half>(a, p, s);
}
template <typename T>
cudaError_t launch_moments(const AdamArgs &a, const Params &p, void *m, void *v, cudaStream_t s)
{
    if (a.state_bits == 8) k_moments<T, true><<<(unsigned)a.chunks, kThreads, 0, s>>>(p, m, v);
    else k_moments<T, false><<<(unsigned)a.chunks, kThreads, 0, s>>>(p, m, v);
    return cudaGetLastError();
}

Params params_of(const AdamArgs &a)
{
    Params p = {};
    p.tensors = a.tensors;
    p.table = a.table;
    for (int i = 0; i < 10; ++i) {
        p.rk0[i] = (uint32_t)a.seed + (uint32_t)i * 0x9E3779B9u;
        p.rk1[i] = (uint32_t)(a.seed >> 32) + (uint32_t)i * 0xBB67AE85u;
    }
    return p;
}

}  // namespace

cudaError_t launch_adamw(const AdamArgs &a, const AdamStep &step, cudaStream_t s)
{
    Params p = params_of(a);
    p.s = step;
    if (a.param_dtype == GQ_FLOAT32) return launch_grad<float>(a, p, s);
    if (a.param_dtype == GQ_BFLOAT16) return launch_grad<__nv_bfloat16>(a, p, s);
    return launch_grad<__half>(a, p, s);
}

cudaError_t launch_adamw_moments(const AdamArgs &a, int dtype, void *m, void *v, cudaStream_t s)
{
    const Params p = params_of(a);
    if (dtype == GQ_FLOAT32) return launch_moments<float>(a, p, m, v, s);
    if (dtype == GQ_BFLOAT16) return launch_moments<__nv_bfloat16>(a, p, m, v, s);
    return launch_moments<__half>(a, p, m, v, s);
}

cudaError_t launch_adamw_norm(const AdamArgs &a, double max_norm, double *parts, float *out, cudaStream_t s)
{
    const unsigned grid = (unsigned)(a.chunks < kNormParts ? a.chunks : kNormParts);
    if (grid) {
        if (a.grad_dtype == GQ_FLOAT32) k_norm<float><<<grid, kThreads, 0, s>>>(a.tensors, a.table, a.chunks, parts);
        else if (a.grad_dtype == GQ_BFLOAT16) k_norm<__nv_bfloat16><<<grid, kThreads, 0, s>>>(a.tensors, a.table, a.chunks, parts);
        else k_norm<__half><<<grid, kThreads, 0, s>>>(a.tensors, a.table, a.chunks, parts);
    }
    k_norm_join<<<1, kThreads, 0, s>>>(parts, (int)grid, max_norm, out);
    return cudaGetLastError();
}

}  // namespace gq
