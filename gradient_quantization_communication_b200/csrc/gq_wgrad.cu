// gq_wgrad.cu -- a linear layer's weight gradient from its input's 8-bit checkpoint:
//   dw[n][k] = sum over tokens t of dy[t][n] * xh[t][k],  xh the decoded input,
// and its bias gradient db[n] = sum over t of dy[t][n].  Sums are binary32.
#include "gq_act.cuh"
#include "gq_act.h"
#include "gq_internal.h"

namespace gq {
namespace {

struct Params {
    int64_t tokens;
    int in, out;
    Ckpt k;
    const void *dy;
    int64_t sdy;
    float *dw;
    int64_t sdw;
    int accumulate;
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

// 64 x 64 outputs per block, 4 x 4 per thread, 16 tokens at a time.
template <typename T>
__global__ void __launch_bounds__(256) k_wgrad_simple(const __grid_constant__ Params p)
{
    __shared__ float sx[16][64], sd[16][64];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int k0 = (int)blockIdx.x * 64, n0 = (int)blockIdx.y * 64;
    float acc[4][4] = {};
    for (int64_t t0 = 0; t0 < p.tokens; t0 += 16) {
        for (int i = threadIdx.x; i < 16 * 64; i += 256) {
            const int64_t t = t0 + (i >> 6);
            const int k = k0 + (i & 63), n = n0 + (i & 63);
            float x = 0.0f, d = 0.0f;
            if (t < p.tokens && k < p.in) {
                const float q = (float)(int8_t)p.k.codes[t * p.k.code_pitch + k];
                x = q * group_scale(p.k.exps[t * p.k.exp_pitch + (k >> 5)]);
                if (sizeof(T) == 2 && __is_same(T, __half)) {
                    x = x > 65504.0f ? 65504.0f : x < -65504.0f ? -65504.0f : x;
                    x = __half2float(__float2half_rn(x));
                }
            }
            if (t < p.tokens && n < p.out) d = to_f(static_cast<const T *>(p.dy)[t * p.sdy + n]);
            sx[i >> 6][i & 63] = x;
            sd[i >> 6][i & 63] = d;
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 16; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __fmaf_rn(sd[t][ty * 4 + i], sx[t][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + ty * 4 + i, k = k0 + tx + 16 * j;
            if (n >= p.out || k >= p.in) continue;
            float *o = p.dw + n * p.sdw + k;
            *o = p.accumulate ? *o + acc[i][j] : acc[i][j];
        }
}

template <typename T>
cudaError_t launch(const Params &p, cudaStream_t s)
{
    k_wgrad_simple<T><<<dim3((unsigned)((p.in + 63) / 64), (unsigned)((p.out + 63) / 64)), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t wgrad_workspace(int dtype, int64_t tokens, int64_t out, int64_t dy_stride, bool bias)
{
    (void)dtype;
    (void)dy_stride;
    return bias ? (size_t)colsum_parts(tokens, out) * (size_t)out * sizeof(float) : 0;
}

cudaError_t launch_wgrad(const WgradArgs &a, cudaStream_t stream)
{
    const CkptLayout l = ckpt_layout(a.tokens, a.in);
    uint8_t *ck = static_cast<uint8_t *>(const_cast<void *>(a.ckpt));
    Params p;
    p.tokens = a.tokens;
    p.in = (int)a.in;
    p.out = (int)a.out;
    p.k = Ckpt{ck, ck + l.exps_off, (int)l.code_pitch, (int)l.exp_pitch};
    p.dy = a.dy.p;
    p.sdy = a.dy.stride;
    p.dw = a.dw;
    p.sdw = a.dw_stride;
    p.accumulate = a.accumulate;
    const cudaError_t e = a.dtype == GQ_FLOAT32    ? launch<float>(p, stream)
                          : a.dtype == GQ_BFLOAT16 ? launch<__nv_bfloat16>(p, stream)
                                                   : launch<__half>(p, stream);
    if (e != cudaSuccess || !a.db) return e;
    return launch_colsum(a.dtype, a.tokens, a.out, a.dy, reinterpret_cast<float *>(a.ws), a.db, a.accumulate, stream);
}

}  // namespace gq
