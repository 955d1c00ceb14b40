// gq_fp8_mm.cu -- products of packed matrices of 8-bit floating point:
//   y[i][j] = sum over blocks b of 2^(Ea + Eb - 254) * sum over c in b of a[i][c] * b[j][c]  + bias[j].
//
// A block of 256 threads takes a tile of 64 x 64, 32 columns at a time, decoded to binary32 in shared memory; a
// thread sums 4 x 4 of it on the ordinary cores.
#include "gq_act.cuh"
#include "gq_device.cuh"
#include "gq_fp8.cuh"
#include "gq_fp8.h"

namespace gq {
namespace {

struct Operand {
    const uint8_t *codes, *exps;
    int64_t rows, code_pitch, exp_pitch;
    int format, shift;  // rows that share an exponent: 1 << shift
};

struct Params {
    Operand a, b;
    int64_t k, sy;
    const float *bias;
    void *y;
    int accumulate, dtype;
    int64_t tiles_n;
};

__device__ __forceinline__ float value(const Operand &o, int64_t row, int64_t c)
{
    if (row >= o.rows || c >= o.code_pitch) return 0.0f;
    const uint32_t q = o.codes[row * o.code_pitch + c], E = o.exps[(row >> o.shift) * o.exp_pitch + (c >> 7)];
    return (o.format == GQ_FP8_E4M3 ? fp8_values<GQ_FP8_E4M3>(q).x : fp8_values<GQ_FP8_E5M2>(q).x) * fp8_scale(E);
}

__global__ void __launch_bounds__(256) k_simple(const __grid_constant__ Params p)
{
    __shared__ float sa[64][33], sb[64][33];
    const int64_t i0 = blockIdx.x / p.tiles_n * 64, j0 = blockIdx.x % p.tiles_n * 64;
    const int ti = (threadIdx.x >> 4) * 4, tj = (threadIdx.x & 15) * 4;
    float acc[4][4] = {};
    for (int64_t c0 = 0; c0 < p.k; c0 += 32) {
        for (int e = threadIdx.x; e < 64 * 32; e += 256) {
            sa[e >> 5][e & 31] = value(p.a, i0 + (e >> 5), c0 + (e & 31));
            sb[e >> 5][e & 31] = value(p.b, j0 + (e >> 5), c0 + (e & 31));
        }
        __syncthreads();
        for (int c = 0; c < 32; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __fmaf_rn(sa[ti + i][c], sb[tj + j][c], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t row = i0 + ti + i, col = j0 + tj + j;
            if (row >= p.a.rows || col >= p.b.rows) continue;
            float v = acc[i][j];
            if (p.bias) v += p.bias[col];
            const int64_t at = row * p.sy + col;
            if (p.dtype == GQ_FLOAT32) {
                float *y = static_cast<float *>(p.y) + at;
                *y = p.accumulate ? *y + v : v;
            } else if (p.dtype == GQ_BFLOAT16) {
                static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(v);
            } else {
                static_cast<__half *>(p.y)[at] = __float2half_rn(v);
            }
        }
}

Operand operand_of(const void *p, int format, int tile, int64_t rows, int64_t cols)
{
    const Fp8Layout l = fp8_layout(tile, rows, cols);
    const uint8_t *b = static_cast<const uint8_t *>(p);
    return Operand{b, b + l.exps_off, rows, l.code_pitch, l.exp_pitch, format, tile ? 7 : 0};
}

}  // namespace

size_t fp8_matmul_workspace(int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_fp8_matmul(const Fp8MatmulArgs &g, cudaStream_t stream)
{
    Params p;
    p.a = operand_of(g.a, g.format_a, g.tile_a, g.m, g.k);
    p.b = operand_of(g.b, g.format_b, g.tile_b, g.n, g.k);
    p.k = g.k;
    p.sy = g.m > 1 ? g.y_stride : 0;
    p.bias = g.bias;
    p.y = g.y;
    p.accumulate = g.accumulate;
    p.dtype = g.dtype;
    p.tiles_n = (g.n + 63) / 64;
    k_simple<<<(unsigned)((g.m + 63) / 64 * p.tiles_n), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gq
