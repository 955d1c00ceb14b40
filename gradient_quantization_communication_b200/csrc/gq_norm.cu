// gq_norm.cu -- layer norm over the rows of a matrix: forward (optionally writing the 8-bit checkpoint
// of its input in the same pass) and backward (from the input or from its checkpoint), with the
// reduction of the weight's and bias's gradients over the rows.
//
//   forward   mean = sum x / C;  var = sum (x - mean)^2 / C;  rstd = 1 / sqrt(var + eps);
//             y = (x - mean) rstd gamma + beta.
//   backward  xh = (x - mean) rstd, g = dy gamma;
//             dx = rstd (g - sum g / C - xh sum(g xh) / C);
//             dgamma = sum over rows of dy xh;  dbeta = sum over rows of dy.
// Measured in a graph at 16384 x 4096 bf16, of 6554 GB/s: forward 51 us (81 %), with the checkpoint 72 us (72 %),
// backward from the input 79 us (78 %), from the checkpoint 80 us (64 %).  Issue alone (22 and 26 instructions an
// element, where full bandwidth leaves 27 slots) would take less than the bytes do, and is 59 and 66 % active: at 128
// registers a thread a quarter of the warps fit, too few to hide a row's way from its load through shuffles and
// the join of its warps to its store.
// Sums are binary32.  The squares are summed around the mean, not as sum x^2 - (sum x)^2 / C, which
// cancels for rows whose mean is large against their spread.
#include "gq_act.cuh"
#include "gq_act.h"
#include "gq_internal.h"

namespace gq {
namespace {

constexpr unsigned kFullMask = 0xffffffffu;

struct Params {
    int64_t rows;
    int cols;
    const void *x, *dy;
    void *y;             // y or dx
    int64_t sx, sdy, sy;
    Ckpt k;              // codes NULL: none
    const void *gamma, *beta;
    int params_f32;      // gamma and beta are float32, else the tensors' type
    float *mean, *rstd;
    float eps;
    float *part_g, *part_b;
    int parts;
    int G, slots;        // rows in registers: warps a row, rows a block
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

// A lane's 8 values of gamma or beta (fill where there is none).
template <typename T>
__device__ __forceinline__ void param_load(float (&v)[8], const void *p, int f32, float fill, int base, int lane, int cols)
{
    if (p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        if (f32) {
            Raw<float, true> r;
            chunk_load<float, true>(r, static_cast<const float *>(p), base, lane, cols);
            to_floats(in_place<float, true>(r, nullptr), v);
        } else {
            Raw<T, true> r;
            chunk_load<T, true>(r, static_cast<const T *>(p), base, lane, cols);
            to_floats(in_place<T, true>(r, nullptr), v);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = base + lane * 8 + j;
        v[j] = fill;
        if (p && c < cols) v[j] = f32 ? __ldg(static_cast<const float *>(p) + c) : to_f(static_cast<const T *>(p)[c]);
    }
}

// A lane's 8 values of a row.
template <typename T, bool AL>
__device__ __forceinline__ void row_floats(float (&v)[8], const T *row, int base, int lane, int cols)
{
    Raw<T, AL> r;
    chunk_load<T, AL>(r, row, base, lane, cols);
    to_floats(in_place<T, AL>(r, row), v);
}
template <typename T, bool AL, bool FULL = false>
__device__ __forceinline__ void row_store(const float (&v)[8], T *row, int base, int lane, int cols)
{
    Words<T> r;
    from_floats(r, v);
    chunk_store<T, AL, FULL>(r, row, base, lane, cols);
}

// Sum over the G warps that share a row; `buf` holds one float per warp.  One barrier: the caller
// alternates buffers, so a buffer is written again only after a later barrier.
__device__ __forceinline__ float row_sum(float v, float *buf, int G, int warp, int lane)
{
    v = warp_sum(v);
    if (G == 1) return v;
    if (lane == 0) buf[warp] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < G; ++i) s += buf[i];
    return s;
}

// ---------------------------------------------------------------------------------------------
// Rows kept in registers.  G warps take a row, NC chunks of 256 columns each (chunk c of warp w is w + c G); a
// block holds `slots` such groups and walks the rows, and loads its next row before it works on the present one.
// ---------------------------------------------------------------------------------------------
constexpr int kForwardCols = 16384, kBackwardCols = 8192;

struct Shape {
    int G, nc, slots;
};
inline Shape shape_of(int64_t cols, int most)
{
    const int n = (int)((cols + kChunk - 1) / kChunk);
    Shape s;
    s.nc = n >= most ? most : n >= 2 ? 2 : 1;
    s.G = (n + s.nc - 1) / s.nc;
    s.slots = s.G >= 8 ? 1 : 8 / s.G;  // blocks of about 8 warps
    return s;
}
// Forward: four chunks a warp where the rows are enough to fill the device, since the reductions and the
// barrier are per warp; for fewer rows one, which has the shortest way from load to store.
inline Shape forward_shape(int64_t rows, int64_t cols)
{
    const int n = (int)((cols + kChunk - 1) / kChunk);
    return shape_of(cols, rows * n <= 148 * 16 && n <= 16 ? 1 : 4);
}
// Backward: two, whose sums and next row still fit 128 registers.
inline Shape backward_shape(int64_t cols) { return shape_of(cols, 2); }

// gamma or beta of all columns in shared memory, binary32, read again for every row: n chunks of 256 columns,
// of which lane l's first four (columns 8 l ..) lie at words 4 l and its others at 128 + 4 l, so that 8 lanes
// read all banks.  What columns past the last hold is not used.
template <typename T>
__device__ __forceinline__ void params_to_shared(float *dst, const void *src, int f32, float fill, int n, int cols, int warp, int lane)
{
    for (int i = warp; i < n; i += blockDim.x >> 5) {
        float v[8];
        param_load<T>(v, src, f32, fill, i * kChunk, lane, cols);
        float4 *d = reinterpret_cast<float4 *>(dst + i * kChunk) + lane;
        d[0] = make_float4(v[0], v[1], v[2], v[3]);
        d[32] = make_float4(v[4], v[5], v[6], v[7]);
    }
}
__device__ __forceinline__ void params_shared(float (&v)[8], const float *src, int base, int lane)
{
    const float4 a = *reinterpret_cast<const float4 *>(src + base + lane * 4);
    const float4 b = *reinterpret_cast<const float4 *>(src + base + 128 + lane * 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Barrier of a slot's G warps.
__device__ __forceinline__ void slot_sync(int slot, int G)
{
    asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(G * 32) : "memory");
}

// How the rows lie: anywhere; from 16-byte boundaries; so, and all of a warp's chunks are whole.
enum Rows { kAnywhere, kAligned, kWhole };

template <typename T, int ROWS, int NC, bool KEEP>
__global__ void __launch_bounds__(512) k_forward(const __grid_constant__ Params p)
{
    constexpr bool AL = ROWS != kAnywhere;
    extern __shared__ float4 shared_params[];
    __shared__ float4 buf[2][16];
    const int lane = threadIdx.x & 31, G = p.G;
    const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0);  // known to be the same in all lanes
    const int slot = warp / G, wslot = warp - slot * G;
    const float inv_c = 1.0f / (float)p.cols;
    float mine = 0.0f;  // columns of this warp
#pragma unroll
    for (int c = 0; c < NC; ++c) mine += (float)min(max(p.cols - (wslot + c * G) * kChunk, 0), kChunk);
    const float inv_mine = 1.0f / mine;
    float *gamma = reinterpret_cast<float *>(shared_params), *beta = gamma + NC * G * kChunk;
    params_to_shared<T>(gamma, p.gamma, p.params_f32, 1.0f, NC * G, p.cols, warp, lane);
    params_to_shared<T>(beta, p.beta, p.params_f32, 0.0f, NC * G, p.cols, warp, lane);
    __syncthreads();
    const int64_t step = (int64_t)gridDim.x * p.slots;
    int64_t row = (int64_t)blockIdx.x * p.slots + slot;
    Raw<T, AL> next[NC];
    auto inner = [&](int c) { return ROWS == kWhole || inner_chunk<T, AL>((wslot + c * G) * kChunk, p.cols); };
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const T *x = static_cast<const T *>(p.x) + r * p.sx;
            if (inner(c)) chunk_load<T, AL, true>(next[c], x, (wslot + c * G) * kChunk, lane, p.cols);
            else chunk_load<T, AL, false>(next[c], x, (wslot + c * G) * kChunk, lane, p.cols);
        }
    };
    if (row < p.rows) fetch(row);
    int turn = 0;
    for (; row < p.rows; row += step, turn ^= 1) {
        float v[NC][8];
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Words<T> w = in_place<T, AL>(next[c], static_cast<const T *>(p.x) + row * p.sx);
            to_floats(w, v[c]);
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[c][j];
            if constexpr (KEEP) {
                if (inner(c)) ckpt_store<T, true>(w, v[c], p.k, row, (wslot + c * G) * kChunk, lane);
                else ckpt_store<T, false>(w, v[c], p.k, row, (wslot + c * G) * kChunk, lane);
            }
        }
        if (row + step < p.rows) fetch(row + step);
        // the warp's own mean and squares around it, then all warps' put together with one barrier:
        // sum (x - mean)^2 = sum over warps of (their squares + their columns (their mean - mean)^2)
        s = warp_sum(s);
        const float wmean = s * inv_mine;
        float ss = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int c0 = (wslot + c * G) * kChunk;
            if (ROWS == kWhole || c0 + kChunk <= p.cols) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = v[c][j] - wmean;
                    ss = __fmaf_rn(d, d, ss);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = c0 + lane * 8 + j < p.cols ? v[c][j] - wmean : 0.0f;
                    ss = __fmaf_rn(d, d, ss);
                }
            }
        }
        ss = warp_sum(ss);
        float mean = wmean;
        if (G > 1) {
            if (lane == 0) buf[turn][warp] = make_float4(mine, s, wmean, ss);
            slot_sync(slot, G);
            const float4 *b = buf[turn] + slot * G;
            s = 0.0f;
            for (int g = 0; g < G; ++g) s += b[g].y;
            mean = s * inv_c;
            ss = 0.0f;
            for (int g = 0; g < G; ++g) {
                const float d = b[g].z - mean;
                ss += __fmaf_rn(b[g].x * d, d, b[g].w);
            }
        }
        const float rstd = 1.0f / sqrtf(ss * inv_c + p.eps);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int base = (wslot + c * G) * kChunk;
            float g[8], b[8];
            params_shared(g, gamma, base, lane);
            params_shared(b, beta, base, lane);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[c][j] = __fmaf_rn((v[c][j] - mean) * rstd, g[j], b[j]);
            T *y = static_cast<T *>(p.y) + row * p.sy;
            if (inner(c)) row_store<T, AL, true>(v[c], y, base, lane, p.cols);
            else row_store<T, AL, false>(v[c], y, base, lane, p.cols);
        }
        if (wslot == 0 && lane == 0) {
            p.mean[row] = mean;
            p.rstd[row] = rstd;
        }
    }
}

// dx, and the block's partial sums of dgamma and dbeta (part_g, part_b: one row a block).
template <typename T, int ROWS, int NC, bool FROM_CKPT>
__global__ void __launch_bounds__(512) k_backward(const __grid_constant__ Params p)
{
    constexpr bool AL = ROWS != kAnywhere;
    extern __shared__ float4 shared_params[];
    __shared__ float2 buf[2][16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = p.G;
    const int slot = warp / G, wslot = warp - slot * G;
    const float inv_c = 1.0f / (float)p.cols;
    const int64_t step = (int64_t)gridDim.x * p.slots;
    int64_t row = (int64_t)blockIdx.x * p.slots + slot;
    Raw<T, AL> ndy[NC], nx[FROM_CKPT ? 1 : NC];
    RawCkpt nk[FROM_CKPT ? NC : 1];
    float nmean = 0.0f, nrstd = 0.0f;
    auto inner = [&](int c) { return ROWS == kWhole || inner_chunk<T, AL>((wslot + c * G) * kChunk, p.cols); };
    auto fetch = [&](int64_t r) {
        nmean = __ldg(p.mean + r);
        nrstd = __ldg(p.rstd + r);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int base = (wslot + c * G) * kChunk;
            if (inner(c)) {
                chunk_load<T, AL, true>(ndy[c], static_cast<const T *>(p.dy) + r * p.sdy, base, lane, p.cols);
                if constexpr (FROM_CKPT) ckpt_load<true>(nk[c], p.k, r, base, lane);
                else chunk_load<T, AL, true>(nx[c], static_cast<const T *>(p.x) + r * p.sx, base, lane, p.cols);
            } else {
                chunk_load<T, AL, false>(ndy[c], static_cast<const T *>(p.dy) + r * p.sdy, base, lane, p.cols);
                if constexpr (FROM_CKPT) ckpt_load<false>(nk[c], p.k, r, base, lane);
                else chunk_load<T, AL, false>(nx[c], static_cast<const T *>(p.x) + r * p.sx, base, lane, p.cols);
            }
        }
    };
    float sg[NC][8], sb[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) sg[c][j] = sb[c][j] = 0.0f;
    if (row < p.rows) fetch(row);
    float *gamma = reinterpret_cast<float *>(shared_params);
    params_to_shared<T>(gamma, p.gamma, p.params_f32, 1.0f, NC * G, p.cols, warp, lane);
    __syncthreads();
    int turn = 0;
    for (; row < p.rows; row += step, turn ^= 1) {
        float x[NC][8], d[NC][8];
        const float mean = nmean, rstd = nrstd;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            to_floats(in_place<T, AL>(ndy[c], static_cast<const T *>(p.dy) + row * p.sdy), d[c]);
            if constexpr (FROM_CKPT) {
                const float sc = group_scale(nk[c].e);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[c][j] = __fmaf_rn(code_float(nk[c], j), sc, -mean) * rstd;
            } else {
                to_floats(in_place<T, AL>(nx[c], static_cast<const T *>(p.x) + row * p.sx), x[c]);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[c][j] = (x[c][j] - mean) * rstd;
            }
        }
        if (row + step < p.rows) fetch(row + step);
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float g[8];
            params_shared(g, gamma, (wslot + c * G) * kChunk, lane);
#pragma unroll
            for (int j = 0; j < 8; ++j) {  // past the last column d is 0
                sg[c][j] = __fmaf_rn(d[c][j], x[c][j], sg[c][j]);
                sb[c][j] += d[c][j];
                d[c][j] *= g[j];
                s0 += d[c][j];
                s1 = __fmaf_rn(d[c][j], x[c][j], s1);
            }
        }
        s0 = warp_sum(s0);
        s1 = warp_sum(s1);
        if (G > 1) {
            if (lane == 0) buf[turn][warp] = make_float2(s0, s1);
            slot_sync(slot, G);
            s0 = s1 = 0.0f;
            for (int g = 0; g < G; ++g) {
                const float2 b = buf[turn][slot * G + g];
                s0 += b.x;
                s1 += b.y;
            }
        }
        const float a0 = -(s0 * inv_c) * rstd, a1 = -(s1 * inv_c) * rstd;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
#pragma unroll
            for (int j = 0; j < 8; ++j) d[c][j] = __fmaf_rn(x[c][j], a1, __fmaf_rn(d[c][j], rstd, a0));
            T *y = static_cast<T *>(p.y) + row * p.sy;
            if (inner(c)) row_store<T, AL, true>(d[c], y, (wslot + c * G) * kChunk, lane, p.cols);
            else row_store<T, AL, false>(d[c], y, (wslot + c * G) * kChunk, lane, p.cols);
        }
    }
    if (!p.part_b) return;
    // the slots' sums, slot by slot in order (slots > 1: in shared memory behind gamma, chunks of 256 columns as
    // gamma's, so that 8 lanes use all banks)
    float *fold = gamma + NC * G * kChunk;
    for (int t = 0; t < p.slots; ++t) {
        if (slot == t) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int base = (wslot + c * G) * kChunk, col = base + lane * 8;
#pragma unroll
                for (int k = 0; k < 2; ++k) {  // dgamma, dbeta
                    float(&a)[8] = k ? sb[c] : sg[c];
                    float *f = fold + k * NC * G * kChunk;
                    if (t > 0) {
                        float old[8];
                        params_shared(old, f, base, lane);
#pragma unroll
                        for (int j = 0; j < 8; ++j) a[j] += old[j];
                    }
                    if (t + 1 < p.slots) {
                        float4 *d = reinterpret_cast<float4 *>(f + base) + lane;
                        d[0] = make_float4(a[0], a[1], a[2], a[3]);
                        d[32] = make_float4(a[4], a[5], a[6], a[7]);
                        continue;
                    }
                    float *o = (k ? p.part_b : p.part_g) + (int64_t)blockIdx.x * p.cols + col;
                    if (p.cols % 4 == 0 && col + 8 <= p.cols) {
                        reinterpret_cast<float4 *>(o)[0] = make_float4(a[0], a[1], a[2], a[3]);
                        reinterpret_cast<float4 *>(o)[1] = make_float4(a[4], a[5], a[6], a[7]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (col + j < p.cols) o[j] = a[j];
                    }
                }
            }
        }
        if (p.slots > 1) __syncthreads();
    }
}

// ---------------------------------------------------------------------------------------------
// Wider rows: one block per row at a time, any number of columns; the row is read three times (twice from
// cache).
// ---------------------------------------------------------------------------------------------
template <typename T, bool AL>
__global__ void __launch_bounds__(512) k_forward_any(const __grid_constant__ Params p)
{
    __shared__ float buf[2][16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = blockDim.x >> 5;
    const float inv_c = 1.0f / (float)p.cols;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T *x = static_cast<const T *>(p.x) + row * p.sx;
        T *y = static_cast<T *>(p.y) + row * p.sy;
        float s = 0.0f;
        for (int base = warp * kChunk; base < p.cols; base += G * kChunk) {
            float v[8];
            row_floats<T, AL>(v, x, base, lane, p.cols);
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[j];
        }
        const float mean = row_sum(s, buf[0], G, warp, lane) * inv_c;
        float ss = 0.0f;
        for (int base = warp * kChunk; base < p.cols; base += G * kChunk) {
            float v[8];
            row_floats<T, AL>(v, x, base, lane, p.cols);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = base + lane * 8 + j < p.cols ? v[j] - mean : 0.0f;
                ss = __fmaf_rn(d, d, ss);
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum(ss, buf[1], G, warp, lane) * inv_c + p.eps);
        for (int base = warp * kChunk; base < p.cols; base += G * kChunk) {
            float v[8], g[8], b[8];
            Raw<T, AL> r;
            chunk_load<T, AL>(r, x, base, lane, p.cols);
            const Words<T> w = in_place<T, AL>(r, x);
            to_floats(w, v);
            if (p.k.codes) ckpt_store<T>(w, v, p.k, row, base, lane);
            param_load<T>(g, p.gamma, p.params_f32, 1.0f, base, lane, p.cols);
            param_load<T>(b, p.beta, p.params_f32, 0.0f, base, lane, p.cols);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __fmaf_rn((v[j] - mean) * rstd, g[j], b[j]);
            row_store<T, AL>(v, y, base, lane, p.cols);
        }
        if (threadIdx.x == 0) {
            p.mean[row] = mean;
            p.rstd[row] = rstd;
        }
    }
}

// A lane's 8 values of the input, from the input or its checkpoint.
template <typename T, bool AL>
__device__ __forceinline__ void input_load(float (&v)[8], const Params &p, int64_t row, int base, int lane)
{
    if (p.x) {
        row_floats<T, AL>(v, static_cast<const T *>(p.x) + row * p.sx, base, lane, p.cols);
    } else {
        RawCkpt r;
        ckpt_load(r, p.k, row, base, lane);
        ckpt_floats(r, v);
    }
}

// dx for any number of columns, one block per row.
template <typename T, bool AL>
__global__ void __launch_bounds__(512) k_backward_rows_any(const __grid_constant__ Params p)
{
    __shared__ float buf[2][16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = blockDim.x >> 5;
    const float inv_c = 1.0f / (float)p.cols;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T *dy = static_cast<const T *>(p.dy) + row * p.sdy;
        const float mean = p.mean[row], rstd = p.rstd[row];
        float s0 = 0.0f, s1 = 0.0f;
        for (int base = warp * kChunk; base < p.cols; base += G * kChunk) {
            float x[8], d[8], g[8];
            row_floats<T, AL>(d, dy, base, lane, p.cols);
            input_load<T, AL>(x, p, row, base, lane);
            param_load<T>(g, p.gamma, p.params_f32, 1.0f, base, lane, p.cols);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (base + lane * 8 + j >= p.cols) continue;
                const float gd = g[j] * d[j];
                s0 += gd;
                s1 = __fmaf_rn(gd, (x[j] - mean) * rstd, s1);
            }
        }
        const float c0 = row_sum(s0, buf[0], G, warp, lane) * inv_c;
        const float c1 = row_sum(s1, buf[1], G, warp, lane) * inv_c;
        for (int base = warp * kChunk; base < p.cols; base += G * kChunk) {
            float x[8], d[8], g[8];
            row_floats<T, AL>(d, dy, base, lane, p.cols);
            input_load<T, AL>(x, p, row, base, lane);
            param_load<T>(g, p.gamma, p.params_f32, 1.0f, base, lane, p.cols);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                d[j] = rstd * __fmaf_rn(-(x[j] - mean) * rstd, c1, __fmaf_rn(g[j], d[j], -c0));
            row_store<T, AL>(d, static_cast<T *>(p.y) + row * p.sy, base, lane, p.cols);
        }
    }
}

// Partial sums over the rows: warp (chunk c, part q) walks rows q, q + parts, ..., eight (with the
// input: two) at a time.
template <typename T, bool AL, bool NORM>
__global__ void __launch_bounds__(128) k_cols(const __grid_constant__ Params p)
{
    constexpr int U = NORM ? 2 : 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int base = ((int)blockIdx.x * 4 + warp) * kChunk;
    if (base >= p.cols) return;
    const bool inner = inner_chunk<T, AL>(base, p.cols);
    float sg[8], sb[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sg[j] = sb[j] = 0.0f;
    for (int64_t row = blockIdx.y; row < p.rows; row += (int64_t)U * p.parts) {
        Raw<T, AL> r[U];
        float x[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = row + (int64_t)u * p.parts;
            if (t >= p.rows) break;
            if (inner) chunk_load<T, AL, true>(r[u], static_cast<const T *>(p.dy) + t * p.sdy, base, lane, p.cols);
            else chunk_load<T, AL, false>(r[u], static_cast<const T *>(p.dy) + t * p.sdy, base, lane, p.cols);
            if constexpr (NORM) input_load<T, AL>(x[u], p, t, base, lane);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = row + (int64_t)u * p.parts;
            if (t >= p.rows) break;
            float d[8];
            to_floats(in_place<T, AL>(r[u], static_cast<const T *>(p.dy) + t * p.sdy), d);
            if constexpr (NORM) {
                const float mean = p.mean[t], rstd = p.rstd[t];
#pragma unroll
                for (int j = 0; j < 8; ++j) sg[j] = __fmaf_rn(d[j], (x[u][j] - mean) * rstd, sg[j]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sb[j] += d[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = base + lane * 8 + j;
        if (c >= p.cols) continue;
        const int64_t o = (int64_t)blockIdx.y * p.cols + c;
        if (NORM) p.part_g[o] = sg[j];
        p.part_b[o] = sb[j];
    }
}

// Column sums of few rows in one kernel: a block takes a chunk of 256 columns, its 16 warps every 16th row each,
// eight at a time, and their sums are added in warp order.  Against partial rows and their reduction, a launch
// more: 64 rows 16.8 and 18.6 us (with the rest of the weight gradient, in a graph), 1024 rows 22.9 and 18.2 us; 512
// rows 19.6 and 21.8 us by calls, which set the border, but 16.0 and 15.1 us in a graph, which would have it lower.
constexpr int kFewRows = 512;

template <typename T, bool AL>
__global__ void __launch_bounds__(512) k_cols_few(const T *dy, int64_t sdy, int rows, int cols, float *out, int accumulate)
{
    __shared__ float s[16][kChunk];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int base = (int)blockIdx.x * kChunk;
    const bool inner = inner_chunk<T, AL>(base, cols);
    float sum[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
    for (int row = warp; row < rows; row += 8 * 16) {
        Raw<T, AL> r[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const T *p = dy + (int64_t)(row + 16 * u) * sdy;
            if (row + 16 * u >= rows) break;
            if (inner) chunk_load<T, AL, true>(r[u], p, base, lane, cols);
            else chunk_load<T, AL, false>(r[u], p, base, lane, cols);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (row + 16 * u >= rows) break;
            float d[8];
            to_floats(in_place<T, AL>(r[u], dy + (int64_t)(row + 16 * u) * sdy), d);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += d[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s[warp][j * 32 + lane] = sum[j];
    __syncthreads();
    const int c = base + (threadIdx.x & 31) * 8 + (threadIdx.x >> 5);  // element j = warp of lane's columns
    if (threadIdx.x < kChunk && c < cols) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += s[i][threadIdx.x];
        out[c] = accumulate ? out[c] + v : v;
    }
}

// Column sums of the partial rows, in a fixed order: 16 warps take 16 interleaved sets of rows of 32 columns,
// eight loads at a time, and their sums are added in warp order.  It is launched to start as the kernel before
// it drains, and waits here for its rows.
__global__ void __launch_bounds__(512) k_parts_reduce(const float *part0, const float *part1, int64_t parts, int cols,
                                                      float *out0, float *out1, int accumulate)
{
    cudaGridDependencySynchronize();
    __shared__ float s[16][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float *part = blockIdx.y ? part1 : part0;
    float *out = blockIdx.y ? out1 : out0;
    if (!out) return;
    const int c = (int)blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < cols) {
        const float *p = part + c;
        int64_t q = warp;
        for (; q + 7 * 16 < parts; q += 8 * 16) {
            float x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = p[(q + u * 16) * cols];
#pragma unroll
            for (int u = 0; u < 8; ++u) v += x[u];
        }
        for (; q < parts; q += 16) v += p[q * cols];
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < cols) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += s[i][lane];
        out[c] = accumulate ? out[c] + v : v;
    }
}

Params params(const NormArgs &a)
{
    Params p;
    p.rows = a.rows;
    p.cols = (int)a.cols;
    p.x = a.x.p;
    p.sx = a.x.stride;
    p.dy = a.dy.p;
    p.sdy = a.dy.stride;
    p.y = const_cast<void *>(a.y.p);
    p.sy = a.y.stride;
    const CkptLayout l = ckpt_layout(a.rows, a.cols);
    p.k = Ckpt{static_cast<uint8_t *>(a.ckpt), a.ckpt ? static_cast<uint8_t *>(a.ckpt) + l.exps_off : nullptr,
               (int)l.code_pitch, (int)l.exp_pitch};
    p.gamma = a.gamma;
    p.beta = a.beta;
    p.params_f32 = a.param_dtype == GQ_FLOAT32;
    p.mean = a.mean;
    p.rstd = a.rstd;
    p.eps = a.eps;
    p.part_g = a.parts;
    p.parts = (int)norm_parts(a.rows, a.cols);
    p.part_b = a.parts ? a.parts + (int64_t)p.parts * a.cols : nullptr;
    return p;
}

bool rows_aligned(int64_t rows, const Mat &m, int per16) { return !m.p || rows == 1 || m.stride % per16 == 0; }

template <typename T, int NC>
cudaError_t forward_reg(const Params &p, bool al, cudaStream_t s)
{
    const bool whole = al && p.cols == NC * p.G * kChunk;
    auto kern = whole ? (p.k.codes ? k_forward<T, kWhole, NC, true> : k_forward<T, kWhole, NC, false>)
                : al  ? (p.k.codes ? k_forward<T, kAligned, NC, true> : k_forward<T, kAligned, NC, false>)
                      : (p.k.codes ? k_forward<T, kAnywhere, NC, true> : k_forward<T, kAnywhere, NC, false>);
    const int threads = p.G * p.slots * 32;
    const size_t smem = (size_t)NC * p.G * kChunk * 2 * sizeof(float);
    int per_sm = 0, sms = 0;
    const cudaError_t e = kernel_occupancy(reinterpret_cast<const void *>(kern), threads, smem, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    const int64_t need = (p.rows + p.slots - 1) / p.slots, most = (int64_t)per_sm * sms;
    kern<<<(unsigned)(need < most ? need : most), threads, smem, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t forward(const NormArgs &a, cudaStream_t s)
{
    const int per16 = 16 / (int)sizeof(T);
    const bool al = rows_aligned(a.rows, a.x, per16) && rows_aligned(a.rows, a.y, per16);
    Params p = params(a);
    if (a.cols <= kForwardCols) {
        const Shape sh = forward_shape(a.rows, a.cols);
        p.G = sh.G;
        p.slots = sh.slots;
        return sh.nc == 1 ? forward_reg<T, 1>(p, al, s) : sh.nc == 2 ? forward_reg<T, 2>(p, al, s) : forward_reg<T, 4>(p, al, s);
    }
    const int warps = 16;
    auto kern = al ? k_forward_any<T, true> : k_forward_any<T, false>;
    int per_sm = 0, sms = 0;
    const cudaError_t e = kernel_occupancy(reinterpret_cast<const void *>(kern), warps * 32, 0, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    const int64_t grid = a.rows < (int64_t)per_sm * sms ? a.rows : (int64_t)per_sm * sms;
    kern<<<(unsigned)grid, warps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, int NC>
cudaError_t backward_reg(const Params &p, bool al, cudaStream_t s)
{
    const bool whole = al && p.cols == NC * p.G * kChunk;
    auto kern = whole ? (p.x ? k_backward<T, kWhole, NC, false> : k_backward<T, kWhole, NC, true>)
                : al  ? (p.x ? k_backward<T, kAligned, NC, false> : k_backward<T, kAligned, NC, true>)
                      : (p.x ? k_backward<T, kAnywhere, NC, false> : k_backward<T, kAnywhere, NC, true>);
    const size_t smem = (size_t)NC * p.G * kChunk * (p.slots > 1 ? 3 : 1) * sizeof(float);
    int per_sm = 0, sms = 0;
    const cudaError_t e = kernel_occupancy(reinterpret_cast<const void *>(kern), p.G * p.slots * 32, smem, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)p.parts, p.G * p.slots * 32, smem, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward(const NormArgs &a, cudaStream_t s)
{
    const int per16 = 16 / (int)sizeof(T);
    const bool al = rows_aligned(a.rows, a.x, per16) && rows_aligned(a.rows, a.y, per16) && rows_aligned(a.rows, a.dy, per16);
    Params p = params(a);
    if (a.rows > 0 && a.cols <= kBackwardCols) {
        const Shape sh = backward_shape(a.cols);
        p.G = sh.G;
        p.slots = sh.slots;
        const cudaError_t e = sh.nc == 1 ? backward_reg<T, 1>(p, al, s) : backward_reg<T, 2>(p, al, s);
        if (e != cudaSuccess) return e;
    } else if (a.rows > 0) {
        const int64_t chunks = (a.cols + kChunk - 1) / kChunk;
        const int warps = 16;
        auto kern = al ? k_backward_rows_any<T, true> : k_backward_rows_any<T, false>;
        int per_sm = 0, sms = 0;
        cudaError_t e = kernel_occupancy(reinterpret_cast<const void *>(kern), warps * 32, 0, &per_sm, &sms);
        if (e != cudaSuccess) return e;
        const int64_t grid = a.rows < (int64_t)per_sm * sms ? a.rows : (int64_t)per_sm * sms;
        kern<<<(unsigned)grid, warps * 32, 0, s>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        if (a.dgamma || a.dbeta) {
            auto ck = al ? k_cols<T, true, true> : k_cols<T, false, true>;
            ck<<<dim3((unsigned)((chunks + 3) / 4), (unsigned)p.parts), 128, 0, s>>>(p);
            e = cudaGetLastError();
            if (e != cudaSuccess) return e;
        }
    }
    if (!a.dgamma && !a.dbeta) return cudaSuccess;
    return launch_parts_reduce(p.part_g, p.part_b, p.parts, a.cols, a.dgamma, a.dbeta, a.accumulate, s);
}

template <typename T>
cudaError_t colsum_few(int64_t rows, int64_t cols, Mat dy, float *out, int accumulate, cudaStream_t s)
{
    auto kern = rows_aligned(rows, dy, 16 / (int)sizeof(T)) ? k_cols_few<T, true> : k_cols_few<T, false>;
    kern<<<(unsigned)((cols + kChunk - 1) / kChunk), 512, 0, s>>>(static_cast<const T *>(dy.p), dy.stride, (int)rows, (int)cols, out,
                                                                  accumulate);
    return cudaGetLastError();
}

template <typename T>
cudaError_t colsum(int64_t rows, int64_t cols, Mat dy, float *parts, cudaStream_t s)
{
    Params p = {};
    p.rows = rows;
    p.cols = (int)cols;
    p.dy = dy.p;
    p.sdy = dy.stride;
    p.part_b = parts;
    p.parts = (int)colsum_parts(rows, cols);
    const int64_t chunks = (cols + kChunk - 1) / kChunk;
    auto ck = rows_aligned(rows, dy, 16 / (int)sizeof(T)) ? k_cols<T, true, false> : k_cols<T, false, false>;
    ck<<<dim3((unsigned)((chunks + 3) / 4), (unsigned)p.parts), 128, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

int64_t norm_parts(int64_t rows, int64_t cols)
{
    if (rows <= 0) return 0;
    if (cols > kBackwardCols) return rows < 296 ? rows : 296;
    // blocks of the backward pass: two an SM, and at least two rows to each of a block's slots, so that the
    // partial sums stay fewer bytes than the rows
    const int64_t rows_a_block = 2 * backward_shape(cols).slots;
    const int64_t n = (rows + rows_a_block - 1) / rows_a_block;
    return n < 296 ? n : 296;
}

int64_t colsum_parts(int64_t rows, int64_t cols)
{
    if (rows <= kFewRows) return 0;
    // parts of 8 rows, which a warp loads at once, up to eight blocks an SM: waiting for them is most of the time
    const int64_t across = (cols + 4 * kChunk - 1) / (4 * kChunk);
    int64_t n = (8 * 148 + across - 1) / across;
    if (n > (rows + 7) / 8) n = (rows + 7) / 8;
    return n;
}

cudaError_t launch_norm_forward(const NormArgs &a, cudaStream_t stream)
{
    if (a.dtype == GQ_FLOAT32) return forward<float>(a, stream);
    if (a.dtype == GQ_BFLOAT16) return forward<__nv_bfloat16>(a, stream);
    return forward<__half>(a, stream);
}

cudaError_t launch_norm_backward(const NormArgs &a, cudaStream_t stream)
{
    if (a.dtype == GQ_FLOAT32) return backward<float>(a, stream);
    if (a.dtype == GQ_BFLOAT16) return backward<__nv_bfloat16>(a, stream);
    return backward<__half>(a, stream);
}

cudaError_t launch_colsum(int dtype, int64_t rows, int64_t cols, Mat dy, float *parts, float *out, int accumulate,
                          cudaStream_t stream)
{
    if (rows <= kFewRows)
        return dtype == GQ_FLOAT32    ? colsum_few<float>(rows, cols, dy, out, accumulate, stream)
               : dtype == GQ_BFLOAT16 ? colsum_few<__nv_bfloat16>(rows, cols, dy, out, accumulate, stream)
                                      : colsum_few<__half>(rows, cols, dy, out, accumulate, stream);
    const cudaError_t e = dtype == GQ_FLOAT32    ? colsum<float>(rows, cols, dy, parts, stream)
                          : dtype == GQ_BFLOAT16 ? colsum<__nv_bfloat16>(rows, cols, dy, parts, stream)
                                                 : colsum<__half>(rows, cols, dy, parts, stream);
    if (e != cudaSuccess) return e;
    return launch_parts_reduce(parts, nullptr, colsum_parts(rows, cols), cols, out, nullptr, accumulate, stream);
}

cudaError_t launch_parts_reduce(const float *part0, const float *part1, int64_t parts, int64_t cols, float *out0,
                                float *out1, int accumulate, cudaStream_t stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((cols + 31) / 32), out1 ? 2u : 1u);
    cfg.blockDim = dim3(512);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_parts_reduce, part0, part1, parts, (int)cols, out0, out1, accumulate);
}

}  // namespace gq
