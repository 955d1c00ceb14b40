// gq_act.h -- launch entry points of the activation checkpoints' kernels, shared by their
// translation units (not part of the public ABI).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "gq.h"

namespace gq {

// A checkpoint of rows x cols values (include/gq.h, gq_act_layout).
struct CkptLayout {
    int64_t code_pitch, exp_pitch;
    size_t exps_off, bytes;
};
inline CkptLayout ckpt_layout(int64_t rows, int64_t cols)
{
    CkptLayout l;
    l.code_pitch = (cols + 31) / 32 * 32;
    l.exp_pitch = (cols + 127) / 128 * 4;
    l.exps_off = (size_t)((rows * l.code_pitch + 15) / 16 * 16);
    l.bytes = l.exps_off + (size_t)((rows * l.exp_pitch + 15) / 16 * 16);
    return l;
}

// A matrix of rows in device memory: stride counts elements.
struct Mat {
    const void *p;
    int64_t stride;
};

enum ActOp { kPack = 0, kUnpack = 1, kForward = 2, kForwardKeep = 3, kBackward = 4 };

struct ActArgs {
    int dtype, kind;
    int64_t rows, cols;
    Mat a;       // x (pack, forward), dy (backward)
    Mat b;       // y (forward), x (unpack), dx (backward): written
    void *ckpt;  // written by pack and kForwardKeep, read by unpack and backward
};
cudaError_t launch_act(ActOp op, const ActArgs &a, cudaStream_t stream);

struct NormArgs {
    int dtype, param_dtype;
    int64_t rows, cols;
    Mat x;               // forward; backward from the input (p NULL: from the checkpoint)
    Mat y;               // forward: y; backward: dx (written)
    Mat dy;              // backward
    void *ckpt;          // forward: written unless NULL; backward: read if x.p is NULL
    const void *gamma, *beta;
    float *mean, *rstd;
    float eps;
    float *dgamma, *dbeta;
    int accumulate;
    float *parts;        // backward: 2 * norm_parts(rows, cols) rows of cols floats
};
cudaError_t launch_norm_forward(const NormArgs &a, cudaStream_t stream);
cudaError_t launch_norm_backward(const NormArgs &a, cudaStream_t stream);
// Partial rows of dgamma and of dbeta that the backward pass writes.
int64_t norm_parts(int64_t rows, int64_t cols);

struct WgradArgs {
    int dtype;
    int64_t tokens, in, out;
    const void *ckpt;
    Mat dy;
    float *dw;
    int64_t dw_stride;
    float *db;           // NULL: no bias
    int accumulate;
    unsigned char *ws;
};
// Workspace of a weight gradient: the staged gradient, cut tiles and the partial rows of the bias.
size_t wgrad_workspace(int dtype, int64_t tokens, int64_t in, int64_t out, int64_t dy_stride, bool bias);
cudaError_t launch_wgrad(const WgradArgs &a, cudaStream_t stream);

// Sums over rows: part[p][c] = sum over the rows of part p of dy[row][c], then
// out[c] = (accumulate ? out[c] : 0) + sum over p, in a fixed order.  0 parts: few rows, summed in one kernel.
int64_t colsum_parts(int64_t rows, int64_t cols);
cudaError_t launch_colsum(int dtype, int64_t rows, int64_t cols, Mat dy, float *parts, float *out, int accumulate,
                          cudaStream_t stream);
// out0 / out1 (either may be NULL) from parts rows of cols floats each.
cudaError_t launch_parts_reduce(const float *part0, const float *part1, int64_t parts, int64_t cols, float *out0,
                                float *out1, int accumulate, cudaStream_t stream);

}  // namespace gq
