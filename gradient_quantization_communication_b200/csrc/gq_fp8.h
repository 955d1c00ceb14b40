// gq_fp8.h -- launch entry points of the kernels on packed matrices of 8-bit floating point, shared by their
// translation units (not part of the public ABI).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "gq.h"
#include "gq_act.h"

namespace gq {

// The packed form of rows x cols values (include/gq.h, gq_fp8_layout).
struct Fp8Layout {
    int64_t code_pitch, exp_rows, exp_pitch;
    size_t exps_off, bytes;
};
inline Fp8Layout fp8_layout(int tile, int64_t rows, int64_t cols)
{
    Fp8Layout l;
    l.code_pitch = (cols + 127) / 128 * 128;
    l.exp_rows = tile ? (rows + 127) / 128 : rows;
    l.exp_pitch = (cols + 511) / 512 * 4;
    l.exps_off = (size_t)((rows * l.code_pitch + 15) / 16 * 16);
    l.bytes = l.exps_off + (size_t)((l.exp_rows * l.exp_pitch + 15) / 16 * 16);
    return l;
}

struct Fp8PackArgs {
    int dtype, format, tile;
    int64_t rows, cols;
    Mat x;
    void *packed, *packed_t;  // either may be NULL
};
cudaError_t launch_fp8_pack(const Fp8PackArgs &a, cudaStream_t stream);
// x is written, packed read.
cudaError_t launch_fp8_unpack(const Fp8PackArgs &a, cudaStream_t stream);

struct Fp8MatmulArgs {
    int dtype;
    int64_t m, n, k;
    int format_a, tile_a, format_b, tile_b;
    const void *a, *b;
    const float *bias;
    void *y;
    int64_t y_stride;
    int accumulate;
    unsigned char *ws;
};
size_t fp8_matmul_workspace(int64_t m, int64_t n, int64_t k);
cudaError_t launch_fp8_matmul(const Fp8MatmulArgs &a, cudaStream_t stream);

}  // namespace gq
