// gq_fp8_api.cu -- host side of the entry points on packed matrices of 8-bit floating point (include/gq.h):
// argument checks and kernel selection.
#include <cstdint>

#include "gq_check.h"
#include "gq_fp8.h"

namespace {

using namespace gq;

bool kind_ok(int format, int tile) { return (format == GQ_FP8_E4M3 || format == GQ_FP8_E5M2) && (tile == 0 || tile == 1); }

}  // namespace

extern "C" {

gq_status_t gq_fp8_layout(int tile, int64_t rows, int64_t cols, size_t *bytes, size_t *codes_off, size_t *exps_off)
{
    if ((tile != 0 && tile != 1) || !shape_ok(rows, cols)) return GQ_ERR_INVALID;
    const Fp8Layout l = fp8_layout(tile, rows, cols);
    if (bytes) *bytes = l.bytes;
    if (codes_off) *codes_off = 0;
    if (exps_off) *exps_off = l.exps_off;
    return GQ_OK;
}

gq_status_t gq_fp8_pack(int dtype, int format, int tile, int64_t rows, int64_t cols, const void *x, int64_t x_stride,
                        void *packed, void *packed_t, void *stream)
{
    Range range("gq_fp8_pack");
    const int size = elem_size(dtype);
    if (!size || !kind_ok(format, tile) || !shape_ok(rows, cols) || (packed_t && !shape_ok(cols, rows))) return GQ_ERR_INVALID;
    if (rows == 0) return GQ_OK;
    if (!in_ok(x, rows, x_stride) || (!packed && !packed_t) || !aligned(packed, 16) || !aligned(packed_t, 16)) return GQ_ERR_INVALID;
    const Region w[] = {region(packed, fp8_layout(tile, rows, cols).bytes), region(packed_t, fp8_layout(tile, cols, rows).bytes)};
    const Region r[] = {region(x, rows, cols, x_stride, size)};
    if (any_overlap(w, 2, r, 1)) return GQ_ERR_INVALID;
    const Fp8PackArgs a = {dtype, format, tile, rows, cols, {x, x_stride}, packed, packed_t};
    return from_cuda(launch_fp8_pack(a, static_cast<cudaStream_t>(stream)));
}

gq_status_t gq_fp8_unpack(int dtype, int format, int tile, int64_t rows, int64_t cols, const void *packed, void *x,
                          int64_t x_stride, void *stream)
{
    Range range("gq_fp8_unpack");
    const int size = elem_size(dtype);
    if (!size || !kind_ok(format, tile) || !shape_ok(rows, cols)) return GQ_ERR_INVALID;
    if (rows == 0) return GQ_OK;
    if (!out_ok(x, rows, cols, x_stride) || !packed || !aligned(packed, 16)) return GQ_ERR_INVALID;
    const Region w[] = {region(x, rows, cols, x_stride, size)};
    const Region r[] = {region(packed, fp8_layout(tile, rows, cols).bytes)};
    if (any_overlap(w, 1, r, 1)) return GQ_ERR_INVALID;
    const Fp8PackArgs a = {dtype, format, tile, rows, cols, {x, x_stride}, const_cast<void *>(packed), nullptr};
    return from_cuda(launch_fp8_unpack(a, static_cast<cudaStream_t>(stream)));
}

gq_status_t gq_fp8_matmul_workspace(int64_t m, int64_t n, int64_t k, size_t *bytes)
{
    if (!shape_ok(m, k) || !shape_ok(n, k) || n < 1 || !bytes) return GQ_ERR_INVALID;
    *bytes = fp8_matmul_workspace(m, n, k);
    return GQ_OK;
}

gq_status_t gq_fp8_matmul(int dtype, int64_t m, int64_t n, int64_t k, int format_a, int tile_a, const void *a, int format_b,
                          int tile_b, const void *b, const float *bias, void *y, int64_t y_stride, int accumulate,
                          void *workspace, size_t workspace_bytes, void *stream)
{
    Range range("gq_fp8_matmul");
    const int size = elem_size(dtype);
    if (!size || !kind_ok(format_a, tile_a) || !kind_ok(format_b, tile_b) || !shape_ok(m, k) || !shape_ok(n, k) || n < 1)
        return GQ_ERR_INVALID;
    if (accumulate != 0 && accumulate != 1) return GQ_ERR_INVALID;
    if (accumulate && dtype != GQ_FLOAT32) return GQ_ERR_UNSUPPORTED;
    if (m == 0) return GQ_OK;
    if (!a || !b || !y || !aligned(a, 16) || !aligned(b, 16) || !aligned(bias, 4) || !aligned(y, (uintptr_t)size) ||
        (m > 1 && (y_stride < n || y_stride > (int64_t(1) << 40))))
        return GQ_ERR_INVALID;
    const size_t need = fp8_matmul_workspace(m, n, k);
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return GQ_ERR_INVALID;
    const Region w[] = {region(y, m, n, y_stride, size), region(workspace, need)};
    const Region r[] = {region(a, fp8_layout(tile_a, m, k).bytes), region(b, fp8_layout(tile_b, n, k).bytes),
                        region(bias, (size_t)n * 4)};
    if (any_overlap(w, 2, r, 3)) return GQ_ERR_INVALID;
    const Fp8MatmulArgs g = {dtype, m, n, k, format_a, tile_a, format_b, tile_b, a, b, bias, y, y_stride, accumulate,
                             static_cast<unsigned char *>(workspace)};
    return from_cuda(launch_fp8_matmul(g, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
