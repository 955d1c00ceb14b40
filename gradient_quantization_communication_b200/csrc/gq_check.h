// gq_check.h -- argument checks that the stateless entry points share (host only).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "gq.h"

namespace gq {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

// NVTX range around an entry point (free when no profiler is attached).
struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

// A CUDA call's failure as a status.  The runtime keeps it as the thread's last error, which the next launch would report
// as its own although its kernel runs: it is taken from there.
inline gq_status_t cuda_failed()
{
    cudaGetLastError();
    return GQ_ERR_CUDA;
}
inline gq_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? GQ_OK : cuda_failed(); }

inline bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

inline int elem_size(int dtype) { return dtype == GQ_FLOAT32 ? 4 : (dtype == GQ_BFLOAT16 || dtype == GQ_FLOAT16) ? 2 : 0; }

// A region of memory: rows of `width` bytes, `stride` bytes apart.
struct Region {
    uintptr_t p;
    int64_t rows, width, stride;
};

inline Region region(const void *p, int64_t rows, int64_t cols, int64_t stride, int size)
{
    return Region{reinterpret_cast<uintptr_t>(p), rows, cols * size, rows > 1 ? stride * size : cols * size};
}
inline Region region(const void *p, size_t bytes) { return Region{reinterpret_cast<uintptr_t>(p), 1, (int64_t)bytes, (int64_t)bytes}; }

// Whether two regions share a byte.  Rows of one stride that interleave (columns of one wider buffer)
// do not; otherwise the regions' whole extents are compared.
inline bool overlap(const Region &a, const Region &b)
{
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return false;
    const uintptr_t ea = a.p + (uintptr_t)((a.rows - 1) * a.stride + a.width);
    const uintptr_t eb = b.p + (uintptr_t)((b.rows - 1) * b.stride + b.width);
    if (ea <= b.p || eb <= a.p) return false;
    if (a.rows > 1 && b.rows > 1 && a.stride == b.stride && a.stride > 0) {
        const uintptr_t s = (uintptr_t)a.stride;
        const uintptr_t d = b.p >= a.p ? (b.p - a.p) % s : (s - (a.p - b.p) % s) % s;
        if (d >= (uintptr_t)a.width && s - d >= (uintptr_t)b.width) return false;
    }
    return true;
}

// Every written region against all regions before it in the list.
template <int N>
bool any_overlap(const Region (&written)[N], int nw, const Region *read, int nr)
{
    for (int i = 0; i < nw; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(written[i], written[j])) return true;
        for (int j = 0; j < nr; ++j)
            if (overlap(written[i], read[j])) return true;
    }
    return false;
}

inline bool shape_ok(int64_t rows, int64_t cols) { return rows >= 0 && rows <= kMaxRows && cols >= 1 && cols <= GQ_ACT_MAX_COLS; }

// A matrix read (rows may repeat: stride 0) or written (rows may not share elements).
inline bool in_ok(const void *p, int64_t rows, int64_t stride)
{
    return p && aligned(p, 16) && (rows <= 1 || (stride >= 0 && stride <= (int64_t(1) << 36)));
}
inline bool out_ok(const void *p, int64_t rows, int64_t cols, int64_t stride)
{
    return in_ok(p, rows, stride) && (rows <= 1 || stride >= cols);
}

}  // namespace gq
