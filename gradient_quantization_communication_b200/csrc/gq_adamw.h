// gq_adamw.h -- launch entry points of the AdamW kernels, shared by their translation units (not part of the
// public ABI).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "gq.h"

namespace gq {

constexpr int kAdamChunk = 4096;  // elements of a tensor that one block updates

// A moment of n elements in 8 bits.
__host__ __device__ inline size_t adam_exps_off(int64_t n) { return (size_t)((n + 127) / 128 * 128); }
inline size_t adam_bytes(int64_t n) { return adam_exps_off(n) + (size_t)(((n + 127) / 128 + 15) / 16 * 16); }

// A piece of a tensor, up to kAdamChunk elements, as the kernels read it: where each of its arrays starts.  With moments
// in 32 bits a tensor may start a few elements behind the first piece's start, where all arrays are on 16 bytes: slices of
// flat vectors are, wherever they begin (64 tensors of 1000001 float32 values: 395 us with loads that are shifted into place,
// 281 so).
struct alignas(16) AdamChunk {
    void *param;
    const void *grad;
    float *master;
    void *m, *v;          // float32 values, or codes
    uint8_t *em, *ev;     // the codes' exponents
    int64_t group;        // of 8 elements of its tensor, its first one
    int64_t start;        // elements of the pieces before it, in the order of the list
    int32_t n;            // with the head
    uint32_t number;      // its tensor's, in the caller's list
    float decay, lr_scale;
    int32_t head;         // elements before the tensor's first, in the arrays' first 16 bytes or 32: they are not the tensor's
};
static_assert(sizeof(AdamChunk) % 16 == 0, "read by 16 bytes");

struct AdamArgs {
    int param_dtype, grad_dtype, state_bits;
    bool master;
    int64_t aligned, chunks;  // pieces whose arrays all start on 16 bytes come first
    const AdamChunk *table;   // device
    uint64_t seed;
};

struct AdamStep {
    gq_adamw_scalars_t now;
    float beta1, rest1, beta2, rest2, eps;  // rest: 1 - beta
    bool fast;  // eps so large that the root of a subnormal second moment vanishes beside it, beta1 0 or at least 2^-9
    bool spread;  // beta1 so near 1 that a first moment in 8 bits would stand still under rounding to nearest
    const float *scale;
    const gq_adamw_scalars_t *scalars;
};
cudaError_t launch_adamw(const AdamArgs &a, const AdamStep &s, cudaStream_t stream);
cudaError_t launch_adamw_moments(const AdamArgs &a, int dtype, void *m, void *v, cudaStream_t stream);

// Partial sums that the norm writes (binary64).
constexpr int kNormPerSm = 4, kNormParts = 148 * kNormPerSm;
cudaError_t launch_adamw_norm(const AdamArgs &a, double max_norm, double *parts, float *out, cudaStream_t stream);

}  // namespace gq
