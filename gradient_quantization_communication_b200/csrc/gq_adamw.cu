// gq_adamw.cu -- AdamW over many tensors in one launch, the gradients' global norm, and the moments' values.
//
// A block takes 4096 elements of one tensor at a time, found in a table that the optimizer keeps on the device; a lane
// takes 8 consecutive ones, a warp 256: two blocks of 128 where the moments are in 8 bits, so that a block's
// largest value is found by shuffles within 16 lanes and every state is read and written once.
// Every operation rounds on its own, in the formula's order; division and square root are IEEE's, but for `FAST` below.
//
// Moments in 32 bits are bounded by bytes: 64 tensors of 4194304, bf16 parameters with float32 masters and bf16
// gradients, 1105 us, where the bytes take 1147 at the rate of a plain copy.  In 8 bits by instructions and latency: 64
// tensors of 1e6, bf16 parameters and float32 gradients, 146 us, where 770 MB take 118; 61 % of the issue slots are used,
// at 80 registers and 24 warps an SM.  The norm is bounded by bytes (41 us for 256 MB, which take 39).
#include <type_traits>

#include "gq_act.cuh"
#include "gq_adamw.h"
#include "gq_device.cuh"
#include "gq_fp8.cuh"

namespace gq {
namespace {

constexpr int kThreads = 256;
constexpr int kHalf = kThreads / 32 * kChunk;  // elements that a block takes at once
static_assert(2 * kHalf == kAdamChunk, "two halves a chunk");

struct Params {
    AdamStep s;
    const AdamChunk *table;
    int64_t chunks;
    uint32_t rk0[10], rk1[10];  // Philox round keys
};

// The sums are taken one by one: packed sums of packed products come out fused, rounded once.
__device__ __forceinline__ void sum2(Two a, Two b, float &x, float &y)
{
    float a0, a1, b0, b1;
    apart(a, a0, a1);
    apart(b, b0, b1);
    x = __fadd_rn(a0, b0);
    y = __fadd_rn(a1, b1);
}

// The update's square root and quotient: rounded to nearest, or (FAST) off by up to 2 units in the last place each, and
// subnormal second moments as 0.  Only the parameter's own change, lr times something near 1, carries that error.  FAST is
// taken where the moments are in 8 bits and instructions bound the kernel (146 us with it, 202 without, 64 tensors of
// 1e6, bf16 parameters and fp32 gradients), and eps is so large that a subnormal moment's root (below 2^-63) vanishes
// beside it, and beta1 no smaller than update() can join with a block's scale.
template <bool FAST>
__device__ __forceinline__ float root(float x)
{
    if constexpr (!FAST) return __fsqrt_rn(x);
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
template <bool FAST>
__device__ __forceinline__ float quotient(float a, float b)
{
    if constexpr (!FAST) return __fdiv_rn(a, b);
    else return __fmul_rn(a, rcp_approx(b));  // b is at least eps, and below 2^126 unless it is infinite
}

// Bits of the largest |x| of a block of 128, which 16 lanes hold (a NaN's above infinity's).
__device__ __forceinline__ uint32_t block_max(const float (&x)[8])
{
    const float a = fmax3_nan(fabsf(x[0]), fabsf(x[1]), fabsf(x[2])), b = fmax3_nan(fabsf(x[3]), fabsf(x[4]), fabsf(x[5]));
    uint32_t m = __float_as_uint(fmax3_nan(fmax_nan(a, b), fabsf(x[6]), fabsf(x[7])));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
    return m;
}

// What a step does with moments in 8 bits: approximate root and quotient (FAST above) and, for beta1 above 17/18, the first
// moment rounded stochastically.
constexpr int kFast = 1, kSpread = 2;

// Codes of 8 first moments under E, up with the probability that the remainder has: the 16 random bits of w's halves are a
// fraction of a code's step.  From 2^-6 on the step is 2^-3 of the value's own power of two, and the sum's upper bits are the
// code, as for the second moment below; under it the step is 2^-9, and values are counted in 2^-25.
__device__ __forceinline__ uint2 spread_codes(const float (&m)[8], const uint32_t (&w)[4], uint32_t E)
{
    if (E == 255u) return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    const float inv = fp8_inverse(E);
    uint32_t q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t noise = (j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu;
        const float x = __fmul_rn(fabsf(m[j]), inv);
        const uint32_t above = ((__float_as_uint(x) + noise * 16u) >> 20) - (120u << 3);
        const uint32_t below = (__float2uint_rz(__fmul_rn(x, 0x1p25f)) + noise) >> 16;
        q[j] = (x >= 0x1p-6f ? above : below) | (__float_as_uint(m[j]) >> 24 & 0x80u);
    }
    return make_uint2(pack_bytes(q[0], q[1], q[2], q[3]), pack_bytes(q[4], q[5], q[6], q[7]));
}

// The second moment's format (include/gq.h): 5 exponent and 3 mantissa bits of binary32, counted from 31 below E.
__device__ __forceinline__ uint32_t square_exp(uint32_t bits)
{
    return bits >= kInfBits ? 255u : min(max((bits + 0xfffffu) >> 23, 32u), 254u);
}
// Codes of 8 values, whose random halves are those of w: binary32 bits with the fraction's 16 random bits added under
// the code's last, cut off there and counted from E's lowest.
__device__ __forceinline__ uint2 square_codes(const float (&v)[8], const uint32_t (&w)[4], uint32_t E)
{
    const int base = (int)((E - 31u) << 3);
    int q[8], least = 1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t noise = (j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu;
        q[j] = (int)((noise * 16u + __float_as_uint(v[j])) >> 20) - base;
        least = min(least, q[j]);
    }
    if (least < 1 || E >= 254u) {  // values 2^31 below the largest, or 0; beyond binary32's largest powers of two; not finite
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = E == 255u || v[j] == 0.0f ? 0 : min(max(q[j], 1), 255);
    }
    return make_uint2(pack_bytes(q[0], q[1], q[2], q[3]), pack_bytes(q[4], q[5], q[6], q[7]));
}
__device__ __forceinline__ bool zero_byte(uint32_t w) { return ((w - 0x01010101u) & ~w & 0x80808080u) != 0u; }
__device__ __forceinline__ void square_values(uint2 q, uint32_t E, float (&v)[8])
{
    const uint32_t base = (E - 31u) << 23;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = __uint_as_float(__byte_perm(j < 4 ? q.x : q.y, 0u, 0x4440u | (uint32_t)(j & 3)) * (1u << 20) + base);
    if (zero_byte(q.x) || zero_byte(q.y) || E == 255u) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t c = __byte_perm(j < 4 ? q.x : q.y, 0u, 0x4440u | (uint32_t)(j & 3));
            v[j] = E == 255u ? __uint_as_float(0x7fffffffu) : c ? v[j] : 0.0f;
        }
    }
}

// A lane's 8 elements, of which the first `head` of the piece are not the tensor's.
template <typename T, bool AL, bool FULL, bool KEPT = true>
__device__ __forceinline__ void piece_load(Raw<T, AL> &r, const T *row, int base, int lane, int head, int n)
{
    if constexpr (AL && !FULL) {
        if (base + lane * 8 < head) {  // a piece's first lane
#pragma unroll
            for (int j = 0; j < 8; ++j) elem_set<T>(r.w, j, j >= head && j < n ? elem_bits(row[j]) : 0u);
            return;
        }
    }
    chunk_load<T, AL, FULL, KEPT>(r, row, base, lane, n);
}
template <typename T, bool AL, bool FULL>
__device__ __forceinline__ void piece_store(const Words<T> &r, T *row, int base, int lane, int head, int n)
{
    if constexpr (AL && !FULL) {
        if (base + lane * 8 < head) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j >= head && j < n) row[j] = elem_get<T>(r.w, j);
            return;
        }
    }
    chunk_store<T, AL, FULL>(r, row, base, lane, n);
}

// What a lane has loaded of its 8 elements.
template <typename S, typename G, bool EIGHT, bool AL>
struct Loaded {
    Raw<S, AL> x;  // the parameters, or their master copies
    Raw<G, AL> g;
    Raw<float, AL> m[EIGHT ? 1 : 2];  // and v
};
template <typename S, typename G, bool AL>
struct Loaded<S, G, true, AL> {
    Raw<S, AL> x;
    Raw<G, AL> g;
    uint2 m, v;
    uint32_t em, ev;
};

template <typename S, bool MASTER>
__device__ __forceinline__ S *updated(const AdamChunk &c)
{
    if constexpr (MASTER) return c.master;
    else return static_cast<S *>(c.param);
}

// Unaligned loads take whole 16-byte pieces, with bytes that other warps may be writing: those are dropped.
// FULL: all of the warp's elements exist (aligned tensors).
template <typename S, typename G, bool MASTER, bool EIGHT, bool AL, bool FULL>
__device__ __forceinline__ void load(Loaded<S, G, EIGHT, AL> &l, const AdamChunk &c, int base, int lane)
{
    const int n = c.n, head = EIGHT ? 0 : c.head;
    piece_load<S, AL, FULL, false>(l.x, updated<S, MASTER>(c), base, lane, head, n);
    piece_load<G, AL, FULL>(l.g, static_cast<const G *>(c.grad), base, lane, head, n);
    if constexpr (EIGHT) {
        const int at = base + lane * 8;
        if (!FULL) {
            l.m = l.v = make_uint2(0u, 0u);
            l.em = 0;
            l.ev = 32;
        }
        if (FULL || at < n) {
            l.m = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(c.m) + at);
            l.v = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(c.v) + at);
            l.em = c.em[at >> 7];
            l.ev = c.ev[at >> 7];
        }
    } else {
        piece_load<float, AL, FULL, false>(l.m[0], static_cast<const float *>(c.m), base, lane, head, n);
        piece_load<float, AL, FULL, false>(l.m[1], static_cast<const float *>(c.v), base, lane, head, n);
    }
}

// One warp's 256 elements from `base` of a chunk.
template <typename P, typename S, typename G, bool MASTER, bool EIGHT, int MODE, bool AL, bool FULL>
__device__ __forceinline__ void update(const Params &p, const Loaded<S, G, EIGHT, AL> &l, const AdamChunk &c,
                                       const gq_adamw_scalars_t &now, float scale, int base, int lane)
{
    constexpr bool FAST = (MODE & kFast) != 0;
    const int n = c.n, at = base + lane * 8, head = EIGHT ? 0 : c.head;
    S *const param = updated<S, MASTER>(c);
    float x[8], g[8], m[8], v[8], beta1 = p.s.beta1;
    to_floats(in_place<S, AL>(l.x, param), x);
    to_floats(in_place<G, AL>(l.g, static_cast<const G *>(c.grad)), g);
    if constexpr (EIGHT) {
        // FAST: the scale, a power of two and at least 2^-117, joins beta1, which is 0 or at least 2^-9: their product is exact
        fp8_decode8<GQ_FP8_E4M3>(l.m, FAST ? 1.0f : fp8_scale(l.em), m);
        if (FAST) beta1 = __fmul_rn(fp8_scale(l.em), beta1);
        square_values(l.v, l.ev, v);
    } else {
        to_floats(in_place<float, AL>(l.m[0], static_cast<const float *>(c.m)), m);
        to_floats(in_place<float, AL>(l.m[1], static_cast<const float *>(c.v)), v);
    }
    const float lr = __fmul_rn(now.lr, c.lr_scale);
    const float keep = __fsub_rn(1.0f, __fmul_rn(lr, c.decay)), size = __fmul_rn(lr, now.inv1);
    const Two scale2 = two(scale, scale), beta1s = two(beta1, beta1), rest1s = two(p.s.rest1, p.s.rest1),
              beta2s = two(p.s.beta2, p.s.beta2), rest2s = two(p.s.rest2, p.s.rest2), inv2s = two(now.inv2, now.inv2),
              epss = two(p.s.eps, p.s.eps), keeps = two(keep, keep), sizes = two(-size, -size);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const Two gj = mul2(two(g[j], g[j + 1]), scale2);
        sum2(mul2(two(m[j], m[j + 1]), beta1s), mul2(gj, rest1s), m[j], m[j + 1]);
        sum2(mul2(two(v[j], v[j + 1]), beta2s), mul2(mul2(gj, gj), rest2s), v[j], v[j + 1]);
        float a, b;
        sum2(mul2(two(root<FAST>(v[j]), root<FAST>(v[j + 1])), inv2s), epss, a, b);
        const Two u = two(quotient<FAST>(m[j], a), quotient<FAST>(m[j + 1], b));
        sum2(mul2(two(x[j], x[j + 1]), keeps), mul2(sizes, u), x[j], x[j + 1]);
    }
    Words<S> ws;
    from_floats(ws, x);
    piece_store<S, AL, FULL>(ws, param, base, lane, head, n);
    if constexpr (MASTER) {
        Words<P> wp;
        from_floats(wp, x);
        piece_store<P, AL, FULL>(wp, static_cast<P *>(c.param), base, lane, head, n);
    }
    if constexpr (EIGHT) {
        // elements past the tensor's last are zeros
        if (!FULL && at + 8 > n) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (at + j >= n) m[j] = v[j] = 0.0f;
        }
        const uint32_t em = fp8_exp<GQ_FP8_E4M3>(block_max(m)), ev = square_exp(block_max(v));
        // Philox's counter (element / 8, step, tensor + 2^31; for the first moment + 2^30 too)
        const uint64_t group = (uint64_t)(c.group + (at >> 3));
        const uint32_t c0 = (uint32_t)group, c2 = now.step;
        const unsigned long long p0 = (unsigned long long)0xD2511F53u * c0, p1 = (unsigned long long)0xCD9E8D57u * c2;
        auto draw = [&](uint32_t which, uint32_t (&w)[4]) {
            const uint4 d = philox_rounds_2_to_10((uint32_t)(p1 >> 32) ^ (uint32_t)(group >> 32) ^ p.rk0[0], (uint32_t)p1,
                                                  (uint32_t)(p0 >> 32) ^ (c.number | which) ^ p.rk1[0], (uint32_t)p0,
                                                  p.rk0 + 1, p.rk1 + 1);
            w[0] = d.x; w[1] = d.y; w[2] = d.z; w[3] = d.w;
        };
        uint32_t w[4];
        uint2 qm;
        if constexpr ((MODE & kSpread) != 0) {
            draw(0xc0000000u, w);
            qm = spread_codes(m, w, em);
        } else {
            qm = fp8_codes8<GQ_FP8_E4M3>(m, em);
        }
        draw(0x80000000u, w);
        const uint2 qv = square_codes(v, w, ev);
        // whole blocks are written, the last one's codes past the tensor as 0
        if (FULL || base + (lane & 16) * 8 < n) {
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(c.m) + at) = qm;
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(c.v) + at) = qv;
            if ((lane & 15) == 0) {
                c.em[at >> 7] = (uint8_t)em;
                c.ev[at >> 7] = (uint8_t)ev;
            }
        }
    } else {
        Words<float> w;
        from_floats(w, m);
        piece_store<float, AL, FULL>(w, static_cast<float *>(c.m), base, lane, head, n);
        from_floats(w, v);
        piece_store<float, AL, FULL>(w, static_cast<float *>(c.v), base, lane, head, n);
    }
}

// Blocks walk the table in strides of the grid.  Entries are fetched two chunks ahead, and with moments in 8 bits the
// elements 256 x 8 ahead: the way from an entry to its elements and back, which a block would wait for twice a chunk,
// is otherwise much of its time (244 us without either, 146 with, 64 tensors of 1e6, bf16 parameters).
// Blocks an SM: three, but two where 8-bit moments leave room for a float32 parameter's and gradient's elements on the
// way only so (184 us against 206; with a bf16 parameter 168 against 146), or where loads that are shifted take more (64
// x 1000001, bf16 parameters: 227 against 268).
constexpr int blocks_of(bool eight, bool al, int updated, int grad) { return eight && (!al || updated + grad == 8) ? 2 : 3; }

template <typename P, typename G, bool MASTER, bool EIGHT, int MODE, bool AL>
__global__ void __launch_bounds__(kThreads, blocks_of(EIGHT, AL, MASTER ? 4 : sizeof(P), sizeof(G))) k_adamw(const __grid_constant__ Params p)
{
    using S = typename std::conditional<MASTER, float, P>::type;  // what is updated
    constexpr int kWords = sizeof(AdamChunk) / 16;
    __shared__ AdamChunk entry[3];
    const int lane = threadIdx.x & 31, first = (int)(threadIdx.x >> 5) * kChunk, tid = threadIdx.x;
    const int64_t step = gridDim.x;
    int64_t i = blockIdx.x;
    auto fetch = [&](int64_t at) { return __ldg(reinterpret_cast<const uint4 *>(p.table + at) + tid); };
    if (tid < kWords) {
        reinterpret_cast<uint4 *>(&entry[0])[tid] = fetch(i);
        if (i + step < p.chunks) reinterpret_cast<uint4 *>(&entry[1])[tid] = fetch(i + step);
    }
    cudaGridDependencySynchronize();  // the table never changes; all else may be written by the kernel before
    const float scale = p.s.scale ? *p.s.scale : 1.0f;
    if (scale != scale) return;
    gq_adamw_scalars_t now = p.s.now;
    if (p.s.scalars) now = *p.s.scalars;
    __syncthreads();
    Loaded<S, G, EIGHT, AL> a;
    auto whole = [](const AdamChunk &c, int base) { return AL && base + kChunk <= c.n && (EIGHT || base >= c.head); };
    auto fetch_elements = [&](Loaded<S, G, EIGHT, AL> &l, const AdamChunk &c, int base) {
        if (whole(c, base)) load<S, G, MASTER, EIGHT, AL, AL>(l, c, base, lane);
        else if (base < c.n) load<S, G, MASTER, EIGHT, AL, false>(l, c, base, lane);
    };
    auto work = [&](const Loaded<S, G, EIGHT, AL> &l, const AdamChunk &c, int base) {
        if (whole(c, base)) update<P, S, G, MASTER, EIGHT, MODE, AL, AL>(p, l, c, now, scale, base, lane);
        else if (base < c.n) update<P, S, G, MASTER, EIGHT, MODE, AL, false>(p, l, c, now, scale, base, lane);
    };
    if (EIGHT) fetch_elements(a, entry[0], first);
    for (int k = 0; i < p.chunks; i += step) {
        const int next = k == 2 ? 0 : k + 1, after = next == 2 ? 0 : next + 1;
        const AdamChunk &c = entry[k];
        uint4 ahead;
        const bool more = i + 2 * step < p.chunks && tid < kWords;
        if (more) ahead = fetch(i + 2 * step);
        if constexpr (EIGHT) {
            Loaded<S, G, EIGHT, AL> b;
            fetch_elements(b, c, first + kHalf);
            work(a, c, first);
            if (i + step < p.chunks) fetch_elements(a, entry[next], first);
            work(b, c, first + kHalf);
        } else {
#pragma unroll 1
            for (int base = first; base < c.n; base += kHalf) {
                fetch_elements(a, c, base);
                work(a, c, base);
            }
        }
        if (more) reinterpret_cast<uint4 *>(&entry[after])[tid] = ahead;
        __syncthreads();
        k = next;
    }
}

// ---------------------------------------------------------------------------------------------
// The moments' values.
// ---------------------------------------------------------------------------------------------
// What a lane has loaded of its 8 elements of a moment.  Those in 32 bits may start elsewhere than the output.
template <bool EIGHT>
struct Moment {
    Raw<float, false> r;
};
template <>
struct Moment<true> {
    uint2 q;
    uint32_t E;
};
template <bool EIGHT>
__device__ __forceinline__ void load(Moment<EIGHT> &l, const void *x, const uint8_t *exps, int n, int base, int lane)
{
    if constexpr (EIGHT) {
        const int at = base + lane * 8;
        l.q = make_uint2(0u, 0u);
        l.E = 32;
        if (at < n) {
            l.q = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(x) + at));
            l.E = __ldg(exps + (at >> 7));
        }
    } else {
        chunk_load<float, false>(l.r, static_cast<const float *>(x), base, lane, n);
    }
}
template <typename T, bool EIGHT, bool AL>
__device__ __forceinline__ void put(const Moment<EIGHT> &l, const AdamChunk &c, bool second, int base, int lane, void *m, void *v)
{
    void *const out = second ? v : m;
    if (!out) return;
    float x[8];
    if constexpr (!EIGHT) to_floats(in_place<float, false>(l.r, static_cast<const float *>(second ? c.v : c.m)), x);
    else if (second) square_values(l.q, l.E, x);
    else fp8_decode8<GQ_FP8_E4M3>(l.q, fp8_scale(l.E), x);
    saturate<T>(x);
    Words<T> w;
    from_floats(w, x);
    chunk_store<T, AL>(w, static_cast<T *>(out) + c.start, base, lane, c.n);
}

// Registers for as many warps as an SM holds: at 47 instead of 32 the 8-bit form takes 95 us instead of 75 (64 x 1e6).
template <typename T, bool EIGHT>
__global__ void __launch_bounds__(kThreads, EIGHT ? 8 : 6) k_moments(const __grid_constant__ Params p, void *m, void *v)
{
    AdamChunk c = p.table[blockIdx.x];
    if constexpr (!EIGHT) {
        c.m = static_cast<float *>(c.m) + c.head;
        c.v = static_cast<float *>(c.v) + c.head;
        c.n -= c.head;
        c.start += c.head;
    }
    cudaGridDependencySynchronize();
    const int lane = threadIdx.x & 31;
    const bool al = c.start % (16 / (int)sizeof(T)) == 0;
    for (int base = (int)(threadIdx.x >> 5) * kChunk; base < c.n; base += kHalf) {
        Moment<EIGHT> l[2];
        if (m) load<EIGHT>(l[0], c.m, c.em, c.n, base, lane);
        if (v) load<EIGHT>(l[1], c.v, c.ev, c.n, base, lane);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (al) put<T, EIGHT, true>(l[w], c, w == 1, base, lane, m, v);
            else put<T, EIGHT, false>(l[w], c, w == 1, base, lane, m, v);
        }
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
struct Grads {
    Raw<G, AL> r[2];
    const G *at;
    __device__ __forceinline__ void load(const AdamChunk &c, int first, int lane)
    {
        at = static_cast<const G *>(c.grad);
        piece_load<G, AL, false>(r[0], at, first, lane, c.head, c.n);
        chunk_load<G, AL>(r[1], at, first + kHalf, lane, c.n);
    }
    __device__ __forceinline__ double squares() const
    {
        double s[2] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float g[8];
            to_floats(in_place<G, AL>(r[h], at), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[h] = __fma_rn((double)g[j], (double)g[j], s[h]);
        }
        return s[0] + s[1];
    }
};

// The squares of the chunks i, i + gridDim.x, ... before `end`; i is left at the first behind.  A chunk's gradients are
// on their way while the one before is summed, and its table entry an iteration longer (64 x 4194304: float32 178 us
// without, 151 with, bf16 138 and 88).
template <typename G, bool AL>
__device__ __forceinline__ double walk(const AdamChunk *table, int64_t &i, int64_t end, int first, int lane)
{
    if (i >= end) return 0.0;
    const int64_t step = gridDim.x;
    double s = 0.0;
    Grads<G, AL> now, next;
    now.load(table[i], first, lane);
    AdamChunk c = table[i + step < end ? i + step : i];
    for (;;) {
        i += step;
        const bool more = i < end;
        if (more) {
            next.load(c, first, lane);
            if (i + step < end) c = table[i + step];
        }
        s += now.squares();
        if (!more) return s;
        now = next;
    }
}

template <typename G>
__global__ void __launch_bounds__(kThreads, kNormPerSm) k_norm(const AdamChunk *table, int64_t aligned, int64_t chunks, double *parts)
{
    __shared__ double shared[kThreads / 32];
    const int lane = threadIdx.x & 31, first = (int)(threadIdx.x >> 5) * kChunk;
    cudaGridDependencySynchronize();
    int64_t i = blockIdx.x;
    double s = walk<G, true>(table, i, aligned, first, lane);
    s += walk<G, false>(table, i, chunks, first, lane);
    s = block_sum(s, shared);
    if (threadIdx.x == 0) parts[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads) k_norm_join(const double *parts, int n, double max_norm, float *out)
{
    __shared__ double shared[kThreads / 32];
    cudaGridDependencySynchronize();
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) s += parts[i];
    s = block_sum(s, shared);
    if (threadIdx.x == 0) {
        const double norm = sqrt(s), f = norm > max_norm ? max_norm / norm : 1.0;
        out[0] = (float)norm;
        out[1] = norm <= 1.7e308 ? (float)f : __uint_as_float(0x7fffffffu);
    }
}

// Launched to start as the kernel before it on the stream drains: these kernels follow one another, some of a few
// microseconds, and each waits for the one before by itself.
template <typename... A, typename... B>
cudaError_t launch_after(void (*kern)(A...), unsigned grid, cudaStream_t s, B... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename P, typename G, bool MASTER, bool EIGHT, int MODE, bool AL>
cudaError_t launch_part(Params p, int64_t first, int64_t chunks, cudaStream_t s)
{
    if (chunks == 0) return cudaSuccess;
    auto kern = k_adamw<P, G, MASTER, EIGHT, MODE, AL>;
    int per_sm = 0, sms = 0;
    const cudaError_t e = kernel_occupancy(reinterpret_cast<const void *>(kern), kThreads, 0, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    p.table += first;
    p.chunks = chunks;
    // 32 bits: a block a chunk, replaced by the next as it ends (268 us against 286 for a grid that stays, 64 x 1e6)
    const int64_t most = EIGHT ? (int64_t)per_sm * sms : chunks;
    return launch_after(kern, (unsigned)(chunks < most ? chunks : most), s, p);
}
template <typename P, typename G, bool MASTER, bool EIGHT, int MODE>
cudaError_t launch_parts(const AdamArgs &a, const Params &p, cudaStream_t s)
{
    const cudaError_t e = launch_part<P, G, MASTER, EIGHT, MODE, true>(p, 0, a.aligned, s);
    return e != cudaSuccess ? e : launch_part<P, G, MASTER, EIGHT, MODE, false>(p, a.aligned, a.chunks - a.aligned, s);
}
template <typename P, typename G, bool MASTER>
cudaError_t launch_state(const AdamArgs &a, const Params &p, cudaStream_t s)
{
    if (a.state_bits != 8) return launch_parts<P, G, MASTER, false, 0>(a, p, s);
    if (p.s.spread)
        return p.s.fast ? launch_parts<P, G, MASTER, true, kSpread | kFast>(a, p, s) : launch_parts<P, G, MASTER, true, kSpread>(a, p, s);
    return p.s.fast ? launch_parts<P, G, MASTER, true, kFast>(a, p, s) : launch_parts<P, G, MASTER, true, 0>(a, p, s);
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
    return launch_after(a.state_bits == 8 ? k_moments<T, true> : k_moments<T, false>, (unsigned)a.chunks, s, p, m, v);
}

Params params_of(const AdamArgs &a)
{
    Params p = {};
    p.table = a.table;
    p.chunks = a.chunks;
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
        auto kern = a.grad_dtype == GQ_FLOAT32 ? k_norm<float> : a.grad_dtype == GQ_BFLOAT16 ? k_norm<__nv_bfloat16> : k_norm<__half>;
        const cudaError_t e = launch_after(kern, grid, s, a.table, a.aligned, a.chunks, parts);
        if (e != cudaSuccess) return e;
    }
    return launch_after(k_norm_join, 1, s, (const double *)parts, (int)grid, max_norm, out);
}

}  // namespace gq
