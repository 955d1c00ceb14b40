// gq_fp8.cu -- packing matrices into 8-bit floating point along their rows and columns, and back.
//
// A block's exponent needs its largest value before its first code, so the 128 values wait in registers: along rows in
// the 16 lanes that loaded them, along columns in a tile of 128 x 128 that a block holds, whose codes leave by way of
// shared memory.  Bounded by bytes and by latency; 16384 x 8192 bf16, along rows 68 us, along columns 67, both 97, in
// tiles both ways 85, back 64, where the bytes take 62, 62, 82, 82 and 62; a row of 16384 x 4095 whose start is not
// aligned takes up to 1.6 times as long.
#include "gq_act.cuh"
#include "gq_device.cuh"
#include "gq_fp8.cuh"
#include "gq_fp8.h"

namespace gq {
namespace {

// A packed matrix in memory.
struct Packed {
    uint8_t *codes, *exps;
    int64_t code_pitch, exp_pitch;
    int blocks;  // of a row
};
Packed packed_of(void *p, int tile, int64_t rows, int64_t cols)
{
    const Fp8Layout l = fp8_layout(tile, rows, cols);
    uint8_t *b = static_cast<uint8_t *>(p);
    return Packed{b, b ? b + l.exps_off : nullptr, l.code_pitch, l.exp_pitch, (int)((cols + 127) / 128)};
}

struct Params {
    const void *x;
    int64_t sx, rows;
    int cols, per_row;  // items a row
    Packed p, t;        // along the rows, along the columns
};

// Largest absolute values: bits of binary32, or two 16-bit patterns in a word, which order like integers.
template <typename T>
__device__ __forceinline__ uint32_t abs_word(uint32_t w)
{
    return w & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu);
}
template <typename T>
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b)
{
    if constexpr (sizeof(T) == 4) return max(a, b);
    else return max_u16x2(a, b);
}
// Binary32 bits of a pattern (the low 16 bits of a word for 16-bit types).
template <typename T>
__device__ __forceinline__ uint32_t float_bits(uint32_t b)
{
    if constexpr (sizeof(T) == 4) return b;
    else if constexpr (__is_same(T, __half)) return __float_as_uint(__half2float(__ushort_as_half((unsigned short)b)));
    else return b << 16;
}
// Of a lane's words of one row: the largest of the 128 columns that its 16 lanes hold, as binary32 bits.
template <typename T>
__device__ __forceinline__ uint32_t row_max(const Words<T> &w)
{
    uint32_t m = abs_word<T>(w.w[0]);
#pragma unroll
    for (int i = 1; i < (int)(2 * sizeof(T)); ++i) m = max_word<T>(m, abs_word<T>(w.w[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_word<T>(m, __shfl_xor_sync(kFull, m, o));
    return float_bits<T>(sizeof(T) == 4 ? m : max(m & 0xffffu, m >> 16));
}

// Columns 2 k and 2 k + 1 of a lane's 8.
template <typename T>
__device__ __forceinline__ void two_floats(const Words<T> &w, int k, float &a, float &b)
{
    if constexpr (sizeof(T) == 4) {
        a = __uint_as_float(w.w[2 * k]);
        b = __uint_as_float(w.w[2 * k + 1]);
    } else if constexpr (__is_same(T, __half)) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w.w[k]));
        a = f.x;
        b = f.y;
    } else {
        a = __uint_as_float(w.w[k] << 16);
        b = __uint_as_float(w.w[k] & 0xffff0000u);
    }
}

// A lane's 8 codes of a row, its block's exponent, and, behind the row's last block, the exponents' padding.
__device__ __forceinline__ void store_row(const Packed &p, int64_t row, int64_t exp_row, int base, int lane, uint2 q, uint32_t E,
                                          bool exps)
{
    const int c = base + lane * 8;
    if (c >= p.code_pitch) return;
    *reinterpret_cast<uint2 *>(p.codes + row * p.code_pitch + c) = q;
    if (exps && (lane & 15) == 0) {
        uint8_t *e = p.exps + exp_row * p.exp_pitch;
        const int b = c >> 7;
        e[b] = (uint8_t)E;
        if (b + 1 == p.blocks)
            for (int i = b + 1; i < p.exp_pitch; ++i) e[i] = 0;
    }
}

// ---------------------------------------------------------------------------------------------
// Along the rows only: a warp takes up to N chunks of 256 columns of a row at a time, all loaded before the first is
// used.  One where there are no more chunks than warps that the device holds (16 x 4096 bf16: 2.0 us against 2.8 with
// four), else four (16384 x 8192: 67 us against 92 with one).
// ---------------------------------------------------------------------------------------------
constexpr int kAhead = 4;
constexpr int64_t kFewChunks = 148 * 16 * 2;

template <typename T, int FMT, bool AL, bool FULL, int N>
__device__ __forceinline__ void pack_item(const Params &p, int64_t row, int base, int lane)
{
    const T *const x = static_cast<const T *>(p.x) + row * p.sx;
    Raw<T, AL> r[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        if (!FULL && u > 0 && base + u * kChunk >= p.cols) break;
        chunk_load<T, AL, FULL>(r[u], x, base + u * kChunk, lane, p.cols);
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
        if (!FULL && u > 0 && base + u * kChunk >= p.cols) break;
        const Words<T> w = in_place<T, AL>(r[u], x);
        const uint32_t E = fp8_exp<FMT>(row_max<T>(w));
        float v[8];
        to_floats(w, v);
        store_row(p.p, row, row, base + u * kChunk, lane, fp8_codes8<FMT>(v, E), E, true);
    }
}

template <typename T, int FMT, bool AL, int N>
__global__ void __launch_bounds__(256) k_pack_rows(const __grid_constant__ Params p)
{
    const int lane = threadIdx.x & 31;
    const int64_t n = p.rows * p.per_row, warps = (int64_t)gridDim.x * 8;
    for (int64_t id = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); id < n; id += warps) {
        const int64_t row = id / p.per_row;
        const int base = (int)(id - row * p.per_row) * (N * kChunk);
        if (AL && base + N * kChunk <= p.cols) pack_item<T, FMT, AL, AL, N>(p, row, base, lane);
        else pack_item<T, FMT, AL, false, N>(p, row, base, lane);
    }
}

// ---------------------------------------------------------------------------------------------
// 128 rows x 128 columns a block: along the columns, along both, and square tiles.  Half a warp takes 8 rows, a lane 8
// columns of them, so that a lane's 8 codes of a column are one 8-byte piece of the transpose.  A block loads, finds its
// largest values, and stores, with barriers between: as many blocks an SM as registers allow hide that from one another
// (16384 x 8192 bf16 both ways: 130 us with two blocks of 512 threads on 256 columns, 97 with three of these; with four
// 103, their registers spilled).  Two where an element has 32 bits or rows start anywhere: a lane's loads take more
// registers (16384 x 4095 bf16 in tiles both ways: 64 us with two, 77 with three).
// ---------------------------------------------------------------------------------------------
constexpr int kTileWarps = 8;

// Exponents of the 8 rows that 16 lanes hold 8 columns each of: byte i of the two words is row i's.  Lanes keep half of
// the rows at each of the first steps, so that 5 exchanges (8 of binary32) find all largest values instead of 32, and an
// exponent is formed once, not by all 16 lanes.
template <typename T, int FMT>
__device__ __forceinline__ void row_exps(const Words<T> (&w)[8], uint32_t (&e)[2])
{
    constexpr int W = 2 * (int)sizeof(T);
    const int lane = threadIdx.x & 31;
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m[i] = abs_word<T>(w[i].w[0]);
#pragma unroll
        for (int k = 1; k < W; ++k) m[i] = max_word<T>(m[i], abs_word<T>(w[i].w[k]));
    }
    auto halve = [&](uint32_t a, uint32_t b, int bit) {  // lanes with the bit keep b
        const uint32_t keep = (lane & bit) ? b : a, send = (lane & bit) ? a : b;
        return max_word<T>(keep, __shfl_xor_sync(kFull, send, bit));
    };
    uint32_t E;
    if constexpr (sizeof(T) == 2) {
        uint32_t p[4];  // rows 2 k and 2 k + 1 in a word
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = max_u16x2(__byte_perm(m[2 * k], m[2 * k + 1], 0x5410), __byte_perm(m[2 * k], m[2 * k + 1], 0x7632));
        uint32_t q = halve(halve(p[0], p[2], 8), halve(p[1], p[3], 8), 4);
        q = max_u16x2(q, __shfl_xor_sync(kFull, q, 2));
        q = max_u16x2(q, __shfl_xor_sync(kFull, q, 1));
        E = fp8_exp<FMT>(float_bits<T>(q & 0xffffu)) | fp8_exp<FMT>(float_bits<T>(q >> 16)) << 8;
        // lanes 8 (k / 2) + 4 (k mod 2) have rows 2 k and 2 k + 1
        const int from = lane & 16;
        e[0] = __shfl_sync(kFull, E, from) | __shfl_sync(kFull, E, from | 4) << 16;
        e[1] = __shfl_sync(kFull, E, from | 8) | __shfl_sync(kFull, E, from | 12) << 16;
    } else {
        uint32_t a[4], b[2];
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] = halve(m[k], m[k + 4], 8);
#pragma unroll
        for (int k = 0; k < 2; ++k) b[k] = halve(a[k], a[k + 2], 4);
        uint32_t q = halve(b[0], b[1], 2);
        q = max(q, __shfl_xor_sync(kFull, q, 1));
        E = fp8_exp<FMT>(q);
        // lanes 8 (i / 4) + 4 (i / 2 mod 2) + 2 (i mod 2) have row i
        e[0] = e[1] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i >> 2] |= __shfl_sync(kFull, E, (lane & 16) | (i >> 2) << 3 | (i >> 1 & 1) << 2 | (i & 1) << 1) << (8 * (i & 3));
    }
}

template <typename T, int FMT, bool TILE, bool AL, bool FULL>
__device__ __forceinline__ void pack_tile(const Params &p, uint8_t *codes, uint8_t *exps)
{
    constexpr int W = 2 * (int)sizeof(T);  // words of a lane's 8 columns
    uint32_t *const most = reinterpret_cast<uint32_t *>(codes);  // the halves' largest values, before the codes
    const int lane = threadIdx.x & 15, piece = threadIdx.x >> 4;  // of 8 rows
    const int64_t tile = blockIdx.x / p.per_row;
    const int base = (int)(blockIdx.x - tile * p.per_row) * kBlock;
    const int64_t row0 = tile * kBlock + piece * 8;

    Words<T> w[8];
    {
        Raw<T, AL> r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const T *const x = static_cast<const T *>(p.x) + (row0 + i) * p.sx;
            if (FULL || row0 + i < p.rows) {
                chunk_load<T, AL, FULL>(r[i], x, base, lane, p.cols);
            } else {
#pragma unroll
                for (int k = 0; k < (int)(sizeof(r[i].w) / 4); ++k) r[i].w[k] = 0u;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = in_place<T, AL>(r[i], static_cast<const T *>(p.x) + (row0 + i) * p.sx);
    }

    uint32_t col[W];  // largest of the 8 rows
#pragma unroll
    for (int k = 0; k < W; ++k) {
        col[k] = abs_word<T>(w[0].w[k]);
#pragma unroll
        for (int i = 1; i < 8; ++i) col[k] = max_word<T>(col[k], abs_word<T>(w[i].w[k]));
    }
    if constexpr (TILE) {
        Words<T> c;
#pragma unroll
        for (int k = 0; k < W; ++k) c.w[k] = col[k];
        const uint32_t m = row_max<T>(c);
        if (lane == 0) most[piece] = m;
    } else {
#pragma unroll
        for (int k = 0; k < W; ++k) most[(piece * W + k) * 16 + lane] = col[k];
    }
    __syncthreads();
    uint32_t E = 0;
    if constexpr (TILE) {
        if (threadIdx.x == 0) {
            uint32_t m = 0;
            for (int i = 0; i < 2 * kTileWarps; ++i) m = max(m, most[i]);
            E = fp8_exp<FMT>(m);
        }
    } else if (threadIdx.x < kBlock) {
        // column 8 l + j: word j (or half of word j / 2) of lane l
        const int l = threadIdx.x >> 3, j = threadIdx.x & 7;
        uint32_t m = 0;
        for (int i = 0; i < 2 * kTileWarps; ++i) m = max_word<T>(m, most[(i * W + (sizeof(T) == 4 ? j : j >> 1)) * 16 + l]);
        if (sizeof(T) == 2) m = (j & 1) ? m >> 16 : m & 0xffffu;
        E = fp8_exp<FMT>(float_bits<T>(m));
    }
    if (threadIdx.x < (TILE ? 1 : kBlock)) {
        exps[threadIdx.x] = (uint8_t)E;
        if (p.t.codes) {
            // the transpose's row: the column (TILE: 128 of them), its block: this one's rows
            const int64_t r = TILE ? base / kBlock : base + threadIdx.x;
            if (TILE || r < p.cols) {
                uint8_t *e = p.t.exps + r * p.t.exp_pitch;
                e[tile] = (uint8_t)E;
                if (tile + 1 == p.t.blocks)
                    for (int64_t i = tile + 1; i < p.t.exp_pitch; ++i) e[i] = 0;
            }
        }
    }
    __syncthreads();

    if (p.p.codes) {
        uint32_t of_rows[2] = {};
        if constexpr (!TILE) row_exps<T, FMT>(w, of_rows);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t e = TILE ? exps[0] : of_rows[i >> 2] >> (8 * (i & 3)) & 0xffu;
            float v[8];
            to_floats(w[i], v);
            const uint2 q = fp8_codes8<FMT>(v, e);
            if (FULL || row0 + i < p.rows)
                store_row(p.p, row0 + i, TILE ? tile : row0 + i, base, lane, q, e, !TILE || (piece == 0 && i == 0));
        }
    }
    if (!p.t.codes) return;
    // Piece i (8 rows) of column c lies at piece i ^ (c / 8 mod 16) of its 128 bytes: the 16 lanes that store a piece, 8
    // columns apart, then store to different banks.
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float x[2][8];  // columns 2 k and 2 k + 1
#pragma unroll
        for (int i = 0; i < 8; ++i) two_floats<T>(w[i], k, x[0][i], x[1][i]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = lane * 8 + 2 * k + h;
            const uint32_t e = exps[TILE ? 0 : c];
            *reinterpret_cast<uint2 *>(codes + c * kBlock + ((piece ^ lane) << 3)) = fp8_codes8<FMT>(x[h], e);
        }
    }
    __syncthreads();
    // 16-byte pieces, two of 8, in order; a column's 128 bytes by 8 lanes
#pragma unroll
    for (int i = threadIdx.x; i < kBlock * 8; i += kTileWarps * 32) {
        const int c = i >> 3, f = (c >> 3) & 15, at = (i & 7) * 2;
        if (!FULL && base + c >= p.cols) break;
        uint4 q = *reinterpret_cast<const uint4 *>(codes + c * kBlock + (((at ^ f) & 14) << 3));
        if (f & 1) q = make_uint4(q.z, q.w, q.x, q.y);
        *reinterpret_cast<uint4 *>(p.t.codes + (int64_t)(base + c) * p.t.code_pitch + tile * kBlock + at * 8) = q;
    }
}

template <typename T, int FMT, bool TILE, bool AL>
__global__ void __launch_bounds__(kTileWarps * 32, sizeof(T) == 4 || !AL ? 2 : 3) k_pack_tile(const __grid_constant__ Params p)
{
    __shared__ __align__(16) uint8_t codes[kBlock * kBlock];  // transposed
    __shared__ uint8_t exps[kBlock];                          // of every column (TILE: the first, of all)
    const int64_t tile = blockIdx.x / p.per_row;
    const int base = (int)(blockIdx.x - tile * p.per_row) * kBlock;
    const bool whole = AL ? base + kBlock <= p.cols : base > 0 && base + kBlock + 8 <= p.cols;
    if (whole && (tile + 1) * kBlock <= p.rows) pack_tile<T, FMT, TILE, AL, true>(p, codes, exps);
    else pack_tile<T, FMT, TILE, AL, false>(p, codes, exps);
}

template <typename T, int FMT, bool TILE, bool AL, bool FULL>
__device__ __forceinline__ void unpack_item(const Params &p, T *out, int64_t row, int base, int lane)
{
    const uint8_t *const codes = p.p.codes + row * p.p.code_pitch;
    const uint8_t *const exps = p.p.exps + (TILE ? row / kBlock : row) * p.p.exp_pitch;
    uint2 q[kAhead];
    uint32_t E[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
        const int c = base + u * kChunk + lane * 8;
        q[u] = make_uint2(0u, 0u);
        E[u] = 0;
        if (FULL || c < p.cols) {
            q[u] = __ldg(reinterpret_cast<const uint2 *>(codes + c));
            E[u] = __ldg(exps + (c >> 7));
        }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
        if (!FULL && u > 0 && base + u * kChunk >= p.cols) break;
        float v[8];
        fp8_decode8<FMT>(q[u], fp8_scale_any(E[u]), v);
        saturate<T>(v);
        Words<T> w;
        from_floats(w, v);
        chunk_store<T, AL, FULL>(w, out + row * p.sx, base + u * kChunk, lane, p.cols);
    }
}

template <typename T, int FMT, bool TILE, bool AL>
__global__ void __launch_bounds__(256) k_unpack(const __grid_constant__ Params p, T *out)
{
    const int lane = threadIdx.x & 31;
    const int64_t n = p.rows * p.per_row, warps = (int64_t)gridDim.x * 8;
    for (int64_t id = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); id < n; id += warps) {
        const int64_t row = id / p.per_row;
        const int base = (int)(id - row * p.per_row) * (kAhead * kChunk);
        if (base + kAhead * kChunk <= p.cols) unpack_item<T, FMT, TILE, AL, true>(p, out, row, base, lane);
        else unpack_item<T, FMT, TILE, AL, false>(p, out, row, base, lane);
    }
}

template <typename T>
bool rows_aligned(const Params &p) { return p.rows <= 1 || p.sx % (16 / (int64_t)sizeof(T)) == 0; }

bool few_chunks(int64_t rows, int64_t cols) { return rows * ((cols + kChunk - 1) / kChunk) <= kFewChunks; }

unsigned warp_grid(const Params &p)
{
    const int64_t need = (p.rows * p.per_row + 7) / 8;
    return (unsigned)(need < 148 * 16 ? need : 148 * 16);
}

template <typename T, int FMT>
cudaError_t pack(const Params &p, int tile, cudaStream_t s)
{
    const bool al = rows_aligned<T>(p);
    if (!tile && !p.t.codes) {
        if (few_chunks(p.rows, p.cols)) {
            if (al) k_pack_rows<T, FMT, true, 1><<<warp_grid(p), 256, 0, s>>>(p);
            else k_pack_rows<T, FMT, false, 1><<<warp_grid(p), 256, 0, s>>>(p);
        } else {
            if (al) k_pack_rows<T, FMT, true, kAhead><<<warp_grid(p), 256, 0, s>>>(p);
            else k_pack_rows<T, FMT, false, kAhead><<<warp_grid(p), 256, 0, s>>>(p);
        }
        return cudaGetLastError();
    }
    const int64_t blocks = (p.rows + kBlock - 1) / kBlock * p.per_row;
    if (blocks > (int64_t(1) << 31) - 1) return cudaErrorInvalidConfiguration;
    const unsigned grid = (unsigned)blocks, threads = kTileWarps * 32;
    if (tile) {
        if (al) k_pack_tile<T, FMT, true, true><<<grid, threads, 0, s>>>(p);
        else k_pack_tile<T, FMT, true, false><<<grid, threads, 0, s>>>(p);
    } else {
        if (al) k_pack_tile<T, FMT, false, true><<<grid, threads, 0, s>>>(p);
        else k_pack_tile<T, FMT, false, false><<<grid, threads, 0, s>>>(p);
    }
    return cudaGetLastError();
}

template <typename T, int FMT>
cudaError_t unpack(const Params &p, int tile, T *out, cudaStream_t s)
{
    const bool al = rows_aligned<T>(p);
    if (tile) {
        if (al) k_unpack<T, FMT, true, true><<<warp_grid(p), 256, 0, s>>>(p, out);
        else k_unpack<T, FMT, true, false><<<warp_grid(p), 256, 0, s>>>(p, out);
    } else {
        if (al) k_unpack<T, FMT, false, true><<<warp_grid(p), 256, 0, s>>>(p, out);
        else k_unpack<T, FMT, false, false><<<warp_grid(p), 256, 0, s>>>(p, out);
    }
    return cudaGetLastError();
}

// width: columns of an item
Params params_of(const Fp8PackArgs &a, int width)
{
    Params p = {};
    p.x = a.x.p;
    p.sx = a.rows > 1 ? a.x.stride : 0;
    p.rows = a.rows;
    p.cols = (int)a.cols;
    p.per_row = (int)((a.cols + width - 1) / width);
    p.p = packed_of(a.packed, a.tile, a.rows, a.cols);
    p.t = packed_of(a.packed_t, a.tile, a.cols, a.rows);
    return p;
}

template <typename T>
cudaError_t pack_type(const Fp8PackArgs &a, cudaStream_t s)
{
    const Params p = params_of(a, a.tile || a.packed_t ? kBlock : few_chunks(a.rows, a.cols) ? kChunk : kAhead * kChunk);
    return a.format == GQ_FP8_E4M3 ? pack<T, GQ_FP8_E4M3>(p, a.tile, s) : pack<T, GQ_FP8_E5M2>(p, a.tile, s);
}
template <typename T>
cudaError_t unpack_type(const Fp8PackArgs &a, cudaStream_t s)
{
    const Params p = params_of(a, kAhead * kChunk);
    T *const out = static_cast<T *>(const_cast<void *>(a.x.p));
    return a.format == GQ_FP8_E4M3 ? unpack<T, GQ_FP8_E4M3>(p, a.tile, out, s) : unpack<T, GQ_FP8_E5M2>(p, a.tile, out, s);
}

}  // namespace

cudaError_t launch_fp8_pack(const Fp8PackArgs &a, cudaStream_t s)
{
    if (a.dtype == GQ_FLOAT32) return pack_type<float>(a, s);
    if (a.dtype == GQ_BFLOAT16) return pack_type<__nv_bfloat16>(a, s);
    return pack_type<__half>(a, s);
}

cudaError_t launch_fp8_unpack(const Fp8PackArgs &a, cudaStream_t s)
{
    if (a.dtype == GQ_FLOAT32) return unpack_type<float>(a, s);
    if (a.dtype == GQ_BFLOAT16) return unpack_type<__nv_bfloat16>(a, s);
    return unpack_type<__half>(a, s);
}

}  // namespace gq
