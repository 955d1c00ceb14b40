// gq_wgrad.cu -- a linear layer's weight gradient from its input's 8-bit checkpoint:
//   dw[n][k] = sum over tokens t of dy[t][n] * xh[t][k],  xh the decoded input,
// and its bias gradient db[n] = sum over t of dy[t][n].
//
// The contraction runs over the tokens, which is the outer axis of both operands, so both are fed to the
// tensor cores "MN-major": 64 columns (128 bytes) by 8 tokens form one swizzled block of shared memory,
// and no operand is transposed on the way.  One tcgen05.mma (kind::f16, cta_group::2) makes a 256 x 256
// tile of dw^T over 16 tokens, binary32 sums in TMEM:
//   A  256 k: decoded from int8 in shared memory, 128 k by each CTA of the pair;
//   B  256 n: dy as it is, 128 n in each CTA.
// Decoding is exact (q * 2^e has 7 significant bits), so the products are too, and rounding happens in
// the binary32 sums only.  A is the decoded operand because the M side holds 128 columns a CTA however
// wide the tile is: a stage's 64 x 128 codes cost some 250 issue slots of each scheduler, under the 512
// cycles that its four MMAs take.
//
// Bounded for long batches by shared memory, through which 80 KB a stage pass in each CTA: B and the codes in
// (24), the codes out (8), A in (16), the MMAs' operands out (32); at 128 bytes a cycle 640 cycles, where the
// MMAs take 512 and a stage some 700.  Fetching the codes into registers instead leaves 64 KB, but the signal
// that A is decoded then waits for the loads ahead (twice the time).  For few tokens bounded by the bytes of dw.
// Measured, bf16, in graphs of ten calls: 8192 tokens, 4096 x 4096 226 us (1.22 PFLOP/s); 16384 tokens, 4096 x 16384
// 1.73 ms (1.27, 78 % of the library's measured peak); 64 tokens, 4096 x 4096 21 us.  In a long run of calls, under
// the power cap, 267 us (1.03) and 2.01 ms (1.09).  gq_act_unpack and a library product after it, which round the sums
// less well and need the decoded tensor, take 186 us, 1.33 ms and 12 us in the same graphs.
//
// A few tokens of a small layer go to a kernel of their own, k_few.
//
// float32 gradients are cut into three bf16 planes (8 significant bits each, by truncation) by a pass before, and
// the contraction runs over 3 x tokens.  The planes add up to the gradient exactly, but for what lies below bf16's
// smallest value, 2^-133, which is cut off (gradients under 2^-110 may have such bits).  Rows that TMA cannot
// fetch (a stride that is no multiple of 16 bytes, or rows that overlap) are copied to aligned ones.
#include "gq_act.cuh"
#include "gq_act.h"
#include "gq_device.cuh"
#include "gq_internal.h"
#include "gq_ring.cuh"
#include "gq_tc.cuh"

namespace gq {
namespace {

constexpr int kTile = 256;               // tile of k and of n, per CTA pair
constexpr int kHalf = 128;               // k rows, and n columns, of one CTA
constexpr int kTok = 64;                 // tokens of a stage
constexpr int kABytes = kHalf * kTok * 2;
constexpr int kBBytes = kHalf * kTok * 2;
constexpr int kCodeBytes = kHalf * kTok;
constexpr int kExpBytes = kTok * 4;      // four groups' exponents of every token
constexpr int kBlockBytes = kTok * 128;  // 64 columns x 64 tokens of a 16-bit operand
constexpr int kStageBytes = kABytes + kBBytes + kCodeBytes;
constexpr int kSmemBytes = kStages * (kStageBytes + kExpBytes) + 1024;
// Stages summed in TMEM before their sums are added to registers.  The tensor cores' binary32 sums round
// toward zero, 16 products at a time: over 8192 tokens they came out 7e-6 small (relative), over 16384
// 1.6e-5, where a chain rounded to nearest is off by 1e-6.  512 tokens lose 4e-7, and sums of such runs,
// rounded to nearest, keep that.
constexpr int kRun = 8;
// Warps: 4 of control (copies, MMA, exponents, one idle), 8 of epilogue, 8 that decode.  The epilogue holds
// 128 sums in each thread's registers, more than an even split gives: see kRegs*.
constexpr int kCtlWarps = 4, kEpiWarps = 8, kConvWarps = 8;
constexpr int kThreads = (kCtlWarps + kEpiWarps + kConvWarps) * 32;
constexpr int kRegsLaunch = 96, kRegsCtl = 48, kRegsEpi = 168, kRegsConv = 48;
static_assert(kCtlWarps * kRegsCtl + kEpiWarps * kRegsEpi + kConvWarps * kRegsConv <= kThreads / 32 * kRegsLaunch,
              "setmaxnreg: the shares come from the block's own registers at launch");
constexpr int kPairs = 74;               // CTA pairs of the 148 SMs: the schedule is made for these

// How the tiles are spread over the pairs: whole rounds of a tile a pair first; the stages of the last, partial
// round's tiles are one line, tile after tile, cut into `ranges` equal ranges, one a pair.  A range's part of a
// tile goes to the workspace, where a second kernel joins them, unless it is the whole tile.
struct Schedule {
    int tiles_k, tiles_n;
    int64_t whole, cut;  // tiles of the whole rounds; tiles of the last
    int pairs, ranges;   // pairs launched; of them, those with a range
    int64_t blocks;      // stages of a tile: planes x ceil(tokens / 64)
    int64_t tok_blocks;  // ceil(tokens / 64)
    // from here on worked out before the launch: divisions of 64 bits in every thread took 5 us a call
    int64_t start[kPairs + 1];               // each range's first stage, counted from the first cut tile's first
    uint8_t tile[kPairs];                    // the cut tile that it lies in
    uint8_t from[kPairs], to[kPairs];        // the ranges of each cut tile's first and last stage
};

struct Params {
    CUtensorMap codes, dy;
    Schedule s;
    int64_t tokens;
    int in, out;
    Ckpt k;
    float *dw;
    int64_t sdw;
    int accumulate;
    float *parts;
    long long limit;          // cycles after which a wait gives up
};

Schedule schedule(int dtype, int64_t tokens, int64_t in, int64_t out)
{
    Schedule s;
    s.tiles_k = (int)((in + kTile - 1) / kTile);
    s.tiles_n = (int)((out + kTile - 1) / kTile);
    s.tok_blocks = (tokens + kTok - 1) / kTok;
    s.blocks = s.tok_blocks * (dtype == GQ_FLOAT32 ? 3 : 1);
    const int64_t tiles = (int64_t)s.tiles_k * s.tiles_n;
    s.cut = tiles % kPairs;
    s.whole = tiles - s.cut;
    s.ranges = (int)s.cut;
    if (s.cut) {
        // A tile a pair, as many equal parts of every tile as there are pairs for, or equal ranges for all pairs.
        // A partial tile, written and read again, costs the others' stages about 0.3 of one; the second kernel
        // ten; ranges under 8 stages do not pay.
        const int64_t total = s.cut * s.blocks, most = total / 8 < kPairs ? total / 8 : kPairs;
        double best = (double)s.blocks;
        for (int64_t r = 2 * s.cut; r < most + s.cut; r += s.cut) {
            if (r > most) r = most;
            if (r <= s.cut) break;
            const double parts = r % s.cut == 0 ? (double)r : (double)(s.cut + r - 1);
            const double cost = (double)((total + r - 1) / r) + 0.3 * parts + 10.0;
            if (cost < best) {
                best = cost;
                s.ranges = (int)r;
            }
            if (r == most) break;
        }
    }
    s.pairs = s.whole ? kPairs : s.ranges;
    for (int p = 0; p <= s.ranges; ++p) s.start[p] = s.ranges ? s.cut * s.blocks * p / s.ranges : 0;
    for (int p = 0; p < s.ranges; ++p) s.tile[p] = (uint8_t)(s.start[p] / s.blocks);
    for (int c = 0, p = 0; c < s.cut; ++c) {
        while (s.start[p + 1] <= c * s.blocks) ++p;
        s.from[c] = (uint8_t)p;
        while (s.start[p + 1] < (c + 1) * s.blocks) ++p;
        s.to[c] = (uint8_t)p;
    }
    return s;
}
// Partial tiles that the workspace holds: range p's part of tile c at c + p.
int64_t part_tiles(const Schedule &s) { return s.ranges > s.cut ? s.cut + s.ranges - 1 : 0; }

// ---------------------------------------------------------------------------------------------
// Operands and the MMA
// ---------------------------------------------------------------------------------------------
// Shared-memory operand, MN-major with the 128-byte swizzle: blocks of 64 columns `kBlockBytes` apart,
// groups of 8 tokens 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3fffu) | (uint64_t)(kBlockBytes >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// kind::f16, D binary32, both operands MN-major, M = N = 256.
__device__ __forceinline__ constexpr uint32_t instr_desc(bool bf16)
{
    return 1u << 4 | (bf16 ? 1u : 0u) << 7 | (bf16 ? 1u : 0u) << 10 | 1u << 15 | 1u << 16 | (uint32_t)(kTile >> 3) << 17 |
           (uint32_t)(kTile >> 4) << 24;
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// ---------------------------------------------------------------------------------------------
// Decoding 16 codes of one group.  Of four codes in a word, the even and the odd ones make a pair each
// (a mask instead of a byte permutation), so columns 1 and 2 of every four change places in A; the
// epilogue's threads store them back in order.
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ __nv_bfloat162 bf2(uint32_t x) { return *reinterpret_cast<const __nv_bfloat162 *>(&x); }
__device__ __forceinline__ __half2 h2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t bits2(__nv_bfloat162 x) { return *reinterpret_cast<const uint32_t *>(&x); }
__device__ __forceinline__ uint32_t bits2(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }
// 16-bit lanes holding the codes' bytes, even (i = 0) or odd (i = 1) ones of a word.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i) { return (i ? w >> 8 : w) & 0x00ff00ffu; }

// Exponents whose codes decode16 takes; decode16_any takes all.
template <bool BF16>
__device__ __forceinline__ bool usual(uint32_t E)
{
    return BF16 ? E - 7u <= 245u : E - 109u <= 32u;
}

template <bool BF16>
__device__ __forceinline__ void decode16(const uint4 &codes, uint32_t E, uint32_t (&o)[8])
{
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    if constexpr (BF16) {
        // 2^-126 <= s <= 2^119.  bf16 0x4300 | (q + 128) is 256 + q for q < 0 and 256 + 2 q for q >= 0 (its
        // step doubles at 256).  y = that less 256, times s, is q s or 2 q s; half of y where it is positive,
        // taken off, leaves q s.  Every step is exact.
        const __nv_bfloat162 s = bf2(E * 0x00800080u - 6u * 0x00800080u);
        const __nv_bfloat162 half = __hmul2(s, bf2(0x3f003f00u)), c = __hmul2(s, bf2(0xc380c380u)),
                             hc = __hmul2(s, bf2(0xc300c300u));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 v = bf2(code_pair(w[i >> 1], i & 1) ^ 0x43804380u);
            o[i] = bits2(__hsub2(__hfma2(v, s, c), __hfma2_relu(v, half, hc)));
        }
    } else {
        // 2^-24 <= s <= 2^8.  fp16 0x6400 | m is 1024 + m; (1024 + q + 128) - 1152 is exact, the product with
        // the scale rounds once at most and stays below 65504
        const uint32_t b = E >= 119u ? (E - 118u) << 10 : 1u << (E - 109u);
        const __half2 s = h2(b | b << 16);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[i] = bits2(__hmul2(__hsub2(h2(code_pair(w[i >> 1], i & 1) ^ 0x64806480u), h2(0x64806480u)), s));
    }
}

template <bool BF16>
__device__ __forceinline__ void decode16_any(const uint4 &codes, uint32_t E, uint32_t (&o)[8])
{
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    if constexpr (BF16) {
        // 0x4300 | m is 128 + m for 7 bits m, and q its low 7 bits less 128 times its sign bit: exact, and so
        // is the product with the scale, down to bf16's smallest subnormal
        const uint32_t b = E == 255u ? 0x7fffu : E > 6u ? (E - 6u) << 7 : 0x40u >> (6u - E);
        const __nv_bfloat162 s = bf2(b | b << 16);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t p = code_pair(w[i >> 1], i & 1);
            o[i] = bits2(__hmul2(__hsub2(bf2((p & 0x007f007fu) | 0x43004300u), bf2((p & 0x00800080u) | 0x43004300u)), s));
        }
    } else {
        // also groups beyond fp16's range: below half its smallest step, or saturated, or NaN
        const float s = group_scale(E);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t p = code_pair(w[i >> 1], i & 1);
            float v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float f = (float)(int)(int8_t)(p >> (16 * h)) * s;
                v[h] = f > 65504.0f ? 65504.0f : f < -65504.0f ? -65504.0f : f;
            }
            o[i] = bits2(__floats2half2_rn(v[0], v[1]));
        }
    }
}

// ---------------------------------------------------------------------------------------------
// The kernel: one CTA pair per SM pair, walking work items (whole tiles, then the parts of its range).
// ---------------------------------------------------------------------------------------------
struct Item {
    int tk, tn;              // tile
    int64_t first, last;     // its stages
    int64_t part;            // partial tile in the workspace, -1: the whole tile
};

// Bands of 8 k tiles, walked along n: pairs that run together share their operands in L2.
__device__ __forceinline__ void tile_place(const Schedule &s, int64_t tile, Item &it)
{
    const int64_t band = (int64_t)8 * s.tiles_n;
    const int64_t g = tile / band;
    const int rest = (int)(tile - g * band);
    const int wide = min(8, s.tiles_k - (int)g * 8);
    it.tn = rest / wide;
    it.tk = (int)g * 8 + rest - it.tn * wide;
}

__device__ __forceinline__ bool item_of(const Schedule &s, int64_t i, Item &it)
{
    int64_t tile;
    if (i < s.whole) {
        tile = i;
        it.first = 0;
        it.last = s.blocks;
        it.part = -1;
    } else {
        // part m of pair p's range, which lies in the m-th tile that the range touches
        const uint32_t j = (uint32_t)(i - s.whole), m = j / (uint32_t)s.pairs, p = j - m * (uint32_t)s.pairs;
        if (p >= (uint32_t)s.ranges) return false;
        const int64_t lo = s.start[p], hi = s.start[p + 1];
        const int64_t c = s.tile[p] + m, at = c * s.blocks;
        it.first = (lo > at ? lo : at) - at;
        it.last = (hi < at + s.blocks ? hi : at + s.blocks) - at;
        if (it.first >= it.last) return false;
        it.part = it.first == 0 && it.last == s.blocks ? -1 : c + p;
        tile = s.whole + c;
    }
    tile_place(s, tile, it);
    return true;
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// n (1 .. 4) values to o, or added to what is there.
__device__ __forceinline__ void store4(float *o, float4 v, int n, int accumulate)
{
    if (n == 4 && (reinterpret_cast<uintptr_t>(o) & 15u) == 0) {
        float4 *p = reinterpret_cast<float4 *>(o);
        if (accumulate) {
            const float4 a = *p;
            v = make_float4(a.x + v.x, a.y + v.y, a.z + v.z, a.w + v.w);
        }
        *p = v;
        return;
    }
    const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) o[i] = accumulate ? o[i] + e[i] : e[i];
}

struct Shared {
    unsigned long long full[kFullBars]; // codes, exponents and B have arrived (this CTA): Ring::full
    unsigned long long ready[kStages];  // both CTAs have decoded A (the leader's is used)
    unsigned long long empty[kStages];  // the MMAs have read A and B
    unsigned long long acc_full[2];     // a run's sums are complete
    unsigned long long acc_empty[2];    // both CTAs have read them (the leader's is used)
    uint32_t tmem;
};

// 128 n of a tile from TMEM to dw, or to the workspace; a wait that gave up (ok false) leaves NaN.
__device__ __forceinline__ void store_tile(const Params &p, const Item &it, uint32_t cols, int n_off, int kl, bool ok)
{
    const int64_t k = (int64_t)it.tk * kTile + kl;
    const int n0 = it.tn * kTile + n_off;
    const bool part = it.part >= 0;
    const int n = part ? kTile / 2 : k < p.in ? p.out - n0 : 0;  // how many of the lane's n exist
    const bool add = !part && p.accumulate;
    const int64_t step = part ? kTile : p.sdw;
    float *o = part ? p.parts + (it.part * kTile + n_off) * kTile + kl : p.dw + (int64_t)n0 * p.sdw + k;
#pragma unroll 1
    for (int c = 0; c < kTile / 2; c += 16) {
        float v[16];
        tmem_load16(cols + c, v);
        if (!ok) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(0x7fffffffu);
        }
        if (add) {
            float old[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) old[j] = c + j < n ? o[j * step] : 0.0f;
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] += old[j];
        }
        if (c + 16 <= n) {
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j * step] = v[j];
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (c + j < n) o[j * step] = v[j];
        }
        o += 16 * step;
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1) k_wgrad(const __grid_constant__ Params p)
{
    extern __shared__ unsigned char raw_smem[];
    __shared__ Shared sh;
    const uint32_t stages = (smem_u32(raw_smem) + 1023u) & ~1023u;
    const uint32_t exps = stages + kStages * kStageBytes;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank();
    const int64_t pair = blockIdx.x >> 1, pairs = p.s.pairs;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kFullBars; ++i) mbar_init(&sh.full[i], 1 + 32);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.ready[i], kConvWarps);  // half of the warps, of two CTAs
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 2 * kEpiWarps);
        }
        fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = sh.tmem;

    if (warp < kCtlWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
        if (warp == 0 && lane == 0) {
            // TMA: codes and B of every stage
            Ring r;
            bool ok = true;
            Item it;
            for (int64_t i = pair; ok && item_of(p.s, i, it); i += pairs) {
                const int k0 = it.tk * kTile + (int)rank * kHalf, n0 = it.tn * kTile + (int)rank * kHalf;
                int plane = (int)(it.first / p.s.tok_blocks);
                int64_t tb = it.first - plane * p.s.tok_blocks;
                for (int64_t b = it.first; b < it.last; ++b) {
                    if (r.wrapped && !mbar_wait_cycles(smem_u32(&sh.empty[r.st]), r.parity_before(), p.limit)) {
                        ok = false;
                        break;
                    }
                    const int t0 = (int)tb * kTok;
                    const uint32_t base = stages + r.st * kStageBytes, bar = smem_u32(&sh.full[r.full()]);
                    mbar_arrive_expect_tx(&sh.full[r.full()], kBBytes + kCodeBytes);
                    tma_load_2d(base + kABytes + kBBytes, &p.codes, k0, t0, bar);
                    tma_load_3d(base + kABytes, &p.dy, n0, t0, plane, bar);
                    tma_load_3d(base + kABytes + kBlockBytes, &p.dy, n0 + 64, t0, plane, bar);
                    r.next();
                    if (++tb == p.s.tok_blocks) {
                        tb = 0;
                        ++plane;
                    }
                }
            }
            // what is still under way into this CTA's shared memory arrives before the CTA may leave: the
            // MMAs' signals (after which the copies have been read), or, where a wait gave up, the copies
            const int left = r.wrapped ? kStages : r.st;
            for (int i = 0; i < left; ++i) {
                r.back();
                if (ok) mbar_wait_cycles(smem_u32(&sh.empty[r.st]), r.parity(), p.limit);
                else mbar_wait_cycles(smem_u32(&sh.full[r.full()]), r.full_parity(), p.limit);
            }
        } else if (warp == 1 && rank == 0) {
            // MMA, by the leader CTA: the warp stays together, so that descriptors are uniform values, and one
            // lane issues
            const bool one = elect_one();
            const uint32_t idesc = instr_desc(BF16);
            Ring r;
            int64_t runs = 0;
            bool ok = true;
            Item it;
            for (int64_t i = pair; ok && item_of(p.s, i, it); i += pairs) {
                for (int64_t b = it.first; ok && b < it.last; ++runs) {
                    const int buf = (int)(runs & 1);
                    if (runs >= 2 && !mbar_wait_cycles_warp(smem_u32(&sh.acc_empty[buf]), ((uint32_t)(runs >> 1) + 1u) & 1u, p.limit)) {
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t d = tmem + buf * kTile;
                    const int n = (int)(it.last - b < kRun ? it.last - b : kRun);
                    b += n;
                    for (int j = 0; j < n; ++j) {
                        if (!mbar_wait_cycles_warp(smem_u32(&sh.ready[r.st]), r.parity(), p.limit)) {
                            ok = false;
                            break;
                        }
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        const uint32_t base = stages + r.st * kStageBytes;
                        const uint64_t da = operand_desc(base), db = operand_desc(base + kABytes);
                        if (one) {
#pragma unroll
                            for (int k = 0; k < kTok / 16; ++k)  // 16 tokens: two groups of 8, 2048 bytes
                                mma(d, da + (uint64_t)(k * 2048 >> 4), db + (uint64_t)(k * 2048 >> 4), idesc, j > 0 || k > 0);
                            commit_pair(smem_u32(&sh.empty[r.st]));
                        }
                        __syncwarp();
                        r.next();
                    }
                    if (ok && one) commit_pair(smem_u32(&sh.acc_full[buf]));
                    __syncwarp();
                }
            }
        } else if (warp == 2) {
            // Exponents of every stage: one word a token, two tokens a lane.  Loaded here and not by the warps
            // that decode: their signals would wait for loads of their own.
            Ring r;
            bool ok = true;
            Item it;
            for (int64_t i = pair; ok && item_of(p.s, i, it); i += pairs) {
                const int k0 = it.tk * kTile + (int)rank * kHalf;
                const bool any = k0 < p.in;
                const int64_t end = p.s.tok_blocks * kTok;
                int64_t t = it.first % p.s.tok_blocks * kTok + lane;
                const uint8_t *src = p.k.exps + (any ? t * p.k.exp_pitch + (k0 >> 5) : 0);
                for (int64_t b = it.first; b < it.last; ++b) {
                    if (r.wrapped && !mbar_wait_cycles_warp(smem_u32(&sh.empty[r.st]), r.parity_before(), p.limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = exps + r.st * kExpBytes + lane * 4;
                    // tokens past the last, and columns past the last, read as 0 (their codes are 0)
                    const bool in0 = any && t < p.tokens, in1 = any && t + 32 < p.tokens;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(in0 ? src : p.k.exps), "r"(in0 ? 4 : 0)
                                 : "memory");
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + 128),
                                 "l"(in1 ? src + 32 * p.k.exp_pitch : p.k.exps), "r"(in1 ? 4 : 0)
                                 : "memory");
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sh.full[r.full()])) : "memory");
                    r.next();
                    t += kTok;
                    if (any) src += kTok * p.k.exp_pitch;
                    if (t >= end) {  // the next plane
                        if (any) src -= end * p.k.exp_pitch;
                        t -= end;
                    }
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else if (warp < kCtlWarps + kEpiWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
        // Epilogue: TMEM lane = k (1 and 2 of every four exchanged), column = n; four warps take 128 n each.
        // A warp's 32 lanes store 32 adjacent k of one n.
        const int quarter = warp & 3;  // the TMEM lanes this warp may read
        const int n_off = (warp - kCtlWarps >= 4) ? kTile / 2 : 0;
        const uint32_t acc_empty = in_cta(smem_u32(&sh.acc_empty[0]), 0);
        const uint32_t cols = tmem + ((uint32_t)(quarter * 32) << 16) + n_off;
        const int kl = (int)rank * kHalf + quarter * 32 + (lane & 28) + ((lane & 1) << 1) + (lane >> 1 & 1);
        int64_t runs = 0;
        bool ok = true;
        Item it;
        for (int64_t i = pair; item_of(p.s, i, it); i += pairs) {
            float acc[kTile / 2];
#pragma unroll
            for (int j = 0; j < kTile / 2; ++j) acc[j] = 0.0f;
            for (int64_t b = it.first; b < it.last; b += kRun, ++runs) {
                const int buf = (int)(runs & 1);
                ok = ok && mbar_wait_cycles_warp(smem_u32(&sh.acc_full[buf]), (uint32_t)(runs >> 1) & 1u, p.limit);
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
                for (int c = 0; c < kTile / 2; c += 16) {
                    float v[16];
                    tmem_load16(cols + buf * kTile + c, v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[c + j] += v[j];
                }
                if (b + kRun >= it.last) {
                    // The tile's sums go back to TMEM, and from there to memory 16 at a time, in a loop that stays
                    // in the instruction cache: storing the registers takes 128 stores of straight code, which
                    // ran once a tile and took 20000 cycles.
#pragma unroll
                    for (int c = 0; c < kTile / 2; c += 16) tmem_store16(cols + buf * kTile + c, acc + c);
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    store_tile(p, it, cols + buf * kTile, n_off, kl, ok);
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) arrive_cluster(acc_empty + buf * 8);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConv));
        // Decode: four warps take the even stages, four the odd ones; a warp 16 tokens, a lane 16 codes at a
        // time.  Eight lanes read 64 bytes of codes of tokens t and t ^ 5 and store 8 pieces of 16 bytes: with
        // the 128-byte swizzle of both (piece ^ (token & 7)) either access covers all banks.
        const int w = warp - kCtlWarps - kEpiWarps;
        const uint32_t ready = in_cta(smem_u32(&sh.ready[0]), 0);
        int64_t total = 0;
        Item it;
        for (int64_t i = pair; item_of(p.s, i, it); i += pairs) total += it.last - it.first;
        const int c = lane & 3, block = lane >> 3 & 1;
        const int pr = lane >> 4, x = (lane & 4) ? pr ^ 5 : pr;      // token & 7 of the first of four
        const int t = (w & 3) * 16 + x;
        const uint32_t from = stages + kABytes + kBBytes + t * 128 + (((block * 4 + c) ^ x) << 4);
        const uint32_t to = stages + block * kBlockBytes + t * 128 + (((2 * c) ^ x) << 4);  // and the piece beside it
        const uint32_t ex = exps + t * 4 + block * 2 + (c >> 1);
        Ring r;
        r.next(w >> 2);
        for (int64_t i = w >> 2; i < total; i += 2, r.next(2)) {
            if (!mbar_wait_cycles_warp(smem_u32(&sh.full[r.full()]), r.full_parity(), p.limit)) break;
            const uint32_t off = r.st * kStageBytes;
            // tokens t, t + 2 (whose swizzle differs in bit 1), and 8 on
            const uint32_t f[2] = {from + off, (from ^ 32u) + off};
            const uint32_t at[4] = {to + off, (to ^ 16u) + off, (to ^ 32u) + off, (to ^ 48u) + off};
            uint4 q[4];
            uint32_t E[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(q[h].x), "=r"(q[h].y), "=r"(q[h].z), "=r"(q[h].w)
                             : "r"(f[h & 1] + (h & 1) * 256 + (h >> 1) * 1024));
                asm volatile("ld.shared.u8 %0, [%1];"
                             : "=r"(E[h])
                             : "r"(ex + (h & 1) * 8 + (h >> 1) * 32 + r.st * kExpBytes));
            }
            auto put = [&](int h, const uint32_t (&o)[8]) {
                const int d = (h & 1) * 256 + (h >> 1) * 1024;
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at[(h & 1) * 2] + d), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                             "r"(o[3])
                             : "memory");
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at[(h & 1) * 2 + 1] + d), "r"(o[4]), "r"(o[5]),
                             "r"(o[6]), "r"(o[7])
                             : "memory");
            };
            if (usual<BF16>(E[0]) && usual<BF16>(E[1]) && usual<BF16>(E[2]) && usual<BF16>(E[3])) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t o[8];
                    decode16<BF16>(q[h], E[h], o);
                    put(h, o);
                }
            } else {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t o[8];
                    decode16_any<BF16>(q[h], E[h], o);
                    put(h, o);
                }
            }
            __syncwarp();
            // A is in this CTA's shared memory, whose stores the fence has made visible to its tensor cores: the
            // signal carries no more than that, and a release to the cluster would take some 1300 cycles
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive_cluster(ready + r.st * 8);
        }
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// The cut tiles' sums, range by range in order, into dw.  A block takes 4 n of a tile, a thread 4 adjacent k of one.
__global__ void __launch_bounds__(256) k_join(const __grid_constant__ Params p)
{
    cudaGridDependencySynchronize();  // launched to start as k_wgrad drains
    const int64_t c = blockIdx.x / (kTile / 4);
    const int n = (int)(blockIdx.x % (kTile / 4)) * 4 + (int)(threadIdx.x >> 6), kl = (int)(threadIdx.x & 63) * 4;
    const int lo = p.s.from[c], hi = p.s.to[c];
    if (lo == hi) return;  // one range has the whole tile, and has stored it
    Item it;
    tile_place(p.s, p.s.whole + c, it);
    const int64_t k = (int64_t)it.tk * kTile + kl, row = (int64_t)it.tn * kTile + n;
    if (k >= p.in || row >= p.out) return;
    const float *s = p.parts + ((c + lo) * kTile + n) * kTile + kl;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int r = 0; r <= hi - lo; ++r) {
        const float4 a = *reinterpret_cast<const float4 *>(s + (int64_t)r * kTile * kTile);
        v.x += a.x;
        v.y += a.y;
        v.z += a.z;
        v.w += a.w;
    }
    store4(p.dw + row * p.sdw + k, v, (int)min((int64_t)4, p.in - k), p.accumulate);
}

__global__ void __launch_bounds__(256) k_zero(float *dw, int64_t sdw, int in, int out)
{
    for (int64_t n = blockIdx.x; n < out; n += gridDim.x)
        for (int k = threadIdx.x; k < in; k += 256) dw[n * sdw + k] = 0.0f;
}

// ---------------------------------------------------------------------------------------------
// A few tokens and not many columns: tiles of 256 x 256 leave most SMs without one.  A block
// takes 64 n x 128 k, a lane 4 k of the 8 n of its warp, on the ordinary cores: every type as it is, and the
// bias's gradient along with it.
// ---------------------------------------------------------------------------------------------
constexpr int kFewTokens = 32, kFewN = 64, kFewK = 128;
// Measured in a graph, this kernel against the tiles: 1024 x 1024 with 1, 16, 32 and 64 tokens 3, 5, 8 and 13.6 us
// against 12 to 13 us; 4096 x 4096 with 16 tokens 36 against 21 us, with 64 117 against 21 us.
inline bool few(int64_t tokens, int64_t in, int64_t out)
{
    return tokens <= kFewTokens && tokens * in * out <= int64_t(1) << 26;
}

template <typename T>
__global__ void __launch_bounds__(256) k_few(const __grid_constant__ Params p, const T *dy, int64_t sdy, float *db)
{
    __shared__ float sd[kFewTokens][kFewN];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tiles_k = (p.in + kFewK - 1) / kFewK;
    const int64_t tn = blockIdx.x / tiles_k;
    const int k = (int)(blockIdx.x - tn * tiles_k) * kFewK + lane * 4, tokens = (int)p.tokens;
    const int64_t n0 = tn * kFewN;
    for (int i = threadIdx.x; i < tokens * kFewN; i += 256) {
        const int t = i / kFewN, n = i % kFewN;
        sd[t][n] = n0 + n < p.out ? to_float(dy[t * sdy + n0 + n]) : 0.0f;
    }
    __syncthreads();
    float acc[8][4] = {};
    const bool in = k < p.k.code_pitch;
    for (int t0 = 0; t0 < tokens; t0 += 8) {  // eight tokens' codes at once: their latency is most of the time
        uint32_t q[8], e[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const bool has = in && t0 + u < tokens;
            q[u] = has ? __ldg(reinterpret_cast<const uint32_t *>(p.k.codes + (int64_t)(t0 + u) * p.k.code_pitch + k)) : 0u;
            e[u] = has ? __ldg(p.k.exps + (int64_t)(t0 + u) * p.k.exp_pitch + (k >> 5)) : 0u;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int t = t0 + u;
            if (t >= tokens) break;
            const float scale = group_scale(e[u]);
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = (float)(int)(int8_t)(q[u] >> (8 * j)) * scale;
                if constexpr (__is_same(T, __half)) {
                    x[j] = x[j] > 65504.0f ? 65504.0f : x[j] < -65504.0f ? -65504.0f : x[j];
                    x[j] = __half2float(__float2half_rn(x[j]));
                }
            }
            float d[8];
            *reinterpret_cast<float4 *>(d) = *reinterpret_cast<const float4 *>(&sd[t][warp * 8]);
            *reinterpret_cast<float4 *>(d + 4) = *reinterpret_cast<const float4 *>(&sd[t][warp * 8 + 4]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __fmaf_rn(d[i], x[j], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t n = n0 + warp * 8 + i;
        if (n < p.out && k < p.in)
            store4(p.dw + n * p.sdw + k, make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]), min(4, p.in - k), p.accumulate);
    }
    if (db && k == lane * 4 && threadIdx.x < kFewN && n0 + threadIdx.x < p.out) {
        float v = 0.0f;
        for (int t = 0; t < tokens; ++t) v += sd[t][threadIdx.x];
        float *o = db + n0 + threadIdx.x;
        *o = p.accumulate ? *o + v : v;
    }
}

// dy into rows of `pitch` 16-bit values: float32 as three bf16 planes that add up to it (smallest first; bits
// below 2^-133 cut off), 16-bit types as they are.  A warp takes 256 columns of a row.
template <typename T, bool AL>
__global__ void __launch_bounds__(256) k_stage(const T *dy, int64_t sdy, int64_t tokens, int out, int64_t pitch, uint16_t *dst)
{
    const int per_row = (out + kChunk - 1) / kChunk, lane = threadIdx.x & 31;
    const int64_t n = tokens * per_row, warps = (int64_t)gridDim.x * 8;
    for (int64_t id = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); id < n; id += warps) {
        const int64_t t = id / per_row;
        const int base = (int)(id - t * per_row) * kChunk, c = base + lane * 8;
        const T *row = dy + t * sdy;
        Raw<T, AL> r;
        if (inner_chunk<T, AL>(base, out)) chunk_load<T, AL, true>(r, row, base, lane, out);
        else chunk_load<T, AL, false>(r, row, base, lane, out);
        const Words<T> w = in_place<T, AL>(r, row);
        if (c >= pitch) continue;  // pitch and c are multiples of 8
        uint16_t *o = dst + t * pitch + c;
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4 *>(o) = make_uint4(w.w[0], w.w[1], w.w[2], w.w[3]);
        } else {
            uint32_t part[3][4];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t bits = w.w[j];
                uint32_t hi = bits >> 16, mid = 0, lo = 0;
                if ((bits & 0x7f800000u) == 0x7f800000u) {
                    if (bits & 0x007fffffu) hi |= 0x40u;  // a NaN stays one
                } else {
                    const float rest = __uint_as_float(bits) - __uint_as_float(bits & 0xffff0000u);
                    const uint32_t m = __float_as_uint(rest);
                    mid = m >> 16;
                    lo = __float_as_uint(rest - __uint_as_float(m & 0xffff0000u)) >> 16;
                }
                const uint32_t e[3] = {lo, mid, hi};
#pragma unroll
                for (int i = 0; i < 3; ++i) part[i][j >> 1] = (j & 1) ? part[i][j >> 1] | e[i] << 16 : e[i];
            }
#pragma unroll
            for (int i = 0; i < 3; ++i)
                *reinterpret_cast<uint4 *>(o + i * tokens * pitch) = make_uint4(part[i][0], part[i][1], part[i][2], part[i][3]);
        }
    }
}

template <typename T>
cudaError_t launch_stage(const void *dy, int64_t sdy, int64_t tokens, int64_t out, int64_t pitch, unsigned char *dst, cudaStream_t s)
{
    const int64_t need = (tokens * ((out + kChunk - 1) / kChunk) + 7) / 8;
    const unsigned grid = (unsigned)(need < 148 * 8 ? need : 148 * 8);
    auto kern = tokens == 1 || sdy % (16 / (int)sizeof(T)) == 0 ? k_stage<T, true> : k_stage<T, false>;
    kern<<<grid, 256, 0, s>>>(static_cast<const T *>(dy), sdy, tokens, (int)out, pitch, reinterpret_cast<uint16_t *>(dst));
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_few(const Params &p, const WgradArgs &a, cudaStream_t s)
{
    const int64_t blocks = ((a.in + kFewK - 1) / kFewK) * ((a.out + kFewN - 1) / kFewN);
    k_few<T><<<(unsigned)blocks, 256, 0, s>>>(p, static_cast<const T *>(a.dy.p), a.dy.stride, a.db);
    return cudaGetLastError();
}

bool staged(int dtype, int64_t tokens, int64_t out, int64_t dy_stride)
{
    return dtype == GQ_FLOAT32 || (tokens > 1 && (dy_stride % 8 != 0 || dy_stride < out));
}
int64_t staged_pitch(int64_t out) { return (out + 7) / 8 * 8; }

struct Spaces {
    size_t staged, parts, cols, bytes;  // offsets of the staged gradient, the cut tiles, the bias's partial rows
};
Spaces spaces(int dtype, int64_t tokens, int64_t in, int64_t out, int64_t dy_stride, bool bias)
{
    Spaces w;
    w.staged = w.parts = w.cols = w.bytes = 0;
    if (few(tokens, in, out)) return w;  // no tokens among them
    const Schedule s = schedule(dtype, tokens, in, out);
    w.parts = staged(dtype, tokens, out, dy_stride)
                  ? (size_t)(tokens * staged_pitch(out)) * (dtype == GQ_FLOAT32 ? 6 : 2) : 0;
    w.cols = w.parts + (size_t)part_tiles(s) * kTile * kTile * sizeof(float);
    w.bytes = w.cols + (bias ? (size_t)(colsum_parts(tokens, out) * out) * sizeof(float) : 0);
    return w;
}

}  // namespace

size_t wgrad_workspace(int dtype, int64_t tokens, int64_t in, int64_t out, int64_t dy_stride, bool bias)
{
    return spaces(dtype, tokens, in, out, dy_stride, bias).bytes;
}

cudaError_t launch_wgrad(const WgradArgs &a, cudaStream_t stream)
{
    if (a.tokens == 0) {
        if (a.accumulate) return cudaSuccess;
        k_zero<<<(unsigned)(a.out < 1024 ? a.out : 1024), 256, 0, stream>>>(a.dw, a.dw_stride, (int)a.in, (int)a.out);
        const cudaError_t e = cudaGetLastError();
        return e == cudaSuccess && a.db ? cudaMemsetAsync(a.db, 0, (size_t)a.out * sizeof(float), stream) : e;
    }
    const CkptLayout l = ckpt_layout(a.tokens, a.in);
    const Spaces w = spaces(a.dtype, a.tokens, a.in, a.out, a.dy.stride, a.db != nullptr);
    int per_sm = 0, sms = 0;
    cudaError_t e = cudaSuccess;

    Params p;
    p.tokens = a.tokens;
    p.in = (int)a.in;
    p.out = (int)a.out;
    uint8_t *ck = static_cast<uint8_t *>(const_cast<void *>(a.ckpt));
    p.k = Ckpt{ck, ck + l.exps_off, (int)l.code_pitch, (int)l.exp_pitch};
    p.dw = a.dw;
    p.sdw = a.dw_stride;
    p.accumulate = a.accumulate;
    p.parts = reinterpret_cast<float *>(a.ws + w.parts);
    // two seconds at 1.97 GHz, three at the 1.39 GHz of the power cap; the longest wait, for a run of stages, is some
    // microseconds
    p.limit = 4000000000ll;

    if (few(a.tokens, a.in, a.out)) {
        if (a.dtype == GQ_FLOAT32) return launch_few<float>(p, a, stream);
        if (a.dtype == GQ_BFLOAT16) return launch_few<__nv_bfloat16>(p, a, stream);
        return launch_few<__half>(p, a, stream);
    }

    p.s = schedule(a.dtype, a.tokens, a.in, a.out);
    const void *dy = a.dy.p;
    int64_t pitch = a.tokens > 1 ? a.dy.stride : staged_pitch(a.out);
    const int planes = a.dtype == GQ_FLOAT32 ? 3 : 1;
    if (staged(a.dtype, a.tokens, a.out, a.dy.stride)) {
        pitch = staged_pitch(a.out);
        e = a.dtype == GQ_FLOAT32 ? launch_stage<float>(dy, a.dy.stride, a.tokens, a.out, pitch, a.ws, stream)
                                  : launch_stage<__half>(dy, a.dy.stride, a.tokens, a.out, pitch, a.ws, stream);
        if (e != cudaSuccess) return e;
        dy = a.ws;
    }
    const EncodeFn encode = encode_fn();
    if (!encode) return cudaErrorNotSupported;
    const cuuint32_t ones[3] = {1, 1, 1};
    {
        const cuuint64_t dims[2] = {(cuuint64_t)l.code_pitch, (cuuint64_t)a.tokens};
        const cuuint64_t strides[1] = {(cuuint64_t)l.code_pitch};
        const cuuint32_t box[2] = {kHalf, kTok};
        if (encode(&p.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(a.ckpt), dims, strides, box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    {
        const cuuint64_t dims[3] = {(cuuint64_t)a.out, (cuuint64_t)a.tokens, (cuuint64_t)planes};
        const cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, (cuuint64_t)pitch * 2 * (cuuint64_t)(planes > 1 ? a.tokens : 1)};
        const cuuint32_t box[3] = {64, kTok, 1};
        if (encode(&p.dy, a.dtype == GQ_FLOAT16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                   const_cast<void *>(dy), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }

    auto kern = a.dtype == GQ_FLOAT16 ? k_wgrad<false> : k_wgrad<true>;
    e = kernel_occupancy(reinterpret_cast<const void *>(kern), kThreads, kSmemBytes, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    static const int regs[2] = {num_regs(k_wgrad<false>), num_regs(k_wgrad<true>)};
    if (regs[0] < kRegsLaunch || regs[1] < kRegsLaunch) return cudaErrorInvalidKernelImage;  // setmaxnreg would wait
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * p.s.pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e != cudaSuccess) return e;
    if (part_tiles(p.s)) {
        cfg.gridDim = dim3((unsigned)(p.s.cut * (kTile / 4)));
        cfg.blockDim = dim3(256);
        cfg.dynamicSmemBytes = 0;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        e = cudaLaunchKernelEx(&cfg, k_join, p);
        if (e != cudaSuccess) return e;
    }
    if (!a.db) return cudaSuccess;
    return launch_colsum(a.dtype, a.tokens, a.out, a.dy, reinterpret_cast<float *>(a.ws + w.cols), a.db, a.accumulate, stream);
}

}  // namespace gq
