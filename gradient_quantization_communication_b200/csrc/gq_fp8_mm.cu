// gq_fp8_mm.cu -- products of packed matrices of 8-bit floating point on the tensor cores:
//   y[i][j] = sum over blocks b of 2^(Ea + Eb - 254) * sum over c in b of a[i][c] * b[j][c]  + bias[j].
//
// The scales are powers of two, which tcgen05.mma (kind::mxf8f6f4, block_scale) takes as they are, one byte for every
// 32 columns: a block's byte serves four MMAs, and the loop has no arithmetic besides them.  The M side of an MMA is
// b (j, the features: a warp's 32 TMEM lanes are then adjacent columns of y), the N side is a (i, the tokens).  A
// stage is 128 columns of both, K-major rows of 128 bytes with the 128-byte swizzle, fetched by TMA.  The exponents
// of four stages (512 columns) are one word a row; four warps put them into TMEM, where row r's word belongs into
// lane r mod 32 of column r / 32, once in each quarter of the lanes.
//
// Two shapes (gq_fp8_tiles.h): CTA pairs on tiles of 256 features x up to 256 tokens, and, for up to 128 tokens, single
// CTAs on 128 features whose clusters cut the columns.  In either, one thread fetches, one issues the MMAs, four warps
// bring the exponents, and four or eight store tiles while the next ones are summed in a second accumulator.
//
// Bounded for many tokens by the SMs' way to L2 and then by power: a stage of a pair's CTA is 32 KB for 512 cycles of
// MMAs, and arrives after 650 (13.5 TB/s over all SMs); the tensor pipe is active 72 % of the time.  Measured in graphs of
// ten calls, bf16: 8192 tokens, 4096 x 4096 100 us (2.75 PFLOP/s), 16384 tokens, 4096 x 16384 757 us (2.90, 89 % of twice
// the library's measured bf16 rate); in a long run of calls, under the power cap, some 2.3.  For few tokens by latency:
// 16 tokens, 4096 x 4096 8.4 us, of which 1 us until the first copy is issued, 1.2 until it arrives, 1.1 for all stages, 1.2
// for the sums' way out of TMEM and 2.7 for the cluster's join, where the weight's bytes would take 2.6.
#include "gq_act.cuh"
#include "gq_device.cuh"
#include "gq_fp8.cuh"
#include "gq_fp8.h"
#include "gq_fp8_tiles.h"
#include "gq_internal.h"
#include "gq_tc.cuh"

namespace gq {
namespace {

using namespace tiles;

// Warps: 4 of control (copies, MMA, two idle), 4 of exponents, 8 or 4 of epilogue.  A pair's epilogue holds 128 sums in
// each thread's registers, more than an even split gives.
constexpr int kRegsLaunch = 128, kRegsCtl = 48, kRegsEpi = 184, kRegsExp = 96;
static_assert(4 * kRegsCtl + 8 * kRegsEpi + 4 * kRegsExp <= 16 * kRegsLaunch, "setmaxnreg: the shares come from the launch's registers");

int run_of(int dtype) { return dtype == GQ_FLOAT32 ? kRunWide : kRun16; }

// An operand's exponents.
struct Exps {
    const uint8_t *p;
    int64_t rows, pitch;
    int shift;  // 1 << shift rows share one
};

struct Params {
    CUtensorMap w, x;
    Schedule s;
    Exps ew, ex;
    uint32_t idesc;     // without the exponents' byte numbers
    int run;            // kRunWide or kRun16
    int64_t tokens, features;
    const float *bias;
    void *y;
    int64_t sy;
    int accumulate;
    bool quads;         // four adjacent features of y start on 8 bytes
    float *parts;
    long long limit;    // cycles after which a wait gives up
};

// Position in the ring of stages.  Every role sees every use of every stage, so a phase's parity names it.
template <int N>
struct Ring {
    int st = 0;
    uint32_t turn = 0;
    __device__ __forceinline__ void next()
    {
        if (++st == N) {
            st = 0;
            ++turn;
        }
    }
    __device__ __forceinline__ uint32_t parity() const { return turn & 1u; }
    __device__ __forceinline__ uint32_t parity_before() const { return (turn & 1u) ^ 1u; }
};

// K-major rows of 128 bytes, 128-byte swizzle: groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3fffu) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// kind::mxf8f6f4, D binary32, both operands K-major, exponents ue8m0.
constexpr uint32_t instr_desc(int fw, int fx, int m, int n)
{
    return (uint32_t)fw << 7 | (uint32_t)fx << 10 | (uint32_t)(n >> 3) << 17 | 1u << 23 | (uint32_t)(m >> 7) << 27;
}
// The byte of the exponents' words that counts.
__device__ __forceinline__ uint32_t exp_byte(uint32_t b) { return b << 4 | b << 29; }

template <int GROUP>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t ea, uint32_t eb, bool add)
{
    if constexpr (GROUP == 2)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d), "l"(a), "l"(b),
            "r"(idesc), "r"(ea), "r"(eb), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.u32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d), "l"(a), "l"(b),
            "r"(idesc), "r"(ea), "r"(eb), "r"((uint32_t)add)
            : "memory");
}
// Arrives on the barrier (of both CTAs of a pair) once the MMAs issued so far are done.
template <int GROUP>
__device__ __forceinline__ void commit(uint32_t bar)
{
    if constexpr (GROUP == 2) commit_pair(bar);
    else asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_store4(uint32_t addr, const uint32_t *v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0, %1, %2, %3};" ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(addr)
                 : "memory");
}

// A box of 128 bytes a row into this CTA's shared memory; of a pair, either CTA's copies complete on the leader's barrier.
template <int GROUP>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    if constexpr (GROUP == 1)
        tma_load_2d(dst, map, x, y, bar);
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                dst),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
}

// 16 columns, to be had after tmem_wait16.
__device__ __forceinline__ void tmem_begin16(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

struct Shared {
    unsigned long long full[8];       // both CTAs' operands have arrived (the leader's)
    unsigned long long empty[8];      // the MMAs have read them
    unsigned long long exp_full[2];   // the exponents of four stages are in TMEM, of both CTAs (the leader's)
    unsigned long long exp_empty[2];  // the MMAs have read them
    unsigned long long acc_full[2];   // a run's sums are complete
    unsigned long long acc_empty[2];  // both CTAs have read them (the leader's)
    unsigned long long edge[2];       // both CTAs have read the columns that the other accumulator shares (the leader's)
    uint32_t tmem;
    int failed;                       // a single CTA's wait gave up
};

template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half rounded<__half>(float v) { return __float2half_rn(v); }

// Two values of a 16-bit type as a word.
template <typename T>
__device__ __forceinline__ uint32_t pair16(float a, float b)
{
    if constexpr (__is_same(T, __half)) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Where a lane's column of a tile goes: its feature of `count` tokens from token x0 of the tile on.
template <typename T, class S>
struct Out {
    T *y;
    float *part;      // the workspace, or (single CTAs) shared memory; nullptr: y
    int64_t sy;
    int n;            // tokens that exist, of `count`
    float bias;
    bool in, add, ok;     // in: the lane's feature exists
    bool fast;            // the warp may store by put16_whole
    uint32_t mine, other, first, second;  // byte selectors of the exchange

    __device__ __forceinline__ Out(const Params &p, const Item &it, float *shared, int x0, int count, int row, bool ok_) : sy(p.sy), ok(ok_)
    {
        const int64_t feature = (int64_t)it.tw * S::kFeatures + row, token = (int64_t)it.tx * p.s.tokens + x0;
        const int64_t left = p.tokens - token;
        in = feature < p.features;
        float *const tile = S::kGroup == 1 ? shared : p.parts + (int64_t)it.part * S::kTokens * S::kFeatures;
        part = it.part < 0 ? nullptr : tile + x0 * S::kFeatures + row;
        n = (int)(left < 0 ? 0 : left < count ? left : count);
        y = static_cast<T *>(p.y) + token * sy + feature;
        bias = p.bias && in && !part ? p.bias[feature] : 0.0f;
        add = p.accumulate != 0;
        // four lanes that share stores exist together, or not at all
        const bool four = p.features % 4 == 0 || __all_sync(kFull, in);
        fast = ok && (sizeof(T) == 4 || part || (p.quads && four));
        const bool odd = threadIdx.x & 1;
        mine = odd ? 0x7632 : 0x5410;
        other = odd ? 0x5410 : 0x7632;
        first = odd ? 0x1054 : 0x5410;
        second = odd ? 0x3276 : 0x7632;
    }
    // Tokens c .. c + 15, some of which may not exist; a wait that gave up (ok false) leaves NaN.
    __device__ __forceinline__ void put16(const uint32_t (&r)[16], int c) const
    {
        const int m = in ? n - c : 0;
        T *o = y + c * sy;
#pragma unroll
        for (int j = 0; j < 16; ++j, o += sy) {
            if (j >= m) continue;
            float v = ok ? __uint_as_float(r[j]) : __uint_as_float(0x7fffffffu);
            if (part) {
                part[(c + j) * S::kFeatures] = v;
                continue;
            }
            v += bias;
            if constexpr (sizeof(T) == 4) {
                if (add) v += *o;
            }
            *o = rounded<T>(v);
        }
    }
    // Whichever of the two it takes.
    __device__ __forceinline__ void put(const uint32_t (&r)[16], int c) const
    {
        if (fast && c + 16 <= n) put16_whole(r, c);
        else if (c < n) put16(r, c);
    }
    // The same where all 16 tokens exist, and where `fast`.  16-bit values go four features of a token at a time: of four
    // tokens the lanes 4 q .. 4 q + 3 exchange theirs, and lane 4 q + i stores token i's (a store of 2 bytes by each lane
    // takes four times as many; with a check for each of them a tile of 256 x 256 took 5.9 us, so it takes 3).
    __device__ __forceinline__ void put16_whole(const uint32_t (&r)[16], int c) const
    {
        if (part) {
            float *o = part + c * S::kFeatures;
            if (in) {
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j * S::kFeatures] = __uint_as_float(r[j]);
            }
            return;
        }
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]) + bias;
        if constexpr (sizeof(T) == 4) {
            T *o = y + c * sy;
            if (!in) return;
            if (add) {
                float old[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) old[j] = o[j * sy];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] += old[j];
            }
#pragma unroll
            for (int j = 0; j < 16; ++j, o += sy) *o = v[j];
        } else {
            const int i = threadIdx.x & 3;
            T *to = y + (c + i) * sy - i;
#pragma unroll
            for (int j = 0; j < 16; j += 4, to += 4 * sy) {
                const uint32_t ab = pair16<T>(v[j], v[j + 1]), cd = pair16<T>(v[j + 2], v[j + 3]);
                // even lanes keep tokens 0 and 2, odd ones 1 and 3, of two features
                const uint32_t a = __byte_perm(ab, cd, mine), b = __shfl_xor_sync(kFull, __byte_perm(ab, cd, other), 1);
                const uint32_t x = __byte_perm(a, b, first), z = __byte_perm(a, b, second);
                // lanes 0 and 1 keep the first of those, lanes 2 and 3 the second, of four features
                const uint32_t got = __shfl_xor_sync(kFull, (i & 2) ? x : z, 2);
                if (in) *reinterpret_cast<uint2 *>(to) = make_uint2((i & 2) ? got : x, (i & 2) ? z : got);
            }
        }
    }
};

__device__ __forceinline__ uint32_t load_cluster(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 load_cluster4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// The parts of a cluster's tile, one in each CTA's shared memory, in order to y: a warp takes a token's 128 features, a
// lane four of them, and all parts' are on their way at once (another CTA's shared memory answers after some 700 cycles).
template <typename T, class S>
__device__ __forceinline__ void join_cluster(const Params &p, const Item &it, Shared &sh, const float *shared, uint32_t rank)
{
    const int splits = p.s.splits, lane = threadIdx.x & 31;
    const int64_t feature = (int64_t)it.tw * S::kFeatures + lane * 4, token = (int64_t)it.tx * S::kTokens;
    const int n = (int)min((int64_t)S::kTokens, p.tokens - token), some = (int)max((int64_t)0, min((int64_t)4, p.features - feature));
    float bias[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) bias[j] = p.bias && j < some ? p.bias[feature + j] : 0.0f;
    cluster_sync();
    const uint32_t from = smem_u32(shared + lane * 4);
    const bool failed = __any_sync(kFull, lane < splits && load_cluster(in_cta(smem_u32(&sh.failed), (uint32_t)lane % splits)) != 0);
    for (int x = (int)rank + splits * (int)(threadIdx.x >> 5); x < n; x += splits * (S::kThreads / 32)) {
        float4 part[kMaxSplits];
#pragma unroll
        for (int r = 0; r < kMaxSplits; ++r)
            if (r < splits) part[r] = load_cluster4(in_cta(from + x * S::kFeatures * 4, (uint32_t)r));
        float4 sum = part[0];
#pragma unroll
        for (int r = 1; r < kMaxSplits; ++r)
            if (r < splits) sum = make_float4(sum.x + part[r].x, sum.y + part[r].y, sum.z + part[r].z, sum.w + part[r].w);
        float v[4] = {sum.x + bias[0], sum.y + bias[1], sum.z + bias[2], sum.w + bias[3]};
        T *const y = static_cast<T *>(p.y) + (token + x) * p.sy + feature;
        if (failed) v[0] = v[1] = v[2] = v[3] = __uint_as_float(0x7fffffffu);
        if constexpr (sizeof(T) == 2) {
            if (p.quads && some == 4) {
                *reinterpret_cast<uint2 *>(y) = make_uint2(pair16<T>(v[0], v[1]), pair16<T>(v[2], v[3]));
                continue;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j >= some) continue;
            if constexpr (sizeof(T) == 4) {
                if (p.accumulate) v[j] += y[j];
            }
            y[j] = rounded<T>(v[j]);
        }
    }
    cluster_sync();  // until all have read
}

// SUMS: runs' sums are added up in registers, rounded to nearest; else a tile is one run.
template <typename T, int GROUP, int TN, bool SUMS>
__global__ void __launch_bounds__(Shape<GROUP, TN>::kThreads, Shape<GROUP, TN>::kPerSm) k_mm(const __grid_constant__ Params p)
{
    using S = Shape<GROUP, TN>;
    extern __shared__ unsigned char raw_smem[];
    __shared__ Shared sh;
    const uint32_t stages = ring_start(smem_u32(raw_smem));
    float *const part = reinterpret_cast<float *>(raw_smem + (stages - smem_u32(raw_smem)));  // a single CTA's, in the end
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank(), leader = GROUP == 2 ? 0u : rank;  // whose barriers the MMAs go by
    const int pair_rank = GROUP == 2 ? (int)rank : 0;
    const int second = min(p.s.tokens, S::kSecond);
    const bool shares = p.s.tokens > S::kSecond;

    if (threadIdx.x == 32) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&p.w) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&p.x) : "memory");
    }
    if (threadIdx.x == 0) {
        sh.failed = 0;
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.exp_full[i], 4 * GROUP);
            mbar_init(&sh.exp_empty[i], 1);
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], S::kEpiWarps * GROUP);
            mbar_init(&sh.edge[i], 4 * GROUP);
        }
        fence_barrier_init();
    }
    __syncthreads();
    if constexpr (GROUP == 2) cluster_sync();
    // Up to here it runs as the kernel before it on the stream drains.  TMEM is not taken before: that kernel might still
    // want it, and this one would wait for its end.
    cudaGridDependencySynchronize();
    if (warp == 1) {
        if constexpr (GROUP == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)), "n"(S::kTmem) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)), "n"(S::kTmem) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = sh.tmem;

    if (warp < 4) {
        if constexpr (GROUP == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
        if (warp == 0 && lane == 0) {
            // TMA: 128 features and this CTA's tokens of every stage.  The leader's barrier expects both CTAs' bytes; the
            // other's may arrive first, but not in an earlier phase: that one had ended when its stage was free again.
            const uint32_t full = in_cta(smem_u32(&sh.full[0]), leader);
            const int xrows = GROUP == 2 ? p.s.tokens / 2 : TN;
            const uint32_t bytes = GROUP * (S::kWBytes + xrows * 128);
            Ring<S::kStages> r;
            bool ok = true;
            Item it;
            for (int i = 0; ok && item_of<GROUP>(p.s, blockIdx.x, i, rank, it); ++i) {
                const int w0 = it.tw * S::kFeatures + pair_rank * 128, x0 = it.tx * p.s.tokens + pair_rank * xrows;
                for (int b = it.first; b < it.last; ++b) {
                    if (r.turn > 0 && !mbar_wait_cycles(smem_u32(&sh.empty[r.st]), r.parity_before(), p.limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t base = stages + r.st * S::kStageBytes, bar = full + r.st * 8;
                    if (rank == leader) mbar_arrive_expect_tx(&sh.full[r.st], bytes);
                    load_box<GROUP>(base, &p.w, b * 128, w0, bar);
                    load_box<GROUP>(base + S::kWBytes, &p.x, b * 128, x0, bar);
                    r.next();
                }
            }
            // what is still under way into this CTA's shared memory arrives before the CTA may leave: the MMAs'
            // signals (after which the copies have been read), or, where a wait gave up, the copies, for which the
            // leader waits (and the other for the leader, at the end)
            const int used = r.turn > 0 ? S::kStages : r.st;
            for (int i = 0; i < used; ++i) {
                if (r.st == 0) {
                    r.st = S::kStages;
                    --r.turn;
                }
                --r.st;
                if (ok || rank == leader) mbar_wait_cycles(smem_u32(ok ? &sh.empty[r.st] : &sh.full[r.st]), r.parity(), p.limit);
            }
        } else if (warp == 1 && rank == leader) {
            // MMA, by the leader CTA: the warp stays together, so that descriptors are uniform values, and one lane
            // issues
            const bool one = elect_one();
            Ring<S::kStages> r;
            uint32_t runs = 0, groups = 0;
            bool ok = true;
            Item it;
            for (int i = 0; ok && item_of<GROUP>(p.s, blockIdx.x, i, rank, it); ++i) {
                uint32_t ew = 0;
                for (int b = it.first; ok && b < it.last; ++runs) {
                    const int buf = (int)(runs & 1);
                    if (runs >= 2) ok = mbar_wait_cycles_warp(smem_u32(&sh.acc_empty[buf]), ((uint32_t)(runs >> 1) + 1u) & 1u, p.limit);
                    if (shares && ok && runs >= 1)
                        ok = mbar_wait_cycles_warp(smem_u32(&sh.edge[buf ^ 1]), (uint32_t)((runs - 1) >> 1) & 1u, p.limit);
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t d = tmem + buf * second;
                    const int end = it.last - b < p.run ? it.last : b + p.run;
                    for (bool add = false; b < end; ++b, add = true) {
                        const int eb = (int)(groups & 1);
                        if (b == it.first || (b & 3) == 0) {
                            if (!mbar_wait_cycles_warp(smem_u32(&sh.exp_full[eb]), (uint32_t)(groups >> 1) & 1u, p.limit)) {
                                ok = false;
                                break;
                            }
                            ew = tmem + S::kExps + eb * S::kExpCols;
                        }
                        if (!mbar_wait_cycles_warp(smem_u32(&sh.full[r.st]), r.parity(), p.limit)) {
                            ok = false;
                            break;
                        }
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        const uint32_t base = stages + r.st * S::kStageBytes;
                        const uint64_t dw = operand_desc(base), dx = operand_desc(base + S::kWBytes);
                        const uint32_t idesc = p.idesc | exp_byte((uint32_t)b & 3u);
                        const bool last = (b & 3) == 3 || b + 1 == it.last;  // of the four stages' exponents
                        if (one) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)  // 32 columns each
                                mma<GROUP>(d, dw + 2 * k, dx + 2 * k, idesc, ew, ew + 4, add || k > 0);
                            commit<GROUP>(smem_u32(&sh.empty[r.st]));
                            if (last) commit<GROUP>(smem_u32(&sh.exp_empty[eb]));
                        }
                        __syncwarp();
                        if (last) ++groups;
                        r.next();
                    }
                    if (ok && one) commit<GROUP>(smem_u32(&sh.acc_full[buf]));
                    __syncwarp();
                }
            }
        }
    } else if (warp >= 8) {
        if constexpr (GROUP == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
        // Epilogue: TMEM lane = feature, column = token; of a pair four warps take the lower half of the tokens, four the
        // upper.
        constexpr int kLower = TN > 128 ? 128 : TN, kFirst = GROUP == 2 && !SUMS ? kHeld : 0;
        const int quarter = warp & 3;  // the TMEM lanes this warp may read
        const bool upper = warp >= 12;
        const int x0 = upper ? kLower : 0;
        const int count = GROUP == 2 ? min(max(p.s.tokens - x0, 0), kLower) : TN;  // a multiple of 32
        const uint32_t acc_empty = in_cta(smem_u32(&sh.acc_empty[0]), leader), edge = in_cta(smem_u32(&sh.edge[0]), leader);
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + x0;
        const int row = pair_rank * 128 + quarter * 32 + lane;
        // The columns are taken in this order: the first kFirst are those that the other accumulator may share, the first
        // accumulator's last and the second one's first.  (Tiles of several runs are narrower and share none.)
        const int turn = !SUMS && shares && upper ? kLower - kFirst : 0;
        auto col = [&](int c) { return (c + turn) & (kLower - 1); };
        auto release = [&](int buf) {
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) arrive_cluster(acc_empty + buf * 8);
        };
        uint32_t runs = 0;
        bool ok = true;
        Item it;
        for (int i = 0; item_of<GROUP>(p.s, blockIdx.x, i, rank, it); ++i) {
            float acc[SUMS ? kLower : 1];
            if constexpr (SUMS) {
#pragma unroll
                for (int j = 0; j < kLower; ++j) acc[j] = 0.0f;
            }
            uint32_t held[2][16], cols = 0;
            int buf = 0;
            // A tile of one run, or (SUMS) the sums of several; the last one's columns of TMEM are kept until all is stored
            for (int b = it.first; b < it.last; b += p.run, ++runs) {
                if (SUMS && b > it.first) release(buf);
                buf = (int)(runs & 1);
                ok = ok && mbar_wait_cycles_warp(smem_u32(&sh.acc_full[buf]), (uint32_t)(runs >> 1) & 1u, p.limit);
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                cols = lanes + buf * second;
                if constexpr (SUMS) {
#pragma unroll
                    for (int c = 0; c < kLower; c += 16) {
                        if (c >= count) break;
                        tmem_begin16(cols + c, held[0]);
                        tmem_wait16(held[0]);
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[c + j] += __uint_as_float(held[0][j]);
                    }
                }
            }
            if constexpr (SUMS) {
                // The tile's sums go back to TMEM, and from there to memory in a loop that stays in the instruction cache.
#pragma unroll
                for (int c = 0; c < kLower; c += 16) {
                    if (c >= count) break;
                    tmem_store16(cols + c, acc + c);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            } else if constexpr (kFirst != 0) {
                if (count > 0) {
                    tmem_begin16(cols + col(0), held[0]);
                    tmem_begin16(cols + col(16), held[1]);
                    tmem_wait16(held[0]);
                    tmem_wait16(held[1]);
                }
                if (shares && upper == (buf == 0)) {
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) arrive_cluster(edge + buf * 8);
                }
            }
            if (GROUP == 1 && !ok) sh.failed = 1;
            if (count > 0) {
                const Out<T, S> out(p, it, part, x0, count, row, ok);
                if (kFirst == 0) {
                    tmem_begin16(cols, held[0]);
                    tmem_wait16(held[0]);
                }
                // the next 16 columns on their way
#pragma unroll 1
                for (int c = 0; c < count; c += 32) {
                    if (kFirst == 0 || c > 0) tmem_begin16(cols + col(c + 16), held[1]);
                    out.put(held[0], col(c));
                    if (kFirst == 0 || c > 0) tmem_wait16(held[1]);
                    const bool more = c + 32 < count;
                    if (more) tmem_begin16(cols + col(c + 32), held[0]);
                    out.put(held[1], col(c + 16));
                    if (more) tmem_wait16(held[0]);
                }
            }
            release(buf);
        }
    } else {
        if constexpr (GROUP == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsExp));
        // Exponents: each warp its quarter of the lanes, all four the same words.  A tile's first words come from memory
        // (the next ones from the same sectors): they are fetched a group ahead, across tiles.
        constexpr int kN = S::kExpCols;
        const uint32_t to = in_cta(smem_u32(&sh.exp_full[0]), leader);
        const uint32_t lanes = tmem + S::kExps + ((uint32_t)((warp & 3) * 32) << 16);
        const uint8_t *rows[kN];
        Item it;
        int next = 0;
        int g = 0, end = 0;  // groups of the item that is fetched
        uint32_t groups = 0;
        bool ok = true, held = false;  // whether v[0] holds words; v[1] receives the next ones meanwhile
        uint32_t v[2][kN] = {};
#pragma unroll 1
        for (bool more = true; ok && (more || held);) {
            if (more && g == end) {
                more = item_of<GROUP>(p.s, blockIdx.x, next, rank, it);
                ++next;
                if (more) {
                    g = it.first >> 2;
                    end = ((it.last - 1) >> 2) + 1;
#pragma unroll
                    for (int c = 0; c < kN; ++c) {
                        const Exps &e = c < 4 ? p.ew : p.ex;
                        const int64_t row = c < 4 ? (int64_t)it.tw * S::kFeatures + pair_rank * 128 + c * 32 + lane
                                                  : (int64_t)it.tx * p.s.tokens + (c - 4) * 32 + lane;
                        const bool in = row < e.rows && (c < 4 || (c - 4) * 32 + lane < p.s.tokens);
                        rows[c] = in ? e.p + (row >> e.shift) * e.pitch : nullptr;
                    }
                }
            }
            if (more) {
#pragma unroll
                for (int c = 0; c < kN; ++c) v[1][c] = rows[c] ? __ldg(reinterpret_cast<const uint32_t *>(rows[c]) + g) : 0u;
                ++g;
            }
            if (held) {
                const int eb = (int)(groups & 1);
                if (groups >= 2) ok = mbar_wait_cycles_warp(smem_u32(&sh.exp_empty[eb]), ((groups >> 1) + 1u) & 1u, p.limit);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
                for (int c = 0; c < kN; c += 4) tmem_store4(lanes + eb * kN + c, v[0] + c);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) arrive_cluster(to + eb * 8);
                ++groups;
            }
            held = more;
#pragma unroll
            for (int c = 0; c < kN; ++c) v[0][c] = v[1][c];
        }
        // the MMAs' last signals arrive before the CTA may leave
        for (uint32_t g = groups >= 2 ? groups - 2 : 0; ok && g < groups; ++g)
            ok = mbar_wait_cycles_warp(smem_u32(&sh.exp_empty[g & 1]), (uint32_t)(g >> 1) & 1u, p.limit);
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (GROUP == 2) cluster_sync();
    else if (p.s.splits > 1) {
        Item it;
        item_of<GROUP>(p.s, blockIdx.x, 0, rank, it);
        join_cluster<T, S>(p, it, sh, part, rank);
    }
    if (warp == 1) {
        if constexpr (GROUP == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kTmem));
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kTmem));
    }
}

// The cut tiles' sums, range by range in order, to y.  A block takes 4 tokens of 256 features, a thread 4 adjacent
// features of one.
template <typename T, class S>
__global__ void __launch_bounds__(256) k_join(const __grid_constant__ Params p)
{
    constexpr int kAcross = S::kFeatures / 4, kRows = 256 / kAcross;
    cudaGridDependencySynchronize();  // launched to start as k_mm drains
    const int c = (int)(blockIdx.x / (S::kTokens / kRows));
    const int x = (int)(blockIdx.x % (S::kTokens / kRows)) * kRows + (int)threadIdx.x / kAcross, w = (int)(threadIdx.x % kAcross) * 4;
    const int lo = p.s.from[c], hi = p.s.to[c];
    if (lo == hi) return;  // one range has the whole tile, and has stored it
    Item it;
    tile_place(p.s, p.s.whole + (uint32_t)c, it);
    const int64_t feature = (int64_t)it.tw * S::kFeatures + w, token = (int64_t)it.tx * p.s.tokens + x;
    if (feature >= p.features || x >= p.s.tokens || token >= p.tokens) return;
    const int n = (int)min((int64_t)4, p.features - feature);
    const float *s = p.parts + ((int64_t)(c + lo) * S::kTokens + x) * S::kFeatures + w;
    float v[4] = {};
#pragma unroll 4
    for (int r = 0; r <= hi - lo; ++r) {
        // columns of features that do not exist were not written
        float a[4];
        if (n == 4) {
            *reinterpret_cast<float4 *>(a) = *reinterpret_cast<const float4 *>(s + (int64_t)r * S::kTokens * S::kFeatures);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] = j < n ? s[(int64_t)r * S::kTokens * S::kFeatures + j] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += a[j];
    }
    T *const y = static_cast<T *>(p.y) + token * p.sy + feature;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < n) {
            if (p.bias) v[j] += p.bias[feature + j];
            if constexpr (sizeof(T) == 4) {
                if (p.accumulate) v[j] += y[j];
            }
            y[j] = rounded<T>(v[j]);
        }
}

template <class S>
size_t workspace_of(int64_t m, int64_t n, int64_t k)
{
    return (size_t)part_tiles(schedule<S>(n, m, k)) * S::kTokens * S::kFeatures * sizeof(float);
}

bool encode_rows(CUtensorMap *map, const void *p, int64_t rows, int64_t pitch, int box_rows)
{
    const EncodeFn encode = encode_fn();
    const cuuint64_t dims[2] = {(cuuint64_t)pitch, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows}, ones[2] = {1, 1};
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, box, ones,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

Exps exps_of(const void *p, int tile, int64_t rows, const Fp8Layout &l)
{
    return Exps{static_cast<const uint8_t *>(p) + l.exps_off, rows, l.exp_pitch, tile ? 7 : 0};
}

template <typename T, class S, bool SUMS>
cudaError_t launch_kernels(const Params &p, cudaStream_t stream)
{
    auto kern = k_mm<T, S::kGroup, S::kTokens, SUMS>;
    int per_sm = 0, sms = 0;
    cudaError_t e = kernel_occupancy(reinterpret_cast<const void *>(kern), S::kThreads, S::kSmemBytes, &per_sm, &sms);
    if (e != cudaSuccess) return e;
    static const int regs = num_regs(kern);
    if (S::kGroup == 2 && regs < kRegsLaunch) return cudaErrorInvalidKernelImage;  // setmaxnreg would wait
    const int64_t ctas = S::kGroup == 2 ? 2 * (int64_t)p.s.units : (int64_t)p.s.tiles_w * p.s.tiles_x * p.s.splits;
    if (ctas > (int64_t(1) << 31) - 1) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)(S::kGroup == 2 ? 2 : p.s.splits);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    if (S::kGroup == 1 || e != cudaSuccess || !part_tiles(p.s)) return e;
    cfg.gridDim = dim3((unsigned)(p.s.cut * (S::kTokens / (1024 / S::kFeatures))));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_join<T, S>, p);
}

template <class S>
cudaError_t launch_shape(const Fp8MatmulArgs &g, cudaStream_t stream)
{
    Params p;
    const Fp8Layout lx = fp8_layout(g.tile_a, g.m, g.k), lw = fp8_layout(g.tile_b, g.n, g.k);
    p.s = schedule<S>(g.n, g.m, g.k);
    p.ew = exps_of(g.b, g.tile_b, g.n, lw);
    p.ex = exps_of(g.a, g.tile_a, g.m, lx);
    p.idesc = instr_desc(g.format_b, g.format_a, S::kFeatures, p.s.tokens);
    p.tokens = g.m;
    p.features = g.n;
    p.bias = g.bias;
    p.y = g.y;
    p.sy = g.m > 1 ? g.y_stride : 0;
    p.accumulate = g.accumulate;
    p.quads = reinterpret_cast<uintptr_t>(g.y) % 8 == 0 && (g.m == 1 || g.y_stride % 4 == 0);
    p.parts = reinterpret_cast<float *>(g.ws);
    // two seconds at 1.97 GHz, three at the power cap's 1.39 GHz; the longest wait, for a tile, is some microseconds a
    // thousand columns
    p.limit = 4000000000ll;
    if (!encode_rows(&p.w, g.b, g.n, lw.code_pitch, 128) ||
        !encode_rows(&p.x, g.a, g.m, lx.code_pitch, S::kGroup == 2 ? p.s.tokens / 2 : S::kTokens))
        return cudaErrorInvalidValue;
    p.run = run_of(g.dtype);
    const bool sums = p.s.blocks > p.run;
    if (g.dtype == GQ_FLOAT32) return sums ? launch_kernels<float, S, true>(p, stream) : launch_kernels<float, S, false>(p, stream);
    if (g.dtype == GQ_BFLOAT16)
        return sums ? launch_kernels<__nv_bfloat16, S, true>(p, stream) : launch_kernels<__nv_bfloat16, S, false>(p, stream);
    return sums ? launch_kernels<__half, S, true>(p, stream) : launch_kernels<__half, S, false>(p, stream);
}

}  // namespace

size_t fp8_matmul_workspace(int64_t m, int64_t n, int64_t k)
{
    if (m == 0) return 0;
    return kind_of(m) == kByPairs ? workspace_of<Pair>(m, n, k) : 0;
}

cudaError_t launch_fp8_matmul(const Fp8MatmulArgs &g, cudaStream_t stream)
{
    switch (kind_of(g.m)) {
    case kByPairs: return launch_shape<Pair>(g, stream);
    case kOne128: return launch_shape<Shape<1, 128>>(g, stream);
    case kOne64: return launch_shape<Shape<1, 64>>(g, stream);
    default: return launch_shape<Shape<1, 32>>(g, stream);
    }
}

}  // namespace gq
