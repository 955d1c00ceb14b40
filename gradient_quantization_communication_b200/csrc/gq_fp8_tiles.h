// gq_fp8_tiles.h -- how the products of packed matrices are cut into tiles, and how these are spread over the device:
// the shapes, the schedule that the host makes, and the items that each role of the kernel takes from it.  Host and
// device: a test walks over all items on the CPU.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define GQ_TILES_FN __host__ __device__ __forceinline__
#else
#define GQ_TILES_FN inline
#endif

namespace gq {
namespace tiles {

// How a tile is made: 128 * group features x up to TN tokens by `group` CTAs.
//   2  a pair of CTAs shares the operands of a large tile, and walks over tiles.  Their tokens are chosen by the call
//      (schedule_pairs).  Two accumulators and the exponents leave room for 224; with 256 the accumulators share 32
//      columns, which the epilogue reads first, and the MMAs of the next tile or run wait for that;
//   1  a CTA makes a tile of few tokens, or a part of it: clusters of CTAs cut the columns among them and add their
//      sums up through each other's shared memory.
template <int GROUP, int TN>
struct Shape {
    static constexpr int kGroup = GROUP, kTokens = TN, kFeatures = 128 * GROUP;
    static constexpr int kPerSm = GROUP == 2 || TN > 64 ? 1 : 2;  // CTAs of an SM
    static constexpr int kEpiWarps = GROUP == 2 ? 8 : 4, kThreads = (8 + kEpiWarps) * 32;
    static constexpr int kWBytes = 128 * 128, kXRows = TN / GROUP, kXBytes = kXRows * 128;
    static constexpr int kStageBytes = kWBytes + kXBytes;
    static constexpr int kStages = 229376 / kPerSm / kStageBytes < 8 ? 229376 / kPerSm / kStageBytes : 8;
    static constexpr int kSmemBytes = kStages * kStageBytes + 1024;
    // single CTAs: a part of a tile, binary32, in the stages' place once the last MMA has read them
    static constexpr int kPartBytes = GROUP == 1 ? TN * 128 * 4 : 0;
    static_assert(kPartBytes <= kStages * kStageBytes, "a part takes the stages' place");
    // TMEM: two accumulators, the second from column kSecond on (or at a tile's fewer tokens), then two buffers of
    // exponents (4 columns for 128 features, TN / 32 but at least 4 for the tokens)
    static constexpr int kExpCols = 4 + (TN > 128 ? 8 : 4);
    static constexpr int kSecond = TN > 128 ? 224 : TN;
    static constexpr int kExps = kSecond + TN;
    static constexpr int kTmem = kExps + 2 * kExpCols <= 128 ? 128 : kExps + 2 * kExpCols <= 256 ? 256 : 512;
    // all CTAs that fit an SM get theirs at once, those of calls on other streams too: none waits for TMEM that another
    // keeps until its cluster's join
    static_assert(kPerSm * kTmem <= 512 && (kPerSm == 1 || 3 * kSmemBytes > 232448), "TMEM");
};
// The stages' (and a part's) address in dynamic shared memory that begins at `base`: the 128-byte swizzle wants 1024 bytes, a
// part's loads 16, and where dynamic shared memory begins behind the static is the toolchain's matter.
GQ_TILES_FN constexpr uint32_t ring_start(uint32_t base) { return (base + 1023u) & ~1023u; }

constexpr int kMostTokens = 256;
using Pair = Shape<2, kMostTokens>;
static_assert(Pair::kExps + 2 * Pair::kExpCols <= 512, "TMEM");
constexpr int kHeld = 32;  // columns that the epilogue reads first: those that two accumulators may share
static_assert(Pair::kTokens - Pair::kSecond <= kHeld, "shared columns");

// Stages summed in TMEM before their sums are added to registers, rounded.  The tensor cores cut off: of every 32 products and
// the sum so far what lies below 2^-25 of the largest one's power of two, then of their sum what lies below 2^-23 (found by
// single products of powers of two beside a large one).  A run of 4096 columns is so off by at most 128 (2^-20 + 2^-23) =
// 1.4e-4 of its largest partial sum, the most where one product outweighs all others; by 7e-7 with positive products of about
// one size (e^N(0, 2)), and up to 3.5e-5 with some thousand times larger among them (e^N(0, 8)).  16384 columns: four times
// that, 5.5e-4 at most, beside half a step of the result's own rounding, 3.9e-3 in bfloat16 and 4.9e-4 in float16.
constexpr int kRunWide = 32, kRun16 = 128;
constexpr int kPairs = 74;        // CTA pairs of the 148 SMs
constexpr int kMaxSplits = 8;     // CTAs of a portable cluster

// How the tiles are spread over the pairs: whole rounds of a tile a pair first; the stages of the last, partial round's
// tiles are one line, cut into `ranges` equal ranges, one a pair.  A range's part of a tile goes to the workspace, where a
// second kernel joins them, unless it is the whole tile.
struct Schedule {
    int tokens;            // of a tile
    int tiles_w, tiles_x;
    int blocks;            // stages of a tile
    int splits;            // single CTAs: parts of each tile; nothing of the following
    uint32_t whole;        // tiles of the whole rounds
    int cut, ranges;       // tiles of the last one, and the ranges that they are cut into
    int units;             // pairs launched
    int64_t start[kPairs + 1];
    uint8_t tile[kPairs], from[kPairs], to[kPairs];
};

template <class S>
Schedule schedule_single(int64_t features, int64_t tokens, int64_t k)
{
    Schedule s = {};
    s.tokens = S::kTokens;
    s.tiles_w = (int)((features + 127) / 128);
    s.tiles_x = (int)((tokens + S::kTokens - 1) / S::kTokens);
    s.blocks = (int)((k + 127) / 128);
    // as many parts as there is room for, of two stages at least; of fewer than eight only to fill the SMs (16 tokens,
    // 4096 columns: 4096 features 8.2 us with four parts, 8.6 with eight; 1000 features 8.4 and 7.0)
    const int64_t tiles = (int64_t)s.tiles_w * s.tiles_x;
    s.splits = 1;
    while (s.splits < kMaxSplits && tiles * s.splits * 2 <= 148 * S::kPerSm && s.splits * 4 <= s.blocks &&
           (tiles * s.splits < 128 || s.blocks / s.splits > 8))
        s.splits *= 2;
    return s;
}

// The pairs' tiles: of the widths that TMEM holds the one that is done first, in cycles as measured.
inline Schedule schedule_pairs(int64_t features, int64_t tokens, int64_t k)
{
    Schedule s = {};
    s.splits = 1;
    s.tiles_w = (int)((features + Pair::kFeatures - 1) / Pair::kFeatures);
    s.blocks = (int)((k + 127) / 128);
    double best = 1e300;
    for (int tx = kMostTokens; tx >= 64; tx -= 32) {  // pairs take their N in steps of 32
        const int64_t tiles_x = (tokens + tx - 1) / tx, tiles = s.tiles_w * tiles_x;
        // a stage: 550 cycles with 128 tokens, 620 with 224, 650 with 256, for its way through L2 (13.5 TB/s in all)
        const double stage = 430 + 0.85 * tx;
        const int64_t cut = tiles % kPairs, rounds = tiles / kPairs;
        if (tx > Pair::kSecond && s.blocks > kRunWide) continue;  // the MMAs would wait at every run: 890 us against 810
        const double before = (double)rounds * s.blocks * stage;
        auto take = [&](int64_t ranges, double cycles) {
            if (cycles >= best) return;
            best = cycles;
            s.tokens = tx;
            s.tiles_x = (int)tiles_x;
            s.cut = (int)cut;
            s.whole = (uint32_t)(tiles - cut);
            s.ranges = (int)ranges;
        };
        if (!cut) {
            take(0, before + 24.0 * tx);
            continue;
        }
        // the last, partial round: a tile a pair, as many equal parts of every tile as there are pairs for, or equal ranges
        // for all pairs.  The second kernel, and its parts' way through L2, cost some microseconds.
        take(cut, before + s.blocks * stage + 24.0 * tx);
        const int64_t total = cut * s.blocks, most = total / 4 < kPairs ? total / 4 : kPairs;
        for (int64_t r = 2 * cut; r < most + cut; r += cut) {
            if (r > most) r = most;
            if (r <= cut) break;
            const double parts = r % cut == 0 ? (double)r : (double)(cut + r - 1);
            take(r, before + (double)((total + r - 1) / r) * stage + 24.0 * tx + 5000.0 + 0.25 * parts * tx);
            if (r == most) break;
        }
    }
    s.units = s.whole ? kPairs : s.ranges;
    const int64_t total = (int64_t)s.cut * s.blocks;
    for (int p = 0; p <= s.ranges; ++p) s.start[p] = s.ranges ? total * p / s.ranges : 0;
    for (int p = 0; p < s.ranges; ++p) s.tile[p] = (uint8_t)(s.start[p] / s.blocks);
    for (int c = 0, p = 0; c < s.cut; ++c) {
        while (s.start[p + 1] <= (int64_t)c * s.blocks) ++p;
        s.from[c] = (uint8_t)p;
        while (s.start[p + 1] < (int64_t)(c + 1) * s.blocks) ++p;
        s.to[c] = (uint8_t)p;
    }
    return s;
}
template <class S>
Schedule schedule(int64_t features, int64_t tokens, int64_t k)
{
    if constexpr (S::kGroup == 1) return schedule_single<S>(features, tokens, k);
    else return schedule_pairs(features, tokens, k);
}
// Partial tiles that the workspace holds: range p's part of tile c at c + p.
inline int64_t part_tiles(const Schedule &s) { return s.ranges > s.cut ? s.cut + s.ranges - 1 : 0; }

// Which shape: tiles of 256 features by CTA pairs, or, for up to 128 tokens, 128 features by single CTAs.
enum Kind { kByPairs, kOne128, kOne64, kOne32 };
inline Kind kind_of(int64_t tokens) { return tokens > 128 ? kByPairs : tokens > 64 ? kOne128 : tokens > 32 ? kOne64 : kOne32; }

struct Item {
    int tw, tx;        // tile
    int first, last;   // its stages
    int part;          // partial tile in the workspace, -1: the whole tile
};

// Bands of 8 feature tiles, walked along the tokens: units that run together share their operands in L2.
GQ_TILES_FN void tile_place(const Schedule &s, uint32_t tile, Item &it)
{
    const uint32_t band = 8u * (uint32_t)s.tiles_x, g = tile / band, rest = tile - g * band;
    const uint32_t wide = (uint32_t)s.tiles_w - g * 8u < 8u ? (uint32_t)s.tiles_w - g * 8u : 8u;
    it.tx = (int)(rest / wide);
    it.tw = (int)(g * 8u + rest - (uint32_t)it.tx * wide);
}

// The i-th item of the pair that a block belongs to, or a single CTA's only one (i = 0); rank: in its cluster.
template <int GROUP>
GQ_TILES_FN bool item_of(const Schedule &s, uint32_t block, int i, uint32_t rank, Item &it)
{
    if constexpr (GROUP == 1) {
        if (i != 0) return false;
        const uint32_t tile = block / (uint32_t)s.splits;
        it.tx = (int)(tile / (uint32_t)s.tiles_w);
        it.tw = (int)(tile - (uint32_t)it.tx * (uint32_t)s.tiles_w);
        it.first = (int)((int64_t)s.blocks * rank / s.splits);
        it.last = (int)((int64_t)s.blocks * (rank + 1) / s.splits);
        it.part = s.splits > 1 ? 0 : -1;
        return true;
    }
    const uint32_t at = (block >> 1) + (uint32_t)i * (uint32_t)s.units;
    uint32_t tile = at;
    if (at < s.whole) {
        it.first = 0;
        it.last = s.blocks;
        it.part = -1;
    } else {
        // part m of unit p's range, which lies in the m-th tile that the range touches
        const uint32_t j = at - s.whole, m = j / (uint32_t)s.units, p = j - m * (uint32_t)s.units;
        if (p >= (uint32_t)s.ranges) return false;
        const int64_t lo = s.start[p], hi = s.start[p + 1];
        const int c = (int)(s.tile[p] + m);
        const int64_t from = (int64_t)c * s.blocks;
        it.first = (int)((lo > from ? lo : from) - from);
        it.last = (int)((hi < from + s.blocks ? hi : from + s.blocks) - from);
        if (it.first >= it.last) return false;
        it.part = it.first == 0 && it.last == s.blocks ? -1 : c + (int)p;
        tile = s.whole + (uint32_t)c;
    }
    tile_place(s, tile, it);
    return true;
}

}  // namespace tiles
}  // namespace gq
