// Walks over the items of every pair and cluster of the 8-bit products' schedules and checks that each stage of each
// tile is taken exactly once, that partial tiles have places of their own inside the workspace, and that the second
// kernel's ranges name exactly these.
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <vector>

#include "gq_fp8_tiles.h"

using namespace gq::tiles;

static void fail(const char *what, int64_t n, int64_t m, int64_t k)
{
    std::printf("%s: features %lld tokens %lld columns %lld\n", what, (long long)n, (long long)m, (long long)k);
    std::exit(1);
}

template <class S>
static void check(int64_t n, int64_t m, int64_t k)
{
    const Schedule s = schedule<S>(n, m, k);
    const int64_t blocks = (k + 127) / 128;
    if (s.blocks != blocks) fail("stages", n, m, k);
    if (s.tokens < 32 || s.tokens > S::kTokens || s.tokens % 32 || (S::kGroup == 1 && s.tokens != S::kTokens)) fail("tile", n, m, k);
    if ((int64_t)s.tiles_w * S::kFeatures < n || (int64_t)(s.tiles_w - 1) * S::kFeatures >= n) fail("features", n, m, k);
    if ((int64_t)s.tiles_x * s.tokens < m || (int64_t)(s.tiles_x - 1) * s.tokens >= m) fail("tokens", n, m, k);
    // a tile that is more than a run may not share columns of its accumulators
    if (S::kGroup == 2 && s.tokens > S::kSecond && blocks > kRunWide) fail("shared columns over runs", n, m, k);
    const int64_t ctas = S::kGroup == 2 ? 2 * (int64_t)s.units : (int64_t)s.tiles_w * s.tiles_x * s.splits;
    if (S::kGroup == 2 && (s.units < 1 || s.units > kPairs)) fail("pairs", n, m, k);
    if (S::kGroup == 1 && (s.splits < 1 || s.splits > kMaxSplits || s.splits > blocks)) fail("splits", n, m, k);
    std::map<std::pair<int, int>, std::vector<std::pair<int, int>>> tiles;
    std::set<int> parts;
    for (int64_t block = 0; block < ctas; block += S::kGroup == 2 ? 2 : 1) {
        const uint32_t rank = S::kGroup == 2 ? 0 : (uint32_t)(block % s.splits);
        Item a, b;
        for (int i = 0; item_of<S::kGroup>(s, (uint32_t)block, i, rank, a); ++i) {
            if (S::kGroup == 2 && (!item_of<2>(s, (uint32_t)block + 1, i, 1, b) || a.tw != b.tw || a.tx != b.tx ||
                                   a.first != b.first || a.last != b.last || a.part != b.part))
                fail("the pair's CTAs differ", n, m, k);
            if (a.tw < 0 || a.tw >= s.tiles_w || a.tx < 0 || a.tx >= s.tiles_x || a.first < 0 || a.first >= a.last || a.last > blocks)
                fail("item", n, m, k);
            tiles[{a.tw, a.tx}].push_back({a.first, a.last});
            const bool whole = a.first == 0 && a.last == blocks;
            if (S::kGroup == 2 && whole != (a.part < 0)) fail("part of a whole tile", n, m, k);
            if (S::kGroup == 1 && (s.splits > 1) != (a.part >= 0)) fail("part", n, m, k);
            if (S::kGroup == 2 && a.part >= 0 && (a.part >= part_tiles(s) || !parts.insert(a.part).second)) fail("place of a part", n, m, k);
        }
        if (S::kGroup == 2 && item_of<2>(s, (uint32_t)block + 1, 1 << 20, 1, b)) fail("endless", n, m, k);
    }
    if ((int64_t)tiles.size() != (int64_t)s.tiles_w * s.tiles_x) fail("tiles", n, m, k);
    for (auto &t : tiles) {
        std::vector<char> seen((size_t)blocks, 0);
        for (auto &r : t.second)
            for (int b = r.first; b < r.second; ++b)
                if (seen[(size_t)b]++) fail("a stage twice", n, m, k);
        for (char c : seen)
            if (!c) fail("a stage missing", n, m, k);
    }
    std::set<int> joined;
    for (int c = 0; c < s.cut && S::kGroup == 2; ++c)
        for (int p = s.from[c]; p <= s.to[c] && s.from[c] != s.to[c]; ++p) joined.insert(c + p);
    if (joined != parts) fail("parts and ranges", n, m, k);
}

static void check_all(int64_t n, int64_t m, int64_t k)
{
    switch (kind_of(m)) {
    case kByPairs: check<Pair>(n, m, k); break;
    case kOne128: check<Shape<1, 128>>(n, m, k); break;
    case kOne64: check<Shape<1, 64>>(n, m, k); break;
    default: check<Shape<1, 32>>(n, m, k);
    }
}

int main()
{
    std::mt19937 g(1);
    auto log_uniform = [&](double lo, double hi) {
        return (int64_t)std::exp(std::uniform_real_distribution<double>(std::log(lo), std::log(hi + 1))(g));
    };
    for (int64_t m : {1, 16, 32, 33, 64, 65, 128, 129, 256, 257, 512, 3001, 8192})
        for (int64_t n : {1, 127, 128, 129, 256, 257, 1000, 2499, 4096, 11008})
            for (int64_t k : {1, 127, 128, 129, 256, 300, 512, 1000, 4096, 4097, 8192, 70000}) check_all(n, m, k);
    for (int i = 0; i < 4000; ++i) check_all(log_uniform(1, 20000), log_uniform(1, 20000), log_uniform(1, 40000));
    std::printf("ok\n");
    return 0;
}
