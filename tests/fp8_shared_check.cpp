// Where the 8-bit products' kernels put their stages and parts in dynamic shared memory, for every place at which that may
// begin: on 1024 bytes, and inside what the launch asks for.
#include <cstdio>

#include "gq_fp8_tiles.h"

using namespace gq::tiles;

template <class S>
static bool holds()
{
    for (uint32_t base = 0; base < 4096; base += 4) {
        const uint32_t at = ring_start(base), end = base + S::kSmemBytes;
        if (at % 1024 || at < base || at + S::kStages * S::kStageBytes > end || at + S::kPartBytes > end) {
            std::printf("tokens %d, base %u\n", S::kTokens, base);
            return false;
        }
    }
    // stages and both operands in them stay on 1024 bytes
    return S::kStageBytes % 1024 == 0 && S::kWBytes % 1024 == 0 && S::kSmemBytes <= 232448;
}

int main()
{
    const bool ok = holds<Pair>() && holds<Shape<1, 128>>() && holds<Shape<1, 64>>() && holds<Shape<1, 32>>();
    std::printf(ok ? "ok\n" : "wrong\n");
    return !ok;
}
