// gq_ring.cuh -- the ring of stages that the weight gradient's warps pass through, and which phase of which
// barrier each of them waits for.  Host and device: tests run it under a model of the barriers.
//
// A wait names a phase by its parity alone: it passes as soon as the barrier's present phase has the other parity.
// That is the phase meant only if the waiter knows the phase before it to be complete.  The warps that decode take
// every second stage in turn, so of a ring of five they see every second use of each, and nothing tells them that
// the use between is past: its data may still be on the way when later stages, which the memory answered sooner,
// have been decoded.  So the barriers that say "full" are two a stage, one for its even uses and one for its
// odd ones, and each of them is waited for at every one of its phases by the same warps.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define GQ_RING_FN __host__ __device__ __forceinline__
#else
#define GQ_RING_FN inline
#endif

namespace gq {

// Five stages of everything.  A ring of its own for the decoded A, so that six stages could be under way,
// needs one more signal and wait a stage and measured slower (1.81 against 1.74 ms, 16384 x 4096 x 16384).
constexpr int kStages = 5;
constexpr int kFullBars = 2 * kStages;

// Position in the ring.
struct Ring {
    int st = 0;            // stage
    uint32_t turn = 0;     // times around
    bool wrapped = false;  // every stage has been used before

    GQ_RING_FN void next(int by = 1)
    {
        st += by;
        if (st >= kStages) {
            st -= kStages;
            ++turn;
            wrapped = true;
        }
    }
    GQ_RING_FN void back()
    {
        if (--st < 0) {
            st = kStages - 1;
            --turn;
        }
    }
    // The barrier that says that this use's data have arrived, and its phase's parity.
    GQ_RING_FN int full() const { return st + ((turn & 1u) ? kStages : 0); }
    GQ_RING_FN uint32_t full_parity() const { return (turn >> 1) & 1u; }
    // Parity of this use's phase of the stage's other barriers, which their waiters see at every use, and of the
    // use before.
    GQ_RING_FN uint32_t parity() const { return turn & 1u; }
    GQ_RING_FN uint32_t parity_before() const { return (turn & 1u) ^ 1u; }
};

}  // namespace gq
