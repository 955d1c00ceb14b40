// The roles of the weight gradient's kernel (gq_wgrad.cu) as far as they wait and signal, run with the ring that
// the kernel uses (gq_ring.cuh) under a model of the barriers, with random delays of every step and of every
// copy, some of them very long.  A wait names its phase by parity, as the hardware's do; the model knows which
// phase was meant, and a wait that passes before it is complete is a failure.
//
// Arguments: seed, number of runs, and "plain" to wait on one "full" barrier a stage by the use's parity (which the
// decoding warps, seeing every second use, must not: the model has to find it).  Exit status 0: no failure.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <deque>
#include <random>
#include <vector>
#include "gq_ring.cuh"
using gq::kFullBars;
using gq::kStages;
using gq::Ring;

struct Barrier {
    int count = 0, pending = 0, phase = 0;
    void init(int n) { count = pending = n; }
    void arrive()
    {
        if (--pending == 0) {
            pending = count;
            ++phase;
        }
    }
    bool passes(uint32_t parity) const { return ((uint32_t)phase & 1u) != parity; }
};

struct Cta {
    Barrier full[kFullBars], empty[kStages];
};

struct Sim {
    std::mt19937 rng;
    int total = 0;
    bool plain = false;
    Cta cta[2];
    Barrier ready[kStages];
    struct Event {
        long at;
        Barrier *b;
    };
    std::vector<Event> events;
    long now = 0;
    bool bad = false;

    int full_bar(const Ring &r) const { return plain ? r.st : r.full(); }
    uint32_t full_parity(const Ring &r) const { return plain ? r.parity() : r.full_parity(); }
    // Phases of the barrier complete once use `use` (0, 1, ...) of the stage has arrived.
    int full_phases(int use) const { return plain ? use + 1 : use / 2 + 1; }

    long delay()
    {
        const unsigned k = rng() % 64;
        return (long)(k == 0 ? 200 + rng() % 800 : k < 8 ? 20 + rng() % 40 : 1 + rng() % 8);
    }
    // A wait: passes or not; the phase meant must be complete if it does.
    bool wait(const Barrier &b, uint32_t parity, int phases)
    {
        if (!b.passes(parity)) return false;
        if (b.phase < phases) bad = true;
        return true;
    }
    // An actor: next step's time, what it waits for.
    struct Actor {
        int role, cta, i = 0;  // role 0: copies, 1: exponents, 2: MMA, 3 and 4: a decoding warp of even / odd stages
        Ring r;
        long at = 0;
        bool started = false;
    };

    bool step(Actor &a)  // true: it made progress
    {
        Cta &c = cta[a.cta];
        const int use = a.i / kStages;  // of its stage
        switch (a.role) {
        case 0:
        case 1:
            if (a.r.wrapped && !wait(c.empty[a.r.st], a.r.parity_before(), use)) return false;
            // the copy's bytes are one arrival, the 32 of the exponents another
            events.push_back({now + delay(), &c.full[full_bar(a.r)]});
            a.r.next();
            ++a.i;
            break;
        case 2:
            if (!wait(ready[a.r.st], a.r.parity(), use + 1)) return false;
            {
                const long at = now + delay();
                events.push_back({at, &cta[0].empty[a.r.st]});
                events.push_back({at + (long)(rng() % 4), &cta[1].empty[a.r.st]});
            }
            a.r.next();
            ++a.i;
            break;
        default:
            if (!a.started) {
                a.started = true;
                a.r.next(a.role - 3);
                a.i = a.role - 3;
                break;
            }
            if (!wait(c.full[full_bar(a.r)], full_parity(a.r), full_phases(use))) return false;
            events.push_back({now + delay(), &ready[a.r.st]});
            a.at = events.back().at;  // it decodes until then
            a.r.next(2);
            a.i += 2;
            return true;
        }
        a.at = now + delay();
        return true;
    }

    int run(int stages)
    {
        total = stages;
        std::vector<Actor> actors;
        for (int k = 0; k < 2; ++k) {
            for (auto &b : cta[k].full) b.init(2);
            for (auto &b : cta[k].empty) b.init(1);
            actors.push_back({0, k});
            actors.push_back({1, k});
            for (int w = 0; w < 8; ++w) actors.push_back({3 + (w >> 2), k});
        }
        for (auto &b : ready) b.init(8);
        actors.push_back({2, 0});
        for (long idle = 0; idle < 20000 && !bad; ++now) {
            bool any = false, left = false;
            for (size_t e = 0; e < events.size();) {
                if (events[e].at > now) {
                    ++e;
                    continue;
                }
                events[e].b->arrive();
                events[e] = events.back();
                events.pop_back();
                any = true;
            }
            for (Actor &a : actors) {
                if (a.started && a.i >= total) continue;
                if (a.role < 3 && a.i >= total) continue;
                left = true;
                if (a.at <= now) any |= step(a);
                else any = true;
            }
            if (!left && events.empty()) return 0;
            idle = any || !events.empty() ? 0 : idle + 1;
        }
        return bad ? 1 : 2;  // 2: nobody moves any more
    }
};

int main(int argc, char **argv)
{
    const unsigned seed = argc > 1 ? (unsigned)atoi(argv[1]) : 1;
    const int runs = argc > 2 ? atoi(argv[2]) : 100;
    int early = 0, stuck = 0;
    for (int k = 0; k < runs; ++k) {
        Sim s;
        s.rng.seed(seed * 100003u + (unsigned)k);
        s.plain = argc > 3 && !strcmp(argv[3], "plain");
        const int r = s.run(k % 8 == 0 ? k / 8 % 24 : 100);
        early += r == 1;
        stuck += r == 2;
    }
    printf("runs %d, waits that passed early in %d, stuck %d\n", runs, early, stuck);
    return early || stuck ? 1 : 0;
}
