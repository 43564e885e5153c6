// Drives ring_places.cuh as a warp of the few-row kernels does: DEPTH loads ahead, then read one, load one.
// Loads land in any order and at any time; in some runs one wait gives up on a load that is still in flight.
// Exit code 0: in no run was a slot read before its load had landed, or waited for without a load, or written
// by a load after the end.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "ring_places.cuh"

namespace {

struct Slot { int phases = 0, load = -1; bool flying = false; };   // phases: finished ones of its barrier

template <int DEPTH>
bool run(unsigned seed, int pieces, int gives_up_at) {
    std::mt19937 rng(seed);
    std::vector<Slot> slots(DEPTH);
    RingPlaces<DEPTH> ring;
    int issued = 0, waits = 0, bad = 0;
    bool gave_up = false;
    auto land = [&](Slot& s) { s.flying = false; ++s.phases; };
    auto some_land = [&] { for (Slot& s : slots) if (s.flying && rng() % 3 == 0) land(s); };
    auto put = [&] {
        if (issued == pieces) return;
        ring.put([&](int i) {
            if (gave_up || slots[i].flying) ++bad;
            slots[i].flying = true;
            slots[i].load = issued++;
        });
    };
    auto wait = [&](int i, uint32_t parity) {
        some_land();
        Slot& s = slots[i];
        if (((s.phases - 1) & 1) == (int)parity) return true;
        if (!s.flying) { ++bad; return false; }   // a wait for a load that nobody made
        if (waits++ == gives_up_at) { gave_up = true; return false; }
        land(s);   // waited long enough
        return true;
    };
    for (int d = 0; d < DEPTH; ++d) put();
    for (int i = 0; i < pieces; ++i) {
        const int slot = ring.take(wait);
        if (!gave_up && (slots[slot].flying || slots[slot].load != i)) ++bad;
        put();
    }
    for (Slot& s : slots) bad += s.flying;
    return bad == 0 && ring.ok != gave_up && (gave_up || issued == pieces);
}

}  // namespace

int main() {
    for (unsigned seed = 0; seed < 3000; ++seed) {
        const int pieces = 1 + seed % 37, at = seed % 3 ? (int)(seed / 3 % 23) : -1;
        if (!run<3>(seed, pieces, at) || !run<4>(seed, pieces, at) || !run<6>(seed, pieces, at)) {
            std::printf("unsound: seed %u, %d pieces, wait %d gives up\n", seed, pieces, at);
            return 1;
        }
    }
    return 0;
}
