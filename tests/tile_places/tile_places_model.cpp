// Drives tile_places.cuh on the host: quotients against the division, the tiles of uneven segments, which have to cover each
// row and channel tile once, and the stage ring of the FP8 product's two issuing warps with loads that land late.
// CONFIGS: X(stages, accumulators) of each configuration in the kernel's source.
// Exit code 0: everything holds.
#include <algorithm>
#include <cstdio>
#include <deque>
#include <random>
#include <set>
#include <tuple>
#include <vector>

#include "tile_places.cuh"

namespace {

std::mt19937_64 rng(1);
uint32_t below(uint64_t n) { return (uint32_t)(rng() % n); }
const float kErrors[] = {-3.0f / 8388608.0f, 0.0f, 3.0f / 8388608.0f};   // (the device's division is within 2 units)

bool quotients() {
    std::vector<uint32_t> ds;
    for (uint32_t d = 1; d < 260; ++d) ds.push_back(d);
    for (int k = 8; k < 32; ++k)
        for (int s = -1; s <= 1; ++s) ds.push_back((1u << k) + s);
    for (int i = 0; i < 500; ++i) ds.push_back(1 + below(0xffffffffull));
    for (uint32_t d : ds) {
        const Divisor by = divisor(d);
        const uint32_t most = 0xffffffffu / d;
        std::vector<uint64_t> ns = {0, 1, 1ull << 31, 0xffffffffull};
        for (int i = 0; i < 40; ++i) ns.push_back(below(1ull << 32));
        for (uint64_t k : {1u, 2u, 3u, most / 2, most})
            for (int s = -1; s <= 1; ++s) ns.push_back(k * d + s);
        for (uint64_t n : ns)
            if (n < 1ull << 32 && (uint32_t)n / by != (uint32_t)n / d) return std::printf("%u / %u\n", (uint32_t)n, d), false;
        if (d >= 1u << 26) continue;
        for (float e : kErrors) {
            quotient_error = e;
            for (uint64_t q : {0u, 1u, 7u, 8u, 255u, 4096u, 1u << 19})
                for (uint64_t rest : {0u, 1u % d, d / 2, d - 1}) {
                    const uint64_t n = q * d + rest;
                    if (n >= 1ull << 31) continue;
                    const Quotient got = divide((uint32_t)n, d);
                    if (got.whole != q || got.rest != rest) return std::printf("divide(%u, %u)\n", (uint32_t)n, d), false;
                }
        }
    }
    return true;
}

bool tiles(int tile, int ctiles) {
    std::vector<int> rows = {0, 1, 31, 32, 33, tile - 1, tile, tile + 1, 0, 8 * tile, 8 * tile + 1, 17 * tile - 5};
    for (int i = 0; i < 12; ++i) rows.push_back((int)below(12 * tile));
    const int E = (int)rows.size();
    std::vector<int> first(E + 1), base(E + 1, 7);
    for (int e = 0; e < E; ++e) {
        first[e + 1] = first[e] + (rows[e] + tile - 1) / tile;
        base[e + 1] = base[e] + rows[e];
    }
    std::vector<std::vector<int>> covered(E);   // how often each row
    for (int e = 0; e < E; ++e) covered[e].resize(rows[e]);
    std::set<std::tuple<int, int64_t, int>> seen;
    const Divisor by = divisor((uint32_t)ctiles);
    for (int item = 0; item < first[E] * ctiles; ++item) {
        quotient_error = kErrors[below(3)];
        const uint32_t at = (uint32_t)item / by;
        int e = E - 1;
        while (first[e] > (int)at || first[e + 1] == first[e]) --e;
        const Tile t = tile_in_segment((uint32_t)item, at, by, e, (uint32_t)first[e], (uint32_t)(first[e + 1] - first[e]), base[e], rows[e]);
        if (t.expert != e || t.m <= 0 || t.m > tile || t.n != (t.m + 31) / 32 * 32 || t.n > tile || t.channel < 0 || t.channel >= ctiles ||
            t.row0 < base[e] || t.row0 + t.m > base[e + 1] || !seen.insert({e, t.row0, t.channel}).second)
            return std::printf("tile %d of %d rows and %d channel tiles\n", item, tile, ctiles), false;
        for (int r = 0; r < t.m; ++r) ++covered[e][t.row0 - base[e] + r];
    }
    for (auto& c : covered)
        for (int n : c)
            if (n != ctiles) return std::printf("rows covered %d times of %d\n", n, ctiles), false;
    return true;
}

// Whether, in one random schedule, a warp issued a block whose load had not landed.  Barriers: finished phases, of which a
// waiter sees the parity of the last.
template <int STAGES, int ACCS>
bool lapped(unsigned seed) {
    std::mt19937 rng(seed);
    constexpr int kBlocks = 60;
    int full[STAGES] = {}, empty[STAGES] = {}, acc_full[ACCS] = {}, acc_empty[ACCS] = {};
    auto passed = [](int done, uint32_t parity) { return ((unsigned)(done - 1) & 1) == parity; };
    Ring<STAGES> load, issue[2];
    Ring<ACCS> out[2], in;
    issue[1].next();
    out[1].next();
    std::vector<std::pair<int, int>> flying;   // block, stage
    std::deque<std::pair<int, int>> running;   // accumulator, stage
    bool landed[kBlocks] = {}, ready[2] = {};
    int armed = 0, read = 0, at[2] = {0, 1};
    const int slow = (int)(rng() % kBlocks);   // one load that comes late
    while (read < kBlocks) {
        struct Move { int kind, of; };
        std::vector<Move> moves;
        if (armed < kBlocks && passed(empty[load.stage], load.parity ^ 1)) moves.push_back({0, 0});
        for (int i = 0; i < (int)flying.size(); ++i)
            if (flying[i].first != slow || rng() % 50 == 0) moves.push_back({1, i});
        for (int w = 0; w < 2; ++w) {
            if (at[w] < kBlocks && !ready[w] && passed(full[issue[w].stage], issue[w].parity)) moves.push_back({2, w});
            if (at[w] < kBlocks && ready[w] && passed(acc_empty[out[w].stage], out[w].parity ^ 1)) moves.push_back({3, w});
        }
        if (!running.empty()) moves.push_back({4, 0});
        if (passed(acc_full[in.stage], in.parity)) moves.push_back({5, 0});
        if (moves.empty()) {
            if (flying.empty()) return false;   // nothing can move: a lost schedule of an unsound ring
            moves.push_back({1, 0});
        }
        const Move m = moves[rng() % moves.size()];
        if (m.kind == 0) {
            flying.push_back({armed++, load.stage});
            load.next();
        } else if (m.kind == 1) {
            landed[flying[m.of].first] = true;
            ++full[flying[m.of].second];
            flying.erase(flying.begin() + m.of);
        } else if (m.kind == 2) {
            if (!landed[at[m.of]]) return true;
            ready[m.of] = true;
        } else if (m.kind == 3) {
            running.push_back({out[m.of].stage, issue[m.of].stage});
            at[m.of] += 2;
            ready[m.of] = false;
            for (int i = 0; i < 2; ++i) { issue[m.of].next(); out[m.of].next(); }
        } else if (m.kind == 4) {   // products end in the order of their issue
            ++acc_full[running.front().first];
            ++empty[running.front().second];
            running.pop_front();
        } else {
            ++acc_empty[in.stage];
            in.next();
            ++read;
        }
    }
    return false;
}

// Sound as the rule has it: no schedule laps; unsound: one of many does.
template <int STAGES, int ACCS>
bool ring(bool sound) {
    if (no_warp_laps(STAGES, ACCS) != sound) return std::printf("the rule on %d stages, %d accumulators\n", STAGES, ACCS), false;
    for (unsigned seed = 0; seed < (sound ? 400u : 2000u); ++seed)
        if (lapped<STAGES, ACCS>(seed)) return !sound || (std::printf("%d stages, %d accumulators\n", STAGES, ACCS), false);
    return sound || (std::printf("no schedule laps %d stages, %d accumulators\n", STAGES, ACCS), false);
}

template <int STAGES>
bool back_and_forth() {
    Ring<STAGES> r;
    std::vector<std::pair<int, uint32_t>> seen;
    for (int i = 0; i < 4 * STAGES; ++i, r.next()) {
        if (r.stage != i % STAGES || r.parity != (uint32_t)(i / STAGES & 1)) return false;
        seen.push_back({r.stage, r.parity});
    }
    while (!seen.empty()) {
        r.back();
        if (seen.back() != std::make_pair(r.stage, r.parity)) return false;
        seen.pop_back();
    }
    return true;
}

}  // namespace

int main() {
    bool ok = quotients();
    for (int tile : {32, 64, 128, 256, 288})
        for (int ctiles : {1, 3, 8, 55}) ok = tiles(tile, ctiles) && ok;
#define X(stages, accs) ok = ring<stages, accs>(true) && ok;
    CONFIGS X(5, 2) X(9, 4) X(7, 4) X(4, 4) X(6, 4) X(4, 2) X(6, 8)
#undef X
    ok = ring<5, 4>(false) && ring<3, 2>(false) && ring<3, 4>(false) && ring<7, 8>(false) && ok;
    ok = back_and_forth<2>() && back_and_forth<5>() && back_and_forth<10>() && ok;
    return ok ? 0 : 1;
}
