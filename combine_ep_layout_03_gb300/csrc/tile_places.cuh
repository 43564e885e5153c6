// tile_places.cuh -- where a tile of a grouped product lies, and positions in rings of stages.  Plain C++ as well as device
// code, so that the same arithmetic is tested on the host, with every error that the device's approximate division may have.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define EP_TILES __host__ __device__ __forceinline__
#else
#define EP_TILES inline
#endif

namespace {

struct Tile { int64_t row0; int expert, m, n, channel; };   // n: MMA columns, channel: tile of output channels

EP_TILES uint32_t high_product(uint32_t a, uint32_t b) {
#ifdef __CUDA_ARCH__
    return __umulhi(a, b);
#else
    return (uint32_t)((uint64_t)a * b >> 32);
#endif
}

#ifndef __CUDACC__
inline float quotient_error = 0.0f;   // a host test's, relative
#endif

// The whole part of a / b, which is taken to two units in the last place (0 of a negative one).
EP_TILES uint32_t whole_quotient(float a, float b) {
#ifdef __CUDA_ARCH__
    return __float2uint_rz(__fdividef(a, b));
#else
    float q = a / b;
#ifndef __CUDACC__
    q += q * quotient_error;
#endif
    return q > 0.0f ? (uint32_t)q : 0;
#endif
}

// A number that many are divided by, with a reciprocal: floor((2^32 - 1) / of).  A quotient by it is at most one too small.
struct Divisor { uint32_t of, reciprocal; };
inline Divisor divisor(uint32_t d) { return {d, 0xffffffffu / d}; }
EP_TILES uint32_t operator/(uint32_t n, const Divisor& d) {
    const uint32_t q = high_product(n, d.reciprocal);
    return q + (n - q * d.of >= d.of);
}

// n / d, n - d * (n / d) where the quotient is small (below 2^20): by an approximate reciprocal, one off at most.
struct Quotient { uint32_t whole, rest; };
EP_TILES Quotient divide(uint32_t n, uint32_t d) {
    uint32_t q = whole_quotient((float)n, (float)d);
    int32_t rest = (int32_t)(n - q * d);
    if (rest < 0) q -= 1, rest += d;
    else if (rest >= (int32_t)d) q += 1, rest -= d;
    return {q, (uint32_t)rest};
}

// In which order the tiles of a matrix are taken: token tiles in groups of eight, all channels of a group before the next
// one, its token tiles fastest.  What runs at a time then covers about as many token tiles as channel tiles, and reads
// few of either.  local: of the matrix's tiles (of token tiles and channel tiles), at: local / ctiles.
struct Place { int tile, channel; };
EP_TILES Place place_of(uint32_t local, uint32_t at, uint32_t tiles, uint32_t ctiles) {
    constexpr uint32_t kGroup = 8;
    const uint32_t before = at / kGroup * kGroup, left = tiles - before;
    const Quotient q = divide(local - before * ctiles, kGroup < left ? kGroup : left);
    return {(int)(before + q.rest), (int)q.whole};
}

// Tile `item` of a product, which is one of expert e's: at: item / ctiles, of token tiles; the expert's first one and how
// many it has; its first row and how many.  The segment's groups of 32 rows are dealt out evenly: no tile is much shorter,
// and none pays for a row more.
EP_TILES Tile tile_in_segment(uint32_t item, uint32_t at, const Divisor& ctiles, int e, uint32_t first_tile, uint32_t tiles, int base, int rows) {
    const Place p = place_of(item - first_tile * ctiles.of, at - first_tile, tiles, ctiles.of);
    const Quotient q = divide((uint32_t)(rows + 31) / 32, tiles);
    const int j = p.tile, each = (int)q.whole, more = (int)q.rest;
    const int first = 32 * (j * each + (j < more ? j : more)), most = 32 * (each + (j < more));
    Tile t;
    t.expert = e;
    t.row0 = (int64_t)base + first;
    t.m = most < rows - first ? most : rows - first;
    t.n = (t.m + 31) / 32 * 32;
    t.channel = p.channel;
    return t;
}

// A ring position: stage and parity of use i.
template <int STAGES>
struct Ring {
    int stage = 0;
    uint32_t parity = 0;
    EP_TILES void next() {
        if (++stage == STAGES) { stage = 0; parity ^= 1; }
    }
    EP_TILES void back() {
        if (stage-- == 0) { stage = STAGES - 1; parity ^= 1; }
    }
};

// Whether two warps that issue every other block each can trust a stage's parity.  Each looks at the stages of every other
// block only, and a parity tells two neighbouring phases apart, no more: with an odd number of stages a warp meets a stage at
// every second of its loads.  When it asks for block b there, block b - stages must be over.  It has issued b - 2, for which
// the accumulator of b - 2 - accs was read, and that is done in order.  (With five stages and four accumulators a warp could
// take a load that came late for the next one, and free its stage twice.)
constexpr bool no_warp_laps(int stages, int accs) { return stages % 2 == 0 || stages >= accs + 2; }

}  // namespace
