// expert_tiles.cuh -- what the tensor-core kernels over expert segments share: where a tile lies, ring
// positions, a warp's wait, and SwiGLU of float32 accumulators.
#pragma once

#include "expert_ops.cuh"
#include "tcgen05.cuh"

namespace {

struct Tile { int64_t row0; int expert, m, n, channel; };   // n: MMA columns, channel: tile of output channels

// A number that many are divided by, with a reciprocal: floor((2^32 - 1) / of).  A quotient by it is at most one too small.
struct Divisor { uint32_t of, reciprocal; };
inline Divisor divisor(uint32_t d) { return {d, 0xffffffffu / d}; }
__device__ __forceinline__ uint32_t operator/(uint32_t n, const Divisor& d) {
    const uint32_t q = __umulhi(n, d.reciprocal);
    return q + (n - q * d.of >= d.of);
}

// n / d, n - d * (n / d) where the quotient is small (below 2^20): by an approximate reciprocal, one off at most.
struct Quotient { uint32_t whole, rest; };
__device__ __forceinline__ Quotient divide(uint32_t n, uint32_t d) {
    uint32_t q = __float2uint_rz(__fdividef((float)n, (float)d));
    int32_t rest = (int32_t)(n - q * d);
    if (rest < 0) q -= 1, rest += d;
    else if (rest >= (int32_t)d) q += 1, rest -= d;
    return {q, (uint32_t)rest};
}

// In which order the tiles of a matrix are taken: token tiles in groups of eight, all channels of a group before the next
// one, its token tiles fastest.  What runs at a time then covers about as many token tiles as channel tiles, and reads
// few of either.  local: of the matrix's tiles (of token tiles and channel tiles), at: local / ctiles.
struct Place { int tile, channel; };
__device__ __forceinline__ Place place_of(uint32_t local, uint32_t at, uint32_t tiles, uint32_t ctiles) {
    constexpr uint32_t kGroup = 8;
    const uint32_t before = at / kGroup * kGroup;
    const Quotient q = divide(local - before * ctiles, min(kGroup, tiles - before));
    return {(int)(before + q.rest), (int)q.whole};
}

// Tiles of one expert are neighbours: concurrent pairs share weights and tokens in L2.
// The roles look tiles up between one tile's work and the next, so it has to be quick: a whole warp goes on from
// its last expert, 32 experts at a time, all counts are 32 bits wide, and nothing is divided by a number whose reciprocal
// could be known (32 experts of 1152 rows, 1024 x 4096: 217 us, with a binary search and 64-bit quotients 233; 512 experts of
// 8 rows, 4096 x 1024: 319, 331).  A single thread searches anew.
template <bool WARP>
__device__ __forceinline__ Tile tile_of(const Segments& s, int E, const Divisor& ctiles, int item, int& e) {
    const int at = (int)((uint32_t)item / ctiles);
    if (WARP) {
        for (int n = 32; n == 32; e += n)
            n = __popc(__ballot_sync(0xffffffffu, s.tile[min(e + 1 + (int)(threadIdx.x & 31), E)] <= at));
    } else {
        e = expert_of_tile(s, E, at);
    }
    const uint32_t first_tile = s.tile[e], tiles = s.tile[e + 1] - first_tile;
    // the segment's groups of 32 rows dealt out evenly: no tile is much shorter, and none pays for a row more
    const Place p = place_of(item - first_tile * ctiles.of, at - first_tile, tiles, ctiles.of);
    const Quotient q = divide((uint32_t)(s.rows[e] + 31) / 32, tiles);
    const int j = p.tile, each = (int)q.whole, more = (int)q.rest;
    const int first = 32 * (j * each + min(j, more));
    Tile t;
    t.expert = e;
    t.row0 = (int64_t)s.base[e] + first;
    t.m = min(32 * (each + (j < more)), s.rows[e] - first);
    t.n = (t.m + 31) / 32 * 32;
    t.channel = p.channel;
    return t;
}

// A ring position: stage and parity of use i.
template <int STAGES>
struct Ring {
    int stage = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++stage == STAGES) { stage = 0; parity ^= 1; }
    }
    __device__ __forceinline__ void back() {
        if (stage-- == 0) { stage = STAGES - 1; parity ^= 1; }
    }
};

__device__ __forceinline__ void sts_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// A warp's wait, the same answer in all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_parked(bar, parity));
}

// silu(gate s0) * (up s1), of quarter = s1 / 4.  Up is multiplied by the sigmoid first: where its exponential passes
// the range the result is 0, however large gate times up would be.  (A gate of -inf gives NaN, the formula's
// -inf / inf.)  The reciprocal of a quarter of 1 + exp is not yet one of the numbers that are taken for 0, so the
// result is the formula's in float32 as far as that goes.  The approximations are within 2^-22, and the exponent's
// rounding within 2^-17 where the sigmoid is smallest; the output's is 2^-8.
__device__ __forceinline__ float swiglu(float gate, float up, float s0, float quarter) {
    float e, r;
    const float g = gate * s0;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmaf_rn(g, -1.4426950408889634f, -2.0f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(0.25f + e));
    return g * (r * (up * quarter));
}

}  // namespace
