// expert_tiles.cuh -- what the tensor-core kernels over expert segments share: looking up a tile (where it lies and ring
// positions: tile_places.cuh), a warp's wait, and SwiGLU of float32 accumulators.
#pragma once

#include "expert_ops.cuh"
#include "tcgen05.cuh"
#include "tile_places.cuh"

namespace {

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
    return tile_in_segment(item, at, ctiles, e, s.tile[e], s.tile[e + 1] - s.tile[e], s.base[e], s.rows[e]);
}

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
