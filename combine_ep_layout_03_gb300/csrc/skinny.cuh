// skinny.cuh -- the inner loop of matrix products with few token rows, where
// reading the weights once is the work: 16 weight rows against up to 64 tokens a
// warp, straight from global memory to the tensor cores.
//
// mma.sync m16n8k16 takes the weights as its 16-row operand and the tokens as its 8
// columns.  A dot product does not care in which order its terms are taken, so the
// 16 columns k that one instruction covers need not be neighbours: each lane loads 16
// contiguous bytes of a weight row and the same k of a token row, and feeds them to
// consecutive instructions as they lie.  No shared memory, no shuffles; the four lanes
// of a row cover 64 contiguous bytes, two such loads a whole 128-byte line.  The legacy
// tensor path is ample here: at 6.8 TB/s the weights arrive at 22 bytes a clock an SM.
#pragma once

#include "ep_internal.cuh"

namespace {

__device__ __forceinline__ void mma_bf16(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two int8 (bytes SEL of w) as bf16x2, exactly: with 0x43 above it a byte's low seven
// bits read as 128 + (q & 127), and its sign bit alone as 128 or 256, the part to take off.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t int8x2_to_bf16x2(uint32_t w) {
    const uint32_t p = __byte_perm(w, 0x43434343u, SEL);
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(p & 0xff7fff7fu), "r"(p & 0xff80ff80u));
    return r;
}

__device__ __forceinline__ void int8x4_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    lo = int8x2_to_bf16x2<0x4140>(w);
    hi = int8x2_to_bf16x2<0x4342>(w);
}

__device__ __forceinline__ uint4 ld_weights(const uint8_t* p) {   // read once: no L1 line is kept
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// One 128-byte piece of two weight rows (this lane's part): rows g and g + 8 of the tile.
struct Piece { uint4 lo[2], hi[2]; };

// k_bytes: bytes of a weight row; a lane's 16 bytes past its end read as zero.
__device__ __forceinline__ void load_piece(Piece& p, const uint8_t* r0, const uint8_t* r1, int piece, int lane_off,
                                           int k_bytes) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int off = piece * 128 + h * 64 + lane_off;
        const bool in = off < k_bytes;
        p.lo[h] = in ? ld_weights(r0 + off) : make_uint4(0, 0, 0, 0);
        p.hi[h] = in ? ld_weights(r1 + off) : make_uint4(0, 0, 0, 0);
    }
}

// acc += the piece's products with NT tiles of eight token rows.  tok[j]: the row of this
// lane's column in tile j (bf16, or int8 with T8); PLANES 2 adds a second row `plane`
// elements further (a value's remainder, see few_tokens.cu).
template <bool W8, bool T8, int NT, int PLANES>
__device__ __forceinline__ void mma_piece(float (*acc)[4], const Piece& p, const uint8_t* const* tok, int64_t plane,
                                          int piece, int lane_off, int k_bytes) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int off = piece * 128 + h * 64 + lane_off;
        const bool in = off < k_bytes;
        uint32_t a0[8], a1[8];   // the lane's weights of rows g and g + 8 as bf16 pairs
        if constexpr (W8) {
            int8x4_to_bf16(p.lo[h].x, a0[0], a0[1]); int8x4_to_bf16(p.lo[h].y, a0[2], a0[3]);
            int8x4_to_bf16(p.lo[h].z, a0[4], a0[5]); int8x4_to_bf16(p.lo[h].w, a0[6], a0[7]);
            int8x4_to_bf16(p.hi[h].x, a1[0], a1[1]); int8x4_to_bf16(p.hi[h].y, a1[2], a1[3]);
            int8x4_to_bf16(p.hi[h].z, a1[4], a1[5]); int8x4_to_bf16(p.hi[h].w, a1[6], a1[7]);
        } else {
            a0[0] = p.lo[h].x; a0[1] = p.lo[h].y; a0[2] = p.lo[h].z; a0[3] = p.lo[h].w;
            a1[0] = p.hi[h].x; a1[1] = p.hi[h].y; a1[2] = p.hi[h].z; a1[3] = p.hi[h].w;
        }
#pragma unroll
        for (int pl = 0; pl < PLANES; ++pl) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                uint32_t b[8];
                const uint4 zero = make_uint4(0, 0, 0, 0);
                if constexpr (T8) {
                    const uint4 v = in ? *reinterpret_cast<const uint4*>(tok[j] + off) : zero;
                    int8x4_to_bf16(v.x, b[0], b[1]); int8x4_to_bf16(v.y, b[2], b[3]);
                    int8x4_to_bf16(v.z, b[4], b[5]); int8x4_to_bf16(v.w, b[6], b[7]);
                } else {
                    const uint8_t* t = tok[j] + pl * plane + (int64_t)off * (W8 ? 2 : 1);
                    const uint4 v = in ? *reinterpret_cast<const uint4*>(t) : zero;
                    b[0] = v.x; b[1] = v.y; b[2] = v.z; b[3] = v.w;
                    if constexpr (W8) {
                        const uint4 w = in ? *reinterpret_cast<const uint4*>(t + 16) : zero;
                        b[4] = w.x; b[5] = w.y; b[6] = w.z; b[7] = w.w;
                    }
                }
#pragma unroll
                for (int i = 0; i < (W8 ? 4 : 2); ++i)
                    mma_bf16(acc[j], a0[2 * i], a1[2 * i], a0[2 * i + 1], a1[2 * i + 1], b[2 * i], b[2 * i + 1]);
            }
        }
    }
}

// Pieces first, first + step, ... below end, the loads of the next DEPTH pieces in flight.
template <bool W8, bool T8, int NT, int PLANES, int DEPTH = 2>
__device__ __forceinline__ void mma_pieces(float (*acc)[4], const uint8_t* r0, const uint8_t* r1,
                                           const uint8_t* const* tok, int64_t plane, int first, int end, int step,
                                           int lane_off, int k_bytes) {
    Piece p[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        load_piece(p[d], r0, r1, first + d * step, lane_off, first + d * step < end ? k_bytes : 0);
    for (int c = first; c < end; c += DEPTH * step) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int now = c + d * step, next = now + DEPTH * step;
            if (now < end) {
                mma_piece<W8, T8, NT, PLANES>(acc, p[d], tok, plane, now, lane_off, k_bytes);
                if (next < end) load_piece(p[d], r0, r1, next, lane_off, k_bytes);
            }
        }
    }
}

}  // namespace
