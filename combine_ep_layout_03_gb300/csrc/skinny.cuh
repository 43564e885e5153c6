// skinny.cuh -- the inner loop of matrix products with few token rows, where
// reading the weights once is the work: 16 weight rows against up to 64 tokens a warp.
//
// mma.sync m16n8k16 takes the weights as its 16-row operand and the tokens as its 8
// columns.  A dot product does not care in which order its terms are taken, so the
// 16 columns k that one instruction covers need not be neighbours: each lane loads 16
// contiguous bytes of a weight row and the same k of a token row, and feeds them to
// consecutive instructions as they lie, without a shuffle; the four lanes of a row cover 64
// contiguous bytes, two such loads a whole 128-byte line.  The legacy
// tensor path is ample here: at 6.8 TB/s the weights arrive at 22 bytes a clock an SM.
#pragma once

#include <type_traits>

#include "tcgen05.cuh"
#include "ep_internal.cuh"
#include "ring_places.cuh"

namespace {

__device__ __forceinline__ void mma_bf16(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same of e4m3, 32 k.
__device__ __forceinline__ void mma_e4m3(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
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

// A warp's weights arrive through a ring of DEPTH slots of its own in shared memory, each one
// 128-byte piece of 16 weight rows (2 KB), by TMA: one lane issues a slot's box, the warp waits
// on the slot's mbarrier, reads, and the slot is filled again.  No warp waits for another, so the
// ring keeps running through the barriers and sums between one unit of work and the next.
// (cp.async in 16-byte chunks, and loads to registers, reach two thirds of the rate: what arrives
// in 32-byte sectors is written to shared memory or registers a sector at a time, 20 accesses for
// 512 bytes.)  Every wait is bounded; ring_places.cuh says what happens after one that gave up.
template <int DEPTH>
struct WeightRing {
    static constexpr int kSlot = 2048, kWarpBytes = DEPTH * kSlot;
    uint8_t* slots;
    uint64_t* bars;
    uint32_t lane_off;   // of this lane's chunk in a slot (row g, the first half of a piece)
    RingPlaces<DEPTH> places;

    // smem: 1024-byte aligned, kWarpBytes a warp; barriers: DEPTH a warp.
    __device__ __forceinline__ WeightRing(uint8_t* smem, uint64_t* barriers, int warp, int lane)
        : slots(smem + warp * kWarpBytes), bars(barriers + warp * DEPTH) {
        const int g = lane >> 2, q = lane & 3;
        lane_off = (uint32_t)__cvta_generic_to_shared(slots) + g * 128 + ((q ^ g) * 16);   // 128-byte swizzle
        if (lane == 0) {
            for (int i = 0; i < DEPTH; ++i) mbar_init(&bars[i], 1);
            mbar_fence_init();
        }
        __syncwarp();
    }

    // load(slot, barrier) issues the box of `bytes` bytes (one lane).
    template <class Load>
    __device__ __forceinline__ void put(int lane, uint32_t bytes, Load load) {
        places.put([&](int slot) {
            if (lane != 0) return;
            mbar_arrive_expect_tx(&bars[slot], bytes);
            load(slots + slot * kSlot, &bars[slot]);
        });
    }

    // This lane's part of the oldest slot: rows g (lo) and g + 8 (hi) of the two 64-byte halves.
    __device__ __forceinline__ void take(uint4 lo[2], uint4 hi[2]) {
        const uint32_t at = lane_off + kSlot * places.take([&](int slot, uint32_t parity) { return wait(slot, parity); });
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            lo[h] = lds(at ^ (h * 64));
            hi[h] = lds((at ^ (h * 64)) + 1024);
        }
    }

    // False: a wait gave up.
    __device__ __forceinline__ bool ok() const { return places.ok; }

    // The same answer in all lanes.
    __device__ __forceinline__ bool wait(int slot, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(&bars[slot], parity, kMaxPolls));
    }

    static __device__ __forceinline__ uint4 lds(uint32_t addr) {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
        return v;
    }
};

// Part of the token side of one piece for a tile of eight tokens, this lane's values as they lie: with bf16
// weights all of the piece, which is one 128-byte line of a token; with int8 weights half of it, so that
// half of the weights at a time is converted and held (64 tokens over 512 experts, bf16, by halves: 886 us
// for 856; 8 over 256 experts, int8, by whole pieces: 242 us for 233).
template <bool W8, bool T8>
struct TokenPart {
    static constexpr int kOfPiece = W8 ? 2 : 1;   // parts of a piece
    uint4 v[T8 ? 1 : 2];
};

// tok: the token's row (bf16, or int8 with T8); a lane's values past the row's end read as zero (the weights
// there are zeros too, but zero times what lies behind the row may not be).
template <bool W8, bool T8>
__device__ __forceinline__ void load_tokens(TokenPart<W8, T8>& t, const uint8_t* tok, int piece, int part, int lane_off, int k_bytes) {
    constexpr int kWide = W8 && !T8 ? 2 : 1;   // bytes of a token's value to those of a weight
    const int off = piece * 128 + (W8 ? part * 64 : 0) + lane_off;
    const uint8_t* p = tok + (int64_t)off * kWide;
    if ((piece + 1) * 128 <= k_bytes) {
#pragma unroll
        for (int i = 0; i < (T8 ? 1 : 2); ++i) t.v[i] = *reinterpret_cast<const uint4*>(p + i * (W8 ? 16 : 64));
    } else {
#pragma unroll
        for (int i = 0; i < (T8 ? 1 : 2); ++i)
            t.v[i] = off + (W8 ? 0 : i * 64) < k_bytes ? *reinterpret_cast<const uint4*>(p + i * (W8 ? 16 : 64))
                                                       : make_uint4(0, 0, 0, 0);
    }
}

// Calls f with the number of tiles of eight columns as a constant: 1, 2, 4 or 8, at most MAXNT.
template <int MAXNT, class F>
__device__ __forceinline__ int with_tiles(int tiles, F&& f) {
    using std::integral_constant;
    if constexpr (MAXNT >= 2) {
        if (tiles > 1) {
            if constexpr (MAXNT >= 8) {
                if (tiles > 4) return f(integral_constant<int, 8>{});
            }
            if constexpr (MAXNT >= 4) {
                if (tiles > 2) return f(integral_constant<int, 4>{});
            }
            return f(integral_constant<int, 2>{});
        }
    }
    return f(integral_constant<int, 1>{});
}

// Sixteen int8, or eight bf16, as bf16 pairs.
template <bool W8>
__device__ __forceinline__ void unpack_weights(const uint4& v, uint32_t* a) {
    if constexpr (W8) {
        int8x4_to_bf16(v.x, a[0], a[1]); int8x4_to_bf16(v.y, a[2], a[3]);
        int8x4_to_bf16(v.z, a[4], a[5]); int8x4_to_bf16(v.w, a[6], a[7]);
    } else {
        a[0] = v.x; a[1] = v.y; a[2] = v.z; a[3] = v.w;
    }
}

// acc += one piece's products with NT tiles of eight tokens.  part(i) gives the token parts in the order of
// use: with `sides` = NT PLANES, part i / sides of side i % sides, which is plane i % PLANES of its tile.
// PLANES 2 multiplies by a second set of token rows as well (a value's remainder).
template <bool W8, bool T8, int NT, int PLANES, class Part>
__device__ __forceinline__ void mma_piece(float (*acc)[4], const uint4 lo[2], const uint4 hi[2], Part part) {
    constexpr int kParts = TokenPart<W8, T8>::kOfPiece, kSides = NT * PLANES;
#pragma unroll
    for (int h = 0; h < kParts; ++h) {
        // an int8 part's 16 codes, or a bf16 part's two times 8 values, of each row
        uint32_t a0[8], a1[8];
#pragma unroll
        for (int n = 0; n < 3 - kParts; ++n) {
            unpack_weights<W8>(lo[h + n], a0 + 4 * n);
            unpack_weights<W8>(hi[h + n], a1 + 4 * n);
        }
#pragma unroll
        for (int i = 0; i < kSides; ++i) {
            const TokenPart<W8, T8> t = part(h * kSides + i);
            uint32_t b[8];
            if constexpr (T8) {
                unpack_weights<true>(t.v[0], b);
            } else {
                unpack_weights<false>(t.v[0], b);
                unpack_weights<false>(t.v[1], b + 4);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n)
                mma_bf16(acc[i / PLANES], a0[2 * n], a1[2 * n], a0[2 * n + 1], a1[2 * n + 1], b[2 * n], b[2 * n + 1]);
        }
    }
}

// Token parts on their way: the first EARLY of a piece are asked for before its weights are waited for,
// each later one when the one EARLY before it is used.
template <bool W8, bool T8, int PARTS, int EARLY>
struct TokenQueue {
    static constexpr int kEarly = EARLY < PARTS ? EARLY : PARTS;
    TokenPart<W8, T8> t[kEarly];
    // load(part, i)
    template <class Load>
    __device__ __forceinline__ void start(Load load) {
#pragma unroll
        for (int i = 0; i < kEarly; ++i) load(t[i], i);
    }
    template <class Load>
    __device__ __forceinline__ TokenPart<W8, T8> take(int i, Load load) {
        const TokenPart<W8, T8> now = t[i % kEarly];
        if (i + kEarly < PARTS) load(t[i % kEarly], i + kEarly);
        return now;
    }
};

}  // namespace
