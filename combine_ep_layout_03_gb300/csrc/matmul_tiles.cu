// matmul_tiles.cu -- the 8-bit integer product of expert rows on the tensor cores:
//   c[r, n] = a_scales[r] * w_scales[e, n] * sum_k a[r, k] * w[e, n, k]
//
// sm_103a has no fast integer tensor path, but every int8 code is a float16 number, a
// product of two is exact in float32, and sums stay exact up to 2^24.  So the codes are
// read from memory as the 8 bits they are and become float16 inside the SM, on the way to
// tcgen05.mma kind::f16.
//
// What bounds such a kernel is shared-memory traffic: a code is written by TMA, read, and
// written and read again in 16 bits, against 128 bytes a clock.  Hence
//  - pairs of CTAs (cta_group::2): 256 weight rows x up to 192 token rows a tile, each CTA
//    converting its own 128 weight rows and only half of the token rows;
//  - weights as the M operand, converted into tensor memory: written once, and neither that
//    write nor the MMA's read of it touches shared memory;
//  - tokens as the N operand, whose size an instruction can choose: a segment of few rows
//    pays for few.
// For 64 k a CTA moves 52 KB through shared memory (406 clocks) under 384 clocks of MMA
// with 192 tokens.  Two accumulators of 192 columns and four 64-k stages of weights (32
// columns each) fill the 512 columns of tensor memory, so a tile's epilogue runs under the
// next tile's products.
//
// Warps: 0 TMA, 1 MMA (of the pair's first CTA), 2 tensor memory, 4-7 epilogue, 8-23 four groups
// that turn the codes of weights and tokens into float16 and take the stages in turn (a group's way
// from its wait to its arrival takes several times as long as the MMAs of a stage).  Every wait is
// bounded (EP_ERR_TIMEOUT).
//
// Measured: 8192^3 614 us, 1791 TFLOP/s (0.93 of the measured float16 rate); 32 experts of 1152 rows,
// 4096 x 2048, 366 us, 1690 TFLOP/s, with SwiGLU 385 us (both by the box, 359 to 382 and 374 to 403); a 64-k step takes some 500 clocks where its
// MMAs take 384, with shared memory about 0.9 busy.  Thin segments read weights: 8 rows for each of 512
// experts, 4096 x 1024, 324 us, 6.7 TB/s (0.99 of the copy bandwidth).  One tile of 128 rows takes 15 us
// at k = 4096.
#include "expert_ops.cuh"
#include "tcgen05.cuh"
#include "tensor_maps.cuh"

namespace {

constexpr int kRows = 128;             // weight rows of a CTA
constexpr int kRawK = 128;             // k of a TMA stage (bytes of a row)
constexpr int kRawA = kRows * kRawK;
constexpr uint32_t kColumns = 512;     // of tensor memory
constexpr int kBoxTokens = 32;         // rows of a token box
constexpr int kSets = 4;               // groups of four warps that convert in turn
constexpr int kThreads = 32 * (8 + 4 * kSets);

// TILE: token rows of a tile, both CTAs.  RAW TMA stages of 128 k, CVT float16 stages of HALVES * 64 k.
template <int TILE, int RAW, int CVT, int HALVES>
struct Config {
    static constexpr int tile = TILE, half = TILE / 2;   // half: token rows that one CTA converts
    static constexpr int raw_stages = RAW, cvt_stages = CVT, halves = HALVES;
    static constexpr int raw_bytes = kRawA + half * kRawK;
    static constexpr int half_bytes = half * 128, cvt_bytes = HALVES * half_bytes;   // rows of 64 float16, HALVES times
    static constexpr int cvt_columns = HALVES * 32;
    static constexpr uint32_t col_a = 2 * TILE;          // weights, behind two accumulators
    static constexpr int smem = 1024 + RAW * raw_bytes + CVT * cvt_bytes;
    static_assert(col_a + CVT * cvt_columns <= kColumns, "tensor memory");
    static_assert((CVT & (CVT - 1)) == 0 && CVT % kSets == 0, "uses take stages in turn");
    // A group of warps looks at the mbarrier of every `turn`-th TMA stage only, and a parity tells two
    // neighbouring phases apart, no more: when it asks for use i of a stage, use i - RAW must be over.
    // It has handed over use i - turn, for which the MMAs of use i - turn - (CVT in TMA stages) were
    // done, and with them, in order, everything before.  (With seven stages in the thin form a group
    // could overtake a load that came late, take its stage for the next one, and free it twice.)
    static constexpr int turn = kSets * HALVES / 2;
    static_assert(turn + CVT * HALVES / 2 <= RAW || RAW % turn == 0, "stages that no group can lap");
    static_assert(raw_bytes % 1024 == 0 && half_bytes % 1024 == 0 && half % kBoxTokens == 0, "swizzled rows");
};

// Segments of many rows: the largest tile of which tensor memory holds two.
using Thick = Config<192, 5, 4, 1>;
// Segments of up to 64 rows: the tile's work is the weights', so more TMA stages are in flight.  The
// MMAs of 64 k with few columns are over before the words about them have been exchanged between
// the warps, so a stage is 128 k (tensor memory has the columns that the accumulators leave).
using Thin = Config<64, 8, 4, 2>;

template <class C>
struct Shared {
    Segments seg;
    uint64_t raw_full[C::raw_stages], raw_empty[C::raw_stages];
    uint64_t cvt_full[C::cvt_stages], cvt_empty[C::cvt_stages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drained;
    uint32_t tmem;
};

struct Tile { int64_t row0; int expert, m, n, channel; };   // n: MMA columns, channel: tile of output channels

// Tiles of one expert are neighbours, its token tiles fastest: concurrent pairs share weights and tokens in L2.
// The roles look tiles up between one tile's work and the next, so it has to be quick: a whole warp goes on from
// its last expert, 32 experts at a time, and all counts are 32 bits wide (32 experts of 1152 rows, 1024 x 4096:
// 217 us, with a binary search and 64-bit quotients 233; 512 experts of 8 rows, 4096 x 1024: 319, 331).
// A single thread searches anew.
template <class C, bool WARP>
__device__ __forceinline__ Tile tile_of(const Segments& s, const MatmulArgs& a, int ctiles, int item, int& e) {
    const int at = (int)((uint32_t)item / (uint32_t)ctiles);
    if (WARP) {
        for (int n = 32; n == 32; e += n)
            n = __popc(__ballot_sync(0xffffffffu, s.tile[min(e + 1 + (int)(threadIdx.x & 31), a.E)] <= at));
    } else {
        e = expert_of_tile(s, a.E, at);
    }
    const uint32_t tiles = s.tile[e + 1] - s.tile[e];
    const uint32_t local = item - s.tile[e] * ctiles;
    // the segment's groups of 32 rows dealt out evenly: no tile is much shorter, and none pays for a row more
    const int groups = (s.rows[e] + 31) / 32, j = (int)(local % tiles), each = (int)((uint32_t)groups / tiles);
    const int more = groups - each * (int)tiles;
    const int first = 32 * (j * each + min(j, more));
    Tile t;
    t.expert = e;
    t.row0 = (int64_t)s.base[e] + first;
    t.m = min(32 * (each + (j < more)), s.rows[e] - first);
    t.n = (t.m + 31) / 32 * 32;
    t.channel = (int)(local / tiles);
    return t;
}

// Two of the bytes of w (each a code + 128) as float16: 0x64xx is 1024 + xx.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t bytes_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(__byte_perm(w, 0x64646464u, SEL)), "r"(0x64806480u));
    return r;
}

__device__ __forceinline__ void codes_to_f16(const uint4& v, uint32_t r[8]) {
    const uint32_t w[4] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u, v.w ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = bytes_to_f16x2<0x4140>(w[i]);
        r[2 * i + 1] = bytes_to_f16x2<0x4342>(w[i]);
    }
}

__device__ __forceinline__ uint4 lds_at(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ void sts_at(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
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

// A warp's wait, the same answer in all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_parked(bar, parity));
}

// What every role of a CTA knows.
template <class C>
struct Work {
    const MatmulArgs& a;
    Shared<C>& sh;
    uint8_t* raw;    // TMA stages: 128 weight rows, then token rows, of 128 codes
    uint8_t* cvt;    // float16 token rows of 64 k
    uint32_t tmem, cta;
    int outs, per_pair, ctiles, raws;
    int first, items, step;
};

template <class C, bool GLU>
__device__ __forceinline__ bool load_tiles(const Work<C>& w, const CUtensorMap* map_w, const CUtensorMap* map_a,
                                           const CUtensorMap* map_half) {
    Ring<C::raw_stages> r;
    int used = 0;   // stages armed so far, at most all
    int expert = 0;
    bool ok = true;
    for (int item = w.first; ok && item < w.items; item += w.step) {
        const Tile t = tile_of<C, false>(w.sh.seg, w.a, w.ctiles, item, expert);
        // token rows in one box where the tile is full, else in boxes of 32
        const int half = t.n / 2, boxes = (half + kBoxTokens - 1) / kBoxTokens;
        const int ch = t.channel * w.per_pair + (int)w.cta * (GLU ? kRows / 2 : kRows);
        const int trow = (int)t.row0 + (int)w.cta * half;
        for (int k = 0; k < w.raws; ++k, r.next()) {
            if (!mbar_wait_parked(&w.sh.raw_empty[r.stage], r.parity ^ 1)) { ok = false; break; }
            uint8_t* dst = w.raw + r.stage * C::raw_bytes;
            uint64_t* bar = &w.sh.raw_full[r.stage];
            mbar_arrive_expect_tx(bar, kRawA + boxes * kBoxTokens * kRawK);
            if (GLU) {
                tma_load_4d(dst, map_w, k * kRawK, ch, 0, t.expert, bar);   // 64 gates, then their ups
            } else {
                tma_load_2d(dst, map_w, k * kRawK, t.expert * w.a.N + ch, bar);
            }
            if (boxes == C::half / kBoxTokens) {
                tma_load_2d(dst + kRawA, map_half, k * kRawK, trow, bar);
            } else {
                for (int b = 0; b < boxes; ++b)
                    tma_load_2d(dst + kRawA + b * kBoxTokens * kRawK, map_a, k * kRawK, trow + b * kBoxTokens, bar);
            }
            used = min(used + 1, C::raw_stages);
        }
    }
    // copies in flight end before the CTA does, also when a wait gave up
    for (int i = 0; i < used; ++i) {
        r.back();
        ok = mbar_wait_parked(&w.sh.raw_full[r.stage], r.parity) && ok;
    }
    return ok;
}

// The whole warp walks the loop and one elected lane issues, so that descriptors stay in uniform
// registers.  Whether the next stage is full is asked before the MMAs of this one are issued:
// the answer takes longer than they do.
template <class C>
__device__ __forceinline__ bool issue_mma(const Work<C>& w) {
    Ring<C::cvt_stages> c;
    Ring<2> acc;
    const uint32_t cvt0 = smem_addr(w.cvt);
    bool ready = false, ok = true;
    int expert = 0;
    for (int item = w.first; ok && item < w.items; item += w.step, acc.next()) {
        const Tile t = tile_of<C, true>(w.sh.seg, w.a, w.ctiles, item, expert);
        const uint32_t idesc = mma_desc_f16(2 * kRows, t.n);
        if (!warp_wait(&w.sh.acc_empty[acc.stage], acc.parity ^ 1)) { ok = false; break; }
        tmem_fence_after();
        const uint32_t d = w.tmem + acc.stage * C::tile;
        for (int k = 0; k < 2 / C::halves * w.raws; ++k) {
            if (!ready && !warp_wait(&w.sh.cvt_full[c.stage], c.parity)) { ok = false; break; }
            tmem_fence_after();
            const uint32_t at = w.tmem + C::col_a + c.stage * C::cvt_columns;
            const uint64_t b = smem_desc_k128(cvt0 + c.stage * C::cvt_bytes);
            uint64_t* const empty = &w.sh.cvt_empty[c.stage];
            c.next();
            ready = __all_sync(0xffffffffu, mbar_test(&w.sh.cvt_full[c.stage], c.parity));
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < 4 * C::halves; ++j)
                    mma_pair_f16(d, at + 8 * j, b + (j >> 2) * (C::half_bytes >> 4) + 2 * (j & 3), idesc, k > 0 || j > 0);
                commit_pair(empty);
            }
            __syncwarp();
        }
        if (ok && elect_one()) commit_pair(&w.sh.acc_full[acc.stage]);
        __syncwarp();
    }
    // no MMA is left when the CTAs part, also when a wait gave up
    if (elect_one()) commit_leader(&w.sh.drained);
    __syncwarp();
    return warp_wait(&w.sh.drained, 0) && ok;
}

// Four warps turn a converted stage's codes into float16 at a time; group `set` takes every kSets-th
// use.  With one half, use u of the converted stages is half u & 1 of TMA stage u >> 1; with two, use
// u is TMA stage u.
template <class C, bool GLU>
__device__ __forceinline__ bool convert(const Work<C>& w, int warp, int set) {
    const int lane = threadIdx.x & 31;
    const uint32_t full0 = cluster_addr(smem_addr(&w.sh.cvt_full[0]), 0);
    const int rr = lane & 7, q = lane >> 3, h0 = C::halves == 1 ? set & 1 : 0;
    constexpr int kChunks = C::half / 32;
    static_assert(kSets % 2 == 0, "a group keeps to one half");
    // weights: a thread per row (tensor-memory lane), its four chunks of 16 codes of a half where the swizzle put
    // them; tokens: a lane per chunk, eight rows and four chunks a warp, free of bank conflicts.  The other half
    // of a row lies 64 bytes across (rows are 128-byte aligned).
    // With gates and ups, lanes 0-15 of a warp take 16 gates and lanes 16-31 their ups (rows 64 further on).
    const int weight = GLU ? warp * 16 + (lane & 15) + (lane & 16) * 4 : warp * 32 + lane;
    uint32_t from_w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) from_w[i] = smem_addr(w.raw) + weight * kRawK + (((4 * h0 + i) ^ rr) * 16);
    const uint32_t from_t = smem_addr(w.raw) + kRawA + (warp * 8 + rr) * kRawK + (((4 * h0 + q) ^ rr) * 16);
    const uint32_t row = smem_addr(w.cvt) + (warp * 8 + rr) * 128;
    const uint32_t to0 = row + (((2 * q) ^ rr) * 16), to1 = row + (((2 * q + 1) ^ rr) * 16);
    const uint32_t col = w.tmem + ((uint32_t)(warp * 32) << 16) + C::col_a;
    Ring<C::raw_stages> r;
    uint32_t use = h0;
    int expert = 0;
    bool ok = true;
    for (int item = w.first; ok && item < w.items; item += w.step) {
        const int rows = tile_of<C, true>(w.sh.seg, w.a, w.ctiles, item, expert).n / 2 - warp * 8;
        for (int k = 0; ok && k < w.raws; ++k, use += 2 / C::halves, r.next()) {
            if (use % kSets != (uint32_t)set) continue;
            const uint32_t stage = use % C::cvt_stages, parity = (use / C::cvt_stages) & 1;
            if (!warp_wait(&w.sh.raw_full[r.stage], r.parity)) { ok = false; break; }
            const uint32_t at = r.stage * C::raw_bytes;
#pragma unroll
            for (int h = 0; h < C::halves; ++h) {
                uint32_t v[32];
                uint4 in[kChunks];
#pragma unroll
                for (int i = 0; i < 4; ++i) codes_to_f16(lds_at((from_w[i] + at) ^ (h * 64)), v + 8 * i);
#pragma unroll
                for (int g = 0; g < kChunks; ++g)   // some past the tile's rows
                    in[g] = lds_at((from_t + at + g * 32 * kRawK) ^ (h * 64));
                if (h == 0) {
                    if (!warp_wait(&w.sh.cvt_empty[stage], parity ^ 1)) { ok = false; break; }
                    tmem_fence_after();
                }
                tmem_store32(col + stage * C::cvt_columns + h * 32, v);
                const uint32_t to = stage * C::cvt_bytes + h * C::half_bytes;
#pragma unroll
                for (int g = 0; g < kChunks; ++g) {
                    if (g * 32 >= rows) break;
                    uint32_t f[8];
                    codes_to_f16(in[g], f);
                    sts_at(to0 + to + g * 32 * 128, f[0], f[1], f[2], f[3]);
                    sts_at(to1 + to + g * 32 * 128, f[4], f[5], f[6], f[7]);
                }
            }
            if (!ok) break;
            fence_proxy_async_smem();
            tmem_wait_stores();
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive_cluster(full0 + stage * 8);
                mbar_arrive(&w.sh.raw_empty[r.stage]);
            }
        }
    }
    // the commits that free the last stages reach this CTA before it ends
    use -= h0;
    for (uint32_t i = 0; ok && i < C::cvt_stages && i < use; ++i)
        ok = warp_wait(&w.sh.cvt_empty[(use - 1 - i) % C::cvt_stages], ((use - 1 - i) / C::cvt_stages) & 1);
    return ok;
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

// Lane: an output channel; with gates and ups, lanes 0-15 hold the gates of lanes 16-31's ups.
template <class C, bool GLU>
__device__ __forceinline__ bool epilogue(const Work<C>& w, int warp, float* scales) {
    const int lane = threadIdx.x & 31;
    const uint32_t acc_empty0 = cluster_addr(smem_addr(&w.sh.acc_empty[0]), 0);
    const int64_t outs = w.outs;
    // two channels a store where rows keep them on four bytes
    const bool wide = (outs & 1) == 0 && ((uintptr_t)w.a.out & 3) == 0;
    Ring<2> acc;
    int expert = 0;
    for (int item = w.first; item < w.items; item += w.step, acc.next()) {
        const Tile t = tile_of<C, true>(w.sh.seg, w.a, w.ctiles, item, expert);
        const int ch = t.channel * w.per_pair + (int)w.cta * (GLU ? kRows / 2 : kRows) + warp * (GLU ? 16 : 32) +
                       (GLU ? lane & 15 : lane);
        const bool in = ch < outs;
        const float* sw = w.a.w_scales + (int64_t)t.expert * w.a.N + (in ? ch : 0);
        const float s0 = sw[0], quarter = GLU ? 0.25f * sw[outs] : 0.0f;   // of the ups' scale
        for (int c = lane; c < t.n; c += 32) scales[c] = c < t.m ? w.a.a_scales[t.row0 + c] : 0.0f;
        __syncwarp();
        if (!warp_wait(&w.sh.acc_full[acc.stage], acc.parity)) return false;
        tmem_fence_after();
        const uint32_t d = w.tmem + ((uint32_t)(warp * 32) << 16) + acc.stage * C::tile;
        for (int c0 = 0; c0 < t.m; c0 += 32) {
            uint32_t v[32];
            tmem_load32(d + c0, v);
            const int left = t.m - c0;
            if (GLU) {
                // lanes 0-15 finish the even tokens, lanes 16-31 the odd ones
                const int odd = lane >> 4;
                float y[16];
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float other = __shfl_xor_sync(0xffffffffu, __uint_as_float(odd ? v[i] : v[i + 1]), 16);
                    const float s = scales[c0 + i + odd];
                    y[i / 2] = swiglu((odd ? other : __uint_as_float(v[i])) * s, (odd ? __uint_as_float(v[i + 1]) : other) * s, s0, quarter);
                }
                if (wide) {
                    // neighbours trade as below: an even lane stores its pair of channels of token
                    // i + odd, an odd lane that of token i + 2 + odd
                    const int last = lane & 1;
                    const uint32_t sel = last ? 0x3276u : 0x5410u;
                    uint16_t* out = w.a.out + (t.row0 + c0 + odd + 2 * last) * outs + (ch - last);
#pragma unroll
                    for (int i = 0; i < 32; i += 4, out += 4 * outs) {
                        const uint32_t p = pack_bf16x2_rn(y[i / 2], y[i / 2 + 1]);
                        const uint32_t both = __byte_perm(p, __shfl_xor_sync(0xffffffffu, p, 1), sel);
                        if (in && i + odd + 2 * last < left) *reinterpret_cast<uint32_t*>(out) = both;
                    }
                } else {
                    uint16_t* out = w.a.out + (t.row0 + c0 + odd) * outs + ch;
#pragma unroll
                    for (int i = 0; i < 32; i += 2, out += 2 * outs)
                        if (in && i + odd < left) *out = (uint16_t)pack_bf16x2_rn(y[i / 2], 0.0f);
                }
            } else if (wide) {
                // neighbours trade halves: an even lane stores both channels of the even token
                const int odd = lane & 1;
                const uint32_t sel = odd ? 0x3276u : 0x5410u;
                uint16_t* out = w.a.out + (t.row0 + c0 + odd) * outs + (ch - odd);
#pragma unroll
                for (int i = 0; i < 32; i += 2, out += 2 * outs) {
                    const float2 s = *reinterpret_cast<const float2*>(&scales[c0 + i]);
                    const uint32_t y = pack_bf16x2_rn(__uint_as_float(v[i]) * s.x * s0, __uint_as_float(v[i + 1]) * s.y * s0);
                    const uint32_t both = __byte_perm(y, __shfl_xor_sync(0xffffffffu, y, 1), sel);
                    if (in && i + odd < left) *reinterpret_cast<uint32_t*>(out) = both;
                }
            } else {
                uint16_t* out = w.a.out + (t.row0 + c0) * outs + ch;
#pragma unroll
                for (int i = 0; i < 32; ++i, out += outs) {
                    const float y = __uint_as_float(v[i]) * scales[c0 + i] * s0;
                    if (in && i < left) *out = (uint16_t)pack_bf16x2_rn(y, 0.0f);
                }
            }
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty0 + acc.stage * 8);
    }
    return true;
}

template <class C, bool GLU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
matmul_tiles_kernel(const MatmulArgs a, const __grid_constant__ CUtensorMap map_w,
                    const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_half) {
    extern __shared__ uint8_t dynamic[];
    __shared__ Shared<C> sh;
    __shared__ __align__(16) float scales[4][C::tile];   // of the epilogue warps
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        prefetch_map(&map_w);
        prefetch_map(&map_a);
        prefetch_map(&map_half);
    }
    const uint32_t cta = cluster_rank();
    uint8_t* raw = dynamic + ((1024 - (smem_addr(dynamic) & 1023)) & 1023);
    if (tid == 0) {
        for (int i = 0; i < C::raw_stages; ++i) { mbar_init(&sh.raw_full[i], 1); mbar_init(&sh.raw_empty[i], 8 / C::halves); }
        for (int i = 0; i < C::cvt_stages; ++i) { mbar_init(&sh.cvt_full[i], 8); mbar_init(&sh.cvt_empty[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&sh.acc_full[i], 1); mbar_init(&sh.acc_empty[i], 8); }
        mbar_init(&sh.drained, 1);
        mbar_fence_init();
    }
    if (warp == 2) tmem_alloc_pair(&sh.tmem, kColumns);
    wait_for_previous();
    const bool fits = load_segments<kThreads>(sh.seg, a, C::tile);   // the same answer in both CTAs
    tmem_fence_before();
    __syncthreads();
    cluster_sync();
    tmem_fence_after();

    const int outs = GLU ? a.N / 2 : a.N;
    const int per_pair = GLU ? kRows : 2 * kRows;   // output channels of a tile
    const int ctiles = (outs + per_pair - 1) / per_pair;
    // (overlapping segments can name more tiles than there is output; items + step stays a number)
    const int64_t all = fits ? (int64_t)sh.seg.tile[a.E] * ctiles : 0, limit = INT32_MAX - (int64_t)gridDim.x;
    const Work<C> w = {a, sh, raw, raw + C::raw_stages * C::raw_bytes, sh.tmem, cta, outs, per_pair, ctiles,
                    (a.K + kRawK - 1) / kRawK, (int)(blockIdx.x >> 1), (int)(all < limit ? all : limit), (int)(gridDim.x >> 1)};
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) ok = load_tiles<C, GLU>(w, &map_w, &map_a, &map_half);
    } else if (warp == 1) {
        if (cta == 0) ok = issue_mma(w);
    } else if (warp >= 8) {
        ok = convert<C, GLU>(w, warp & 3, (warp >> 2) - 2);
    } else if (warp >= 4) {
        ok = epilogue<C, GLU>(w, warp & 3, scales[warp & 3]);
    }
    if (!ok && a.status) ep_set_status(a.status, EP_ERR_TIMEOUT);
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    cluster_sync();   // neither CTA's shared or tensor memory goes while the pair's MMAs may read it
    if (warp == 2) tmem_free_pair(w.tmem, kColumns);
}

template <class C>
cudaError_t launch(const MatmulArgs& a, int sms, cudaStream_t st) {
    const int64_t per_pair = a.swiglu ? kRows : 2 * kRows, outs = a.swiglu ? a.N / 2 : a.N;
    CUtensorMap map_w, map_a, map_half;
    if (!(a.swiglu ? make_pairs_map(&map_w, a.w, a.E, outs, a.K, kRows / 2)
                   : make_rows_map(&map_w, a.w, (int64_t)a.E * a.N, a.K, kRows)) ||
        !make_rows_map(&map_a, a.a, a.rows, a.K, kBoxTokens) ||
        !make_rows_map(&map_half, a.a, a.rows, a.K, C::half))
        return cudaErrorInvalidValue;
    const int64_t most = ((a.rows + C::tile - 1) / C::tile + (a.E > 1 ? a.E : 0)) * ((outs + per_pair - 1) / per_pair);
    if (most > INT32_MAX - sms) return cudaErrorInvalidValue;   // more output than any memory holds
    const int64_t pairs = most < sms / 2 ? most : sms / 2;
    auto kernel = a.swiglu ? matmul_tiles_kernel<C, true> : matmul_tiles_kernel<C, false>;
    static std::atomic<uint64_t> done[2];
    const cudaError_t e = allow_smem(kernel, C::smem, done[a.swiglu]);
    if (e != cudaSuccess) return e;
    return launch_overlapped(kernel, dim3((unsigned)(2 * pairs)), kThreads, C::smem, st, a, map_w, map_a, map_half);
}

// Segments of up to this many rows take the thin form, and so do larger ones if its rounds of tiles, which
// take three quarters as long, are that few (half-empty rounds cost whole ones).  Measured, us (thin,
// thick): 128 rows x 4096 x 4096: 15.8, 22.1; 500 x 4096 x 1000: 15.7, 22.3; 2000 x 2048 x 1000: 16.9,
// 14.9; 4000 x 2048 x 2000: 44.7, 34.1; 64 experts of 96 rows, 2048 x 1024: 49.0, 43.5; 128 experts of
// 64 rows, 4096 x 2048: 183, 258; 16 experts of 166 rows, 1024 x 1400: 22.5, 18.6.
constexpr int kThinRows = 64;

}  // namespace

cudaError_t launch_matmul_tiles(const MatmulArgs& a, int sms, cudaStream_t st) {
    const int64_t rows = (a.rows + a.E - 1) / a.E, per_pair = a.swiglu ? kRows : 2 * kRows;
    const int64_t columns = ((a.swiglu ? a.N / 2 : a.N) + per_pair - 1) / per_pair * a.E, pairs = sms / 2;
    const int64_t thin = ((rows + Thin::tile - 1) / Thin::tile * columns + pairs - 1) / pairs;
    const int64_t thick = ((rows + Thick::tile - 1) / Thick::tile * columns + pairs - 1) / pairs;
    return rows <= kThinRows || 4 * thin <= 3 * thick + 1 ? launch<Thin>(a, sms, st) : launch<Thick>(a, sms, st);
}
