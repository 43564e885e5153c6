// matmul_fp8.cu -- the FP8 product of expert rows with a scale for each block of 128, on the tensor cores:
//   c[r, n] = sum over blocks b of 128 k:  a_scales[r, b] w_scales[e, n / 128, b] * sum_{k in b} a[r, k] w[e, n, k]
//
// The scales are float32 and change with every block of k, so no instruction can apply them: the sum of a block is
// taken by tcgen05.mma kind::f8f6f4 into a fresh accumulator in tensor memory, and warps read it, multiply it by the
// two scales and add it to sums in registers, while the next block's products go into another accumulator.
// Tokens are the M operand: a thread has a token (a lane of tensor memory), so that a block costs it one product of
// scales for each 128 channels and one FMA for each value.
//
// Tiles: 256 rows by 256 channels a pair of CTAs (cta_group::2, 512 clocks of products a block, of which the FMAs take
// half), for segments of many rows; 128 rows by 128 channels, or fewer of either, a CTA otherwise.  With SwiGLU half of the
// channels are gates and half their ups, and a thread has both.  A finished row leaves through a row of shared memory of its
// own, from which a warp stores whole 16 bytes (by a bulk copy of each row, 64 experts of 512 rows, 256 x 1024, took 40.5 us
// in a graph where they now take 29.2, and a single tile 4.9 where it takes 3.9).
//
// Warps: four of the epilogue for 64 channels (128 rows), then one for TMA, two that issue MMAs, every other block each,
// and one that brings the products of scales to shared memory (read where they are used, four bytes of 32 rows at a
// time, they cost more than the FMAs).  Every wait is bounded (EP_ERR_TIMEOUT).
//
// Measured: 8192^3 440 us, 2500 TFLOP/s (without scales a library product takes 283); 128 experts of 1024 rows, 4096 x 2
// x 1024 with SwiGLU 1100 to 1150 us (at 1970 MHz and the power limit, as the library's product is at 1460 MHz); thin segments read
// weights: 8 rows for each of 512 experts, 4096 x 1024, 316 us, 6.8 TB/s.  What bounds the large tile is a warp's way through a
// block, some 1020 clocks: wait, four reads of tensor memory with their FMAs, the word that the accumulator is free.  With
// everything else as it was then, 8192^3 took 320 us without the epilogue's waits, reads and FMAs, as much with the reads alone,
// 392 with the FMAs alone, and 496 with both (then 517 in all).
// The tile of 128 by 128 is bound by its loads, 64 bytes a clock of an SM: half the sums a thread, or twice the accumulators, left it
// as it is (8.9 us for 1000 rows x 2048 x 2048).
#include "expert_ops.cuh"
#include "expert_tiles.cuh"
#include "tcgen05.cuh"
#include "tensor_maps.cuh"

namespace {

struct Fp8Args {
    const float* a_scales;       // [rows][blocks]
    const float* w_scales;       // [E][wblocks][blocks]
    const int32_t* expert_base;  // [E + 1] first row of each expert, or null: all rows belong to one matrix
    int32_t* status;             // or null
    uint16_t* out;               // [rows][outs] bf16
    int64_t rows;
    int32_t E;
    int32_t outs;                // n, or n / 2 with swiglu
    int32_t blocks;              // of 128 k
    int32_t wblocks;             // of 128 rows of a matrix (with swiglu: of the gates, then of the ups)
    Divisor ctiles;              // tiles of output channels
};

constexpr int kBoxTokens = 32;   // rows of a small token box
constexpr int kPart = 32;        // output columns that a thread stages at a time
constexpr int kPitch = kPart * 2 + 16;   // bytes of its row there: 16 more than the row, so that lanes meet different banks

// CTAS: of a tile; ROWS: token rows of a CTA that there is room for; N: channels of a tile; STAGES: of 128 k;
// ACCS: accumulators in tensor memory.
// WIDTH: accumulators of an epilogue thread.
template <int CTAS, int ROWS, int N, int STAGES, int ACCS, int WIDTH>
struct Config {
    static constexpr int ctas = CTAS, rows = ROWS, tile = CTAS * ROWS, n = N, stages = STAGES, accs = ACCS;
    static constexpr int channels = N / CTAS;              // whose weights a CTA loads
    static constexpr int width = WIDTH;
    static constexpr int groups = N / width;               // of four epilogue warps
    static constexpr int load_warp = 4 * groups, mma_warp = load_warp + 1, scale_warp = load_warp + 3;   // two MMA warps
    static constexpr int threads = groups == 1 ? 256 : 32 * (4 * groups + 4);
    static constexpr int bytes_a = ROWS * 128, bytes = bytes_a + channels * 128;
    static constexpr int staged = 128 * groups * kPitch;
    static constexpr int smem = 1024 + STAGES * bytes + staged;
    static constexpr uint32_t columns = ACCS * N;
    static_assert(columns <= 512 && (columns & (columns - 1)) == 0 && columns >= 32, "tensor memory");
    static_assert(bytes_a % 1024 == 0 && bytes % 1024 == 0 && width % 32 == 0 && N % width == 0, "swizzled rows; registers");
    static_assert(no_warp_laps(STAGES, ACCS), "stages that no warp can lap");
    static_assert(ACCS % 2 == 0, "an accumulator is one warp's");
    // an MMA reads 128 token rows, also where a stage has room for fewer: what follows is read for them, inside shared memory
    static_assert(bytes - bytes_a + staged >= (128 - ROWS) * 128, "rows past a stage's");
};

using Thick = Config<2, 128, 256, 5, 2, 64>;
using Mid = Config<1, 128, 128, 5, 2, 64>;
using Small = Config<1, 128, 32, 8, 8, 32>;
using Thin = Config<1, 32, 128, 9, 4, 64>;

// The products of scales of a chunk of blocks, by token row of a CTA: of the tile's first block of channels, and of its
// second (or of the ups).
constexpr int kChunk = 8, kChunks = 2;
struct Scales { float of[2][kChunk][128]; };

template <class C>
struct Shared {
    Segments seg;
    Scales scales[kChunks];
    uint64_t scale_full[kChunks], scale_empty[kChunks];
    uint64_t full[C::stages], empty[C::stages];   // full: of the tile's first CTA
    uint64_t acc_full[C::accs], acc_empty[C::accs];
    uint64_t drained;
    uint32_t tmem;
};

template <class C>
struct Work {
    const Fp8Args& a;
    Shared<C>& sh;
    uint8_t* smem;      // stages: token rows, then weight rows
    uint8_t* staged;    // a row of kPitch bytes for each epilogue thread
    uint32_t tmem, cta;
    int per_tile;       // output channels
    int first, items, step;
};

template <class C>
__device__ __forceinline__ void load_rows(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint64_t* own) {
    if constexpr (C::ctas == 2) tma_pair_2d(dst, map, x, y, bar);
    else tma_load_2d(dst, map, x, y, own);
}

template <class C>
__device__ __forceinline__ void load_weights(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar, uint64_t* own) {
    if constexpr (C::ctas == 2) tma_pair_3d(dst, map, x, y, z, bar);
    else tma_load_3d(dst, map, x, y, z, own);
}

// map_w: matrices of weights (with SwiGLU the gates and the ups are one each); map_a, map_all: token rows in boxes of 32,
// or of all that a stage has room for.
template <class C, bool GLU>
__device__ __forceinline__ bool load_tiles(const Work<C>& w, const CUtensorMap* map_w, const CUtensorMap* map_a, const CUtensorMap* map_all) {
    Ring<C::stages> r;
    const uint32_t full0 = cluster_addr(smem_addr(&w.sh.full[0]), 0);
    int used = 0, expert = 0;   // used: stages filled so far, at most all
    bool ok = true;
    for (int item = w.first; ok && item < w.items; item += w.step) {
        const Tile t = tile_of<false>(w.sh.seg, w.a.E, w.a.ctiles, item, expert);
        // rows in one box where the tile is nearly full (each box takes its time to issue, and rows that are not the
        // tile's do no harm), else in boxes of 32
        const int mine = t.n / C::ctas, filled = (mine + kBoxTokens - 1) / kBoxTokens;
        const int boxes = 2 * filled > C::rows / kBoxTokens ? C::rows / kBoxTokens : filled;
        const int bytes = C::channels * 128 + boxes * kBoxTokens * 128;
        const int ch = t.channel * w.per_tile, row = (int)t.row0 + (int)w.cta * mine;
        for (int k = 0; k < w.a.blocks; ++k, r.next()) {
            if (!mbar_wait_parked(&w.sh.empty[r.stage], r.parity ^ 1)) { ok = false; break; }
            uint8_t* dst = w.smem + r.stage * C::bytes;
            uint64_t* own = &w.sh.full[r.stage];
            const uint32_t bar = full0 + r.stage * 8;
            if (w.cta == 0) mbar_arrive_expect_tx(own, C::ctas * bytes);
            if constexpr (!GLU) {
                load_weights<C>(dst + C::bytes_a, map_w, k * 128, ch + (int)w.cta * C::channels, t.expert, bar, own);
            } else if constexpr (C::ctas == 2) {
                load_weights<C>(dst + C::bytes_a, map_w, k * 128, ch, 2 * t.expert + (int)w.cta, bar, own);
            } else {
                load_weights<C>(dst + C::bytes_a, map_w, k * 128, ch, 2 * t.expert, bar, own);
                load_weights<C>(dst + C::bytes_a + C::channels * 64, map_w, k * 128, ch, 2 * t.expert + 1, bar, own);
            }
            if (boxes == C::rows / kBoxTokens) {
                load_rows<C>(dst, map_all, k * 128, row, bar, own);
            } else {
                for (int b = 0; b < boxes; ++b) load_rows<C>(dst + b * kBoxTokens * 128, map_a, k * 128, row + b * kBoxTokens, bar, own);
            }
            used = min(used + 1, C::stages);
        }
    }
    // every load has arrived and been used when its stage is free again: none is in flight when the CTA ends (also
    // when a wait gave up, here or elsewhere: a wait of seconds has passed since the last load then)
    bool over = true;
    for (int i = 0; over && i < used; ++i) {
        r.back();
        over = mbar_wait_parked(&w.sh.empty[r.stage], r.parity);
    }
    return ok && over;
}

// The waits and words of the loop over blocks, which is one chain of latencies: without branches on the lane (50 to 100
// clocks each).  Polls and limit are mbar_wait_parked()'s: every 64 polls the clock is read.  The answer is the warp's: lanes
// need not leave the loop together, and what follows (loads of tensor memory, elections) asks for a converged warp.
__device__ __forceinline__ bool wait_block(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t.reg .u32 n, r;\n\t.reg .u64 start, now;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "@p bra OVER%=;\n\t"
                 "mov.u32 n, 0;\n\tmov.u64 start, 0;\n"
                 "POLL%=:\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "@p bra OVER%=;\n\t"
                 "add.u32 n, n, 1;\n\tand.b32 r, n, 63;\n\tsetp.ne.u32 p, r, 0;\n\t@p bra POLL%=;\n\t"
                 "mov.u64 now, %%globaltimer;\n\tsetp.eq.u32 p, n, 64;\n\t@p mov.u64 start, now;\n\t"
                 "sub.u64 now, now, start;\n\tsetp.le.u64 p, now, %4;\n\t@p bra POLL%=;\n\t"
                 "setp.ne.u32 p, 0, 0;\n"
                 "OVER%=:\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity), "r"(kParkNs), "l"(kWaitNs) : "memory");
    return __all_sync(0xffffffffu, ok != 0);
}

// One lane of a converged warp arrives on this CTA's barrier, or on either CTA's.
__device__ __forceinline__ void arrive_one(int lane, uint32_t bar) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}"
                 :: "r"(bar), "r"(lane) : "memory");
}

__device__ __forceinline__ void arrive_one_cluster(int lane, uint32_t bar) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}"
                 :: "r"(bar), "r"(lane) : "memory");
}

__device__ __forceinline__ float lds_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Two warps issue, every other block each: a block's products start a fresh accumulator, so that their order does not
// matter, and the words to be exchanged for a block (some 350 clocks) are exchanged while the other's products run.
template <class C>
__device__ __forceinline__ bool issue_mma(const Work<C>& w, int which) {
    Ring<C::stages> r;
    Ring<C::accs> acc;
    const uint32_t smem0 = smem_addr(w.smem), idesc = mma_desc_e4m3(128 * C::ctas, C::n);
    if (which) {
        r.next();
        acc.next();
    }
    const int tiles = w.items > w.first ? (w.items - w.first + w.step - 1) / w.step : 0;
    const int64_t blocks = (int64_t)tiles * w.a.blocks;
    bool ok = true;
    for (int64_t k = which; k < blocks; k += 2) {
        const uint32_t at = smem0 + r.stage * C::bytes, d = w.tmem + acc.stage * C::n;
        const uint64_t a = smem_desc_k128(at), b = smem_desc_k128(at + C::bytes_a);
        if (!wait_block(smem_addr(&w.sh.full[r.stage]), r.parity) || !wait_block(smem_addr(&w.sh.acc_empty[acc.stage]), acc.parity ^ 1)) {
            ok = false;
            break;
        }
        tmem_fence_after();
        __syncwarp();
        if (elect_one()) {
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_f8_ss<C::ctas>(d, a + 2 * j, b + 2 * j, idesc, j > 0);
            commit_all<C::ctas>(&w.sh.acc_full[acc.stage]);
            commit_all<C::ctas>(&w.sh.empty[r.stage]);
        }
        __syncwarp();
        r.next();
        r.next();
        acc.next();
        acc.next();
    }
    // no MMA is left when the CTAs part, also when a wait gave up
    if (elect_one()) commit_own<C::ctas>(&w.sh.drained);
    __syncwarp();
    return warp_wait(&w.sh.drained, 0) && ok;
}

// COLS columns of a warp's rows, in bf16 pairs, to out + row * outs + col.  They pass through rows of shared memory of the warp's own,
// so that its lanes store whole 16 bytes, the rows' pieces side by side; where rows are not whole 16 bytes, it writes its rows one by one.
// row: of lane 0; rows: of the warp's 32 that are there.
template <int COLS>
__device__ __forceinline__ void store_part(const uint32_t y[COLS / 2], uint8_t* mine, uint16_t* row, int64_t outs, int cols, int rows, bool whole) {
    const int lane = threadIdx.x & 31;
    __syncwarp();   // the part before has been read
#pragma unroll
    for (int i = 0; i < COLS / 8; ++i) sts_v4(smem_addr(mine) + 16 * i, y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
    __syncwarp();
    const uint32_t warp_rows = smem_addr(mine) - lane * kPitch;
    if (whole) {
        constexpr int kLanes = COLS / 8, kRows = 32 / kLanes;   // of a row's piece; rows at a time
        const int r = lane / kLanes, c = 8 * (lane % kLanes);
        uint16_t* to = row + r * outs + c;
#pragma unroll
        for (int i = 0; i < 32; i += kRows, to += kRows * outs) {
            const uint4 v = lds_v4(warp_rows + (r + i) * kPitch + 2 * c);
            if (r + i < rows && c < cols) *reinterpret_cast<uint4*>(to) = v;
        }
        return;
    }
    for (int r = 0; r < min(rows, 32); ++r, row += outs) {
        for (int c = lane; c < min(cols, COLS); c += 32) {
            uint16_t v;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(warp_rows + r * kPitch + 2 * c) : "memory");
            row[c] = v;
        }
    }
}

// Scales go through shared memory, by a warp of their own: read by the threads that use them, 4 bytes of 32 rows at a
// time, they cost more than the additions.
template <class C, bool GLU>
__device__ __forceinline__ bool load_scales(const Work<C>& w) {
    const int lane = threadIdx.x & 31, blocks = w.a.blocks;
    Ring<kChunks> r;
    int expert = 0;
    for (int item = w.first; item < w.items; item += w.step) {
        const Tile t = tile_of<true>(w.sh.seg, w.a.E, w.a.ctiles, item, expert);
        const int mine = t.n / C::ctas, rows = (min(mine, t.m - (int)w.cta * mine) + 31) / 32;   // in 32s (perhaps none)
        const float* row[C::rows / 32];
#pragma unroll
        for (int i = 0; i < C::rows / 32; ++i)
            row[i] = w.a.a_scales + (t.row0 + min((int)w.cta * mine + 32 * i + lane, t.m - 1)) * blocks;
        // lanes 0 to 15: the eight blocks of k of the first block of channels, and of the second (or of the ups)
        const int half = (lane >> 3) & 1, ch = t.channel * w.per_tile;
        const int wb = GLU ? (ch >> 7) + half * (w.a.wblocks / 2) : min((ch >> 7) + half, w.a.wblocks - 1);
        const float* sw = w.a.w_scales + ((int64_t)t.expert * w.a.wblocks + wb) * blocks;
        for (int k = 0; k < blocks; k += kChunk, r.next()) {
            float v[C::rows / 32][kChunk];
#pragma unroll
            for (int i = 0; i < C::rows / 32; ++i)
#pragma unroll
                for (int b = 0; b < kChunk; ++b) v[i][b] = i < rows && k + b < blocks ? row[i][k + b] : 0.0f;
            const float c = sw[min(k + (lane & 7), blocks - 1)];
            if (!warp_wait(&w.sh.scale_empty[r.stage], r.parity ^ 1)) return false;
            Scales& s = w.sh.scales[r.stage];
#pragma unroll
            for (int h = 0; h < (GLU || C::n > 128 ? 2 : 1); ++h)
#pragma unroll
                for (int b = 0; b < kChunk; ++b) {
                    const float of = __shfl_sync(0xffffffffu, c, 8 * h + b);
#pragma unroll
                    for (int i = 0; i < C::rows / 32; ++i) s.of[h][b][32 * i + lane] = v[i][b] * of;
                }
            __syncwarp();
            if (lane == 0) mbar_arrive(&w.sh.scale_full[r.stage]);
        }
    }
    return true;
}

// sum += s * v.  Volatile, so that it stays behind the wait for the load of v.
__device__ __forceinline__ void add_scaled(float& sum, uint32_t v, float s) {
    asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(sum) : "f"(__uint_as_float(v)), "f"(s));
}

template <class C, bool GLU>
__device__ __forceinline__ bool epilogue(const Work<C>& w, int warp) {
    constexpr int kWidth = C::width, kHalf = kWidth / 2;
    const int lane = threadIdx.x & 31, quarter = warp & 3, group = warp >> 2, mine_row = quarter * 32 + lane;
    const uint32_t acc_empty0 = cluster_addr(smem_addr(&w.sh.acc_empty[0]), 0);
    uint8_t* const mine = w.staged + (group * 128 + mine_row) * kPitch;
    const int outs = w.a.outs, blocks = w.a.blocks;
    const bool whole = outs % 8 == 0 && ((uintptr_t)w.a.out & 15) == 0;
    constexpr uint32_t kUps = sizeof(w.sh.scales[0].of[0]);   // from a gates' product of scales to the ups'
    const uint32_t acc_full = smem_addr(&w.sh.acc_full[0]);
    const uint32_t columns = w.tmem + ((uint32_t)(quarter * 32) << 16) + group * (GLU ? kHalf : kWidth);
    // (all lanes' loads of an accumulator are over: the wait for them is the warp's)
    auto release = [&](uint32_t at) {
        tmem_fence_before();
        if (C::ctas == 1) arrive_one(lane, smem_addr(&w.sh.acc_empty[0]) + 8 * at);
        else arrive_one_cluster(lane, acc_empty0 + 8 * at);
    };
    Ring<kChunks> scales;
    Ring<C::accs> acc;
    int expert = 0;
    bool ok = true;
    for (int item = w.first; ok && item < w.items; item += w.step) {
        const Tile t = tile_of<true>(w.sh.seg, w.a.E, w.a.ctiles, item, expert);
        const int each = t.n / C::ctas;
        const bool some = quarter * 32 < min(each, t.m - (int)w.cta * each);   // of this CTA's rows (perhaps none)
        const int cb = GLU ? 0 : group * kWidth >> 7;   // the thread's channels' block of the tile's (with SwiGLU: the gates' is the first, the ups' the second)
        float sum[kWidth];
#pragma unroll
        for (int i = 0; i < kWidth; ++i) sum[i] = 0.0f;
        for (int k = 0; ok && k < blocks; k += kChunk, scales.next()) {
            if (!wait_block(smem_addr(&w.sh.scale_full[scales.stage]), scales.parity)) { ok = false; break; }
            const int n = min(kChunk, blocks - k);
            uint32_t of = smem_addr(&w.sh.scales[scales.stage].of[cb][0][mine_row]);
            for (const uint32_t end = of + n * 512; of != end; of += 512, acc.next()) {
                const float s = lds_f32(of), u = GLU ? lds_f32(of + kUps) : 0.0f;
                const uint32_t at = acc.stage;
                if (!wait_block(acc_full + 8 * at, acc.parity)) { ok = false; break; }
                tmem_fence_after();
                if (some) {
                    const uint32_t d = columns + at * C::n;
#pragma unroll
                    for (int c = 0; c < kWidth / 16; ++c) {
                        const bool up = GLU && 16 * c >= kHalf;
                        uint32_t v[16];
                        tmem_start16(d + (up ? C::n / 2 - kHalf : 0) + 16 * c, v);
                        tmem_wait_loads();
                        if (c == kWidth / 16 - 1) release(at);
#pragma unroll
                        for (int i = 0; i < 16; ++i) add_scaled(sum[16 * c + i], v[i], up ? u : s);
                    }
                } else {
                    release(at);
                }
            }
            __syncwarp();
            arrive_one(lane, smem_addr(&w.sh.scale_empty[scales.stage]));
        }
        if (!ok || !some) continue;
        // where the tile lies, looked up again: kept over the loop, it would cost the registers that the sums need
        int again = item;
        asm volatile("" : "+r"(again));
        const Tile o = tile_of<true>(w.sh.seg, w.a.E, w.a.ctiles, again, expert);
        const int first = (int)w.cta * (o.n / C::ctas) + quarter * 32, rows = min(o.n / C::ctas - quarter * 32, o.m - first);   // of the warp
        const int ch = o.channel * w.per_tile + group * (GLU ? kHalf : kWidth);   // of the thread
        const int64_t row = o.row0 + first;
        constexpr int kOuts = GLU ? kHalf : kWidth, kCols = kOuts < kPart ? kOuts : kPart;
#pragma unroll
        for (int p = 0; p < kOuts / kCols; ++p) {
            uint32_t y[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) {
                float a = sum[p * kCols + 2 * i], b = sum[p * kCols + 2 * i + 1];
                if constexpr (GLU) {
                    a = swiglu(a, sum[kHalf + p * kCols + 2 * i], 1.0f, 0.25f);
                    b = swiglu(b, sum[kHalf + p * kCols + 2 * i + 1], 1.0f, 0.25f);
                }
                y[i] = pack_bf16x2_rn(a, b);
            }
            store_part<kCols>(y, mine, w.a.out + row * outs + ch + p * kCols, outs, outs - ch - p * kCols, rows, whole);
        }
    }
    return ok;
}

template <class C, bool GLU>
__global__ void __launch_bounds__(C::threads, 1)
matmul_fp8_kernel(const Fp8Args a, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
                  const __grid_constant__ CUtensorMap map_all) {
    extern __shared__ uint8_t dynamic[];
    __shared__ Shared<C> sh;
    static_assert(C::smem + sizeof(sh) <= 227 * 1024, "shared memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        prefetch_map(&map_w);
        prefetch_map(&map_a);
        prefetch_map(&map_all);
    }
    const uint32_t cta = C::ctas == 2 ? cluster_rank() : 0;
    uint8_t* smem = dynamic + ((1024 - (smem_addr(dynamic) & 1023)) & 1023);
    if (tid == 0) {
        for (int i = 0; i < C::stages; ++i) { mbar_init(&sh.full[i], 1); mbar_init(&sh.empty[i], 1); }
        for (int i = 0; i < C::accs; ++i) { mbar_init(&sh.acc_full[i], 1); mbar_init(&sh.acc_empty[i], 4 * C::groups * C::ctas); }
        for (int i = 0; i < kChunks; ++i) { mbar_init(&sh.scale_full[i], 1); mbar_init(&sh.scale_empty[i], 4 * C::groups); }
        mbar_init(&sh.drained, 2);
        mbar_fence_init();
    }
    if (warp == C::mma_warp) tmem_alloc<C::ctas>(&sh.tmem, C::columns);
    wait_for_previous();
    const bool fits = load_segments<C::threads>(sh.seg, a, C::tile);   // the same answer in both CTAs
    tmem_fence_before();
    __syncthreads();
    if constexpr (C::ctas == 2) cluster_sync();
    tmem_fence_after();

    const int per_tile = GLU ? C::n / 2 : C::n;
    const int64_t all = fits ? (int64_t)sh.seg.tile[a.E] * a.ctiles.of : 0, limit = INT32_MAX - (int64_t)gridDim.x;   // (items + step stays a number)
    const Work<C> w = {a, sh, smem, smem + C::stages * C::bytes, sh.tmem, cta, per_tile,
                       (int)(blockIdx.x / C::ctas), (int)(all < limit ? all : limit), (int)(gridDim.x / C::ctas)};
    bool ok = true;
    if (warp < 4 * C::groups) {
        ok = epilogue<C, GLU>(w, warp);
    } else if (warp == C::load_warp) {
        if (lane == 0) ok = load_tiles<C, GLU>(w, &map_w, &map_a, &map_all);
    } else if (warp == C::mma_warp || warp == C::mma_warp + 1) {
        if (cta == 0) ok = issue_mma(w, warp - C::mma_warp);
    } else if (warp == C::scale_warp) {
        ok = load_scales<C, GLU>(w);
    }
    if (!ok && a.status) ep_set_status(a.status, EP_ERR_TIMEOUT);
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    if constexpr (C::ctas == 2) cluster_sync();   // neither CTA's shared or tensor memory goes while the pair's MMAs may read it
    if (warp == C::mma_warp) tmem_free<C::ctas>(w.tmem, C::columns);
}

template <class C, bool GLU>
cudaError_t launch(const Fp8Args& a, const void* rows, const void* weights, int sms, cudaStream_t st) {
    const int64_t per_tile = GLU ? C::n / 2 : C::n, ctiles = (a.outs + per_tile - 1) / per_tile, k = 128 * (int64_t)a.blocks;
    CUtensorMap map_w, map_a, map_all;
    if (!make_experts_map(&map_w, weights, GLU ? 2 * a.E : a.E, a.outs, k, GLU && C::ctas == 1 ? C::channels / 2 : C::channels) ||
        !make_rows_map(&map_a, rows, a.rows, k, kBoxTokens) || !make_rows_map(&map_all, rows, a.rows, k, C::rows))
        return cudaErrorInvalidValue;
    const int64_t most = ((a.rows + C::tile - 1) / C::tile + (a.E > 1 ? a.E : 0)) * ctiles;
    if (most > INT32_MAX - sms) return cudaErrorInvalidValue;   // more output than any memory holds
    const int64_t tiles = most < sms / C::ctas ? most : sms / C::ctas;
    Fp8Args b = a;
    b.ctiles = divisor((uint32_t)ctiles);
    static std::atomic<uint64_t> done;
    const cudaError_t e = allow_smem(matmul_fp8_kernel<C, GLU>, C::smem, done);
    if (e != cudaSuccess) return e;
    return launch_overlapped_clusters(matmul_fp8_kernel<C, GLU>, C::ctas, dim3((unsigned)(C::ctas * tiles)), C::threads, C::smem, st,
                                      b, map_w, map_a, map_all);
}

// The way that is over first by this estimate in us, of rounds of tiles: so much for each block of k and for each tile.  Few
// rows may take matmul_skinny.cu instead, whose items are 16 channels by 32 rows: so much for each round of items and for
// each eight 128-byte pieces of a row.
// Measured, us in a graph (Thick, Mid, Small):
//   one matrix: 100 rows x 4096 x 4096: 21.5, 12.7, 10.3; 500 x 4096 x 1024: 21.2, 12.9, 10.4; 1000 x 2048 x 2048: 14.5, 8.9, 18.9;
//   4000 x 2048 x 2048 with SwiGLU: 24.9, 26.0, 60.1; experts: 8 of 128 rows, 2944 x 330: 18.4, 11.2, 9.1; 16 of 166, 4096 x
//   2048: 42.6, 47.9, 101; of 1024 x 1400 with SwiGLU: 17.4, 14.9, 28.9; 64 of 100, 2048 x 1024: 45.3, 34.0, 57.8; 64 of 512, 256 x
//   1024: 28.4, 29.3, 64.1; 128 of 200, 4096 x 2048 with SwiGLU: 266, 310, 873; 32 of 640, 128 x 592 with SwiGLU: 16.0, 12.8, 23.2.
// Measured, us in a graph (few rows' kernel, Thin): one matrix, 4096 x 4096: 8 rows 6.6, 12.1; 32 rows 11.1, 12.1; 7168 x 4096 with
// SwiGLU: 8 rows 8.8, 19.8; 32 rows 18.3, 19.7; 1024 x 8192: 16 rows 6.8, 5.7; experts of 2048 x 1024: 8 of 16 rows 9.9, 8.4; 8 of
// 32 with SwiGLU 14.9, 9.3; 16 of 8 rows 13.9, 8.6; 32 of 8 rows 24.3, 14.0; 64 of 4 rows, 4096 x 1024: 73.7, 49.5.
template <bool GLU>
struct Plan {
    const Fp8Args& a;
    const int sms;
    int tile = 0, n = 0;
    double us = 1e30;
    template <class C>
    void consider(double block, double of_tile) {
        const int64_t each = (a.rows + a.E - 1) / a.E, experts = a.rows < a.E ? a.rows : a.E, per_tile = GLU ? C::n / 2 : C::n;
        const int64_t tiles = (each + C::tile - 1) / C::tile * experts * ((a.outs + per_tile - 1) / per_tile);
        const double t = 2.8 + (double)((tiles + sms / C::ctas - 1) / (sms / C::ctas)) * (a.blocks * block + of_tile);
        if (t < us) us = t, tile = C::tile, n = C::n;
    }
    bool is_few_rows() const {
        const int64_t each = (a.rows + a.E - 1) / a.E, experts = a.rows < a.E ? a.rows : a.E;
        if (each > 32) return false;
        const double more[4] = {1.0, 1.25, 1.7, 2.1};   // by tiles of eight rows
        const double rounds = (double)(experts * ((a.outs + (GLU ? 7 : 15)) / (GLU ? 8 : 16))) / (2 * sms);
        return 3.0 + (rounds > 0.6 ? rounds : 0.6) * (0.9 + 1.05 * ((a.blocks + 7) / 8) * more[(each - 1) / 8]) <= us;
    }
};

template <bool GLU>
cudaError_t run(const Fp8Args& a, const void* rows, const void* weights, int sms, cudaStream_t st) {
    Plan<GLU> plan{a, sms};
    if ((a.rows + a.E - 1) / a.E <= Thin::tile) plan.template consider<Thin>(0.29, 0.8);
    else plan.template consider<Small>(0.19, 1.1);   // (for so few rows it was never first)
    plan.template consider<Mid>(0.31, 1.5);
    plan.template consider<Thick>(0.52, 2.9);
    if (plan.is_few_rows()) {
        MatmulArgs m{};
        m.a = (const uint8_t*)rows;
        m.a_scales = a.a_scales;
        m.w = (const uint8_t*)weights;
        m.w_scales = a.w_scales;
        m.expert_base = a.expert_base;
        m.out = a.out;
        m.status = a.status;
        m.rows = a.rows;
        m.K = 128 * a.blocks; m.N = GLU ? 2 * a.outs : a.outs; m.E = a.E;
        m.swiglu = GLU;
        return launch_matmul_skinny_fp8(m, sms, st);
    }
    if (plan.tile == Thin::tile) return launch<Thin, GLU>(a, rows, weights, sms, st);
    if (plan.tile == Thick::tile) return launch<Thick, GLU>(a, rows, weights, sms, st);
    return plan.n == Small::n ? launch<Small, GLU>(a, rows, weights, sms, st) : launch<Mid, GLU>(a, rows, weights, sms, st);
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

}  // namespace

extern "C" ep_status ep_expert_matmul_fp8(const void* a, const float* a_scales, int64_t rows, int32_t k, const void* w,
                                          const float* w_scales, int32_t n, int32_t num_experts, const int32_t* expert_base,
                                          int32_t swiglu, void* out, int32_t* status, ep_stream_t stream) {
    if (rows < 0 || rows >= INT32_MAX || k < 128 || k > 65536 || k % 128 != 0 || n < 1 || n > 65536) return EP_ERR_INVALID_ARG;
    if ((swiglu != 0 && swiglu != 1) || (swiglu && n % 2 != 0)) return EP_ERR_INVALID_ARG;
    if (num_experts < 1 || num_experts > kMaxExperts || (num_experts > 1 && !expert_base)) return EP_ERR_INVALID_ARG;
    if (!aligned(expert_base, 4) || !aligned(status, 4)) return EP_ERR_INVALID_ARG;
    if (!w || !aligned(w, 16) || !w_scales || !aligned(w_scales, 4)) return EP_ERR_INVALID_ARG;
    if (rows == 0) return EP_OK;
    if (!a || !aligned(a, 16) || !a_scales || !aligned(a_scales, 4) || !out || !aligned(out, 2)) return EP_ERR_INVALID_ARG;
    Fp8Args f{};
    f.a_scales = a_scales;
    f.w_scales = w_scales;
    f.expert_base = expert_base;
    f.status = status;
    f.out = (uint16_t*)out;
    f.rows = rows;
    f.E = num_experts;
    f.outs = swiglu ? n / 2 : n;
    f.blocks = k / 128;
    f.wblocks = (swiglu ? 2 : 1) * ((f.outs + 127) / 128);
    const int sms = ep_current_sms();
    if (sms <= 0) return EP_ERR_CUDA;
    const cudaError_t e = swiglu ? run<true>(f, a, w, sms, (cudaStream_t)stream) : run<false>(f, a, w, sms, (cudaStream_t)stream);
    return e == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}
