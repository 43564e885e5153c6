// matmul_bf16.cu -- the bf16 product of expert rows and its gradients on the tensor cores:
//   c[r, n] = sum_k a[r, k] w[e, n, k]        (plain, or with SwiGLU of gates and ups)
//   da[r, k] = sum_n dc[r, n] w[e, n, k],     dw[e, n, k] = sum over expert e's rows of dc[r, n] a[r, k]
//
// One kernel in four forms.  A tile is 256 "channels" (the contiguous index of the output: n, k and k) by up to 256
// "rows" (token rows of one expert, or n for dw), which a pair of CTAs computes (tcgen05.mma, cta_group::2): channels
// are the M operand, 128 a CTA, and rows the N operand, whose size an instruction can choose, so that a segment of few
// rows pays for few.  The operands lie as they do in memory: an operand whose reduced index is contiguous is K-major,
// else MN-major (w for da, both for dw), and no transposed copy is made of anything.
//
// Warps: 0 TMA, 1 MMA (of the pair's first CTA), 2 tensor memory, 3 ends of segments (dw), 4-11 epilogue.  Both CTAs'
// loads report to the first one's barriers.  Two accumulators take turns, so a tile's epilogue runs under the next
// one's products.  Every wait is bounded (EP_ERR_TIMEOUT).
//
// Few tiles with a long sum are shared by two or four pairs of a cluster: each takes a part of the sum, leaves its
// accumulators in shared memory, and finishes every second or fourth 32 rows of the tile with the other parts' read from
// there, in the order of the parts, whoever adds them.
//
// dw reduces over token rows, and a segment ends anywhere: the rows of its last 16 that belong to others (to the next
// expert, or to nobody, with any contents) are set to zero in shared memory, in both operands, between their arrival
// and their product.  That the second CTA has done so the first one learns by a copy of 16 bytes, whose completion is a
// release to the cluster (16 experts of 166 rows, 1024 x 1408 in float32: 21.6 us in a graph at that; by an arrival that
// releases to the cluster, which waits for the epilogue's stores, 32.1; with the rows loaded one by one and nothing cleared
// 25.6).  Its sums are taken 1024 rows at a time: sum_steps().
//
// Measured: 8192^3 578 us, 1902 TFLOP/s (0.99 of the measured rate); 128 experts of 1088 rows, 4096 x 2048: 1520 us one after
// the other (at 1390 MHz and the power limit; 1310 after a rest), dw of the same 1410 to 1630; 6 rows for each of 128 experts,
// 4096 x 2 x 1024: 308 us, 7.0 TB/s.  Large tiles are bound by the tensor cores (0.96 of a CTA's time) and by power; short sums
// by a tile's way out, of which an SM stores some 27 bytes a clock in float32 and 24 in bf16 (whose instructions take as long as its
// stores: without the stores themselves dw of 16 experts of 16 rows took 19 us where it took 22).
#include "expert_ops.cuh"
#include "expert_tiles.cuh"
#include "tcgen05.cuh"
#include "tensor_maps.cuh"

#include <type_traits>

namespace {

enum Form { FORWARD, GLU, ROWS, WEIGHTS };

struct Bf16Args {
    const int32_t* expert_base;  // [E + 1] first row of each expert, or null: all rows belong to one matrix
    int32_t* status;             // or null
    void* out;
    int64_t rows;
    int32_t E;
    int32_t outs;                // channels of an output row
    int32_t reduced;             // length of the sum (FORWARD, GLU: k; ROWS: n)
    int32_t n;                   // WEIGHTS: rows of a matrix
    int32_t wide, accumulate;    // WEIGHTS: float32 output; added to what is there
    int32_t split;               // pairs that share a tile's sum: 1, 2 or 4
    Divisor ctiles, rtiles;      // tiles of channels; WEIGHTS: of a matrix's rows
};

constexpr int kGroups = 2;                // of four epilogue warps, which take every other 32 rows of a tile
constexpr int kThreads = 32 * (4 + 4 * kGroups);
constexpr int kRows = 128;                // channels of a CTA
constexpr int kStep = 64;                 // of the sum a stage: 128 bytes
constexpr int kBytesA = kRows * 128;
constexpr int kBoxTokens = 32;            // rows of a small token box
constexpr int kBlock = 64 * 128;          // MN-major: 64 channels or rows by 64 of the sum
constexpr uint32_t kColumns = 512;        // of tensor memory
constexpr int kMostParts = 4;             // of a tile's sum
constexpr int kSteps = 16;                // WEIGHTS: of a sum that the tensor cores take in one go

// TILE: rows of a tile, both CTAs.
template <int TILE, int STAGES>
struct Config {
    static constexpr int tile = TILE, half = TILE / 2, stages = STAGES;
    static constexpr int bytes = kBytesA + half * 128;
    static constexpr int smem = 1024 + STAGES * bytes;
    static_assert(2 * TILE <= (int)kColumns && bytes % 1024 == 0 && half % kBoxTokens == 0, "layout");
};

using Thick = Config<256, 6>;
using Mid = Config<128, 8>;
using Thin = Config<64, 10>;

template <class C>
struct Shared {
    Segments seg;
    uint64_t full[C::stages], empty[C::stages];   // full: of the pair's first CTA
    uint64_t tail[C::stages];                     // WEIGHTS: this CTA's bytes of a stage that ends a segment
    alignas(16) uint8_t word[16];                 // WEIGHTS: where the second CTA's words arrive that it has cleared rows
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drained;
    uint32_t tmem;
};

// What every role of a CTA knows.
template <class C, Form F>
struct Work {
    const Bf16Args& a;
    Shared<C>& sh;
    uint8_t* smem;      // stages: 128 channels, then rows
    uint32_t tmem, cta;
    uint32_t lead;                  // the pair's first CTA in its cluster
    int part;                       // of a tile's sum
    int per_pair;                   // channels of a tile
    int first, items, step;

    // The first of the steps of a sum that part p takes.
    __device__ __forceinline__ int begin(int steps, int p) const { return steps * p / a.split; }
    // Up to which step those from `first` on go to one accumulator.
    __device__ __forceinline__ int until(int first, int end) const { return F == WEIGHTS ? min(first + kSteps, end) : end; }

    // The tile, and its stages of the sum.
    template <bool WARP>
    __device__ __forceinline__ Tile tile(int item, int& e, int& steps) const {
        if constexpr (F == WEIGHTS) {
            const uint32_t at = (uint32_t)item / a.ctiles, matrix = at / a.rtiles, before = matrix * a.rtiles.of;
            Tile t;
            e = (int)matrix;
            t.expert = e;
            const Place p = place_of((uint32_t)item - before * a.ctiles.of, at - before, a.rtiles.of, a.ctiles.of);
            t.channel = p.channel;
            t.row0 = (int64_t)p.tile * C::tile;
            t.m = min(C::tile, a.n - (int)t.row0);
            t.n = (t.m + 31) / 32 * 32;
            steps = (sh.seg.rows[e] + kStep - 1) / kStep;
            return t;
        } else {
            steps = (a.reduced + kStep - 1) / kStep;
            return tile_of<WARP>(sh.seg, a.E, a.ctiles, item, e);
        }
    }
    // Of the sum in step k, at most 64.
    __device__ __forceinline__ int left(const Tile& t, int k) const {
        return min(kStep, (F == WEIGHTS ? sh.seg.rows[t.expert] : a.reduced) - k * kStep);
    }
    // Whether warp 3 has to clear rows before step k's products.
    __device__ __forceinline__ bool ragged(const Tile& t, int k) const { return F == WEIGHTS && left(t, k) % 16 != 0; }
};

template <class C, Form F>
__device__ __forceinline__ bool load_tiles(const Work<C, F>& w, const CUtensorMap* map_c, const CUtensorMap* map_r, const CUtensorMap* map_half) {
    Ring<C::stages> r;
    const uint32_t full0 = cluster_addr(smem_addr(&w.sh.full[0]), w.lead);
    int used = 0, expert = 0;   // used: stages filled so far, at most all
    bool ok = true;
    for (int item = w.first; ok && item < w.items; item += w.step) {
        int steps;
        const Tile t = w.template tile<false>(item, expert, steps);
        const int half = t.n / 2;
        // rows in one box where the tile is nearly full (each box takes its time to issue, and rows that are not the
        // tile's do no harm), else in boxes of 32
        const int filled = (half + kBoxTokens - 1) / kBoxTokens, all = C::half / kBoxTokens;
        const int boxes = F == WEIGHTS ? (half + 63) / 64 : 2 * filled > all ? all : filled;
        const int bytes = kBytesA + boxes * (F == WEIGHTS ? kBlock : kBoxTokens * 128);
        const int ch = t.channel * w.per_pair + (int)w.cta * (F == GLU ? kRows / 2 : kRows);
        const int row = (int)t.row0 + (int)w.cta * half;
        for (int k = w.begin(steps, w.part), end = w.begin(steps, w.part + 1); k < end; ++k, r.next()) {
            if (!mbar_wait_parked(&w.sh.empty[r.stage], r.parity ^ 1)) { ok = false; break; }
            uint8_t* dst = w.smem + r.stage * C::bytes;
            uint32_t bar = full0 + r.stage * 8;
            if (w.ragged(t, k)) {
                bar = smem_addr(&w.sh.tail[r.stage]);
                mbar_arrive_expect_tx(&w.sh.tail[r.stage], bytes);
                if (w.cta == 0) mbar_arrive_expect_tx(&w.sh.full[r.stage], 16);   // the second CTA's word
            } else if (w.cta == 0) {
                mbar_arrive_expect_tx(&w.sh.full[r.stage], 2 * bytes);
            } else if (F == WEIGHTS) {
                mbar_arrive_cluster(bar);
            }
            if constexpr (F == FORWARD) {
                tma_pair_3d(dst, map_c, k * 128, ch, t.expert, bar);
            } else if constexpr (F == GLU) {
                for (int i = 0; i < 4; ++i)   // 16 gates and their ups: a warp of the epilogue has both
                    tma_pair_4d(dst + i * 4096, map_c, k * 128, ch + 16 * i, 0, t.expert, bar);
            } else if constexpr (F == ROWS) {
                for (int i = 0; i < 2; ++i) tma_pair_3d(dst + i * kBlock, map_c, (ch + 64 * i) * 2, k * kStep, t.expert, bar);
            } else {
                const int sum0 = w.sh.seg.base[t.expert] + k * kStep;
                for (int i = 0; i < 2; ++i) tma_pair_2d(dst + i * kBlock, map_c, (ch + 64 * i) * 2, sum0, bar);
                for (int i = 0; i < boxes; ++i) tma_pair_2d(dst + kBytesA + i * kBlock, map_r, (row + 64 * i) * 2, sum0, bar);
            }
            if constexpr (F != WEIGHTS) {
                if (boxes == all) {
                    tma_pair_2d(dst + kBytesA, map_half, k * 128, row, bar);
                } else {
                    for (int b = 0; b < boxes; ++b)
                        tma_pair_2d(dst + kBytesA + b * kBoxTokens * 128, map_r, k * 128, row + b * kBoxTokens, bar);
                }
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

// Warp 3, WEIGHTS: of a stage whose last 16 rows are not all the segment's, those that are not become zeros.
template <class C, Form F>
__device__ __forceinline__ bool clear_tails(const Work<C, F>& w) {
    Ring<C::stages> r;
    const uint32_t full0 = cluster_addr(smem_addr(&w.sh.full[0]), w.lead);
    const uint32_t word = cluster_addr(smem_addr(w.sh.word), w.lead);
    uint32_t parity = 0;   // of each stage's tail barrier
    const int lane = threadIdx.x & 31;
    int expert = 0;
    for (int item = w.first; item < w.items; item += w.step) {
        int steps;
        const Tile t = w.template tile<true>(item, expert, steps);
        const int begin = w.begin(steps, w.part), end = w.begin(steps, w.part + 1);
        if (begin == end) continue;
        for (int k = begin; k < end - 1; ++k) r.next();
        if (w.ragged(t, end - 1)) {
            if (!warp_wait(&w.sh.tail[r.stage], (parity >> r.stage) & 1)) return false;
            parity ^= 1u << r.stage;
            const int blocks = 2 + (t.n / 2 + 63) / 64, first = w.left(t, end - 1), past = (first + 15) / 16 * 16;
            const uint32_t at = smem_addr(w.smem + r.stage * C::bytes);
            for (int i = lane; i < blocks * (past - first) * 8; i += 32) {
                const int piece = i & 7, row = first + (i >> 3) % (past - first), block = (i >> 3) / (past - first);
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};"
                             :: "r"(at + block * kBlock + row * 128 + piece * 16), "r"(0) : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (w.cta == 0) mbar_arrive(&w.sh.full[r.stage]);
                else copy16_to_cluster(word, at + first * 128, full0 + r.stage * 8);
            }
        }
        r.next();
    }
    return true;
}

// The whole warp walks the loop and one elected lane issues, so that descriptors stay in uniform registers.
// Whether the next stage is full is asked before the MMAs of this one are issued: the answer takes longer than they do.
template <class C, Form F>
__device__ __forceinline__ bool issue_mma(const Work<C, F>& w) {
    constexpr bool a_mn = F == ROWS || F == WEIGHTS, b_mn = F == WEIGHTS;
    Ring<C::stages> r;
    Ring<2> acc;
    const uint32_t smem0 = smem_addr(w.smem);
    bool ready = false, ok = true;
    int expert = 0;
    for (int item = w.first; ok && item < w.items; item += w.step) {
        int steps;
        const Tile t = w.template tile<true>(item, expert, steps);
        const uint32_t idesc = mma_desc_bf16(2 * kRows, t.n, a_mn, b_mn);
        for (int first = w.begin(steps, w.part), end = w.begin(steps, w.part + 1); ok && first < end; first = w.until(first, end)) {
            if (!warp_wait(&w.sh.acc_empty[acc.stage], acc.parity ^ 1)) { ok = false; break; }
            tmem_fence_after();
            const uint32_t d = w.tmem + acc.stage * C::tile;
            for (int k = first; k < w.until(first, end); ++k) {
                if (!ready && !warp_wait(&w.sh.full[r.stage], r.parity)) { ok = false; break; }
                tmem_fence_after();
                const uint32_t at = smem0 + r.stage * C::bytes;
                const uint64_t a = a_mn ? smem_desc_mn128(at, kBlock) : smem_desc_k128(at);
                const uint64_t b = b_mn ? smem_desc_mn128(at + kBytesA, kBlock) : smem_desc_k128(at + kBytesA);
                const int pieces = (w.left(t, k) + 15) / 16;
                uint64_t* const empty = &w.sh.empty[r.stage];
                r.next();
                ready = __all_sync(0xffffffffu, mbar_test(&w.sh.full[r.stage], r.parity));
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < kStep / 16; ++j)   // 16 of the sum: 32 bytes further on, or 16 rows of 128
                        if (j < pieces) mma_pair_f16_ss(d, a + j * (a_mn ? 128 : 2), b + j * (b_mn ? 128 : 2), idesc, k > first || j > 0);
                    commit_pair_of(empty, w.lead);
                }
                __syncwarp();
            }
            if (ok && elect_one()) commit_pair_of(&w.sh.acc_full[acc.stage], w.lead);
            __syncwarp();
            acc.next();
        }
    }
    // no MMA is left when the CTAs part, also when a wait gave up
    if (elect_one()) commit_leader(&w.sh.drained);
    __syncwarp();
    return warp_wait(&w.sh.drained, 0) && ok;
}

// Eight sums += what the accumulators hold.  Volatile, as what reads tmem_start8()'s registers has to be.
__device__ __forceinline__ void add_columns(float* sum, uint32_t addr) {
    uint32_t v[8];
    tmem_start8(addr, v);
    tmem_wait_loads();
#pragma unroll
    for (int i = 0; i < 8; ++i) asm volatile("add.rn.f32 %0, %0, %1;" : "+f"(sum[i]) : "f"(__uint_as_float(v[i])));
}

// WEIGHTS: a sum of more than kSteps steps, [begin, end).  The tensor cores cut what passes float32 wherever they add, always
// towards zero, so they take kSteps at a time, and each thread adds up its columns of these in registers, rounding to nearest; the
// last accumulator then gets the sums, as if it were the only one.  (A gradient of 16384 rows was off by 1.9e-5 of its norm,
// 8.2e-5 where all terms have one sign; it is by 1.0e-6 and 2.2e-6.  Us in a graph, before and now: 2 experts of 16384 rows, 4096 x
// 2048: 375, 375; 32 of 1088 rows, added: 500, 525, and 600 with eight steps at a time, which are half as far off; 4 of 2000 rows, 512 x
// 2048: 17.0, 17.9; 16 of 166 rows, which has no long sums: 23.3, 24.0.)
template <class C, Form F>
__device__ __forceinline__ bool sum_steps(const Work<C, F>& w, const Tile& t, int begin, int end, int warp, int group, Ring<2>& acc) {
    if (w.until(begin, end) == end) return true;
    constexpr int kTurns = C::tile / (32 * kGroups);
    const uint32_t acc_empty0 = cluster_addr(smem_addr(&w.sh.acc_empty[0]), w.lead);
    float sum[kTurns][32];
#pragma unroll
    for (int i = 0; i < kTurns; ++i)
#pragma unroll
        for (int j = 0; j < 32; ++j) sum[i][j] = 0.0f;
    uint32_t d;
#pragma unroll 1
    while (true) {
        if (!warp_wait(&w.sh.acc_full[acc.stage], acc.parity)) return false;
        tmem_fence_after();
        d = w.tmem + ((uint32_t)(warp * 32) << 16) + acc.stage * C::tile + 32 * group;
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            if (32 * (group + kGroups * i) >= t.m) break;
#pragma unroll
            for (int j = 0; j < 32; j += 8) add_columns(sum[i] + j, d + 32 * kGroups * i + j);
        }
        begin = w.until(begin, end);
        if (begin == end) break;
        tmem_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive_cluster(acc_empty0 + acc.stage * 8);
        acc.next();
    }
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        if (32 * (group + kGroups * i) >= t.m) break;
        uint32_t v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(sum[i][j]);
        tmem_store32(d + 32 * kGroups * i, v);
    }
    tmem_wait_stores();
    return true;
}

// A part of a tile's sum: its accumulators go to shared memory, whose stages have been used by then, a column of 128
// channels after the other.
template <class C, Form F>
__device__ __forceinline__ bool leave_part(const Work<C, F>& w, int warp, int group) {
    if (w.first >= w.items) return true;
    int steps, expert = 0;
    const Tile t = w.template tile<true>(w.first, expert, steps);
    const int begin = w.begin(steps, w.part), end = w.begin(steps, w.part + 1);
    if (begin == end) return true;
    Ring<2> acc;
    if (!sum_steps(w, t, begin, end, warp, group, acc)) return false;
    if (!warp_wait(&w.sh.acc_full[acc.stage], acc.parity)) return false;
    tmem_fence_after();
    const uint32_t to = smem_addr(w.smem) + (warp * 32 + (threadIdx.x & 31)) * 4;
    for (int c0 = 32 * group; c0 < t.m; c0 += 32 * kGroups) {
        uint32_t v[32];
        tmem_load32(w.tmem + ((uint32_t)(warp * 32) << 16) + acc.stage * C::tile + c0, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) asm volatile("st.shared.u32 [%0], %1;" :: "r"(to + (c0 + i) * 512), "r"(v[i]) : "memory");
    }
    return true;
}

// The sum of all parts of 32 rows of a channel, at this address of each pair's shared memory.  All parts of 16 rows are asked
// for at once: the way there and back takes most of a microsecond.
template <class C, Form F>
__device__ __forceinline__ void add_parts(const Work<C, F>& w, int steps, uint32_t at, uint32_t v[32]) {
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
        float x[kMostParts][16];
#pragma unroll
        for (int p = 0; p < kMostParts; ++p) {
            const bool left = p < w.a.split && w.begin(steps, p) < w.begin(steps, p + 1);   // (else nothing was)
            const uint32_t there = cluster_addr(at + h * 512, left ? 2 * p + w.cta : 0);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[p][i] = 0.0f;
                if (left) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x[p][i]) : "r"(there + i * 512) : "memory");
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float sum = x[0][i];
#pragma unroll
            for (int p = 1; p < kMostParts; ++p) sum += x[p][i];
            v[h + i] = __float_as_uint(sum);
        }
    }
}

// The address of row i, `pitch` bytes each.  Volatile, so that the 32 offsets are not kept from one tile to the next: with them the
// registers did not do, and 16 experts of 16 rows, dw of 1024 x 1408 in float32, took 28 us in a graph where it takes 18.8.
__device__ __forceinline__ void* row_at(void* base, uint32_t pitch, int i) {
    uint64_t p;
    asm volatile("mad.wide.u32 %0, %1, %2, %3;" : "=l"(p) : "r"(pitch), "r"(i), "l"(base));
    return (void*)p;
}

// 32 rows of a warp's channels, of which this lane's first n are stored (ALL: all 32, in every lane); ch: of this lane.
template <Form F, bool ADD, class ALL>
__device__ __forceinline__ void store_rows(const Bf16Args& a, const uint32_t v[32], int64_t row0, int ch, int n, bool wide, ALL) {
    constexpr bool all = ALL::value;
    const int lane = threadIdx.x & 31;
    if (F == WEIGHTS && a.wide) {
        const uint32_t pitch = 4 * (uint32_t)a.outs;
        void* const to = (float*)a.out + row0 * a.outs + ch;
        if (ADD) {
            float* const out = (float*)to;
            float before[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) before[i] = all || i < n ? out[i * (int64_t)a.outs] : 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (all || i < n) out[i * (int64_t)a.outs] = before[i] + __uint_as_float(v[i]);
        } else {
            // one row's address from the last one's: no offsets are kept
            void* row = to;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                if (all || i < n) *(float*)row = __uint_as_float(v[i]);
                asm volatile("add.s64 %0, %0, %1;" : "+l"(row) : "l"((uint64_t)pitch));
            }
        }
        return;
    }
    const uint32_t pitch = 2 * (uint32_t)a.outs;
    uint16_t* const out = (uint16_t*)a.out + row0 * a.outs + ch;
    if (F == GLU) {
        // lanes 0-15 finish the even rows, lanes 16-31 the odd ones
        const int odd = lane >> 4;
        float y[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const float other = __shfl_xor_sync(0xffffffffu, __uint_as_float(odd ? v[i] : v[i + 1]), 16);
            y[i / 2] = swiglu(odd ? other : __uint_as_float(v[i]), odd ? __uint_as_float(v[i + 1]) : other, 1.0f, 0.25f);
        }
        if (wide) {
            // neighbours trade as below: an even lane stores its pair of channels of row i + odd, an odd lane that of
            // row i + 2 + odd
            const int last = lane & 1, mine = odd + 2 * last;
            const uint32_t sel = last ? 0x3276u : 0x5410u;
            void* const to = out + (int64_t)mine * a.outs - last;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const uint32_t p = pack_bf16x2_rn(y[i / 2], y[i / 2 + 1]);
                const uint32_t both = __byte_perm(p, __shfl_xor_sync(0xffffffffu, p, 1), sel);
                if (all || i + mine < n) *(uint32_t*)row_at(to, pitch, i) = both;
            }
        } else {
            void* const to = out + (int64_t)odd * a.outs;
#pragma unroll
            for (int i = 0; i < 32; i += 2)
                if (all || i + odd < n) *(uint16_t*)row_at(to, pitch, i) = (uint16_t)pack_bf16x2_rn(y[i / 2], 0.0f);
        }
    } else if (wide) {
        // neighbours trade halves: an even lane stores both channels of the even row
        const int odd = lane & 1;
        const uint32_t sel = odd ? 0x3276u : 0x5410u;
        void* const to = out + (int64_t)odd * a.outs - odd;
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const uint32_t y = pack_bf16x2_rn(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
            const uint32_t both = __byte_perm(y, __shfl_xor_sync(0xffffffffu, y, 1), sel);
            if (all || i + odd < n) *(uint32_t*)row_at(to, pitch, i) = both;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (all || i < n) *(uint16_t*)row_at(out, pitch, i) = (uint16_t)pack_bf16x2_rn(__uint_as_float(v[i]), 0.0f);
    }
}

// Lane: a channel; with gates and ups, lanes 0-15 hold the gates of lanes 16-31's ups.
template <class C, Form F, bool ADD>
__device__ __forceinline__ bool epilogue(const Work<C, F>& w, int warp, int group) {
    const int lane = threadIdx.x & 31;
    const uint32_t acc_empty0 = cluster_addr(smem_addr(&w.sh.acc_empty[0]), w.lead);
    const int64_t outs = w.a.outs;
    // two channels a store where rows keep them on four bytes
    const bool wide = (outs & 1) == 0 && ((uintptr_t)w.a.out & 3) == 0;
    Ring<2> acc;
    int expert = 0;
    for (int item = w.first; item < w.items; item += w.step) {
        int steps;
        const Tile t = w.template tile<true>(item, expert, steps);
        if (ADD && steps == 0) continue;
        const int ch = t.channel * w.per_pair + (int)w.cta * (F == GLU ? kRows / 2 : kRows) + warp * (F == GLU ? 16 : 32) +
                       (F == GLU ? lane & 15 : lane);
        const bool in = ch < outs;
        const int64_t row0 = F == WEIGHTS ? (int64_t)t.expert * w.a.n + t.row0 : t.row0;
        const bool some = F != WEIGHTS || steps > 0;   // an expert without rows: zeros
        if (ADD && ch - lane < outs) {
            // what the tile is added to, on its way to L2 under the products, a row a lane: 128 experts of 64 rows, 2048 x 1024:
            // 335 us in a graph, 461 without (its bytes take 324); of 500 rows 420 to 428, 465 (of the next tile instead 397, 546)
            const float* to = (const float*)w.a.out + row0 * outs + ch - lane;
            for (int c0 = 32 * (group + kGroups * w.part) + lane; c0 < t.m; c0 += 32 * kGroups * w.a.split)
                asm volatile("prefetch.global.L2 [%0];" :: "l"(to + c0 * outs));
        }
        if (some && w.a.split == 1) {   // (parts have been waited for)
            if (!sum_steps(w, t, 0, steps, warp, group, acc)) return false;
            if (!warp_wait(&w.sh.acc_full[acc.stage], acc.parity)) return false;
            tmem_fence_after();
        }
        const uint32_t d = w.tmem + ((uint32_t)(warp * 32) << 16) + acc.stage * C::tile;
        for (int c0 = 32 * (group + kGroups * w.part); c0 < t.m; c0 += 32 * kGroups * w.a.split) {
            uint32_t v[32];
            if (some && w.a.split > 1) {
                add_parts(w, steps, smem_addr(w.smem) + (warp * 32 + lane) * 4 + c0 * 512, v);
            } else if (some) {
                tmem_load32(d + c0, v);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0;
            }
            // rows of the 32 that this lane stores, and whether that is all of them for the whole warp
            const int n = in ? t.m - c0 : 0;
            if (__all_sync(0xffffffffu, n >= 32)) store_rows<F, ADD>(w.a, v, row0 + c0, ch, 32, wide, std::true_type());
            else store_rows<F, ADD>(w.a, v, row0 + c0, ch, n, wide, std::false_type());
        }
        if (some && w.a.split == 1) {
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_empty0 + acc.stage * 8);
            acc.next();
        }
    }
    return true;
}

template <class C, Form F, bool ADD>   // ADD: WEIGHTS, to what is there
__global__ void __launch_bounds__(kThreads, 1)
matmul_bf16_kernel(const Bf16Args a, const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_r,
                   const __grid_constant__ CUtensorMap map_half) {
    extern __shared__ uint8_t dynamic[];
    __shared__ Shared<C> sh;
    static_assert(C::smem + sizeof(sh) <= 227 * 1024, "shared memory");
    static_assert(F != WEIGHTS || C::half % 64 == 0, "a box of rows of dw is 64 wide");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        prefetch_map(&map_c);
        prefetch_map(&map_r);
        prefetch_map(&map_half);
    }
    const uint32_t rank = cluster_rank(), cta = rank & 1;
    uint8_t* smem = dynamic + ((1024 - (smem_addr(dynamic) & 1023)) & 1023);
    if (tid == 0) {
        // full: the first CTA's bytes announced; with segments that may end anywhere, a word of either CTA, or at an end two of
        // the first and 16 bytes of the second
        for (int i = 0; i < C::stages; ++i) { mbar_init(&sh.full[i], F == WEIGHTS ? 2 : 1); mbar_init(&sh.empty[i], 1); mbar_init(&sh.tail[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&sh.acc_full[i], 1); mbar_init(&sh.acc_empty[i], 8 * kGroups); }
        mbar_init(&sh.drained, 1);
        mbar_fence_init();
    }
    if (warp == 2) tmem_alloc_pair(&sh.tmem, kColumns);
    tmem_fence_before();
    __syncthreads();
    cluster_sync();
    tmem_fence_after();
    wait_for_previous();   // (what is above runs while the kernel before ends: one tile 4.0 us, 4.2 with the clusters' wait below)
    let_next_start();
    const bool fits = load_segments<kThreads>(sh.seg, a, C::tile);   // the same answer in both CTAs

    const int per_pair = F == GLU ? kRows : 2 * kRows;
    const int64_t all = !fits ? 0 : (F == WEIGHTS ? (int64_t)a.E * a.rtiles.of : (int64_t)sh.seg.tile[a.E]) * a.ctiles.of;
    const int64_t limit = INT32_MAX - (int64_t)gridDim.x;   // (items + step stays a number)
    const Work<C, F> w = {a, sh, smem, sh.tmem, cta, rank - cta, (int)(rank >> 1), per_pair,
                          (int)(blockIdx.x / (2 * a.split)), (int)(all < limit ? all : limit), (int)(gridDim.x / (2 * a.split))};
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) ok = load_tiles(w, &map_c, &map_r, &map_half);
    } else if (warp == 1) {
        if (cta == 0) ok = issue_mma(w);
    } else if (warp == 3) {
        if (F == WEIGHTS) ok = clear_tails(w);
    } else if (warp >= 4) {
        ok = a.split == 1 ? epilogue<C, F, ADD>(w, warp & 3, (warp >> 2) - 1) : leave_part(w, warp & 3, (warp >> 2) - 1);
    }
    if (a.split > 1) {   // all parts are there; then each finishes its share of the tile
        __syncwarp();
        __syncthreads();
        cluster_sync();
        if (warp >= 4) ok = epilogue<C, F, ADD>(w, warp & 3, (warp >> 2) - 1) && ok;
    }
    if (!ok && a.status) ep_set_status(a.status, EP_ERR_TIMEOUT);
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    cluster_sync();   // neither CTA's shared or tensor memory goes while the pair's MMAs may read it
    if (warp == 2) tmem_free_pair(w.tmem, kColumns);
}

// How many tiles can be shared by `split` pairs each at a time: clusters that the device holds, asked once for each
// device and kernel (152 SMs hold fewer clusters of eight than 19).
template <class C, Form F>
int64_t clusters_of(int split) {
    static std::atomic<int> known[64][2];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::atomic<int>& mine = known[dev][split == 4];
    int n = mine.load(std::memory_order_relaxed);
    if (n == 0) {
        static std::atomic<uint64_t> done;
        if (allow_smem(matmul_bf16_kernel<C, F, false>, C::smem, done) != cudaSuccess) return 0;
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute attr{};
        cfg.gridDim = dim3((unsigned)(2 * split) * 64);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = C::smem;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = (unsigned)(2 * split);
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, matmul_bf16_kernel<C, F, false>, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            n = 0;
        }
        mine.store(n > 0 ? n : -1, std::memory_order_relaxed);
    }
    return n > 0 ? n : 0;
}

// c: the channels' operand, r: the rows' one.
template <class C, Form F>
cudaError_t launch(const Bf16Args& a, const void* c, const void* r, int split, int sms, cudaStream_t st) {
    static_assert(C::tile * 512 <= C::stages * C::bytes, "accumulators in the stages' place");
    const int64_t per_pair = F == GLU ? kRows : 2 * kRows, ctiles = (a.outs + per_pair - 1) / per_pair;
    CUtensorMap map_c, map_r, map_half;
    bool ok;
    const int64_t rows = a.rows > 0 ? a.rows : 1;   // (of no rows none is read)
    if constexpr (F == FORWARD) ok = make_experts_map(&map_c, c, a.E, a.outs, 2 * (int64_t)a.reduced, kRows);
    else if constexpr (F == GLU) ok = make_pairs_map(&map_c, c, a.E, a.outs, 2 * (int64_t)a.reduced, 16);
    else if constexpr (F == ROWS) ok = make_experts_map(&map_c, c, a.E, a.reduced, 2 * (int64_t)a.outs, kStep);
    else ok = make_rows_map(&map_c, c, rows, 2 * (int64_t)a.outs, kStep);
    if constexpr (F == WEIGHTS) {
        ok = ok && make_rows_map(&map_r, r, rows, 2 * (int64_t)a.n, kStep);
        map_half = map_r;
    } else {
        ok = ok && make_rows_map(&map_r, r, rows, 2 * (int64_t)a.reduced, kBoxTokens) &&
             make_rows_map(&map_half, r, rows, 2 * (int64_t)a.reduced, C::half);
    }
    if (!ok) return cudaErrorInvalidValue;
    const int64_t rtiles = F == WEIGHTS ? (int64_t)a.E * ((a.n + C::tile - 1) / C::tile) : (a.rows + C::tile - 1) / C::tile + (a.E > 1 ? a.E : 0);
    const int64_t most = rtiles * ctiles;
    if (most > INT32_MAX - sms) return cudaErrorInvalidValue;   // more output than any memory holds
    Bf16Args b = a;
    b.split = split;
    b.ctiles = divisor((uint32_t)ctiles);
    b.rtiles = divisor((uint32_t)(F == WEIGHTS ? (a.n + C::tile - 1) / C::tile : 1));
    const int64_t tiles = b.split > 1 || most < sms / 2 ? most : sms / 2;   // (a shared tile has a cluster of its own)
    auto kernel = matmul_bf16_kernel<C, F, false>;
    if constexpr (F == WEIGHTS) {
        if (a.accumulate) kernel = matmul_bf16_kernel<C, F, true>;
    }
    static std::atomic<uint64_t> done[2];
    const cudaError_t e = allow_smem(kernel, C::smem, done[a.accumulate]);
    if (e != cudaSuccess) return e;
    return launch_overlapped_clusters(kernel, 2 * b.split, dim3((unsigned)(2 * b.split * tiles)), kThreads, C::smem, st, b,
                                      map_c, map_r, map_half);
}

// What few rows take in matmul_skinny.cu, in us: 3.0 for its start, and its items are 16 channels by 32 rows, so much for each
// round of items and for each eight 128-byte pieces of a row.  (Plan's estimates are of tiles alone: kStartUs before them.)
// Measured, us in a graph (that kernel, Thin): one matrix: 8 rows x 4096 x 4096 7.1, 17.8; 32 rows 11.3, 17.8; 32 rows x 7168 x
// 512 10.1, 27.2; experts of 2048 x 1024: 8 of 32 rows with SwiGLU 13.3, 14.4; 16 of 8 rows 14.4, 12.5; 32 of 8 rows 33.6,
// 27.6; 64 of 4 rows, 4096 x 1024: 95.8, 87.9.
double few_rows_us(const Bf16Args& a, bool glu, int sms) {
    const int64_t experts = a.rows < a.E ? a.rows : a.E, each = (a.rows + a.E - 1) / a.E;
    if (each > 32) return 1e30;
    const double more[4] = {1.0, 1.15, 1.35, 1.6};   // by tiles of eight rows
    const double rounds = (double)(experts * ((a.outs + (glu ? 7 : 15)) / (glu ? 8 : 16))) / (2 * sms);
    return 3.0 + (rounds > 0.6 ? rounds : 0.6) * (0.9 + 0.75 * ((a.reduced + 511) / 512) * more[(each - 1) / 8]);
}

// Which tile, and how many pairs share its sum: whatever is over first by this estimate in us, of rounds of tiles of so many
// steps of 64 and of their way out.  The larger tiles do more products for what they read, the smaller ones are more, and pay for fewer rows that
// are none; to share a sum takes a meeting, and clusters that find room.
// Measured, us in a graph (256, 128, 64 rows a tile):
//   one matrix: 500 rows x 4096 x 1024: 22.9, 18.4, 18.4; 1000 x 2048 x 2048: 14.7, 12.6, 19.2; 4000 x 2048 x 2048 with SwiGLU: 25.9,
//   42.8, 69.2; experts: 64 of 100 rows, 2048 x 1024: 58.4, 54.2, 59.7; 16 of 166, 4096 x 2048: 55.3, 67.3, 87.3; 64 of 512, 256 x
//   1024: 26.5, 33.2, 51.3; 128 of 200, 4096 x 2048 with SwiGLU: 377, 572, 983; 32 of 64, 1024 x 2048 with SwiGLU: 31.5, 31.3, 30.2.
//   dw: 2000 rows, 1024 x 1024: 17.6, 14.8; 16384 rows: 93.2, 75.9; 4 experts of 2000 rows, 2048 x 512: 17.1, 22.8; 128 of 64
//   rows, 2048 x 1024: 108, 130, in float32 199, 200.
// Measured, us in a graph (one, two, four pairs): 50 rows x 4096 x 512: 21.1, 15.8, 13.2; 300 x 7168 x 512 with SwiGLU: 35.8,
// 23.5, 18.2; 128 x 2048 x 1024: 11.8, 11.4, 11.9; dw of 13922 rows, 992 x 376: 59.6, 35.5, 24.9; of 1000 rows, 512 x 512: 9.9,
// 10.2, 11.2.
struct Plan {
    int tile = 0, split = 1;
    double us = 1e30;
    // tiles: that there may be
    template <class C, Form F>
    void consider(double per_step, double per_row, int64_t tiles, int64_t steps, int sms) {
        const double meeting[3] = {0.0, 2.8, 4.2}, store = per_row * C::tile;
        for (int s = 0; s < 3; ++s) {
            if (s > 0 && (tiles > sms / 4 || steps < 16 || tiles > clusters_of<C, F>(1 << s))) break;
            const int64_t rounds = (tiles + sms / 2 - 1) / (sms / 2), part = (steps + (1 << s) - 1) >> s;
            // a tile is stored under the next one's products
            const double sum = (double)part * per_step, longer = sum > store ? sum : store;
            const double t = (double)rounds * (longer + 0.45) + sum + store - longer + meeting[s];
            if (t < us) us = t, tile = C::tile, split = 1 << s;
        }
    }
};

// Clusters, barriers, tensor memory and the first loads: a tile of 8 rows, 8 channels and 8 of the sum takes 3.7 to 4.0 us in
// a graph.
constexpr double kStartUs = 4.0;

template <Form F>
cudaError_t choose(const Bf16Args& a, const void* c, const void* r, int sms, cudaStream_t st) {
    const int64_t per_pair = F == GLU ? kRows : 2 * kRows, ctiles = (a.outs + per_pair - 1) / per_pair;
    const int64_t each = F == WEIGHTS ? a.n : (a.rows + a.E - 1) / a.E;   // rows of a segment, or of a matrix
    const int64_t E = F == WEIGHTS || a.rows > a.E ? a.E : a.rows;
    // tiles of rows, of segments that end inside one
    auto rtiles = [&](int64_t tile) {
        if (F == WEIGHTS || E == 1) return (each + tile - 1) / tile * E;
        const int64_t n = a.rows / tile + (3 * E + 4) / 5;
        return n > E ? n : E;
    };
    const int64_t steps = ((F == WEIGHTS ? (a.rows + a.E - 1) / a.E : a.reduced) + kStep - 1) / kStep;
    // a CTA's part of a tile leaves at about 27 bytes a clock in float32, 24 in bf16.  (Us in a graph, 256 rows a tile, 128: 128 experts
    // of 200 rows, 256 x 512: 13.6, 17.2; dw of 16 experts of 166 rows, 1024 x 1408: 18.2, 20.2.)
    const double per_row = a.wide ? 0.0102 : F == GLU ? 0.004 : 0.0055;
    Plan plan;
    if constexpr (F != WEIGHTS) {
        if (each <= 32) plan.consider<Thin, F>(0.22, per_row, rtiles(Thin::tile) * ctiles, steps, sms);
    }
    plan.consider<Mid, F>(0.24, per_row, rtiles(Mid::tile) * ctiles, steps, sms);
    if (each > Mid::tile) plan.consider<Thick, F>(0.30, per_row, rtiles(Thick::tile) * ctiles, steps, sms);
    if constexpr (F == FORWARD || F == GLU) {
        if (few_rows_us(a, F == GLU, sms) <= kStartUs + plan.us) {
            MatmulArgs m{};
            m.a = (const uint8_t*)r;
            m.w = (const uint8_t*)c;
            m.expert_base = a.expert_base;
            m.out = (uint16_t*)a.out;
            m.status = a.status;
            m.rows = a.rows;
            m.K = a.reduced; m.N = F == GLU ? 2 * a.outs : a.outs; m.E = a.E;
            m.swiglu = F == GLU;
            return launch_matmul_skinny_bf16(m, sms, st);
        }
    }
    if (plan.tile == Thick::tile) return launch<Thick, F>(a, c, r, plan.split, sms, st);
    if constexpr (F != WEIGHTS) {
        if (plan.tile == Thin::tile) return launch<Thin, F>(a, c, r, plan.split, sms, st);
    }
    return launch<Mid, F>(a, c, r, plan.split, sms, st);
}

template <Form F>
ep_status run(const Bf16Args& a, const void* c, const void* r, cudaStream_t st) {
    const int sms = ep_current_sms();
    if (sms <= 0) return EP_ERR_CUDA;
    return choose<F>(a, c, r, sms, st) == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

bool sizes_ok(int64_t rows, int32_t reduced, int32_t n, int32_t E, const void* base, const void* status) {
    return rows >= 0 && rows < INT32_MAX && reduced >= 8 && reduced <= 65536 && reduced % 8 == 0 && n >= 1 && n <= 65536 && E >= 1 &&
           E <= kMaxExperts && (E == 1 || base) && aligned(base, 4) && aligned(status, 4);
}

Bf16Args args_of(int64_t rows, int32_t E, const int32_t* base, void* out, int32_t* status) {
    Bf16Args a{};
    a.expert_base = base;
    a.status = status;
    a.out = out;
    a.rows = rows;
    a.E = E;
    return a;
}

}  // namespace

extern "C" ep_status ep_expert_matmul_bf16(const void* a, int64_t rows, int32_t k, const void* w, int32_t n, int32_t num_experts,
                                           const int32_t* expert_base, int32_t swiglu, void* out, int32_t* status,
                                           ep_stream_t stream) {
    if (!sizes_ok(rows, k, n, num_experts, expert_base, status)) return EP_ERR_INVALID_ARG;
    if ((swiglu != 0 && swiglu != 1) || (swiglu && n % 2 != 0) || !w || !aligned(w, 16)) return EP_ERR_INVALID_ARG;
    if (rows == 0) return EP_OK;
    if (!a || !aligned(a, 16) || !out || !aligned(out, 2)) return EP_ERR_INVALID_ARG;
    Bf16Args b = args_of(rows, num_experts, expert_base, out, status);
    b.outs = swiglu ? n / 2 : n;
    b.reduced = k;
    return swiglu ? run<GLU>(b, w, a, (cudaStream_t)stream) : run<FORWARD>(b, w, a, (cudaStream_t)stream);
}

extern "C" ep_status ep_expert_matmul_grad_rows(const void* grad_c, int64_t rows, int32_t n, const void* w, int32_t k,
                                                int32_t num_experts, const int32_t* expert_base, void* grad_a, int32_t* status,
                                                ep_stream_t stream) {
    if (!sizes_ok(rows, n, k, num_experts, expert_base, status) || k < 8 || k % 8 != 0 || !w || !aligned(w, 16)) return EP_ERR_INVALID_ARG;
    if (rows == 0) return EP_OK;
    if (!grad_c || !aligned(grad_c, 16) || !grad_a || !aligned(grad_a, 4)) return EP_ERR_INVALID_ARG;
    Bf16Args b = args_of(rows, num_experts, expert_base, grad_a, status);
    b.outs = k;
    b.reduced = n;
    return run<ROWS>(b, w, grad_c, (cudaStream_t)stream);
}

extern "C" ep_status ep_expert_matmul_grad_weights(const void* grad_c, const void* a, int64_t rows, int32_t n, int32_t k,
                                                   int32_t num_experts, const int32_t* expert_base, int32_t float32_out,
                                                   int32_t accumulate, void* grad_w, int32_t* status, ep_stream_t stream) {
    if (!sizes_ok(rows, n, k, num_experts, expert_base, status) || k < 8 || k % 8 != 0) return EP_ERR_INVALID_ARG;
    if ((float32_out != 0 && float32_out != 1) || (accumulate != 0 && accumulate != 1)) return EP_ERR_INVALID_ARG;
    if (!grad_w || !aligned(grad_w, 4)) return EP_ERR_INVALID_ARG;
    if (accumulate && !float32_out) return EP_ERR_UNSUPPORTED;
    if (rows > 0 && (!grad_c || !aligned(grad_c, 16) || !a || !aligned(a, 16))) return EP_ERR_INVALID_ARG;
    Bf16Args b = args_of(rows, num_experts, expert_base, grad_w, status);
    b.outs = k;
    b.n = n;
    b.wide = float32_out;
    b.accumulate = accumulate;
    if (rows == 0) a = grad_c = (const void*)((uintptr_t)grad_w & ~(uintptr_t)15);   // an address for tensor maps that nothing reads
    return run<WEIGHTS>(b, a, grad_c, (cudaStream_t)stream);
}
