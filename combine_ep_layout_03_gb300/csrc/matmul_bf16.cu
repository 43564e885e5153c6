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
// dw reduces over token rows, and a segment ends anywhere: the rows of its last 16 that belong to others (to the next
// expert, or to nobody, with any contents) are set to zero in shared memory, in both operands, between their arrival
// and their product.
#include "expert_ops.cuh"
#include "expert_tiles.cuh"
#include "tcgen05.cuh"
#include "tensor_maps.cuh"

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
};

constexpr int kGroups = 2;                // of four epilogue warps, which take every other 32 rows of a tile
constexpr int kThreads = 32 * (4 + 4 * kGroups);
constexpr int kRows = 128;                // channels of a CTA
constexpr int kStep = 64;                 // of the sum a stage: 128 bytes
constexpr int kBytesA = kRows * 128;
constexpr int kBoxTokens = 32;            // rows of a small token box
constexpr int kBlock = 64 * 128;          // MN-major: 64 channels or rows by 64 of the sum
constexpr uint32_t kColumns = 512;        // of tensor memory

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
    int per_pair, ctiles, rtiles;   // channels of a tile, tiles of channels, WEIGHTS: tiles of rows
    int first, items, step;

    // The tile, and its stages of the sum.
    template <bool WARP>
    __device__ __forceinline__ Tile tile(int item, int& e, int& steps) const {
        if constexpr (F == WEIGHTS) {
            const uint32_t each = (uint32_t)(ctiles * rtiles), local = (uint32_t)item % each;
            Tile t;
            e = (int)((uint32_t)item / each);
            t.expert = e;
            const Place p = place_of(local, (uint32_t)rtiles, (uint32_t)ctiles);
            t.channel = p.channel;
            t.row0 = (int64_t)p.tile * C::tile;
            t.m = min(C::tile, a.n - (int)t.row0);
            t.n = (t.m + 31) / 32 * 32;
            steps = (sh.seg.rows[e] + kStep - 1) / kStep;
            return t;
        } else {
            steps = (a.reduced + kStep - 1) / kStep;
            return tile_of<WARP>(sh.seg, a.E, ctiles, item, e);
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
    const uint32_t full0 = cluster_addr(smem_addr(&w.sh.full[0]), 0);
    int used = 0, expert = 0;   // used: stages filled so far, at most all
    bool ok = true;
    for (int item = w.first; ok && item < w.items; item += w.step) {
        int steps;
        const Tile t = w.template tile<false>(item, expert, steps);
        const int half = t.n / 2;
        const int boxes = F == WEIGHTS ? (half + 63) / 64 : (half + kBoxTokens - 1) / kBoxTokens;
        const int bytes = kBytesA + boxes * (F == WEIGHTS ? kBlock : kBoxTokens * 128);
        const int ch = t.channel * w.per_pair + (int)w.cta * (F == GLU ? kRows / 2 : kRows);
        const int row = (int)t.row0 + (int)w.cta * half;
        for (int k = 0; k < steps; ++k, r.next()) {
            if (!mbar_wait_parked(&w.sh.empty[r.stage], r.parity ^ 1)) { ok = false; break; }
            uint8_t* dst = w.smem + r.stage * C::bytes;
            uint32_t bar = full0 + r.stage * 8;
            if (w.ragged(t, k)) {
                bar = smem_addr(&w.sh.tail[r.stage]);
                mbar_arrive_expect_tx(&w.sh.tail[r.stage], bytes);
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
            if constexpr (F != WEIGHTS) {   // rows in one box where the tile is full, else in boxes of 32
                if (boxes == C::half / kBoxTokens) {
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
    const uint32_t full0 = cluster_addr(smem_addr(&w.sh.full[0]), 0);
    uint32_t parity = 0;   // of each stage's tail barrier
    const int lane = threadIdx.x & 31;
    int expert = 0;
    for (int item = w.first; item < w.items; item += w.step) {
        int steps;
        const Tile t = w.template tile<true>(item, expert, steps);
        if (steps == 0) continue;
        for (int k = 0; k < steps - 1; ++k) r.next();
        if (w.ragged(t, steps - 1)) {
            if (!warp_wait(&w.sh.tail[r.stage], (parity >> r.stage) & 1)) return false;
            parity ^= 1u << r.stage;
            const int blocks = 2 + (t.n / 2 + 63) / 64, first = w.left(t, steps - 1), end = (first + 15) / 16 * 16;
            const uint32_t at = smem_addr(w.smem + r.stage * C::bytes);
            for (int i = lane; i < blocks * (end - first) * 8; i += 32) {
                const int piece = i & 7, row = first + (i >> 3) % (end - first), block = (i >> 3) / (end - first);
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};"
                             :: "r"(at + block * kBlock + row * 128 + piece * 16), "r"(0) : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(full0 + r.stage * 8);
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
        if (steps == 0) continue;
        const uint32_t idesc = mma_desc_bf16(2 * kRows, t.n, a_mn, b_mn);
        if (!warp_wait(&w.sh.acc_empty[acc.stage], acc.parity ^ 1)) { ok = false; break; }
        tmem_fence_after();
        const uint32_t d = w.tmem + acc.stage * C::tile;
        for (int k = 0; k < steps; ++k) {
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
                    if (j < pieces) mma_pair_f16_ss(d, a + j * (a_mn ? 128 : 2), b + j * (b_mn ? 128 : 2), idesc, k > 0 || j > 0);
                commit_pair(empty);
            }
            __syncwarp();
        }
        if (ok && elect_one()) commit_pair(&w.sh.acc_full[acc.stage]);
        __syncwarp();
        acc.next();
    }
    // no MMA is left when the CTAs part, also when a wait gave up
    if (elect_one()) commit_leader(&w.sh.drained);
    __syncwarp();
    return warp_wait(&w.sh.drained, 0) && ok;
}

// Lane: a channel; with gates and ups, lanes 0-15 hold the gates of lanes 16-31's ups.
template <class C, Form F>
__device__ __forceinline__ bool epilogue(const Work<C, F>& w, int warp, int group) {
    const int lane = threadIdx.x & 31;
    const uint32_t acc_empty0 = cluster_addr(smem_addr(&w.sh.acc_empty[0]), 0);
    const int64_t outs = w.a.outs;
    uint16_t* const out16 = (uint16_t*)w.a.out;
    // two channels a store where rows keep them on four bytes
    const bool wide = (outs & 1) == 0 && ((uintptr_t)w.a.out & 3) == 0;
    Ring<2> acc;
    int expert = 0;
    for (int item = w.first; item < w.items; item += w.step) {
        int steps;
        const Tile t = w.template tile<true>(item, expert, steps);
        if (F == WEIGHTS && steps == 0 && w.a.accumulate) continue;
        const int ch = t.channel * w.per_pair + (int)w.cta * (F == GLU ? kRows / 2 : kRows) + warp * (F == GLU ? 16 : 32) +
                       (F == GLU ? lane & 15 : lane);
        const bool in = ch < outs;
        const int64_t row0 = F == WEIGHTS ? (int64_t)t.expert * w.a.n + t.row0 : t.row0;
        const bool some = F != WEIGHTS || steps > 0;   // an expert without rows: zeros
        if (some) {
            if (!warp_wait(&w.sh.acc_full[acc.stage], acc.parity)) return false;
            tmem_fence_after();
        }
        const uint32_t d = w.tmem + ((uint32_t)(warp * 32) << 16) + acc.stage * C::tile;
        for (int c0 = 32 * group; c0 < t.m; c0 += 32 * kGroups) {
            uint32_t v[32];
            if (some) {
                tmem_load32(d + c0, v);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0;
            }
            const int left = t.m - c0;
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
                    // neighbours trade as below: an even lane stores its pair of channels of row i + odd, an odd
                    // lane that of row i + 2 + odd
                    const int last = lane & 1;
                    const uint32_t sel = last ? 0x3276u : 0x5410u;
                    uint16_t* out = out16 + (row0 + c0 + odd + 2 * last) * outs + (ch - last);
#pragma unroll
                    for (int i = 0; i < 32; i += 4, out += 4 * outs) {
                        const uint32_t p = pack_bf16x2_rn(y[i / 2], y[i / 2 + 1]);
                        const uint32_t both = __byte_perm(p, __shfl_xor_sync(0xffffffffu, p, 1), sel);
                        if (in && i + odd + 2 * last < left) *reinterpret_cast<uint32_t*>(out) = both;
                    }
                } else {
                    uint16_t* out = out16 + (row0 + c0 + odd) * outs + ch;
#pragma unroll
                    for (int i = 0; i < 32; i += 2, out += 2 * outs)
                        if (in && i + odd < left) *out = (uint16_t)pack_bf16x2_rn(y[i / 2], 0.0f);
                }
            } else if (F == WEIGHTS && w.a.wide) {
                float* out = (float*)w.a.out + (row0 + c0) * outs + ch;
                if (w.a.accumulate) {
                    float before[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) before[i] = in && i < left ? out[i * outs] : 0.0f;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (in && i < left) out[i * outs] = before[i] + __uint_as_float(v[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (in && i < left) out[i * outs] = __uint_as_float(v[i]);
                }
            } else if (wide) {
                // neighbours trade halves: an even lane stores both channels of the even row
                const int odd = lane & 1;
                const uint32_t sel = odd ? 0x3276u : 0x5410u;
                uint16_t* out = out16 + (row0 + c0 + odd) * outs + (ch - odd);
#pragma unroll
                for (int i = 0; i < 32; i += 2, out += 2 * outs) {
                    const uint32_t y = pack_bf16x2_rn(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                    const uint32_t both = __byte_perm(y, __shfl_xor_sync(0xffffffffu, y, 1), sel);
                    if (in && i + odd < left) *reinterpret_cast<uint32_t*>(out) = both;
                }
            } else {
                uint16_t* out = out16 + (row0 + c0) * outs + ch;
#pragma unroll
                for (int i = 0; i < 32; ++i, out += outs)
                    if (in && i < left) *out = (uint16_t)pack_bf16x2_rn(__uint_as_float(v[i]), 0.0f);
            }
        }
        if (some) {
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_empty0 + acc.stage * 8);
            acc.next();
        }
    }
    return true;
}

template <class C, Form F>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
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
    const uint32_t cta = cluster_rank();
    uint8_t* smem = dynamic + ((1024 - (smem_addr(dynamic) & 1023)) & 1023);
    if (tid == 0) {
        // full: the first CTA's bytes announced; with segments that may end anywhere, a word of either CTA
        for (int i = 0; i < C::stages; ++i) { mbar_init(&sh.full[i], F == WEIGHTS ? 2 : 1); mbar_init(&sh.empty[i], 1); mbar_init(&sh.tail[i], 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(&sh.acc_full[i], 1); mbar_init(&sh.acc_empty[i], 8 * kGroups); }
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

    const int per_pair = F == GLU ? kRows : 2 * kRows;
    const int ctiles = (a.outs + per_pair - 1) / per_pair, rtiles = F == WEIGHTS ? (a.n + C::tile - 1) / C::tile : 0;
    const int64_t all = !fits ? 0 : F == WEIGHTS ? (int64_t)a.E * ctiles * rtiles : (int64_t)sh.seg.tile[a.E] * ctiles;
    const int64_t limit = INT32_MAX - (int64_t)gridDim.x;   // (items + step stays a number)
    const Work<C, F> w = {a, sh, smem, sh.tmem, cta, per_pair, ctiles, rtiles,
                          (int)(blockIdx.x >> 1), (int)(all < limit ? all : limit), (int)(gridDim.x >> 1)};
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) ok = load_tiles(w, &map_c, &map_r, &map_half);
    } else if (warp == 1) {
        if (cta == 0) ok = issue_mma(w);
    } else if (warp == 3) {
        if (F == WEIGHTS) ok = clear_tails(w);
    } else if (warp >= 4) {
        ok = epilogue(w, warp & 3, (warp >> 2) - 1);
    }
    if (!ok && a.status) ep_set_status(a.status, EP_ERR_TIMEOUT);
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    cluster_sync();   // neither CTA's shared or tensor memory goes while the pair's MMAs may read it
    if (warp == 2) tmem_free_pair(w.tmem, kColumns);
}

// c: the channels' operand, r: the rows' one.
template <class C, Form F>
cudaError_t launch(const Bf16Args& a, const void* c, const void* r, int sms, cudaStream_t st) {
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
    const int64_t pairs = most < sms / 2 ? most : sms / 2;
    static std::atomic<uint64_t> done;
    const cudaError_t e = allow_smem(matmul_bf16_kernel<C, F>, C::smem, done);
    if (e != cudaSuccess) return e;
    return launch_overlapped(matmul_bf16_kernel<C, F>, dim3((unsigned)(2 * pairs)), kThreads, C::smem, st, a, map_c, map_r, map_half);
}

// Few enough rows and weights for matmul_skinny.cu, which is on every SM from the start, and reads weights the slower the
// more rows there are; a tile here takes 0.3 us for 64 k, however few its rows.
// Measured, us in a graph (that kernel, Thin): one matrix: 8 rows x 4096 x 4096 7.1, 17.8; 32 rows 11.3, 17.8; 32 rows x 7168 x
// 512 10.1, 27.2; experts of 2048 x 1024: 8 of 32 rows with SwiGLU 13.3, 14.4; 16 of 8 rows 14.4, 12.5; 32 of 8 rows 33.6,
// 27.6; 64 of 4 rows, 4096 x 1024: 95.8, 87.9.
bool few_rows(const Bf16Args& a, bool glu, int sms) {
    const int64_t experts = a.rows < a.E ? a.rows : a.E, rows = (a.rows + a.E - 1) / a.E, per_pair = glu ? kRows : 2 * kRows;
    if (rows > 32) return false;
    const double rate[4] = {5.0, 4.5, 4.0, 3.5};   // bytes of weights a picosecond, by tiles of eight rows
    const double here = 3.5 + 2e-6 * (double)(experts * a.outs * (glu ? 2 : 1)) * a.reduced / rate[(rows - 1) / 8];
    const int64_t rounds = (experts * ((a.outs + per_pair - 1) / per_pair) + sms / 2 - 1) / (sms / 2);
    return here <= 4.0 + 0.3 * (double)(rounds * ((a.reduced + kStep - 1) / kStep));
}

// Which tile: the larger ones do more products for what they read, the smaller ones are more, and pay for fewer rows that
// are none.  Measured, us (256, 128, 64 rows a tile):
//   one matrix: 128 rows x 4096 x 4096: 29.3, 23.2, 23.2; 2000 x 2048 x 1000: 19.1, 17.1, 23.2; 4000 x 2048 x 2000: 29.3,
//   39.6, 60.1; experts: 64 of 96 rows, 2048 x 1024: 73.7, 68.3, 70.4; 64 of 128, 4096 x 2048: 201, 193, 218; 128 of 200:
//   392, 441, 734; 128 of 6 with SwiGLU: 361, 353, 334.
//   dw: 2000 rows, 1024 x 1024: 21.2, 17.1; 16384 rows: 88.7, 72.4; 4 experts of 2000 rows, 2048 x 512: 23.2, 27.3; 128 of 64
//   rows, 2048 x 1024: 132, 156.
// So: 64 up to 32 rows an expert; 128 where its rounds of tiles, which take 0.8 of the time of 256's, are that few, or
// segments are no longer than that.
template <Form F>
cudaError_t choose(const Bf16Args& a, const void* c, const void* r, int sms, cudaStream_t st) {
    const int64_t per_pair = F == GLU ? kRows : 2 * kRows, ctiles = (a.outs + per_pair - 1) / per_pair, pairs = sms / 2;
    const int64_t each = F == WEIGHTS ? a.n : (a.rows + a.E - 1) / a.E;   // rows of a segment, or of a matrix
    if constexpr (F == FORWARD || F == GLU) {
        if (few_rows(a, F == GLU, sms)) {
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
    if constexpr (F != WEIGHTS) {
        if (each <= 32) return launch<Thin, F>(a, c, r, sms, st);
    }
    const int64_t mid = ((each + Mid::tile - 1) / Mid::tile * a.E * ctiles + pairs - 1) / pairs;
    const int64_t thick = ((each + Thick::tile - 1) / Thick::tile * a.E * ctiles + pairs - 1) / pairs;
    return each <= Mid::tile || 4 * mid < 5 * thick ? launch<Mid, F>(a, c, r, sms, st) : launch<Thick, F>(a, c, r, sms, st);
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
