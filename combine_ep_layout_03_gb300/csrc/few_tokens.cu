// few_tokens.cu -- the whole expert layer for up to 64 tokens in two kernels:
//   inner[t, e] = weight[t, e] * silu(Wg[e] x[t]) * (Wu[e] x[t])        few_inner_kernel
//   out[t]      = sum over e of W2[e] inner[t, e] (+ shared rows)       few_out_kernel
// Every expert that a token chose is read once, whole, and nothing else of the weights:
// the floor is those bytes.  Both kernels find the chosen experts and their tokens from
// topk_idx by themselves (a bit mask of tokens for each expert in shared memory), so
// there is no layout, dispatch or combine pass and no row moves.
//
// The inner rows are float32 results that the second product needs as bf16.  One
// rounding there would cost as much as the output's own; they are kept as a bf16 value
// and a bf16 remainder (16 significant bits) instead, and the second kernel multiplies
// by both: the tensor cores have time to spare while the weights arrive.
//
// Sums run in a fixed order (warps take fixed pieces, their partial sums are added in
// warp order): results do not vary from run to run.
//
// Measured (both kernels): 64 tokens over 512 experts of 4096 x 512, bf16: 865 us, 6.45 TB/s (0.95 of
// the copy bandwidth); 16 tokens over 128 experts of 4096 x 1024: 316 us, 6.6 TB/s; one token 39 us,
// 5.1 TB/s, of which about 9 us are the two starts.  int8 weights are bound by instruction issue,
// most of it their conversion: 8 tokens of 256 experts of 7168 x 1024 233 us, 5.3 TB/s;
// one token of 128 experts of 4096 x 1024 33 us, 3.1 TB/s.  Many tokens on few experts are bound by
// the token values' way from L2, each time for 16 weight rows: 64 tokens over 8 experts of 4096 x 1024,
// bf16, 69 us by two and 139 us by eight (the weights' bytes are 30).
#include <algorithm>

#include "expert_ops.cuh"
#include "skinny.cuh"
#include "tensor_maps.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxEntries = kFewMaxTokens * kMaxTopk;

// What a CTA knows of the routing: the experts with a token, in ascending order, and the
// rows of their tokens (ascending; rows of one expert are neighbours in `inner`).
struct Routing {
    unsigned long long mask[kMaxExperts];
    int16_t expert[kMaxExperts];
    int16_t base[kMaxExperts + 1];
    uint8_t token[kMaxEntries];
    int32_t warp_sum[kWarps];
    int32_t count;   // experts with a token
};

__device__ __forceinline__ void build_routing(Routing& r, const FewArgs& a) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < a.E; e += kThreads) r.mask[e] = 0;
    __syncthreads();
    for (int i = tid; i < a.T * a.K; i += kThreads) {
        const int64_t e = a.topk[i];
        if (e >= 0 && e < a.E) atomicOr(&r.mask[e], 1ull << (i / a.K));
        else if (e != -1 && a.status) ep_set_status(a.status, EP_ERR_BAD_EXPERT_ID);
    }
    __syncthreads();
    // thread t holds experts 2t and 2t + 1; experts in the high half of the sums, rows in the low
    const int e0 = 2 * tid;
    const unsigned long long m0 = e0 < a.E ? r.mask[e0] : 0, m1 = e0 + 1 < a.E ? r.mask[e0 + 1] : 0;
    const int v0 = m0 ? (1 << 16) + __popcll(m0) : 0, v1 = m1 ? (1 << 16) + __popcll(m1) : 0;
    int s = v0 + v1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += n;
    }
    if (lane == 31) r.warp_sum[warp] = s;
    __syncthreads();
    for (int w = 0; w < warp; ++w) s += r.warp_sum[w];
    int at = s - v0 - v1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const unsigned long long m = h ? m1 : m0;
        if (m) {
            const int pos = at >> 16;
            int row = at & 0xffff;
            r.expert[pos] = (int16_t)(e0 + h);
            r.base[pos] = (int16_t)row;
            for (unsigned long long left = m; left; left &= left - 1) r.token[row++] = (uint8_t)(__ffsll(left) - 1);
        }
        at += h ? v1 : v0;
    }
    if (tid == kThreads - 1) {
        r.count = s >> 16;
        r.base[s >> 16] = (int16_t)(s & 0xffff);
    }
    __syncthreads();
}

static_assert(kMaxExperts <= 2 * kThreads, "a thread holds two experts");
static_assert(kFewMaxTokens <= 64, "a token mask is 64 bits");

// Router weight of (token, expert): its entries' weights in slot order (one, unless a
// token names an expert twice).
__device__ __forceinline__ float routing_weight(const FewArgs& a, int token, int expert) {
    float w = 0.0f;
    for (int k = 0; k < a.K; ++k) {
        const float v = a.topk_w[token * a.K + k];
        w += a.topk[token * a.K + k] == expert ? v : 0.0f;
    }
    return w;
}

// Sizes of both kernels by weight type and largest number of token tiles.
//   ctas     CTAs of an SM; what the routing and the sums leave of its shared memory goes to the rings (depth).
//   early    token parts that are asked for before the weights of their piece are waited for.  64 tokens, bf16,
//            over 8 experts by two: 64 us with 3, 68 with 4 (spills), 69 with 2, 96 with none, in one run.
//   prefetch whether with one token tile those of the next piece are loaded under this one's products.  It
//            helps bf16 weights (64 tokens over 512 experts: 914 us with, 1015 us without); int8 weights
//            need the registers for their conversion and gain more from other warps (8 tokens of 256 experts:
//            276 us with it and two CTAs, 255 us without, 238 us without and with three CTAs).
template <bool W8, int MAXNT>
struct Sizes {
    static constexpr int ctas = W8 && MAXNT == 1 ? 3 : 2;
    static constexpr int depth = ctas == 3 ? 3 : W8 ? (MAXNT == 2 ? 4 : 3) : MAXNT == 1 ? 6 : MAXNT == 2 ? 5 : 4;
    static constexpr int early = 3;
    static constexpr bool prefetch = !W8;
    using Ring = WeightRing<depth>;
    static constexpr int ring_bytes = kWarps * Ring::kWarpBytes;
    // inner: [buffer][warp][column][16 rows]; two buffers in turn, so that one barrier an item is enough, but one
    // where 64 columns make them large
    static constexpr int buffers = MAXNT > 2 ? 1 : 2;
    static constexpr int inner_smem = 1024 + ring_bytes + buffers * kWarps * MAXNT * 8 * 16 * 4;
    static constexpr int out_smem = 1024 + ring_bytes + kWarps * MAXNT * 8 * 16 * 4;   // [warp][token][16 columns]
    static_assert(ctas * (inner_smem + (int)sizeof(Routing) + 1536) <= 228 * 1024, "shared memory of an SM");
};

__device__ __forceinline__ uint8_t* aligned_smem(uint8_t* p) {
    return p + ((1024 - (smem_addr(p) & 1023)) & 1023);
}

// Work of few_inner_kernel.  A tile is eight inner channels of one expert: their gate rows are rows 0-7
// of the 16 rows and their up rows 8-15, so a lane ends with both of a channel.  1 << share_log warps
// share a tile's k and add their parts in shared memory; an item is the `sets` tiles side by side that a
// CTA works on at a time.  Where the items past the last full round of CTAs have no more tiles than there
// are CTAs they are dealt out tile by tile, each to all eight warps of a CTA, so that the last round is a
// short one (6 tokens over 32 experts of 6416 x 1232, int8: 103 us for 110; no gain from tiles of a few
// pieces, or from two short rounds for a long one: 12.7 us for 14.3, 94 for 98).
struct InnerPlan {
    int share_log, sets_log, tiles, groups, full, units;
    __device__ __forceinline__ InnerPlan(int share_log, int tiles, int experts, int step, int pieces)
        : share_log(share_log), sets_log(3 - share_log), tiles(tiles) {
        groups = (tiles + (1 << sets_log) - 1) >> sets_log;
        const int items = experts * groups;
        full = items / step * step;
        if (pieces < 2 * kWarps || (items - full) << sets_log > step) full = items;
        units = full + ((items - full) << sets_log);
    }
    struct Unit { int pos, tile0, share_log; };   // place of the expert in the routing, first tile, warps of a tile
    __device__ __forceinline__ Unit unit(int u) const {
        const int tail = u - full, item = tail < 0 ? u : full + (tail >> sets_log);
        const int pos = item / groups, tile0 = (item - pos * groups) << sets_log;
        if (tail < 0) return {pos, tile0, share_log};
        return {pos, tile0 + (tail & ((1 << sets_log) - 1)), 3};
    }
};
static_assert(kWarps == 8, "share_log is at most 3");

// A warp's way through its pieces: units unit, unit + step, ... and in each the pieces rank, rank + share, ...
// of its tile, if it has one there.
struct InnerCursor {
    int unit, tile, piece, expert, rank, share;
    __device__ __forceinline__ void place(const Routing& r, const InnerPlan& p, int step, int warp, int pieces) {
        for (; unit < p.units; unit += step) {
            const InnerPlan::Unit n = p.unit(unit);
            share = 1 << n.share_log;
            rank = warp & (share - 1);
            tile = n.tile0 + (warp >> n.share_log);
            if (tile < p.tiles && rank < pieces) {
                expert = r.expert[n.pos];
                piece = rank;
                return;
            }
        }
    }
};

template <bool W8, int MAXNT>
__global__ void __launch_bounds__(kThreads, Sizes<W8, MAXNT>::ctas) few_inner_kernel(const FewArgs a, int share_log, const __grid_constant__ CUtensorMap map_w) {
    extern __shared__ uint8_t dynamic[];
    __shared__ Routing r;
    using S = Sizes<W8, MAXNT>;
    __shared__ uint64_t bars[kWarps * S::depth];
    uint8_t* const slots = aligned_smem(dynamic);
    constexpr int kBuffers = S::buffers, kSums = kWarps * MAXNT * 8 * 16;
    float* const red = reinterpret_cast<float*>(slots + S::ring_bytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    if (tid == 0) prefetch_map(&map_w);
    wait_for_previous();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    build_routing(r, a);
    const int step = gridDim.x;
    const int k_bytes = a.H * (W8 ? 1 : 2), pieces = (k_bytes + 127) / 128;
    const InnerPlan plan(share_log, a.I / 8, r.count, step, pieces);
    typename S::Ring ring(slots, bars, warp, lane);
    InnerCursor ahead;
    ahead.unit = blockIdx.x;
    ahead.place(r, plan, step, warp, pieces);
    auto fetch = [&]() {
        if (ahead.unit >= plan.units) return;
        ring.put(lane, 2048, [&](uint8_t* slot, uint64_t* bar) {
            tma_load_4d(slot, &map_w, ahead.piece * 128, ahead.tile * 8, 0, ahead.expert, bar);
        });
        ahead.piece += ahead.share;
        if (ahead.piece >= pieces) {
            ahead.unit += step;
            ahead.place(r, plan, step, warp, pieces);
        }
    };
    for (int d = 0; d < S::depth; ++d) fetch();

    int buffer = 0;
    for (int u = blockIdx.x; u < plan.units; u += step, buffer ^= 1) {
        const InnerPlan::Unit unit = plan.unit(u);
        const int tile0 = unit.tile0, log = unit.share_log, share = 1 << log, rank = warp & (share - 1);
        const int e = r.expert[unit.pos], row0 = r.base[unit.pos], m = r.base[unit.pos + 1] - row0;
        const int nt = (m + 7) / 8, my_pieces = tile0 + (warp >> log) < plan.tiles ? pieces : 0;
        const int width_log = 6 - log, width = 1 << width_log;   // channels of the unit
        float* sums = red + (kBuffers == 2 ? buffer * kSums : 0);
        // what the sums below will be multiplied by arrives meanwhile
        struct Factors { float gate, up, weight; };
        auto factors = [&](int i) {
            Factors f = {1.0f, 1.0f, routing_weight(a, r.token[row0 + (i >> width_log)], e)};
            if constexpr (W8) {
                const float* sc = a.w13_scales + (int64_t)e * 2 * a.I + tile0 * 8 + (i & (width - 1));
                f.gate = sc[0];
                f.up = sc[a.I];
            }
            return f;
        };
        auto in_item = [&](int i) { return i < m << width_log && tile0 * 8 + (i & (width - 1)) < a.I; };
        const Factors mine = in_item(tid) ? factors(tid) : Factors{};
        auto run = [&](auto count) {
            constexpr int NT = decltype(count)::value;
            uint32_t tok[NT];   // offsets of the tokens' rows: half the registers of addresses
            float acc[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int col = min(j * 8 + g, m - 1);   // columns past the last token repeat it and are not stored
                tok[j] = (uint32_t)(r.token[row0 + col] * a.H * 2);
                acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
            }
            auto load = [&](TokenPart<W8, false>& t, int i, int c) {
                load_tokens<W8, false>(t, reinterpret_cast<const uint8_t*>(a.x) + tok[i % NT], c, i / NT,
                                       q * 16, k_bytes);
            };
            constexpr bool kAhead = NT == 1 && S::prefetch;
            TokenQueue<W8, false, TokenPart<W8, false>::kOfPiece * NT, S::early> queue, next;   // next: with one tile, the tokens of the next piece
            if (kAhead && rank < my_pieces) next.start([&](auto& t, int i) { load(t, i, rank); });
            for (int c = rank; c < my_pieces; c += share) {
                uint4 lo[2], hi[2];
                if constexpr (kAhead) {
                    queue = next;
                    if (c + share < pieces) next.start([&](auto& t, int i) { load(t, i, c + share); });
                } else {
                    queue.start([&](auto& t, int i) { load(t, i, c); });
                }
                ring.take(lo, hi);
                mma_piece<W8, false, NT, 1>(acc, lo, hi, [&](int i) {
                    return queue.take(i, [&](auto& t, int n) { load(t, n, c); });
                });
                __syncwarp();
                fetch();
            }
            float* part = sums + warp * NT * 8 * 16;   // [warp][column][16 rows]
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                part[(j * 8 + 2 * q) * 16 + g] = acc[j][0];
                part[(j * 8 + 2 * q + 1) * 16 + g] = acc[j][1];
                part[(j * 8 + 2 * q) * 16 + g + 8] = acc[j][2];
                part[(j * 8 + 2 * q + 1) * 16 + g + 8] = acc[j][3];
            }
            return NT * 8;
        };
        const int cols = with_tiles<MAXNT>(nt, run);
        __syncthreads();
        for (int i = tid; i < m << width_log; i += kThreads) {
            if (!in_item(i)) continue;
            const int col = i >> width_log, at = i & (width - 1), c = at & 7, channel = tile0 * 8 + at;
            const float* part = sums + (((at >> 3) << log) * cols + col) * 16 + c;
            float gate = 0.0f, up = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w < share) {
                    gate += part[w * cols * 16];
                    up += part[w * cols * 16 + 8];
                }
            }
            const Factors f = i == tid ? mine : factors(i);
            gate *= f.gate;
            const float h = gate / (1.0f + expf(-gate)) * (up * f.up) * f.weight;
            // value and remainder; past the largest bf16 the value is the truncated one, and an infinity has none
            uint32_t hi = pack_bf16x2_rn(h, 0.0f) & 0xffffu;
            if ((hi & 0x7fffu) == 0x7f80u) hi = __float_as_uint(h) >> 16;
            const float rest = (hi & 0x7fffu) == 0x7f80u ? 0.0f : h - bf16_bits_to_float(hi);
            uint16_t* dst = a.inner + (int64_t)(row0 + col) * 2 * a.I + channel;
            dst[0] = (uint16_t)hi;
            dst[a.I] = (uint16_t)pack_bf16x2_rn(rest, 0.0f);
        }
        if (kBuffers == 1) __syncthreads();
    }
    if (!ring.ok() && a.status) ep_set_status(a.status, EP_ERR_TIMEOUT);
}

// The CTAs of a cluster (or one) own `rows` <= 16 columns of the output at a time (tiles tile, tile +
// clusters, ...) for every token.  The pieces of all experts form one line, of which each warp takes an
// equal stretch; a CTA adds its warps' sums, then the CTAs' sums are added in rank order.
struct OutCursor {
    int tile, at, piece, expert;   // at: place in the line of pieces
    __device__ __forceinline__ void place(const Routing& r, int pieces) {
        piece = at % pieces;
        expert = r.expert[at / pieces];
    }
};

template <bool W8, int MAXNT>
__global__ void __launch_bounds__(kThreads, Sizes<W8, MAXNT>::ctas) few_out_kernel(const FewArgs a, int rows, int split, const __grid_constant__ CUtensorMap map_w) {
    extern __shared__ uint8_t dynamic[];
    __shared__ Routing r;
    using S = Sizes<W8, MAXNT>;
    __shared__ uint64_t bars[kWarps * S::depth];
    uint8_t* const slots = aligned_smem(dynamic);
    float* const sums = reinterpret_cast<float*>(slots + S::ring_bytes);   // [warp][token][16]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    if (tid == 0) prefetch_map(&map_w);
    for (int i = tid; i < kWarps * a.T * 16; i += kThreads) sums[i] = 0.0f;
    build_routing(r, a);
    const int k_bytes = a.I * (W8 ? 1 : 2), pieces = (k_bytes + 127) / 128;
    const int total = r.count * pieces, tiles = (a.H + rows - 1) / rows;
    const int first_tile = split > 1 ? (int)blockIdx.x / split : (int)blockIdx.x, step = split > 1 ? (int)gridDim.x / split : (int)gridDim.x;
    const int rank = (int)blockIdx.x - first_tile * split, part = rank * kWarps + warp, parts = split * kWarps;
    const int begin = (int)((uint32_t)(total * part) / (uint32_t)parts), end = (int)((uint32_t)(total * (part + 1)) / (uint32_t)parts);
    const uint32_t plane = (uint32_t)a.I * 2;
    typename S::Ring ring(slots, bars, warp, lane);
    OutCursor ahead;
    ahead.tile = begin < end ? first_tile : tiles;
    ahead.at = begin;
    if (ahead.tile < tiles) ahead.place(r, pieces);
    auto fetch = [&]() {
        if (ahead.tile >= tiles) return;
        ring.put(lane, 128 * rows, [&](uint8_t* slot, uint64_t* bar) {
            tma_load_3d(slot, &map_w, ahead.piece * 128, ahead.tile * rows, ahead.expert, bar);
        });
        ++ahead.piece;
        if (++ahead.at == end) {
            ahead.at = begin;
            ahead.tile += step;
            if (ahead.tile < tiles) ahead.place(r, pieces);
        } else if (ahead.piece == pieces) {
            ahead.place(r, pieces);
        }
    };
    // the weights do not depend on the first kernel: they are on their way while it ends
    for (int d = 0; d < S::depth; ++d) fetch();
    wait_for_previous();

    float* mine = sums + warp * a.T * 16;
    for (int tile = first_tile; tile < tiles; tile += step) {
        const int h0 = tile * rows;
        for (int at = begin; at < end;) {
            const int pos = at / pieces, first = at % pieces, last = min(pieces, first + end - at);
            const int e = r.expert[pos], row0 = r.base[pos], m = r.base[pos + 1] - row0;
            // count 0: up to four tokens, whose values and remainders share one tile of eight columns
            auto run = [&](auto count) {
                constexpr bool kFold = decltype(count)::value == 0;
                constexpr int NT = kFold ? 1 : decltype(count)::value, PLANES = kFold ? 1 : 2;
                uint32_t tok[NT];   // offsets, at most 64 tokens x 16 entries x 65536 x 4 bytes
                float acc[NT][4];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int col = kFold ? g & 3 : j * 8 + g;
                    tok[j] = (uint32_t)(row0 + min(col, m - 1)) * a.I * 4 + (kFold && g >= 4 ? plane : 0);
                    acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
                }
                constexpr int kSides = NT * PLANES;
                auto load = [&](TokenPart<W8, false>& t, int i, int c) {
                    const int side = i % kSides;
                    load_tokens<W8, false>(t, reinterpret_cast<const uint8_t*>(a.inner) + tok[side / PLANES] + side % PLANES * plane,
                                           c, i / kSides, q * 16, k_bytes);
                };
                constexpr bool kAhead = NT == 1 && S::prefetch;
                TokenQueue<W8, false, TokenPart<W8, false>::kOfPiece * kSides, S::early> queue, next;   // next: with one tile, the inner rows of the next piece
                if (kAhead) next.start([&](auto& t, int i) { load(t, i, first); });
                for (int c = first; c < last; ++c) {
                    uint4 lo[2], hi[2];
                    if constexpr (kAhead) {
                        queue = next;
                        if (c + 1 < last) next.start([&](auto& t, int i) { load(t, i, c + 1); });
                    } else {
                        queue.start([&](auto& t, int i) { load(t, i, c); });
                    }
                    ring.take(lo, hi);
                    mma_piece<W8, false, NT, PLANES>(acc, lo, hi, [&](int i) {
                        return queue.take(i, [&](auto& t, int n) { load(t, n, c); });
                    });
                    __syncwarp();
                    fetch();
                }
                if constexpr (kFold) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[0][i] += __shfl_xor_sync(0xffffffffu, acc[0][i], 2);
                }
                float sa = 1.0f, sb = 1.0f;
                if constexpr (W8) {
                    sa = a.w2_scales[(int64_t)e * a.H + min(h0 + g, a.H - 1)];
                    sb = a.w2_scales[(int64_t)e * a.H + min(h0 + g + 8, a.H - 1)];
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int col = j * 8 + 2 * q + c;
                        if (col < m) {
                            float* s = mine + r.token[row0 + col] * 16 + g;
                            s[0] += sa * acc[j][c];
                            s[8] += sb * acc[j][c + 2];
                        }
                    }
                }
                __syncwarp();
                return 0;
            };
            if (m <= 4) run(std::integral_constant<int, 0>{});
            else with_tiles<MAXNT>((m + 7) / 8, run);
            at += last - first;
        }
        __syncthreads();
        if (split > 1) {   // the CTA's sum to its first warp's place, for its peers
            for (int i = tid; i < a.T * 16; i += kThreads) {
                float s = sums[i];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    s += sums[w * a.T * 16 + i];
                    sums[w * a.T * 16 + i] = 0.0f;
                }
                sums[i] = s;
            }
            __syncwarp();
            cluster_sync();
        }
        for (int i = rank * kThreads + tid; i < a.T * 16; i += split * kThreads) {
            const int t = i >> 4, h = h0 + (i & 15);
            float s = 0.0f;
            if (split > 1) {
                for (int c = 0; c < split; ++c) s += load_of_peer(&sums[i], c);
            } else {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    s += sums[w * a.T * 16 + i];
                    sums[w * a.T * 16 + i] = 0.0f;
                }
            }
            if ((i & 15) >= rows || h >= a.H) continue;
            for (int k = 0; k < a.S; ++k) s += bf16_bits_to_float(a.shared[((int64_t)k * a.T + t) * a.H + h]);
            a.out[(int64_t)t * a.H + h] = (uint16_t)pack_bf16x2_rn(s, 0.0f);
        }
        if (split > 1) {
            __syncwarp();
            cluster_sync();   // the peers have read
            for (int i = tid; i < a.T * 16; i += kThreads) sums[i] = 0.0f;
        }
        __syncthreads();
    }
    if (!ring.ok() && a.status) ep_set_status(a.status, EP_ERR_TIMEOUT);
}

// Warps that share a tile of few_inner_kernel.  All eight keep the most CTAs busy where there are few
// tiles (one token on 8 of 128 experts, bf16: 39.2 us with 8, 41.8 with 4); with more, fewer barriers and
// longer stretches of k win (15 tokens over 256 experts of 4208 x 336, int8: 95 us with 4, 111 with 8;
// 64 tokens, bf16: 861 with 4, 887 with 8), and short rows of int8 weights are better off with two
// (32 tokens, 4096 x 1024: 305 us with 2, 311 with 4, 342 with 8; but 8 of 7168 x 1024 320, 244, 253).
template <bool W8>
int tile_share_log(int64_t tiles, int ctas, int pieces) {
    int share_log = 2;
    if (tiles <= 4 * (int64_t)ctas) share_log = 3;
    else if (W8 && pieces <= 32 && tiles >= 32 * (int64_t)ctas) share_log = 1;
    while (share_log > 0 && 1 << share_log > pieces) --share_log;
    return share_log;
}

// Tiles of few_out_kernel: their columns, 12 to 16, those that leave the last round of clusters fullest;
// and the CTAs of a cluster, up to three where there would be fewer tiles than SMs (8 tokens, 1584 columns,
// int8: 160 us with 1, 128 with 2, 127 with 3, 135 with 4; 1024 columns, bf16: 184, 141, 129, 148; but a line
// of 30 pieces 9.5, 11.9, 11.1).  From one tile an SM on, splitting costs more than it gives (2992 columns,
// 56.2 us for 57.2).
struct OutShape { int rows, split; };

OutShape out_shape(int H, int sms, int ctas, int64_t most_pieces) {
    OutShape best = {16, 1};
    const int least_tiles = (H + 15) / 16;
    if (least_tiles < sms && most_pieces >= 10 * kWarps) best.split = std::min(3, ctas / least_tiles);
    const int clusters = ctas / best.split;
    int64_t least = INT64_MAX;
    for (int rows = 16; rows >= 12; --rows) {
        const int tiles = (H + rows - 1) / rows;
        const int64_t time = (int64_t)((tiles + clusters - 1) / clusters) * (rows + 3);
        if (time < least) { least = time; best.rows = rows; }
    }
    return best;
}

template <bool W8, int MAXNT>
cudaError_t launch(const FewArgs& a, int sms, cudaStream_t st) {
    const int64_t entries = (int64_t)a.T * a.K, experts = entries < a.E ? entries : a.E, width = W8 ? 1 : 2;
    const int64_t inner_tiles = experts * (a.I / 8);
    using S = Sizes<W8, MAXNT>;
    // As many CTAs as fit, or fewer if that fills the rounds of tiles better (one token: 8 x 128 tiles are
    // 3.4 rounds of two CTAs an SM, but 2.2 of three).
    int per_sm = S::ctas;
    if (per_sm == 3 && (inner_tiles + 3 * sms - 1) / (3 * sms) * 3 > (inner_tiles + 2 * sms - 1) / (2 * sms) * 2) per_sm = 2;
    const int ctas = sms * per_sm;
    const int share_log = tile_share_log<W8>(inner_tiles, ctas, (int)((a.H * width + 127) / 128));
    const OutShape o = out_shape(a.H, sms, ctas, experts * ((a.I * width + 127) / 128));
    const int tiles = (a.H + o.rows - 1) / o.rows, clusters = ctas / o.split;
    CUtensorMap map13, map2;
    if (!make_pairs_map(&map13, a.w13, a.E, a.I, a.H * width, 8) || !make_experts_map(&map2, a.w2, a.E, a.H, a.I * width, o.rows))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> inner_done{0}, out_done{0};
    cudaError_t e = allow_smem(few_inner_kernel<W8, MAXNT>, S::inner_smem, inner_done);
    if (e == cudaSuccess) e = allow_smem(few_out_kernel<W8, MAXNT>, S::out_smem, out_done);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(few_inner_kernel<W8, MAXNT>, dim3((unsigned)(inner_tiles < ctas ? inner_tiles : ctas)), kThreads, S::inner_smem, st,
                          a, share_log, map13);
    if (e != cudaSuccess) return e;
    // The second kernel reads the routing and fetches its first weights while the first drains.  Both have waited
    // for what came before, so neither reads them before they are there.
    return launch_overlapped_clusters(few_out_kernel<W8, MAXNT>, o.split, dim3((unsigned)((tiles < clusters ? tiles : clusters) * o.split)), kThreads,
                             S::out_smem, st, a, o.rows, o.split, map2);
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

size_t workspace_bytes(int64_t T, int64_t K, int64_t I) { return (size_t)(T * K * I * 4); }

ep_status check_sizes(int32_t T, int32_t H, int32_t E, int32_t K, int32_t I) {
    if (T < 0 || H < 8 || H > 8192 || E < 1 || E > kMaxExperts || K < 1 || K > kMaxTopk || K > E)
        return EP_ERR_INVALID_ARG;
    if (I < 8 || I > 65536 || H % 8 != 0 || I % 8 != 0) return EP_ERR_INVALID_ARG;
    return T > kFewMaxTokens ? EP_ERR_UNSUPPORTED : EP_OK;
}

}  // namespace

// The number of tile columns is a template bound: with at most 8 or 16 tokens the
// accumulators of wider tiles would only cost registers, and so loads in flight.
cudaError_t launch_few_tokens(const FewArgs& a, bool w8, int sms, cudaStream_t st) {
    if (a.T <= 8) return w8 ? launch<true, 1>(a, sms, st) : launch<false, 1>(a, sms, st);
    if (a.T <= 16) return w8 ? launch<true, 2>(a, sms, st) : launch<false, 2>(a, sms, st);
    return w8 ? launch<true, 8>(a, sms, st) : launch<false, 8>(a, sms, st);
}

extern "C" ep_status ep_moe_few_tokens_workspace_size(int32_t num_tokens, int32_t hidden, int32_t num_experts,
                                                      int32_t topk, int32_t inner, size_t* bytes) {
    const ep_status s = check_sizes(num_tokens, hidden, num_experts, topk, inner);
    if (s != EP_OK) return s;
    if (!bytes) return EP_ERR_INVALID_ARG;
    *bytes = workspace_bytes(num_tokens, topk, inner);
    return EP_OK;
}

extern "C" ep_status ep_moe_few_tokens(const void* x, const int64_t* topk_idx, const float* topk_weights,
                                       int32_t num_tokens, int32_t hidden, int32_t num_experts, int32_t topk,
                                       int32_t inner, const void* w13, const float* w13_scales, const void* w2,
                                       const float* w2_scales, const void* shared, int32_t num_shared, void* out,
                                       void* workspace, size_t workspace_size, int32_t* status,
                                       ep_stream_t stream) {
    const ep_status s = check_sizes(num_tokens, hidden, num_experts, topk, inner);
    if (s != EP_OK) return s;
    if (!w13 || !w2 || !aligned(w13, 16) || !aligned(w2, 16)) return EP_ERR_INVALID_ARG;
    if ((w13_scales == nullptr) != (w2_scales == nullptr)) return EP_ERR_INVALID_ARG;
    const bool w8 = w13_scales != nullptr;
    if (w8 && (hidden % 16 != 0 || inner % 16 != 0 || !aligned(w13_scales, 4) || !aligned(w2_scales, 4)))
        return EP_ERR_INVALID_ARG;
    if (num_shared < 0 || num_shared > kMaxShared || (num_shared > 0 && (!shared || !aligned(shared, 2))))
        return EP_ERR_INVALID_ARG;
    if (status && !aligned(status, 4)) return EP_ERR_INVALID_ARG;
    if (num_tokens == 0) return EP_OK;
    if (!x || !aligned(x, 16) || !topk_idx || !aligned(topk_idx, 8) || !topk_weights || !aligned(topk_weights, 4) ||
        !out || !aligned(out, 2))
        return EP_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16) || workspace_size < workspace_bytes(num_tokens, topk, inner))
        return EP_ERR_INVALID_ARG;
    FewArgs a;
    a.x = (const uint16_t*)x;
    a.topk = topk_idx;
    a.topk_w = topk_weights;
    a.w13 = (const uint8_t*)w13;
    a.w13_scales = w13_scales;
    a.w2 = (const uint8_t*)w2;
    a.w2_scales = w2_scales;
    a.shared = (const uint16_t*)shared;
    a.out = (uint16_t*)out;
    a.inner = (uint16_t*)workspace;
    a.status = status;
    a.T = num_tokens; a.K = topk; a.E = num_experts; a.H = hidden; a.I = inner; a.S = num_shared;
    const int sms = ep_current_sms();
    if (sms <= 0) return EP_ERR_CUDA;
    return launch_few_tokens(a, w8, sms, (cudaStream_t)stream) == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}
