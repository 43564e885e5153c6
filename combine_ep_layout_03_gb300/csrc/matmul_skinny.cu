// matmul_skinny.cu -- the products of expert rows for experts with few rows each, where reading the weights is the
// work: 8-bit integers, FP8 with scales for each block of 128, and bf16 (ep_expert_matmul and its two relatives).
//   c[r, n] = a_scales[r] * w_scales[e, n] * sum_k a[r, k] * w[e, n, k]      (8-bit integers; others likewise)
// An item is 16 weight rows (eight gates and their eight ups with swiglu) against up to
// 32 rows of one expert: the warps of a CTA share the item's k and add their parts in
// shared memory, in warp order.  Integer codes become bf16 on the way to the tensor cores,
// which is exact, and a product of two codes is exact in float32; sums stay exact up to
// 2^24 (1024 terms of the largest size, any number of ordinary ones).  A 128-byte piece of FP8 rows is a block: its
// sum is taken alone, scaled and added.
//
// Measured: 8 rows x 4096 x 4096 7.0 us (its floor, 17 MB, is 2.5 us); 32 rows 12.9 us.  FP8 6.4 and 10.9 us in a graph, bf16
// 7.1 (33 MB) and 11.3.  What bounds
// it is a warp's start, its first loads and its few pieces one after another; the host takes 5.1 us a call.
#include "expert_ops.cuh"
#include "skinny.cuh"
#include "tensor_maps.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTileRows = 32;
constexpr int kDepth = 4;                              // pieces in flight a warp
using Ring = WeightRing<kDepth>;
constexpr int kRingBytes = kWarps * Ring::kWarpBytes;
constexpr int kSums = kWarps * kTileRows * 16;         // [warp][column][16 rows]
constexpr int kSmem = 1024 + kRingBytes + 2 * kSums * (int)sizeof(float);

// Where an item lies: tiles of one expert are neighbours, its token tiles fastest (they read the same weights).
struct Item { int e, channel, first, m; };

__device__ __forceinline__ Item item_of(const Segments& s, const MatmulArgs& a, int ctiles, int64_t item) {
    Item t;
    t.e = expert_of_tile(s, a.E, (int)(item / ctiles));
    const int tiles = s.tile[t.e + 1] - s.tile[t.e];
    const int local = (int)(item - (int64_t)s.tile[t.e] * ctiles);
    t.first = local % tiles * kTileRows;
    t.channel = local / tiles;
    t.m = min(kTileRows, s.rows[t.e] - t.first);
    return t;
}

// What the rows and matrices hold.
enum Kind { INT8, FP8, BF16 };

template <Kind KIND, bool GLU>
__global__ void __launch_bounds__(kThreads, 2) matmul_skinny_kernel(const MatmulArgs a, const __grid_constant__ CUtensorMap map_w) {
    extern __shared__ uint8_t dynamic[];
    __shared__ uint64_t bars[kWarps * kDepth];
    uint8_t* const slots = dynamic + ((1024 - (smem_addr(dynamic) & 1023)) & 1023);
    __shared__ Segments s;
    float* const red = reinterpret_cast<float*>(slots + kRingBytes);   // two buffers in turn: a barrier an item
    if (threadIdx.x == 0) prefetch_map(&map_w);
    wait_for_previous();
    if (!load_segments<kThreads>(s, a, kTileRows)) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    constexpr int per = GLU ? 8 : 16;   // output channels of an item
    const int outs = GLU ? a.N / 2 : a.N, ctiles = (outs + per - 1) / per;
    const int row_bytes = KIND == BF16 ? 2 * a.K : a.K, pieces = (row_bytes + 127) / 128;
    const int64_t items = (int64_t)s.tile[a.E] * ctiles;

    Ring ring(slots, bars, warp, lane);
    int64_t ahead = warp < pieces ? (int64_t)blockIdx.x : items;
    int ahead_piece = warp;
    Item at{};
    if (ahead < items) at = item_of(s, a, ctiles, ahead);
    auto fetch = [&]() {
        if (ahead >= items) return;
        ring.put(lane, 2048, [&](uint8_t* slot, uint64_t* bar) {
            if (GLU) tma_load_4d(slot, &map_w, ahead_piece * 128, at.channel * per, 0, at.e, bar);
            else tma_load_3d(slot, &map_w, ahead_piece * 128, at.channel * per, at.e, bar);
        });
        ahead_piece += kWarps;
        if (ahead_piece >= pieces) {
            ahead_piece = warp;
            ahead += gridDim.x;
            if (ahead < items) at = item_of(s, a, ctiles, ahead);
        }
    };
    for (int d = 0; d < kDepth; ++d) fetch();

    int buffer = 0;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x, buffer ^= 1) {
        const Item t = item_of(s, a, ctiles, item);
        const int64_t row0 = (int64_t)s.base[t.e] + t.first;
        float* sums = red + buffer * kSums;
        // the scales of this thread's first result arrive meanwhile (FP8's change with every piece)
        struct Scales { float row, gate, up; };
        auto scales = [&](int i) {
            if constexpr (KIND != INT8) return Scales{1.0f, 1.0f, 1.0f};
            const float* sw = a.w_scales + (int64_t)t.e * a.N + min(t.channel * per + i % per, outs - 1);
            return Scales{a.a_scales[row0 + i / per], sw[0], GLU ? sw[outs] : 0.0f};
        };
        const Scales mine = tid < t.m * per ? scales(tid) : Scales{};
        auto run = [&](auto count) {
            constexpr int NT = decltype(count)::value;
            const uint8_t* tok[NT];
            float acc[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                tok[j] = a.a + (row0 + min(j * 8 + g, t.m - 1)) * row_bytes;   // columns past the last repeat it
                acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
            }
            constexpr bool kInt8 = KIND == INT8;
            using Part = TokenPart<kInt8, kInt8>;
            auto load = [&](Part& t, int i, int c) { load_tokens<kInt8, kInt8>(t, tok[i % NT], c, i / NT, q * 16, row_bytes); };
            TokenQueue<kInt8, kInt8, Part::kOfPiece * NT, 8> queue, next;   // next: with one tile, the tokens of the next piece
            const float* sa[KIND == FP8 ? 2 * NT : 1];   // of this lane's two columns of each tile
            const float* sw[2];                          // of rows g and g + 8 (with SwiGLU: gates and ups)
            if constexpr (KIND == FP8) {
#pragma unroll
                for (int j = 0; j < 2 * NT; ++j) sa[j] = a.a_scales + (row0 + min((j / 2) * 8 + 2 * q + (j & 1), t.m - 1)) * pieces;
                const int blocks = (outs + 127) / 128;
                sw[0] = a.w_scales + ((int64_t)t.e * (GLU ? 2 : 1) * blocks + (t.channel * per >> 7)) * pieces;
                sw[1] = sw[0] + (GLU ? (int64_t)blocks * pieces : 0);
            }
            if (NT == 1 && warp < pieces) next.start([&](auto& t, int i) { load(t, i, warp); });
            for (int c = warp; c < pieces; c += kWarps) {
                if constexpr (NT == 1) {
                    queue = next;
                    if (c + kWarps < pieces) next.start([&](auto& t, int i) { load(t, i, c + kWarps); });
                } else {
                    queue.start([&](auto& t, int i) { load(t, i, c); });
                }
                float row_scale[KIND == FP8 ? 2 * NT : 1], weight_scale[2];
                if constexpr (KIND == FP8) {
#pragma unroll
                    for (int j = 0; j < 2 * NT; ++j) row_scale[j] = sa[j][c];
                    weight_scale[0] = sw[0][c];
                    weight_scale[1] = sw[1][c];
                }
                uint4 lo[2], hi[2];
                ring.take(lo, hi);
                auto tokens = [&](int i) { return queue.take(i, [&](auto& t, int n) { load(t, n, c); }); };
                if constexpr (KIND == FP8) {
                    // a piece is a block: its sum is scaled and added to the blocks' before
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const Part t = tokens(j);
                        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            mma_e4m3(sum, lo[h].x, hi[h].x, lo[h].y, hi[h].y, t.v[h].x, t.v[h].y);
                            mma_e4m3(sum, lo[h].z, hi[h].z, lo[h].w, hi[h].w, t.v[h].z, t.v[h].w);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[j][i] = __fmaf_rn(sum[i], row_scale[2 * j + (i & 1)] * weight_scale[i >> 1], acc[j][i]);
                    }
                } else {
                    mma_piece<kInt8, kInt8, NT, 1>(acc, lo, hi, tokens);
                }
                __syncwarp();
                fetch();
            }
            float* part = sums + warp * NT * 8 * 16;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                part[(j * 8 + 2 * q) * 16 + g] = acc[j][0];
                part[(j * 8 + 2 * q + 1) * 16 + g] = acc[j][1];
                part[(j * 8 + 2 * q) * 16 + g + 8] = acc[j][2];
                part[(j * 8 + 2 * q + 1) * 16 + g + 8] = acc[j][3];
            }
            return NT * 8;
        };
        const int cols = with_tiles<4>((t.m + 7) / 8, run);
        __syncthreads();
        for (int i = tid; i < t.m * per; i += kThreads) {
            const int col = i / per, c = i % per, ch = t.channel * per + c;
            if (ch >= outs) continue;
            float v = 0.0f, u = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                v += sums[(k * cols + col) * 16 + c];
                if constexpr (GLU) u += sums[(k * cols + col) * 16 + c + 8];
            }
            const int64_t row = row0 + col;
            if constexpr (KIND == INT8) {
                const Scales f = i == tid ? mine : scales(i);
                v = v * f.row * f.gate;
                u = u * f.row * f.up;
            }
            if constexpr (GLU) v = v / (1.0f + expf(-v)) * u;
            a.out[row * outs + ch] = (uint16_t)pack_bf16x2_rn(v, 0.0f);
        }
    }
    if (!ring.ok() && a.status) ep_set_status(a.status, EP_ERR_TIMEOUT);
}

// Few enough rows and weights for the kernel above.  Its loop reads weights at about 3 TB/s for up to
// eight rows an expert and less for more, but on every SM and from the start; matmul_tiles.cu reads at
// 6 TB/s, starts later, and a round of its tiles takes as long as their k, however few they are.
// Measured, us (this kernel, that one): 8 rows x 4096 x 4096: 7.1, 15.1; 32 rows: 12.5, 15.2;
// 8 rows x 7168 x 4096: 10.8, 22.5; experts of 2048 x 1024: 16 of 8 rows 14.0, 11.1; 8 of 16 rows
// 10.5, 11.1; 8 of 32 rows 15.0, 11.1; 32 of 8 rows 27.2, 17.4; 16 of 8 rows, 1024 x 1400: 13.9, 13.4.
bool is_skinny(const MatmulArgs& a, int sms) {
    const int64_t experts = a.rows < a.E ? a.rows : a.E, rows = (a.rows + a.E - 1) / a.E;
    if (rows > 32) return false;
    const double rate[4] = {3.2, 2.7, 2.2, 1.7};   // bytes of weights a picosecond, by tiles of eight rows
    const double here = 4.5 + 1e-6 * (double)(experts * a.N * a.K) / rate[(rows - 1) / 8];
    const int64_t tiles = experts * (((a.swiglu ? a.N / 2 : a.N) + (a.swiglu ? 127 : 255)) / (a.swiglu ? 128 : 256));
    const int64_t rounds = (tiles + sms / 2 - 1) / (sms / 2);
    return here <= 6.0 + (double)rounds * a.K / 420.0;
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

template <Kind KIND>
cudaError_t launch(const MatmulArgs& a, int sms, cudaStream_t st) {
    const int64_t ctiles = a.swiglu ? (a.N / 2 + 7) / 8 : (a.N + 15) / 16, row_bytes = KIND == BF16 ? 2 * (int64_t)a.K : a.K;
    const int64_t most_tiles = (a.rows + kTileRows - 1) / kTileRows + (a.E > 1 ? a.E : 0);
    const int64_t items = ctiles * most_tiles;
    const unsigned grid = (unsigned)(items < 2 * sms ? items : 2 * sms);
    auto kernel = a.swiglu ? matmul_skinny_kernel<KIND, true> : matmul_skinny_kernel<KIND, false>;
    CUtensorMap map_w;
    if (!(a.swiglu ? make_pairs_map(&map_w, a.w, a.E, a.N / 2, row_bytes, 8) : make_experts_map(&map_w, a.w, a.E, a.N, row_bytes, 16)))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done[2];
    const cudaError_t e = allow_smem(kernel, kSmem, done[a.swiglu]);
    if (e != cudaSuccess) return e;
    return launch_overlapped(kernel, dim3(grid), kThreads, kSmem, st, a, map_w);
}

}  // namespace

cudaError_t launch_matmul_skinny(const MatmulArgs& a, int sms, cudaStream_t st) { return launch<INT8>(a, sms, st); }
cudaError_t launch_matmul_skinny_fp8(const MatmulArgs& a, int sms, cudaStream_t st) { return launch<FP8>(a, sms, st); }
cudaError_t launch_matmul_skinny_bf16(const MatmulArgs& a, int sms, cudaStream_t st) { return launch<BF16>(a, sms, st); }

extern "C" ep_status ep_expert_matmul(const void* a, const float* a_scales, int64_t rows, int32_t k, const void* w,
                                      const float* w_scales, int32_t n, int32_t num_experts,
                                      const int32_t* expert_base, int32_t swiglu, void* out, int32_t* status,
                                      ep_stream_t stream) {
    if (rows < 0 || rows >= INT32_MAX || k < 16 || k > 65536 || k % 16 != 0 || n < 1 || n > 65536)
        return EP_ERR_INVALID_ARG;
    if (swiglu != 0 && swiglu != 1) return EP_ERR_INVALID_ARG;
    if (swiglu && n % 2 != 0) return EP_ERR_INVALID_ARG;
    if (num_experts < 1 || num_experts > kMaxExperts || (num_experts > 1 && !expert_base)) return EP_ERR_INVALID_ARG;
    if (!aligned(expert_base, 4) || !aligned(status, 4)) return EP_ERR_INVALID_ARG;
    if (!w || !aligned(w, 16) || !w_scales || !aligned(w_scales, 4)) return EP_ERR_INVALID_ARG;
    if (rows == 0) return EP_OK;
    if (!a || !aligned(a, 16) || !a_scales || !aligned(a_scales, 4) || !out || !aligned(out, 2))
        return EP_ERR_INVALID_ARG;
    MatmulArgs m;
    m.a = (const uint8_t*)a;
    m.a_scales = a_scales;
    m.w = (const uint8_t*)w;
    m.w_scales = w_scales;
    m.expert_base = expert_base;
    m.out = (uint16_t*)out;
    m.status = status;
    m.rows = rows;
    m.K = k; m.N = n; m.E = num_experts;
    m.swiglu = swiglu;
    const int sms = ep_current_sms();
    if (sms <= 0) return EP_ERR_CUDA;
    const cudaError_t e = is_skinny(m, sms) ? launch_matmul_skinny(m, sms, (cudaStream_t)stream)
                                       : launch_matmul_tiles(m, sms, (cudaStream_t)stream);
    return e == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}
