// matmul_skinny.cu -- the 8-bit integer product of expert rows for experts with few
// rows each, where reading the weights is the work:
//   c[r, n] = a_scales[r] * w_scales[e, n] * sum_k a[r, k] * w[e, n, k]
// An item is 16 weight rows (eight gates and their eight ups with swiglu) against up to
// 64 rows of one expert: the warps of a CTA share the item's k and add their parts in
// shared memory, in warp order.  The codes become bf16 on the way to the tensor cores,
// which is exact, and a product of two codes is exact in float32; sums stay exact up to
// 2^24 (1040 terms of the largest size, any number of ordinary ones).
#include "expert_ops.cuh"
#include "skinny.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTileRows = 64;

template <bool GLU, int NT>
__device__ __forceinline__ void matmul_item(const MatmulArgs& a, int e, int64_t row0, int m, int tile, float* red) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    const int outs = GLU ? a.N / 2 : a.N, ch0 = tile * (GLU ? 8 : 16);
    // rows past the last repeat it and are not stored
    const int n0 = min(ch0 + g, outs - 1), n1 = GLU ? n0 + outs : min(ch0 + g + 8, outs - 1);
    const uint8_t* w = a.w + (int64_t)e * a.N * a.K;
    const uint8_t* tok[NT];
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        tok[j] = a.a + (row0 + min(j * 8 + g, m - 1)) * a.K;
        acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
    }
    mma_pieces<true, true, NT, 1>(acc, w + (int64_t)n0 * a.K, w + (int64_t)n1 * a.K, tok, 0, warp, (a.K + 127) / 128,
                                  kWarps, q * 16, a.K);
    float* mine = red + warp * NT * 8 * 16;   // [warp][column][16 rows]
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        mine[(j * 8 + 2 * q) * 16 + g] = acc[j][0];
        mine[(j * 8 + 2 * q + 1) * 16 + g] = acc[j][1];
        mine[(j * 8 + 2 * q) * 16 + g + 8] = acc[j][2];
        mine[(j * 8 + 2 * q + 1) * 16 + g + 8] = acc[j][3];
    }
    __syncthreads();
    constexpr int per = GLU ? 8 : 16;
    for (int i = tid; i < m * per; i += kThreads) {
        const int col = i / per, c = i % per, ch = ch0 + c;
        if (ch >= outs) continue;
        float v = 0.0f, u = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            v += red[(k * NT * 8 + col) * 16 + c];
            if constexpr (GLU) u += red[(k * NT * 8 + col) * 16 + c + 8];
        }
        const int64_t row = row0 + col;
        const float sa = a.a_scales[row];
        const float* sw = a.w_scales + (int64_t)e * a.N + ch;
        v = v * sa * sw[0];
        if constexpr (GLU) v = v / (1.0f + expf(-v)) * (u * sa * sw[outs]);
        a.out[row * outs + ch] = (uint16_t)pack_bf16x2_rn(v, 0.0f);
    }
    __syncthreads();
}

template <bool GLU>
__global__ void __launch_bounds__(kThreads) matmul_skinny_kernel(const MatmulArgs a) {
    __shared__ Segments s;
    __shared__ float red[kWarps * kTileRows * 16];
    if (!load_segments<kThreads>(s, a, kTileRows)) return;
    const int channels = GLU ? 8 : 16, outs = GLU ? a.N / 2 : a.N;
    const int ctiles = (outs + channels - 1) / channels;
    const int64_t items = (int64_t)s.tile[a.E] * ctiles;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        // an expert's items are neighbours, its token tiles fastest: they read the same weights
        const int e = expert_of_tile(s, a.E, (int)(item / ctiles));
        const int tiles = s.tile[e + 1] - s.tile[e];
        const int local = (int)(item - (int64_t)s.tile[e] * ctiles);
        const int first = local % tiles * kTileRows, m = min(kTileRows, s.rows[e] - first);
        const int64_t row0 = (int64_t)s.base[e] + first;
        if (m <= 8) matmul_item<GLU, 1>(a, e, row0, m, local / tiles, red);
        else if (m <= 16) matmul_item<GLU, 2>(a, e, row0, m, local / tiles, red);
        else if (m <= 32) matmul_item<GLU, 4>(a, e, row0, m, local / tiles, red);
        else matmul_item<GLU, 8>(a, e, row0, m, local / tiles, red);
    }
}

#ifndef EP_MATMUL_TILE_ROWS
#define EP_MATMUL_TILE_ROWS 64
#endif

bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

}  // namespace

cudaError_t launch_matmul_skinny(const MatmulArgs& a, int sms, cudaStream_t st) {
    const int64_t ctiles = a.swiglu ? (a.N / 2 + 7) / 8 : (a.N + 15) / 16;
    const int64_t most_tiles = (a.rows + kTileRows - 1) / kTileRows + (a.E > 1 ? a.E : 0);
    const int64_t items = ctiles * most_tiles, most = (int64_t)sms * 8;
    const unsigned grid = (unsigned)(items < most ? items : most);
    if (a.swiglu) matmul_skinny_kernel<true><<<grid, kThreads, 0, st>>>(a);
    else matmul_skinny_kernel<false><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

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
    const bool tiles = rows > (int64_t)num_experts * EP_MATMUL_TILE_ROWS;
    const cudaError_t e = tiles ? launch_matmul_tiles(m, sms, (cudaStream_t)stream)
                                : launch_matmul_skinny(m, sms, (cudaStream_t)stream);
    return e == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}
