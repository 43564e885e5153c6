// expert_ops.cuh -- argument blocks and launchers of the expert-layer operators
// (8-bit rows, integer expert products, the few-token layer).  Internal; not part
// of the ABI.
#pragma once

#include "ep_internal.cuh"

struct RowQuantArgs {
    const uint16_t* x;         // [rows] rows of H bf16, x_stride elements apart
    const uint16_t* residual;  // as x, or null
    const uint16_t* gamma;     // [H] bf16 (normalised form only)
    uint16_t* h_out;           // [rows] rows of H bf16, h_stride apart, or null
    uint16_t* y_out;           // [rows][H] bf16 of y, or null
    uint8_t* data;             // [rows][H] codes
    uint8_t* scales;           // [rows][scale_bytes]
    int64_t x_stride, residual_stride, h_stride;
    int64_t rows;
    int32_t H, nvec, scale_bytes;
    float eps, inv_n;          // inv_n: 1 / H
};

// Launchers return cudaGetLastError() after the launch.
cudaError_t launch_rms_norm_quant(const RowQuantArgs& a, int quant, int sms, cudaStream_t st);
cudaError_t launch_quant_rows(const RowQuantArgs& a, int quant, int sms, cudaStream_t st);

// Launches a kernel that may be set up while the one before it in the stream ends (programmatic
// dependent launch).  It must call wait_for_previous() before it touches global memory.  cluster: CTAs of
// a cluster, a divisor of the grid (1: none but what the kernel declares).
template <class... P, class... A>
cudaError_t launch_overlapped_clusters(void (*kernel)(P...), int cluster, dim3 grid, int threads, size_t smem,
                                       cudaStream_t st, A&&... args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <class... P, class... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A&&... args) {
    return launch_overlapped_clusters(kernel, 1, grid, threads, smem, st, args...);
}

// Everything that earlier kernels of the stream wrote is visible after this.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// SMs of the current device (0 when the query fails).
inline int ep_current_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms;
}

constexpr int kFewMaxTokens = 64;   // tokens of one ep_moe_few_tokens call

struct FewArgs {
    const uint16_t* x;         // [T][H] bf16
    const int64_t* topk;       // [T][K]
    const float* topk_w;       // [T][K]
    const uint8_t* w13;        // [E][2I][H] bf16 or int8: I gate rows, then I up rows
    const float* w13_scales;   // [E][2I], int8 only
    const uint8_t* w2;         // [E][H][I]
    const float* w2_scales;    // [E][H], int8 only
    const uint16_t* shared;    // [S][T][H] bf16 or null
    uint16_t* out;             // [T][H]
    uint16_t* inner;           // workspace: [T * K][2][I], the weighted inner rows as bf16 pairs (value, remainder)
    int32_t* status;           // or null
    int32_t T, K, E, H, I, S;
};

cudaError_t launch_few_tokens(const FewArgs& a, bool int8_weights, int sms, cudaStream_t st);

struct MatmulArgs {
    const uint8_t* a;          // [rows][K] int8 token rows
    const float* a_scales;     // [rows]
    const uint8_t* w;          // [E][N][K] int8
    const float* w_scales;     // [E][N]
    const int32_t* expert_base;  // [E + 1] first row of each expert, or null: all rows belong to one matrix
    uint16_t* out;             // [rows][N] bf16, or [rows][N / 2] with swiglu
    int32_t* status;           // or null
    int64_t rows;              // rows of a and out
    int32_t K, N, E;
    int32_t swiglu;
};

cudaError_t launch_matmul_skinny(const MatmulArgs& a, int sms, cudaStream_t st);

// The segments of a grouped product in shared memory: first row and first token tile of each
// expert.  Device data is not trusted with addresses: the segments have to ascend inside the buffers'
// rows, or none is worked on.  (Each inside but overlapping, their tiles could pass 32 bits together.)
struct Segments {
    int32_t base[kMaxExperts];
    int32_t rows[kMaxExperts];
    int32_t tile[kMaxExperts + 1];   // first token tile of each expert; [E]: all tiles
    int32_t warp_sum[32];
};

// All threads of a CTA of NT threads, kMaxExperts <= 2 NT.  False: the segments do not ascend from a first one
// >= 0 (EP_ERR_INVALID_ARG is set) or need more rows than there are (EP_ERR_CAPACITY), and nothing may be written.
template <int NT>
__device__ __forceinline__ bool load_segments(Segments& s, const MatmulArgs& a, int tile_rows) {
    static_assert(kMaxExperts <= 2 * NT, "a thread holds two experts");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int tiles[2] = {0, 0};
    bool ascend = true, fits = true;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = 2 * tid + h;
        if (e >= a.E) continue;
        int64_t b = 0, end = a.rows;
        if (a.expert_base) {
            b = a.expert_base[e];
            end = a.expert_base[e + 1];
            ascend = ascend && b >= 0 && b <= end;
            fits = fits && end <= a.rows;
        }
        s.base[e] = (int32_t)b;
        s.rows[e] = (int32_t)(end - b);
        tiles[h] = (int)((end - b + tile_rows - 1) / tile_rows);
    }
    int sum = tiles[0] + tiles[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += n;
    }
    if (lane == 31) s.warp_sum[warp] = sum;
    if (!__syncthreads_and(ascend && fits)) {
        ascend = __syncthreads_and(ascend);
        if (tid == 0 && a.status) ep_set_status(a.status, ascend ? EP_ERR_CAPACITY : EP_ERR_INVALID_ARG);
        return false;
    }
    for (int w = 0; w < warp; ++w) sum += s.warp_sum[w];
    const int at = sum - tiles[0] - tiles[1];
    if (2 * tid < a.E) s.tile[2 * tid] = at;
    if (2 * tid + 1 < a.E) s.tile[2 * tid + 1] = at + tiles[0];
    if (tid == NT - 1) s.tile[a.E] = sum;
    __syncthreads();
    return true;
}

// The expert that token tile t belongs to (tiles of empty experts do not exist).
__device__ __forceinline__ int expert_of_tile(const Segments& s, int E, int t) {
    int lo = 0, hi = E;   // last e with tile[e] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.tile[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The tensor-core form for experts with many rows (matmul_tiles.cu).
cudaError_t launch_matmul_tiles(const MatmulArgs& a, int sms, cudaStream_t st);
