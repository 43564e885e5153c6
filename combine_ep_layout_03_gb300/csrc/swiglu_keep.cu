// swiglu_keep.cu -- the activation between an expert's two products, in training:
//   inner = weight * silu(g) * u   of rows [g, u], and g and u in 8 bits for the backward pass,
// and that pass, which has nothing but the 8 bits, the gradient of inner and the row's weight:
//   s = 1 / (1 + exp(-g)),  dg = weight dy u s (1 + g (1 - s)),  du = weight dy g s,
//   inner = weight g s u  (what the next product's weights' gradient reads),  dweight = sum dy g s u.
// Codes are e4m3 with a scale for each 128 columns, max / 448; they are the nearest ones of the real
// quotient (row_codes.cuh).  The weight is the routing weight of the row's token: multiplied in here, where
// all of a row is at hand in the backward pass, it makes the combine a plain sum, whose gradient is a
// dispatch.
//
// Both kernels read and write each value once.  Measured, 131072 rows of 2 x 1024: forward 183 us, 5.9 TB/s (0.87 of the copy
// bandwidth; issue slots are 0.73 busy, with the codes), backward 200 us, 6.7 TB/s (0.99).
#include "expert_ops.cuh"
#include "expert_tiles.cuh"
#include "row_codes.cuh"

namespace {

struct KeepArgs {
    const uint16_t* c;        // [rows][2I] bf16, gates then ups
    const float* weights;     // [rows], or null: 1
    const int32_t* used;      // rows that hold anything (device), or null: all
    uint16_t* inner;          // [rows][I] bf16
    uint8_t* codes;           // [rows][2I] e4m3
    float* scales;            // [rows][2I / 128]
    const uint16_t* dy;       // [rows][I] bf16: gradient of inner
    uint16_t* dc;             // [rows][2I] bf16
    float* dweights;          // [rows]
    int32_t rows, groups;     // groups: I / 128
};

constexpr int kThreads = 256;
constexpr int kUnits = kThreads / 16;   // 16 threads take 128 gates and their ups: 16 bytes a thread of each
constexpr int kEach = 2;                // such units a thread: loads in flight

__device__ __forceinline__ int rows_of(const KeepArgs& a) { return a.used ? min(max(*a.used, 0), a.rows) : a.rows; }

// Codes and scale of a thread's eight values of a group of 128, which the 16 threads of a half warp hold.
__device__ __forceinline__ uint2 keep_group(const f32x2 v[4], float* scale, bool first) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max_abs3(m, v[i]);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(__shfl_xor_sync(kFull, m, o)));
    const bool finite = m <= 3.402823466e38f;   // false of NaN too
    // m / 448, rounded: the quotient and its remainder's
    constexpr float kInv = 1.0f / 448.0f;
    const float q = __fmul_rn(m, kInv);
    if (first) *scale = finite ? __fmaf_rn(__fmaf_rn(q, -448.0f, m), kInv, q) : __uint_as_float(0x7fc00000u);
    return finite && m > 0.0f ? encode_ratio<M_FP8G_E4M3>(v, m) : make_uint2(0, 0);
}

// Five CTAs an SM: 183 us for 131072 rows of 2 x 1024, 193 after a flush of L2 (four 214; six, with one unit a thread, 208).
__global__ void __launch_bounds__(kThreads, 5) swiglu_keep_kernel(const KeepArgs a) {
    const int lane = threadIdx.x & 15;
    wait_for_previous();
    const int rows = rows_of(a);
    const uint32_t groups = (uint32_t)a.groups, unit0 = blockIdx.x * (kUnits * kEach) + (threadIdx.x >> 4);
    uint4 g[kEach], u[kEach];
    uint32_t row[kEach], group[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint32_t unit = unit0 + i * kUnits;
        row[i] = unit / groups;
        group[i] = unit - row[i] * groups;
        const uint16_t* at = a.c + (int64_t)row[i] * groups * 256 + group[i] * 128 + lane * 8;
        g[i] = u[i] = make_uint4(0, 0, 0, 0);
        if ((int)row[i] < rows) {
            g[i] = ld_nc_v4(at);
            u[i] = ld_nc_v4(at + groups * 128);
        }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        f32x2 gv[4], uv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            gv[j] = unpack2(word(g[i], j));
            uv[j] = unpack2(word(u[i], j));
        }
        const bool in = (int)row[i] < rows;
        float* scales = a.scales + (int64_t)row[i] * groups * 2 + group[i];
        const uint2 gc = keep_group(gv, scales, in && lane == 0);
        const uint2 uc = keep_group(uv, scales + groups, in && lane == 0);
        if (!in) continue;
        const float quarter = a.weights ? 0.25f * a.weights[row[i]] : 0.25f;
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float g0, g1, u0, u1;
            halves(gv[j], g0, g1);
            halves(uv[j], u0, u1);
            y[j] = pack_bf16x2_rn(swiglu(g0, u0, 1.0f, quarter), swiglu(g1, u1, 1.0f, quarter));
        }
        const int64_t at = (int64_t)row[i] * groups * 128 + group[i] * 128 + lane * 8;
        st_v4(a.inner + at, make_uint4(y[0], y[1], y[2], y[3]));
        uint8_t* codes = a.codes + (int64_t)row[i] * groups * 256 + group[i] * 128 + lane * 8;
        st_v2(codes, gc);
        st_v2(codes + groups * 128, uc);
    }
}

// The two e4m3 codes of a half word, times scale.
__device__ __forceinline__ void decode2(uint32_t codes, float scale, float& a, float& b) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(a), "=f"(b) : "r"(h));
    a *= scale;
    b *= scale;
}

__device__ __forceinline__ uint2 ld_nc_v2(const void* p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// LANES threads a row, eight gates and their ups each at a time: a warp, so that the weight's gradient is a sum within it;
// half a warp where a row has no more than 128 gates; a CTA where there are few rows, whose warps' sums are added in their
// order (9 rows of 2 x 2688: 7.9 us by warps).  Many
// resident warps, each with few loads in flight: 205 us for 131072 rows of 2 x 1024 after a flush of L2 (three CTAs an SM,
// which hold as many loads: 275; six 236).
template <int LANES>
__global__ void __launch_bounds__(kThreads, 5) swiglu_keep_grad_kernel(const KeepArgs a) {
    const int lane = threadIdx.x % LANES;
    wait_for_previous();
    const int64_t row = (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    const bool in = row < rows_of(a);
    if (LANES >= 32 && !in) return;   // (halves of a warp stay together for their sums)
    const int inner = a.groups * 128;
    const float weight = in && a.weights ? a.weights[row] : 1.0f;
    const uint8_t* codes = a.codes + row * inner * 2;
    const float* scales = a.scales + row * a.groups * 2;
    float sum = 0.0f;
#pragma unroll 1
    for (int col = in ? lane * 8 : inner; col < inner; col += LANES * 8) {
        const uint2 gc = ld_nc_v2(codes + col), uc = ld_nc_v2(codes + inner + col);
        const uint4 dv = ld_nc_v4(a.dy + row * inner + col);
        const float gs = scales[col >> 7], us = scales[a.groups + (col >> 7)];
        uint32_t dg[4], du[4], y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float g[2], u[2], d[2], ng[2], nu[2], ny[2];
            decode2((j < 2 ? gc.x : gc.y) >> (16 * (j & 1)), gs, g[0], g[1]);
            decode2((j < 2 ? uc.x : uc.y) >> (16 * (j & 1)), us, u[0], u[1]);
            halves(unpack2(word(dv, j)), d[0], d[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float e, r;
                // (as swiglu() has it: the reciprocal of a quarter of 1 + exp(-g))
                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmaf_rn(g[h], -1.4426950408889634f, -2.0f)));
                asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(0.25f + e));
                const float s = 0.25f * r, silu = g[h] * s, wd = weight * d[h];
                sum = __fmaf_rn(d[h], silu * u[h], sum);
                ny[h] = silu * (weight * u[h]);   // silu * u alone may pass the range
                nu[h] = wd * silu;
                ng[h] = wd * (u[h] * __fmaf_rn(silu, 1.0f - s, s));
            }
            dg[j] = pack_bf16x2_rn(ng[0], ng[1]);
            du[j] = pack_bf16x2_rn(nu[0], nu[1]);
            y[j] = pack_bf16x2_rn(ny[0], ny[1]);
        }
        uint16_t* dc = a.dc + row * inner * 2 + col;
        st_v4(dc, make_uint4(dg[0], dg[1], dg[2], dg[3]));
        st_v4(dc + inner, make_uint4(du[0], du[1], du[2], du[3]));
        if (a.inner) st_v4(a.inner + row * inner + col, make_uint4(y[0], y[1], y[2], y[3]));
    }
    if (!a.dweights) return;
#pragma unroll
    for (int o = (LANES < 32 ? LANES : 32) / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if constexpr (LANES > 32) {
        __shared__ float sums[LANES / 32];
        if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < LANES / 32; ++i) sum += sums[i];
    }
    if (lane == 0 && in) a.dweights[row] = sum;
}

template <int LANES>
cudaError_t launch_grad(const KeepArgs& a, cudaStream_t st) {
    const int64_t each = kThreads / LANES, blocks = (a.rows + each - 1) / each;
    return launch_overlapped(swiglu_keep_grad_kernel<LANES>, dim3((unsigned)blocks), kThreads, 0, st, a);
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

bool sizes_ok(int64_t rows, int32_t inner) {
    // (units of 128 gates: a grid covers them in 32s, so that the last one's number stays below 2^31 too)
    static_assert(kUnits * kEach == 32, "2^31 is a multiple of a CTA's units");
    return rows >= 0 && inner >= 128 && inner <= 65536 && inner % 128 == 0 && rows <= INT32_MAX / (inner / 128);
}

}  // namespace

extern "C" ep_status ep_swiglu_keep(const void* c, const float* row_weights, int64_t rows, int32_t inner_size,
                                    const int32_t* rows_used, void* inner, void* codes, float* scales, ep_stream_t stream) {
    if (!sizes_ok(rows, inner_size) || !aligned(row_weights, 4) || !aligned(rows_used, 4)) return EP_ERR_INVALID_ARG;
    if (rows == 0) return EP_OK;
    if (!c || !aligned(c, 16) || !inner || !aligned(inner, 16) || !codes || !aligned(codes, 16) || !scales || !aligned(scales, 4))
        return EP_ERR_INVALID_ARG;
    KeepArgs a{};
    a.c = (const uint16_t*)c;
    a.weights = row_weights;
    a.used = rows_used;
    a.inner = (uint16_t*)inner;
    a.codes = (uint8_t*)codes;
    a.scales = scales;
    a.rows = (int32_t)rows;
    a.groups = inner_size / 128;
    const int64_t units = rows * a.groups, blocks = (units + kUnits * kEach - 1) / (kUnits * kEach);
    return launch_overlapped(swiglu_keep_kernel, dim3((unsigned)blocks), kThreads, 0, (cudaStream_t)stream, a) == cudaSuccess
               ? EP_OK : EP_ERR_CUDA;
}

extern "C" ep_status ep_swiglu_keep_grad(const void* codes, const float* scales, const float* row_weights,
                                         const void* grad_inner, int64_t rows, int32_t inner_size, const int32_t* rows_used,
                                         void* grad_c, void* inner, float* grad_row_weights, ep_stream_t stream) {
    if (!sizes_ok(rows, inner_size) || !aligned(row_weights, 4) || !aligned(rows_used, 4) || !aligned(inner, 16) ||
        !aligned(grad_row_weights, 4))
        return EP_ERR_INVALID_ARG;
    if (rows == 0) return EP_OK;
    if (!codes || !aligned(codes, 16) || !scales || !aligned(scales, 4) || !grad_inner || !aligned(grad_inner, 16) || !grad_c ||
        !aligned(grad_c, 16))
        return EP_ERR_INVALID_ARG;
    KeepArgs a{};
    a.codes = (uint8_t*)const_cast<void*>(codes);
    a.scales = const_cast<float*>(scales);
    a.weights = row_weights;
    a.dy = (const uint16_t*)grad_inner;
    a.used = rows_used;
    a.dc = (uint16_t*)grad_c;
    a.inner = (uint16_t*)inner;
    a.dweights = grad_row_weights;
    a.rows = (int32_t)rows;
    a.groups = inner_size / 128;
    // a warp a row fills 152 SMs from 1216 rows on; up to that many, a row of more than two turns has a CTA
    const cudaError_t e = a.groups == 1 ? launch_grad<16>(a, (cudaStream_t)stream)
                          : rows <= 1216 && a.groups > 4 ? launch_grad<kThreads>(a, (cudaStream_t)stream)
                                                         : launch_grad<32>(a, (cudaStream_t)stream);
    return e == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}
