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
    uint8_t* data;             // [rows][H] codes
    uint8_t* scales;           // [rows][scale_bytes]
    int64_t x_stride, residual_stride, h_stride;
    int64_t rows;
    int32_t H, nvec, scale_bytes;
    float eps;
};

// Launchers return cudaGetLastError() after the launch.
cudaError_t launch_rms_norm_quant(const RowQuantArgs& a, int quant, int sms, cudaStream_t st);
cudaError_t launch_quant_rows(const RowQuantArgs& a, int quant, int sms, cudaStream_t st);

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
