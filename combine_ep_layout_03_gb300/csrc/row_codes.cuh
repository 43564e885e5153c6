// row_codes.cuh -- what the kernels that read rows of bf16 and write 8-bit codes share: packed float32
// arithmetic, magnitudes, and the codes of a ratio.
#pragma once

#include "quant.cuh"

namespace {

// Two float32 values in a register pair, for the packed arithmetic of sm_100 and later: the
// kernels of rows have several operations for each byte, and issue slots run out before bandwidth does.
using f32x2 = unsigned long long;

__device__ __forceinline__ f32x2 pair(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void halves(f32x2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// The two bf16 of a word.
__device__ __forceinline__ f32x2 unpack2(uint32_t w) {
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// max(m, |a|, |b|), NaN when any is NaN
__device__ __forceinline__ float max_abs3(float m, f32x2 v) {
    float a, b, r;
    halves(v, a, b);
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

__device__ __forceinline__ uint4 ld_stream_v4(const void* p) {   // not .nc: h_out may be one of the inputs
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// Codes of 8 values t with largest magnitude m (finite, > 0) at TOP: the divisor is
// brought near 1 by a power of two (exact), so that t * top cannot overflow.  The quotient is corrected by its
// remainder, which an FMA gives exactly (Markstein).
template <int Q>
__device__ __forceinline__ uint2 encode_ratio(const f32x2 t[4], float m) {
    constexpr float top = QTraits<Q>::dmax;
    const int e = max((int)(__float_as_uint(m) >> 23) - 127, -110);
    // 2^-e: e = 127 gives the subnormal 2^-127
    const float p = e < 127 ? __uint_as_float((uint32_t)(127 - e) << 23) : 5.877471754111438e-39f;
    const float a = __fmul_rn(top, p), b = __fmul_rn(m, p), inv = __frcp_rn(b);
    const f32x2 a2 = pair(a, a), nb2 = pair(-b, -b), inv2 = pair(inv, inv);
    f32x2 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x2 n = mul2(t[i], a2);
        const f32x2 q0 = mul2(n, inv2);
        q[i] = fma2(fma2(q0, nb2, n), inv2, q0);
    }
    float f[8];
    if constexpr (Q == M_INT8) {
        // adding 1.5 * 2^23 rounds to nearest even and leaves the code in the low byte
        const f32x2 magic = pair(12582912.0f, 12582912.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) halves(add2(q[i], magic), f[2 * i], f[2 * i + 1]);
        return make_uint2(pack4_low_bytes(__float_as_int(f[0]), __float_as_int(f[1]), __float_as_int(f[2]), __float_as_int(f[3])),
                          pack4_low_bytes(__float_as_int(f[4]), __float_as_int(f[5]), __float_as_int(f[6]), __float_as_int(f[7])));
    } else {
        constexpr int C = QTraits<Q>::fp8;
#pragma unroll
        for (int i = 0; i < 4; ++i) halves(q[i], f[2 * i], f[2 * i + 1]);
        return make_uint2(cvt_fp8x2<C>(f[0], f[1]) | (cvt_fp8x2<C>(f[2], f[3]) << 16),
                          cvt_fp8x2<C>(f[4], f[5]) | (cvt_fp8x2<C>(f[6], f[7]) << 16));
    }
}

}  // namespace
