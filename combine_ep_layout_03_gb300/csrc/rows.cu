// rows.cu -- rows of 8-bit codes with scales from bf16 rows: after a residual add
// and RMSNorm (rms_norm_quant_kernel), or as they are (quant_rows_kernel).  Either
// leaves rows that ep_dispatch_ex moves unchanged (EP_DISPATCH_PRE_ENCODED), so a
// token is encoded once however many experts it goes to.
//
// The mathematics of the normalised form, for one row:
//   h = bf16(x + residual),  t = h * gamma,  r = 1 / sqrt(mean(h^2) + eps),  y = t * r
//   per token / per 128 columns:  m = max|t|,  code = nearest(t * top / m),  scale = m * r / top
//   MX blocks of 32 columns:      2^s, s = floor(log2(max|t| * r)) - emax,  code = nearest(y * 2^-s)
// The root cancels in the codes of the first kind, so the maximum does not wait for
// it: one pass over the row, one barrier.  t is exact in float32 (8 x 8 significant
// bits), and so is t * top (top has three or seven); the quotient is corrected once
// with an FMA remainder, which makes every tie between two codes an exact value and
// leaves no non-tie on one: the codes are the formula's, not a float32 neighbour's.
// (Distance of a non-tie from a tie: at least 2^-24 of it, from the widths 23 and 16
// bits of numerator and divisor; the corrected quotient is closer than that.)
// h is rounded to bf16 before the norm: that rounded row is what the residual stream
// stores, and normalising exactly it makes the result the same whether the addition
// was fused or not.
//
// Scales are float32 products of a float32 root, off by a few 2^-24 (41 at most; 5e-8 in the norm).
//
// Measured, against the copy bandwidth: 65536 x 4096 int8 with a residual 269 us, 1.03 (and with y_out 344 us,
// 1.03); without one 144 us, 0.82; 32768 x 7168 MXFP8 without one 158 us, 0.67 (with: 240 us, 1.03); 1237 x 7168
// in groups, with one, 14.2 us, 0.65 (8.1 rows an SM).  With a residual the bytes bound it.  Without one it is
// instructions: issue slots are 0.71 busy (int8) and 0.68 (MXFP8, whose ALU pipe is 0.62), DRAM 0.65 and 0.52;
// what is missing to full is a row's loads, sum and barrier one after another, with 0.40 to 0.45 of the warps
// that an SM holds.  More or fewer resident rows make it slower.
#include <type_traits>

#include "expert_ops.cuh"
#include "quant.cuh"
#include "row_codes.cuh"

namespace {

// Sum of float32 values with its rounding error carried along (Knuth's two-term sum, and the compensated summation
// of Ogita, Rump and Oishi): about 48 bits.
struct Sum2 { float hi, lo; };

__device__ __forceinline__ void sum2_add(Sum2& s, float hi, float lo) {
    const float t = __fadd_rn(s.hi, hi);
    const float b = __fsub_rn(t, s.hi);
    const float e = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, b)), __fsub_rn(hi, b));
    s.hi = t;
    s.lo = __fadd_rn(s.lo, __fadd_rn(e, lo));
}

// What is missing from r, an approximation of 1 / sqrt(s / n + eps): r (n - r^2 s - r^2 n eps) / 2n, with the
// errors of the products taken along.  0 where a product leaves the range.
__device__ __forceinline__ float rsqrt_remainder(float r, float s, float n, float inv_n, float eps) {
    const float p = __fmul_rn(n, eps);
    const float q = __fmul_rn(r, r), q_lo = __fmaf_rn(r, r, -q);
    const float a = __fmul_rn(s, q), a_lo = __fmaf_rn(s, q, -a);
    const float b = __fmul_rn(p, q), b_lo = __fmaf_rn(p, q, -b);
    const float left = __fsub_rn(__fsub_rn(__fsub_rn(n, a), b), __fmaf_rn(__fadd_rn(s, p), q_lo, __fadd_rn(a_lo, b_lo)));
    const float lo = __fmul_rn(__fmul_rn(r, 0.5f * inv_n), left);
    return fabsf(lo) <= r * 0x1p-20f ? lo : 0.0f;
}

// bf16(x + residual) of eight columns
__device__ __forceinline__ uint4 add_rows(const uint4& x, const uint4& residual) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f0, f1;
        halves(add2(unpack2(word(x, i)), unpack2(word(residual, i))), f0, f1);
        h[i] = pack_bf16x2_rn(f0, f1);
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

__device__ __forceinline__ bool finite_bits(uint32_t magnitude) { return magnitude < 0x7f800000u; }

// h of eight columns of a row once more (no register keeps it past the first pass): from h_out, which may have
// taken an input's place, or from the inputs.  The thread that wrote them there reads them.
__device__ __forceinline__ uint4 row_again(const RowQuantArgs& a, int64_t row, int vi) {
    if (a.h_out) return ld_stream_v4(a.h_out + row * a.h_stride + 8 * vi);
    const uint4 x = ld_stream_v4(a.x + row * a.x_stride + 8 * vi);
    return a.residual ? add_rows(x, ld_stream_v4(a.residual + row * a.residual_stride + 8 * vi)) : x;
}

// v in 32 bits for a conversion to 8 or 16 that follows: what the first rounding drops is kept in the last bit,
// so that the second sees no tie where there is none.
__device__ __forceinline__ float sticky(double v) {
    const float f = __double2float_rz(v);
    return (double)f == v ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// A row whose squares leave the range of float32 (values from 2^57 on; or, with an eps below 2^-100, values whose
// mean square is below that too), or that is not finite: all of it in 64 bits, one vector of eight columns at a
// time.  Such rows are rare; what counts is that the others' registers stay as they are (32768 x 7168 MXFP8: 155 us
// without this code in the kernel, 158 with it inlined, where nothing else lives past it, 163 with it as a call,
// 174 as a second pass over values rescaled by a power of two).
template <int Q>
__device__ __forceinline__ void wide_row(const RowQuantArgs& a, int64_t row) {
    using TR = QTraits<Q>;
    using u64 = unsigned long long;
    __shared__ double s_sum[32];
    __shared__ u64 s_max[32];
    const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = nt >> 5;
    auto load = [&](int vi, float h[8], double t[8]) {
        float g[8];
        unpack8(vi < a.nvec ? row_again(a, row, vi) : make_uint4(0, 0, 0, 0), h);
        unpack8(vi < a.nvec ? __ldg(reinterpret_cast<const uint4*>(a.gamma) + vi) : make_uint4(0, 0, 0, 0), g);
        u64 m = 0;   // bits of max|t|, NaN above all
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t[i] = (double)h[i] * (double)g[i];
            m = max(m, (u64)__double_as_longlong(fabs(t[i])));
        }
        return m;
    };
    float h[8];
    double t[8], s = 0.0;
    u64 m = 0;
    for (int vi = tid; vi < a.nvec; vi += nt) {
        m = max(m, load(vi, h, t));
#pragma unroll
        for (int i = 0; i < 8; ++i) s += (double)h[i] * (double)h[i];
    }
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(kFull, s, o);
        m = max(m, __shfl_xor_sync(kFull, m, o));
    }
    if (lane == 0) { s_sum[warp] = s; s_max[warp] = m; }
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < nwarps; ++w) { s += s_sum[w]; m = max(m, s_max[w]); }
    const double n = a.H, mean = s / n + (double)a.eps, r = mean == 0.0 ? 0.0 : 1.0 / sqrt(mean);   // zeros and eps 0: y = 0
    const u64 inf = 0x7ff0000000000000ull;
    const bool row_ok = (u64)__double_as_longlong(s) < inf;
    for (int first = 0; first < a.nvec; first += nt) {
        const int vi = first + tid;
        u64 bm = load(vi, h, t);
        if constexpr (TR::token) bm = m;
        else   // consecutive lanes hold a group or block
            for (int o = 1; o < (TR::group ? 16 : 4); o <<= 1) bm = max(bm, __shfl_xor_sync(kFull, bm, o));
        if (vi >= a.nvec) continue;
        if (a.y_out) {
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = pack_bf16x2_rn(sticky(t[2 * i] * r), sticky(t[2 * i + 1] * r));
            st_v4(a.y_out + row * a.H + 8 * vi, make_uint4(y[0], y[1], y[2], y[3]));
        }
        const bool ok = row_ok && bm < inf;
        const double mf = __longlong_as_double((long long)bm);
        int se = -127;
        if constexpr (TR::mx) {
            if (ok && bm) {   // floor(log2(m r)): m^2 n >= 4^k (s + n eps) tells a power of two from what is just below
                int k = ilogb(mf * r);
                const double lhs = mf * mf * n, rhs = ldexp(s + n * (double)a.eps, 2 * k);
                if (lhs < rhs) --k;
                else if (lhs >= 4.0 * rhs) ++k;
                se = min(max(k - TR::emax, -127), 127);
            }
        }
        uint32_t c[2] = {0, 0};
        if (ok && bm) {
            const double up = TR::mx ? r * ldexp(1.0, -se) : 0.0;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const double q0 = TR::mx ? t[i] * up : t[i] * (double)TR::dmax / mf;
                const double q1 = TR::mx ? t[i + 1] * up : t[i + 1] * (double)TR::dmax / mf;
                uint32_t two;
                if constexpr (Q == M_INT8)
                    two = ((uint32_t)__double2int_rn(q0) & 0xffu) | (((uint32_t)__double2int_rn(q1) & 0xffu) << 8);
                else
                    two = cvt_fp8x2<TR::mx ? Q : TR::fp8>(sticky(q0), sticky(q1));
                c[i >> 2] |= two << (16 * ((i >> 1) & 1));
            }
        }
        st_v2(a.data + row * a.H + 8 * vi, make_uint2(c[0], c[1]));
        if constexpr (TR::mx) {
            if ((vi & 3) == 0) a.scales[row * a.scale_bytes + (vi >> 2)] = (uint8_t)(!ok ? 255 : bm ? se + 127 : 0);
        } else if (TR::group ? (vi & 15) == 0 : vi == 0) {
            reinterpret_cast<float*>(a.scales + row * a.scale_bytes)[TR::group ? vi >> 4 : 0] =
                !ok ? __uint_as_float(0x7fc00000u) : bm ? (float)(mf * r / (double)TR::dmax) : 0.0f;
        }
    }
}

// One CTA per row; thread t holds the 16-byte vectors u * blockDim + t of the row in
// registers between the barrier and the stores.
template <int Q, int VPT>
__global__ void __launch_bounds__(VPT == 4 ? 256 : 1024, VPT == 4 ? 4 : 1) rms_norm_quant_kernel(const RowQuantArgs a) {
    using TR = QTraits<Q>;
    __shared__ float2 s_sum[32];
    __shared__ uint32_t s_max[32];
    const int nt = blockDim.x, tid = threadIdx.x, warp = tid >> 5, nwarps = nt >> 5;
    const int64_t row = blockIdx.x;
    const uint16_t* x = a.x + row * a.x_stride;
    const uint16_t* res = a.residual ? a.residual + row * a.residual_stride : nullptr;
    wait_for_previous();

    uint4 v[VPT], g[VPT];
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int vi = u * nt + tid;
        v[u] = vi < a.nvec ? ld_stream_v4(x + 8 * vi) : make_uint4(0, 0, 0, 0);
    }
    if (res) {
        uint4 w[VPT];
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int vi = u * nt + tid;
            w[u] = vi < a.nvec ? ld_stream_v4(res + 8 * vi) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < VPT; ++u) v[u] = add_rows(v[u], w[u]);
    }
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int vi = u * nt + tid;
        g[u] = vi < a.nvec ? __ldg(reinterpret_cast<const uint4*>(a.gamma) + vi) : make_uint4(0, 0, 0, 0);
    }
    if (a.h_out) {
        uint16_t* h = a.h_out + row * a.h_stride;
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int vi = u * nt + tid;
            if (vi < a.nvec) st_v4(h + 8 * vi, v[u]);
        }
    }

    // the sum of squares, and max|t|: a maximum that keeps NaN, whose bits lie above every number's
    f32x2 t[VPT][4], s2 = pair(0.0f, 0.0f);
    uint32_t m = 0, gm[VPT];
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        float mu = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 h = unpack2(word(v[u], i));
            s2 = fma2(h, h, s2);
            t[u][i] = mul2(h, unpack2(word(g[u], i)));
            mu = max_abs3(mu, t[u][i]);
        }
        gm[u] = __float_as_uint(mu);
        m = max(m, gm[u]);
    }
    float s0, s1;
    halves(s2, s0, s1);
    float s = __fadd_rn(s0, s1);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(kFull, s, o));
    if constexpr (TR::token) m = __reduce_max_sync(kFull, m);
    if ((tid & 31) == 0) {
        s_sum[warp].x = s;
        if constexpr (TR::token) s_max[warp] = m;
    }
    __syncthreads();
    const int from = tid & 31;   // a lane for each warp's sum
    s = from < nwarps ? s_sum[from].x : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(kFull, s, o));
    if constexpr (TR::token) m = __reduce_max_sync(kFull, from < nwarps ? s_max[from] : 0u);
    const float n = (float)a.H, mean = __fmaf_rn(s, a.inv_n, a.eps);
    // from 2^-100 up to infinity, and not NaN; the same answer in every thread, as the sum is
    constexpr uint32_t least = 27u << 23, beyond = 0x7f800000u;
    if (__builtin_expect(__float_as_uint(mean) - least >= beyond - least, 0)) {
        wide_row<Q>(a, row);
        return;
    }
    const float rstd = rsqrtf(mean);
    const float nan = __uint_as_float(0x7fc00000u);
    uint8_t* data = a.data + row * a.H;
    if (a.y_out) {
        const f32x2 r2 = pair(rstd, rstd);
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int vi = u * nt + tid;
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y0, y1;
                halves(mul2(t[u][i], r2), y0, y1);
                y[i] = pack_bf16x2_rn(y0, y1);
            }
            if (vi < a.nvec) st_v4(a.y_out + row * a.H + 8 * vi, make_uint4(y[0], y[1], y[2], y[3]));
        }
    }

    if constexpr (TR::token) {
        const float mf = __uint_as_float(m);
        const bool ok = finite_bits(m);
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int vi = u * nt + tid;
            if (vi < a.nvec) st_v2(data + 8 * vi, ok && m ? encode_ratio<Q>(t[u], mf) : make_uint2(0, 0));
        }
        if (tid == 0)
            reinterpret_cast<float*>(a.scales)[row] =
                !ok ? nan : m ? __fmul_rn(__fmul_rn(mf, rstd), 1.0f / TR::dmax) : 0.0f;
    } else if constexpr (TR::group) {
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int vi = u * nt + tid;
            uint32_t gmax = gm[u];   // 16 consecutive lanes hold a group
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) gmax = max(gmax, __shfl_xor_sync(kFull, gmax, o));
            const float mf = __uint_as_float(gmax);
            const bool ok = finite_bits(gmax);
            if (vi < a.nvec) {
                st_v2(data + 8 * vi, ok && gmax ? encode_ratio<Q>(t[u], mf) : make_uint2(0, 0));
                if ((vi & 15) == 0)
                    reinterpret_cast<float*>(a.scales + row * a.scale_bytes)[vi >> 4] =
                        !ok ? nan : gmax ? __fmul_rn(__fmul_rn(mf, rstd), 1.0f / TR::dmax) : 0.0f;
            }
        }
    } else {
        // The block's exponent is that of max|t| * r.  Within 2^-17 of a power of two the float32
        // product may lie on the wrong side of it (the sum, with 32 + 11 additions, is off by less than 2^-18): then the CTA
        // takes the sum again with its errors carried along, and m * r >= 2^k is decided as
        // m^2 H >= 4^k (sum + H eps) in 64 bits.  A row in some hundreds comes to this.
        uint32_t bm[VPT];
        int ex[VPT];
        bool near[VPT], any = false;
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            bm[u] = gm[u];   // 4 consecutive lanes hold a block
            bm[u] = max(bm[u], __shfl_xor_sync(kFull, bm[u], 1));
            bm[u] = max(bm[u], __shfl_xor_sync(kFull, bm[u], 2));
            const uint32_t p = __float_as_uint(__fmul_rn(__uint_as_float(bm[u]), rstd));
            const uint32_t frac = p & 0x7fffffu;
            ex[u] = (p >> 23) == 0 ? -255 : (int)(p >> 23) - 127;
            near[u] = finite_bits(bm[u]) && bm[u] && (frac < 64u || frac > 0x7fffffu - 64u) && ex[u] > -120 && ex[u] < 128;
            any = any || near[u];
        }
        if (__syncthreads_or(any)) {
            Sum2 e = {0.0f, 0.0f};
            for (int vi = tid; vi < a.nvec; vi += nt) {
                const uint4 h = row_again(a, row, vi);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float h0, h1;
                    halves(unpack2(word(h, i)), h0, h1);
                    sum2_add(e, __fmul_rn(h0, h0), 0.0f);   // the square of a bf16 is exact
                    sum2_add(e, __fmul_rn(h1, h1), 0.0f);
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float hi = __shfl_xor_sync(kFull, e.hi, o);
                sum2_add(e, hi, __shfl_xor_sync(kFull, e.lo, o));
            }
            if ((tid & 31) == 0) s_sum[warp] = make_float2(e.hi, e.lo);
            __syncthreads();
            e = Sum2{0.0f, 0.0f};
            for (int w = 0; w < nwarps; ++w) sum2_add(e, s_sum[w].x, s_sum[w].y);
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                if (!near[u]) continue;
                const double mf = __uint_as_float(bm[u]);
                const uint32_t frac = __float_as_uint(__fmul_rn(__uint_as_float(bm[u]), rstd)) & 0x7fffffu;
                const int k = frac < 64u ? ex[u] : ex[u] + 1;
                const double rhs = ldexp((double)e.hi + (double)e.lo + (double)n * (double)a.eps, 2 * k);
                ex[u] = mf * mf * (double)n >= rhs ? k : k - 1;
            }
        }
        // t r as one rounding, from the root and its remainder: the 8-bit codes then differ from those of the real
        // numbers about as seldom as any rounding to float32 before them allows (some 50 of 90 million; with the
        // root alone, off by up to two steps, and a product rounded again the error of a whole output was up to
        // twice that; 32768 x 7168 took 148 us so, and 154 like this).
        const float rest = rsqrt_remainder(rstd, s, n, a.inv_n, a.eps);
        // The power of two of a block goes into the root, unless some values are so far from 1 that it
        // would leave the range.
        auto store = [&](auto into_root) {
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                const int vi = u * nt + tid;
                const bool ok = finite_bits(bm[u]);
                const int se = min(max(ex[u] - TR::emax, -127), 127);
                const float mul = __uint_as_float((uint32_t)(127 - se) << 23);   // 2^-se; se = 127 only for values
                                                                                 // that no finite row reaches
                uint2 c = make_uint2(0, 0);
                if (ok && bm[u]) {
                    const float rm = into_root ? rstd * mul : rstd, lo = into_root ? rest * mul : rest;
                    const f32x2 r2 = pair(rm, rm), lo2 = pair(lo, lo), m2 = pair(mul, mul);
                    float q[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x2 y = fma2(t[u][i], r2, mul2(t[u][i], lo2));
                        halves(into_root ? y : mul2(y, m2), q[2 * i], q[2 * i + 1]);
                    }
                    c.x = cvt_fp8x2<Q>(q[0], q[1]) | (cvt_fp8x2<Q>(q[2], q[3]) << 16);
                    c.y = cvt_fp8x2<Q>(q[4], q[5]) | (cvt_fp8x2<Q>(q[6], q[7]) << 16);
                }
                if (vi < a.nvec) {
                    st_v2(data + 8 * vi, c);
                    if ((vi & 3) == 0)
                        a.scales[row * a.scale_bytes + (vi >> 2)] = (uint8_t)(!ok ? 255 : bm[u] ? se + 127 : 0);
                }
            }
        };
        bool fits = rstd > 0x1p-60f && rstd < 0x1p60f;
#pragma unroll
        for (int u = 0; u < VPT; ++u) fits = fits && ((ex[u] > -50 && ex[u] < 50) || !bm[u]);
        if (fits) store(std::true_type{});
        else store(std::false_type{});
    }
}

// The rows as they are, with the dispatch kernels' arithmetic (quant.cuh), so that the
// codes and scales are those of a fused dispatch bit for bit.
template <int Q, int VPT>
__global__ void __launch_bounds__(VPT == 4 ? 256 : 1024, VPT == 4 ? 4 : 1) quant_rows_kernel(const RowQuantArgs a) {
    using TR = QTraits<Q>;
    __shared__ uint32_t s_max[32];
    const int nt = blockDim.x, tid = threadIdx.x, warp = tid >> 5, nwarps = nt >> 5;
    const int64_t row = blockIdx.x;
    const uint16_t* x = a.x + row * a.x_stride;
    uint4 v[VPT];
    uint32_t m = 0;
    wait_for_previous();
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int vi = u * nt + tid;
        v[u] = vi < a.nvec ? ld_nc_v4(x + 8 * vi) : make_uint4(0, 0, 0, 0);
    }
    float s = 0.0f;
    if constexpr (TR::token) {
#pragma unroll
        for (int u = 0; u < VPT; ++u) m = max(m, vec_absmax_bits(v[u]));
        m = __reduce_max_sync(kFull, m);
        if ((tid & 31) == 0) s_max[warp] = m;
        __syncthreads();
        for (int w = 0; w < nwarps; ++w) m = max(m, s_max[w]);
        s = __fdiv_rn(TR::dmax, bf16_bits_to_float(m));
        if (tid == 0) reinterpret_cast<float*>(a.scales)[row] = __fdiv_rn(1.0f, s);
    }
    uint8_t* data = a.data + row * a.H;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
        const int vi = u * nt + tid;
        float f[8], ginv = 0.0f;
        uint32_t c[2], sbyte = 0;
        unpack8(v[u], f);
        encode_vec<Q>(v[u], f, s, m != 0, c, sbyte, ginv);
        if (vi < a.nvec) {
            st_v2(data + 8 * vi, make_uint2(c[0], c[1]));
            if constexpr (TR::group) {
                if ((vi & 15) == 0) reinterpret_cast<float*>(a.scales + row * a.scale_bytes)[vi >> 4] = ginv;
            }
            if constexpr (TR::mx) {
                if ((vi & 3) == 0) a.scales[row * a.scale_bytes + (vi >> 2)] = (uint8_t)sbyte;
            }
        }
    }
}

// With fewer rows than SMs a thread has one vector (the shortest dependent chain); otherwise four,
// and a row as few warps as that makes, so that many rows share an SM.  65536 x 1024 int8 without a
// residual: 39 us by one warp a row, 55 us by four of one vector each; 65536 x 4096: 147 us by four
// warps, 166 us by eight; 32768 x 7168: 142 us by seven, 212 us by fourteen.
template <int Q, template <int, int> class K>
cudaError_t launch_rows(const RowQuantArgs& a, int sms, cudaStream_t st) {
    const int vpt = a.rows <= sms || a.nvec <= 32 ? 1 : a.nvec <= 64 ? 2 : 4;
    const int nt = ((a.nvec + vpt - 1) / vpt + 31) / 32 * 32;
    const dim3 grid((unsigned)a.rows);
    if (vpt == 1) return K<Q, 1>::run(a, grid, nt, st);
    if (vpt == 2) return K<Q, 2>::run(a, grid, nt, st);
    return K<Q, 4>::run(a, grid, nt, st);
}

template <int Q, int VPT>
struct NormKernel {
    static cudaError_t run(const RowQuantArgs& a, dim3 grid, int nt, cudaStream_t st) {
        return launch_overlapped(rms_norm_quant_kernel<Q, VPT>, grid, nt, 0, st, a);
    }
};

template <int Q, int VPT>
struct QuantKernel {
    static cudaError_t run(const RowQuantArgs& a, dim3 grid, int nt, cudaStream_t st) {
        return launch_overlapped(quant_rows_kernel<Q, VPT>, grid, nt, 0, st, a);
    }
};

template <template <int, int> class K>
cudaError_t launch_mode(const RowQuantArgs& a, int quant, int sms, cudaStream_t st) {
    switch (quant) {
        case EP_QUANT_INT8_PER_TOKEN: return launch_rows<M_INT8, K>(a, sms, st);
        case EP_QUANT_MXFP8_E4M3: return launch_rows<M_E4M3, K>(a, sms, st);
        case EP_QUANT_MXFP8_E5M2: return launch_rows<M_E5M2, K>(a, sms, st);
        case EP_QUANT_FP8_E4M3_PER_TOKEN: return launch_rows<M_FP8T_E4M3, K>(a, sms, st);
        case EP_QUANT_FP8_E5M2_PER_TOKEN: return launch_rows<M_FP8T_E5M2, K>(a, sms, st);
        case EP_QUANT_FP8_E4M3_PER_GROUP: return launch_rows<M_FP8G_E4M3, K>(a, sms, st);
        case EP_QUANT_FP8_E5M2_PER_GROUP: return launch_rows<M_FP8G_E5M2, K>(a, sms, st);
    }
    return cudaErrorInvalidValue;
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

// Checks shared by both entry points; fills the sizes of `a`.
ep_status check_rows(const void* x, int64_t x_stride, int64_t rows, int32_t hidden, ep_quant_mode q,
                     const void* data, const void* scales, RowQuantArgs* a) {
    if (q == EP_QUANT_NONE || q == EP_QUANT_INT8_STATIC || q == EP_QUANT_MXFP4_E2M1) return EP_ERR_UNSUPPORTED;
    int64_t db = 0, sb = 0;
    const ep_status s = ep_recv_row_bytes(hidden, q, &db, &sb);
    if (s != EP_OK) return s;
    if (hidden > 8192 || rows < 0 || rows > INT32_MAX) return EP_ERR_INVALID_ARG;
    if (x_stride < hidden || x_stride % 8 != 0) return EP_ERR_INVALID_ARG;
    if (rows > 0) {
        if (!x || !data || !scales) return EP_ERR_INVALID_ARG;
        if (!aligned(x, 16) || !aligned(data, 16) || !aligned(scales, 4)) return EP_ERR_INVALID_ARG;
    }
    a->x = (const uint16_t*)x;
    a->x_stride = x_stride;
    a->data = (uint8_t*)const_cast<void*>(data);
    a->scales = (uint8_t*)const_cast<void*>(scales);
    a->rows = rows;
    a->H = hidden;
    a->nvec = hidden / 8;
    a->scale_bytes = (int32_t)sb;
    return EP_OK;
}

}  // namespace

cudaError_t launch_rms_norm_quant(const RowQuantArgs& a, int quant, int sms, cudaStream_t st) {
    return launch_mode<NormKernel>(a, quant, sms, st);
}

cudaError_t launch_quant_rows(const RowQuantArgs& a, int quant, int sms, cudaStream_t st) {
    return launch_mode<QuantKernel>(a, quant, sms, st);
}

extern "C" ep_status ep_rms_norm_quant(const void* x, int64_t x_stride, const void* residual,
                                       int64_t residual_stride, const void* gamma, float eps, int64_t rows,
                                       int32_t hidden, ep_quant_mode quant, void* h_out, int64_t h_stride,
                                       void* y_out, void* data, void* scales, ep_stream_t stream) {
    RowQuantArgs a{};
    const ep_status s = check_rows(x, x_stride, rows, hidden, quant, data, scales, &a);
    if (s != EP_OK) return s;
    if (!(eps >= 0.0f) || eps > 3.0e38f) return EP_ERR_INVALID_ARG;
    if (!gamma || !aligned(gamma, 16)) return EP_ERR_INVALID_ARG;
    if (residual && (!aligned(residual, 16) || residual_stride < hidden || residual_stride % 8 != 0))
        return EP_ERR_INVALID_ARG;
    if (h_out && (!aligned(h_out, 16) || h_stride < hidden || h_stride % 8 != 0)) return EP_ERR_INVALID_ARG;
    if (y_out && !aligned(y_out, 16)) return EP_ERR_INVALID_ARG;
    if (rows == 0) return EP_OK;
    a.y_out = (uint16_t*)y_out;
    a.residual = (const uint16_t*)residual;
    a.residual_stride = residual_stride;
    a.gamma = (const uint16_t*)gamma;
    a.h_out = (uint16_t*)h_out;
    a.h_stride = h_stride;
    a.eps = eps;
    a.inv_n = 1.0f / (float)hidden;
    const int sms = ep_current_sms();
    if (sms <= 0) return EP_ERR_CUDA;
    return launch_rms_norm_quant(a, quant, sms, (cudaStream_t)stream) == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}

extern "C" ep_status ep_quant_rows(const void* x, int64_t x_stride, int64_t rows, int32_t hidden,
                                   ep_quant_mode quant, void* data, void* scales, ep_stream_t stream) {
    RowQuantArgs a{};
    const ep_status s = check_rows(x, x_stride, rows, hidden, quant, data, scales, &a);
    if (s != EP_OK) return s;
    if (rows == 0) return EP_OK;
    const int sms = ep_current_sms();
    if (sms <= 0) return EP_ERR_CUDA;
    return launch_quant_rows(a, quant, sms, (cudaStream_t)stream) == cudaSuccess ? EP_OK : EP_ERR_CUDA;
}
