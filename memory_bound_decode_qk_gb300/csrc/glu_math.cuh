// glu_math.cuh -- the gated activations act(g) * u, shared by the kernels that
// write them in the activation dtype or in 8 bits.
//
//   silu(g)      = g * sigma(g)
//   gelu_tanh(g) = 0.5 g (1 + tanh z) = g * sigma(2z),
//                  z = sqrt(2/pi) (g + 0.044715 g^3)
// The second form is an exact identity, since 0.5 (1 + tanh z) equals the
// logistic sigma(2z).  It avoids the cancellation of 1 + tanh z for negative
// z.  sigma(v) is evaluated as num / (1 + e^-|v|) with num = 1 for v >= 0 and
// e^-|v| otherwise, so nothing overflows.
//
// Two precisions of the exponential, both from this identity:
//   - fp32 outputs: libm expf, an IEEE divide, and the GELU argument 2z
//     carried as an unevaluated sum of two floats.  This keeps the relative
//     error within a few fp32 ulps for every g.
//   - bf16 / fp16 / 8-bit outputs: e^-a = 2^(-a log2 e) through ex2.approx and
//     a reciprocal through rcp.approx.  The error is a few fp32 ulps (plus
//     the |2z| * 2^-24 of the argument's rounding), far inside half an ulp of
//     the output in most cases.  This keeps the kernel HBM-bound rather than
//     issue-bound at full bandwidth.
#pragma once

#include "edge_common.cuh"

namespace edge {

constexpr int kSilu = 0;
constexpr int kGelu = 1;

// Constants from their definitions, split into a float and its remainder.
constexpr double kLog2eD = 1.4426950408889634073599246810019;   // log2(e)
constexpr double kK2D = 1.5957691216057307117597842397375;      // 2 sqrt(2/pi)
constexpr double kCD = 0.044715;
constexpr float kLog2e = (float)kLog2eD;
constexpr float kK2 = (float)kK2D;
// 2 sqrt(2/pi) log2(e): the fast tanh-GELU forms its exponent in base 2
// directly, one product fewer per element
constexpr float kK2L = (float)(kK2D * kLog2eD);
constexpr float kK2lo = (float)(kK2D - (double)(float)kK2D);
constexpr float kC = (float)kCD;
constexpr float kClo = (float)(kCD - (double)(float)kCD);

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Reciprocal of x in [1, 2] (its only use: 1 / (1 + e^-|v|)).  Neither x nor
// 1/x is subnormal there, so the flush-to-zero form gives the same result
// without the subnormal handling of the plain form (measured on GB300: 1.17x
// on the issue-bound tanh-GELU gate with FP8 output).
__device__ __forceinline__ float rcp_approx_1to2(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// act(g) * u, fast form (bf16 / fp16 / FP8 outputs).  vl is the logistic
// argument times log2(e), so that e^-|v| = 2^-|vl|.
template <int ACT>
__device__ __forceinline__ float gate_fast(float g, float u) {
    float vl;
    if constexpr (ACT == kSilu) {
        vl = __fmul_rn(g, kLog2e);
    } else {
        const float c2 = __fmul_rn(__fmul_rn(kC, g), g);
        vl = __fmul_rn(__fmul_rn(kK2L, g), __fadd_rn(1.0f, c2));
    }
    const float t = ex2_approx(-fabsf(vl));
    const float num = vl >= 0.0f ? 1.0f : t;
    // g * sigma(v) first, u last: g * u could overflow where sigma(v) = 0
    return __fmul_rn(__fmul_rn(g, __fmul_rn(num, rcp_approx_1to2(__fadd_rn(1.0f, t)))), u);
}

// gate_fast on a pair of elements: the products and sums as packed two-lane
// instructions (each lane rounded as gate_fast rounds it, so the results are
// the same bits), the exponential and the reciprocal per lane.
template <int ACT>
__device__ __forceinline__ float2 gate_fast2(float2 g, float2 u) {
    float2 vl;
    if constexpr (ACT == kSilu) {
        vl = __fmul2_rn(g, splat2(kLog2e));
    } else {
        const float2 c2 = __fmul2_rn(__fmul2_rn(splat2(kC), g), g);
        vl = __fmul2_rn(__fmul2_rn(splat2(kK2L), g), __fadd2_rn(splat2(1.0f), c2));
    }
    const float2 t = make_float2(ex2_approx(-fabsf(vl.x)), ex2_approx(-fabsf(vl.y)));
    const float2 num = make_float2(vl.x >= 0.0f ? 1.0f : t.x, vl.y >= 0.0f ? 1.0f : t.y);
    const float2 den = __fadd2_rn(splat2(1.0f), t);
    const float2 rc = make_float2(rcp_approx_1to2(den.x), rcp_approx_1to2(den.y));
    // g * sigma(v) first, u last (see gate_fast)
    return __fmul2_rn(__fmul2_rn(g, __fmul2_rn(num, rc)), u);
}

// act(g) * u, accurate form (fp32 outputs).
template <int ACT>
__device__ __forceinline__ float gate_accurate(float g, float u) {
    float a, ae;  // |v| = a + ae, v the logistic argument
    bool neg;
    if constexpr (ACT == kSilu) {
        a = fabsf(g);
        ae = 0.0f;
        neg = g < 0.0f;
    } else {
        // v = 2z = K g (1 + C g^2) in double-float arithmetic.  Past |g| = 2^20,
        // |v| > 2^56 and sigma(v) is exactly 0 or 1 in fp32, so g is clamped
        // there: the double-float terms would overflow to inf - inf.
        const float gc = fminf(fmaxf(g, -1048576.0f), 1048576.0f);
        const float g2 = __fmul_rn(gc, gc);
        const float g2e = __fmaf_rn(gc, gc, -g2);
        const float c = __fmul_rn(kC, g2);
        const float ce = __fmaf_rn(kC, g2, -c) + __fmaf_rn(kC, g2e, __fmul_rn(kClo, g2));
        const float s = __fadd_rn(1.0f, c);
        const float bb = __fsub_rn(s, 1.0f);
        const float se = __fadd_rn(__fadd_rn(__fsub_rn(1.0f, __fsub_rn(s, bb)), __fsub_rn(c, bb)), ce);
        const float pq = __fmul_rn(gc, s);
        const float pe = __fmaf_rn(gc, s, -pq) + __fmul_rn(gc, se);
        const float z = __fmul_rn(kK2, pq);
        const float ze = __fmaf_rn(kK2, pq, -z) + __fmaf_rn(kK2, pe, __fmul_rn(kK2lo, pq));
        neg = z < 0.0f;
        a = fabsf(z);
        ae = neg ? -ze : ze;
    }
    // e^-(a + ae) = e^-a * e^-ae ~= e^-a (1 - ae), |ae| <= a few ulp of a.
    // Wherever e^-a is nonzero (a < 104), |ae| < 2^-15; the clamp only keeps
    // t = +0 past that, where a's ulp can exceed 1.
    const float t = __fmul_rn(expf(-a), __fsub_rn(1.0f, fminf(fmaxf(ae, -0.25f), 0.25f)));
    const float num = neg ? t : 1.0f;
    // g * sigma first, u last (see gate_fast)
    return __fmul_rn(__fmul_rn(g, __fdiv_rn(num, __fadd_rn(1.0f, t))), u);
}

template <typename T, bool FP8, int ACT>
__device__ __forceinline__ float gate(float g, float u) {
    if constexpr (std::is_same<T, float>::value && !FP8) {
        return gate_accurate<ACT>(g, u);
    } else {
        return gate_fast<ACT>(g, u);
    }
}

}  // namespace edge
