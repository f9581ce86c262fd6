// token_activations.cuh -- relu, SiLU and GELU of two fp32 values, with their relative
// accuracy in the negative tail: the row kernels' (token_rows.cuh), and GELU of
// the product's 16-bit outputs (linear_w8a8.cu).
#pragma once
#include "internal.h"

namespace c3d {

// max(v, 0) that keeps a NaN
__device__ __forceinline__ float relu_nan(float v) {
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
    return r;
}

// Two at a time with the two-wide fp32 instructions: the row kernels have about 16
// (ungated) to 27 (gated) instruction slots an element before arithmetic costs
// more than memory does, where erfcf alone takes more.  Two of them are
// special-function operations (2^x and 1/x, a quarter of the rate).

// 2^x within 2 ulp; results below 2^-126 are 0 (keeping them takes three more
// instructions, and the tails are far below their row's scale there).
__device__ __forceinline__ float ex2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// e^m for m <= 0: 2^-t with t = -m log2(e) rounded, times e^(m + t ln 2), what the
// rounding left over, as 1 + (m + t ln 2) (the argument's correction of Cody and
// Waite, "Software Manual for the Elementary Functions", 1980, with ln 2 as one
// fp32 number: 3e-9 |m| off).  Without it t's rounding costs |m| * 2^-24.
__device__ __forceinline__ float2 exp_neg2(float2 m) {
    const float2 t = __fmul2_rn(m, make_float2(-1.44269504f, -1.44269504f));
    const float2 r = __ffma2_rn(t, make_float2(0.693147182f, 0.693147182f), m);
    const float2 e = make_float2(ex2_approx(-t.x), ex2_approx(-t.y));
    return __ffma2_rn(e, r, e);
}

// Both activations are max(v, 0) - |v| T(|v|) with a tail T that falls to 0:
//   v sigmoid(v):  T = e / (1 + e), e = e^-|v|
//   v Phi(v):      T = Phi(-|v|) = e^(-v^2/2) g(|v|)
// Below zero that is the tail alone, with its relative accuracy, and nothing
// overflows on either side; the tail is 0 where e is below 2^-126 (v < -87.3; -13.2).
// n = -|v|, cut where the tail is 0 in any case (128; 64).  Infinities come out as
// the limits 0 and inf; a caller that holds -inf * 0 to be NaN looks at its inputs,
// or has gelu2<true> do it (half an instruction an element more).
__device__ __forceinline__ float2 silu2(float2 v) {
    const float2 n = make_float2(fmaxf(-fabsf(v.x), -128.0f), fmaxf(-fabsf(v.y), -128.0f));
    const float2 e = exp_neg2(n);
    const float2 d = __fadd2_rn(e, make_float2(1.0f, 1.0f));
    const float2 tail = __fmul2_rn(e, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
    return __ffma2_rn(n, tail, make_float2(relu_nan(v.x), relu_nan(v.y)));
}

// g(a) = t Q(t), t = 1 / (1 + 0.35 a); Q, of degree 8, is a minimax fit of
// e^(a^2/2) Phi(-a) / t over 0 <= a <= 14 (reweighted least squares in 64 bits;
// relative error 3.2e-8, 3.4e-7 at most as evaluated in fp32).
template <bool INF_TO_NAN = false>
__device__ __forceinline__ float2 gelu2(float2 v) {
    const float2 n = make_float2(fmaxf(-fabsf(v.x), -64.0f), fmaxf(-fabsf(v.y), -64.0f));
    const float2 d = __ffma2_rn(n, make_float2(-0.35f, -0.35f), make_float2(1.0f, 1.0f));
    const float2 t = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    constexpr float kQ[9] = {0.13962141f, 0.13986187f, 0.11983292f, 0.10550778f, -0.023109227f,
                             0.15917318f, -0.25571328f, 0.14397119f, -0.029145816f};
    float2 q = make_float2(kQ[8], kQ[8]);
#pragma unroll
    for (int i = 7; i >= 0; --i) q = __ffma2_rn(q, t, make_float2(kQ[i], kQ[i]));
    const float2 e = exp_neg2(__fmul2_rn(__fmul2_rn(n, n), make_float2(-0.5f, -0.5f)));
    const float2 tail = __fmul2_rn(__fmul2_rn(q, t), e);
    // max(v, 0), or v + max(-v, 0): the same but for -inf
    const float2 r = INF_TO_NAN ? __fadd2_rn(v, make_float2(fmaxf(-v.x, 0.0f), fmaxf(-v.y, 0.0f)))
                                : make_float2(relu_nan(v.x), relu_nan(v.y));
    return __ffma2_rn(n, tail, r);
}

template <int ACT>
__device__ __forceinline__ float2 act2(float2 v) {
    if (ACT == kActRelu) return make_float2(relu_nan(v.x), relu_nan(v.y));
    if (ACT == kActSilu) return silu2(v);
    if (ACT == kActGelu) return gelu2(v);
    return v;
}

}  // namespace c3d
