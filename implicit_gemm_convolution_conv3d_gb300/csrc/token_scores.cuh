// token_scores.cuh -- device helpers that the attention kernels share: exponentials in
// powers of two, arithmetic on two values at a time, and the cap on scores.
#pragma once
#include "token_common.cuh"

namespace c3d {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two values a register pair: one instruction each
__device__ __forceinline__ uint64_t two(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint64_t two(float v) { return two(__float_as_uint(v), __float_as_uint(v)); }
__device__ __forceinline__ void split(uint64_t v, uint32_t& a, uint32_t& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The cap: cap * tanh(s / cap).  With x = s / cap, |x| <= kTanhReach, tanh(x) / x is a
// polynomial in x^2, within 1.3e-7 of it in fp32 arithmetic (a least-squares fit reweighted
// towards equal relative errors), so that s times it keeps its relative accuracy however
// small s is beside the cap.  Beyond, 1 - 2 / (1 + e^2x), which cancels near 0, is within
// 2.5e-7, less than 2^-20 of a tanh of 0.537 or more.
constexpr float kTanhReach = 0.6f;
__device__ constexpr float kTanh[5] = {0.99999994f, -0.33332309f, 0.133101732f, -0.052101478f, 0.0154754231f};

// Two scores within the reach, capped and in powers of two
__device__ __forceinline__ uint64_t cap_pair(uint64_t s, uint64_t inv_cap) {
    const uint64_t x = mul2(s, inv_cap), u = mul2(x, x);
    uint64_t y = fma2(u, two(kTanh[4] * kLog2e), two(kTanh[3] * kLog2e));
#pragma unroll
    for (int d = 2; d >= 0; --d) y = fma2(u, y, two(kTanh[d] * kLog2e));
    return mul2(s, y);
}

// Any two
__device__ __forceinline__ uint64_t cap_pair_any(uint64_t s, float cap, float inv_cap) {
    uint32_t x[2], near[2], r[2];
    split(mul2(s, two(inv_cap)), x[0], x[1]);
    split(cap_pair(s, two(inv_cap)), near[0], near[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float v = __uint_as_float(x[i]);
        const float far = cap * (kLog2e - 2.0f * kLog2e * rcp_approx(1.0f + ex2(v * (2.0f * kLog2e))));
        r[i] = fabsf(v) <= kTanhReach ? near[i] : __float_as_uint(far);
    }
    return two(r[0], r[1]);
}

// Any score, capped
__device__ __forceinline__ float cap_score(float s, float cap, float inv_cap) {
    const float x = s * inv_cap, u = x * x;
    if (fabsf(x) <= kTanhReach) return s * fmaf(u, fmaf(u, fmaf(u, fmaf(u, kTanh[4], kTanh[3]), kTanh[2]), kTanh[1]), kTanh[0]);
    return cap * (1.0f - 2.0f * rcp_approx(1.0f + ex2(x * (2.0f * kLog2e))));
}

}  // namespace c3d
