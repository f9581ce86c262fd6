// token_rows.cuh -- what the row kernels (token_norm.cu, token_act.cu) share: a
// row held in registers, its reductions, and its codes.
//
// A row of `n` elements is held by `threads` threads, kVec x 8 elements each
// (as fp32): read once, and everything that needs the whole row (its mean
// square, its largest value) is a reduction between registers.  Two layouts:
//   VEC 8: thread t holds the 8-element pieces t, t + threads, ... (16-byte
//          loads of 16-bit types; width, strides and bases in whole pieces)
//   VEC 1: thread t holds the elements t, t + threads, ... (any alignment)
// Rows of up to kMaxRowWidth elements go this way; a wider row is read again
// for each pass.
#pragma once
#include "token_common.cuh"

namespace c3d {

constexpr int kVec = 4;                      // pieces of 8 elements per thread
constexpr int kHeld = 8 * kVec;
constexpr int kMaxRowThreads = 512;         // 128 registers a thread
constexpr int kWideThreads = 1024;
constexpr long long kMaxRowWidth = static_cast<long long>(kHeld) * kMaxRowThreads;
constexpr int kWarpRows = 4;                 // rows of a block when one warp holds a row

// 8 consecutive elements (16- or 32-byte aligned) as fp32
__device__ __forceinline__ void load8(const float* p, float* v) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void load8(const __half* p, float* v) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ void store8(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(__half* p, const float* v) {
    __half2 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h);
}

// Index of the first element of piece j of thread t, and whether the piece (VEC 8)
// or element e of it (VEC 1) lies in the row.
template <int VEC>
__device__ __forceinline__ int piece_at(int j, int t, int threads) {
    return VEC == 8 ? (j * threads + t) * 8 : j * 8 * threads + t;
}

// The thread's elements of a row; those outside it are zeros.
template <int VEC, typename T>
__device__ __forceinline__ void load_row(const T* p, int n, int t, int threads, float (&v)[kHeld]) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const int i0 = piece_at<VEC>(j, t, threads);
        if (VEC == 8) {
            if (i0 < n) {
                load8(p + i0, v + 8 * j);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * j + e] = 0.0f;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + e * threads;
                v[8 * j + e] = i < n ? to_f32(p[i]) : 0.0f;
            }
        }
    }
}

template <int VEC, typename T>
__device__ __forceinline__ void store_row(T* p, int n, int t, int threads, const float (&v)[kHeld]) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const int i0 = piece_at<VEC>(j, t, threads);
        if (VEC == 8) {
            if (i0 < n) store8(p + i0, v + 8 * j);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + e * threads;
                if (i < n) p[i] = from_f32<T>(v[8 * j + e]);
            }
        }
    }
}

// max(a, |b|), a NaN if either is one
__device__ __forceinline__ float max_abs_nan(float a, float b) {
    float r;
    asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %2;\n\tmax.NaN.f32 %0, %1, t;\n\t}" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// ---------------------------------------------------------------- activations
// Two at a time with the two-wide fp32 instructions: the row kernels have about 16
// (ungated) to 27 (gated) instruction slots an element before arithmetic costs
// more than memory does, where erfcf alone takes more.  Two of them are
// special-function operations (2^x and 1/x, a quarter of the rate).

__device__ __forceinline__ float ex2_approx(float x) {   // 2 ulp; subnormal results kept
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// e^-y for y >= 0: 2^-t with t = y log2(e) rounded, times e^(t ln 2 - y), what the
// rounding left over, as 1 + (t ln 2 - y); ln 2 in two parts (Cody and Waite,
// "Software Manual for the Elementary Functions", 1980).  Without it t's rounding
// costs y * 2^-24 of relative error.
__device__ __forceinline__ float2 exp_neg2(float2 y) {
    const float2 t = __fmul2_rn(y, make_float2(1.44269504f, 1.44269504f));
    float2 r = __ffma2_rn(t, make_float2(0.693147182f, 0.693147182f), make_float2(-y.x, -y.y));
    r = __ffma2_rn(t, make_float2(-1.90465421e-9f, -1.90465421e-9f), r);
    const float2 e = make_float2(ex2_approx(-t.x), ex2_approx(-t.y));
    return __ffma2_rn(e, r, e);
}

// v * sigmoid(v) with e = e^-|v|: v / (1 + e), or v e / (1 + e) below zero (no
// overflow on either side; beyond 128 e is 0 in any case).
__device__ __forceinline__ float2 silu2(float2 v) {
    const float2 e = exp_neg2(make_float2(fminf(fabsf(v.x), 128.0f), fminf(fabsf(v.y), 128.0f)));
    const float2 d = __fadd2_rn(e, make_float2(1.0f, 1.0f));
    const float2 r = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    const float2 n = make_float2(v.x < 0.0f ? e.x : 1.0f, v.y < 0.0f ? e.y : 1.0f);
    return __fmul2_rn(__fmul2_rn(v, n), r);
}

// v * Phi(v) through the tail P = Phi(-|v|) = e^(-v^2/2) g(|v|), which keeps its
// relative accuracy: Phi = P below zero and 1 - P above.  g(a) = t Q(t) with
// t = 1 / (1 + 0.35 a); Q, of degree 8, is a minimax fit of e^(a^2/2) Phi(-a) / t over
// 0 <= a <= 14 (reweighted least squares in 64 bits; relative error 3.2e-8,
// 3.4e-7 at most as evaluated in fp32).  Beyond 64 the tail is 0 in any case.
__device__ __forceinline__ float2 gelu2(float2 v) {
    const float2 a = make_float2(fminf(fabsf(v.x), 64.0f), fminf(fabsf(v.y), 64.0f));
    const float2 d = __ffma2_rn(a, make_float2(0.35f, 0.35f), make_float2(1.0f, 1.0f));
    const float2 t = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    constexpr float kQ[9] = {0.13962141f, 0.13986187f, 0.11983292f, 0.10550778f, -0.023109227f,
                             0.15917318f, -0.25571328f, 0.14397119f, -0.029145816f};
    float2 q = make_float2(kQ[8], kQ[8]);
#pragma unroll
    for (int i = 7; i >= 0; --i) q = __ffma2_rn(q, t, make_float2(kQ[i], kQ[i]));
    const float2 e = exp_neg2(__fmul2_rn(__fmul2_rn(a, a), make_float2(0.5f, 0.5f)));
    const float2 tail = __fmul2_rn(__fmul2_rn(q, t), e);
    const float2 rest = __ffma2_rn(tail, make_float2(-1.0f, -1.0f), make_float2(1.0f, 1.0f));
    return __fmul2_rn(v, make_float2(v.x < 0.0f ? tail.x : rest.x, v.y < 0.0f ? tail.y : rest.y));
}

template <int ACT>
__device__ __forceinline__ float2 act2(float2 v) {
    if (ACT == kActRelu) return make_float2(v.x < 0.0f ? 0.0f : v.x, v.y < 0.0f ? 0.0f : v.y);
    if (ACT == kActSilu) return silu2(v);
    if (ACT == kActGelu) return gelu2(v);
    return v;
}

// Four int8 codes of quotients within +-127: adding 1.5 * 2^23 rounds each to the
// nearest integer (ties to even) and leaves its two's complement in the low byte.
__device__ __forceinline__ uint32_t int8x4(float a, float b, float c, float d) {
    constexpr float kMagic = 12582912.0f;
    const uint32_t x = __float_as_uint(a + kMagic), y = __float_as_uint(b + kMagic);
    const uint32_t z = __float_as_uint(c + kMagic), w = __float_as_uint(d + kMagic);
    return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
}

// The thread's codes: the nearest to v / scale, the quotient by the corrected
// reciprocal (quot_corrected's steps, two at a time; the sign of a zero quotient,
// which they may lose, is no matter here) or, for scales that is not valid for, by
// division.
template <int VEC, bool E4M3>
__device__ __forceinline__ void store_codes(uint8_t* q, int n, int t, int threads, float (&v)[kHeld],
                                            float scale, bool blank, bool wide_q) {
    if (quot_corrected_ok(scale)) {
        const float y1 = 1.0f / scale;
        const float2 y = make_float2(y1, y1), ns = make_float2(-scale, -scale);
#pragma unroll
        for (int i = 0; i < kHeld; i += 2) {
            const float2 x = make_float2(v[i], v[i + 1]);
            const float2 q0 = __fmul2_rn(x, y);
            const float2 q1 = __ffma2_rn(__ffma2_rn(ns, q0, x), y, q0);
            v[i] = q1.x;
            v[i + 1] = q1.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) v[i] = v[i] / scale;
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float* c = v + 8 * j + 4 * h;
            if (E4M3)
                w[h] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(c[0], c[1]),
                                                                      __NV_SATFINITE, __NV_E4M3)) |
                       static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(c[2], c[3]),
                                                                      __NV_SATFINITE, __NV_E4M3))
                           << 16;
            else
                w[h] = int8x4(c[0], c[1], c[2], c[3]);
            if (blank) w[h] = 0u;
        }
        const int i0 = piece_at<VEC>(j, t, threads);
        if (VEC == 8) {
            if (i0 < n) {
                if (wide_q) {
                    *reinterpret_cast<uint2*>(q + i0) = make_uint2(w[0], w[1]);
                } else {   // the inputs decide the layout, so that results do not depend on q
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        q[i0 + e] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + e * threads;
                if (i < n) q[i] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
            }
        }
    }
}

// Sum / maximum over a row's threads: a warp, or a whole block of `warps` warps
// through `sh` (32 entries, each array used once per row).
__device__ __forceinline__ float row_sum(float v, int warps, float* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? sh[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ uint32_t row_max(uint32_t v, int warps, uint32_t* sh) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, lane < warps ? sh[lane] : 0u);
}

// The block of a row of n elements, and the grid for `tokens` rows.
inline dim3 row_block(long long n) {
    const int warps = static_cast<int>((n + 32 * kHeld - 1) / (32 * kHeld));
    return warps <= 1 ? dim3(32, kWarpRows) : dim3(static_cast<unsigned>(32 * warps), 1);
}
inline unsigned row_blocks(long long tokens, const dim3& block) {
    return static_cast<unsigned>((tokens + block.y - 1) / block.y);
}

inline bool aligned_rows(const void* p, long long stride, long long tokens, int elt, int bytes) {
    return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && (tokens == 1 || stride * elt % bytes == 0));
}

inline int elt_bytes(int dtype) { return dtype == kTokF32 ? 4 : dtype == kTokBf16 || dtype == kTokF16 ? 2 : 1; }

}  // namespace c3d
