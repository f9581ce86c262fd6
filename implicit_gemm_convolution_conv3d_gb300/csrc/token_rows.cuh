// token_rows.cuh -- what the row kernels (token_norm.cu, token_act.cu) share: a
// row held in registers, its reductions, and its codes.
//
// A row of `n` elements is held by `threads` threads, kVec pieces of 8 elements each
// (as fp32): read once, and everything that needs the whole row (its mean square,
// its largest value) is a reduction between registers.  Thread t holds the pieces
// t, t + threads, ...; a piece is one 16-byte access of a 16-bit matrix.  With
// PHASED rows (any width, stride and base) the pieces start `lead` elements before
// the row, where x's 16-byte blocks do: in a dense matrix of odd width every row of
// every operand then has aligned blocks inside, and only the pieces at the row's
// ends (and operands of another phase) go element by element.
// 64 registers a thread, so that 1024 threads an SM keep their loads in flight: with
// 80 (768 threads) the 216000 x 2048 norm took 549 us against 499.
#pragma once
#include "token_activations.cuh"
#include "token_common.cuh"

namespace c3d {

constexpr int kVec = 4;                      // pieces of 8 elements per thread
constexpr int kHeld = 8 * kVec;
constexpr int kMaxRowThreads = 1024;
constexpr long long kMaxRowWidth = static_cast<long long>(kHeld) * kMaxRowThreads - 8;
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

// Eight elements as one (fp32: two) 16-byte accesses.
template <typename T>
struct alignas(16) Block8 {
    uint4 w[sizeof(T) / 2];
};

// Elements of the row that a 16-byte block of x begins before it.
template <typename TX>
__device__ __forceinline__ int row_lead(const TX* x) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(TX));
}

// Whether pieces that start `lead` elements before p lie on boundaries of `bytes`.
template <typename T>
__device__ __forceinline__ bool in_phase(const T* p, int lead, unsigned bytes) {
    return ((reinterpret_cast<uintptr_t>(p) - static_cast<uintptr_t>(lead) * sizeof(T)) & (bytes - 1u)) == 0;
}

// The thread's elements of a row; those outside it are zeros.  inner: rows of the
// same matrix lie before and behind this one, so that a block which it shares with
// them may be read whole.
template <bool PHASED, typename T>
__device__ __forceinline__ void load_row(const T* p, int n, int lead, bool inner, int t, int threads,
                                         float (&v)[kHeld]) {
    if (!PHASED) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int i0 = (j * threads + t) * 8;
            if (i0 < n) {
                load8(p + i0, v + 8 * j);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * j + e] = 0.0f;
            }
        }
        return;
    }
    // loads first, without branches between them: a branch's block would wait for
    // its own load before the next one is issued
    if (in_phase(p, lead, 16u)) {
        Block8<T> raw[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int i0 = (j * threads + t) * 8 - lead;
            raw[j] = Block8<T>{};
            if (i0 < n && (inner || (i0 >= 0 && i0 + 8 <= n))) raw[j] = *reinterpret_cast<const Block8<T>*>(p + i0);
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            load8(reinterpret_cast<const T*>(&raw[j]), v + 8 * j);
            const int i0 = (j * threads + t) * 8 - lead;
            if (i0 < n && (i0 < 0 || i0 + 8 > n)) {   // the row's ends
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const bool in = i0 + e >= 0 && i0 + e < n;
                    if (!in) v[8 * j + e] = 0.0f;
                    else if (!inner) v[8 * j + e] = to_f32(p[i0 + e]);
                }
            }
        }
    } else {
        T raw[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int at = ((i >> 3) * threads + t) * 8 - lead + (i & 7);
            raw[i] = at >= 0 && at < n ? p[at] : from_f32<T>(0.0f);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) v[i] = to_f32(raw[i]);
    }
}

template <bool PHASED, typename T>
__device__ __forceinline__ void store_row(T* p, int n, int lead, int t, int threads,
                                          const float (&v)[kHeld]) {
    const bool wide = !PHASED || in_phase(p, lead, 16u);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const int i0 = (j * threads + t) * 8 - (PHASED ? lead : 0);
        if (PHASED ? wide && i0 >= 0 && i0 + 8 <= n : i0 < n) {
            store8(p + i0, v + 8 * j);
        } else if (PHASED) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (i0 + e >= 0 && i0 + e < n) p[i0 + e] = from_f32<T>(v[8 * j + e]);
        }
    }
}

// max(a, |b|, |c|), a NaN if any is one
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The largest magnitude of the thread's elements, as bits that order like it.
__device__ __forceinline__ uint32_t held_max(const float (&v)[kHeld]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kHeld; i += 2) m = max_abs_nan(m, v[i], v[i + 1]);
    return __float_as_uint(m);
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
template <bool PHASED, bool E4M3>
__device__ __forceinline__ void store_codes(uint8_t* q, int n, int lead, int t, int threads,
                                            float (&v)[kHeld], float scale, bool blank) {
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
    const bool wide = !PHASED || in_phase(q, lead, 8u);
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
        const int i0 = (j * threads + t) * 8 - (PHASED ? lead : 0);
        if (PHASED ? wide && i0 >= 0 && i0 + 8 <= n : i0 < n) {
            *reinterpret_cast<uint2*>(q + i0) = make_uint2(w[0], w[1]);
        } else if (PHASED) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (i0 + e >= 0 && i0 + e < n) q[i0 + e] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
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

// The block of a row of n elements (with a lead of up to 7 before it unless the
// inputs are aligned: the inputs alone decide which thread adds what, so that
// results do not depend on the outputs' alignment), and the grid for `tokens` rows.
inline dim3 row_block(long long n, bool inputs_aligned) {
    const int warps = static_cast<int>((n + (inputs_aligned ? 0 : 7) + 32 * kHeld - 1) / (32 * kHeld));
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
