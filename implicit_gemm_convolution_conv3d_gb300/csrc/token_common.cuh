// token_common.cuh -- what the token kernels (token_norm.cu, token_act.cu,
// linear_w8a8.cu) share: element loads and stores in fp32, the fp32 outputs'
// activations, the row scale and codes of the 8-bit outputs, and launches.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "internal.h"
#include "kernel_common.cuh"

namespace c3d {

// element types of the token operators (values of the C ABI's codes)
constexpr int kTokBf16 = 0, kTokE4m3 = 1, kTokInt8 = 2, kTokF16 = 3, kTokF32 = 4;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The activations to fp32 accuracy (the convolutions' epilogue forms in
// internal.h are shaped for bf16 results): v * sigmoid(v) = v / (1 + e^-v), and
// v * Phi(v) = v/2 * erfc(-v / sqrt 2), which keeps its relative accuracy in
// the negative tail where 1 + erf cancels.  relu keeps a NaN.
__device__ __forceinline__ float activate_f32(float v, int act) {
    if (act == kActRelu) return v < 0.0f ? 0.0f : v;
    if (act == kActSilu) return v / (1.0f + expf(-v));
    if (act == kActGelu) return 0.5f * v * erfcf(v * -0.70710678118654752f);
    return v;
}

// |v| as an integer that orders like the magnitude, infinities and NaNs on top
// (so a maximum over these bits keeps a NaN, which fmaxf would drop)
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u, kNanBits = 0x7FC00000u;

// The row's scale from its largest |v|: max / qmax by IEEE division, 1 for a
// row of zeros, NaN for a row that is not finite; never subnormal, so that
// v / scale stays within qmax (rows below qmax * 2^-126 lose nothing that the
// codes could hold).
__device__ __forceinline__ float row_scale(uint32_t amax_bits, float qmax) {
    if (amax_bits >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
    if (amax_bits == 0u) return 1.0f;
    return fmaxf(__uint_as_float(amax_bits) / qmax, 1.17549435e-38f);
}

// Rows that hold no information for the codes (all zeros, or not finite):
// their codes are 0, where v / scale would give e4m3's negative zero or NaN.
__device__ __forceinline__ bool row_blank(uint32_t amax_bits) {
    return amax_bits == 0u || amax_bits >= 0x7F800000u;
}

// The code of v / scale (nearest, ties to even) as a byte.
template <bool E4M3>
__device__ __forceinline__ uint32_t code_of(float v, float scale) {
    const float c = v / scale;
    if (E4M3) return __nv_cvt_float_to_fp8(c, __NV_SATFINITE, __NV_E4M3);
    return static_cast<uint32_t>(__float2int_rn(c)) & 0xFFu;
}

// Launch with programmatic stream serialization (unless overridden): the kernel
// may start while the previous one in the stream runs, and waits for it
// (griddep_wait) before it touches global memory.  cluster: CTAs of a cluster.
template <typename Kernel, typename... Args>
inline cudaError_t launch_ex(Kernel kern, unsigned grid, dim3 block, size_t smem, int cluster,
                             cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = overrides().pdl != 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace c3d
