// linear_w8a8.cu -- the product of 8-bit tokens and weights with a scale per
// token and per output channel.
#include <cuda_runtime.h>

#include "token_common.cuh"
#include "token_ops_internal.h"

namespace c3d {

namespace {

constexpr int kT = 64;   // outputs and tokens of a tile
constexpr int kKB = 32;  // reduction elements of a step

__device__ __forceinline__ void store_out(void* out, int dtype, long long at, float v) {
    if (dtype == kTokBf16) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
    else if (dtype == kTokF16) static_cast<__half*>(out)[at] = __float2half_rn(v);
    else static_cast<float*>(out)[at] = v;
}

template <bool E4M3>
__device__ __forceinline__ float code_value(uint8_t c) {
    if (E4M3) return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
    return static_cast<float>(static_cast<int8_t>(c));
}

// A 64 x 64 tile per block of 256 threads, 4 x 4 outputs a thread.
template <bool E4M3>
__global__ void __launch_bounds__(256) linear_tile_kernel(const LinearParams p) {
    __shared__ float xs[kKB][kT + 1], ws[kKB][kT + 1];
    const long long n0 = static_cast<long long>(blockIdx.x) * kT;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const long long m_tiles = (p.tokens + kT - 1) / kT;
    for (long long mt = blockIdx.y; mt < m_tiles; mt += gridDim.y) {
        const long long m0 = mt * kT;
        float acc[4][4] = {};
        for (long long k0 = 0; k0 < p.width; k0 += kKB) {
            for (int i = threadIdx.x; i < kT * kKB; i += 256) {
                const int r = i / kKB, c = i % kKB;
                const bool kin = k0 + c < p.width;
                xs[c][r] = kin && m0 + r < p.tokens
                               ? code_value<E4M3>(p.x[(m0 + r) * p.x_stride + k0 + c]) : 0.0f;
                ws[c][r] = kin && n0 + r < p.outputs
                               ? code_value<E4M3>(p.w[(n0 + r) * p.w_stride + k0 + c]) : 0.0f;
            }
            __syncthreads();
            for (int k = 0; k < kKB; ++k)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = fmaf(xs[k][ty + 16 * i], ws[k][tx + 16 * j], acc[i][j]);
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i) {
            const long long m = m0 + ty + 16 * i;
            if (m >= p.tokens) continue;
            const float sx = p.scale_x ? p.scale_x[m] : 1.0f;
            for (int j = 0; j < 4; ++j) {
                const long long n = n0 + tx + 16 * j;
                if (n >= p.outputs) continue;
                float v = acc[i][j] * sx * (p.scale_w ? p.scale_w[n] : 1.0f);
                if (p.bias) v += p.bias[n];
                store_out(p.out, p.out_dtype, m * p.out_stride + n, activate_f32(v, p.act));
            }
        }
    }
}

}  // namespace

cudaError_t launch_linear_w8a8(const LinearParams& p, cudaStream_t stream) {
    const long long mt = (p.tokens + kT - 1) / kT;
    const dim3 grid(static_cast<unsigned>((p.outputs + kT - 1) / kT),
                    static_cast<unsigned>(mt < 65535 ? mt : 65535));
    if (p.e4m3) linear_tile_kernel<true><<<grid, 256, 0, stream>>>(p);
    else linear_tile_kernel<false><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace c3d
