// token_quant.cu -- rows of tokens brought to 8 bits with a scale each: the
// root-mean-square norm with the residual's addition, and the (gated)
// activation.
#include <cuda_runtime.h>

#include "token_common.cuh"
#include "token_ops_internal.h"

namespace c3d {

namespace {

constexpr int kRowThreads = 256;

// sum / maximum over the block; every thread gets the result
__device__ __forceinline__ float block_sum(float v, float* sh) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) s += sh[i];
    return s;
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* sh) {
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    uint32_t s = 0;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) s = max(s, sh[i]);
    return s;
}

// One block per row, three passes over it (sum of squares, maximum, codes).
template <typename TX, typename TR, typename TW, bool E4M3>
__global__ void __launch_bounds__(kRowThreads) norm_rows_kernel(const NormParams p) {
    __shared__ float shf[32];
    __shared__ uint32_t shu[32];
    const int n = static_cast<int>(p.width);
    for (long long row = blockIdx.x; row < p.tokens; row += gridDim.x) {
        const TX* x = static_cast<const TX*>(p.x) + row * p.x_stride;
        const TR* r = p.res ? static_cast<const TR*>(p.res) + row * p.res_stride : nullptr;
        TR* ro = p.res_out ? static_cast<TR*>(p.res_out) + row * p.res_out_stride : nullptr;
        const TW* w = static_cast<const TW*>(p.weight);
        uint8_t* q = p.q + row * p.q_stride;
        auto h_at = [&](int i) { return to_f32(x[i]) + (r ? to_f32(r[i]) : 0.0f); };
        float ss = 0.0f;
        for (int i = threadIdx.x; i < n; i += kRowThreads) {
            const float h = h_at(i) * p.shrink;
            ss = fmaf(h, h, ss);
        }
        const float rms = 1.0f / sqrtf(block_sum(ss, shf) * p.mean_of + p.eps);
        auto v_of = [&](float h, int i) { return h * rms * (w ? to_f32(w[i]) : 1.0f); };
        uint32_t m = 0;
        for (int i = threadIdx.x; i < n; i += kRowThreads) m = max(m, abs_bits(v_of(h_at(i), i)));
        const uint32_t top = block_max(m, shu);
        const float scale = row_scale(top, E4M3 ? 448.0f : 127.0f);
        for (int i = threadIdx.x; i < n; i += kRowThreads) {
            const float h = h_at(i);
            q[i] = row_blank(top) ? 0 : static_cast<uint8_t>(code_of<E4M3>(v_of(h, i), scale));
            if (ro) ro[i] = from_f32<TR>(h);
        }
        if (threadIdx.x == 0) p.scale[row] = scale;
    }
}

template <typename TX, bool E4M3>
__global__ void __launch_bounds__(kRowThreads) act_rows_kernel(const ActParams p) {
    __shared__ uint32_t shu[32];
    const long long n = p.width;
    for (long long row = blockIdx.x; row < p.tokens; row += gridDim.x) {
        const TX* x = static_cast<const TX*>(p.x) + row * p.x_stride;
        uint8_t* q = p.q + row * p.q_stride;
        auto v_at = [&](long long i) {
            const float a = activate_f32(to_f32(x[i]), p.act);
            return p.gated ? a * to_f32(x[n + i]) : a;
        };
        uint32_t m = 0;
        for (long long i = threadIdx.x; i < n; i += kRowThreads) m = max(m, abs_bits(v_at(i)));
        const uint32_t top = block_max(m, shu);
        const float scale = row_scale(top, E4M3 ? 448.0f : 127.0f);
        for (long long i = threadIdx.x; i < n; i += kRowThreads)
            q[i] = row_blank(top) ? 0 : static_cast<uint8_t>(code_of<E4M3>(v_at(i), scale));
        if (threadIdx.x == 0) p.scale[row] = scale;
    }
}

unsigned row_grid(long long tokens) {
    return static_cast<unsigned>(tokens < (1 << 20) ? tokens : (1 << 20));
}

template <typename TX, typename TR, typename TW>
cudaError_t norm_q(const NormParams& p, cudaStream_t stream) {
    if (p.q_dtype == kTokE4m3)
        norm_rows_kernel<TX, TR, TW, true><<<row_grid(p.tokens), kRowThreads, 0, stream>>>(p);
    else
        norm_rows_kernel<TX, TR, TW, false><<<row_grid(p.tokens), kRowThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename TX>
cudaError_t norm_x(const NormParams& p, cudaStream_t stream) {
    const bool rf = p.res && p.res_dtype == kTokF32, wf = p.weight_dtype == kTokF32;
    if (rf) return wf ? norm_q<TX, float, float>(p, stream) : norm_q<TX, float, TX>(p, stream);
    return wf ? norm_q<TX, TX, float>(p, stream) : norm_q<TX, TX, TX>(p, stream);
}

template <typename TX>
cudaError_t act_x(const ActParams& p, cudaStream_t stream) {
    if (p.q_dtype == kTokE4m3)
        act_rows_kernel<TX, true><<<row_grid(p.tokens), kRowThreads, 0, stream>>>(p);
    else
        act_rows_kernel<TX, false><<<row_grid(p.tokens), kRowThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_quant(const NormParams& p, cudaStream_t stream) {
    if (p.x_dtype == kTokBf16) return norm_x<__nv_bfloat16>(p, stream);
    if (p.x_dtype == kTokF16) return norm_x<__half>(p, stream);
    return norm_x<float>(p, stream);
}

cudaError_t launch_act_quant(const ActParams& p, cudaStream_t stream) {
    if (p.x_dtype == kTokBf16) return act_x<__nv_bfloat16>(p, stream);
    if (p.x_dtype == kTokF16) return act_x<__half>(p, stream);
    return act_x<float>(p, stream);
}

}  // namespace c3d
