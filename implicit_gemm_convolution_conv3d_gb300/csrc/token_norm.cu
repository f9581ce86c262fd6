// token_norm.cu -- the root-mean-square norm with the residual's addition and an
// 8-bit output:
//
//   h = x + residual;  r = 1 / sqrt(mean(h^2) + eps);  v = h r w
//   scale = max|v| / qmax;  q = nearest code of v / scale
//
// Bound by memory: x and the residual are read once and h, q and the scale
// written once (7 bytes an element for a bf16 stream); the row waits in registers
// for its two reductions.  216000 x 2048 takes 500 us (6.2 TB/s).
#include <cuda_runtime.h>

#include "token_ops_internal.h"
#include "token_rows.cuh"

namespace c3d {

namespace {

constexpr float kMaxFinite = 3.4028235e38f;

// A square loses up to 2^-150 at fp32's lower end, fewer than 2^31 of them up to
// 2^-117 of the mean: 2^-53 of this mean square (eps included) and above.  Rows
// below it (an eps near 0 and tokens below 2^-32) are taken times 2^94, which is
// exact, and eps times 2^188; their squares then add up to less than 2^124.
constexpr float kTinyMean = 5.421010862427522e-20f;   // 2^-64
constexpr float kLift = 1.98070406285660844e28f;      // 2^94

// 1 / sqrt(mean); a row of zeros without an eps stays a row of zeros.
__device__ __forceinline__ float inverse_rms(float mean) { return mean == 0.0f ? 0.0f : 1.0f / sqrtf(mean); }

// TINY: a mean square below kTinyMean can occur.  An instance of its own: that
// branch costs 60000 unaligned rows of 2047 5% (273 us, 287 with it), 2000 rows of
// 40000 (norm_wide_kernel) 6% (367, 387).
template <typename TX, typename TR, bool E4M3, bool PHASED, bool TINY>
__global__ void __launch_bounds__(kMaxRowThreads)
    norm_row_kernel(const NormParams p) {
    __shared__ float shf[TINY ? 64 : 32];
    __shared__ uint32_t shu[32];
    griddep_launch_dependents();
    griddep_wait();
    const int n = static_cast<int>(p.width), t = threadIdx.x, threads = blockDim.x;
    const int warps = threads >> 5;
    const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= p.tokens) return;   // whole warps: a row's threads leave together
    const TX* x = static_cast<const TX*>(p.x) + row * p.x_stride;
    const int lead = PHASED ? row_lead(x) : 0;
    const bool inner = row > 0 && row + 1 < p.tokens && n >= 8;   // neighbours of a block or more
    float h[kHeld];
    load_row<PHASED>(x, n, lead, inner, t, threads, h);
    if (p.res) {
        float r[kHeld];
        load_row<PHASED>(static_cast<const TR*>(p.res) + row * p.res_stride, n, lead, inner, t, threads, r);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) h[i] += r[i];
        if (p.res_out)
            store_row<PHASED>(static_cast<TR*>(p.res_out) + row * p.res_out_stride, n, lead, t, threads, h);
    }
    auto mean_square = [&](float* sh) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const float s = h[i] * p.shrink;
            ss = fmaf(s, s, ss);
        }
        return row_sum(ss, warps, sh) * p.mean_of;
    };
    float mean = mean_square(shf) + p.eps;
    if (TINY && mean < kTinyMean) {   // the same for all of the row's threads
#pragma unroll
        for (int i = 0; i < kHeld; ++i) h[i] *= kLift;
        mean = mean_square(shf + 32) + p.eps * kLift * kLift;
    }
    const float rms = TINY ? inverse_rms(mean) : 1.0f / sqrtf(mean);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) h[i] *= rms;
    if (p.weight) {
        float w[kHeld];
        if (p.weight_dtype == kTokF32)
            load_row<PHASED>(static_cast<const float*>(p.weight), n, lead, false, t, threads, w);
        else
            load_row<PHASED>(static_cast<const TX*>(p.weight), n, lead, false, t, threads, w);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) h[i] *= w[i];
    }
    uint32_t top = row_max(held_max(h), warps, shu);
    if (!(mean <= kMaxFinite)) top = 0x7FC00000u;   // the mean square is not finite
    const float scale = row_scale(top, E4M3 ? 448.0f : 127.0f);
    store_codes<PHASED, E4M3>(p.q + row * p.q_stride, n, lead, t, threads, h, scale, row_blank(top));
    if (t == 0) p.scale[row] = scale;
}

// Rows that do not fit: read again for each pass (mean square, maximum, codes).
template <typename TX, typename TR, bool E4M3, bool TINY>
__global__ void __launch_bounds__(kMaxRowThreads)
    norm_wide_kernel(const NormParams p) {
    __shared__ float shf[TINY ? 64 : 32];
    __shared__ uint32_t shu[32];
    griddep_launch_dependents();
    griddep_wait();
    // unsigned: the last turn's index passes 2^31 where the width is near it
    const unsigned n = static_cast<unsigned>(p.width);
    const int warps = blockDim.x >> 5;
    const long long row = blockIdx.x;
    const TX* x = static_cast<const TX*>(p.x) + row * p.x_stride;
    const TR* r = p.res ? static_cast<const TR*>(p.res) + row * p.res_stride : nullptr;
    TR* ro = p.res_out ? static_cast<TR*>(p.res_out) + row * p.res_out_stride : nullptr;
    uint8_t* q = p.q + row * p.q_stride;
    auto h_at = [&](unsigned i) { return to_f32(x[i]) + (r ? to_f32(r[i]) : 0.0f); };
    auto mean_square = [&](float shrink, float* sh) {
        float ss = 0.0f;
        for (unsigned i = threadIdx.x; i < n; i += blockDim.x) {
            const float h = h_at(i) * shrink;
            ss = fmaf(h, h, ss);
        }
        return row_sum(ss, warps, sh) * p.mean_of;
    };
    float mean = mean_square(p.shrink, shf) + p.eps, lift = 1.0f;
    if (TINY && mean < kTinyMean) {
        lift = kLift;
        mean = mean_square(p.shrink * kLift, shf + 32) + p.eps * kLift * kLift;
    }
    const float rms = TINY ? inverse_rms(mean) : 1.0f / sqrtf(mean);
    auto v_of = [&](float h, unsigned i) {
        const float w = !p.weight ? 1.0f
                        : p.weight_dtype == kTokF32 ? static_cast<const float*>(p.weight)[i]
                                                    : to_f32(static_cast<const TX*>(p.weight)[i]);
        return (TINY ? h * lift : h) * rms * w;
    };
    uint32_t m = 0;
    for (unsigned i = threadIdx.x; i < n; i += blockDim.x) m = max(m, abs_bits(v_of(h_at(i), i)));
    uint32_t top = row_max(m, warps, shu);
    if (!(mean <= kMaxFinite)) top = 0x7FC00000u;   // the mean square is not finite
    const float scale = row_scale(top, E4M3 ? 448.0f : 127.0f);
    // each element is read before this thread writes it: residual_out may be an input
    for (unsigned i = threadIdx.x; i < n; i += blockDim.x) {
        const float h = h_at(i);
        q[i] = row_blank(top) ? 0 : static_cast<uint8_t>(code_of<E4M3>(v_of(h, i), scale));
        if (ro) ro[i] = from_f32<TR>(h);
    }
    if (threadIdx.x == 0) p.scale[row] = scale;
}

template <typename TX, typename TR, bool E4M3>
cudaError_t norm_launch(const NormParams& p, cudaStream_t stream) {
    const bool tiny = p.eps < kTinyMean;
    if (p.width > kMaxRowWidth) {
        auto kern = tiny ? norm_wide_kernel<TX, TR, E4M3, true> : norm_wide_kernel<TX, TR, E4M3, false>;
        return launch_ex(kern, static_cast<unsigned>(p.tokens), dim3(kMaxRowThreads), 0, 1, stream, p);
    }
    const int xb = elt_bytes(p.x_dtype), rb = elt_bytes(p.res_dtype);
    const bool inputs = p.width % 8 == 0 && aligned_rows(p.x, p.x_stride, p.tokens, xb, 16) &&
                      aligned_rows(p.res, p.res_stride, p.tokens, rb, 16) &&
                      aligned_rows(p.weight, 0, 1, 1, 16);
    const bool wide = inputs && aligned_rows(p.res_out, p.res_out_stride, p.tokens, rb, 16) &&
                      aligned_rows(p.q, p.q_stride, p.tokens, 1, 8);
    const dim3 block = row_block(p.width, inputs);
    const unsigned grid = row_blocks(p.tokens, block);
#define C3D_NORM(V, Y) launch_ex(norm_row_kernel<TX, TR, E4M3, V, Y>, grid, block, 0, 1, stream, p)
    if (tiny) return wide ? C3D_NORM(false, true) : C3D_NORM(true, true);
    return wide ? C3D_NORM(false, false) : C3D_NORM(true, false);
#undef C3D_NORM
}

template <typename TX>
cudaError_t norm_types(const NormParams& p, cudaStream_t stream) {
    const bool e4m3 = p.q_dtype == kTokE4m3;
    if (p.res && p.res_dtype == kTokF32)
        return e4m3 ? norm_launch<TX, float, true>(p, stream) : norm_launch<TX, float, false>(p, stream);
    return e4m3 ? norm_launch<TX, TX, true>(p, stream) : norm_launch<TX, TX, false>(p, stream);
}

}  // namespace

cudaError_t launch_norm_quant(const NormParams& p, cudaStream_t stream) {
    if (p.x_dtype == kTokBf16) return norm_types<__nv_bfloat16>(p, stream);
    if (p.x_dtype == kTokF16) return norm_types<__half>(p, stream);
    return norm_types<float>(p, stream);
}

}  // namespace c3d
