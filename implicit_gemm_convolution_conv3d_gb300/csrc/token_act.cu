// token_act.cu -- the (gated) activation with an 8-bit output:
//
//   v = act(x), or act(gate) * value for a row [gate | value]
//   scale = max|v| / qmax;  q = nearest code of v / scale
//
// Read once, held in registers for the row's maximum, written as codes: 3 bytes an
// element for 16-bit inputs, 5 gated.  Bound by memory and, with SiLU or GELU, by
// issue slots: 16384 x 4096 gated silu 64 us (5.3 TB/s), 9500 x 5120 gelu 46 us, none
// 26 us (5.6 TB/s).
#include <cuda_runtime.h>

#include "token_ops_internal.h"
#include "token_rows.cuh"

namespace c3d {

namespace {

template <typename TX, int ACT, bool GATED, bool E4M3, bool PHASED>
__global__ void __launch_bounds__(kMaxRowThreads)
    act_row_kernel(const ActParams p) {
    __shared__ uint32_t shu[32];
    griddep_launch_dependents();
    griddep_wait();
    const int n = static_cast<int>(p.width), t = threadIdx.x, threads = blockDim.x;
    const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= p.tokens) return;   // whole warps: a row's threads leave together
    const TX* x = static_cast<const TX*>(p.x) + row * p.x_stride;
    const int lead = PHASED ? row_lead(x) : 0;
    const bool inner = row > 0 && row + 1 < p.tokens && n >= 8;   // neighbours of a block or more
    float v[kHeld];
    load_row<PHASED>(x, n, lead, inner, t, threads, v);
    float b[GATED ? kHeld : 1];
    if constexpr (GATED) load_row<PHASED>(x + n, n, lead, inner, t, threads, b);
    // SiLU and GELU of -inf are NaN: kept as a sum of 0 * x beside them, half an
    // instruction an element (inside them the gated instances spill)
    constexpr bool kTails = ACT == kActSilu || ACT == kActGelu;
    float2 spoilt = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kHeld; i += 2) {
        if (kTails) spoilt = __ffma2_rn(make_float2(v[i], v[i + 1]), make_float2(0.0f, 0.0f), spoilt);
        const float2 y = act2<ACT>(make_float2(v[i], v[i + 1]));
        v[i] = y.x;
        v[i + 1] = y.y;
    }
    if (GATED) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) v[i] *= b[i];
    }
    const uint32_t top = row_max(isnan(spoilt.x + spoilt.y) ? kNanBits : held_max(v), threads >> 5, shu);
    const float scale = row_scale(top, E4M3 ? 448.0f : 127.0f);
    store_codes<PHASED, E4M3>(p.q + row * p.q_stride, n, lead, t, threads, v, scale, row_blank(top));
    if (t == 0) p.scale[row] = scale;
}

// Rows that do not fit: read twice; two elements a turn where the activation's
// arithmetic is two-wide (one else: 2000 x 40000 none 155 us against 212).
template <typename TX, int ACT, bool E4M3>
__global__ void __launch_bounds__(kMaxRowThreads)
    act_wide_kernel(const ActParams p) {
    __shared__ uint32_t shu[32];
    griddep_launch_dependents();
    griddep_wait();
    const long long n = p.width, row = blockIdx.x;
    const TX* x = static_cast<const TX*>(p.x) + row * p.x_stride;
    uint8_t* q = p.q + row * p.q_stride;
    constexpr bool kTails = ACT == kActSilu || ACT == kActGelu;
    const int pace = blockDim.x, turn = kTails ? 2 * pace : pace;
    auto v_at = [&](long long i) {   // elements i and (kTails; zero behind the row) i + pace
        const bool two = kTails && i + pace < n;
        const float2 x2 = make_float2(to_f32(x[i]), two ? to_f32(x[i + pace]) : 0.0f);
        float2 v = act2<ACT>(x2);
        if (kTails) v = __ffma2_rn(x2, make_float2(0.0f, 0.0f), v);   // NaN of +-inf
        if (p.gated) {
            v.x *= to_f32(x[n + i]);
            if (two) v.y *= to_f32(x[n + i + pace]);
        }
        return v;
    };
    uint32_t m = 0;
    for (long long i = threadIdx.x; i < n; i += turn) {
        const float2 v = v_at(i);
        m = max(m, max(abs_bits(v.x), abs_bits(v.y)));
    }
    const uint32_t top = row_max(m, blockDim.x >> 5, shu);
    const float scale = row_scale(top, E4M3 ? 448.0f : 127.0f);
    for (long long i = threadIdx.x; i < n; i += turn) {
        const float2 v = v_at(i);
        q[i] = row_blank(top) ? 0 : static_cast<uint8_t>(code_of<E4M3>(v.x, scale));
        if (kTails && i + pace < n) q[i + pace] = row_blank(top) ? 0 : static_cast<uint8_t>(code_of<E4M3>(v.y, scale));
    }
    if (threadIdx.x == 0) p.scale[row] = scale;
}

template <typename TX, int ACT, bool E4M3>
cudaError_t act_launch(const ActParams& p, cudaStream_t stream) {
    if (p.width > kMaxRowWidth)
        return launch_ex(act_wide_kernel<TX, ACT, E4M3>, static_cast<unsigned>(p.tokens),
                         dim3(kMaxRowThreads), 0, 1, stream, p);
    const int xb = elt_bytes(p.x_dtype);
    const bool inputs = p.width % 8 == 0 && aligned_rows(p.x, p.x_stride, p.tokens, xb, 16);
    const bool wide = inputs && aligned_rows(p.q, p.q_stride, p.tokens, 1, 8);
    const dim3 block = row_block(p.width, inputs);
    const unsigned grid = row_blocks(p.tokens, block);
#define C3D_ACT(G, V) launch_ex(act_row_kernel<TX, ACT, G, E4M3, V>, grid, block, 0, 1, stream, p)
    if (p.gated) return wide ? C3D_ACT(true, false) : C3D_ACT(true, true);
    return wide ? C3D_ACT(false, false) : C3D_ACT(false, true);
#undef C3D_ACT
}

template <typename TX, bool E4M3>
cudaError_t act_kind(const ActParams& p, cudaStream_t stream) {
    if (p.act == kActRelu) return act_launch<TX, kActRelu, E4M3>(p, stream);
    if (p.act == kActSilu) return act_launch<TX, kActSilu, E4M3>(p, stream);
    if (p.act == kActGelu) return act_launch<TX, kActGelu, E4M3>(p, stream);
    return act_launch<TX, kActNone, E4M3>(p, stream);
}

template <typename TX>
cudaError_t act_types(const ActParams& p, cudaStream_t stream) {
    return p.q_dtype == kTokE4m3 ? act_kind<TX, true>(p, stream) : act_kind<TX, false>(p, stream);
}

}  // namespace

cudaError_t launch_act_quant(const ActParams& p, cudaStream_t stream) {
    if (p.x_dtype == kTokBf16) return act_types<__nv_bfloat16>(p, stream);
    if (p.x_dtype == kTokF16) return act_types<__half>(p, stream);
    return act_types<float>(p, stream);
}

}  // namespace c3d
