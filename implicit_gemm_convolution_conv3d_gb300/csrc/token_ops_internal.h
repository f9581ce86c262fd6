// token_ops_internal.h -- parameter blocks and launch entry points shared by
// token_api.cu and the token kernels.  Not part of the public ABI.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace c3d {

struct NormParams {
    const void* x;
    const void* res;      // NULL: no residual
    const void* weight;   // NULL: ones
    void* res_out;        // NULL: not stored
    uint8_t* q;
    float* scale;
    long long x_stride, res_stride, res_out_stride, q_stride;
    long long tokens, width;
    float eps;
    // the sum of squares is taken of h * shrink (a power of two near
    // 1/sqrt(width), so that it overflows only where the mean does) and the
    // mean is that sum * mean_of
    float shrink, mean_of;
    int x_dtype, res_dtype, weight_dtype, q_dtype;
};

struct ActParams {
    const void* x;
    uint8_t* q;
    float* scale;
    long long x_stride, q_stride;
    long long tokens, width;
    int x_dtype, q_dtype, act, gated;
};

struct LinearParams {
    // operands as the kernels read them: rows at 16-byte aligned pitches
    const uint8_t* x;
    const uint8_t* w;
    const float* scale_x;   // NULL: ones
    const float* scale_w;   // NULL: ones
    const float* bias;      // NULL: none
    void* out;
    long long x_stride, w_stride, out_stride;
    long long tokens, outputs, width;
    int e4m3, act, out_dtype;
    int* status;            // device status word and the bound on every wait
    unsigned long long wait_ns;
};

// How linear_w8a8_fwd runs a problem (plan_linear)
struct LinearPlan {
    int pair;               // CTA-pair kernel for many tokens, else the split kernel
    int tok_tile;           // split: tokens of a tile
    int tok_box, out_box;   // rows of a TMA box of either operand
    int out_tiles, tok_tiles;
    int splits;             // split: CTAs of a cluster that share a tile's reduction
    int stages, cvt_stages; // split: rings of TMA boxes and of converted (int8) operands
    int tma_out;            // pair: the output's rows can be stored by TMA
    int grid;               // pair: CTAs
    size_t smem;
};
// whether the pair form runs this product; its int8 weights are then f16 rows in
// the workspace (launch_stage_rows)
bool linear_pair_form(long long tokens, long long outputs);
// whether the form for few tokens runs it: any alignment, no tensor maps
bool linear_thin_form(long long tokens);
cudaError_t launch_linear_thin(const LinearParams& p, int num_sms, cudaStream_t stream);
cudaError_t plan_linear(const LinearParams& p, int num_sms, LinearPlan* plan);

struct LinearMaps {
    CUtensorMap x, w, out;  // out: pair kernel with tma_out only
};

cudaError_t launch_norm_quant(const NormParams& p, cudaStream_t stream);
cudaError_t launch_act_quant(const ActParams& p, cudaStream_t stream);
cudaError_t launch_linear(const LinearMaps& maps, const LinearParams& p, const LinearPlan& plan,
                          cudaStream_t stream);

// Rows of `cols` bytes, `stride` apart, to rows of `pitch` elements (a multiple of
// 16; dst 16-byte aligned) with zeros behind them: bytes, or f16 (widen, of int8).
// rows 0: no job.
struct RowJob {
    const uint8_t* src;
    uint8_t* dst;
    long long stride, rows, cols, pitch;
    int widen;
    int aligned, small;   // the rest is filled at launch
    FastDiv by_words;
};
struct RowJobs {
    RowJob job[2];
    unsigned blocks0;
};
cudaError_t launch_stage_rows(RowJobs jobs, cudaStream_t stream);

}  // namespace c3d
