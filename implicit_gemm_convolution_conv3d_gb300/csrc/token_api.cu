// token_api.cu -- the C ABI of the token operators (declared in
// include/token_ops.h): argument checks and launches.  No allocation.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdio>

#include "internal.h"
#include "token_common.cuh"
#include "token_ops.h"
#include "token_ops_internal.h"

namespace c3d {

namespace {

constexpr int64_t kMaxDim = (1ll << 31) - 1;

int invalid(const char* what) {
    set_last_error(what);
    return CONV_ERR_INVALID;
}

int launched(cudaError_t e, const char* where) {
    if (e == cudaSuccess) return CONV_OK;
    char msg[160];
    std::snprintf(msg, sizeof msg, "%s: %s", where, cudaGetErrorString(e));
    set_last_error(msg);
    return CONV_ERR_CUDA;
}

bool is_float_type(int t) { return t == CONV_DTYPE_BF16 || t == CONV_DTYPE_F16 || t == CONV_DTYPE_F32; }
bool is_code_type(int t) { return t == CONV_DTYPE_INT8 || t == CONV_DTYPE_FP8_E4M3; }
int size_of(int t) {
    return t == CONV_DTYPE_F32 ? 4 : t == CONV_DTYPE_BF16 || t == CONV_DTYPE_F16 ? 2 : 1;
}
bool aligned_to(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) % bytes) == 0; }

// the checks that every matrix of rows shares
const char* bad_rows(const void* p, int64_t stride, int64_t row, int64_t rows, int elt) {
    if (!p) return "null pointer";
    if (stride < row && rows > 1) return "a row stride is below the row's length";
    if (!aligned_to(p, elt)) return "a pointer is not aligned to its element type";
    return nullptr;
}

long long round16(int64_t b) { return (b + 15) / 16 * 16; }

// whether TMA can address these rows (one row has no stride to align)
bool tma_rows(const void* p, int64_t stride, int64_t rows) {
    return aligned_to(p, 16) && (rows == 1 || stride % 16 == 0);
}

}  // namespace

}  // namespace c3d

using namespace c3d;

extern "C" {

int rms_norm_quant_fwd(const void* x, int x_dtype, int64_t x_stride, const void* residual,
                       int res_dtype, int64_t res_stride, const void* weight, int weight_dtype,
                       float eps, int64_t tokens, int64_t width, int q_dtype, void* q,
                       int64_t q_stride, float* scale, void* residual_out,
                       int64_t res_out_stride, cudaStream_t stream) {
    if (tokens < 0 || tokens > kMaxDim || width < 1 || width > kMaxDim)
        return invalid("tokens must be 0 or more and width 1 or more, below 2^31");
    if (!is_float_type(x_dtype)) return invalid("x_dtype must be BF16, F16 or F32");
    if (!is_code_type(q_dtype)) return invalid("q_dtype must be INT8 or FP8_E4M3");
    if (residual && res_dtype != x_dtype && res_dtype != CONV_DTYPE_F32)
        return invalid("res_dtype must be x_dtype or F32");
    if (weight && weight_dtype != x_dtype && weight_dtype != CONV_DTYPE_F32)
        return invalid("weight_dtype must be x_dtype or F32");
    if (residual_out && !residual) return invalid("residual_out needs a residual");
    if (!(eps >= 0.0f)) return invalid("eps must be 0 or more");
    if (tokens == 0) return CONV_OK;
    if (const char* e = bad_rows(x, x_stride, width, tokens, size_of(x_dtype))) return invalid(e);
    if (const char* e = bad_rows(q, q_stride, width, tokens, 1)) return invalid(e);
    if (const char* e = bad_rows(scale, 1, 1, tokens, 4)) return invalid(e);
    if (residual)
        if (const char* e = bad_rows(residual, res_stride, width, tokens, size_of(res_dtype)))
            return invalid(e);
    if (residual_out)
        if (const char* e = bad_rows(residual_out, res_out_stride, width, tokens, size_of(res_dtype)))
            return invalid(e);
    if (weight && !aligned_to(weight, size_of(weight_dtype)))
        return invalid("a pointer is not aligned to its element type");
    NormParams p{};
    p.x = x;
    p.res = residual;
    p.weight = weight;
    p.res_out = residual_out;
    p.q = static_cast<uint8_t*>(q);
    p.scale = scale;
    p.x_stride = x_stride;
    p.res_stride = res_stride;
    p.res_out_stride = res_out_stride;
    p.q_stride = q_stride;
    p.tokens = tokens;
    p.width = width;
    p.eps = eps;
    p.shrink = 1.0f;
    while (static_cast<double>(p.shrink) * p.shrink * static_cast<double>(width) > 1.0) p.shrink *= 0.5f;
    p.mean_of = static_cast<float>(
        1.0 / (static_cast<double>(p.shrink) * p.shrink * static_cast<double>(width)));
    p.x_dtype = x_dtype;
    p.res_dtype = residual ? res_dtype : x_dtype;
    p.weight_dtype = weight ? weight_dtype : x_dtype;
    p.q_dtype = q_dtype;
    return launched(launch_norm_quant(p, stream), "rms_norm_quant_fwd launch");
}

int act_quant_fwd(const void* x, int x_dtype, int64_t x_stride, int act, int gated,
                  int64_t tokens, int64_t width, int q_dtype, void* q, int64_t q_stride,
                  float* scale, cudaStream_t stream) {
    if (tokens < 0 || tokens > kMaxDim || width < 1 || width > kMaxDim / 2)
        return invalid("tokens must be 0 or more and width 1 or more, below 2^31 (2^30)");
    if (!is_float_type(x_dtype)) return invalid("x_dtype must be BF16, F16 or F32");
    if (!is_code_type(q_dtype)) return invalid("q_dtype must be INT8 or FP8_E4M3");
    if (act < CONV_ACT_NONE || act > CONV_ACT_GELU) return invalid("unknown activation");
    if (tokens == 0) return CONV_OK;
    if (const char* e = bad_rows(x, x_stride, gated ? 2 * width : width, tokens, size_of(x_dtype)))
        return invalid(e);
    if (const char* e = bad_rows(q, q_stride, width, tokens, 1)) return invalid(e);
    if (const char* e = bad_rows(scale, 1, 1, tokens, 4)) return invalid(e);
    ActParams p{};
    p.x = x;
    p.q = static_cast<uint8_t*>(q);
    p.scale = scale;
    p.x_stride = x_stride;
    p.q_stride = q_stride;
    p.tokens = tokens;
    p.width = width;
    p.x_dtype = x_dtype;
    p.q_dtype = q_dtype;
    p.act = act;
    p.gated = gated != 0;
    return launched(launch_act_quant(p, stream), "act_quant_fwd launch");
}

size_t linear_w8a8_workspace_size(const void* x, int64_t x_stride, const void* w,
                                  int64_t w_stride, int dtype, int64_t tokens, int64_t outputs,
                                  int64_t width) {
    if (tokens < 1 || outputs < 1 || width < 1 || linear_thin_form(tokens)) return 0;
    const size_t pitch = static_cast<size_t>(round16(width));
    const bool widen = dtype == CONV_DTYPE_INT8 && linear_pair_form(tokens, outputs);
    return (tma_rows(x, x_stride, tokens) ? 0 : pitch * static_cast<size_t>(tokens)) +
           (widen ? 2 : tma_rows(w, w_stride, outputs) ? 0 : 1) * pitch * static_cast<size_t>(outputs);
}

int linear_w8a8_fwd(const void* x, int64_t x_stride, const void* w, int64_t w_stride, int dtype,
                    int64_t tokens, int64_t outputs, int64_t width, const float* scale_x,
                    const float* scale_w, const float* bias, int act, void* out, int out_dtype,
                    int64_t out_stride, void* workspace, size_t workspace_bytes,
                    cudaStream_t stream) {
    if (tokens < 0 || tokens > kMaxDim || outputs < 0 || outputs > kMaxDim || width < 1 ||
        width > kMaxDim)
        return invalid("tokens and outputs must be 0 or more and width 1 or more, below 2^31");
    if (!is_code_type(dtype)) return invalid("dtype must be INT8 or FP8_E4M3");
    if (!is_float_type(out_dtype)) return invalid("out_dtype must be BF16, F16 or F32");
    if (act < CONV_ACT_NONE || act > CONV_ACT_GELU) return invalid("unknown activation");
    if (tokens == 0 || outputs == 0) return CONV_OK;
    if (const char* e = bad_rows(x, x_stride, width, tokens, 1)) return invalid(e);
    if (const char* e = bad_rows(w, w_stride, width, outputs, 1)) return invalid(e);
    if (const char* e = bad_rows(out, out_stride, outputs, tokens, size_of(out_dtype)))
        return invalid(e);
    if (!aligned_to(scale_x, 4) || !aligned_to(scale_w, 4) || !aligned_to(bias, 4))
        return invalid("a pointer is not aligned to its element type");
    LinearParams p{};
    p.x = static_cast<const uint8_t*>(x);
    p.w = static_cast<const uint8_t*>(w);
    p.scale_x = scale_x;
    p.scale_w = scale_w;
    p.bias = bias;
    p.out = out;
    p.x_stride = x_stride;
    p.w_stride = w_stride;
    p.out_stride = out_stride;
    p.tokens = tokens;
    p.outputs = outputs;
    p.width = width;
    p.e4m3 = dtype == CONV_DTYPE_FP8_E4M3;
    p.act = act;
    p.out_dtype = out_dtype;
    const size_t need =
        linear_w8a8_workspace_size(x, x_stride, w, w_stride, dtype, tokens, outputs, width);
    if (need && (!workspace || workspace_bytes < need || !aligned_to(workspace, 16)))
        return invalid("this product needs a 16-byte aligned workspace of "
                       "linear_w8a8_workspace_size bytes");
    LaunchLimits lim;
    int rc = launch_limits(&lim);
    if (rc) return rc;
    p.status = lim.status;
    p.wait_ns = lim.wait_ns;
    if (linear_thin_form(tokens))
        return launched(launch_linear_thin(p, lim.num_sms, stream), "linear_w8a8_fwd launch");
    // operands that TMA cannot address are copied to an aligned pitch first, and
    // the pair form's int8 weights are widened to f16
    const bool widen = !p.e4m3 && linear_pair_form(tokens, outputs);
    const bool copy_x = !tma_rows(x, x_stride, tokens);
    const bool copy_w = !widen && !tma_rows(w, w_stride, outputs);
    const long long pitch = round16(width);
    uint8_t* at = static_cast<uint8_t*>(workspace);
    const uint8_t *src_x = p.x, *src_w = p.w;
    if (copy_x) {
        p.x = at;
        at += pitch * tokens;
    }
    if (copy_w || widen) p.w = at;
    p.x_stride = copy_x || tokens == 1 ? pitch : x_stride;
    p.w_stride = copy_w || widen || outputs == 1 ? pitch : w_stride;
    LinearPlan plan;
    if ((rc = launched(plan_linear(p, lim.num_sms, &plan), "linear_w8a8_fwd plan"))) return rc;
    const long long tiles = static_cast<long long>(plan.out_tiles) * plan.tok_tiles * plan.splits;
    const long long pairs = plan.pair ? plan.grid / 2 : 1;   // each counts its k-steps in 32 bits
    if (tiles > kMaxDim || (plan.pair && (tiles / pairs + 1) * ((width + 127) / 128) > kMaxDim)) {
        set_last_error("the output has more tiles than the kernels count");
        return CONV_ERR_UNSUPPORTED;
    }
    const long long elt = size_of(out_dtype);
    // TMA stores whole 16-byte words: an output row's last one has to be its own
    plan.tma_out = aligned_to(out, 16) && out_stride * elt % 16 == 0 && outputs * elt % 16 == 0;
    LinearMaps maps{};
    if ((rc = encode_rows(&maps.x, p.x, 1, width, tokens, p.x_stride, plan.tok_box, 128))) return rc;
    if ((rc = encode_rows(&maps.w, p.w, widen ? 2 : 1, width, outputs, p.w_stride * (widen ? 2 : 1),
                          plan.out_box, 128)))
        return rc;
    if (plan.pair && plan.tma_out &&
        (rc = encode_rows(&maps.out, out, static_cast<int>(elt), outputs, tokens, out_stride * elt, 32, 64)))
        return rc;
    cudaError_t e = cudaSuccess;
    if (copy_x || copy_w || widen) {
        RowJobs jobs{};
        if (copy_x)
            jobs.job[0] = RowJob{src_x, const_cast<uint8_t*>(p.x), x_stride, tokens, width, pitch, 0, 0, 0, {}};
        if (copy_w || widen)
            jobs.job[1] = RowJob{src_w, const_cast<uint8_t*>(p.w), w_stride, outputs, width, pitch, widen, 0, 0, {}};
        e = launch_stage_rows(jobs, stream);
    }
    if (e == cudaSuccess) e = launch_linear(maps, p, plan, stream);
    return launched(e, "linear_w8a8_fwd launch");
}

}  // extern "C"
