// kv_cache.cu -- rows of keys and values into a paged cache and back.
//
// Writing takes each row's largest magnitude, scale = max / qmax, and stores the
// nearest codes (the rules of token_common.cuh: the same codes and scales as
// act_quant_fwd); reading multiplies codes by their scale and rounds once.
// Memory-bound: every row is read and written once.  A row is a group of 8, 16 or
// 32 lanes with 8 elements each, so a row's maximum takes three to five shuffles
// and nothing leaves the warp; keys and values are rows of one launch.
#include "attention_internal.h"
#include "paging.cuh"
#include "token_common.cuh"

namespace c3d {

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* src, int count, bool aligned, float (&v)[8]) {
    if (aligned && count >= 8) {
        constexpr int W = 16 / sizeof(T);
        alignas(16) T e[8];
#pragma unroll
        for (int i = 0; i < 8 / W; ++i)
            reinterpret_cast<uint4*>(e)[i] = reinterpret_cast<const uint4*>(src)[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < count ? to_f32(src[i]) : 0.0f;
    }
}

template <typename T>
__device__ __forceinline__ void store8(T* dst, int count, bool aligned, const float (&v)[8]) {
    alignas(16) T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(v[i]);
    if (aligned && count >= 8) {
        constexpr int W = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < 8 / W; ++i)
            reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(e)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < count) dst[i] = e[i];
    }
}

// The unit of a group of lanes: a token's key or value row of one head.  A warp's
// groups are neighbours; `first` is the warp's first unit.
struct Unit {
    long long token, pos;
    int head, value, sequence;
    bool in;   // belongs to a sequence
};

template <int G>
__device__ __forceinline__ Unit unit_of(const CacheParams& p, long long first) {
    Unit u;
    const int per = 2 * p.heads;
    const long long token0 = first / per;
    const uint32_t at = static_cast<uint32_t>(first - token0 * per) + (threadIdx.x & 31) / G;
    const uint32_t more = fdiv(at, p.by_units);
    const int k = static_cast<int>(at - more * per);
    u.token = token0 + more;
    u.value = k >= p.heads;
    u.head = u.value ? k - p.heads : k;
    u.in = u.token < p.tokens;
    if (!p.offsets) {
        u.sequence = static_cast<int>(u.token);
        u.pos = u.in ? p.starts[u.token] : 0;
        return u;
    }
    int s = find_sequence(p.offsets, p.sequences, token0);
    while (s + 1 < p.sequences && p.offsets[s + 1] <= u.token) ++s;
    u.sequence = s;
    const long long begin = p.offsets[s];
    u.in = u.in && u.token >= begin && u.token < p.offsets[s + 1];
    u.pos = u.token - begin + (p.starts && u.in ? p.starts[s] : 0);
    return u;
}

template <typename T, int CACHE, int G>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ CacheParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const long long first =
        (static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32) * (32 / G);
    const Unit u = unit_of<G>(p, first);
    const int e = (threadIdx.x % G) * 8;
    const int count = p.width - e;   // elements of this lane (0 or less: none)
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (u.in && count > 0)
        load8(reinterpret_cast<const T*>(u.value ? p.rows_v : p.rows_k) + u.token * p.tok_stride +
                  u.head * p.head_stride + e,
              count, p.aligned, v);
    long long row = 0, at = 0;
    const bool there = u.in && token_row(p.map, u.sequence, u.pos, u.head, &row, &at);
    unsigned char* dst = (u.value ? p.v : p.k) + row;
    if (CACHE == kTokBf16 || CACHE == kTokF16) {
        if (there && count > 0) store8(reinterpret_cast<T*>(dst) + e, 8, true, v);
    } else {
        constexpr bool E4 = CACHE == kTokE4m3;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, abs_bits(v[i]));
#pragma unroll
        for (int d = G / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        if (!there) return;
        const float scale = row_scale(top, E4 ? 448.0f : 127.0f);
        if (threadIdx.x % G == 0) (u.value ? p.v_scale : p.k_scale)[at] = scale;
        if (count <= 0) return;
        uint32_t w[2] = {0u, 0u};
        if (!row_blank(top)) {
            const float r = 1.0f / scale;
            const bool quick = quot_corrected_ok(scale);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float c = quick ? quot_corrected(v[i], scale, r) : v[i] / scale;
                const uint32_t b = E4 ? __nv_cvt_float_to_fp8(c, __NV_SATFINITE, __NV_E4M3)
                                      : static_cast<uint32_t>(__float2int_rn(c)) & 0xFFu;
                w[i / 4] |= b << (8 * (i % 4));
            }
        }
        *reinterpret_cast<uint2*>(dst + e) = make_uint2(w[0], w[1]);
    }
}

template <typename T, int CACHE, int G>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const long long first =
        (static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32) * (32 / G);
    const Unit u = unit_of<G>(p, first);
    const int e = (threadIdx.x % G) * 8;
    if (!u.in || e >= p.width) return;
    long long row = 0, at = 0;
    const bool there = token_row(p.map, u.sequence, u.pos, u.head, &row, &at);
    const unsigned char* src = (u.value ? p.v : p.k) + row;
    float v[8];
    if (!there) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(kNanBits);
    } else if (CACHE == kTokBf16) {
        load8(reinterpret_cast<const __nv_bfloat16*>(src) + e, 8, true, v);
    } else if (CACHE == kTokF16) {
        load8(reinterpret_cast<const __half*>(src) + e, 8, true, v);
    } else {
        const uint2 w = *reinterpret_cast<const uint2*>(src + e);
        const float scale = (u.value ? p.v_scale : p.k_scale)[at];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = ((i < 4 ? w.x : w.y) >> (8 * (i % 4))) & 0xFFu;
            if (CACHE == kTokE4m3)
                v[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3))) * scale;
            else
                v[i] = static_cast<float>(static_cast<signed char>(b)) * scale;
        }
    }
    store8(reinterpret_cast<T*>(u.value ? p.rows_v : p.rows_k) + u.token * p.tok_stride +
               u.head * p.head_stride + e,
           8, p.aligned, v);
}

template <typename T, int CACHE, bool WRITE>
cudaError_t by_width(CacheParams p, cudaStream_t stream) {
    const int g = p.width <= 64 ? 8 : p.width <= 128 ? 16 : 32;
    const long long units = p.tokens * 2 * p.heads;
    const long long per = (kThreads / 32) * (32 / g);
    const unsigned blocks = static_cast<unsigned>((units + per - 1) / per);
    p.by_units = make_fastdiv(static_cast<uint32_t>(2 * p.heads));
    auto go = [&](auto kern) { return launch_ex(kern, blocks, dim3(kThreads), 0, 1, stream, p); };
    if (WRITE)
        return g == 8 ? go(cache_write_kernel<T, CACHE, 8>)
                      : g == 16 ? go(cache_write_kernel<T, CACHE, 16>) : go(cache_write_kernel<T, CACHE, 32>);
    return g == 8 ? go(cache_read_kernel<T, CACHE, 8>)
                  : g == 16 ? go(cache_read_kernel<T, CACHE, 16>) : go(cache_read_kernel<T, CACHE, 32>);
}

template <typename T, bool WRITE>
cudaError_t by_cache(const CacheParams& p, int cache, cudaStream_t stream) {
    if (cache == kTokInt8) return by_width<T, kTokInt8, WRITE>(p, stream);
    if (cache == kTokE4m3) return by_width<T, kTokE4m3, WRITE>(p, stream);
    // unquantised rows are written as they are: the types are the same
    if (cache == kTokBf16) {
        if constexpr (WRITE) return by_width<__nv_bfloat16, kTokBf16, true>(p, stream);
        else return by_width<T, kTokBf16, false>(p, stream);
    }
    if constexpr (WRITE) return by_width<__half, kTokF16, true>(p, stream);
    else return by_width<T, kTokF16, false>(p, stream);
}

}  // namespace

cudaError_t launch_cache_write(const CacheParams& p, int row, int cache, cudaStream_t stream) {
    if (row == kTokBf16) return by_cache<__nv_bfloat16, true>(p, cache, stream);
    if (row == kTokF16) return by_cache<__half, true>(p, cache, stream);
    return by_cache<float, true>(p, cache, stream);
}

cudaError_t launch_cache_read(const CacheParams& p, int row, int cache, cudaStream_t stream) {
    if (row == kTokBf16) return by_cache<__nv_bfloat16, false>(p, cache, stream);
    if (row == kTokF16) return by_cache<__half, false>(p, cache, stream);
    return by_cache<float, false>(p, cache, stream);
}

}  // namespace c3d
