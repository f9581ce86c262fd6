// token_kv_cache.cu -- rows of keys and values into a paged cache and back.
//
// Writing takes each row's largest magnitude, scale = max / qmax, and stores the
// nearest codes (the rules of token_common.cuh: the same codes and scales as
// act_quant_fwd); reading multiplies codes by their scale and rounds once.
// Memory-bound: every row is read and written once.  To write, a row is a group of 8, 10,
// 16 or 32 lanes with 8 elements each, so a row's maximum takes three to five shuffles
// and nothing leaves the warp; keys and values are rows of one launch, and a group
// takes several of a token's rows at once.
// Measured: bf16 caches 6.5 TB/s both ways (108000 x 16 x 64; a copy runs at 6.8);
// 8 bits, 216000 x 8 x 128: reading 225 us (5.9 TB/s), writing 309 (4.3 TB/s: the maximum,
// two divisions a row and the codes' rounding are about 30 instructions for eight
// elements, and the issue slots what it waits for).  One new token of each of 64
// sequences: 8 us, the host's time for a call.
#include "token_attention_internal.h"
#include "token_paging.cuh"
#include "token_common.cuh"

#include <type_traits>

namespace c3d {

namespace {

constexpr int kThreads = 256;

// Eight elements of a row as they lie in memory.
template <typename T>
struct Raw {
    uint32_t w[2 * sizeof(T)];
};

template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* src, int count, bool aligned) {
    Raw<T> r;
    if (aligned) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
            const uint4 v = reinterpret_cast<const uint4*>(src)[i];
            r.w[4 * i] = v.x;
            r.w[4 * i + 1] = v.y;
            r.w[4 * i + 2] = v.z;
            r.w[4 * i + 3] = v.w;
        }
    } else {
        T* e = reinterpret_cast<T*>(r.w);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = i < count ? src[i] : from_f32<T>(0.0f);
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void widen8(const Raw<T>& r, float (&v)[8]) {
    const T* e = reinterpret_cast<const T*>(r.w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
}

template <typename T>
__device__ __forceinline__ void store8(T* dst, bool aligned, const float (&v)[8]) {
    alignas(16) T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(v[i]);
    if (aligned) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
            reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(e)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) dst[i] = e[i];
    }
}

// The unit of a group of G lanes: one of `parts` shares of a token's 2 * heads rows (the
// keys' heads, then the values').  One look at the offsets and the table serves it.
struct Unit {
    long long token, row, scale;   // row, scale: of head 0 in the pool
    int part;
    bool in, there;                // belongs to a sequence; has a page
};

template <int G>
__device__ __forceinline__ Unit unit_of(const CacheParams& p) {
    const long long first =
        (static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32) * (32 / G);
    Unit u;
    const long long token0 = first / p.parts;
    const uint32_t group = (threadIdx.x & 31) / G;
    const uint32_t at = static_cast<uint32_t>(first - token0 * p.parts) + group;
    const uint32_t more = fdiv(at, p.by_parts);
    u.token = token0 + more;
    u.part = static_cast<int>(at - more * p.parts);
    u.in = u.token < p.tokens && group < 32 / G;   // (ten lanes a row leave two over)
    u.row = u.scale = 0;
    long long sequence = u.token, pos = 0;
    if (!p.offsets) {
        if (u.in) pos = p.starts[u.token];
    } else {
        int s = find_sequence(p.offsets, p.sequences, token0);
        while (s + 1 < p.sequences && p.offsets[s + 1] <= u.token) ++s;
        const long long begin = p.offsets[s], end = p.offsets[s + 1];
        u.in = u.in && u.token >= begin && u.token < end;
        sequence = s;
        pos = u.token - begin + (p.starts ? p.starts[s] : 0);
    }
    u.there = u.in && token_row(p.map, sequence, pos, 0, &u.row, &u.scale);
    return u;
}

// The largest magnitude of eight elements, as fp32 bits that order like it (abs_bits).
template <typename T>
__device__ __forceinline__ uint32_t top_of(const Raw<T>& r) {
    if constexpr (sizeof(T) == 4) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, r.w[i] & 0x7FFFFFFFu);
        return top;
    } else {
        // magnitudes of 16-bit floats order like their bits, two at a time
        uint32_t m = r.w[0] & 0x7FFF7FFFu;
#pragma unroll
        for (int i = 1; i < 4; ++i) m = __vmaxu2(m, r.w[i] & 0x7FFF7FFFu);
        const uint32_t top = max(m & 0xFFFFu, m >> 16);
        if constexpr (std::is_same<T, __half>::value)
            return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(top))));
        return top << 16;
    }
}

// Two quotients by one scale, rounded once (quot_corrected's steps, two values an
// instruction); the sign of a zero quotient is put back for e4m3, which has one.
template <bool E4>
__device__ __forceinline__ float2 quotients(float x, float y, float scale, float inv, bool quick) {
    if (!quick) return make_float2(x / scale, y / scale);
    float2 q;
    asm("{\n\t.reg .b64 v, s, r, q;\n\t"
        "mov.b64 v, {%2, %3};\n\tmov.b64 s, {%4, %4};\n\tmov.b64 r, {%5, %5};\n\t"
        "mul.rn.f32x2 q, v, r;\n\t"
        "fma.rn.f32x2 s, s, q, v;\n\t"
        "fma.rn.f32x2 q, s, r, q;\n\t"
        "mov.b64 {%0, %1}, q;\n\t}"
        : "=f"(q.x), "=f"(q.y)
        : "f"(x), "f"(y), "f"(-scale), "f"(inv));
    if (E4) {
        q.x = __uint_as_float(__float_as_uint(q.x) | (__float_as_uint(x) & 0x80000000u));
        q.y = __uint_as_float(__float_as_uint(q.y) | (__float_as_uint(y) & 0x80000000u));
    }
    return q;
}

// G lanes a row: 8, 10, 16 or 32.  A lane's rows are reduced side by side; lane r of the
// group then takes row r's two divisions for all.
template <typename T, int CACHE, int G, int R>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ CacheParams p) {
    static_assert(R <= G, "a lane for each row's scale");
    griddep_launch_dependents();
    griddep_wait();
    const Unit u = unit_of<G>(p);
    const int lane = threadIdx.x & 31, in_row = lane % G, e = in_row * 8;
    const bool mine = u.there && e < p.width;
    Raw<T> raw[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = u.part + r * p.parts;
#pragma unroll
        for (int i = 0; i < static_cast<int>(2 * sizeof(T)); ++i) raw[r].w[i] = 0u;
        if (!mine || row >= 2 * p.heads) continue;
        const bool value = row >= p.heads;
        const T* src = reinterpret_cast<const T*>(value ? p.rows_v : p.rows_k) + u.token * p.tok_stride +
                       (value ? row - p.heads : row) * p.head_stride + e;
        raw[r] = load_raw(src, p.width - e, p.aligned);
    }
    if (CACHE == kTokBf16 || CACHE == kTokF16) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = u.part + r * p.parts;
            if (!mine || row >= 2 * p.heads) continue;
            const bool value = row >= p.heads;
            unsigned char* dst = (value ? p.v : p.k) + u.row + (value ? row - p.heads : row) * p.map.head_stride;
            reinterpret_cast<uint4*>(dst)[in_row] = make_uint4(raw[r].w[0], raw[r].w[1], raw[r].w[2], raw[r].w[3]);
        }
        return;
    }
    constexpr bool E4 = CACHE == kTokE4m3;
    uint32_t top[R];
#pragma unroll
    for (int r = 0; r < R; ++r) top[r] = top_of(raw[r]);
    constexpr int kReach = G == 32 ? 16 : G > 8 ? 8 : 4;
#pragma unroll
    for (int d = kReach; d > 0; d >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t o = __shfl_down_sync(0xffffffffu, top[r], d);
            if (in_row + d < G) top[r] = max(top[r], o);
        }
    // lane r of the group: row r
    uint32_t own = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t t = __shfl_sync(0xffffffffu, top[r], lane - in_row);
        if (in_row == r) own = t;
    }
    const float own_scale = row_scale(own, E4 ? 448.0f : 127.0f);
    // 0 for a row that is blank
    const float own_inv = row_blank(own) ? 0.0f : 1.0f / own_scale;
    {
        const int row = u.part + in_row * p.parts;
        if (u.there && in_row < R && row < 2 * p.heads) {
            const bool value = row >= p.heads;
            (value ? p.v_scale : p.k_scale)[u.scale + (value ? row - p.heads : row) * p.map.scale_head_stride] =
                own_scale;
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float scale = __shfl_sync(0xffffffffu, own_scale, lane - in_row + r);
        const float inv = __shfl_sync(0xffffffffu, own_inv, lane - in_row + r);
        const int row = u.part + r * p.parts;
        if (!mine || row >= 2 * p.heads) continue;
        const bool value = row >= p.heads;
        unsigned char* dst = (value ? p.v : p.k) + u.row + (value ? row - p.heads : row) * p.map.head_stride;
        uint32_t w[2] = {0u, 0u};
        if (inv != 0.0f) {
            float v[8];
            widen8(raw[r], v);
            const bool quick = quot_corrected_ok(scale);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 q = quotients<E4>(v[i], v[i + 1], scale, inv, quick);
                // int8: nearest (ties to even) by the addition of 1.5 * 2^23, |q| <= 127.5
                const uint32_t b = E4 ? __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3)
                                      : __byte_perm(__float_as_uint(q.x + 12582912.0f),
                                                    __float_as_uint(q.y + 12582912.0f), 0x0040);
                w[i / 4] = i % 4 == 0 ? b : __byte_perm(w[i / 4], b, 0x5410);
            }
        }
        *reinterpret_cast<uint2*>(dst + e) = make_uint2(w[0], w[1]);
    }
}

// Eight codes (or 16-bit elements) as fp32, times their scale
template <int CACHE>
__device__ __forceinline__ void values8(const uint32_t (&w)[4], float scale, float (&v)[8]) {
    if (CACHE == kTokBf16 || CACHE == kTokF16) {
        Raw<__half> r{{w[0], w[1], w[2], w[3]}};
        if (CACHE == kTokF16) widen8(r, v);
        else widen8(*reinterpret_cast<Raw<__nv_bfloat16>*>(&r), v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint32_t b = w[i / 4] >> (8 * (i % 4));
        if (CACHE == kTokE4m3) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(b), __NV_E4M3);
            const float2 f = __half22float2(__half2(h));
            v[i] = f.x * scale;
            v[i + 1] = f.y * scale;
        } else {
            // 2^23 + 128 + code as fp32 bits, less 2^23 + 128
            const uint32_t o = b ^ 0x8080u;
            v[i] = (__uint_as_float(__byte_perm(o, 0x4B000000u, 0x7440)) - 8388736.0f) * scale;
            v[i + 1] = (__uint_as_float(__byte_perm(o, 0x4B000000u, 0x7441)) - 8388736.0f) * scale;
        }
    }
}

// A share is every parts * G-th run of eight elements of the token's rows, so that lanes
// take neighbours whatever the width is; up to R of them a lane.
template <typename T, int CACHE, int G, int R>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 4 : 5) cache_read_kernel(const __grid_constant__ CacheParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const Unit u = unit_of<G>(p);
    if (!u.in) return;
    constexpr bool kCodes = CACHE == kTokInt8 || CACHE == kTokE4m3;
    const int runs = p.width / 8, all = 2 * p.heads * runs;
    const int first = u.part * G + threadIdx.x % G, step = p.parts * G;
    // the first one's row and element; the next is `rows` rows and `on` elements further
    const int row0 = fdiv(first, p.by_runs), e0 = (first - row0 * runs) * 8;
    const int rows = fdiv(step, p.by_runs), on = (step - rows * runs) * 8;
    uint32_t w[R][4];
    float scale[R];
    int row = row0, e = e0;
    auto next = [&]() {
        row += rows;
        e += on;
        if (e >= p.width) {
            e -= p.width;
            ++row;
        }
    };
#pragma unroll
    for (int r = 0; r < R; ++r, next()) {
        if (!u.there || first + r * step >= all) continue;
        const bool value = row >= p.heads;
        const int head = value ? row - p.heads : row;
        const unsigned char* src = (value ? p.v : p.k) + u.row + head * p.map.head_stride;
        if (kCodes) {
            const uint2 c = *reinterpret_cast<const uint2*>(src + e);
            w[r][0] = c.x;
            w[r][1] = c.y;
            scale[r] = (value ? p.v_scale : p.k_scale)[u.scale + head * p.map.scale_head_stride];
        } else {
            const uint4 c = *reinterpret_cast<const uint4*>(src + 2 * e);
            w[r][0] = c.x;
            w[r][1] = c.y;
            w[r][2] = c.z;
            w[r][3] = c.w;
        }
    }
    row = row0;
    e = e0;
#pragma unroll
    for (int r = 0; r < R; ++r, next()) {
        if (first + r * step >= all) break;
        const bool value = row >= p.heads;
        float v[8];
        if (u.there) {
            values8<CACHE>(w[r], kCodes ? scale[r] : 1.0f, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(kNanBits);
        }
        store8(reinterpret_cast<T*>(value ? p.rows_v : p.rows_k) + u.token * p.tok_stride +
                   (value ? row - p.heads : row) * p.head_stride + e,
               p.aligned, v);
    }
}

template <typename Kernel>
cudaError_t run(Kernel kern, CacheParams p, int parts, int lanes, cudaStream_t stream) {
    p.parts = parts;
    p.by_parts = make_fastdiv(static_cast<uint32_t>(parts));
    p.by_runs = make_fastdiv(static_cast<uint32_t>(p.width / 8));
    const long long units = p.tokens * parts, per = kThreads / 32 * (32 / lanes);
    return launch_ex(kern, static_cast<unsigned>((units + per - 1) / per), dim3(kThreads), 0, 1, stream, p);
}

// Several rows a lane where that leaves the SMs two blocks each: their loads are in flight
// together behind one look at the table.  Eight, or four where that wastes fewer lanes'
// rows (2, 4, 10 or 12 rows a token) and of fp32, for the registers.  216000 tokens x 8
// heads x 128, e4m3: 309 us with eight, 332 with four, 611 with one; 108000 x 1 x 128: 60, 43
// and 50; 64 x 8 x 128 (too few): 10.2 with eight, 8.2 with one.
template <typename T, int CACHE, int G>
cudaError_t write_by_rows(const CacheParams& p, cudaStream_t stream) {
    const int rows = 2 * p.heads;
    const bool eight = sizeof(T) < 4 && (rows + 7) / 8 * 8 == (rows + 3) / 4 * 4;
    const bool many = p.tokens * rows / (eight ? 8 : 4) * G >= 2 * 152 * kThreads;
    if (!many) return run(cache_write_kernel<T, CACHE, G, 1>, p, rows, G, stream);
    if constexpr (sizeof(T) < 4)
        if (eight) return run(cache_write_kernel<T, CACHE, G, 8>, p, (rows + 7) / 8, G, stream);
    return run(cache_write_kernel<T, CACHE, G, 4>, p, (rows + 3) / 4, G, stream);
}

// Reads: up to eight runs of elements a lane (four of 16-bit ones, for the registers), as
// above: 216000 x 8 x 128, e4m3: 225 us, 254 with four, 453 with one.  Eight lanes share a
// token's runs: 32 took 182 us for 108000 x 16 x 80 int8 where eight take 158, and twice as
// long for one or two heads.
template <typename T, int CACHE>
cudaError_t read_by_runs(const CacheParams& p, cudaStream_t stream) {
    constexpr int G = 8, kMany = CACHE == kTokInt8 || CACHE == kTokE4m3 ? 8 : 4;
    const int runs = 2 * p.heads * (p.width / 8);
    const bool many = p.tokens * runs / kMany >= 2 * 152 * kThreads;
    return many ? run(cache_read_kernel<T, CACHE, G, kMany>, p, (runs + kMany * G - 1) / (kMany * G), G, stream)
                : run(cache_read_kernel<T, CACHE, G, 1>, p, (runs + G - 1) / G, G, stream);
}

// Lanes of a written row: the fewest that hold it, eight elements each.  (80-wide rows in 16
// lanes: 310 us where ten lanes take 215, 108000 x 16 x 80 int8.)
template <typename T, int CACHE, bool WRITE>
cudaError_t by_width(const CacheParams& p, cudaStream_t stream) {
    if constexpr (WRITE)
        return p.width <= 64    ? write_by_rows<T, CACHE, 8>(p, stream)
               : p.width <= 80  ? write_by_rows<T, CACHE, 10>(p, stream)
               : p.width <= 128 ? write_by_rows<T, CACHE, 16>(p, stream)
                                : write_by_rows<T, CACHE, 32>(p, stream);
    else
        return read_by_runs<T, CACHE>(p, stream);
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
