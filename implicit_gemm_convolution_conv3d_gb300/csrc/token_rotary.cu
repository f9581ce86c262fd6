// token_rotary.cu -- rotary positions with several axes (time, height, width).
//
// A pair (a, b) of a head becomes (a cos t - b sin t, b cos t + a sin t) with
// t = position[axis] * frequency.  The turn is taken in whole numbers: with
// F = 2^64 * frequency / 2 pi, to the nearest whole number, position * F modulo 2^64
// is the angle's fraction of a turn, within |position| 2^-65 of a turn for every 64-bit
// position (no argument reduction), of which the sine and cosine are taken in fp32.
// Memory-bound: every element is read and written once.  The sines of a block's
// tokens are computed once into shared memory and shared by all heads; a thread
// keeps those of its pairs in registers over the heads it rotates.
// Measured: 216000 x 32 x 128 bf16 598 us interleaved (5.9 TB/s of 6.8), 610 in halves;
// 100000 x 16 x 64 fp32 122 us (6.7 TB/s); 200000 x 2 x 128 82 us: with two heads to share
// them the sines are what it computes.  One token: 6 us, the host's time for a call.
#include "token_attention_internal.h"
#include "token_common.cuh"

namespace c3d {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 32;   // tokens of a block
constexpr int kSinCos = 2048;    // (cos, sin) of a block

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
    T v[VEC];
};

// Heads whose loads a thread has in flight, and blocks of an SM that its registers have to
// allow: for 16-bit elements by four or eight many threads with a few loads each, else
// few with many.  216000 x 32 x 128 bf16 interleaved: two heads and five blocks 596 us, four heads
// and two blocks 640, two and six (spills) 715; in halves (two loads a head) one head and
// five blocks 608, two and four 649, four and two 665; 100000 x 16 x 64 fp32 in halves 127
// with one and five, 122 with four and two.
template <typename T, int VEC>
constexpr bool kManyThreads = sizeof(T) == 2 && VEC >= 4;

// VEC elements a load: VEC (half) or VEC / 2 (interleaved) pairs of a unit; VEC == 1
// is the form for any alignment (interleaved: two elements apart).
template <typename T, int VEC, bool HALF>
__global__ void __launch_bounds__(kThreads, kManyThreads<T, VEC> ? 5 : 0)
    rotary_kernel(const __grid_constant__ RotaryParams p, int units, int lanes, int tokens_block) {
    __shared__ float2 table[kSinCos];
    griddep_launch_dependents();
    griddep_wait();
    constexpr int NP = HALF ? VEC : (VEC > 1 ? VEC / 2 : 1);   // pairs of a unit
    const long long tok0 = static_cast<long long>(blockIdx.x) * tokens_block;
    const int here = static_cast<int>(min(static_cast<long long>(tokens_block), p.tokens - tok0));
    // a thread: unit `u` of token `t`, heads h0, h0 + lanes, ...
    const int u = threadIdx.x % units, rest = threadIdx.x / units;
    const int h0 = rest % lanes, t = rest / lanes;
    const T* x = static_cast<const T*>(p.x) + (tok0 + t) * p.x_tok;
    T* out = static_cast<T*>(p.out) + (tok0 + t) * p.out_tok;
    const int rot_units = p.pairs / NP;
    using V = Vec<T, VEC>;
    constexpr int kUnroll = !kManyThreads<T, VEC> ? 4 : HALF ? 1 : 2;
    const int ea = HALF ? u * VEC : u * 2 * NP;
    const int eb = HALF ? ea + p.pairs : ea + 1;
    constexpr bool kTwo = HALF || VEC == 1;   // two loads a unit
    V a[kUnroll], b[kUnroll];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int hh = h + i * lanes;
            if (hh < p.heads) {
                a[i] = *reinterpret_cast<const V*>(x + hh * p.x_head + ea);
                if (kTwo) b[i] = *reinterpret_cast<const V*>(x + hh * p.x_head + eb);
            }
        }
    };
    // (on their way while the sines are taken)
    const bool turns = t < here && u < rot_units;
    if (turns) load(h0);
    for (int i = threadIdx.x; i < here * p.pairs; i += kThreads) {
        const int tt = i / p.pairs, pair = i - tt * p.pairs;
        // (a lane's own entry: by its generic address, as the constant path takes one lane's at a time)
        unsigned long long per;
        uint32_t axis;
        asm("ld.u64 %0, [%1];" : "=l"(per) : "l"(p.turns + pair));
        asm("ld.u8 %0, [%1];" : "=r"(axis) : "l"(p.axis + pair));
        const long long at = (tok0 + tt) * p.axes + axis;
        const long long pos = p.pos64 ? static_cast<const long long*>(p.positions)[at]
                                      : static_cast<const int*>(p.positions)[at];
        const long long turn = static_cast<long long>(static_cast<unsigned long long>(pos) * per);
        float s, c;
        sincospif(__ll2float_rn(turn) * 1.0842021724855044e-19f, &s, &c);   // 2^-63: half turns
        table[i] = make_float2(c, p.inverse ? -s : s);
    }
    __syncthreads();
    if (t >= here) return;
    if (!turns) {   // elements that are not rotated
        for (int e = 2 * p.pairs + (u - rot_units) * VEC; e < p.width; e += (units - rot_units) * VEC)
            for (int h = h0; h < p.heads; h += lanes)
                *reinterpret_cast<V*>(out + h * p.out_head + e) =
                    *reinterpret_cast<const V*>(x + h * p.x_head + e);
        return;
    }
    float c[NP], s[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const float2 cs = table[t * p.pairs + u * NP + i];
        c[i] = cs.x;
        s[i] = cs.y;
    }
    for (int h = h0; h < p.heads; h += kUnroll * lanes) {
        if (h != h0) load(h);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int hh = h + i * lanes;
            if (hh >= p.heads) break;
            if (kTwo) {
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    const float va = to_f32(a[i].v[j]), vb = to_f32(b[i].v[j]);
                    a[i].v[j] = from_f32<T>(va * c[j] - vb * s[j]);
                    b[i].v[j] = from_f32<T>(vb * c[j] + va * s[j]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    const float va = to_f32(a[i].v[2 * j]), vb = to_f32(a[i].v[2 * j + 1]);
                    a[i].v[2 * j] = from_f32<T>(va * c[j] - vb * s[j]);
                    a[i].v[2 * j + 1] = from_f32<T>(vb * c[j] + va * s[j]);
                }
            }
            *reinterpret_cast<V*>(out + hh * p.out_head + ea) = a[i];
            if (kTwo) *reinterpret_cast<V*>(out + hh * p.out_head + eb) = b[i];
        }
    }
}

template <typename T, int VEC, bool HALF>
cudaError_t run(const RotaryParams& p, cudaStream_t stream) {
    constexpr int NP = HALF ? VEC : (VEC > 1 ? VEC / 2 : 1);
    const int rest = p.copy_rest ? (p.width - 2 * p.pairs) / VEC : 0;
    const int units = p.pairs / NP + (rest < kThreads / 2 ? rest : kThreads / 2);
    // heads side by side: all, as far as a block reaches; fewer, so that a thread's
    // sines serve up to four heads, where there are blocks enough without them (216000 x
    // 32 x 128: 640 us so, 888 with all side by side; 1000 x 24 x 128: 9.5 and 13.3)
    int lanes = kThreads / units < 1 ? 1 : kThreads / units;
    if (lanes > p.heads) lanes = p.heads;
    if (p.tokens * p.heads > 152 * 64 && lanes > (p.heads + 3) / 4) lanes = (p.heads + 3) / 4;
    int toks = kThreads / (units * lanes);
    if (toks > kMaxTokens) toks = kMaxTokens;
    if (toks * p.pairs > kSinCos) toks = kSinCos / p.pairs;
    const long long blocks = (p.tokens + toks - 1) / toks;
    return launch_ex(rotary_kernel<T, VEC, HALF>, static_cast<unsigned>(blocks), dim3(kThreads), 0, 1,
                     stream, p, units, lanes, toks);
}

// The widest loads that the rows' alignment, the pairs' distance and the elements left
// over allow: 16 bytes, 8, 4 (of 16-bit elements), or one element at a time.  100000 x 32 x
// 72 in halves of 36: 224 us by 8 bytes, 343 by elements; 68 in halves of 34: 325 by 4 bytes,
// 341 by elements.
template <typename T>
cudaError_t by_form(const RotaryParams& p, int align, cudaStream_t stream) {
    const int per = p.interleaved ? 2 * p.pairs : p.pairs, rest = p.width - 2 * p.pairs;
    auto fits = [&](int vec) {
        return align >= vec * static_cast<int>(sizeof(T)) && per % vec == 0 && rest % vec == 0;
    };
    constexpr int W = 16 / sizeof(T);
    if (fits(W)) return p.interleaved ? run<T, W, false>(p, stream) : run<T, W, true>(p, stream);
    if (fits(W / 2)) return p.interleaved ? run<T, W / 2, false>(p, stream) : run<T, W / 2, true>(p, stream);
    if constexpr (W == 8)
        if (fits(2)) return p.interleaved ? run<T, 2, false>(p, stream) : run<T, 2, true>(p, stream);
    return p.interleaved ? run<T, 1, false>(p, stream) : run<T, 1, true>(p, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, int dtype, int align, cudaStream_t stream) {
    if (dtype == kTokBf16) return by_form<__nv_bfloat16>(p, align, stream);
    if (dtype == kTokF16) return by_form<__half>(p, align, stream);
    return by_form<float>(p, align, stream);
}

}  // namespace c3d
