// linear_w8a8.cu -- the product of 8-bit tokens and weights with a scale per
// token and per output channel:
//
//   out[m,n] = act(scale_x[m] * scale_w[n] * sum_k x[m,k] w[n,k] + bias[n])
//
// sm_103a has no tensor-core product of 8-bit integers (tcgen05 kind::i8 is not
// among its features), so int8 codes go through kind::f16: every code is exact in
// f16, every product in fp32, and the fp32 sums are exact up to 2^24.  e4m3
// codes go through kind::f8f6f4 as they are.
#include <cuda_runtime.h>

#include <algorithm>

#include "token_activations.cuh"
#include "token_common.cuh"
#include "token_ops.h"
#include "token_ops_internal.h"

namespace c3d {

namespace {

constexpr int kRows = 128;        // weight rows of a tile (tcgen05 M)
constexpr int kStep = 128;        // reduction elements (bytes) of a k-step
constexpr int kMaxTok = 128;      // tokens of a tile at most
template <bool E4M3>
constexpr int kSplitThreads = 128 + 32 * (E4M3 ? 8 : 16);   // converters / epilogue behind four warps
constexpr int kMaxStages = 8, kMaxCvt = 4, kMaxSplits = 8;
constexpr uint32_t kBarBytes = 16u * (kMaxStages + kMaxCvt) + 16u;
// Rings (200 KB at most), barriers, alignment.  Every launch asks for all of it: the
// kernel holds all of an SM's tensor memory, and where two of its CTAs could share
// an SM, two clusters could each hold what the other waits for.
constexpr int kSplitRings = 200 * 1024, kSplitSmem = 206 * 1024;
static_assert(kSplitRings + kBarBytes + 32 + 1024 <= kSplitSmem, "");
constexpr int kSmSmem = 228 * 1024;      // of an SM; a CTA takes 1 KB more than it asks for
static_assert(2 * (kSplitSmem + 1024) > kSmSmem, "one split CTA an SM");

// No kernel here loads through the read-only path (__ldg): it starts while earlier
// kernels of the stream run, and what they write (codes, scales, also weights) is
// then not read-only for its lifetime.

// Bounded wait (see wait_bar) of a role that may wait for thousands of cycles:
// it sleeps in hardware between looks, so that its polling leaves the issue slots
// to the converters and the epilogue.
__device__ __forceinline__ bool wait_long_slow(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                            int* status, unsigned long long limit_ns) {
    const long long t0 = clock64();
    const long long limit = static_cast<long long>(limit_ns > (1ull << 61) ? (1ull << 61) : limit_ns) * 2;
    while (!mbar_try_wait_for(bar, parity, 100000u)) {
        if (*abort_flag) return false;
        if (clock64() - t0 > limit) {
            *abort_flag = 1u;
            atomicExch(status, kStatusTimeout);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                          int* status, unsigned long long limit_ns) {
    return mbar_try_wait_for(bar, parity, 100000u) ||
           wait_long_slow(bar, parity, abort_flag, status, limit_ns);
}

// After an abort: the loads into a ring of `slots` that `issued` k-steps armed.  Each
// slot's last load is waited for, whoever has seen it: an earlier one has landed
// (the slot was filled again), and the parity of the last is the barrier's
// current phase, so that the wait neither passes early nor runs out.
constexpr __host__ __device__ uint32_t drain_from(uint32_t issued, uint32_t slots) {
    return issued > slots ? issued - slots : 0u;
}
static_assert(drain_from(0, 4) == 0 && drain_from(4, 4) == 0 && drain_from(5, 4) == 1 && drain_from(13, 6) == 7, "");

__device__ __noinline__ void drain_ring(uint32_t full0, uint32_t issued, uint32_t slots) {
    for (uint32_t i = drain_from(issued, slots); i < issued; ++i) drain_wait(full0 + 8 * (i % slots), (i / slots) & 1u);
}

// The byte of the 16-byte chunk `c` of row `r` in a 128-byte-swizzled tile.
__device__ __forceinline__ uint32_t swz(int r, int c) {
    return static_cast<uint32_t>(r) * 128u + (static_cast<uint32_t>(c ^ (r & 7)) << 4);
}

// The same for 64-byte rows in the 64-byte swizzle.
__device__ __forceinline__ uint32_t swz64(int r, int c) {
    return static_cast<uint32_t>(r) * 64u + (static_cast<uint32_t>(c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t cluster_addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(cluster_addr) : "memory");
    return v;
}

__device__ __forceinline__ float ld_cluster_f1(uint32_t cluster_addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t cluster_addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// Four int8 codes as four f16 values: with the sign bit flipped a byte is the
// code + 128, and below the byte 0x64 it is the f16 number 1024 + 128 + code;
// 1152 subtracts exactly.  Five instructions for four codes.
__device__ __forceinline__ void i8x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

// One 16-byte chunk (16 codes) as 8 registers of f16 pairs.
__device__ __forceinline__ void cvt_chunk(const uint4& v, uint32_t* o) {
    i8x4_to_f16x4(v.x, o[0], o[1]);
    i8x4_to_f16x4(v.y, o[2], o[3]);
    i8x4_to_f16x4(v.z, o[4], o[5]);
    i8x4_to_f16x4(v.w, o[6], o[7]);
}

// A k-step of `rows` int8 rows (a multiple of 16; 128 bytes each, swizzled) as two
// boxes of f16 rows (64 elements each, swizzled), by the 128 threads `t`.  Eight
// threads that share a shared-memory cycle take four neighbouring chunks of row
// r and of row r^5: bit 2 keeps their reads, bit 0 their writes off each other's
// banks.  A thread's rows are 32 apart, which the swizzle does not see.
__device__ __forceinline__ void cvt_rows(uint32_t src, uint32_t dst, int rows, int t) {
    const int c4 = t & 3, r0 = (2 * (t >> 3)) ^ ((t & 4) ? 5 : 0);
    const int n = (rows - r0 + 31) >> 5;   // this thread's rows
    const uint32_t d0 = dst + swz(r0, 2 * c4), d1 = dst + swz(r0, 2 * c4 + 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t s0 = src + swz(r0, 4 * h + c4), box = static_cast<uint32_t>(h * rows) * 128u;
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)   // at most 128 rows
            if (i < n) w[i] = lds128(s0 + 4096u * i);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= n) break;
            uint32_t v[8];
            cvt_chunk(w[i], v);
            sts128(d0 + box + 4096u * i, v[0], v[1], v[2], v[3]);
            sts128(d1 + box + 4096u * i, v[4], v[5], v[6], v[7]);
        }
    }
}

// Epilogue activation: for 16-bit outputs the convolutions' SiLU and the row kernels'
// GELU (the convolutions' is off by 1.5e-7 in erf, more than its value below -5,
// which both types can hold), for fp32 outputs the fp32-accurate forms; all keep a
// NaN.  Out of line: the code behind a mainloop runs once and cold, and the fp32
// forms are long.
__device__ __noinline__ float epi_act_call(float v, int act, int out_dtype) {
    if (act == kActRelu || out_dtype == kTokF32) return activate_f32(v, act);
    return act == kActSilu ? activate_c<kActSilu>(v) : gelu2<true>(make_float2(v, 0.0f)).x;
}

__device__ __forceinline__ float epi_act(float v, int act, int out_dtype) {
    return act == kActNone ? v : epi_act_call(v, act, out_dtype);
}

__device__ __forceinline__ void store_one(void* out, int dtype, long long at, float v) {
    if (dtype == kTokBf16) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
    else if (dtype == kTokF16) static_cast<__half*>(out)[at] = __float2half_rn(v);
    else static_cast<float*>(out)[at] = v;
}

__device__ __forceinline__ uint32_t pack2(float a, float b, int dtype) {
    if (dtype == kTokBf16) return pack_bf16x2(a, b);
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Up to 16 bytes (left < 16: the rest zeros) from any address, put together from
// the aligned 4-byte words that hold at least one of them.
__device__ __forceinline__ uint4 load_bytes(const uint8_t* src, long long left) {
    const int n = static_cast<int>(min(16ll, left));
    uint32_t o[4] = {0u, 0u, 0u, 0u};
    if (n > 0) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(src);
        const int sh = static_cast<int>(a & 3u);
        const uint32_t* q = reinterpret_cast<const uint32_t*>(a - sh);
        const int need = (sh + n + 3) >> 2;
        uint32_t v[5];
#pragma unroll
        for (int j = 0; j < 5; ++j) v[j] = j < need ? q[j] : 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            o[j] = __funnelshift_r(v[j], v[j + 1], 8 * sh);
            const int in = n - 4 * j;   // bytes of this word that were asked for
            if (in < 4) o[j] = in <= 0 ? 0u : o[j] & ((1u << (8 * in)) - 1u);
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// ---------------------------------------------------------------- few tokens
// Up to 16 tokens: the weights are all there is to read, once, and latency is what
// is left.  A CTA takes 16 weight rows, its warps interleave over the reduction
// in steps of 64 bytes, and everything goes from global memory to registers to
// mma.sync (m16n8k16, f16): a dot product does not care in which order its terms
// come, so a lane's 16 contiguous bytes of a weight row and of a token serve as
// the k pairs that the instruction's fragments want (lane t of a quad: bytes
// 16 t .. 16 t + 15 of the step, four k16 products).  tcgen05's detour (TMA ring,
// tensor memory, a cluster's reduction) took 8.1 us for one token through
// 8192 x 2048 int8 against 5.0 here; its 128-row operand would be 1/16 full.
// Rows of any alignment: the unaligned ones are put together from aligned words.
constexpr int kThinRows = 16, kThinTok = LINEAR_W8A8_NO_WORKSPACE_TOKENS, kThinMaxWarps = 16;
static_assert(kThinTok == 16, "two blocks of eight tokens");

template <bool E4M3>
__device__ __forceinline__ void thin_cvt(const uint4& v, uint32_t (&o)[8]) {
    if (!E4M3) {
        cvt_chunk(v, o);
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(o[2 * i]), "=r"(o[2 * i + 1]) : "r"(w[i]));
}

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes of global memory, kept in the L1 cache (tokens: other CTAs of the SM read
// them) or not.  As asm volatile these loads stay in the order and number they are
// written in: plain ones took 5.3 us for one token through 8192 x 2048 against 4.9.
template <bool KEEP>
__device__ __forceinline__ uint4 ldg128(const uint8_t* p) {
    uint4 v;
    if (KEEP)
        asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    else
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// The 16 bytes at column c of a row (zeros outside it, or where the row is NULL).
template <bool ALIGNED, bool KEEP>
__device__ __forceinline__ uint4 thin_load(const uint8_t* row, long long c, long long width) {
    if (!row || c >= width) return make_uint4(0u, 0u, 0u, 0u);
    if (ALIGNED && c + 16 <= width) return ldg128<KEEP>(row + c);
    return load_bytes(row + c, width - c);
}

// NB blocks of 8 tokens; AHEAD steps whose loads are in flight together
template <bool E4M3, int NB, bool ALIGNED, int AHEAD>
__global__ void __launch_bounds__(32 * kThinMaxWarps)
    linear_thin_kernel(const LinearParams p) {
    __shared__ float part[kThinMaxWarps][8 * NB][kThinRows];
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const long long n0 = static_cast<long long>(blockIdx.x) * kThinRows;
    const uint8_t* w0 = n0 + g < p.outputs ? p.w + (n0 + g) * p.w_stride : nullptr;
    const uint8_t* w1 = n0 + g + 8 < p.outputs ? p.w + (n0 + g + 8) * p.w_stride : nullptr;
    const uint8_t* xr[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) xr[b] = 8 * b + g < p.tokens ? p.x + (8 * b + g) * p.x_stride : nullptr;
    float acc[NB][4] = {};
    const long long step = 64ll * warps;
    for (long long c = 64ll * warp + 16 * t; c - 16 * t < p.width; c += AHEAD * step) {
        uint4 a[AHEAD][2], x[AHEAD][NB];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            a[i][0] = thin_load<ALIGNED, false>(w0, c + i * step, p.width);
            a[i][1] = thin_load<ALIGNED, false>(w1, c + i * step, p.width);
#pragma unroll
            for (int b = 0; b < NB; ++b) x[i][b] = thin_load<ALIGNED, true>(xr[b], c + i * step, p.width);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            uint32_t u[8], v[8];
            thin_cvt<E4M3>(a[i][0], u);
            thin_cvt<E4M3>(a[i][1], v);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t y[8];
                thin_cvt<E4M3>(x[i][b], y);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma_f16_16816(acc[b], u[2 * j], v[2 * j], u[2 * j + 1], v[2 * j + 1], y[2 * j],
                                  y[2 * j + 1]);
            }
        }
    }
    // the warps' partial sums, added in warp order
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        part[warp][8 * b + 2 * t][g] = acc[b][0];
        part[warp][8 * b + 2 * t + 1][g] = acc[b][1];
        part[warp][8 * b + 2 * t][g + 8] = acc[b][2];
        part[warp][8 * b + 2 * t + 1][g + 8] = acc[b][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 8 * NB * kThinRows; i += blockDim.x) {
        const int m = i / kThinRows, r = i % kThinRows;
        const long long n = n0 + r;
        if (m >= p.tokens || n >= p.outputs) continue;
        float v = 0.0f;
        for (int k = 0; k < warps; ++k) v += part[k][m][r];
        v = v * (p.scale_x ? p.scale_x[m] : 1.0f) * (p.scale_w ? p.scale_w[n] : 1.0f) +
            (p.bias ? p.bias[n] : 0.0f);
        store_one(p.out, p.out_dtype, m * p.out_stride + n, epi_act(v, p.act, p.out_dtype));
    }
}

// ---------------------------------------------------------------- split tiles
// One tile (128 outputs x up to 128 tokens) per cluster, its reduction split
// over the cluster's CTAs: the form for few tokens, where the weights are all
// there is to read and 128-row tiles alone would leave most SMs idle.  The
// weights are the MMA's 128-row operand, so that a tile holds as few tokens as
// there are; partial tiles meet in distributed shared memory and are summed in
// rank order.
//   warp 0     TMA producer: raw 128-byte rows of weights and tokens
//   warp 1     TMEM, MMA issuer
//   warps 4-11  int8: weights to f16 into TMEM (lane = row); epilogue
//   warps 12-19 int8 only: tokens to f16 into shared memory;  epilogue
// The converters of either operand are two groups of four warps on alternate
// k-steps: a group's step is 600 to 1600 cycles of latency (wait, read, convert,
// write, fence) that the other's hides.
// What bounds it: latency (launch, first loads, the partials' way between CTAs, about
// 4 us in all) and, for int8, the token converters (about 1200 cycles a k-step at
// 128 tokens): 128 x 8192 x 2048 e4m3 8.4 us, int8 11.2 us, where the weights'
// bytes take 2.5.
struct SplitParams {
    LinearParams p;
    int tok_tile, out_tiles;
    int splits, k_steps, stages, cvt;
    uint32_t stage_bytes, cvt_bytes;
};

template <bool E4M3>
__global__ void __launch_bounds__(kSplitThreads<E4M3>, 1)
    linear_split_kernel(const __grid_constant__ CUtensorMap w_map,
                        const __grid_constant__ CUtensorMap x_map, const SplitParams s) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    constexpr int kCvtWarps = kSplitThreads<E4M3> / 32 - 4;
    const LinearParams& p = s.p;
    const int nt = s.tok_tile;
    const uint32_t ring = base;
    const uint32_t cvt0 = ring + static_cast<uint32_t>(s.stages) * s.stage_bytes;
    const uint32_t bars = cvt0 + static_cast<uint32_t>(s.cvt) * s.cvt_bytes;
    const uint32_t full0 = bars, empty0 = full0 + 8u * kMaxStages;
    const uint32_t cfull0 = empty0 + 8u * kMaxStages, cempty0 = cfull0 + 8u * kMaxCvt;
    const uint32_t acc_bar = cempty0 + 8u * kMaxCvt, drain_bar = acc_bar + 8u;
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem_raw + (drain_bar + 8u - raw));
    // misc[0] TMEM base, [1] abort flag, [2] k-steps issued
    volatile uint32_t* abort_flag = misc + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x % static_cast<unsigned>(s.splits));
    const int tile = static_cast<int>(blockIdx.x / static_cast<unsigned>(s.splits));
    const int n0 = (tile % s.out_tiles) * kRows;
    const long long m0 = static_cast<long long>(tile / s.out_tiles) * nt;
    const int ks0 = static_cast<int>(static_cast<long long>(s.k_steps) * rank / s.splits);
    const int ks1 = static_cast<int>(static_cast<long long>(s.k_steps) * (rank + 1) / s.splits);
    const int steps = ks1 - ks0;   // at least one: splits <= k_steps

    if (threadIdx.x == 0) {
        for (int i = 0; i < s.stages; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, E4M3 ? 1 : 8);
        }
        for (int i = 0; i < s.cvt; ++i) {
            mbar_init(cfull0 + 8 * i, 8);
            mbar_init(cempty0 + 8 * i, 1);
        }
        mbar_init(acc_bar, 1);
        mbar_init(drain_bar, 1);
        misc[1] = 0u;
        misc[2] = 0u;
        fence_mbar_init();
        prefetch_tmap(&w_map);
        prefetch_tmap(&x_map);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(misc), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    const uint32_t tmem_a = tmem + kMaxTok;   // converted weights behind the accumulator
    griddep_launch_dependents();
    griddep_wait();

    if (warp == 0) {
        if (lane == 0) {
            int st = 0;
            uint32_t ph = 0;
            for (int i = 0; i < steps; ++i) {
                if (!wait_bar(empty0 + 8 * st, ph ^ 1u, abort_flag, p.status, p.wait_ns)) break;
                const uint32_t fb = full0 + 8 * st, dst = ring + st * s.stage_bytes;
                mbar_arrive_expect_tx(fb, s.stage_bytes);
                tma_load_2d(dst, &w_map, fb, (ks0 + i) * kStep, n0);
                tma_load_2d(dst + kRows * kStep, &x_map, fb, (ks0 + i) * kStep, static_cast<int>(m0));
                misc[2] = i + 1;
                if (++st == s.stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // D: fp32, operands f16 (or e4m3: both codes are 0), N tokens, M 128
            const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(nt >> 3) << 17) | ((kRows >> 4) << 24);
            const uint64_t adesc = make_smem_desc(ring, 1024u, 2u);
            const uint64_t bdesc = make_smem_desc(E4M3 ? ring + kRows * kStep : cvt0, 1024u, 2u);
            const uint32_t step = (E4M3 ? s.stage_bytes : s.cvt_bytes) >> 4;
            const int depth = E4M3 ? s.stages : s.cvt;
            int st = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int i = 0; i < steps; ++i) {
                const uint32_t fb = (E4M3 ? full0 : cfull0) + 8 * st;
                if (!wait_bar(fb, ph, abort_flag, p.status, p.wait_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(st) * step);
                if (E4M3) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_f8(tmem, adesc + off + 2 * k, bdesc + off + 2 * k, idesc, (i | k) != 0);
                } else {
                    const uint32_t box = static_cast<uint32_t>(nt) * 128u >> 4;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        tc_mma_f16_ta(tmem, tmem_a + st * 64 + k * 8,
                                      bdesc + off + (k >> 2) * box + 2 * (k & 3), idesc, (i | k) != 0);
                }
                tc_commit((E4M3 ? empty0 : cempty0) + 8 * st);
                if (++st == depth) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (ok) tc_commit(acc_bar);
        }
    } else if (warp >= 4) {
        bool ok = true;
        if (!E4M3) {
            // even rings: a group sees every phase of the slots it waits for
            const int group = ((warp - 4) >> 2) & 1;
            int st = group, c = group;
            uint32_t ph = 0, cph = 0;
            for (int i = group; i < steps; i += 2) {
                ok = wait_bar(full0 + 8 * st, ph, abort_flag, p.status, p.wait_ns) &&
                     wait_bar(cempty0 + 8 * c, cph ^ 1u, abort_flag, p.status, p.wait_ns);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                const uint32_t src = ring + st * s.stage_bytes;
                if (warp < 12) {
                    tc_fence_after();
                    const int r = (warp & 3) * 32 + lane;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[32];
#pragma unroll
                        for (int j = 0; j < 4; ++j) cvt_chunk(lds128(src + swz(r, 4 * h + j)), v + 8 * j);
                        tmem_st_32x32b_x32(tmem_a + (static_cast<uint32_t>((warp & 3) * 32) << 16) +
                                               c * 64 + h * 32, v);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                } else {
                    cvt_rows(src + kRows * kStep, cvt0 + c * s.cvt_bytes, nt, threadIdx.x & 127);
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(empty0 + 8 * st);
                    mbar_arrive(cfull0 + 8 * c);
                }
                st += 2;
                if (st >= s.stages) {
                    st -= s.stages;
                    ph ^= 1u;
                }
                c += 2;
                if (c >= s.cvt) {
                    c -= s.cvt;
                    cph ^= 1u;
                }
            }
        }
        // the accumulator as [token][output] fp32 over the ring, which every
        // load and MMA has left by now
        if (warp < 12 && ok &&
            __all_sync(0xffffffffu, wait_bar(acc_bar, 0, abort_flag, p.status, p.wait_ns))) {
            tc_fence_after();
            const int q = warp & 3, half = warp >= 8;
            const int valid = static_cast<int>(min(static_cast<long long>(nt), p.tokens - m0));
            for (int t0 = half * (nt / 2); t0 < (half + 1) * (nt / 2); t0 += 8) {
                if (t0 >= valid) break;
                uint32_t v[8];
                tmem_ld_32x32b_x8(tmem + (static_cast<uint32_t>(q * 32) << 16) + t0, v);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(
                                     ring + static_cast<uint32_t>((t0 + j) * kRows + q * 32 + lane) * 4u),
                                 "r"(v[j]) : "memory");
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    if (s.splits > 1) cluster_sync();
    else __syncthreads();
    if (warp >= 4 && !*abort_flag) {
        // this rank's share of the tile's tokens, a row of 128 outputs per warp and turn
        const int t_lo = nt * rank / s.splits;
        const int t_hi = static_cast<int>(min(static_cast<long long>(nt * (rank + 1) / s.splits), p.tokens - m0));
        // a lane's outputs: four neighbours where rows are aligned for one store of
        // them, else every 32nd, so that a warp's stores lie side by side
        const int elt = p.out_dtype == kTokF32 ? 4 : 2;
        const bool wide = ((reinterpret_cast<uintptr_t>(p.out) | static_cast<uintptr_t>(p.out_stride * elt)) &
                           (4 * elt - 1)) == 0;
        const int first = wide ? 4 * lane : lane, pace = wide ? 1 : 32;
        const int n = n0 + first;
        float sw[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = n + j * pace < p.outputs;
            sw[j] = in && p.scale_w ? p.scale_w[n + j * pace] : 1.0f;
            b[j] = in && p.bias ? p.bias[n + j * pace] : 0.0f;
        }
        auto finish = [&](float (&v)[4], int t, float sx) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = epi_act(v[j] * sx * sw[j] + b[j], p.act, p.out_dtype);
            const long long at = (m0 + t) * p.out_stride + n;
            if (wide && n + 3 < p.outputs) {
                if (elt == 4)
                    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) =
                        make_float4(v[0], v[1], v[2], v[3]);
                else
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
                        make_uint2(pack2(v[0], v[1], p.out_dtype), pack2(v[2], v[3], p.out_dtype));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j * pace < p.outputs) store_one(p.out, p.out_dtype, at + j * pace, v[j]);
            }
        };
        // one token's row in this CTA's or a peer's partial tile
        auto own = [&](uint32_t a) {
            if (wide) return lds128(a);
            return make_uint4(lds32(a), lds32(a + 128u), lds32(a + 256u), lds32(a + 384u));
        };
        auto peer = [&](uint32_t a) {
            if (wide) return ld_cluster_f4(a);
            return make_float4(ld_cluster_f1(a), ld_cluster_f1(a + 128u), ld_cluster_f1(a + 256u),
                               ld_cluster_f1(a + 384u));
        };
        if (s.splits > 1) {
            // the ranks' partials of a token or two at once (a peer's shared memory is
            // far away), then added in rank order
            constexpr int kTurns = E4M3 ? 2 : 1;
            for (int t0 = t_lo + warp - 4; t0 < t_hi; t0 += kTurns * kCvtWarps) {
                float4 f[kTurns][kMaxSplits];
                float sx[kTurns];
#pragma unroll
                for (int u = 0; u < kTurns; ++u) {
                    const int t = min(t0 + u * kCvtWarps, t_hi - 1);
                    const uint32_t a = ring + static_cast<uint32_t>(t * kRows + first) * 4u;
                    sx[u] = p.scale_x ? p.scale_x[m0 + t] : 1.0f;
#pragma unroll
                    for (int r = 0; r < kMaxSplits; ++r)
                        f[u][r] = r < s.splits ? peer(mapa_shared(a, r)) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int u = 0; u < kTurns; ++u) {
                    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int r = 0; r < kMaxSplits; ++r) {
                        v[0] += f[u][r].x;
                        v[1] += f[u][r].y;
                        v[2] += f[u][r].z;
                        v[3] += f[u][r].w;
                    }
                    if (t0 + u * kCvtWarps < t_hi) finish(v, t0 + u * kCvtWarps, sx[u]);
                }
            }
        } else {
            constexpr int kTurns = 4;   // tokens whose loads are in flight together
            for (int t0 = t_lo + warp - 4; t0 < t_hi; t0 += kTurns * kCvtWarps) {
                float v[kTurns][4], sx[kTurns];
#pragma unroll
                for (int u = 0; u < kTurns; ++u) {
                    const int t = min(t0 + u * kCvtWarps, t_hi - 1);
                    const uint4 w = own(ring + static_cast<uint32_t>(t * kRows + first) * 4u);
                    v[u][0] = __uint_as_float(w.x);
                    v[u][1] = __uint_as_float(w.y);
                    v[u][2] = __uint_as_float(w.z);
                    v[u][3] = __uint_as_float(w.w);
                    sx[u] = p.scale_x ? p.scale_x[m0 + t] : 1.0f;
                }
#pragma unroll
                for (int u = 0; u < kTurns; ++u)
                    if (t0 + u * kCvtWarps < t_hi) finish(v[u], t0 + u * kCvtWarps, sx[u]);
            }
        }
    }
    __syncwarp();
    if (s.splits > 1) cluster_sync();   // the peers have read this CTA's partial tile
    else __syncthreads();
    if (*abort_flag) {
        // drain: the loads, then the MMAs in flight
        if (threadIdx.x == 0) drain_ring(full0, misc[2], static_cast<uint32_t>(s.stages));
        if (warp == 1 && lane == 0) {
            tc_commit(drain_bar);
            drain_wait(drain_bar, 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- paired tiles
// Persistent CTA pairs, 256 tokens x up to 256 outputs a tile: the form for many
// tokens.  Here the tokens are the MMA's row operand (128 per CTA) and each CTA
// holds half of the tile's weight rows.
//   warp 0       TMA producer (int8: of the weights)
//   warp 1       TMEM, MMA issuer (leader CTA)
//   warp 2       int8: TMA producer of the tokens
//   warps 4-     epilogue (e4m3 16 warps, int8 8): lane = token, 64 or 128 outputs a warp
//   warps 12-19  int8: tokens to f16 into TMEM, two groups on alternate k-steps
// int8: the tokens cross shared memory once as bytes (their f16 form goes to
// TMEM); the weights come as f16 from the workspace, where one short launch has
// put them.  What decides this is shared memory, 128 bytes a cycle: per k-step
// (1024 cycles of MMA) it moves 16 KB of raw tokens in and out, 32 KB of weights
// in and 32 KB of the MMA's reads, 96 bytes a cycle.  Converting the weights here
// too takes 128 (raw in and out, f16 in and out), and measured 1475 TFLOP/s at
// 16384 x 8192 x 8192 against 1907; the launch moves 3 bytes per weight.
// What bounds it now: the tensor pipe under the power cap at long reductions (1057
// cycles a k-step of 1024; e4m3 3600 to 3700 TFLOP/s), and between tiles the hand-over
// of the accumulator (int8, about 2000 cycles a tile).  e4m3's k-steps fill the
// shared memory's 128 bytes a cycle by themselves, so that at 1024-long reductions
// the epilogue's staging and scales are what is added (2840 TFLOP/s at 16384 x
// 8192 x 1024).  Measured and not kept: outputs stored from the registers, a sector
// per lane (0.88x there), tiles of 128 outputs (a k-step costs the same).
//
// Rings: the tokens' raw slots are free once converted, so that their loads run
// ahead of the MMAs by both rings (4 raw slots, 4 in TMEM); one ring for both
// operands refilled a stage in 4100 cycles, over the 3072 that it had.
// Accumulators: e4m3 has two, int8 one (its tokens take the other half of
// TMEM), which the epilogue therefore first loads into registers as a whole
// (128 a thread; setmaxnreg gives its warps what the others do not need) and
// hands back before it scales, packs and stores: the MMAs wait for the loads
// only, not for the 6000 cycles that a tile's epilogue took chunk by chunk.
struct PairParams {
    LinearParams p;
    int m_tiles, n_tiles, group_m;
    int k_steps;
    FastDiv f_group, f_gm;
};

constexpr int kPairOut = 256;                             // outputs of a tile
constexpr uint32_t kTokBytes = kRows * kStep;             // tokens of a k-step and CTA
constexpr uint32_t kTmemA = 256;                          // TMEM columns of the converted tokens
template <bool E4M3>
struct PairShape {
    static constexpr uint32_t kWBytes = kRows * kStep * (E4M3 ? 1u : 2u);   // weights of a k-step
    // a ring stage: e4m3 tokens and weights, int8 weights (f16) alone
    static constexpr uint32_t kStage = kWBytes + (E4M3 ? kTokBytes : 0u);
    static constexpr int kStages = E4M3 ? 6 : 4;
    static constexpr int kAcc = E4M3 ? 2 : 1;        // accumulators in TMEM
    static constexpr int kTokSlots = E4M3 ? 0 : 4;   // int8: raw tokens
    // The two converter groups take alternate k-steps.  A parity wait tells a phase
    // from its neighbours only, so a group has to see every phase of the slots it
    // waits for: rings of even length, each slot one group's.
    static_assert(kTokSlots % 2 == 0 && kStages % 2 == 0, "");
    // epilogue warps, and the 32-column chunks that each takes of a tile
    static constexpr int kEpiWarps = E4M3 ? 16 : 8, kChunks = 32 / kEpiWarps;
    static constexpr uint32_t kStaging = E4M3 ? 2048u : 4096u;   // of a warp: one or two 2 KB buffers
    static constexpr int kThreads = 128 + 32 * kEpiWarps + (E4M3 ? 0 : 256);
    static constexpr uint32_t kEpi0 = kStages * kStage + kTokSlots * kTokBytes;
    static constexpr uint32_t kBars0 = kEpi0 + kEpiWarps * kStaging;
    static constexpr uint32_t kBytes = kBars0 + 5u * 8u * kMaxStages + 40u + 32u;
};
static_assert(PairShape<true>::kBytes <= 227u * 1024u && PairShape<false>::kBytes <= 227u * 1024u, "");

// Two accumulators: v * sx * f + b, with the two-wide fp32 instructions.
__device__ __forceinline__ void scale2(uint32_t& v0, uint32_t& v1, float sx, uint32_t f0, uint32_t f1,
                                       uint32_t b0, uint32_t b1) {
    asm("{\n\t.reg .b64 v, s, f, b;\n\t"
        "mov.b64 v, {%0, %1};\n\tmov.b64 s, {%2, %2};\n\t"
        "mov.b64 f, {%3, %4};\n\tmov.b64 b, {%5, %6};\n\t"
        "mul.rn.f32x2 v, v, s;\n\tfma.rn.f32x2 v, v, f, b;\n\t"
        "mov.b64 {%0, %1}, v;\n\t}"
        : "+r"(v0), "+r"(v1)
        : "r"(__float_as_uint(sx)), "r"(f0), "r"(f1), "r"(b0), "r"(b1));
}

// The same without a bias.
__device__ __forceinline__ void mul2(uint32_t& v0, uint32_t& v1, float sx, uint32_t f0, uint32_t f1) {
    asm("{\n\t.reg .b64 v, s, f;\n\t"
        "mov.b64 v, {%0, %1};\n\tmov.b64 s, {%2, %2};\n\tmov.b64 f, {%3, %4};\n\t"
        "mul.rn.f32x2 v, v, s;\n\tmul.rn.f32x2 v, v, f;\n\t"
        "mov.b64 {%0, %1}, v;\n\t}"
        : "+r"(v0), "+r"(v1)
        : "r"(__float_as_uint(sx)), "r"(f0), "r"(f1));
}

// The activation of a chunk in registers, in the forms for 16-bit outputs.
__device__ __forceinline__ void act_chunk(uint32_t (&v)[32], int act) {
    auto each = [&](auto f) {
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            const float2 y = f(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])));
            v[j] = __float_as_uint(y.x);
            v[j + 1] = __float_as_uint(y.y);
        }
    };
    if (act == kActRelu) each([](float2 y) { return make_float2(y.x < 0.0f ? 0.0f : y.x, y.y < 0.0f ? 0.0f : y.y); });
    else if (act == kActSilu)
        each([](float2 y) { return make_float2(activate_c<kActSilu>(y.x), activate_c<kActSilu>(y.y)); });
    else each([](float2 y) { return gelu2<true>(y); });
}

struct PairTile {
    int mt, nt;
};

// Groups of group_m token tiles, token tile fastest: the tiles in flight form a
// near-square block, whose token and weight rows are read from L2.
__device__ __forceinline__ PairTile pair_tile(int t, const PairParams& s) {
    const int g = static_cast<int>(fdiv(static_cast<uint32_t>(t), s.f_group));
    const int first = g * s.group_m, local = t - g * s.group_m * s.n_tiles;
    const int gm = min(s.group_m, s.m_tiles - first);
    const int nt = gm == s.group_m ? static_cast<int>(fdiv(static_cast<uint32_t>(local), s.f_gm)) : local / gm;
    return PairTile{first + local - nt * gm, nt};
}

// Outputs that tile nt's MMAs compute: kPairOut, or the rest rounded up to 32.
__device__ __forceinline__ int pair_cols(int nt, const PairParams& s) {
    const long long rest = s.p.outputs - static_cast<long long>(nt) * kPairOut;
    return rest >= kPairOut ? kPairOut : static_cast<int>((rest + 31) & ~31ll);
}

// TMA_OUT: TMA can address the output's rows; else they are stored element by
// element, by an instance of its own (that code's registers cost the other 2%).
template <bool E4M3, bool TMA_OUT>
__global__ void __launch_bounds__(PairShape<E4M3>::kThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap x_map,
                       const __grid_constant__ CUtensorMap w_map,
                       const __grid_constant__ CUtensorMap o_map, const PairParams s) {
    using Shape = PairShape<E4M3>;
    extern __shared__ __align__(1024) unsigned char smem_pair[];
    const LinearParams& p = s.p;
    const uint32_t ring = smem_u32(smem_pair);
    const uint32_t toks = ring + Shape::kStages * Shape::kStage;
    // wfull: both CTAs' weights (and e4m3 tokens), on the leader; xfull, xempty:
    // this CTA's int8 tokens; ready: both CTAs' 4 converter warps of the step, on
    // the leader; empty: the stage's MMAs
    const uint32_t wfull0 = ring + Shape::kBars0, xfull0 = wfull0 + 8u * kMaxStages;
    const uint32_t xempty0 = xfull0 + 8u * kMaxStages, ready0 = xempty0 + 8u * kMaxStages;
    const uint32_t empty0 = ready0 + 8u * kMaxStages;
    const uint32_t tfull0 = empty0 + 8u * kMaxStages, tempty0 = tfull0 + 16u;
    const uint32_t drain_bar = tempty0 + 16u;
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem_pair + (drain_bar + 8u - ring));
    // misc[0] TMEM base, [1] abort flag, [2] weights' k-steps issued, [3] tokens'
    volatile uint32_t* abort_flag = misc + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int tiles = s.m_tiles * s.n_tiles;
    const int first = static_cast<int>(blockIdx.x) >> 1, stride = static_cast<int>(gridDim.x) >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < Shape::kStages; ++i) {
            mbar_init(wfull0 + 8 * i, 1);
            mbar_init(xfull0 + 8 * i, 1);
            mbar_init(xempty0 + 8 * i, 4);
            mbar_init(ready0 + 8 * i, 8);
            mbar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull0 + 8 * i, 1);
            mbar_init(tempty0 + 8 * i, 2 * Shape::kEpiWarps);
        }
        mbar_init(drain_bar, 1);
        for (int i = 1; i < 4; ++i) misc[i] = 0u;
        fence_mbar_init();
        prefetch_tmap(&x_map);
        prefetch_tmap(&w_map);
        if (TMA_OUT) prefetch_tmap(&o_map);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(misc), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers exist before any cross-CTA signal
    tc_fence_after();
    const uint32_t tmem = misc[0];
    griddep_launch_dependents();
    griddep_wait();
    // k-steps of this pair's tiles
    const int total = first < tiles ? ((tiles - first + stride - 1) / stride) * s.k_steps : 0;

    // Each warpgroup takes its share of the launch's registers, 20 warps of 96:
    // e4m3 4 x 56 + 16 x 104, int8 4 x 40 + 8 x 168 + 8 x 48, both <= 1920.
    if (warp < 4) {
        set_max_regs_dec<E4M3 ? 56 : 40>();
        if (warp == 0) {
            // ------------------------------------------------------ TMA producer
            if (lane == 0) {
                int st = 0;
                uint32_t ph = 0, issued = 0;
                bool ok = true;
                for (int t = first; t < tiles && ok; t += stride) {
                    const PairTile tl = pair_tile(t, s);
                    const int m0 = tl.mt * 256 + rank * kRows;
                    const int n0 = tl.nt * kPairOut + rank * (pair_cols(tl.nt, s) >> 1);
                    for (int i = 0; i < s.k_steps; ++i) {
                        if (!wait_long(empty0 + 8 * st, ph ^ 1u, abort_flag, p.status, p.wait_ns)) {
                            ok = false;
                            break;
                        }
                        const uint32_t dst = ring + st * Shape::kStage;
                        // the leader's barrier counts both CTAs' bytes
                        if (rank == 0) mbar_arrive_expect_tx(wfull0 + 8 * st, 2u * Shape::kStage);
                        const uint32_t fb = mapa_shared(wfull0 + 8 * st, 0);
                        if (E4M3) {
                            tma_load_2d_pair(dst, &x_map, fb, i * kStep, m0);
                            tma_load_2d_pair(dst + kTokBytes, &w_map, fb, i * kStep, n0);
                        } else {
                            // f16: two boxes of 64 elements
                            tma_load_2d_pair(dst, &w_map, fb, i * kStep, n0);
                            tma_load_2d_pair(dst + kTokBytes, &w_map, fb, i * kStep + 64, n0);
                        }
                        misc[2] = ++issued;
                        if (++st == Shape::kStages) {
                            st = 0;
                            ph ^= 1u;
                        }
                    }
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------ MMA issuer
            if (lane == 0 && rank == 0) {
                const uint64_t adesc = make_smem_desc(ring, 1024u, 2u);
                const uint64_t bdesc = make_smem_desc(ring + (E4M3 ? kTokBytes : 0u), 1024u, 2u);
                int st = 0, it = 0;
                uint32_t ph = 0;
                bool ok = true, landed = false;   // landed: this stage's operands were seen
                auto here = [&](int stage, uint32_t phase) {
                    return mbar_test_wait(wfull0 + 8 * stage, phase) &&
                           (E4M3 || mbar_test_wait(ready0 + 8 * stage, phase));
                };
                for (int t = first; t < tiles && ok; t += stride, ++it) {
                    const PairTile tl = pair_tile(t, s);
                    // D fp32, operands f16 (or e4m3: both codes are 0), N, M 256
                    const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(pair_cols(tl.nt, s) >> 3) << 17) |
                                           ((256u >> 4) << 24);
                    const int acc = it % Shape::kAcc;
                    const uint32_t aph = static_cast<uint32_t>(it / Shape::kAcc) & 1u;
                    if (!wait_bar(tempty0 + 8 * acc, aph ^ 1u, abort_flag, p.status, p.wait_ns)) break;
                    const uint32_t d = tmem + static_cast<uint32_t>(acc * kPairOut);
                    for (int i = 0; i < s.k_steps; ++i) {
                        if (!landed &&
                            (!wait_bar(wfull0 + 8 * st, ph, abort_flag, p.status, p.wait_ns) ||
                             (!E4M3 && !wait_bar(ready0 + 8 * st, ph, abort_flag, p.status, p.wait_ns)))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t off =
                            static_cast<uint64_t>(static_cast<uint32_t>(st) * (Shape::kStage >> 4));
                        const int nst = st + 1 == Shape::kStages ? 0 : st + 1;
                        const uint32_t nph = nst ? ph : ph ^ 1u;
                        // The pipe queues a couple of MMAs: the next stage is looked at
                        // before the last one of this stage, while they run.
                        constexpr int kMma = E4M3 ? 4 : 8;
#pragma unroll
                        for (int k = 0; k < kMma; ++k) {
                            if (k == kMma - 1) landed = here(nst, nph);
                            if (E4M3)
                                tc_mma_f8_pair(d, adesc + off + 2 * k, bdesc + off + 2 * k, idesc,
                                               (i | k) != 0);
                            else
                                tc_mma_f16_ta_pair(d, tmem + kTmemA + st * 64 + k * 8,
                                                   bdesc + off + (k >> 2) * (kTokBytes >> 4) + 2 * (k & 3),
                                                   idesc, (i | k) != 0);
                        }
                        tc_commit_pair(empty0 + 8 * st, 3);
                        st = nst;
                        ph = nph;
                    }
                    if (ok) tc_commit_pair(tfull0 + 8 * acc, 3);
                }
            }
        } else if (warp == 2) {
            // ------------------------------------------------------ tokens' producer (int8)
            if (!E4M3 && lane == 0) {
                int xs = 0;
                uint32_t ph = 0, issued = 0;
                bool ok = true;
                for (int t = first; t < tiles && ok; t += stride) {
                    const int m0 = pair_tile(t, s).mt * 256 + rank * kRows;
                    for (int i = 0; i < s.k_steps; ++i) {
                        if (!wait_long(xempty0 + 8 * xs, ph ^ 1u, abort_flag, p.status, p.wait_ns)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(xfull0 + 8 * xs, kTokBytes);
                        tma_load_2d(toks + xs * kTokBytes, &x_map, xfull0 + 8 * xs, i * kStep, m0);
                        misc[3] = ++issued;
                        if (++xs == Shape::kTokSlots) {
                            xs = 0;
                            ph ^= 1u;
                        }
                    }
                }
            }
        }
    } else if (warp < 4 + Shape::kEpiWarps) {
        // ------------------------------------------------------ epilogue
        set_max_regs_inc<E4M3 ? 104 : 168>();
        const int q = warp & 3, col0 = ((warp - 4) >> 2) * 32 * Shape::kChunks;
        const uint32_t tempty_dst = mapa_shared(tempty0, 0);
        const uint32_t buf0 = ring + Shape::kEpi0 + static_cast<uint32_t>(warp - 4) * Shape::kStaging;
        const bool f32 = p.out_dtype == kTokF32;
        int it = 0, nbuf = 0;
        for (int t = first; t < tiles; t += stride, ++it) {
            const PairTile tl = pair_tile(t, s);
            const int ncols = pair_cols(tl.nt, s);
            const long long nbase = static_cast<long long>(tl.nt) * kPairOut;
            const long long m0 = static_cast<long long>(tl.mt) * 256 + rank * kRows + q * 32;
            // this lane's scale and bias of each 32-column chunk
            float csw[Shape::kChunks], cbi[Shape::kChunks];
#pragma unroll
            for (int j = 0; j < Shape::kChunks; ++j) {
                const int c = col0 + 32 * j + lane;
                const bool in = c < ncols && nbase + c < p.outputs;
                csw[j] = in && p.scale_w ? p.scale_w[nbase + c] : 1.0f;
                cbi[j] = in && p.bias ? p.bias[nbase + c] : 0.0f;
            }
            const float sx = p.scale_x && m0 + lane < p.tokens ? p.scale_x[m0 + lane] : 1.0f;
            const int acc = it % Shape::kAcc;
            const uint32_t aph = static_cast<uint32_t>(it / Shape::kAcc) & 1u;
            if (!__all_sync(0xffffffffu,
                            wait_long(tfull0 + 8 * acc, aph, abort_flag, p.status, p.wait_ns)))
                break;
            tc_fence_after();
            const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) +
                                static_cast<uint32_t>(acc * kPairOut + col0);
            // chunks that have outputs; all are loaded (the columns exist), so that the
            // accumulator goes back at once
            const int chunks = max(0, min(Shape::kChunks, (ncols - col0 + 31) >> 5));
            uint32_t v[Shape::kChunks][32];
#pragma unroll
            for (int j = 0; j < Shape::kChunks; ++j) tmem_ld_32x32b_x32(tb + 32 * j, v[j]);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(tempty_dst + 8 * acc);
            if (m0 >= p.tokens) continue;
            // Outputs leave through 2 KB buffers of 32 rows x 64 bytes.  free_buffer:
            // the next one, when its last store has read it; store_buffer: its
            // columns [c0, c0 + width) to the output.
            auto free_buffer = [&]() {
                const uint32_t buf = buf0 + (E4M3 ? 0u : static_cast<uint32_t>(nbuf++ & 1) * 2048u);
                if (TMA_OUT && lane == 0) bulk_wait_read<E4M3 ? 0 : 1>();
                __syncwarp();
                return buf;
            };
            auto store_buffer = [&](uint32_t buf, int c0) {
                if constexpr (TMA_OUT) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        // columns and rows outside the output are not written (its rows end on
                        // 16 bytes)
                        tma_store_2d(&o_map, buf, static_cast<int>(nbase) + c0, static_cast<int>(m0));
                        bulk_commit();
                    }
                } else {
                    // rows that TMA cannot address: element stores, 64 bytes of a row at once,
                    // eight reads of the buffer ahead of their stores
                    __syncwarp();
                    const int rows = static_cast<int>(min(32ll, p.tokens - m0));
                    if (f32) {
                        const int c = lane & 15, r0 = lane >> 4;
                        float* dst = static_cast<float*>(p.out) + (m0 + r0) * p.out_stride + nbase + c0 + c;
                        const bool in = nbase + c0 + c < p.outputs;
#pragma unroll
                        for (int g = 0; g < 32; g += 16) {
                            uint32_t x[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[i] = lds32(buf + swz64(g + 2 * i + r0, c >> 2) + 4u * (c & 3));
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (in && g + 2 * i + r0 < rows)
                                    dst[(g + 2 * i) * p.out_stride] = __uint_as_float(x[i]);
                        }
                    } else {
                        uint16_t* dst = static_cast<uint16_t*>(p.out) + m0 * p.out_stride + nbase + c0 + lane;
                        const bool in = nbase + c0 + lane < p.outputs;
// e4m3's 16 epilogue warps have the fewer registers: unrolled they spill 344 bytes
// (16384 x 8191 x 1024: 178 us rolled, 226 unrolled; int8 311 and 297)
#pragma unroll(E4M3 ? 1 : 4)
                        for (int g = 0; g < 32; g += 8) {
                            uint16_t x[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                asm volatile("ld.shared.b16 %0, [%1];" : "=h"(x[i])
                                             : "r"(buf + swz64(g + i, lane >> 3) + 2u * (lane & 7)) : "memory");
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (in && g + i < rows) dst[(g + i) * p.out_stride] = x[i];
                        }
                    }
                    __syncwarp();
                }
            };
#pragma unroll
            for (int j = 0; j < Shape::kChunks; ++j) {
                if (j >= chunks) break;
                uint32_t(&y)[32] = v[j];
                uint32_t buf = free_buffer();
                // the chunk's 32 scales and 32 biases, through the buffer as broadcasts
                sts32(buf + 4u * lane, __float_as_uint(csw[j]));
                if (p.bias) sts32(buf + 128u + 4u * lane, __float_as_uint(cbi[j]));
                __syncwarp();
                if (p.bias) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 f = lds128(buf + 16u * i), b = lds128(buf + 128u + 16u * i);
                        scale2(y[4 * i], y[4 * i + 1], sx, f.x, f.y, b.x, b.y);
                        scale2(y[4 * i + 2], y[4 * i + 3], sx, f.z, f.w, b.z, b.w);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 f = lds128(buf + 16u * i);
                        mul2(y[4 * i], y[4 * i + 1], sx, f.x, f.y);
                        mul2(y[4 * i + 2], y[4 * i + 3], sx, f.z, f.w);
                    }
                }
                __syncwarp();
                const int c0 = col0 + 32 * j;
                if (f32) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {   // 16 columns a buffer
                        if (h == 1) buf = free_buffer();
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sts128(buf + swz64(lane, i), y[16 * h + 4 * i], y[16 * h + 4 * i + 1],
                                   y[16 * h + 4 * i + 2], y[16 * h + 4 * i + 3]);
                        // the fp32 activations are long: a loop over the staged row
                        for (int i = 0; p.act != kActNone && i < 16; ++i) {
                            float* e = reinterpret_cast<float*>(
                                smem_pair + (buf - ring) + swz64(lane, i >> 2) + 4 * (i & 3));
                            *e = activate_f32(*e, p.act);
                        }
                        store_buffer(buf, c0 + 16 * h);
                    }
                    continue;
                }
                if (p.act != kActNone) act_chunk(y, p.act);
                // one branch a chunk: the compiler would test the type at every pair
                if (p.out_dtype == kTokBf16) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        y[i] = pack_bf16x2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]));
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        y[i] = pack2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]), kTokF16);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sts128(buf + swz64(lane, i), y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                store_buffer(buf, c0);
            }
        }
        // the staging buffers are read out before the CTA leaves
        if (TMA_OUT && lane == 0) bulk_wait_read<0>();
    } else if (!E4M3) {
        // ------------------------------------------------------ converters (int8)
        set_max_regs_dec<48>();
        const int group = (warp - 12) >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t ta = tmem + kTmemA + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t ready_dst = mapa_shared(ready0, 0);
        int xs = group, ts = group;   // raw slot, TMEM slot (the weights' stage)
        uint32_t xph = 0, tph = 0;
        for (int i = group; i < total; i += 2) {
            const bool ok = wait_long(xfull0 + 8 * xs, xph, abort_flag, p.status, p.wait_ns) &&
                            wait_long(empty0 + 8 * ts, tph ^ 1u, abort_flag, p.status, p.wait_ns);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const uint32_t src = toks + xs * kTokBytes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t v[32];
#pragma unroll
                for (int j = 0; j < 4; ++j) cvt_chunk(lds128(src + swz(r, 4 * h + j)), v + 8 * j);
                tmem_st_32x32b_x32(ta + ts * 64 + h * 32, v);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(xempty0 + 8 * xs);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(ready_dst + 8 * ts);
            xs += 2;
            if (xs >= Shape::kTokSlots) {
                xs -= Shape::kTokSlots;
                xph ^= 1u;
            }
            ts += 2;
            if (ts >= Shape::kStages) {
                ts -= Shape::kStages;
                tph ^= 1u;
            }
        }
    }

    __syncthreads();
    // both CTAs finish their roles before either drains, frees TMEM or leaves
    cluster_sync();
    if (*abort_flag) {
        // the peer's loads signal the leader's barriers, so it cannot watch them
        // land: after an abort ~100 us pass first
        const long long t0 = clock64();
        while (clock64() - t0 < 200000) {
        }
        if (threadIdx.x == 0) {
            if (rank == 0) {
                // the peer's half of a step that it gave up before is not coming
                const uint32_t theirs = ld_cluster_u32(mapa_shared(smem_u32(misc + 2), 1));
                for (uint32_t i = max(theirs, drain_from(misc[2], Shape::kStages)); i < misc[2]; ++i)
                    mbar_complete_tx(wfull0 + 8 * (i % Shape::kStages), Shape::kStage);
                drain_ring(wfull0, misc[2], Shape::kStages);
            }
            if (!E4M3) drain_ring(xfull0, misc[3], PairShape<false>::kTokSlots);
        }
        if (warp == 1 && lane == 0 && rank == 0) {
            tc_commit_pair(drain_bar, 1);
            drain_wait(drain_bar, 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// Operands brought to rows that TMA can address, in one launch: bytes copied to a
// 16-byte pitch, or int8 widened to f16; zeros behind each row.  One thread per 16
// bytes read, as one word where the source's rows allow it.
__device__ __forceinline__ void stage_job(const RowJob& j, unsigned block, unsigned blocks) {
    const long long words = j.pitch >> 4, total = j.rows * words;
    for (long long k = static_cast<long long>(block) * 256 + threadIdx.x; k < total;
         k += static_cast<long long>(blocks) * 256) {
        const long long r = j.small ? static_cast<long long>(fdiv(static_cast<uint32_t>(k), j.by_words)) : k / words;
        const long long c = (k - r * words) << 4;
        const uint8_t* src = j.src + r * j.stride + c;
        const uint4 v = j.aligned && c + 16 <= j.cols ? *reinterpret_cast<const uint4*>(src)
                                                      : load_bytes(src, j.cols - c);
        if (j.widen) {
            uint32_t o[8];
            cvt_chunk(v, o);
            uint4* d = reinterpret_cast<uint4*>(j.dst + 2 * (r * j.pitch + c));
            d[0] = make_uint4(o[0], o[1], o[2], o[3]);
            d[1] = make_uint4(o[4], o[5], o[6], o[7]);
        } else {
            *reinterpret_cast<uint4*>(j.dst + r * j.pitch + c) = v;
        }
    }
}

__global__ void __launch_bounds__(256) stage_rows_kernel(const __grid_constant__ RowJobs jobs) {
    griddep_launch_dependents();
    griddep_wait();
    if (blockIdx.x < jobs.blocks0) stage_job(jobs.job[0], blockIdx.x, jobs.blocks0);
    else stage_job(jobs.job[1], blockIdx.x - jobs.blocks0, gridDim.x - jobs.blocks0);
}

// Clusters of 2, 4 and 8 split-kernel CTAs (one per SM) that the current device
// runs at once; asked once per device (the GPCs' sizes decide it, not the SM count).
struct ClusterRoom {
    int of[4];   // by log2 of the cluster's size
};

template <bool E4M3>
cudaError_t cluster_room(int num_sms, ClusterRoom* room) {
    static std::atomic<int> known[kMaxDevices][4];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    room->of[0] = num_sms;
    for (int i = 1; i < 4; ++i) {
        int n = dev < kMaxDevices ? known[dev][i].load(std::memory_order_acquire) : 0;
        if (n == 0) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(num_sms / (1 << i) * (1 << i)), 1, 1);
            cfg.blockDim = dim3(kSplitThreads<E4M3>, 1, 1);
            cfg.dynamicSmemBytes = kSplitSmem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 1u << i;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if ((e = cudaOccupancyMaxActiveClusters(&n, linear_split_kernel<E4M3>, &cfg)) != cudaSuccess)
                return e;
            n = std::max(n, 1);
            if (dev < kMaxDevices) known[dev][i].store(n, std::memory_order_release);
        }
        room->of[i] = n;
    }
    return cudaSuccess;
}

// the split kernel may use kSplitSmem bytes
template <bool E4M3>
cudaError_t allow_split_smem() {
    static std::atomic<int> smem_set[kMaxDevices];
    return ensure_dynamic_smem(linear_split_kernel<E4M3>, kSplitSmem, smem_set);
}

template <bool E4M3>
cudaError_t launch_split(const CUtensorMap& w_map, const CUtensorMap& x_map, const SplitParams& s,
                         const LinearPlan& plan, cudaStream_t stream) {
    cudaError_t e = allow_split_smem<E4M3>();
    if (e != cudaSuccess) return e;
    const long long grid = static_cast<long long>(plan.out_tiles) * plan.tok_tiles * plan.splits;
    return launch_ex(linear_split_kernel<E4M3>, static_cast<unsigned>(grid), kSplitThreads<E4M3>, plan.smem,
                     plan.splits, stream, w_map, x_map, s);
}

template <bool E4M3, bool TMA_OUT>
cudaError_t launch_pair(const LinearMaps& maps, const PairParams& s, const LinearPlan& plan,
                        cudaStream_t stream) {
    static std::atomic<int> smem_set[kMaxDevices];
    auto kern = linear_pair_kernel<E4M3, TMA_OUT>;
    cudaError_t e = ensure_dynamic_smem(kern, plan.smem, smem_set);
    if (e != cudaSuccess) return e;
    return launch_ex(kern, static_cast<unsigned>(plan.grid), PairShape<E4M3>::kThreads, plan.smem, 2, stream,
                     maps.x, maps.w, maps.out, s);
}

void plan_pair(const LinearParams& p, int num_sms, LinearPlan* r) {
    r->pair = 1;
    r->tok_box = r->out_box = kRows;
    r->tok_tiles = static_cast<int>((p.tokens + 255) / 256);
    r->out_tiles = static_cast<int>((p.outputs + kPairOut - 1) / kPairOut);
    r->splits = 1;
    r->smem = p.e4m3 ? PairShape<true>::kBytes : PairShape<false>::kBytes;
    const long long tiles = static_cast<long long>(r->tok_tiles) * r->out_tiles;
    r->grid = static_cast<int>(2 * std::min<long long>(tiles, num_sms / 2));
}

void plan_split(const LinearParams& p, const ClusterRoom& room, LinearPlan* r) {
    r->pair = 0;
    r->tok_tiles = static_cast<int>((p.tokens + kMaxTok - 1) / kMaxTok);
    const long long per = (p.tokens + r->tok_tiles - 1) / r->tok_tiles;
    r->tok_tile = static_cast<int>((per + 15) / 16 * 16);
    r->out_box = kRows;
    r->tok_box = r->tok_tile;
    r->tok_tiles = static_cast<int>((p.tokens + r->tok_tile - 1) / r->tok_tile);
    r->out_tiles = static_cast<int>((p.outputs + kRows - 1) / kRows);
    const long long tiles = static_cast<long long>(r->tok_tiles) * r->out_tiles;
    const long long k_steps = (p.width + kStep - 1) / kStep;
    // the reduction over as many CTAs as can run at once (a second wave costs more
    // than it gives) and have a step each
    r->splits = 1;
    for (int i = 1; i < 4; ++i)
        if (tiles <= room.of[i] && (1 << i) <= k_steps) r->splits = 1 << i;
    // rings within kSplitRings: raw stages of both operands, converted tokens (f16)
    const int stage = (kRows + r->tok_tile) * kStep, cvt = r->tok_tile * 256;
    r->cvt_stages = p.e4m3 ? 0 : (r->tok_tile <= 64 ? kMaxCvt : 2);
    r->stages = std::min(kMaxStages, (kSplitRings - r->cvt_stages * cvt) / stage);
    const long long per_rank = (k_steps + r->splits - 1) / r->splits;
    r->stages = static_cast<int>(std::min<long long>(r->stages, per_rank));
    // even (see the converters); two stages also hold the fp32 partial tile: (128 + t) 256
    // bytes against 512 t, t <= 128
    r->stages = std::max(2, r->stages / 2 * 2);
    r->smem = kSplitSmem;
}

}  // namespace

// The pair form's tile is 256 tokens high and its k-step costs the same at any
// width, so it pays where the split form's 128 x 128 tiles need a second wave
// (us, split and pair: 300 x 8192 x 2048 int8 27.7, 24.8, e4m3 17.7, 10.5; 512 x
// 8192 x 2048 28.6, 25.1 and 19.3, 10.8; 1280 x 2048 x 2048 27.8, 19.4 and 18.7,
// 10.3).  Within one wave the split form wins or is within 5%, the more the longer
// the reduction that it splits and the fewer the tiles (1024 x 2048 x 2048 14.5,
// 19.2 and 9.8, 9.9; 600 x 640 x 8192 15.3, 44.0 and 10.3, 23.3; 1024 x 2048 x 8192
// e4m3 22.1, 23.8; 4000 x 512 x 512 7.7, 10.2 and 6.5, 6.2).  Up to 256 tokens the
// pair's second CTA would have nothing to do, and int8 weights are not worth
// widening (256 x 8192 x 2048 14.5, 23.9 and 9.8, 9.9).
// A wave is counted in sm_103a's 152 SMs, not the current device's: the workspace's
// size follows from this rule, and its query asks no device.
bool linear_pair_form(long long tokens, long long outputs) {
    constexpr int kWave = 152;
    if (tokens <= 256) return false;
    return (tokens + kMaxTok - 1) / kMaxTok * ((outputs + kRows - 1) / kRows) > kWave;
}
bool linear_thin_form(long long tokens) { return tokens <= kThinTok; }

cudaError_t launch_linear_thin(const LinearParams& p, int num_sms, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>((p.outputs + kThinRows - 1) / kThinRows);
    // Few row blocks: 16 warps each, four steps ahead (95 registers).  Many: as many
    // warps as fill the GPU to 48 an SM, two steps ahead, so that more of them are
    // resident.  Measured each way: 2048 x 8192 int8 5.6 us against 7.5, 8192 x 2048
    // 6.2 against 5.0, 8192 x 8192 e4m3 16.9 against 12.7.
    const bool many = grid >= 2u * static_cast<unsigned>(num_sms);
    int warps = kThinMaxWarps;
    while (warps > 2 && ((many && static_cast<long long>(grid) * warps > 48ll * num_sms) ||
                         64ll * warps / 2 >= p.width))
        warps /= 2;
    const bool aligned = (reinterpret_cast<uintptr_t>(p.x) & 15u) == 0 &&
                         (reinterpret_cast<uintptr_t>(p.w) & 15u) == 0 &&
                         (p.tokens == 1 || p.x_stride % 16 == 0) && (p.outputs == 1 || p.w_stride % 16 == 0);
    const dim3 block(static_cast<unsigned>(32 * warps));
#define C3D_THIN(F8, NB, AL)                                                                     \
    (many ? launch_ex(linear_thin_kernel<F8, NB, AL, 2>, grid, block, 0, 1, stream, p)          \
          : launch_ex(linear_thin_kernel<F8, NB, AL, 4>, grid, block, 0, 1, stream, p))
    if (p.tokens <= 8) {
        if (p.e4m3) return aligned ? C3D_THIN(true, 1, true) : C3D_THIN(true, 1, false);
        return aligned ? C3D_THIN(false, 1, true) : C3D_THIN(false, 1, false);
    }
    if (p.e4m3) return aligned ? C3D_THIN(true, 2, true) : C3D_THIN(true, 2, false);
    return aligned ? C3D_THIN(false, 2, true) : C3D_THIN(false, 2, false);
#undef C3D_THIN
}

cudaError_t plan_linear(const LinearParams& p, int num_sms, LinearPlan* r) {
    *r = LinearPlan{};
    if (linear_pair_form(p.tokens, p.outputs)) {
        plan_pair(p, num_sms, r);
        return cudaSuccess;
    }
    ClusterRoom room;
    cudaError_t e = p.e4m3 ? allow_split_smem<true>() : allow_split_smem<false>();
    if (e == cudaSuccess) e = p.e4m3 ? cluster_room<true>(num_sms, &room) : cluster_room<false>(num_sms, &room);
    if (e == cudaSuccess) plan_split(p, room, r);
    return e;
}

cudaError_t launch_linear(const LinearMaps& maps, const LinearParams& p, const LinearPlan& plan,
                          cudaStream_t stream) {
    const int k_steps = static_cast<int>((p.width + kStep - 1) / kStep);
    if (plan.pair) {
        PairParams s{};
        s.p = p;
        s.m_tiles = plan.tok_tiles;
        s.n_tiles = plan.out_tiles;
        s.group_m = 8;
        s.k_steps = k_steps;
        s.f_group = make_fastdiv(static_cast<uint32_t>(s.group_m * s.n_tiles));
        s.f_gm = make_fastdiv(static_cast<uint32_t>(s.group_m));
        if (p.e4m3)
            return plan.tma_out ? launch_pair<true, true>(maps, s, plan, stream)
                                : launch_pair<true, false>(maps, s, plan, stream);
        return plan.tma_out ? launch_pair<false, true>(maps, s, plan, stream)
                            : launch_pair<false, false>(maps, s, plan, stream);
    }
    SplitParams s{};
    s.p = p;
    s.tok_tile = plan.tok_tile;
    s.out_tiles = plan.out_tiles;
    s.splits = plan.splits;
    s.k_steps = k_steps;
    s.stages = plan.stages;
    s.cvt = plan.cvt_stages;
    s.stage_bytes = static_cast<uint32_t>((kRows + plan.tok_tile) * kStep);
    s.cvt_bytes = static_cast<uint32_t>(plan.tok_tile * 256);
    return p.e4m3 ? launch_split<true>(maps.w, maps.x, s, plan, stream)
                  : launch_split<false>(maps.w, maps.x, s, plan, stream);
}

cudaError_t launch_stage_rows(RowJobs jobs, cudaStream_t stream) {
    unsigned blocks[2];
    for (int i = 0; i < 2; ++i) {
        RowJob& j = jobs.job[i];
        const long long words = j.pitch >> 4, total = j.rows * words;
        j.aligned = (reinterpret_cast<uintptr_t>(j.src) & 15u) == 0 && j.stride % 16 == 0;
        j.small = total < (1ll << 31) ? 1 : 0;
        j.by_words = make_fastdiv(static_cast<uint32_t>(words));
        blocks[i] = static_cast<unsigned>(std::min((total + 255) / 256, 152ll * 32));
    }
    jobs.blocks0 = blocks[0];
    return launch_ex(stage_rows_kernel, blocks[0] + blocks[1], 256, 0, 1, stream, jobs);
}

}  // namespace c3d
