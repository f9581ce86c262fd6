// token_paged_attention.cu -- attention of one new token of each sequence over a paged
// cache of keys and values in 8 or 16 bits.
//
// For a sequence of n cached tokens and each of its query heads
//     out = sum_t p_t v_t / sum_t p_t,   p_t = e^(s_t - m),   s_t = f(scale q.k_t)
// in one pass over the tokens with a running maximum m.  Memory-bound: a key and a
// value row are read once for the `group` query heads that share them.
//
// The work is every sequence's every key head, cut into units of a block of tokens for
// each warp and dealt to the CTAs in equal runs, whatever the lengths are (they are on the device
// only).  A run's ends may lie inside a key head: those CTAs leave (maximum, sum,
// output) in the workspace and a second launch joins them in order, so results do
// not depend on timing.  Within a CTA each warp takes blocks of 16 or 32 tokens (4 KB of
// keys and values at least: what a block costs beside its data is the same) on its own,
// through its own ring of TMA loads: two a run of 32, 16 or 8 tokens, as many as pages
// hold a multiple of, which leaves the load units to the shared-memory side.  Blocks at an
// edge of what is seen, in pages of other sizes, or in pages that are not there come word
// by word.
//
// Measured, 200 sequences of 1 to 8192 tokens, 8 key heads of 128 for 32 query heads, back
// to back: fp16 492 us; int8, capped, 297 us (84% of the floor's bytes at 6.8 TB/s): there the
// widening of codes and the weights are what it spends its time on beside memory, one
// instruction for two elements at best.  So are 64- and 80-wide heads (4.1 and 3.3 TB/s
// alone): a block's scores, exponentials and join cost the same for fewer bytes.  256-wide:
// 6.2 TB/s.  One sequence of 216000 tokens, e4m3: 86 us (5.3 TB/s).
//
// A block is two small matrix products per warp, tokens on the 16-row side:
//     S^T[16 tokens, 8 heads] = K q^T,    O^T[width, 8 heads] += V^T P^T
// The reduction index of the first, the rows of the second and the tokens' order may be
// permuted at will, so that a thread's operands are whole 16-byte words of the cache as
// it lies in memory, read without bank conflicts from 128-byte swizzled rows: row r of
// the product is token r ^ ((r & 1) << 2) of the block's eight.  Nothing is transposed
// but P (one 8 x 8 exchange).  Memory-bound work
// at 8 heads cannot fill a 128-row tensor-memory tile; the warp-level product reads
// its operands from registers, where 8-bit codes have to be widened anyway.
// int8 and e4m3 codes are exact in f16, as are queries times a power of two, so the
// scores carry fp32 sums of exact products; keys' scales multiply the scores.
// Values' scales go into the weights: p'_t = 2^(log2 p_t + log2 vscale_t - m'), m' the
// running maximum of that exponent, so that the f16 weights of the product have all
// of f16's 11 bits next to their maximum whatever the scales are; the sum of the
// weights takes 2^(log2 p_t - m') in fp32.
#include "token_attention_internal.h"
#include "token_paging.cuh"
#include "token_scores.cuh"

namespace c3d {

namespace {

constexpr float kTinyScale = 7.8886091e-31f;   // 2^-100
// Weights may exceed 1 by 2^4 before what they are relative to follows: the outputs are
// rarely rescaled, and a block of tokens without a new maximum needs no exchange of it.
constexpr float kLag = 4.0f;
// f16 weights are taken 2^11 times as large, next to f16's largest (2^15 of 2^16): those of
// 2^-35 of the largest one still count, where 2^-24 would be the least otherwise.  bf16
// weights have fp32's range and are taken 2^-24 times as large, so that sums over 2^20
// tokens hold for values up to the type's largest (results below 2^-112 lose bits instead).
constexpr float kUp = 11.0f, kDown = 1.0f / 2048.0f, kUpBf16 = -24.0f;
// Scores from here on (powers of two) are in steps of a quarter and more: f16 weights follow
// the maximum at once, as the steps could take lagging ones out of f16's range.
constexpr float kCoarse = 2097152.0f;

template <int ES, int DP>
struct Form {
    static constexpr int kWarps = 4;
    static constexpr int kStages = 2;
    static constexpr int kBoxes = (DP * ES + 127) / 128;   // 128-byte columns of a row
    static constexpr int kSubs = kBoxes == 1 ? 2 : 1;      // products of 16 tokens in a block
    static constexpr int kBlock = 16 * kSubs;
    static constexpr int kUnit = kWarps * kBlock;
    static constexpr int kKWords = DP * ES / 64;           // 16-byte words of a key row per thread
    static constexpr int kVBytes = DP * ES / 8;            // bytes of a value row per thread
    static constexpr int kVWord = kVBytes < 16 ? kVBytes : 16;
    static constexpr int kVWords = kVBytes / kVWord;
    static constexpr uint32_t kBox = 16u * 128u;           // 16 rows of 128 bytes, swizzled
    static constexpr uint32_t kVOff = kSubs * kBoxes * kBox;
    static constexpr uint32_t kStage = 2 * kVOff;
    static constexpr uint32_t kRing = kWarps * kStages * kStage;
    // behind the rings: a block's scales of keys and of values for each stage, then the
    // stages' barriers; 1024 for the rings' alignment
    static constexpr uint32_t kScales = 2u * kBlock * 4u;
    static constexpr uint32_t kBars = kRing + kWarps * kStages * kScales;
    static constexpr uint32_t kBytes = kBars + kWarps * kStages * 8u + 1024u;
};

// CTAs of an SM: three of one group of query heads, two of two (their registers), as far
// as shared memory goes: some compute while another joins its warps' results at a key
// head's end.  (Two instead of three: 200 ragged sequences of up to 8192, 8 key heads of 128,
// int8 340 us for 292, fp16 533 for 504; 16 key heads of 64, int8, 490 for 389; one of 216000
// e4m3 83 for 85.)
constexpr int ctas_of(int es, int dp, int ng) { return es * dp >= 512 ? 1 : ng == 1 ? 3 : 2; }

// Byte of 16-byte word `c` of row `r` in boxes of 16 rows (of 32, if there is one column).
__device__ __forceinline__ uint32_t word_at(int r, int c) {
    return static_cast<uint32_t>((c >> 3) * 2048 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    if (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// four codes as two f16 pairs
template <bool E4>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if (E4) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        // 0x6400 + u is 1024 + u in f16, u = code + 128
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 off = __half2half2(__ushort_as_half(0x6480));   // 1152
        const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
        lo = *reinterpret_cast<const uint32_t*>(&x);
        hi = *reinterpret_cast<const uint32_t*>(&y);
    }
}

template <int BYTES>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&w)[BYTES / 4]) {
    if constexpr (BYTES == 16)
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(addr));
    else
        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
}

// Bounded wait for a stage by the whole warp (see wait_bar).
__device__ __forceinline__ bool wait_block(uint32_t bar, uint32_t parity, int* status, unsigned long long limit_ns) {
    constexpr uint32_t kAll = 0xffffffffu;
    if (__all_sync(kAll, limit_ns ? mbar_try_wait(bar, parity) : mbar_test_wait(bar, parity))) return true;
    const long long t0 = clock64();
    const long long limit = static_cast<long long>(limit_ns > (1ull << 61) ? (1ull << 61) : limit_ns) * 2;
    while (!__any_sync(kAll, clock64() - t0 >= limit))
        if (__all_sync(kAll, mbar_try_wait(bar, parity))) return true;
    atomicExch(status, kStatusTimeout);
    return false;
}

// What a sequence's query sees: tokens [0, lead) and [from, length), as blocks:
// first those of the lead, then those from block `skip` on.
struct Seen {
    int length, lead, from;
    int lead_blocks, skip, blocks, units;
    bool bad;   // more tokens than the table holds
};

template <typename F>
__device__ __forceinline__ Seen seen_by(const PagedParams& p, int s) {
    constexpr int kBlock = F::kBlock;
    Seen v;
    const int n = p.lengths[s];
    v.bad = n > p.map.capacity;
    v.length = v.bad ? 1 : max(n, 0);
    v.from = p.window > 0 ? max(0, v.length - p.window) : 0;
    v.lead = p.prefix ? min(max(p.prefix[s], 0), v.length) : 0;
    if (v.from == 0) v.lead = 0;
    v.lead_blocks = (v.lead + kBlock - 1) / kBlock;
    v.skip = max(v.from / kBlock, v.lead_blocks);
    v.blocks = v.lead_blocks + max((v.length + kBlock - 1) / kBlock - v.skip, 0);
    v.units = p.whole ? v.blocks != 0 : (v.blocks + F::kWarps - 1) / F::kWarps;
    return v;
}

// Units of all sequences (one key head), summed over the block, and where unit
// `first` of the run falls: its sequence and the units before it.
template <typename F>
__device__ __forceinline__ long long sum_units(const PagedParams& p, long long* scratch) {
    constexpr int THREADS = 32 * F::kWarps;
    long long mine = 0;
    for (int s = threadIdx.x; s < p.sequences; s += THREADS) mine += seen_by<F>(p, s).units;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x / 32] = mine;
    __syncthreads();
    long long all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) all += scratch[w];
    __syncthreads();
    return all;
}

// The sequence s with before(s) <= unit < before(s) + units(s) (units of one key head
// row: `per` = key heads x blocks times its units), found by the first warp.
template <typename F>
__device__ __forceinline__ void find_unit(const PagedParams& p, long long per, long long unit,
                                          int* sequence, long long* before) {
    const int lane = threadIdx.x & 31;
    long long sum = 0;
    for (int s0 = 0; s0 < p.sequences; s0 += 32) {
        const int s = s0 + lane;
        const long long n = s < p.sequences ? seen_by<F>(p, s).units * per : 0;
        long long run = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, run, d);
            if (lane >= d) run += o;
        }
        const uint32_t over = __ballot_sync(0xffffffffu, sum + run > unit);
        if (over) {
            const int k = __ffs(over) - 1;
            *sequence = s0 + k;
            *before = sum + __shfl_sync(0xffffffffu, run - n, k);
            return;
        }
        sum += __shfl_sync(0xffffffffu, run, 31);
    }
    *sequence = p.sequences;
    *before = sum;
}

// A partial result in the workspace: [query][max, sum, out[DP]]
template <int DP>
constexpr int kPartial = 16 * (DP + 2);

// KIND: kTokInt8, kTokE4m3, kTokBf16 or kTokF16; QBF: the queries are bf16; NG: groups
// of eight query heads.
template <int KIND, bool QBF, int DP, int NG>
__global__ void __launch_bounds__(32 * Form<KIND == kTokBf16 || KIND == kTokF16 ? 2 : 1, DP>::kWarps,
                                  ctas_of(KIND == kTokBf16 || KIND == kTokF16 ? 2 : 1, DP, NG))
    paged_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                 const __grid_constant__ PagedParams p) {
    constexpr bool kCodes = KIND == kTokInt8 || KIND == kTokE4m3;
    constexpr int ES = kCodes ? 1 : 2;
    using F = Form<ES, DP>;
    constexpr int kWarps = F::kWarps, kBlock = F::kBlock;
    constexpr bool kBf = KIND == kTokBf16;
    constexpr int kSteps = DP / 16;   // k-steps of the first product
    constexpr int kTiles = DP / 16;   // 16-row tiles of the second's output
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    unsigned char* smem = smem_raw + (base - raw);
    __shared__ long long s_scratch[kWarps];
    __shared__ int s_seq;
    __shared__ long long s_before;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3;
    const uint32_t ring = base + warp * (F::kStages * F::kStage);
    const uint32_t scales = base + F::kRing + warp * (F::kStages * F::kScales);
    const uint32_t full0 = base + F::kBars + warp * (F::kStages * 8u);
    if (lane == 0) {
        for (int i = 0; i < F::kStages; ++i) mbar_init(full0 + 8 * i, 1);
        fence_mbar_init();
        if (p.rows_box) {
            prefetch_tmap(&k_map);
            prefetch_tmap(&v_map);
        }
    }
    __syncwarp();
    // (the next launch is not let in early: its CTAs, waiting, kept this one's and the join's
    // from their places: 200 ragged sequences back to back 423 us so, 297 without)
    griddep_wait();

    // this CTA's run of units
    const long long per = static_cast<long long>(p.kv_heads) * p.blocks;
    const long long c = blockIdx.x, grid = gridDim.x;
    // (equal runs; the first total % grid are one longer.  Key heads that are not split have a
    // unit and a CTA each, those of sequences that see nothing too)
    const long long total = p.whole ? grid : sum_units<F>(p, s_scratch) * per;
    const long long share = total / grid, longer = total % grid;
    long long unit = c * share + min(c, longer);
    const long long end = unit + share + (c < longer ? 1 : 0);
    if (threadIdx.x == 0 && !p.whole) p.jobs[c] = make_int4(0, 0, 0, 0);
    // sequences that see nothing get zeros
    for (long long s = c; s < p.sequences; s += grid) {
        if (seen_by<F>(p, static_cast<int>(s)).units) continue;
        for (int i = threadIdx.x; i < p.kv_heads * p.group * p.width; i += kWarps * 32) {
            unsigned char* o = p.out + (s * p.out_seq + (i / p.width) * p.out_head + i % p.width) * 2;
            *reinterpret_cast<uint16_t*>(o) = 0;
        }
    }
    if (unit >= end) return;
    int seq = static_cast<int>(c / per);
    long long before = seq * per;
    if (p.whole) {
        if (seen_by<F>(p, seq).units == 0) return;
    } else {
        if (warp == 0) {
            int s;
            long long b;
            find_unit<F>(p, per, unit, &s, &b);
            if (lane == 0) {
                s_seq = s;
                s_before = b;
            }
        }
        __syncthreads();
        seq = s_seq;
        before = s_before;
    }

    int stage = 0;        // the ring's next stage, and its phase
    uint32_t phase = 0;
    bool dead = false;    // a wait ran out: no more work, but the CTA's barriers are kept
    // where this thread's words lie: the key rows r0 and r0 + 8 (8 rows: 1024 bytes on) and the
    // values' rows of the product's 2q, 2q + 1, 2q + 8 and 2q + 9
    const int r0 = r ^ ((r & 1) << 2);
    const uint32_t k_at = word_at(r0, q), v_at0 = word_at(2 * q, F::kVWord == 16 ? r : r >> 1),
                   v_at1 = word_at((2 * q + 1) ^ 4, F::kVWord == 16 ? r : r >> 1);
    const uint32_t v_half = F::kVOff + (F::kVWord == 16 ? 0u : (r & 1) * 8u);
    const uint32_t block_bytes = F::kStage + (kCodes ? F::kScales : 0u);
    // lanes that load a block's runs of rows_box tokens
    const int runs = p.rows_box ? kBlock / p.rows_box : 1, run_at = min(lane, runs - 1) * p.rows_box;
    while (unit < end) {
        const Seen see = seen_by<F>(p, seq);
        if (see.units == 0) {
            ++seq;
            continue;
        }
        const long long in = unit - before;
        const int hb = static_cast<int>(in / see.units);
        const int u0 = static_cast<int>(in - static_cast<long long>(hb) * see.units);
        const int u1 = static_cast<int>(min(static_cast<long long>(see.units), u0 + (end - unit)));
        const int head = hb / p.blocks, qb = hb - head * p.blocks;
        const int heads_here = min(p.group - qb * 8 * NG, 8 * NG);
        const int qh0 = head * p.group + qb * 8 * NG;

        // ---- the queries: B operands of the first product
        uint32_t bq[NG][kSteps][2];
        float qscale[NG][2];   // of columns 2q, 2q + 1: multiplies the scores
        float slope[NG][2];
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            const int h = 8 * n + r;
            const bool have = h < heads_here;
            const uint16_t* src = reinterpret_cast<const uint16_t*>(p.q) + seq * p.q_seq +
                                  static_cast<long long>(qh0 + (have ? h : 0)) * p.q_head;
            float top = 0.0f;
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                // the elements of this thread's word of the key rows
                constexpr int E = 16 / ES;   // elements of a word
                const int d = (st / (E / 4)) * 4 * E + q * E + (st % (E / 4)) * 4;
                uint32_t w[2] = {0u, 0u};
                if (have && d < p.width) {
                    w[0] = src[d] | static_cast<uint32_t>(src[d + 1]) << 16;
                    w[1] = src[d + 2] | static_cast<uint32_t>(src[d + 3]) << 16;
                }
                bq[n][st][0] = w[0];
                bq[n][st][1] = w[1];
                if (kCodes && QBF) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        top = fmaxf(top, fabsf(__uint_as_float(w[i] << 16)));
                        top = fmaxf(top, fabsf(__uint_as_float(w[i] & 0xFFFF0000u)));
                    }
                }
            }
            float back = 1.0f;
            if (kCodes && QBF) {
                // bf16 queries to f16 by a power of two that brings the largest to [2^7, 2^8):
                // exact but for elements below 2^-21 of it, off by 2^-33 of it at most
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int ex = static_cast<int>(__float_as_uint(top) >> 23);   // biased
                const int sh = min(max(261 - ex, 1), 253);                     // 2^(sh - 127): ex -> 134
                const float up = __uint_as_float(static_cast<uint32_t>(sh) << 23);
                back = __uint_as_float(static_cast<uint32_t>(254 - sh) << 23);
#pragma unroll
                for (int st = 0; st < kSteps; ++st)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t w = bq[n][st][i];
                        const __half2 x = __floats2half2_rn(__uint_as_float(w << 16) * up,
                                                            __uint_as_float(w & 0xFFFF0000u) * up);
                        bq[n][st][i] = *reinterpret_cast<const uint32_t*>(&x);
                    }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // row 2q + j of this group is held by lanes 4 * (2q + j) ...
                // (without a cap the change to powers of two goes along)
                qscale[n][j] = __shfl_sync(0xffffffffu, back, 4 * (2 * q + j)) * p.scale * (p.cap > 0.0f ? 1.0f : kLog2e);
                const int hh = 8 * n + 2 * q + j;
                slope[n][j] = p.slopes && hh < heads_here ? p.slopes[qh0 + hh] * kLog2e : 0.0f;
            }
        }

        float o[NG][kTiles][4];
        float m[NG][2], l[NG][2];
#pragma unroll
        for (int n = 0; n < NG; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[n][j] = -INFINITY;
                l[n][j] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][i][j] = 0.0f;
        }

        // ---- the warp's blocks
        const int b0 = u0 * kWarps, b1 = p.whole ? see.blocks : min(u1 * kWarps, see.blocks);
        auto token_of = [&](int b) {
            return (b < see.lead_blocks ? b : b - see.lead_blocks + see.skip) * kBlock;
        };
        auto visible = [&](int t) { return t < see.length && (t >= see.from || t < see.lead); };
        const int32_t* table = p.map.table + seq * p.map.table_stride;
        // the page of this lane's run of the next block to ask for
        const bool look = p.rows_box != 0 && !see.bad;
        int page_ahead = 0;
        auto look_ahead = [&](int b) {
            if (!look || b >= b1) return;
            const int t = min(token_of(b) + run_at, see.length - 1);
            page_ahead = table[fdiv(static_cast<uint32_t>(t), p.map.by_page)];
        };
        look_ahead(b0 + warp);
        uint32_t slow = 0;   // stages that were filled word by word (bits)
        auto issue = [&](int b, int st) {
            const uint32_t dst = ring + st * F::kStage, sdst = scales + st * F::kScales, bar = full0 + 8 * st;
            const int t0 = token_of(b), page = page_ahead;
            look_ahead(b + kWarps);
            // (all tokens are seen, in pages that are there)
            if (look && t0 + kBlock <= see.length && (t0 >= see.from || t0 + kBlock <= see.lead) &&
                __all_sync(0xffffffffu, page >= 0 && page < p.map.pages)) {
                slow &= ~(1u << st);
                if (lane == 0) mbar_arrive_expect_tx(bar, block_bytes);
                __syncwarp();
                if (lane < runs) {
                    const int t = t0 + run_at;
                    const int off = t - static_cast<int>(fdiv(static_cast<uint32_t>(t), p.map.by_page) * p.map.by_page.d);
#pragma unroll
                    for (int x = 0; x < F::kBoxes; ++x) {
                        tma_load_4d(dst + x * F::kBox + run_at * 128u, &k_map, bar, x * (128 / ES), off, head, page);
                        tma_load_4d(dst + F::kVOff + x * F::kBox + run_at * 128u, &v_map, bar, x * (128 / ES), off, head,
                                    page);
                    }
                    if (kCodes) {
                        const long long at = page * p.map.scale_page_stride + head * p.map.scale_head_stride + off;
                        bulk_load_1d(sdst + run_at * 4u, p.k_scale + at, p.rows_box * 4u, bar);
                        bulk_load_1d(sdst + (kBlock + run_at) * 4u, p.v_scale + at, p.rows_box * 4u, bar);
                    }
                }
                return;
            }
            // word by word: a block's edge, pages that end in it, pages that are not there.  Each
            // lane looks its token up, so that the table is waited for once: every sequence has
            // such a block at its end (200 ragged sequences, int8: 336 us, 408 token by token)
            slow |= 1u << st;
            const int mine = t0 + lane % kBlock;
            long long row = 0, sc = 0;
            const bool seen = visible(mine), have = !see.bad && seen && token_row(p.map, seq, mine, head, &row, &sc);
            const uint32_t all = __ballot_sync(0xffffffffu, have);
            // (rows of one column: two tokens at a time)
            constexpr int kWords = F::kBoxes * 16, kAtOnce = kWords == 16 ? 2 : 1;   // a key's words, then a value's
#pragma unroll 1
            for (int i0 = 0; i0 < kBlock; i0 += kAtOnce) {
                const int i = i0 + (kAtOnce == 2 ? lane >> 4 : 0);
                const long long at = __shfl_sync(0xffffffffu, row, i);
#pragma unroll
                for (int c = lane % kWords; c < kWords; c += 32) {
                    const int w = c % (F::kBoxes * 8);
                    const bool value = c >= F::kBoxes * 8, load = (all >> i & 1u) && w * 16 < p.width * ES;
                    cp_async<16>(dst + (value ? F::kVOff : 0u) + word_at(i, w),
                                 (value ? p.v : p.k) + (load ? at + w * 16 : 0), load ? 16u : 0u);
                }
            }
            // NaN for the scale of a token whose page is missing, which spoils the row
            const bool want = seen || see.bad;
#pragma unroll
            for (int e = lane; e < 2 * kBlock; e += 32) {
                if (kCodes && (have || !want))
                    cp_async<4>(sdst + e * 4u, (e < kBlock ? p.k_scale : p.v_scale) + sc, have ? 4u : 0u);
                else
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(sdst + e * 4u),
                                 "f"(want && !have ? __uint_as_float(kNanBits) : 1.0f)
                                 : "memory");
            }
        };
        {
            int st = stage;
#pragma unroll
            for (int i = 0; i < F::kStages - 1; ++i) {
                const int b = b0 + warp + i * kWarps;
                if (b < b1 && !dead) issue(b, st);
                if (++st == F::kStages) st = 0;
            }
        }
        for (int b = b0 + warp; b < b1 && !dead; b += kWarps) {
            {
                const int nb = b + (F::kStages - 1) * kWarps;
                int ns = stage + F::kStages - 1;
                if (ns >= F::kStages) ns -= F::kStages;
                if (nb < b1) issue(nb, ns);
            }
            const bool by_words = slow >> stage & 1u;
            if (by_words) {
                // (the barrier's phase passes without a load)
                cp_async_wait_all();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full0 + 8 * stage);
            }
            if (!wait_block(full0 + 8 * stage, phase, p.status, p.wait_ns)) {
                // what is on its way lands before the shared memory is given up
                cp_async_wait_all();
                dead = true;
                for (int i = 0; i < F::kStages && b + i * kWarps < b1; ++i) {
                    const int st = (stage + i) % F::kStages;
                    if (!(slow >> st & 1u)) drain_wait(full0 + 8 * st, stage + i < F::kStages ? phase : phase ^ 1u);
                }
                break;
            }
            const uint32_t src = ring + stage * F::kStage, ssrc = scales + stage * F::kScales;
            const int t0 = token_of(b);

            // ---- scores (two sums: a product waits for the one before in its own)
            float s2[F::kSubs][NG][4];   // in powers of two, but before a cap
            float lv[F::kSubs][2];
            bool none[F::kSubs][2];      // values too small to count
#pragma unroll
            for (int u = 0; u < F::kSubs; ++u) {
                float sc[NG][4], sd[NG][4];
#pragma unroll
                for (int n = 0; n < NG; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[n][j] = sd[n][j] = 0.0f;
#pragma unroll
                for (int w = 0; w < F::kKWords; ++w) {
                    uint32_t x[4], y[4];
                    // (the next word is in the other half of the row, its eighth in the next box)
                    const uint32_t at = src + (u + (w >> 1)) * F::kBox + (k_at ^ ((w & 1) * 64u));
                    lds<16>(at, x);
                    lds<16>(at + 1024u, y);
                    if constexpr (kCodes) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t x0, x1, y0, y1;
                            widen4<KIND == kTokE4m3>(x[i], x0, x1);
                            widen4<KIND == kTokE4m3>(y[i], y0, y1);
#pragma unroll
                            for (int n = 0; n < NG; ++n)
                                mma16816<false>(i & 1 ? sd[n] : sc[n], x0, y0, x1, y1, bq[n][4 * w + i][0],
                                                bq[n][4 * w + i][1]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int n = 0; n < NG; ++n)
                                mma16816<kBf>(i & 1 ? sd[n] : sc[n], x[2 * i], y[2 * i], x[2 * i + 1], y[2 * i + 1],
                                              bq[n][2 * w + i][0], bq[n][2 * w + i][1]);
                    }
                }
                // this thread's tokens are t0 + 16 u + r0 and the eighth after it
                float ks[2] = {1.0f, 1.0f};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    lv[u][i] = 0.0f;
                    none[u][i] = false;
                    if (!kCodes && !by_words) continue;
                    const uint32_t at = ssrc + (16 * u + r0 + 8 * i) * 4u;
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ks[i]) : "r"(at));
                    if (kCodes) {
                        float vs;
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vs) : "r"(at + kBlock * 4u));
                        none[u][i] = vs < kTinyScale;
                        lv[u][i] = none[u][i] ? -100.0f : lg2(vs);
                    }
                }
#pragma unroll
                for (int n = 0; n < NG; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s2[u][n][j] = (sc[n][j] + sd[n][j]) * (ks[j >> 1] * qscale[n][j & 1]);
            }
            if (p.cap > 0.0f) {
                // all of the warp's scores within the polynomial's reach (most blocks), or each as it lies
                float top = 0.0f;
#pragma unroll
                for (int u = 0; u < F::kSubs; ++u)
#pragma unroll
                    for (int n = 0; n < NG; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) top = fmaxf(top, fabsf(s2[u][n][j]));
                const bool small = __all_sync(0xffffffffu, top * p.inv_cap <= kTanhReach);
#pragma unroll
                for (int u = 0; u < F::kSubs; ++u)
#pragma unroll
                    for (int n = 0; n < NG; ++n)
#pragma unroll
                        for (int j = 0; j < 4; j += 2) {
                            float (&s)[4] = s2[u][n];
                            if (small) {
                                uint32_t a, b;
                                split(cap_pair(two(__float_as_uint(s[j]), __float_as_uint(s[j + 1])), two(p.inv_cap)), a, b);
                                s[j] = __uint_as_float(a);
                                s[j + 1] = __uint_as_float(b);
                            } else {
                                s[j] = cap_score(s[j], p.cap, p.inv_cap) * kLog2e;
                                s[j + 1] = cap_score(s[j + 1], p.cap, p.inv_cap) * kLog2e;
                            }
                        }
            }
            if (p.slopes) {
#pragma unroll
                for (int u = 0; u < F::kSubs; ++u)
#pragma unroll
                    for (int n = 0; n < NG; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            s2[u][n][j] -= slope[n][j & 1] *
                                           static_cast<float>(see.length - 1 - (t0 + 16 * u + r0 + 8 * (j >> 1)));
            }
            // ---- weights
            if (by_words) {   // (others are seen whole)
#pragma unroll
                for (int u = 0; u < F::kSubs; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (!visible(t0 + 16 * u + r0 + 8 * i) && !see.bad) {
#pragma unroll
                            for (int n = 0; n < NG; ++n) s2[u][n][2 * i] = s2[u][n][2 * i + 1] = -INFINITY;
                        }
            }
            float best[NG][2];   // of this thread's tokens
            bool rise = false;
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    best[n][j] = fmaxf(s2[0][n][j] + lv[0][0], s2[0][n][j + 2] + lv[0][1]);
                    if (F::kSubs == 2)
                        best[n][j] = fmaxf(best[n][j], fmaxf(s2[F::kSubs - 1][n][j] + lv[F::kSubs - 1][0],
                                                             s2[F::kSubs - 1][n][j + 2] + lv[F::kSubs - 1][1]));
                    rise |= best[n][j] > m[n][j] + kLag || (!kBf && fabsf(best[n][j]) >= kCoarse);
                }
            if (__any_sync(0xffffffffu, rise)) {
                // all tokens' maximum, and everything relative to it
#pragma unroll
                for (int n = 0; n < NG; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float top = best[n][j];
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        const float now = fmaxf(m[n][j], top);
                        const float fall = now == -INFINITY ? 1.0f : ex2(m[n][j] - now);
                        m[n][j] = now;
                        l[n][j] *= fall;
#pragma unroll
                        for (int i = 0; i < kTiles; ++i) {
                            o[n][i][j] *= fall;
                            o[n][i][j + 2] *= fall;
                        }
                    }
            }
            // ---- output
#pragma unroll
            for (int u = 0; u < F::kSubs; ++u) {
                uint32_t bp[NG][2];
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    float pw[4];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        // (the sum of weights without values' scales: the factor stays out of it, as it
                        // is large enough where these are small)
                        const float base = m[n][j] == -INFINITY ? 0.0f : m[n][j] - (kCodes ? 0.0f : kBf ? kUpBf16 : kUp);
                        const float x = s2[u][n][j] - base, y = s2[u][n][j + 2] - base;
                        pw[j] = none[u][0] ? 0.0f : ex2(x + (kCodes ? lv[u][0] + kUp : 0.0f));
                        pw[j + 2] = none[u][1] ? 0.0f : ex2(y + (kCodes ? lv[u][1] + kUp : 0.0f));
                        l[n][j] += kCodes ? ex2(x) + ex2(y) : pw[j] + pw[j + 2];
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t w16;
                        if (kBf) {
                            w16 = pack_bf16x2(pw[2 * i], pw[2 * i + 1]);
                        } else {
                            const __half2 x = __floats2half2_rn(pw[2 * i], pw[2 * i + 1]);
                            w16 = *reinterpret_cast<const uint32_t*>(&x);
                        }
                        bp[n][i] = transpose8x8(w16);
                    }
                }
#pragma unroll
                for (int w = 0; w < F::kVWords; ++w) {
                    uint32_t x[4][F::kVWord / 4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        lds<F::kVWord>(src + v_half + (i & 1 ? v_at1 : v_at0) + (i >> 1) * 1024u + (u + w) * F::kBox, x[i]);
#pragma unroll
                    for (int i = 0; i < F::kVWord / 4; ++i) {
                        // pairs of tokens side by side, an element (and the next) each
                        if constexpr (kCodes) {
                            uint32_t a[2][4];   // [tokens of the half][elements 0..3]
#pragma unroll
                            for (int hlf = 0; hlf < 2; ++hlf) {
                                const uint32_t lo = __byte_perm(x[2 * hlf][i], x[2 * hlf + 1][i], 0x5140);
                                const uint32_t hi = __byte_perm(x[2 * hlf][i], x[2 * hlf + 1][i], 0x7362);
                                widen4<KIND == kTokE4m3>(lo, a[hlf][0], a[hlf][1]);
                                widen4<KIND == kTokE4m3>(hi, a[hlf][2], a[hlf][3]);
                            }
                            constexpr int kPer = F::kVWord / 2;   // tiles of a word
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int n = 0; n < NG; ++n)
                                    mma16816<false>(o[n][w * kPer + 2 * i + k], a[0][2 * k], a[0][2 * k + 1],
                                                    a[1][2 * k], a[1][2 * k + 1], bp[n][0], bp[n][1]);
                        } else {
                            const uint32_t a0 = __byte_perm(x[0][i], x[1][i], 0x5410);
                            const uint32_t a1 = __byte_perm(x[0][i], x[1][i], 0x7632);
                            const uint32_t a2 = __byte_perm(x[2][i], x[3][i], 0x5410);
                            const uint32_t a3 = __byte_perm(x[2][i], x[3][i], 0x7632);
#pragma unroll
                            for (int n = 0; n < NG; ++n)
                                mma16816<kBf>(o[n][w * 4 + i], a0, a1, a2, a3, bp[n][0], bp[n][1]);
                        }
                    }
                }
            }
            __syncwarp();   // all lanes have read this stage
            if (++stage == F::kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }

        // ---- the warps' results meet in shared memory, over the rings
        __syncthreads();
        constexpr int kRow = DP + 4;
        float* so = reinterpret_cast<float*>(smem);                   // [warp][query][kRow]
        float* sm = so + kWarps * 8 * NG * kRow;                      // [warp][query][2]
#pragma unroll
        for (int n = 0; n < NG; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float sum = l[n][j];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int at = warp * 8 * NG + 8 * n + 2 * q + j;
                if (r == 0) {
                    sm[2 * at] = m[n][j];
                    sm[2 * at + 1] = sum;
                }
                constexpr int E = F::kVWord / ES;   // elements of a word
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    const int d = (2 * i / E) * 8 * E + r * E + (2 * i) % E;
                    *reinterpret_cast<float2*>(so + at * kRow + d) = make_float2(o[n][i][j], o[n][i][j + 2]);
                }
            }
        }
        __syncthreads();
        const bool whole = u0 == 0 && u1 == see.units;
        const int slot = u0 == 0 ? 1 : 0;
        float* part = p.partial + (c * 2 + slot) * kPartial<DP>;
        for (int i = threadIdx.x; i < heads_here * (DP / 2); i += kWarps * 32) {
            const int h = i / (DP / 2), d = 2 * (i - h * (DP / 2));
            if (d >= p.width) continue;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[2 * (w * 8 * NG + h)]);
            const float base = top == -INFINITY ? 0.0f : top;
            float x = 0.0f, y = 0.0f, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const int at = w * 8 * NG + h;
                const float f = ex2(sm[2 * at] - base);
                const float2 v = *reinterpret_cast<const float2*>(so + at * kRow + d);
                x += v.x * f;
                y += v.y * f;
                sum += sm[2 * at + 1] * f;
            }
            if (kCodes) {
                x *= kDown;
                y *= kDown;
            }
            if (whole) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                uint32_t w;
                if (QBF) {
                    w = pack_bf16x2(x * inv, y * inv);
                } else {
                    const __half2 hv = __floats2half2_rn(x * inv, y * inv);
                    w = *reinterpret_cast<const uint32_t*>(&hv);
                }
                uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) + seq * p.out_seq +
                                static_cast<long long>(qh0 + h) * p.out_head + d;
                dst[0] = static_cast<uint16_t>(w);
                dst[1] = static_cast<uint16_t>(w >> 16);
            } else {
                if (d == 0) {
                    part[h * (DP + 2)] = top;
                    part[h * (DP + 2) + 1] = sum;
                }
                *reinterpret_cast<float2*>(part + h * (DP + 2) + 2 + d) = make_float2(x, y);
            }
        }
        if (u0 == 0 && !whole && threadIdx.x == 0) {
            // this CTA owns the join: how many CTAs share this key head
            const long long last = before + static_cast<long long>(hb + 1) * see.units - 1;
            const long long split = longer * (share + 1);
            const long long c1 = last < split ? last / (share + 1) : longer + (last - split) / share;
            p.jobs[c] = make_int4(seq, qh0, heads_here, static_cast<int>(c1 - c));
        }
        fence_proxy_async_smem();   // the next loads come over what was written here
        __syncthreads();
        unit += u1 - u0;
        if (u1 == see.units && hb + 1 == per) {
            before += static_cast<long long>(see.units) * per;
            ++seq;
        }
    }
}

// Joins the partial results of the key heads that several CTAs share, in the order of
// their tokens: block c joins the one that begins in CTA c's run and goes on beyond it.
// Every part's weight is taken first, so that the sums' loads do not wait for one another.
constexpr int kWholeTokens = 384;
constexpr int kMaxParts = 480;   // and CTAs of the first launch

template <bool QBF, int DP>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedParams p) {
    __shared__ float weight[16][kMaxParts];
    __shared__ float total[16];
    griddep_wait();
    const int c = blockIdx.x, lane = threadIdx.x & 31;
    const int4 job = p.jobs[c];   // sequence, first query head, heads, further parts
    if (job.w == 0) return;
    // part k of head h: the owner's second slot, then the others' first ones
    auto part = [&](int k, int h) {
        return p.partial + ((static_cast<long long>(c) + k) * 2 + (k == 0)) * kPartial<DP> + h * (DP + 2);
    };
    // a few parts: every thread takes their weights itself, all loads at once (16 heads of 64,
    // bf16, in a graph: 400 tokens, 4 parts, 7.5 us, 8.3 through the warps' weights; 800, 7
    // parts, 8.0 and 8.5; but 900, 8 parts, 8.4 and 7.6)
    constexpr int kFew = 7;
    const bool few = job.w < kFew;
    for (int h = threadIdx.x >> 5; h < job.z && !few; h += 8) {
        float top = -INFINITY;
        for (int k = lane; k <= job.w; k += 32) top = fmaxf(top, part(k, h)[0]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float base = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
        for (int k = lane; k <= job.w; k += 32) {
            const float f = ex2(part(k, h)[0] - base);
            weight[h][k] = f;
            sum += part(k, h)[1] * f;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) total[h] = sum;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < job.z * (DP / 2); i += 256) {
        const int h = i / (DP / 2), d = 2 * (i - h * (DP / 2));
        if (d >= p.width) continue;
        float x = 0.0f, y = 0.0f, all = 0.0f;
        if (few) {
            float2 ms[kFew], v[kFew];
#pragma unroll
            for (int k = 0; k < kFew; ++k) {
                const float* f = part(min(k, job.w), h);
                ms[k] = *reinterpret_cast<const float2*>(f);
                v[k] = *reinterpret_cast<const float2*>(f + 2 + d);
            }
            float top = ms[0].x;
#pragma unroll
            for (int k = 1; k < kFew; ++k) top = fmaxf(top, ms[k].x);
            const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int k = 0; k < kFew; ++k) {
                if (k > job.w) break;
                const float f = ex2(ms[k].x - base);
                x = fmaf(v[k].x, f, x);
                y = fmaf(v[k].y, f, y);
                all = fmaf(ms[k].y, f, all);
            }
        } else {
#pragma unroll 8
            for (int k = 0; k <= job.w; ++k) {
                const float f = weight[h][k];
                const float2 v = *reinterpret_cast<const float2*>(part(k, h) + 2 + d);
                x = fmaf(v.x, f, x);
                y = fmaf(v.y, f, y);
            }
            all = total[h];
        }
        const float inv = all == 0.0f ? 0.0f : 1.0f / all;
        uint32_t w;
        if (QBF) {
            w = pack_bf16x2(x * inv, y * inv);
        } else {
            const __half2 hv = __floats2half2_rn(x * inv, y * inv);
            w = *reinterpret_cast<const uint32_t*>(&hv);
        }
        uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) + job.x * p.out_seq +
                        static_cast<long long>(job.y + h) * p.out_head + d;
        dst[0] = static_cast<uint16_t>(w);
        dst[1] = static_cast<uint16_t>(w >> 16);
    }
}

int padded(int width) { return width <= 64 ? 64 : width <= 128 ? 128 : 256; }

template <int KIND, bool QBF, int DP, int NG>
cudaError_t run(const PagedMaps& maps, const PagedParams& p0, cudaStream_t stream) {
    constexpr int ES = KIND == kTokBf16 || KIND == kTokF16 ? 2 : 1;
    using F = Form<ES, DP>;
    constexpr int kCtas = ctas_of(ES, DP, NG);
    PagedParams p = p0;
    p.grid = p.whole ? p.sequences * p.kv_heads * p.blocks : p0.grid < kCtas * p0.num_sms ? p0.grid : kCtas * p0.num_sms;
    constexpr size_t meet = sizeof(float) * F::kWarps * 8 * NG * (DP + 4 + 2);
    static_assert(meet <= F::kRing, "the warps' results meet over the rings");
    constexpr size_t smem = F::kBytes;
    static std::atomic<int> slots[kMaxDevices];
    cudaError_t e = ensure_dynamic_smem(paged_kernel<KIND, QBF, DP, NG>, smem, slots);
    if (e != cudaSuccess) return e;
    e = launch_ex(paged_kernel<KIND, QBF, DP, NG>, static_cast<unsigned>(p.grid), dim3(32 * F::kWarps), smem, 1,
                  stream, maps.k, maps.v, p);
    // (a table of no more than a unit's tokens leaves nothing to join)
    if (e != cudaSuccess || p.whole || p.grid == 1 || p.map.capacity <= F::kUnit) return e;
    return launch_ex(paged_join_kernel<QBF, DP>, static_cast<unsigned>(p.grid), dim3(256), 0, 1, stream, p);
}

template <int KIND, bool QBF>
cudaError_t by_width(const PagedMaps& m, const PagedParams& p, cudaStream_t stream) {
    const bool two = p.group > 8;
    if (p.width <= 64) return two ? run<KIND, QBF, 64, 2>(m, p, stream) : run<KIND, QBF, 64, 1>(m, p, stream);
    if (p.width <= 128) return two ? run<KIND, QBF, 128, 2>(m, p, stream) : run<KIND, QBF, 128, 1>(m, p, stream);
    return run<KIND, QBF, 256, 1>(m, p, stream);
}

}  // namespace

// Query heads of one pass: 8, or 16 where more share a key head (256-wide heads have no
// registers for 16).
static int pass_heads(long long group, int width) { return group > 8 && width <= 128 ? 16 : 8; }

// Key heads are not split where tables hold few tokens and each head has a CTA of its own
// among those that run at once: there is nothing to join then, no workspace to allocate,
// and no unit to look for.  A CTA alone takes longer than several and the join from about 450
// tokens on (one sequence in a graph, 8 key heads of 128, e4m3: 333 tokens 7.4 us for 8.0, 384
// 6.6 for 7.8, 450 8.5 for 8.0, 650 10.6 for 8.5; 16 of 64, bf16: 384 5.4 for 7.0, 450 6.9 for
// 7.7, 650 8.4 for 7.9); outside a graph the host's time of a second launch and the workspace
// is 2 us of 17.
bool paged_whole(long long sequences, long long kv_heads, long long group, int width,
                 long long capacity, int num_sms) {
    const long long blocks = (group + pass_heads(group, width) - 1) / pass_heads(group, width);
    return capacity <= kWholeTokens && sequences <= num_sms && kv_heads * blocks * sequences <= 2ll * num_sms;
}

int paged_grid(long long sequences, long long kv_heads, long long group, int width,
               long long capacity, int num_sms) {
    // three CTAs an SM at most, as far as there can be units
    const long long blocks = (group + pass_heads(group, width) - 1) / pass_heads(group, width);
    const long long units = (capacity + 63) / 64;   // (the smallest form's)
    const long long most = 3ll * num_sms < kMaxParts ? 3ll * num_sms : kMaxParts;
    if (units >= most) return static_cast<int>(most);
    long long n = units * kv_heads * blocks;
    n = n >= most || sequences >= most ? most : n * sequences;
    return static_cast<int>(n < 1 ? 1 : n > most ? most : n);
}

size_t paged_workspace(int grid, int width) {
    const size_t part = 16 * (static_cast<size_t>(padded(width)) + 2) * sizeof(float);
    return static_cast<size_t>(grid) * (2 * part + sizeof(int4));
}

cudaError_t launch_paged(const PagedMaps& maps, const PagedParams& p0, int q_dtype, int cache_dtype,
                         cudaStream_t stream) {
    PagedParams p = p0;
    p.blocks = (p.group + pass_heads(p.group, p.width) - 1) / pass_heads(p.group, p.width);
    const bool bf = q_dtype == kTokBf16;
    if (cache_dtype == kTokInt8)
        return bf ? by_width<kTokInt8, true>(maps, p, stream) : by_width<kTokInt8, false>(maps, p, stream);
    if (cache_dtype == kTokE4m3)
        return bf ? by_width<kTokE4m3, true>(maps, p, stream) : by_width<kTokE4m3, false>(maps, p, stream);
    return bf ? by_width<kTokBf16, true>(maps, p, stream) : by_width<kTokF16, false>(maps, p, stream);
}

}  // namespace c3d
