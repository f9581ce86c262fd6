// token_packed_attention.cu -- attention within documents packed one after the other.
//
// For each document, head and query i:  out = sum_j p_ij v_j / sum_j p_ij,
// p_ij = e^(s_ij - m_i), in one pass over the keys i sees with a running maximum.
//
// A job is one head of NQ tiles of 128 query rows; it walks the 128-key tiles that any
// of them sees.  CTAs stay on their SM and take one job after the other (kDealtFrom).  Both
// products run on the tensor cores, with everything between them in tensor memory:
// S = Q K^T (128 x 128 fp32) is read by the four warps of its tile, a row per thread, so
// that a row's maximum and sum need no exchange; the weights go back as 16-bit words over
// S, where the second product O += P V takes them as its first operand.  V is read as it
// lies in memory (its rows are the reduction).
//   warp 0      TMA producer: Q, then K and V tiles in a ring
//   warp 1      tensor memory; issues the first tile's products, warp 2 the second's
//   warp 3      finds the jobs and plans them, up to four ahead (one, where they are dealt)
//   warps 4-7   the first tile's rows: softmax, then the output; 8-11 the second's
// The next job's loads and first scores run under the last softmax and the output of the
// one before.
//
// With two tiles a job the tensor cores work on one while the other's weights are
// computed, and K and V are read once for 256 rows; with one tile two CTAs share an SM.
// Two are taken where documents are longer than a tile and their jobs reach every SM:
// 14400 x 16 x 128 948 against 1104 us, 1024-long documents of 64-wide heads 81 against 89,
// 256-long ones 34 each; between 256 and 768 either is ahead by up to 14%, as the number of
// tiles is even or odd (54 of 300 63 against 57, 32 of 500 50 against 58).
// What bounds it: at 128-wide heads the tensor cores (14400 x 16 x 128: 1790 TFLOP/s of
// 1915 back to back on the same inputs, 1600 on changing ones, under the power cap); at 64
// the chain of one tile's steps, as its scores and weights share their place:
// of 2400 cycles for a key tile of both query tiles 1700 are a softmax from scores to
// weights, the rest its two products and the hand-overs.  So the weights are handed over in
// two halves, and a turn's scores are issued right behind its product, their keys having
// been waited for before it (822 to 799 us at 64, 788 by now; leaving out the exponentials and the
// maximum gains 10%).  Without the turns 128-wide heads take 1304 us.
// The maximum that weights are relative to follows the running one only when that has
// grown by more than 2^8 (weights up to 256 keep their 11 or 8 bits, sums are fp32), so
// that O is rarely rescaled: only then does a softmax warp wait for the product before.
// Weights are rounded to the inputs' 16-bit type for the second product, whose
// operands have one type; the sum of weights takes them unrounded.
#include "token_attention_internal.h"
#include "token_scores.cuh"

namespace c3d {

namespace {

constexpr int kRows = 128;             // query rows and keys of a tile
constexpr uint32_t kBoxBytes = 16384;  // 128 rows of 64 elements
constexpr int kMaxStages = 8;
constexpr uint32_t kJobs = 4;          // jobs planned ahead
constexpr uint32_t kSmallBytes = 896;  // shared memory of the barriers, jobs and the dealer's answers
constexpr uint32_t kAsk = 8;           // asked for at once behind the last job
// Mean tokens of a document above which jobs are dealt to CTAs that ask (cluster launch
// control: a CTA takes the index of one that has not started), so that none waits for
// another's longer documents: 2 x 8192 causal 332 us, 360 with every grid-th job a CTA;
// 24 documents of 100 to 1403 with slopes 210 and 223; 40 of 30 to 1600 causal 169 and 196
// (lengths drawn at random).  The grid then has a CTA for every job that there could be, and
// those behind the last job are taken too, kAsk at a time: a buffer of 65536 rows with 1000
// in use takes 17 us either way.  Of short documents the planner finds 32 jobs at a time
// instead (100 x 100: 21 us, 33 dealt).
constexpr long long kDealtFrom = 384;
constexpr float kLag = 8.0f;           // powers of two that weights may exceed 1 by
// f16 weights (and their sum) are taken 2^7 times as large, up to 2^15 of f16's 2^16: those
// of 2^-31 of the largest one still count, where 2^-24 would be the least otherwise.  bf16
// weights have fp32's range and are taken 2^-24 times as large, so that sums over 2^16 keys
// (2^24, with weights of 1) hold for values up to the type's largest; results below 2^-112
// lose bits instead.
template <bool BF>
constexpr float kUp = BF ? -24.0f : 7.0f;
// Scores from here on (powers of two) are in steps of a quarter and more: f16 weights follow
// the maximum at once, as the steps could take lagging ones out of f16's range.
constexpr float kCoarse = 2097152.0f;

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if (BF) return pack_bf16x2(a, b);
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 128 * NQ rows from `row0` of a document, for one head (negative: no more jobs).
// Its key tiles, in order, are those of the document's lead (lead_tiles), then those from
// tile `skip` on; a query tile sees the first `lead` of them and those from lo to hi.
struct Seen {
    int lead, lo, hi;
    __device__ bool operator()(int n) const { return n < lead || (n >= lo && n < hi); }
};
struct Job {
    int head, row0, rows;    // rows: the document's queries
    int keys, shift;         // its keys; position of row r: r + shift
    int prefix;
    int count, lead_tiles, skip;
    Seen seen[2];
    int unused;
    long long q0, k0;        // packed rows of the document's first query and key
    __device__ int key(int n) const { return (n < lead_tiles ? n : n - lead_tiles + skip) * kRows; }
};
static_assert(352 + kJobs * sizeof(Job) <= kSmallBytes - 16 * kAsk - 8, "barriers, words, jobs, the dealer's answers");

// The keys that rows [a, b) of the job see: [lo, hi) of any of them, and [0, lead).
struct Range {
    int lo, hi, lead;
};
__device__ __forceinline__ Range range_of(const PackedParams& p, const Job& j, int a, int b) {
    Range r{0, j.keys, j.prefix};
    const int i0 = a + j.shift, i1 = b - 1 + j.shift;   // positions, first and last
    if (p.window > 0) {
        r.lo = static_cast<int>(max(0ll, static_cast<long long>(i0) - p.window + 1));
        r.hi = static_cast<int>(min(static_cast<long long>(r.hi), static_cast<long long>(i1) + p.window));
    }
    if (p.causal) r.hi = min(r.hi, i1 + 1);
    if (r.hi <= r.lo || a >= b) r.lo = r.hi = 0;
    if (a >= b) r.lead = 0;
    return r;
}

// The key tiles of a job of nq query tiles
__device__ __forceinline__ void plan_tiles(const PackedParams& p, Job& j, int nq) {
    const Range all = range_of(p, j, j.row0, min(j.row0 + nq * kRows, j.rows));
    j.lead_tiles = (all.lead + kRows - 1) / kRows;
    j.skip = max(all.lo / kRows, j.lead_tiles);
    j.count = j.lead_tiles + max((all.hi + kRows - 1) / kRows - j.skip, 0);
    for (int i = 0; i < 2; ++i) {
        const int a = j.row0 + i * kRows;
        const Range r = range_of(p, j, a, i < nq ? min(a + kRows, j.rows) : a);
        j.seen[i].lead = r.lead ? j.lead_tiles : 0;
        j.seen[i].lo = r.hi > r.lo ? max(r.lo / kRows, j.skip) - j.skip + j.lead_tiles : 0;
        j.seen[i].hi = r.hi > r.lo ? max((r.hi + kRows - 1) / kRows, j.skip) - j.skip + j.lead_tiles : 0;
    }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The largest of 128 values, or of their magnitudes
template <bool ABS>
__device__ __forceinline__ float max128(const uint32_t (&s)[4][32]) {
    float t[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        auto v = [&](int e) { return ABS ? fabsf(__uint_as_float(s[h][e])) : __uint_as_float(s[h][e]); };
        t[h] = fmaxf(v(0), v(1));
#pragma unroll
        for (int e = 2; e < 32; e += 2) t[h] = max3(t[h], v(e), v(e + 1));
    }
    return fmaxf(max3(t[0], t[1], t[2]), t[3]);
}

// A row's score at a key, in powers of two
__device__ __forceinline__ float shaped(const PackedParams& p, float dot, int i, int j, float slope2) {
    float s = dot * p.scale;
    if (p.cap > 0.0f) s = cap_score(s, p.cap, p.inv_cap);
    return s * kLog2e - slope2 * fabsf(static_cast<float>(i - j));
}

__device__ __forceinline__ uint32_t bits_below(int n) {
    return static_cast<uint32_t>((1ull << min(max(n, 0), 32)) - 1ull);
}
struct RowMask {
    int lo, hi, lead, keys;
    // keys j .. j + 31 as bits
    __device__ uint32_t bits(int j) const {
        return ((bits_below(hi - j) & ~bits_below(lo - j)) | bits_below(lead - j)) & bits_below(keys - j);
    }
};
__device__ __forceinline__ RowMask row_mask(const PackedParams& p, const Job& j, int row) {
    const Range r = range_of(p, j, row, row + 1);
    return RowMask{r.lo, r.hi, r.lead, j.keys};
}

// Four elements of a row, as they lie in memory and as fp32
__device__ __forceinline__ uint2 four_raw(const unsigned char* base, long long i) {
    return *reinterpret_cast<const uint2*>(base + 2 * i);
}
template <bool BF>
__device__ __forceinline__ void four(uint2 w, float (&v)[4]) {
    const uint32_t x[2] = {w.x, w.y};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint16_t h = static_cast<uint16_t>(x[e >> 1] >> (16 * (e & 1)));
        v[e] = BF ? __uint_as_float(static_cast<uint32_t>(h) << 16) : __half2float(__ushort_as_half(h));
    }
}

// A row whose result is not finite although what it sees may be: an unseen key of a
// tile that was multiplied (weight 0) has a value that is not finite.  Then the row is
// computed again, over what it sees alone, by the whole warp, four elements a lane and eight
// keys at a time, so that their loads are in flight together: 260 cycles a key, 620 one at a
// time (127 rows over 60000 keys: 265 ms and 625).  The other warps wait meanwhile, and count
// their bounds from its last word that it goes on.
template <bool BF>
__device__ __forceinline__ void redo_row(const PackedParams& p, const Job& job, const Seen& seen, int row, int lane,
                                         uint32_t* goes_on) {
    constexpr int kAtOnce = 8;
    const RowMask m = row_mask(p, job, row);
    const bool in = 4 * lane < p.width;
    const long long base = job.k0 * p.k_tok + static_cast<long long>(job.head / p.group) * p.k_head + 4 * lane;
    const float slope2 = p.slopes ? p.slopes[job.head] * kLog2e : 0.0f;
    float top = -INFINITY, sum = 0.0f, q[4] = {}, o[4] = {};
    if (in) four<BF>(four_raw(p.q, (job.q0 + row) * p.q_tok + static_cast<long long>(job.head) * p.q_head + 4 * lane), q);
    bool spoiled = false, nan = false;
    // pass 0: is an unseen key's value the cause?  1: the row
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        if (pass && !__any_sync(0xffffffffu, spoiled)) return;
#pragma unroll 1
        for (int n = 0; n < 128 / kAtOnce * job.count; ++n) {
            constexpr int kPer = 128 / kAtOnce;   // of a tile
            const int j0 = job.key(n / kPer) + n % kPer * kAtOnce;
            if (lane == 0) atomicAdd(goes_on, 1u);
            uint32_t bits = m.bits(j0);
            if (pass == 0) bits = ~bits & bits_below(job.keys - j0);
            if (!seen(n / kPer)) bits = 0u;
            bits &= (1u << kAtOnce) - 1u;
            if (!bits) continue;
            uint2 kw[kAtOnce], vw[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const bool load = in && (bits >> i & 1u);
                kw[i] = vw[i] = make_uint2(0u, 0u);
                if (load) vw[i] = four_raw(p.v, base + (j0 + i) * p.k_tok);
                if (load && pass) kw[i] = four_raw(p.k, base + (j0 + i) * p.k_tok);
            }
            float s[kAtOnce], v[4], now = top;
            if (pass == 0) {
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    four<BF>(vw[i], v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) spoiled = spoiled || !(fabsf(v[e]) < INFINITY);
                }
                continue;
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                four<BF>(kw[i], v);
                s[i] = q[0] * v[0] + q[1] * v[1] + q[2] * v[2] + q[3] * v[3];
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                s[i] = bits >> i & 1u ? shaped(p, s[i], row + job.shift, j0 + i, slope2) : -INFINITY;
                nan = nan || !(s[i] < INFINITY);
                now = fmaxf(now, s[i]);
            }
            if (now == -INFINITY) continue;
            const float fall = ex2(top - now);
            top = now;
            sum *= fall;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] *= fall;
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const float w = ex2(s[i] - now + kUp<BF>);
                sum += w;
                four<BF>(vw[i], v);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = fmaf(w, v[e], o[e]);
            }
        }
    }
    uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) + (job.q0 + row) * p.out_tok +
                    static_cast<long long>(job.head) * p.out_head + 4 * lane;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float r = nan ? __uint_as_float(kNanBits) : sum == 0.0f ? 0.0f : o[e] / sum;
        if (in) dst[e] = static_cast<uint16_t>(pack2<BF>(r, 0.0f));
    }
}

// Bounded waits without a call (see wait_bar and drain_wait): the compiler makes none from
// warps that have registers of a number of their own.  A role sleeps in hardware between
// looks, so that its polling leaves the issue slots to the others.  Whole warps wait, with
// one answer for all lanes.  The bound counts anew while rows are computed again: their
// warps say so in a word behind the abort flag (kGoesOn).
constexpr int kGoesOn = 5;
__device__ __forceinline__ bool wait_role(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag,
                                          int* status, long long limit_cycles) {
    constexpr uint32_t kAll = 0xffffffffu;
    // (without a limit to wait for, nothing is waited for)
    if (__all_sync(kAll, limit_cycles ? mbar_try_wait(bar, parity) : mbar_test_wait(bar, parity))) return true;
    long long t0 = clock64();
    uint32_t last = abort_flag[kGoesOn];
    while (!__any_sync(kAll, *abort_flag != 0u || clock64() - t0 >= limit_cycles)) {
        if (__all_sync(kAll, mbar_try_wait_for(bar, parity, 20000u))) return true;
        const uint32_t now = abort_flag[kGoesOn];
        if (now != last) t0 = clock64();
        last = now;
    }
    if (atomicExch(const_cast<uint32_t*>(abort_flag), 1u) == 0u) atomicExch(status, kStatusTimeout);
    return false;
}
__device__ __forceinline__ void drain_here(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 <= kDrainNs) {
    }
}
// the last load of each slot of a ring
__device__ __forceinline__ void drain_slots(uint32_t full0, uint32_t issued, uint32_t slots) {
    for (uint32_t n = issued > slots ? issued - slots : 0u; n < issued; ++n)
        drain_here(full0 + 8 * (n % slots), (n / slots) & 1u);
}

// One lane's predicate, and instructions under it
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
}
// (a value that every lane holds alike, said so to the compiler)
__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }

__device__ __forceinline__ void mma_if(uint32_t lane, uint32_t d, uint32_t a_low, uint32_t a_high, uint32_t b_low,
                                       uint32_t b_high, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 q, %0, 0;\n\t"
        "setp.ne.b32 p, %7, 0;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %6, p;\n\t}" ::"r"(lane),
        "r"(d), "r"(a_low), "r"(a_high), "r"(b_low), "r"(b_high), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ta_if(uint32_t lane, uint32_t d, uint32_t a, uint32_t b_low, uint32_t b_high,
                                          uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 q, %0, 0;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 b, {%3, %4};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], b, %5, p;\n\t}" ::"r"(lane),
        "r"(d), "r"(a), "r"(b_low), "r"(b_high), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t lane, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %0, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(lane),
        "r"(bar)
        : "memory");
}

// 32 lanes x 8 consecutive 32-bit columns, the reverse of tmem_ld_32x32b_x8
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
        : "memory");
}

// Takes one of the grid's CTAs that has not started yet: the answer (16 bytes) arrives on
// a barrier.  Nobody asks again who has seen that there was none left.
__device__ __forceinline__ void ask_for_cta(uint32_t answer, uint32_t bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
        "r"(bar)
        : "memory");
}
__device__ __forceinline__ bool taken_cta(uint32_t answer, uint32_t* index) {
    uint32_t taken, x;
    asm volatile(
        "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 a, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
        : "=r"(taken), "=r"(x)
        : "r"(answer)
        : "memory");
    *index = x;
    return taken != 0u;
}

template <int NQ>
constexpr int kThreads = 128 + 128 * NQ;

// What scores go through beside the scale: nothing (the scale then goes into the
// exponent's one multiply-add), the cap, the distance (or a scale that is not positive).
constexpr int kCap = 1, kFar = 2;

// NQ: query tiles of a job.
template <bool BF, int NQ, int MOD>
__global__ void __launch_bounds__(kThreads<NQ>, NQ == 1 ? 2 : 1)
    packed_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map, const __grid_constant__ PackedParams p,
                  const int stages, const int q_bufs, const int dealt) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const int boxes = (p.width + 63) / 64;
    const uint32_t tile_bytes = boxes * kBoxBytes;
    const uint32_t q_smem = base, ring = base + q_bufs * NQ * tile_bytes;
    const uint32_t bars = ring + stages * tile_bytes;
    const uint32_t full0 = bars, empty0 = full0 + 8u * kMaxStages;
    const uint32_t q_full0 = empty0 + 8u * kMaxStages, q_empty0 = q_full0 + 16u;
    const uint32_t job_full0 = q_empty0 + 16u, job_empty0 = job_full0 + 8u * kJobs;
    const uint32_t s_full0 = job_empty0 + 8u * kJobs, p_full0 = s_full0 + 16u, o_done0 = p_full0 + 16u;
    const uint32_t turn_bar0 = o_done0 + 16u, half_full0 = turn_bar0 + 16u, tail_bar = half_full0 + 16u;
    const uint32_t drain_bar = tail_bar + 8u;
    const uint32_t deal_answer = bars + kSmallBytes - 16u * kAsk, deal_bar = deal_answer - 8u;
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem_raw + (drain_bar + 8u - raw));
    // misc[0] TMEM base, [1] abort flag, [2] ring loads issued, [3] Q loads issued, [4] whether a
    // last tile's values are on their way (1 + its phase), [5] to which slot, [6] counts while rows
    // are computed again; then the jobs
    volatile uint32_t* abort_flag = misc + 1;
    Job* jobs = reinterpret_cast<Job*>(misc + 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // (two cycles a nanosecond, as in wait_bar)
    const long long limit = static_cast<long long>(p.wait_ns > (1ull << 61) ? (1ull << 61) : p.wait_ns) * 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, NQ);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full0 + 8 * i, 1);
            mbar_init(q_empty0 + 8 * i, NQ);
            mbar_init(s_full0 + 8 * i, 1);
            mbar_init(half_full0 + 8 * i, 4);
            mbar_init(p_full0 + 8 * i, 4);
            mbar_init(o_done0 + 8 * i, 1);
            mbar_init(turn_bar0 + 8 * i, 1);
        }
        for (uint32_t i = 0; i < kJobs; ++i) {
            mbar_init(job_full0 + 8 * i, 1);
            mbar_init(job_empty0 + 8 * i, 1 + 5 * NQ);
        }
        mbar_init(tail_bar, 1);
        mbar_init(drain_bar, NQ);
        mbar_init(deal_bar, 1);
        misc[1] = 0u;
        misc[2] = 0u;
        misc[3] = 0u;
        misc[4] = 0u;
        misc[1 + kGoesOn] = 0u;
        fence_mbar_init();
        prefetch_tmap(&q_map);
        prefetch_tmap(&k_map);
        prefetch_tmap(&v_map);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(misc), NQ == 2 ? 512 : 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    const uint32_t o_pitch = boxes * 64u;
    griddep_wait();   // (the next launch is not let in early: capped causal prompts 380 us so, 368 without)

    if (warp < 4) {
        set_max_regs_dec<NQ == 2 ? 72 : 56>();
        if (warp == 3) {
            // Documents are looked through 128 at a time, four a lane; a lane plans one of the
            // CTA's next jobs, 32 in all.  Where jobs are dealt, it is one at a time, the next
            // taken when all roles have begun the last; the grid has a CTA for every job that
            // there could be, and behind the last job they are taken kAsk at a time.
            uint32_t ticket = blockIdx.x, have = 1u, deal_ph = 0;   // have: lanes with a ticket
            bool more = true;        // there may be CTAs left to take
            long long total = -1;    // jobs of one head, once known
            auto deal = [&]() {
                const uint32_t ask = total < 0 ? 1u : kAsk;
                if (lane == 0) mbar_arrive_expect_tx(deal_bar, 16u * ask);
                __syncwarp();
                if (lane < ask) ask_for_cta(deal_answer + 16u * lane, deal_bar);
                __syncwarp();
                if (!wait_role(deal_bar, deal_ph, abort_flag, p.status, limit)) {
                    drain_here(deal_bar, deal_ph);   // they land before the shared memory is given up
                    return false;
                }
                deal_ph ^= 1u;
                const bool taken = lane < ask && taken_cta(deal_answer + 16u * lane, &ticket);
                more = __all_sync(0xffffffffu, taken || lane >= ask);
                have = __ballot_sync(0xffffffffu,
                                     taken && (total < 0 || ticket / static_cast<uint32_t>(p.heads) < total));
                fence_proxy_async_smem();
                return true;
            };
            int s0 = -128, n[4] = {0, 0, 0, 0}, off[5] = {0, 0, 0, 0, 0}, mine = 0, run = 0;
            long long before = 0;
            int all = 0;   // jobs (of one head) of these 128
            bool ok = true;
            for (uint32_t k = 0; ok;) {
                if (dealt && !have && more) {
                    const uint32_t last = k - 1;
                    ok = (k == 0 || wait_role(job_empty0 + 8 * (last % kJobs), (last / kJobs) & 1u, abort_flag, p.status,
                                              limit)) &&
                         deal();
                    continue;
                }
                const bool some = !dealt || have;
                const uint32_t at = dealt ? __shfl_sync(0xffffffffu, ticket, have ? __ffs(have) - 1 : 0)
                                          : blockIdx.x + (k + lane) * gridDim.x;
                have &= have - 1u;
                const uint32_t want = dealt && (lane || !some) ? 0xffffffffu : at / static_cast<uint32_t>(p.heads);
                const uint32_t first = __shfl_sync(0xffffffffu, want, 0);
                if (first < before) {   // (dealt out of order)
                    s0 = -128;
                    before = all = 0;
                }
                while (some && before + all <= first && s0 < p.documents) {
                    before += all;
                    s0 += 128;
#pragma unroll
                    for (int i = 0; i < 5; ++i) {
                        const int s = min(s0 + 4 * lane + i, p.documents);
                        off[i] = static_cast<int>(min(max(static_cast<long long>(p.q_offsets[s]), 0ll), p.q_tokens));
                    }
                    mine = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        n[i] = (max(off[i + 1] - off[i], 0) + NQ * kRows - 1) / (NQ * kRows);
                        mine += n[i];
                    }
                    run = mine;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int o = __shfl_up_sync(0xffffffffu, run, d);
                        if (lane >= d) run += o;
                    }
                    all = __shfl_sync(0xffffffffu, run, 31);
                }
                // the jobs among these documents: the first lanes'
                const bool here = want - before < all;
                const int count = __popc(__ballot_sync(0xffffffffu, here));
                if (dealt && some && count == 0) {
                    total = before + all;
                    continue;
                }
                const int in = here ? static_cast<int>(want - before) : 0;
                int src = 0;   // the lane whose four documents hold it
#pragma unroll
                for (int d = 16; d > 0; d >>= 1)
                    if (__shfl_sync(0xffffffffu, run, src + d - 1) <= in) src += d;
                src = min(src, 31);
                int t = in - (__shfl_sync(0xffffffffu, run, src) - __shfl_sync(0xffffffffu, mine, src));
                int s = s0 + 4 * src, tiles = 0, q0 = 0, q1 = 0;
                bool found = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = __shfl_sync(0xffffffffu, n[i], src);
                    const int a = __shfl_sync(0xffffffffu, off[i], src), b = __shfl_sync(0xffffffffu, off[i + 1], src);
                    if (found) continue;
                    if (t < c) {
                        found = true;
                        tiles = c;
                        q0 = a;
                        q1 = b;
                        s += i;
                    } else {
                        t -= c;
                    }
                }
                Job job;
                job.head = -1;
                if (here) {
                    job.rows = q1 - q0;
                    job.row0 = (p.causal ? tiles - 1 - t : t) * NQ * kRows;   // the longest first
                    const long long kb = min(max(static_cast<long long>(p.k_offsets[s]), 0ll), p.k_tokens);
                    const long long ke = min(max(static_cast<long long>(p.k_offsets[s + 1]), kb), p.k_tokens);
                    job.keys = static_cast<int>(ke - kb);
                    job.shift = job.keys - job.rows;
                    job.prefix = p.prefix ? min(max(p.prefix[s], 0), job.keys) : 0;
                    job.q0 = q0;
                    job.k0 = kb;
                    job.head = static_cast<int>(at - want * static_cast<uint32_t>(p.heads));
                    job.unused = 0;
                    plan_tiles(p, job, NQ);
                }
                const int post = max(count, 1);   // behind the last one, the word that it was
                for (int l = 0; l < post; ++l, ++k) {
                    const uint32_t slot = k % kJobs, jph = (k / kJobs) & 1u;
                    ok = wait_role(job_empty0 + 8 * slot, jph ^ 1u, abort_flag, p.status, limit);
                    if (!ok) break;
                    if (lane == l) jobs[slot] = job;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(job_full0 + 8 * slot);
                }
                if (count == 0) break;
            }
        } else if (warp == 0) {
            int st = 0;
            uint32_t ph = 0, issued = 0, q_buf = 0, q_ph = 0, q_issued = 0, tail_ph = 0;
            bool ok = true;
            // The keys of a tile behind the document's last are other documents': their scores are
            // replaced, their values (times a weight of 0) have to be finite.  The last tile's
            // values land on a barrier of their own and are cleared behind the last key before
            // they are handed on; meanwhile the next job's loads go out.
            int tail_first = -1;
            uint32_t tail_slot = 0;
            auto finish_tail = [&]() {
                if (tail_first < 0) return true;
                if (!wait_role(tail_bar, tail_ph, abort_flag, p.status, limit)) return false;
                const uint32_t dst = ring + tail_slot * tile_bytes;
#pragma unroll 1
                for (int i = tail_first * 8 + lane; i < kRows * 8; i += 32)
#pragma unroll 1
                    for (int b = 0; b < boxes; ++b)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + b * kBoxBytes + i * 16u), "r"(0u)
                                     : "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(full0 + 8 * tail_slot);
                    misc[4] = 0u;
                }
                tail_ph ^= 1u;
                tail_first = -1;
                return true;
            };
            // (a job's queries and first keys do not depend on the tail before)
            for (uint32_t k = 0; ok; ++k) {
                ok = wait_role(job_full0 + 8 * (k % kJobs), (k / kJobs) & 1u, abort_flag, p.status, limit);
                if (!ok) break;
                const Job& shared = jobs[k % kJobs];
                const int head = shared.head, keys = shared.keys, lead_tiles = shared.lead_tiles, skip = shared.skip;
                const int q_row = static_cast<int>(shared.q0) + shared.row0, k_row = static_cast<int>(shared.k0);
                const int count = head < 0 ? 0 : shared.count, kv = head / p.group;
                __syncwarp();
                if (lane == 0) mbar_arrive(job_empty0 + 8 * (k % kJobs));
                if (count) {
                    ok = wait_role(q_empty0 + 8 * q_buf, q_ph ^ 1u, abort_flag, p.status, limit);
                    if (!ok) break;
                    ++q_issued;
                    if (lane == 0) {
                        misc[3] = q_issued;
                        mbar_arrive_expect_tx(q_full0 + 8 * q_buf, NQ * tile_bytes);
#pragma unroll 1
                        for (int t = 0; t < NQ * boxes; ++t) {
                            const int i = boxes == 1 ? t : t >> 1, b = boxes == 1 ? 0 : t & 1;
                            tma_load_3d(q_smem + (q_buf * NQ + i) * tile_bytes + b * kBoxBytes, &q_map, q_full0 + 8 * q_buf,
                                        b * 64, head, q_row + i * kRows);
                        }
                    }
                    if (++q_buf == static_cast<uint32_t>(q_bufs)) {
                        q_buf = 0;
                        q_ph ^= 1u;
                    }
                }
#pragma unroll 1
                for (int n2 = 0; n2 < 2 * max(count, 1); ++n2) {
                    const bool value = n2 & 1;
                    if (value && !finish_tail()) {
                        ok = false;
                        break;
                    }
                    if (!count) continue;
                    const int n = n2 >> 1, t0 = (n < lead_tiles ? n : n - lead_tiles + skip) * kRows;
                    const bool tail = value && t0 + kRows > keys;
                    ok = wait_role(empty0 + 8 * st, ph ^ 1u, abort_flag, p.status, limit);
                    if (!ok) break;
                    const uint32_t dst = ring + st * tile_bytes, bar = tail ? tail_bar : full0 + 8 * st;
                    const void* map = value ? &v_map : &k_map;
                    ++issued;
                    if (tail) {
                        tail_first = keys - t0;
                        tail_slot = st;
                    }
                    if (lane == 0) {
                        if (tail) {
                            misc[4] = 1u + tail_ph;
                            misc[5] = st;
                        }
                        misc[2] = issued;
                        mbar_arrive_expect_tx(bar, tile_bytes);
                        tma_load_3d(dst, map, bar, 0, kv, k_row + t0);
                        if (boxes == 2) tma_load_3d(dst + kBoxBytes, map, bar, 64, kv, k_row + t0);
                    }
                    if (++st == stages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                if (head < 0) break;
            }
        } else if (warp <= NQ) {
            // One warp a query tile, all lanes together and one of them issuing: addresses and
            // decisions then stay in uniform registers, which the instructions take them from.
            // Small code counts: it shares its instruction cache with the softmax loops.
            constexpr uint32_t kType = BF ? (1u << 7) | (1u << 10) : 0u;
            const uint32_t ksteps = (p.width + 15) / 16;
            const uint32_t idesc_s = (1u << 4) | kType | ((kRows >> 3) << 17) | ((kRows >> 4) << 24);
            const uint32_t idesc_o = (1u << 4) | kType | (1u << 16) | (ksteps * 2u << 17) | ((kRows >> 4) << 24);
            // descriptors by their words: the address (and the V blocks' distance) below, the
            // 8-row groups' distance, the version and the swizzle above
            constexpr uint32_t kHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
            const uint32_t i = NQ == 1 ? 0u : static_cast<uint32_t>(uniform(warp - 1));
            const uint32_t step = tile_bytes >> 4, el = elect_lane();
            const uint32_t q_low = ((q_smem >> 4) | (1u << 16)) + i * step, k_low = (ring >> 4) | (1u << 16);
            const uint32_t v_low = (ring >> 4) | ((kBoxBytes >> 4) << 16);
            const uint32_t t_s = tmem + i * kRows, t_o = tmem + NQ * kRows + i * o_pitch;
            const uint32_t s_full = s_full0 + 8 * i, o_done = o_done0 + 8 * i;
            const uint32_t half_full = half_full0 + 8 * i, p_full = p_full0 + 8 * i;
            uint32_t slot = 0, ph = 0, q_buf = 0, q_ph = 0, pph = 0, my_turn = 0;
            bool ok = true;
            // The two warps take turns, so that the tensor cores finish one tile's products, then
            // the other's, and not both at once: each softmax then has the SM's other units
            // while the other tile's products run.  A turn is the weights' product with a key
            // tile and the scores with the next.
            auto take_turn = [&]() {
                if (NQ == 1) return true;
                const bool mine = wait_role(turn_bar0 + 8 * i, my_turn ^ (i == 0 ? 1u : 0u), abort_flag, p.status, limit);
                my_turn ^= 1u;
                return mine;
            };
            auto pass_turn = [&]() {
                __syncwarp();
                if (NQ == 2 && lane == 0) mbar_arrive(turn_bar0 + 8 * (i ^ 1u));
            };
            auto next = [&]() {
                if (++slot == static_cast<uint32_t>(stages)) {
                    slot = 0;
                    ph ^= 1u;
                }
            };
            for (uint32_t k = 0; ok; ++k) {
                ok = wait_role(job_full0 + 8 * (k % kJobs), (k / kJobs) & 1u, abort_flag, p.status, limit);
                if (!ok) break;
                const Job& job = jobs[k % kJobs];
                const int count = uniform(job.count);
                const Seen seen{uniform(job.seen[i].lead), uniform(job.seen[i].lo), uniform(job.seen[i].hi)};
                const bool last = uniform(job.head + 1) == 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(job_empty0 + 8 * (k % kJobs));
                if (last) break;
                if (count == 0) continue;
                ok = wait_role(q_full0 + 8 * q_buf, q_ph, abort_flag, p.status, limit) && take_turn();
                if (!ok) break;
                const uint32_t q_at = q_low + q_buf * NQ * step;
                uint32_t add = 0u;
                ok = wait_role(full0 + 8 * slot, ph, abort_flag, p.status, limit);
#pragma unroll 1
                for (int n = 0; ok && n < count; ++n) {
                    const bool active = seen(n);
                    if (active) {
                        // (the scores before were read, and their weights multiplied, by then)
                        tc_fence_after();
                        const uint32_t b = k_low + slot * step;
                        mma_if(el, t_s, q_at, kHigh, b, kHigh, idesc_s, 0u);
#pragma unroll
                        for (uint32_t kk = 1; kk < 8; ++kk) {
                            const uint32_t off = (kk >> 2) * (kBoxBytes >> 4) + 2 * (kk & 3);
                            if (kk < ksteps) mma_if(el, t_s, q_at + off, kHigh, b + off, kHigh, idesc_s, 1u);
                        }
                        commit_if(el, s_full);
                    }
                    commit_if(el, empty0 + 8 * slot);
                    if (n + 1 == count) commit_if(el, q_empty0 + 8 * q_buf);
                    pass_turn();
                    next();
                    const uint32_t at = slot;
                    ok = wait_role(full0 + 8 * slot, ph, abort_flag, p.status, limit);
                    if (!ok) break;
                    // the next keys too, so that their scores follow this product at once
                    next();
                    if (n + 1 < count) ok = wait_role(full0 + 8 * slot, ph, abort_flag, p.status, limit);
                    ok = ok && take_turn();
                    if (!ok) break;
                    if (active) {
                        const uint32_t b = v_low + at * step;
#pragma unroll 1
                        for (uint32_t half = 0; half < 2; ++half) {
                            ok = wait_role(half ? p_full : half_full, pph, abort_flag, p.status, limit);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (uint32_t kk = 0; kk < kRows / 32; ++kk)
                                mma_ta_if(el, t_o, t_s + 32 * half + 8 * kk, b + (4 * half + kk) * 128, kHigh, idesc_o,
                                          kk || half ? 1u : add);
                        }
                        if (!ok) break;
                        pph ^= 1u;
                        commit_if(el, o_done);
                        add = 1u;
                    }
                    commit_if(el, empty0 + 8 * at);
                }
                if (!ok) break;
                pass_turn();
                if (++q_buf == static_cast<uint32_t>(q_bufs)) {
                    q_buf = 0;
                    q_ph ^= 1u;
                }
            }
        }
        __syncwarp();
    } else {
        set_max_regs_inc<NQ == 2 ? 216 : 200>();
        const int i = (warp - 4) >> 2;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + i * kRows, t_o = tmem + lanes + NQ * kRows + i * o_pitch;
        const float per_cap = p.per_cap;
        const float c = MOD ? 1.0f : p.scale * kLog2e;
        uint32_t turn = 0;   // this tile's units so far
        bool ok = true;
        for (uint32_t k = 0; ok; ++k) {
            ok = wait_role(job_full0 + 8 * (k % kJobs), (k / kJobs) & 1u, abort_flag, p.status, limit);
            if (!ok) break;
            const Job job = jobs[k % kJobs];
            __syncwarp();
            if (lane == 0) mbar_arrive(job_empty0 + 8 * (k % kJobs));
            if (job.head < 0) break;
            const Seen mine = NQ == 2 && i == 1 ? job.seen[1] : job.seen[0];
            const int row = job.row0 + i * kRows + (warp & 3) * 32 + lane;
            const bool valid = row < job.rows;
            const RowMask mask = row_mask(p, job, min(row, job.rows - 1));
            const int a = job.row0 + i * kRows, b = min(a + kRows, job.rows);
            // keys that every row of the tile sees
            int all_lo = 0, all_hi = job.keys;
            if (p.window > 0) {
                all_lo = static_cast<int>(max(0ll, static_cast<long long>(b) + job.shift - p.window));
                all_hi = static_cast<int>(min(static_cast<long long>(all_hi), static_cast<long long>(a) + job.shift + p.window));
            }
            if (p.causal) all_hi = min(all_hi, a + job.shift + 1);
            const float slope2 = (MOD & kFar) && p.slopes ? p.slopes[job.head] * kLog2e : 0.0f;
            const int pos = row + job.shift;
            float ref = -INFINITY, sum = 0.0f;   // ref: what the weights are relative to
            bool fresh = true;
            for (int n = 0; n < job.count; ++n) {
                const int t0 = job.key(n);
                if (!mine(n)) continue;
                ok = wait_role(s_full0 + 8 * i, turn & 1u, abort_flag, p.status, limit);
                if (!ok) break;
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int h = 0; h < 4; ++h) tmem_ld_32x32b_x32(t_s + 32 * h, s[h]);
                tmem_ld_wait();
                // Scores that are all within the cap's polynomial go through it with the scale and the
                // cap in its coefficients: a score is then its product times `co` in that product's
                // square, in powers of two, where the exponential's form takes two turns of the
                // special-function unit a value.  (Where these coefficients were no normal numbers,
                // per_cap is infinite and no score is within.)
                uint64_t co[5];
                bool small = false;   // all scores of the warp's tile are within the polynomial's reach
                if (MOD & kCap) {
                    small = __all_sync(0xffffffffu, max128<true>(s) * per_cap <= kTanhReach);
                    float f = p.scale * kLog2e;
#pragma unroll
                    for (int d = 0; d < 5; ++d) {
                        co[d] = two(kTanh[d] * f);
                        f *= per_cap * per_cap;
                    }
                }
                auto factor = [&](uint64_t x) {
                    const uint64_t u = mul2(x, x);
                    uint64_t y = fma2(u, co[4], co[3]);
#pragma unroll
                    for (int d = 2; d >= 0; --d) y = fma2(u, y, co[d]);
                    return y;
                };
                // the cap alone keeps the order of scores: where all are seen their maximum is taken
                // before it, and small ones go through it on their way into the exponent
                const bool open = t0 + kRows <= job.keys &&
                                  (t0 + kRows <= job.prefix || (t0 >= all_lo && t0 + kRows <= all_hi));
                const bool late = MOD == kCap && small && open;
                if ((MOD & kCap) && !small) {
                    // (through tensor memory, 32 at a time: 843 us where, unrolled over the row, it takes
                    // 941, and the usual form 2% longer beside it; causal 2 x 8192 under a cap of 1)
#pragma unroll 1
                    for (int h = 0; h < 4; ++h) {
                        uint32_t t[32];
                        tmem_ld_32x32b_x32(t_s + 32 * h, t);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            split(cap_pair_any(mul2(two(t[e], t[e + 1]), two(p.scale)), p.cap, p.inv_cap), t[e], t[e + 1]);
                        tmem_st_32x32b_x32(t_s + 32 * h, t);
                    }
                    tmem_st_wait();
#pragma unroll
                    for (int h = 0; h < 4; ++h) tmem_ld_32x32b_x32(t_s + 32 * h, s[h]);
                    tmem_ld_wait();
                } else if ((MOD & kCap) && !late) {
#pragma unroll
                    for (int h = 0; h < 4; ++h)
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const uint64_t x = two(s[h][e], s[h][e + 1]);
                            split(mul2(x, factor(x)), s[h][e], s[h][e + 1]);
                        }
                }
                if (MOD & kFar) {
                    const uint64_t f = two(MOD & kCap ? 1.0f : p.scale * kLog2e);
                    if (t0 + kRows <= a + job.shift + 1 || t0 >= b - 1 + job.shift) {
                        // all keys on one side of all rows: the distance is linear
                        const float g = t0 >= b - 1 + job.shift ? -slope2 : slope2;
                        const float g0 = g * static_cast<float>(t0 - pos);
#pragma unroll
                        for (int h = 0; h < 4; ++h)
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                const float d = static_cast<float>(32 * h + e);
                                const uint64_t far = fma2(two(g), two(__float_as_uint(d), __float_as_uint(d + 1.0f)), two(g0));
                                split(fma2(two(s[h][e], s[h][e + 1]), f, far), s[h][e], s[h][e + 1]);
                            }
                    } else {
                        const float rel = static_cast<float>(t0 - pos), ff = MOD & kCap ? 1.0f : p.scale * kLog2e;
#pragma unroll
                        for (int h = 0; h < 4; ++h)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                s[h][e] = __float_as_uint(fmaf(__uint_as_float(s[h][e]), ff,
                                                               -slope2 * fabsf(rel + static_cast<float>(32 * h + e))));
                    }
                }
                if (!open) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const uint32_t m = mask.bits(t0 + 32 * h);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(m >> e & 1u)) s[h][e] = __float_as_uint(-INFINITY);
                    }
                }
                float top = max128<false>(s);
                if (late) {
                    uint32_t x, y;
                    const uint64_t v = two(top);
                    split(mul2(v, factor(v)), x, y);
                    top = top == -INFINITY ? top : __uint_as_float(x);
                }
                if (fresh) {
                    ref = top;
                } else if (__any_sync(0xffffffffu, top * c > ref * c + (BF || fabsf(top * c) < kCoarse ? kLag : 0.0f))) {
                    ok = wait_role(o_done0 + 8 * i, (turn - 1) & 1u, abort_flag, p.status, limit);
                    if (!ok) break;
                    tc_fence_after();
                    const float now = fmaxf(ref, top);
                    const float f = now == -INFINITY ? 1.0f : ex2((ref - now) * c);
                    ref = now;
                    sum *= f;
#pragma unroll 1
                    for (uint32_t d = 0; d < o_pitch; d += 8) {
                        uint32_t o[8];
                        tmem_ld_32x32b_x8(t_o + d, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st_32x32b_x8(t_o + d, o);
                    }
                }
                fresh = false;
                const uint64_t off = two(ref == -INFINITY ? 0.0f : fmaf(-ref, c, kUp<BF>)), cc = two(c);
                uint64_t sums[2] = {0ull, 0ull};
                auto weights = [&](auto exponent) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            uint32_t x, y;
                            split(exponent(two(s[h][e], s[h][e + 1])), x, y);
                            const float px = ex2(__uint_as_float(x)), py = ex2(__uint_as_float(y));
                            sums[e / 2 & 1] = add2(sums[e / 2 & 1], two(__float_as_uint(px), __float_as_uint(py)));
                            s[h >> 1][(h & 1) * 16 + e / 2] = pack2<BF>(px, py);
                        }
                        if (h == 1) {   // the first half's product can begin
                            tmem_st_32x32b_x32(t_s, s[0]);
                            tmem_st_wait();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(half_full0 + 8 * i);
                        }
                    }
                };
                if (MOD == 0) weights([&](uint64_t v) { return fma2(v, cc, off); });
                else if (late) weights([&](uint64_t v) { return fma2(v, factor(v), off); });
                else weights([&](uint64_t v) { return add2(v, off); });
                tmem_st_32x32b_x32(t_s + 32, s[1]);
                {
                    uint32_t x, y;
                    split(add2(sums[0], sums[1]), x, y);
                    sum += __uint_as_float(x) + __uint_as_float(y);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full0 + 8 * i);
                ++turn;
            }
            if (!ok) break;
            if (!fresh) {
                ok = wait_role(o_done0 + 8 * i, (turn - 1) & 1u, abort_flag, p.status, limit);
                if (!ok) break;
                tc_fence_after();
            }
            // ---- the output rows
            const float inv = fresh || sum == 0.0f ? 0.0f : 1.0f / sum;
            uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) + (job.q0 + row) * p.out_tok +
                            static_cast<long long>(job.head) * p.out_head;
            float odd = 0.0f;   // becomes NaN with the first result that is not finite
#pragma unroll 1
            for (int d = 0; d < p.width; d += 32) {
                uint32_t o[32];
                if (fresh) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                } else {
                    tmem_ld_32x32b_x32(t_o + d, o);
                    tmem_ld_wait();
                }
                // (a row that saw nothing has a sum of 0, whatever its products are)
                const int left = p.width - d;
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const bool none = inv == 0.0f || 2 * e >= left;
                    const float x = none ? 0.0f : __uint_as_float(o[2 * e]) * inv;
                    const float y = none ? 0.0f : __uint_as_float(o[2 * e + 1]) * inv;
                    odd = fmaf(x, 0.0f, fmaf(y, 0.0f, odd));
                    w[e] = pack2<BF>(x, y);
                }
                __syncwarp();
                if (!valid) {
                } else if (p.out_aligned == 32 && left >= 32) {
#pragma unroll
                    for (int e = 0; e < 16; e += 8)
                        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + d + 2 * e),
                                     "r"(w[e]), "r"(w[e + 1]), "r"(w[e + 2]), "r"(w[e + 3]), "r"(w[e + 4]),
                                     "r"(w[e + 5]), "r"(w[e + 6]), "r"(w[e + 7])
                                     : "memory");
                } else if (p.out_aligned) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        if (2 * e < left)
                            *reinterpret_cast<uint4*>(dst + d + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (e < left) dst[d + e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
                }
                __syncwarp();
            }
            for (uint32_t again = __ballot_sync(0xffffffffu, valid && odd != 0.0f); again; again &= again - 1u)
                redo_row<BF>(p, job, mine, row - lane + __ffs(again) - 1, lane, misc + 1 + kGoesOn);
            __syncwarp();
            tc_fence_before();
        }
    }
    __syncwarp();
    __syncthreads();
    if (*abort_flag) {
        // drain: the loads, then the MMAs in flight
        if (threadIdx.x == 0) {
            if (misc[4]) {
                drain_here(tail_bar, misc[4] - 1u);
                mbar_arrive(full0 + 8 * misc[5]);
            }
            drain_slots(q_full0, misc[3], q_bufs);
            drain_slots(full0, misc[2], stages);
        }
        if (warp >= 1 && warp <= NQ) {
            commit_if(elect_lane(), drain_bar);
            drain_here(drain_bar, 0);
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, NQ == 2 ? 512 : 256);
    }
}

template <bool BF, int NQ, int MOD>
cudaError_t run(const PackedMaps& maps, const PackedParams& p, int num_sms, cudaStream_t stream) {
    const uint32_t tile = static_cast<uint32_t>((p.width + 63) / 64) * kBoxBytes;
    // shared memory of the SM, or half of it for two CTAs; Q twice where tiles are small
    const uint32_t room = (NQ == 2 ? 232448u : 115200u) - 1024u - kSmallBytes;
    const int q_bufs = tile == kBoxBytes ? 2 : 1;
    int stages = static_cast<int>((room - q_bufs * NQ * tile) / tile);
    if (stages > kMaxStages) stages = kMaxStages;
    const size_t smem = 1024u + (q_bufs * NQ + stages) * tile + kSmallBytes;
    static std::atomic<int> slots[kMaxDevices];
    cudaError_t e = ensure_dynamic_smem(packed_kernel<BF, NQ, MOD>, smem, slots);
    if (e != cudaSuccess) return e;
    const long long most = (p.q_tokens / (NQ * kRows) + p.documents) * p.heads;
    const long long resident = static_cast<long long>(num_sms) * (NQ == 1 ? 2 : 1);
    const int dealt = most > resident && p.q_tokens / p.documents > kDealtFrom;
    return launch_ex(packed_kernel<BF, NQ, MOD>, static_cast<unsigned>(most < resident || dealt ? most : resident),
                     dim3(kThreads<NQ>), smem, 1, stream, maps.q, maps.k, maps.v, p, stages, q_bufs, dealt);
}

template <bool BF, int NQ>
cudaError_t by_mod(const PackedMaps& maps, const PackedParams& p, int num_sms, cudaStream_t stream) {
    const bool far = p.slopes || !(p.scale > 0.0f);
    if (p.cap > 0.0f)
        return far ? run<BF, NQ, kCap | kFar>(maps, p, num_sms, stream) : run<BF, NQ, kCap>(maps, p, num_sms, stream);
    return far ? run<BF, NQ, kFar>(maps, p, num_sms, stream) : run<BF, NQ, 0>(maps, p, num_sms, stream);
}

}  // namespace

cudaError_t launch_packed(const PackedMaps& maps, const PackedParams& p, int dtype, int num_sms,
                          cudaStream_t stream) {
    const bool bf = dtype == kTokBf16;
    // two tiles where documents have them and there are jobs enough for all SMs
    const bool two_tiles = p.q_tokens / p.documents > kRows && p.q_tokens / 256 * p.heads >= num_sms;
    if (two_tiles) return bf ? by_mod<true, 2>(maps, p, num_sms, stream) : by_mod<false, 2>(maps, p, num_sms, stream);
    return bf ? by_mod<true, 1>(maps, p, num_sms, stream) : by_mod<false, 1>(maps, p, num_sms, stream);
}

}  // namespace c3d
