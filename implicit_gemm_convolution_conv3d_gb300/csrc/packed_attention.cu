// packed_attention.cu -- attention within documents packed one after the other.
//
// For each document, head and query i:  out = sum_j p_ij v_j / sum_j p_ij,
// p_ij = e^(s_ij - m_i), in one pass over the keys i sees with a running maximum.
//
// A CTA takes one head of NQ tiles of 128 query rows and walks the 128-key tiles that
// any of them sees.  Both products run on the tensor cores, with everything between
// them in tensor memory: S = Q K^T (128 x 128 fp32) is read by the four warps of its
// tile, a row per thread, so that a row's maximum and sum need no exchange; the weights
// go back as 16-bit words over S, where the second product O += P V takes them as its
// first operand.  V is read as it lies in memory (its rows are the reduction).
//   warp 0      TMA producer: Q, then K and V tiles in a ring
//   warp 1      tensor memory, MMA issuer
//   warps 4-7   the first tile's rows: softmax, then the output; 8-11 the second's
// With two tiles the tensor cores work on one while the other's weights are computed,
// and K and V are read once for 256 rows; with one tile two CTAs share an SM instead.
// The maximum that weights are relative to follows the running one only when that has
// grown by more than 2^8 (weights up to 256 keep their 11 or 8 bits, sums are fp32), so
// that O is rarely rescaled: only then does a softmax warp wait for the product before.
// Weights are rounded to the inputs' 16-bit type for the second product, whose
// operands have one type; the sum of weights takes them unrounded.
#include "attention_internal.h"
#include "token_common.cuh"

namespace c3d {

namespace {

constexpr int kRows = 128;             // query rows and keys of a tile
constexpr uint32_t kBoxBytes = 16384;  // 128 rows of 64 elements
constexpr int kMaxStages = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLag = 8.0f;           // powers of two that weights may exceed 1 by

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if (BF) return pack_bf16x2(a, b);
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool BF>
__device__ __forceinline__ float elem(const unsigned char* base, long long i) {
    if (BF) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[i]);
    return __half2float(reinterpret_cast<const __half*>(base)[i]);
}

// A CTA's work: 128 * NQ rows from `row0` of a document, for one head.
struct Job {
    int row0, rows;          // of the document; rows: the document's queries
    int keys, shift;         // its keys; position of row r: r + shift
    int prefix;
    long long q0, k0;        // packed rows of the document's first query and key
    int head;
};

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

// The key tiles of the whole job, in order: those of the lead, then those from `skip` on.
struct Tiles {
    int lead, skip, count;
    __device__ int at(int n) const { return (n < lead ? n : n - lead + skip) * kRows; }
};
__device__ __forceinline__ Tiles tiles_of(const Range& r) {
    Tiles t;
    t.lead = (r.lead + kRows - 1) / kRows;
    t.skip = max(r.lo / kRows, t.lead);
    t.count = t.lead + max((r.hi + kRows - 1) / kRows - t.skip, 0);
    return t;
}
__device__ __forceinline__ bool sees(const Range& r, int t0) {
    return t0 < r.lead || (t0 < r.hi && t0 + kRows > r.lo);
}

template <bool BF>
__device__ bool finite_row(const unsigned char* v, long long at, int width) {
    for (int d = 0; d < width; ++d)
        if (!(fabsf(elem<BF>(v, at + d)) <= 3.4e38f)) return false;
    return true;
}

// A row's score at a key, in powers of two
__device__ __forceinline__ float shaped(const PackedParams& p, float dot, int i, int j, float slope2) {
    float s = dot * p.scale;
    if (p.cap > 0.0f) s = p.cap - 2.0f * p.cap * rcp_approx(1.0f + ex2(s * (2.0f * kLog2e / p.cap)));
    return s * kLog2e - slope2 * fabsf(static_cast<float>(i - j));
}

struct RowMask {
    int lo, hi, lead, keys;
    __device__ bool operator()(int j) const { return j < keys && ((j >= lo && j < hi) || j < lead); }
};
__device__ __forceinline__ RowMask row_mask(const PackedParams& p, const Job& j, int row) {
    const Range r = range_of(p, j, row, row + 1);
    return RowMask{r.lo, r.hi, r.lead, j.keys};
}

// A row whose result is not finite although what it sees may be: an unseen key of a
// tile that was multiplied (weight 0) has a value that is not finite.  Then the row is
// computed again, over what it sees alone.
template <bool BF>
__device__ __noinline__ void redo_row(const PackedParams& p, const Job& job, const Range& tile_range, int row) {
    const int kv = static_cast<int>(static_cast<long long>(job.head) * p.kv_heads / p.heads);
    const RowMask m = row_mask(p, job, row);
    const long long vbase = job.k0 * p.k_tok + static_cast<long long>(kv) * p.k_head;
    bool spoiled = false;
    const Tiles tl = tiles_of(tile_range);
    for (int n = 0; n < tl.count && !spoiled; ++n) {
        const int t0 = tl.at(n);
        for (int j = t0; j < min(t0 + kRows, job.keys) && !spoiled; ++j)
            if (!m(j)) spoiled = !finite_row<BF>(p.v, vbase + j * p.k_tok, p.width);
    }
    if (!spoiled) return;
    const long long qb = (job.q0 + row) * p.q_tok + static_cast<long long>(job.head) * p.q_head;
    const float slope2 = p.slopes ? p.slopes[job.head] * kLog2e : 0.0f;
    auto score = [&](int j) {
        float s = 0.0f;
        for (int d = 0; d < p.width; ++d) s += elem<BF>(p.q, qb + d) * elem<BF>(p.k, vbase + j * p.k_tok + d);
        return shaped(p, s, row + job.shift, j, slope2);
    };
    float top = -INFINITY, sum = 0.0f, o[128];
    bool nan = false;
    for (int pass = 0; pass < 2 && !nan; ++pass) {
        if (pass)
            for (int d = 0; d < p.width; ++d) o[d] = 0.0f;
        for (int part = 0; part < 2; ++part)
            for (int j = part ? max(m.lo, m.lead) : 0; j < (part ? m.hi : min(m.lead, m.keys)); ++j) {
                const float s = score(j);
                if (!pass) {
                    nan = nan || !(s < INFINITY);
                    top = fmaxf(top, s);
                } else if (top > -INFINITY) {
                    const float w = ex2(s - top);
                    sum += w;
                    for (int d = 0; d < p.width; ++d) o[d] += w * elem<BF>(p.v, vbase + j * p.k_tok + d);
                }
            }
    }
    uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) + (job.q0 + row) * p.out_tok +
                    static_cast<long long>(job.head) * p.out_head;
    for (int d = 0; d < p.width; ++d) {
        const float v = nan ? __uint_as_float(kNanBits) : sum == 0.0f ? 0.0f : o[d] / sum;
        dst[d] = static_cast<uint16_t>(pack2<BF>(v, 0.0f));
    }
}

template <int NQ>
constexpr int kThreads = 128 + 128 * NQ;

// NQ: query tiles of a CTA.  MOD: scores are capped, biased or scaled by a number that
// is not positive (else the scale goes into the exponent's one multiply-add).
template <bool BF, int NQ, bool MOD>
__global__ void __launch_bounds__(kThreads<NQ>, NQ == 1 ? 2 : 1)
    packed_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map, const __grid_constant__ PackedParams p,
                  const int stages) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const int boxes = (p.width + 63) / 64;
    const uint32_t tile_bytes = boxes * kBoxBytes;
    const uint32_t q_smem = base, ring = base + NQ * tile_bytes;
    const uint32_t bars = ring + stages * tile_bytes;
    const uint32_t full0 = bars, empty0 = full0 + 8u * kMaxStages, q_full = empty0 + 8u * kMaxStages;
    const uint32_t s_full0 = q_full + 8u, p_full0 = s_full0 + 16u, o_done0 = p_full0 + 16u;
    const uint32_t tail_bar = o_done0 + 16u, drain_bar = tail_bar + 8u;
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem_raw + (drain_bar + 8u - raw));
    // misc[0] TMEM base, [1] abort flag, [2] loads issued, [3] whether there is work; then the job
    volatile uint32_t* abort_flag = misc + 1;
    Job* shared_job = reinterpret_cast<Job*>(misc + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    griddep_launch_dependents();
    griddep_wait();
    if (warp == 0) {
        // which document's rows this CTA takes: 128 documents a step, four a lane
        const int head = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.heads));
        const long long want = blockIdx.x / static_cast<unsigned>(p.heads);
        long long before = 0;
        bool found = false;
        for (int s0 = 0; s0 < p.documents && !found; s0 += 128) {
            int off[5];
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                const int s = min(s0 + 4 * lane + i, p.documents);
                off[i] = static_cast<int>(min(max(static_cast<long long>(p.q_offsets[s]), 0ll), p.q_tokens));
            }
            int n[4], mine = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                n[i] = (max(off[i + 1] - off[i], 0) + NQ * kRows - 1) / (NQ * kRows);
                mine += n[i];
            }
            int run = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, run, d);
                if (lane >= d) run += o;
            }
            const uint32_t over = __ballot_sync(0xffffffffu, before + run > want);
            if (over) {
                found = true;
                if (lane == __ffs(over) - 1) {
                    int at = static_cast<int>(want - before) - (run - mine), i = 0;
                    while (at >= n[i]) at -= n[i++];
                    const int s = s0 + 4 * lane + i;
                    Job j;
                    j.rows = off[i + 1] - off[i];
                    j.row0 = (p.causal ? n[i] - 1 - at : at) * NQ * kRows;   // the longest first
                    const long long kb = min(max(static_cast<long long>(p.k_offsets[s]), 0ll), p.k_tokens);
                    const long long ke = min(max(static_cast<long long>(p.k_offsets[s + 1]), kb), p.k_tokens);
                    j.keys = static_cast<int>(ke - kb);
                    j.shift = j.keys - j.rows;
                    j.prefix = p.prefix ? min(max(p.prefix[s], 0), j.keys) : 0;
                    j.q0 = off[i];
                    j.k0 = kb;
                    j.head = head;
                    *shared_job = j;
                }
            }
            before += __shfl_sync(0xffffffffu, run, 31);
        }
        if (lane == 0) misc[3] = found;
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
        }
        mbar_init(q_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full0 + 8 * i, 1);
            mbar_init(p_full0 + 8 * i, 4);
            mbar_init(o_done0 + 8 * i, 1);
        }
        mbar_init(tail_bar, 1);
        mbar_init(drain_bar, 1);
        misc[1] = 0u;
        misc[2] = 0u;
        fence_mbar_init();
        prefetch_tmap(&q_map);
        prefetch_tmap(&k_map);
        prefetch_tmap(&v_map);
    }
    __syncthreads();
    if (!misc[3]) return;   // behind the last document
    if (warp == 1) {
        tmem_alloc(smem_u32(misc), NQ == 2 ? 512 : 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    const Job job = *shared_job;
    const uint32_t o_pitch = boxes * 64u;
    const int row_end = min(job.row0 + NQ * kRows, job.rows);
    const Tiles tl = tiles_of(range_of(p, job, job.row0, row_end));
    Range part[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i)
        part[i] = range_of(p, job, job.row0 + i * kRows, min(job.row0 + (i + 1) * kRows, job.rows));

    if (warp == 0) {
        const int kv = static_cast<int>(static_cast<long long>(job.head) * p.kv_heads / p.heads);
        int st = 0;
        uint32_t ph = 0, issued = 0;
        bool ok = true;
        if (tl.count > 0 && lane == 0) {
            mbar_arrive_expect_tx(q_full, NQ * tile_bytes);
            for (int i = 0; i < NQ; ++i)
                for (int b = 0; b < boxes; ++b)
                    tma_load_3d(q_smem + i * tile_bytes + b * kBoxBytes, &q_map, q_full, b * 64, job.head,
                                static_cast<int>(job.q0 + job.row0 + i * kRows));
        }
        for (int n = 0; n < 2 * tl.count && ok; ++n) {
            const bool value = n & 1;
            const int t0 = tl.at(n >> 1);
            // the keys of a tile behind the document's last are other documents': their scores
            // are replaced, their values (times a weight of 0) have to be finite
            const bool tail = value && t0 + kRows > job.keys;
            ok = wait_bar(empty0 + 8 * st, ph ^ 1u, abort_flag, p.status, p.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t dst = ring + st * tile_bytes, bar = tail ? tail_bar : full0 + 8 * st;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, tile_bytes);
                for (int b = 0; b < boxes; ++b)
                    tma_load_3d(dst + b * kBoxBytes, value ? &v_map : &k_map, bar, b * 64, kv,
                                static_cast<int>(job.k0 + t0));
            }
            if (tail) {
                ok = wait_bar(tail_bar, 0, abort_flag, p.status, p.wait_ns);
                if (!__all_sync(0xffffffffu, ok)) {
                    drain_wait(tail_bar, 0);
                    break;
                }
                const int first = job.keys - t0;
                for (int i = first * 8 + lane; i < kRows * 8; i += 32)
                    for (int b = 0; b < boxes; ++b)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + b * kBoxBytes + i * 16u), "r"(0u)
                                     : "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full0 + 8 * st);
            }
            if (lane == 0) misc[2] = ++issued;
            if (++st == stages) {
                st = 0;
                ph ^= 1u;
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && tl.count > 0) {
            constexpr uint32_t kType = BF ? (1u << 7) | (1u << 10) : 0u;
            const int cols = (p.width + 15) / 16 * 16;
            const uint32_t idesc_s = (1u << 4) | kType | ((kRows >> 3) << 17) | ((kRows >> 4) << 24);
            const uint32_t idesc_o = (1u << 4) | kType | (1u << 16) | (static_cast<uint32_t>(cols >> 3) << 17) |
                                     ((kRows >> 4) << 24);
            const uint64_t qdesc = make_smem_desc(q_smem, 1024u, 2u);
            const uint64_t kdesc = make_smem_desc(ring, 1024u, 2u);
            const uint64_t vdesc = make_smem_desc(ring, 1024u, 2u, kBoxBytes);
            const uint32_t step = tile_bytes >> 4;
            int st = 0;
            uint32_t ph = 0;
            uint32_t turn[2] = {0u, 0u};   // steps of either tile so far
            auto next = [&]() {
                if (++st == stages) {
                    st = 0;
                    ph ^= 1u;
                }
            };
            auto scores = [&](int i, int slot) {
                for (int k = 0; k < cols / 16; ++k) {
                    const uint64_t off = (k >> 2) * (kBoxBytes >> 4) + 2 * (k & 3);
                    tc_mma_f16(tmem + i * kRows, qdesc + i * step + off, kdesc + slot * step + off, idesc_s, k != 0);
                }
                tc_commit(s_full0 + 8 * i);
            };
            bool ok = wait_bar(q_full, 0, abort_flag, p.status, p.wait_ns) &&
                      wait_bar(full0, 0, abort_flag, p.status, p.wait_ns);
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < NQ; ++i)
                    if (sees(part[i], tl.at(0))) scores(i, 0);
                tc_commit(empty0);
            }
            next();
            for (int n = 0; n < tl.count && ok; ++n) {
                const int t0 = tl.at(n), t1 = tl.at(n + 1);
                const bool more = n + 1 < tl.count;
                const int vs = st;
                const uint32_t vph = ph;
                next();
                const int ks = st;
                const uint32_t kph = ph;
                if (more) next();
                bool v_ready = false, k_ready = false;
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    if (sees(part[i], t0)) {
                        if (!v_ready) ok = ok && wait_bar(full0 + 8 * vs, vph, abort_flag, p.status, p.wait_ns);
                        v_ready = true;
                        ok = ok && wait_bar(p_full0 + 8 * i, turn[i] & 1u, abort_flag, p.status, p.wait_ns);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < kRows / 16; ++k)
                            tc_mma_f16_ta(tmem + NQ * kRows + i * o_pitch, tmem + i * kRows + 8 * k,
                                          vdesc + vs * step + k * 128, idesc_o, (turn[i] | k) != 0);
                        tc_commit(o_done0 + 8 * i);
                        ++turn[i];
                    }
                    if (more && sees(part[i], t1)) {
                        if (!k_ready) ok = ok && wait_bar(full0 + 8 * ks, kph, abort_flag, p.status, p.wait_ns);
                        k_ready = true;
                        if (!ok) break;
                        tc_fence_after();
                        scores(i, ks);
                    }
                }
                if (!ok) break;
                tc_commit(empty0 + 8 * vs);   // (any tile is seen by one of the two)
                if (more) tc_commit(empty0 + 8 * ks);
            }
        }
    } else if (warp >= 4) {
        const int i = (warp - 4) >> 2;
        const int row = job.row0 + i * kRows + (warp & 3) * 32 + lane;
        const bool valid = row < job.rows;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + i * kRows, t_o = tmem + lanes + NQ * kRows + i * o_pitch;
        Range mine = part[0];
        if (NQ == 2 && i == 1) mine = part[NQ - 1];
        const RowMask mask = row_mask(p, job, min(row, job.rows - 1));
        const int a = job.row0 + i * kRows;
        const int b = min(a + kRows, job.rows);
        // keys that every row of the tile sees
        int all_lo = 0, all_hi = job.keys;
        if (p.window > 0) {
            all_lo = static_cast<int>(max(0ll, static_cast<long long>(b) + job.shift - p.window));
            all_hi = static_cast<int>(min(static_cast<long long>(all_hi), static_cast<long long>(a) + job.shift + p.window));
        }
        if (p.causal) all_hi = min(all_hi, a + job.shift + 1);
        const float slope2 = MOD && p.slopes ? p.slopes[job.head] * kLog2e : 0.0f;
        const float c = MOD ? 1.0f : p.scale * kLog2e;
        const int pos = row + job.shift;
        float ref = -INFINITY, sum = 0.0f;   // ref: what the weights are relative to
        uint32_t turn = 0;
        bool ok = true;
        for (int n = 0; n < tl.count; ++n) {
            const int t0 = tl.at(n);
            if (!sees(mine, t0)) continue;
            ok = wait_bar(s_full0 + 8 * i, turn & 1u, abort_flag, p.status, p.wait_ns);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t s[4][32];
#pragma unroll
            for (int h = 0; h < 4; ++h) tmem_ld_32x32b_x32(t_s + 32 * h, s[h]);
            tmem_ld_wait();
            if (MOD) {
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        s[h][e] = __float_as_uint(shaped(p, __uint_as_float(s[h][e]), pos, t0 + 32 * h + e, slope2));
            }
            const bool open = t0 + kRows <= job.keys &&
                              (t0 + kRows <= job.prefix || (t0 >= all_lo && t0 + kRows <= all_hi));
            if (!open) {
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!mask(t0 + 32 * h + e)) s[h][e] = __float_as_uint(-INFINITY);
            }
            float top = -INFINITY;
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
                for (int e = 0; e < 32; ++e) top = fmaxf(top, __uint_as_float(s[h][e]));
            if (turn == 0) {
                ref = top;
            } else {
                const bool rise = top * c > ref * c + kLag;
                if (__any_sync(0xffffffffu, rise)) {
                    ok = wait_bar(o_done0 + 8 * i, (turn - 1) & 1u, abort_flag, p.status, p.wait_ns);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const float now = fmaxf(ref, top);
                    const float f = now == -INFINITY ? 1.0f : ex2((ref - now) * c);
                    ref = now;
                    sum *= f;
                    for (uint32_t d = 0; d < o_pitch; d += 8) {
                        uint32_t o[8];
                        tmem_ld_32x32b_x8(t_o + d, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st_32x32b_x8(t_o + d, o);
                    }
                }
            }
            const float off = ref == -INFINITY ? 0.0f : ref * c;
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float x = ex2(fmaf(__uint_as_float(s[h][e]), c, -off));
                    const float y = ex2(fmaf(__uint_as_float(s[h][e + 1]), c, -off));
                    sum += x + y;
                    s[h >> 1][(h & 1) * 16 + e / 2] = pack2<BF>(x, y);
                }
            tmem_st_32x32b_x32(t_s, s[0]);
            tmem_st_32x32b_x32(t_s + 32, s[1]);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full0 + 8 * i);
            ++turn;
        }
        if (ok && turn > 0) ok = wait_bar(o_done0 + 8 * i, (turn - 1) & 1u, abort_flag, p.status, p.wait_ns);
        if (__all_sync(0xffffffffu, ok)) {
            tc_fence_after();
            const float inv = turn == 0 || sum == 0.0f ? 0.0f : 1.0f / sum;
            uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) + (job.q0 + row) * p.out_tok +
                            static_cast<long long>(job.head) * p.out_head;
            bool odd = false;
            for (int d = 0; d < p.width; d += 8) {
                uint32_t o[8];
                if (turn > 0) {
                    tmem_ld_32x32b_x8(t_o + d, o);
                    tmem_ld_wait();
                }
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = turn > 0 && inv != 0.0f ? __uint_as_float(o[2 * e]) * inv : 0.0f;
                    const float y = turn > 0 && inv != 0.0f ? __uint_as_float(o[2 * e + 1]) * inv : 0.0f;
                    odd = odd || !(fabsf(x) + fabsf(y) < INFINITY);
                    w[e] = pack2<BF>(x, y);
                }
                if (valid && p.out_aligned) {
                    *reinterpret_cast<uint4*>(dst + d) = make_uint4(w[0], w[1], w[2], w[3]);
                } else if (valid) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) dst[d + e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
                }
                __syncwarp();
            }
            if (valid && odd) redo_row<BF>(p, job, mine, row);
        }
        tc_fence_before();
    }
    __syncwarp();
    __syncthreads();
    if (*abort_flag) {
        // drain: the loads, then the MMAs in flight
        if (threadIdx.x == 0) {
            if (tl.count > 0) drain_wait(q_full, 0);
            for (uint32_t n = misc[2] > static_cast<uint32_t>(stages) ? misc[2] - stages : 0u; n < misc[2]; ++n)
                drain_wait(full0 + 8 * (n % stages), (n / stages) & 1u);
        }
        if (threadIdx.x == 32) {
            tc_commit(drain_bar);
            drain_wait(drain_bar, 0);
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, NQ == 2 ? 512 : 256);
    }
}

template <bool BF, int NQ, bool MOD>
cudaError_t run(const PackedMaps& maps, const PackedParams& p, cudaStream_t stream) {
    const uint32_t tile = static_cast<uint32_t>((p.width + 63) / 64) * kBoxBytes;
    // shared memory of the SM, or half of it for two CTAs
    const uint32_t room = (NQ == 2 ? 232448u : 115200u) - 1024u - 512u;
    int stages = static_cast<int>((room - NQ * tile) / tile);
    if (stages > kMaxStages) stages = kMaxStages;
    const size_t smem = 1024u + (NQ + stages) * tile + 512u;
    static std::atomic<int> slots[kMaxDevices];
    cudaError_t e = ensure_dynamic_smem(packed_kernel<BF, NQ, MOD>, smem, slots);
    if (e != cudaSuccess) return e;
    const long long blocks = (p.q_tokens / (NQ * kRows) + p.documents) * p.heads;
    return launch_ex(packed_kernel<BF, NQ, MOD>, static_cast<unsigned>(blocks), dim3(kThreads<NQ>), smem, 1, stream,
                     maps.q, maps.k, maps.v, p, stages);
}

}  // namespace

cudaError_t launch_packed(const PackedMaps& maps, const PackedParams& p, int dtype, int num_sms,
                          cudaStream_t stream) {
    const bool mod = p.cap > 0.0f || p.slopes || !(p.scale > 0.0f);
    const bool bf = dtype == kTokBf16;
    // two tiles where documents are long and there are CTAs enough for all SMs
    const bool two = p.q_tokens / p.documents >= 1024 && p.q_tokens / 256 * p.heads >= num_sms;
    if (two) {
        if (bf) return mod ? run<true, 2, true>(maps, p, stream) : run<true, 2, false>(maps, p, stream);
        return mod ? run<false, 2, true>(maps, p, stream) : run<false, 2, false>(maps, p, stream);
    }
    if (bf) return mod ? run<true, 1, true>(maps, p, stream) : run<true, 1, false>(maps, p, stream);
    return mod ? run<false, 1, true>(maps, p, stream) : run<false, 1, false>(maps, p, stream);
}

}  // namespace c3d
