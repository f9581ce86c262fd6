// token_attention_api.cu -- the C ABI of rotary positions, the key-value cache and
// attention (declared in include/token_attention.h): argument checks and launches.
// No allocation.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <utility>

#include "token_attention_internal.h"
#include "token_common.cuh"

namespace c3d {

namespace {

constexpr int64_t kMaxDim = (1ll << 31) - 1;
constexpr int64_t kMaxTokens = kMaxDim - 256;   // positions that kernels count in 32 bits

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
bool is_half_type(int t) { return t == CONV_DTYPE_BF16 || t == CONV_DTYPE_F16; }
int size_of(int t) {
    return t == CONV_DTYPE_F32 ? 4 : t == CONV_DTYPE_BF16 || t == CONV_DTYPE_F16 ? 2 : 1;
}
bool aligned_to(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) % bytes) == 0; }
bool fits(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

// whether rows of `width` elements share some, for dimensions {size, stride} that lie in
// one another in some order
bool overlap(int64_t width, std::initializer_list<std::pair<int64_t, int64_t>> dims) {
    std::pair<int64_t, int64_t> d[3];
    int n = 0;
    for (const auto& e : dims)
        if (e.first > 1) d[n++] = {e.second, e.first};
    std::sort(d, d + n);
    __int128 extent = width;
    for (int i = 0; i < n; ++i) {
        if (d[i].first < extent) return true;
        extent += static_cast<__int128>(d[i].second - 1) * d[i].first;
    }
    return false;
}

// frequency / 2 pi, modulo 1, in units of 2^-64 (nearest), modulo 2^64.  1 / 2 pi is the sum
// of two doubles, exact to 2^-110, so that the product with the frequency's 53 bits is exact
// beyond 2^-64 for frequencies up to 2^40, and to 2^-105 of the turns themselves beyond.
unsigned long long turns_of(double frequency) {
    constexpr double kHigh = 0x1.45f306dc9c883p-3, kLow = -0x1.6b01ec5417056p-57;
    const double f = std::fabs(frequency);
    const volatile double product = f * kHigh;   // (rounded here, whatever a compiler fuses)
    const double high = product, low = std::fma(f, kHigh, -high) + f * kLow;
    // whole turns of whole positions do not count; what is left is exact in each part
    const double a = (high - std::floor(high)) * 0x1p64, b = (low - std::rint(low)) * 0x1p64;
    const double whole = std::floor(a), rest = b + (a - whole);   // a < 2^64, |rest| <= 2^63 + 1
    unsigned long long t = static_cast<unsigned long long>(whole);
    t += rest < 0.0 ? 0ull - static_cast<unsigned long long>(0.5 - rest) : static_cast<unsigned long long>(rest + 0.5);
    return frequency < 0.0 ? 0ull - t : t;
}

// heads of tokens: [tokens, heads, width] with strides in elements
const char* bad_heads(const void* p, int64_t tok, int64_t head, int64_t tokens, int64_t heads,
                      int64_t width, int elt) {
    if (!p) return "null pointer";
    if (!aligned_to(p, elt)) return "a pointer is not aligned to its element type";
    if (tok < 0 || head < 0) return "strides must be 0 or more";
    if (heads > 1 && head < width) return "a head stride is below the head's width";
    if (tokens > 1 && tok < width) return "a token stride is below the head's width";
    return nullptr;
}
// the same of an output, whose rows nothing else may share
const char* bad_out(const void* p, int64_t tok, int64_t head, int64_t tokens, int64_t heads,
                    int64_t width, int elt) {
    if (const char* e = bad_heads(p, tok, head, tokens, heads, width, elt)) return e;
    return overlap(width, {{tokens, tok}, {heads, head}}) ? "an output's rows overlap" : nullptr;
}
bool words(const void* p, int64_t tok, int64_t head, int elt) {
    return aligned_to(p, 16) && tok * elt % 16 == 0 && head * elt % 16 == 0;
}

const char* bad_cache(const kv_cache* c) {
    if (!c || !c->k || !c->v) return "null pointer";
    if (!is_code_type(c->dtype) && !is_half_type(c->dtype))
        return "a cache must be INT8, FP8_E4M3, BF16 or F16";
    if (!fits(c->pages, 1, kMaxDim) || !fits(c->heads, 1, 1 << 20) || !fits(c->page_size, 1, 1 << 30))
        return "a cache must have pages, heads and tokens in a page";
    if (!fits(c->width, 16, 256) || c->width % 16) return "a cache's width must be a multiple of 16 up to 256";
    const int elt = size_of(c->dtype);
    if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16) || c->page_stride * elt % 16 ||
        c->head_stride * elt % 16 || c->row_stride * elt % 16)
        return "a cache's rows must be 16-byte aligned";
    if (c->row_stride > 1 << 26) return "a cache's row stride must be below 2^26";
    if (c->row_stride < c->width || c->head_stride < 0 || c->page_stride < 0)
        return "a cache's row stride is below its width";
    if (overlap(c->width, {{c->pages, c->page_stride}, {c->heads, c->head_stride}, {c->page_size, c->row_stride}}))
        return "a cache's rows overlap";
    if (is_code_type(c->dtype)) {
        if (!c->k_scale || !c->v_scale) return "an 8-bit cache needs scales";
        if (!aligned_to(c->k_scale, 4) || !aligned_to(c->v_scale, 4))
            return "a pointer is not aligned to its element type";
        if (c->scale_page_stride < 0 || c->scale_head_stride < 0) return "strides must be 0 or more";
        if (overlap(1, {{c->pages, c->scale_page_stride}, {c->heads, c->scale_head_stride}, {c->page_size, 1}}))
            return "a cache's scales overlap";
    }
    return nullptr;
}

const char* bad_table(const int32_t* table, int64_t stride, int64_t pages, int64_t sequences) {
    if (!fits(pages, 0, kMaxDim)) return "a page table's width must be 0 or more, below 2^31";
    if (pages && sequences && (!table || !aligned_to(table, 4))) return "null or unaligned page table";
    if (sequences > 1 && stride < pages) return "a page table's stride is below its width";
    return nullptr;
}

// cuTensorMapEncodeTiled, found in the driver as the convolutions find it
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Tensor map of RANK dimensions, innermost first (strides in bytes, multiples of 16, of all
// but that one): boxes of `box` elements, 128-byte swizzle,
// zeros outside.
template <int RANK>
int encode(CUtensorMap* m, const void* ptr, int elt, const cuuint64_t (&dims)[RANK],
           const cuuint64_t (&strides)[RANK - 1], const cuuint32_t (&box)[RANK]) {
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                           cudaSuccess &&
                       q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<EncodeTiled>(f)
                   : nullptr;
    }();
    if (!fn) {
        set_last_error("the driver's tensor-map encoder is not available");
        return CONV_ERR_CUDA;
    }
    cuuint32_t steps[RANK];
    for (cuuint32_t& s : steps) s = 1;
    const CUresult r = fn(m, elt == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, RANK,
                          const_cast<void*>(ptr), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return CONV_OK;
    char msg[96];
    std::snprintf(msg, sizeof msg, "cuTensorMapEncodeTiled failed (code %d)", static_cast<int>(r));
    set_last_error(msg);
    return CONV_ERR_CUDA;
}

cuuint64_t u64(int64_t v) { return static_cast<cuuint64_t>(v); }

// Heads [rows, heads, width] of 16-bit elements: box_rows rows x 64 elements of one head
int encode_heads(CUtensorMap* m, const void* ptr, int64_t width, int64_t heads, int64_t rows,
                 int64_t head_pitch, int64_t row_pitch, int box_rows) {
    return encode<3>(m, ptr, 2, {u64(width), u64(heads), u64(rows)}, {u64(head_pitch), u64(row_pitch)},
                     {64u, 1u, static_cast<cuuint32_t>(box_rows)});
}

// A cache [pages, heads, rows, width]: box_rows rows x 128 bytes of one head of one page
// (one head or page has no pitch of its own)
int encode_pages(CUtensorMap* m, const void* ptr, int elt, int64_t width, int64_t rows, int64_t heads,
                 int64_t pages, int64_t row_pitch, int64_t head_pitch, int64_t page_pitch, int box_rows) {
    return encode<4>(m, ptr, elt, {u64(width), u64(rows), u64(heads), u64(pages)},
                     {u64(row_pitch), u64(heads > 1 ? head_pitch : row_pitch), u64(pages > 1 ? page_pitch : row_pitch)},
                     {static_cast<cuuint32_t>(128 / elt), static_cast<cuuint32_t>(box_rows), 1u, 1u});
}

PageMap page_map(const kv_cache* c, const int32_t* table, int64_t stride, int64_t pages) {
    PageMap m{};
    const int elt = size_of(c->dtype);
    m.table = table;
    m.table_stride = stride;
    m.capacity = pages > kMaxTokens / c->page_size ? kMaxTokens : pages * c->page_size;
    m.pages = c->pages;
    m.page_stride = c->page_stride * elt;
    m.head_stride = c->head_stride * elt;
    m.row_stride = c->row_stride * elt;
    m.scale_page_stride = c->scale_page_stride;
    m.scale_head_stride = c->scale_head_stride;
    m.by_page = make_fastdiv(static_cast<uint32_t>(c->page_size));
    return m;
}

int cache_rows(const kv_cache* cache, void* k, void* v, int dtype, int64_t token_stride,
               int64_t head_stride, int64_t tokens, const int32_t* offsets, const int32_t* starts,
               const int32_t* page_table, int64_t table_stride, int64_t table_pages, int64_t sequences,
               bool write, cudaStream_t stream) {
    const char* name = write ? "kv_cache_write launch" : "kv_cache_read launch";
    if (!fits(tokens, 0, kMaxDim) || !fits(sequences, 0, kMaxDim))
        return invalid("tokens and sequences must be 0 or more, below 2^31");
    if (const char* e = bad_cache(cache)) return invalid(e);
    if (!is_float_type(dtype)) return invalid("dtype must be BF16, F16 or F32");
    if (write && is_half_type(cache->dtype) && dtype != cache->dtype)
        return invalid("rows must have the type of an unquantised cache");
    if (const char* e = bad_table(page_table, table_stride, table_pages, sequences)) return invalid(e);
    if (write && !offsets && tokens != sequences)
        return invalid("without offsets there is one token for each sequence");
    if (tokens == 0 || sequences == 0) return CONV_OK;
    if (write ? !starts : !offsets) return invalid("null pointer");
    if (write ? cache->k == cache->v : k == v) return invalid("keys and values must be written to places of their own");
    if (!aligned_to(offsets, 4) || !aligned_to(starts, 4))
        return invalid("a pointer is not aligned to its element type");
    for (const void* p : {static_cast<const void*>(k), static_cast<const void*>(v)})
        if (const char* e = (write ? bad_heads : bad_out)(p, token_stride, head_stride, tokens, cache->heads,
                                                          cache->width, size_of(dtype)))
            return invalid(e);
    if (tokens > kMaxDim * 4 / cache->heads) {
        set_last_error("more rows than the kernels count");
        return CONV_ERR_UNSUPPORTED;
    }
    CacheParams p{};
    p.k = static_cast<unsigned char*>(cache->k);
    p.v = static_cast<unsigned char*>(cache->v);
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.map = page_map(cache, page_table, table_stride, table_pages);
    p.rows_k = static_cast<unsigned char*>(k);
    p.rows_v = static_cast<unsigned char*>(v);
    p.tok_stride = token_stride;
    p.head_stride = head_stride;
    p.offsets = offsets;
    p.starts = starts;
    p.tokens = tokens;
    p.sequences = static_cast<int>(sequences);
    p.heads = static_cast<int>(cache->heads);
    p.width = static_cast<int>(cache->width);
    p.aligned = words(k, token_stride, head_stride, size_of(dtype)) &&
                words(v, token_stride, head_stride, size_of(dtype));
    return launched(write ? launch_cache_write(p, dtype, cache->dtype, stream)
                          : launch_cache_read(p, dtype, cache->dtype, stream), name);
}

}  // namespace

}  // namespace c3d

using namespace c3d;

extern "C" {

int rotary_fwd(const void* x, int dtype, int64_t x_token_stride, int64_t x_head_stride,
               const void* positions, int position_bytes, int axes, const int* axis,
               const double* frequency, int pairs, int interleaved, int inverse, int64_t tokens,
               int64_t heads, int64_t width, void* out, int64_t out_token_stride,
               int64_t out_head_stride, cudaStream_t stream) {
    if (!fits(tokens, 0, kMaxDim) || !fits(heads, 0, 1 << 20) || !fits(width, 1, 1 << 20))
        return invalid("tokens must be 0 or more, below 2^31, heads and width up to 2^20");
    if (!is_float_type(dtype)) return invalid("dtype must be BF16, F16 or F32");
    if (position_bytes != 4 && position_bytes != 8) return invalid("positions must be int32 or int64");
    if (axes < 1 || axes > ROTARY_MAX_AXES) return invalid("axes must be 1 to 8");
    if (pairs < 1 || pairs > ROTARY_MAX_PAIRS || 2ll * pairs > width)
        return invalid("pairs must be 1 to 128, and fit the width");
    if (!axis || !frequency) return invalid("null pointer");
    RotaryParams p{};
    for (int i = 0; i < pairs; ++i) {
        if (axis[i] < 0 || axis[i] >= axes) return invalid("a pair's axis is not one of the positions'");
        if (!std::isfinite(frequency[i])) return invalid("a frequency is not finite");
        p.turns[i] = turns_of(frequency[i]);
        p.axis[i] = static_cast<unsigned char>(axis[i]);
    }
    if (tokens == 0 || heads == 0) return CONV_OK;
    const int elt = size_of(dtype);
    if (const char* e = bad_heads(x, x_token_stride, x_head_stride, tokens, heads, width, elt)) return invalid(e);
    if (const char* e = bad_out(out, out_token_stride, out_head_stride, tokens, heads, width, elt))
        return invalid(e);
    if (!positions || !aligned_to(positions, position_bytes)) return invalid("null or unaligned positions");
    p.x = x;
    p.out = out;
    p.positions = positions;
    p.x_tok = x_token_stride;
    p.x_head = x_head_stride;
    p.out_tok = out_token_stride;
    p.out_head = out_head_stride;
    p.tokens = tokens;
    p.heads = static_cast<int>(heads);
    p.width = static_cast<int>(width);
    p.axes = axes;
    p.pairs = pairs;
    p.pos64 = position_bytes == 8;
    p.interleaved = interleaved != 0;
    p.inverse = inverse != 0;
    p.copy_rest = out != x;
    int align = 16;
    const int64_t at[6] = {static_cast<int64_t>(reinterpret_cast<uintptr_t>(x)),
                           static_cast<int64_t>(reinterpret_cast<uintptr_t>(out)), x_token_stride * elt,
                           x_head_stride * elt, out_token_stride * elt, out_head_stride * elt};
    for (int64_t v : at)
        while (v % align) align /= 2;
    return launched(launch_rotary(p, dtype, align, stream), "rotary_fwd launch");
}

int kv_cache_write(const kv_cache* cache, const void* k, const void* v, int dtype,
                   int64_t token_stride, int64_t head_stride, int64_t tokens,
                   const int32_t* offsets, const int32_t* starts, const int32_t* page_table,
                   int64_t table_stride, int64_t table_pages, int64_t sequences,
                   cudaStream_t stream) {
    return cache_rows(cache, const_cast<void*>(k), const_cast<void*>(v), dtype, token_stride, head_stride,
                      tokens, offsets, starts, page_table, table_stride, table_pages, sequences, true, stream);
}

int kv_cache_read(const kv_cache* cache, void* k, void* v, int dtype, int64_t token_stride,
                  int64_t head_stride, int64_t tokens, const int32_t* offsets,
                  const int32_t* starts, const int32_t* page_table, int64_t table_stride,
                  int64_t table_pages, int64_t sequences, cudaStream_t stream) {
    return cache_rows(cache, k, v, dtype, token_stride, head_stride, tokens, offsets, starts, page_table,
                      table_stride, table_pages, sequences, false, stream);
}

size_t paged_attention_workspace_size(int64_t sequences, int64_t heads, int64_t kv_heads,
                                      int64_t width, int64_t page_size, int64_t table_pages) {
    if (sequences < 1 || kv_heads < 1 || heads < kv_heads || heads % kv_heads || !fits(width, 16, 256) ||
        page_size < 1 || table_pages < 0)
        return 0;
    LaunchLimits lim;
    if (launch_limits(&lim)) return 0;
    const int64_t capacity = table_pages > kMaxTokens / page_size ? kMaxTokens : table_pages * page_size;
    const int64_t group = heads / kv_heads;
    if (paged_whole(sequences, kv_heads, group, static_cast<int>(width), capacity, lim.num_sms)) return 0;
    const int grid = paged_grid(sequences, kv_heads, group, static_cast<int>(width), capacity, lim.num_sms);
    return paged_workspace(grid, static_cast<int>(width));
}

int paged_attention_fwd(const void* q, int q_dtype, int64_t q_sequence_stride,
                        int64_t q_head_stride, const kv_cache* cache, const int32_t* page_table,
                        int64_t table_stride, int64_t table_pages, const int32_t* lengths,
                        const int32_t* prefix, const float* slopes, float scale, float cap,
                        int64_t window, int64_t sequences, int64_t heads, void* out,
                        int64_t out_sequence_stride, int64_t out_head_stride, void* workspace,
                        size_t workspace_bytes, cudaStream_t stream) {
    if (!fits(sequences, 0, kMaxDim)) return invalid("sequences must be 0 or more, below 2^31");
    if (const char* e = bad_cache(cache)) return invalid(e);
    if (!is_half_type(q_dtype)) return invalid("q_dtype must be BF16 or F16");
    if (is_half_type(cache->dtype) && q_dtype != cache->dtype)
        return invalid("q must have the type of an unquantised cache");
    if (!fits(heads, 1, 1 << 20) || heads % cache->heads) return invalid("heads must be a multiple of the cache's");
    if (!std::isfinite(scale)) return invalid("scale must be finite");
    if (cap != 0.0f && (!(cap >= 1e-20f) || !std::isfinite(cap))) return invalid("cap must be 0, or 1e-20 or more");
    if (window < 0) return invalid("window must be 0 or more");
    if (const char* e = bad_table(page_table, table_stride, table_pages, sequences)) return invalid(e);
    if (sequences == 0) return CONV_OK;
    if (!lengths) return invalid("null pointer");
    if (!aligned_to(lengths, 4) || !aligned_to(prefix, 4) || !aligned_to(slopes, 4))
        return invalid("a pointer is not aligned to its element type");
    if (const char* e = bad_heads(q, q_sequence_stride, q_head_stride, sequences, heads, cache->width, 2))
        return invalid(e);
    if (const char* e = bad_out(out, out_sequence_stride, out_head_stride, sequences, heads, cache->width, 2))
        return invalid(e);
    LaunchLimits lim;
    if (int rc = launch_limits(&lim)) return rc;
    PagedParams p{};
    p.q = static_cast<const unsigned char*>(q);
    p.out = static_cast<unsigned char*>(out);
    p.k = static_cast<const unsigned char*>(cache->k);
    p.v = static_cast<const unsigned char*>(cache->v);
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.map = page_map(cache, page_table, table_stride, table_pages);
    p.lengths = lengths;
    p.prefix = prefix;
    p.slopes = slopes;
    p.q_seq = q_sequence_stride;
    p.q_head = q_head_stride;
    p.out_seq = out_sequence_stride;
    p.out_head = out_head_stride;
    p.scale = scale;
    p.cap = cap;
    p.inv_cap = cap > 0.0f ? 1.0f / cap : 0.0f;
    p.window = static_cast<int>(window > kMaxTokens ? 0 : window);
    p.sequences = static_cast<int>(sequences);
    p.kv_heads = static_cast<int>(cache->heads);
    p.group = static_cast<int>(heads / cache->heads);
    p.width = static_cast<int>(cache->width);
    p.grid = paged_grid(sequences, cache->heads, p.group, p.width, p.map.capacity, lim.num_sms);
    p.num_sms = lim.num_sms;
    p.whole = paged_whole(sequences, cache->heads, p.group, p.width, p.map.capacity, lim.num_sms);
    // (one of 0 bytes, where that is the size, is none; any other that is given has to do for
    // heads that are split, too)
    const size_t need = paged_workspace(p.grid, p.width);
    const bool given = workspace && (workspace_bytes || !p.whole);
    if (given ? workspace_bytes < need || !aligned_to(workspace, 16) : !p.whole)
        return invalid(p.whole ? "paged_attention_fwd needs no workspace here, and one that is given must be 16-byte "
                                 "aligned and large enough for key heads that are split"
                               : "paged_attention_fwd needs a 16-byte aligned workspace of "
                                 "paged_attention_workspace_size bytes");
    if (!p.whole) {
        p.jobs = static_cast<int4*>(workspace);
        p.partial = reinterpret_cast<float*>(p.jobs + p.grid);
    }
    p.status = lim.status;
    p.wait_ns = lim.wait_ns;
    // blocks of tokens that lie in one page (or in two halves) are loaded by TMA, with their
    // scales where those are 16-byte aligned
    const int elt = size_of(cache->dtype);
    const bool scales = !is_code_type(cache->dtype) ||
                        (aligned_to(cache->k_scale, 16) && aligned_to(cache->v_scale, 16) &&
                         cache->scale_page_stride % 4 == 0 && cache->scale_head_stride % 4 == 0);
    p.rows_box = !scales || cache->page_size % 8           ? 0
                 : cache->page_size % 16                    ? 8
                 : cache->page_size % 32 || p.width * elt > 128 ? 16
                                                            : 32;
    PagedMaps maps{};
    if (p.rows_box)
        for (int i = 0; i < 2; ++i)
            if (int rc = encode_pages(i ? &maps.v : &maps.k, i ? cache->v : cache->k, elt, cache->width,
                                      cache->page_size, cache->heads, cache->pages, p.map.row_stride,
                                      p.map.head_stride, p.map.page_stride, p.rows_box))
                return rc;
    return launched(launch_paged(maps, p, q_dtype, cache->dtype, stream), "paged_attention_fwd launch");
}

int packed_attention_fwd(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                         const void* k, const void* v, int64_t k_token_stride,
                         int64_t k_head_stride, int dtype, const int32_t* q_offsets,
                         const int32_t* k_offsets, int64_t documents, int64_t q_tokens,
                         int64_t k_tokens, int64_t heads, int64_t kv_heads, int64_t width,
                         int causal, int64_t window, const int32_t* prefix, const float* slopes,
                         float scale, float cap, void* out, int64_t out_token_stride,
                         int64_t out_head_stride, cudaStream_t stream) {
    if (!fits(documents, 0, kMaxTokens) || !fits(q_tokens, 0, kMaxTokens) || !fits(k_tokens, 0, kMaxTokens))
        return invalid("documents and tokens must be 0 or more, below 2^31 - 256");
    if (!is_half_type(dtype)) return invalid("dtype must be BF16 or F16");
    if (!fits(width, 8, 128) || width % 8) return invalid("width must be a multiple of 8 up to 128");
    if (!fits(kv_heads, 1, 1 << 20) || !fits(heads, 1, 1 << 20) || heads % kv_heads)
        return invalid("heads must be a multiple of kv_heads");
    if (!std::isfinite(scale)) return invalid("scale must be finite");
    if (cap != 0.0f && (!(cap >= 1e-20f) || !std::isfinite(cap))) return invalid("cap must be 0, or 1e-20 or more");
    if (window < 0) return invalid("window must be 0 or more");
    if (documents == 0 || q_tokens == 0) return CONV_OK;
    if (!q_offsets || !k_offsets) return invalid("null pointer");
    if (!aligned_to(q_offsets, 4) || !aligned_to(k_offsets, 4) || !aligned_to(prefix, 4) || !aligned_to(slopes, 4))
        return invalid("a pointer is not aligned to its element type");
    if (const char* e = bad_heads(q, q_token_stride, q_head_stride, q_tokens, heads, width, 2)) return invalid(e);
    if (const char* e = bad_out(out, out_token_stride, out_head_stride, q_tokens, heads, width, 2))
        return invalid(e);
    if (out == q) return invalid("out may not be q");
    if (k_tokens)
        for (const void* t : {k, v})
            if (const char* e = bad_heads(t, k_token_stride, k_head_stride, k_tokens, kv_heads, width, 2))
                return invalid(e);
    // (one row or head has no stride to align)
    const int64_t qt = q_tokens > 1 ? q_token_stride : heads * 128, qh = heads > 1 ? q_head_stride : 128;
    const int64_t kt = k_tokens > 1 ? k_token_stride : kv_heads * 128, kh = kv_heads > 1 ? k_head_stride : 128;
    if (!words(q, qt, qh, 2) || !words(k, kt, kh, 2) || !words(v, kt, kh, 2))
        return invalid("q, k and v must be 16-byte aligned, and their strides multiples of 16 bytes");
    if (q_tokens / 128 + documents > kMaxDim / heads) {
        set_last_error("more tiles than the kernels count");
        return CONV_ERR_UNSUPPORTED;
    }
    LaunchLimits lim;
    int rc = launch_limits(&lim);
    if (rc) return rc;
    PackedParams p{};
    p.q_offsets = q_offsets;
    p.k_offsets = k_offsets;
    p.prefix = prefix;
    p.slopes = slopes;
    p.out = static_cast<unsigned char*>(out);
    p.q = static_cast<const unsigned char*>(q);
    p.k = static_cast<const unsigned char*>(k);
    p.v = static_cast<const unsigned char*>(v);
    p.q_tok = q_token_stride;
    p.q_head = q_head_stride;
    p.k_tok = k_token_stride;
    p.k_head = k_head_stride;
    p.out_tok = out_token_stride;
    p.out_head = out_head_stride;
    p.q_tokens = q_tokens;
    p.k_tokens = k_tokens;
    p.documents = static_cast<int>(documents);
    p.heads = static_cast<int>(heads);
    p.group = static_cast<int>(heads / kv_heads);
    p.width = static_cast<int>(width);
    p.causal = causal != 0;
    p.window = static_cast<int>(window > kMaxTokens ? 0 : window);
    p.scale = scale;
    p.cap = cap;
    p.inv_cap = cap > 0.0f ? 1.0f / cap : 0.0f;
    // the coefficients of the cap's polynomial go with scale (scale / cap)^2d, d = 0 to 4
    const double first = std::fabs(static_cast<double>(scale)), ratio = cap > 0.0f ? first / cap : 0.0;
    const double last = first * std::pow(ratio, 8);
    p.per_cap = std::min(first, last) > 1e-30 && std::max(first, last) < 1e30 ? static_cast<float>(ratio) : INFINITY;
    p.out_aligned = !words(out, out_token_stride, out_head_stride, 2) ? 0
                    : aligned_to(out, 32) && out_token_stride % 16 == 0 && out_head_stride % 16 == 0 ? 32 : 16;
    p.status = lim.status;
    p.wait_ns = lim.wait_ns;
    PackedMaps maps{};
    // (without a key nothing is loaded: the queries stand in for the maps' addresses)
    const bool none = k_tokens == 0;
    if ((rc = encode_heads(&maps.q, q, width, heads, q_tokens, qh * 2, qt * 2, 128))) return rc;
    if ((rc = none ? encode_heads(&maps.k, q, width, heads, q_tokens, qh * 2, qt * 2, 128)
                   : encode_heads(&maps.k, k, width, kv_heads, k_tokens, kh * 2, kt * 2, 128)))
        return rc;
    if ((rc = none ? encode_heads(&maps.v, q, width, heads, q_tokens, qh * 2, qt * 2, 128)
                   : encode_heads(&maps.v, v, width, kv_heads, k_tokens, kh * 2, kt * 2, 128)))
        return rc;
    return launched(launch_packed(maps, p, dtype, lim.num_sms, stream), "packed_attention_fwd launch");
}

}  // extern "C"
