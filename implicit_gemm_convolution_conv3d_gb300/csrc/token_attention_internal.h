// token_attention_internal.h -- parameter blocks and launch entry points shared by
// token_attention_api.cu and the kernels of rotary positions, the key-value cache and
// attention.  Not part of the public ABI.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "token_attention.h"

namespace c3d {

struct RotaryParams {
    const void* x;
    void* out;
    const void* positions;
    long long x_tok, x_head, out_tok, out_head;
    long long tokens;
    int heads, width, axes, pairs;
    int pos64, interleaved, inverse, copy_rest;
    // turns of a pair for each unit of its position, as a fraction of 2^64: the
    // product with a whole position, modulo 2^64, is the angle's fraction of a turn
    unsigned long long turns[ROTARY_MAX_PAIRS];
    unsigned char axis[ROTARY_MAX_PAIRS];
};
// align: bytes (up to 16) that all rows are aligned to
cudaError_t launch_rotary(const RotaryParams& p, int dtype, int align, cudaStream_t stream);

// where a sequence's tokens lie
struct PageMap {
    const int32_t* table;
    long long table_stride;   // entries between sequences
    long long capacity;       // tokens a row of the table can hold
    long long pages;
    long long page_stride, head_stride, row_stride;   // bytes
    long long scale_page_stride, scale_head_stride;   // elements
    FastDiv by_page;
};

struct CacheParams {
    unsigned char* k;
    unsigned char* v;
    float* k_scale;   // NULL: unquantised
    float* v_scale;
    PageMap map;
    unsigned char* rows_k;
    unsigned char* rows_v;
    long long tok_stride, head_stride;   // of the rows, elements
    const int32_t* offsets;   // NULL: row s is sequence s (write only)
    const int32_t* starts;    // NULL: 0 (read only)
    long long tokens;
    int sequences, heads, width;
    int aligned;   // the rows take 16-byte accesses
    int parts;     // groups of lanes that share a token's rows (filled at launch)
    FastDiv by_parts, by_runs;
};
cudaError_t launch_cache_write(const CacheParams& p, int row_dtype, int cache_dtype,
                               cudaStream_t stream);
cudaError_t launch_cache_read(const CacheParams& p, int row_dtype, int cache_dtype,
                              cudaStream_t stream);

struct PagedParams {
    const unsigned char* q;
    unsigned char* out;
    const unsigned char* k;
    const unsigned char* v;
    const float* k_scale;
    const float* v_scale;
    PageMap map;
    const int32_t* lengths;
    const int32_t* prefix;
    const float* slopes;
    long long q_seq, q_head, out_seq, out_head;   // elements
    float scale, cap, inv_cap;   // inv_cap: 1 / cap
    int window;            // 0: none
    int sequences, kv_heads, group, width;
    int blocks;            // groups of query heads that share a pass over a key head
    int grid, num_sms;     // grid: CTAs at most
    bool whole;            // key heads are not split
    float* partial;        // workspace: see token_paged_attention.cu
    int4* jobs;
    int rows_box;          // tokens of a TMA load: 32 (rows up to 128 bytes), 16, 8, or 0 (none: word by word)
    int* status;           // device status word and the bound on every wait
    unsigned long long wait_ns;
};
struct PagedMaps {
    CUtensorMap k, v;
};
// Whether every key head has a CTA of its own, which needs no workspace
bool paged_whole(long long sequences, long long kv_heads, long long group, int width,
                 long long capacity, int num_sms);
// CTAs of the grid otherwise
int paged_grid(long long sequences, long long kv_heads, long long group, int width,
               long long capacity, int num_sms);
size_t paged_workspace(int grid, int width);
cudaError_t launch_paged(const PagedMaps& maps, const PagedParams& p, int q_dtype, int cache_dtype,
                         cudaStream_t stream);

struct PackedParams {
    const int32_t* q_offsets;
    const int32_t* k_offsets;
    const int32_t* prefix;
    const float* slopes;
    unsigned char* out;
    const unsigned char* q;
    const unsigned char* k;
    const unsigned char* v;
    long long q_tok, q_head, k_tok, k_head, out_tok, out_head;   // elements
    long long q_tokens, k_tokens;
    int documents, heads, group, width;   // group: query heads of a key head
    int causal, window;
    float scale, cap, inv_cap;   // inv_cap: 1 / cap
    float per_cap;               // |scale| / cap, or infinite where the cap's polynomial cannot hold its powers
    int out_aligned;   // bytes that rows of out are aligned to: 32, 16 or fewer (0)
    int* status;
    unsigned long long wait_ns;
};
struct PackedMaps {
    CUtensorMap q, k, v;
};
cudaError_t launch_packed(const PackedMaps& maps, const PackedParams& p, int dtype, int num_sms,
                          cudaStream_t stream);

}  // namespace c3d
