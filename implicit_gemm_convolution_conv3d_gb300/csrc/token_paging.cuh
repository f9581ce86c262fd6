// token_paging.cuh -- device helpers of the paged key-value cache: which sequence a
// packed row belongs to, and where a token's row lies.
#pragma once
#include "token_attention_internal.h"

namespace c3d {

// The sequence of packed row `row`, by the whole warp: the last s in [0, n) with
// offsets[s] <= row (0 if there is none).  32 candidates a step.
__device__ __forceinline__ int find_sequence(const int32_t* offsets, int n, long long row) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;   // the answer is in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const bool le = at < hi && (lane == 0 || offsets[at] <= row);
        const int k = __popc(__ballot_sync(0xffffffffu, le)) - 1;   // offsets ascend
        lo += k * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Byte offset of token `pos`'s row in a page pool, and its scale's index; false
// for a token that the table does not hold or whose page is not in the pool.
__device__ __forceinline__ bool token_row(const PageMap& m, long long sequence, long long pos, int head,
                                          long long* row, long long* scale) {
    if (pos < 0 || pos >= m.capacity) return false;
    const uint32_t slot = fdiv(static_cast<uint32_t>(pos), m.by_page);
    const long long off = pos - static_cast<long long>(slot) * m.by_page.d;
    const long long page = m.table[sequence * m.table_stride + slot];
    if (page < 0 || page >= m.pages) return false;
    *row = page * m.page_stride + head * m.head_stride + off * m.row_stride;
    *scale = page * m.scale_page_stride + head * m.scale_head_stride + off;
    return true;
}

}  // namespace c3d
