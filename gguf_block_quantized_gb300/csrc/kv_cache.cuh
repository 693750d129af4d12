// kv_cache.cuh — the paged key-value cache as the kernels see it, and what its readers share.
//
// A pool (one for keys, one for values) holds n_pages pages, page_stride bytes apart; a page
// holds n_kv tiles, one per kv head; a tile holds page_size = 2^page_shift rows of dim values:
//   F16   [page_size][dim] halves
//   Q8_0  [page_size][dim] int8 codes, then [page_size][dim/32] fp16 scales
// The Q8_0 values are those of the block format (d = fp16(amax/127), value = d * code); codes
// and scales are kept apart because a 34-byte block row starts on no 16-byte boundary, while
// both planes of a tile do: page_size >= 8 and dim % 32 == 0 make page_size*dim and
// page_size*dim/16 multiples of 16.
#pragma once
#include <climits>

#include "common.cuh"

namespace syn {

struct KvCache {
    uint8_t* k;
    uint8_t* v;
    int64_t n_pages;
    int64_t page_stride;  // bytes
    int64_t tile;         // bytes of one head's rows of a page
    int n_kv, dim, page_shift, q8;
};

// The rows of a sequence: a length is cut to what its page table holds (and to what leaves room in 32
// bits for a row number rounded up to a tile); every kernel that reads lens[] goes by this.
__device__ __forceinline__ int held_rows(int len, int64_t max_pages, int page_shift) {
    return (int)min((int64_t)max(len, 0), min(max_pages << page_shift, (int64_t)INT_MAX - 1024));
}

// The keys a query at position pos of a sequence of len rows sees:
//   first <= j < len and (j < pre or (low <= j <= pos)),  low = the window's first key.
// (j < pre: the bidirectional prefix, which the window does not cut.)
struct Visible {
    int first, pre, low, end;  // end: one past the last key of the causal part
    __device__ __forceinline__ bool operator()(int j) const {
        return j >= first && (j < pre || (j >= low && j < end));
    }
    __device__ __forceinline__ bool any(int a, int b) const {  // of the keys a .. b - 1
        return max(a, first) < min(b, pre) || max(a, low) < min(b, end);
    }
};

__device__ __forceinline__ Visible visible_of(int len, int pos, int first, int prefix, int window) {
    Visible w;
    w.first = max(first, 0);
    w.pre = min(prefix, len);
    w.end = min(pos + 1, len);
    w.low = w.first;
    if (window > 0) w.low = max(w.low, pos >= window ? pos - window + 1 : 0);
    return w;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace syn
