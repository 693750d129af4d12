// attn_tokens.cuh — what the two tensor-core forms of the attention share (several new tokens of a sequence:
// attn_prefill.cu; nodes of a tree: attn_tree.cu).
#pragma once
#include <climits>

#include "kv_cache.cuh"
#include "tcgen05.cuh"

namespace syn {

constexpr float PRE_P_LOG2 = 6.0f;    // p is held as 2^6 p
constexpr float PRE_GROW_LOG2 = 8.0f; // the maximum's lag

template <int N>
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// the tiles that hold a key some row of the item sees: [a0, a1) of the prefix, [b0, b1)
struct Tiles {
    int a0, a1, b0, b1;
    __device__ __forceinline__ int count() const { return a1 - a0 + b1 - b0; }
    __device__ __forceinline__ int at(int i) const { return i < a1 - a0 ? a0 + i : b0 + (i - (a1 - a0)); }
};

// bits of the keys 32w .. 32w+31 of a tile that lie in [lo, hi)
__device__ __forceinline__ uint32_t span_bits(int lo, int hi, int w) {
    const int a = min(max(lo - 32 * w, 0), 32), b = min(max(hi - 32 * w, 0), 32);
    const uint32_t below_b = b == 32 ? 0xffffffffu : (1u << b) - 1u, below_a = a == 32 ? 0xffffffffu : (1u << a) - 1u;
    return below_b & ~below_a;
}

// A Q8_0 block's scale, twice, for its expansion to fp16.  From 512 on a block may hold values that fp16 does not:
// it is expanded to NaN, so that the rows that see it are computed again from the cache itself.  (An infinite
// key alone would not show: a score of -inf has no weight.)
__device__ __forceinline__ __half2 expand_scale(uint32_t bits) {
    uint32_t db = __byte_perm((bits & 0x7FFFu) < 0x6000u ? bits : 0x7FFFu, 0, 0x1010);
    return *reinterpret_cast<__half2*>(&db);
}

// (starts that run backwards or past the call's tokens count as none)
__device__ __forceinline__ int new_tokens(const int32_t* starts, int s, int n_tok) {
    const int a = starts[s], b = starts[s + 1];
    return a < 0 || b > n_tok ? 0 : max(b - a, 0);
}

// 8 values of the user's cache from value `at` of a tile on.
template <bool Q8>
__device__ __forceinline__ void cached8(const uint8_t* tile, int64_t scales, int64_t at, float (&x)[8]) {
    if (!Q8) {
        const uint4 w = *reinterpret_cast<const uint4*>(tile + 2 * at);
        const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
            x[2 * i] = y.x;
            x[2 * i + 1] = y.y;
        }
    } else {
        const uint2 w = *reinterpret_cast<const uint2*>(tile + at);
        const float d = h2f_bits(*reinterpret_cast<const uint16_t*>(tile + scales + 2 * (at >> 5)));
#pragma unroll
        for (int i = 0; i < 4; i++) {
            x[i] = d * (float)(int8_t)(w.x >> (8 * i));
            x[4 + i] = d * (float)(int8_t)(w.y >> (8 * i));
        }
    }
}

}  // namespace syn
