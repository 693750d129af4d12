// attn_decode.cu — attention of one new token of each sequence over the paged cache.
//
//   s_j = cap*tanh(scale*q.k_j/cap) - slope*(p - j),  out = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m)
// with x = s*log2(e) and m the running maximum: one pass over the cached rows; a part of the
// rows leaves (m, l = sum, o = weighted sum) per head, and parts join by
//   m = max m_i, l = sum l_i 2^(m_i - m), o = sum o_i 2^(m_i - m).
//
// Bound: HBM; every cached row is read once for all the query heads that share it.
//   - Warps work alone: each copies chunks of 16 rows of K and V into a ring of its own in shared
//     memory (cp.async) and multiplies them with mma.sync m16n8k16, the 16 cached rows as the A
//     operand and up to 8 query heads as the columns: S^T = K Q^T, then O^T += V^T P^T.  A
//     chunk of 128-wide rows is about 430 instructions (F16) or 710 (Q8_0) of a warp, where its bytes
//     take 1400 or 750 issue slots of an SM to arrive.  Q8_0 fills 60 % of the slots, its busiest pipe (integer
//     and conversion) 40 %: four warps a scheduler do not hide what their instructions wait for each other.
//   - p is split into two fp16 numbers (head and tail, 22 bits) and each chunk's product starts
//     from zero and is added to the fp32 sums by fma, because the tensor pipe's own additions
//     truncate.  Scores likewise come from short chains.  So the result is as exact as fp32
//     arithmetic allows, which fp32 outputs show.
//   - Q8_0 codes go into the products as they are, without their scales: exact in fp16.  A key's
//     scale multiplies its block's 32-value sum, a value's scale goes into p, head and tail, relative to the
//     power of two of its row's largest, which goes into the running maximum: what is kept of a row goes by what
//     it adds to the output (a scale relative to the largest so far: 3 % less time, and a row of large
//     values with no weight cost the others up to 1 % of their own).  A code's 128, added to make its byte an
//     fp16 number, is subtracted ahead of the product: left in, and taken off the sum, it costs the small
//     codes beside an outlier channel their last bits in the tensor pipe's truncating sums.
//   - Work is cut by length, not by sequence: the steps (4 chunks, one per warp) of all
//     (sequence, kv head) items, and some for each item's start and end, are dealt to the CTAs in
//     equal contiguous ranges, found on the device from the lengths (a captured graph keeps working
//     as they grow).  A CTA whose range
//     covers an item writes the output; else it leaves a partial in the workspace, and the CTA
//     that finishes an item last (a counter) joins the partials in order.  No CTA waits.
//
// Measured on GB300, 32 / 8 heads of 128 (share of a copy's rate): 300 sequences of 2500 rows, F16 98 %,
// Q8_0 77 %; 48 sequences of 100 to 4000, F16 44.5 us, 71 %; 128 of 500 to 8191, Q8_0, capped 175 us, 65 %;
// one of 130001, F16 92 us, 85 %; one of 77 (heads of 64) 5.3 us.
#include <algorithm>

#include "kernels.h"
#include "kv_cache.cuh"

namespace syn {

constexpr int DEC_WARPS = 4;
constexpr int DEC_SLOTS = 3;    // of a warp's ring: the keys or the values of a chunk each
// What an item's start and end cost, in steps.  Measured (us, 0 / 2 / 8): 58 sequences of 40 to 14210 rows, 32 / 8
// heads of 128, Q8_0 117 / 72 / 80, F16 140 / 101 / 100; 58 of 2500 rows each, Q8_0 75 / 73 / 78.
constexpr int DEC_ITEM = 2;
// A part's share of the join, per value, against a step (blocks of sqrt(steps * values * this)).
// Measured (us, 0 / 2e-4 / 8e-4): one sequence of 32768 rows, F16, 24 / 1 heads of 128 72 / 40 / 49; one of
// 40642, Q8_0, 16 / 2 heads of 64 30 / 27 / 31.
constexpr float DEC_JOIN = 2e-4f;
constexpr int DEC_MAX_SEQ = 1024;  // sequences of one launch (their step counts are in shared memory)
// p is held in fp16 as 2^14 p, so that small p stay normal numbers; Q8_0 as 2^13 p: times a relative scale below 4
template <bool Q8>
constexpr float DEC_P_LOG2 = Q8 ? 13.0f : 14.0f;

struct DecodeParams {
    KvCache c;
    const __half* q;
    int64_t q_stride, out_stride;
    void* out;
    const int32_t* pages;
    int64_t max_pages;
    const int32_t* lens;
    const float* slopes;
    const int32_t* prefix;
    const int32_t* first;
    float* part;  // per CTA two partial slots
    int* count;   // per item, zero between calls
    int* err;
    float scale, cap, inv_cap;
    uint32_t stride16;  // page_stride / 16
    int n_seq, g, n_hg, window, out_f16, whole;
};

// ---- primitives ------------------------------------------------------------------------

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_zero(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }

// (x, y) as fp16 heads and tails: x = hi + lo to 22 bits
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = h2u(h);
    lo = h2u(__floats2half2_rn(x - f.x, y - f.y));
}

// tanh to about 2^-22 of itself without branches: (e - 1)/(e + 1) with e = 2^(2|y| log2 e), and below
// 0.55, where e - 1 would cancel, the fifth convergent of Lambert's continued fraction
__device__ __forceinline__ float tanh_rel(float y) {
    const float a = fminf(fabsf(y), 10.0f), u = a * a;
    const bool small = a < 0.55f;
    const float e = ex2(2.8853900817779268f * a);
    const float num = small ? a * fmaf(u, u + 105.0f, 945.0f) : e - 1.0f;
    const float den = small ? fmaf(u, fmaf(u, 15.0f, 420.0f), 945.0f) : e + 1.0f;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(den));
    return copysignf(y == y ? num * r : y, y);
}

// ---- what a sequence needs ---------------------------------------------------------------

// The chunks (16 rows from a multiple of 16) that hold a visible key: [a0, a1) of the prefix,
// [b0, b1) of the rest.
struct Chunks {
    int a0, a1, b0, b1;
    __device__ __forceinline__ int count() const { return a1 - a0 + b1 - b0; }
    __device__ __forceinline__ int at(int i) const { return i < a1 - a0 ? a0 + i : b0 + (i - (a1 - a0)); }
};

__device__ __forceinline__ int seq_len(const DecodeParams& p, int s) {
    return held_rows(p.lens[s], p.max_pages, p.c.page_shift);
}

__device__ __forceinline__ Visible seq_visible(const DecodeParams& p, int s, int len) {
    return visible_of(len, len - 1, p.first ? p.first[s] : 0, p.prefix ? p.prefix[s] : 0, p.window);
}

__device__ __forceinline__ Chunks seq_chunks(const Visible& w) {
    Chunks c;
    const int pre_end = min(w.pre, w.low);
    c.a0 = w.first >> 4;
    c.a1 = pre_end > w.first ? (pre_end + 15) >> 4 : c.a0;
    c.b0 = w.low >> 4;
    c.b1 = w.end > w.low ? (w.end + 15) >> 4 : c.b0;
    if (c.a1 > c.b0) c.a1 = max(c.a0, c.b0);
    return c;
}

template <int D, bool Q8>
struct DecLayout {
    // row pitch in shared memory: the 8 rows of one 16-byte piece that ldmatrix reads lie on different
    // banks.  F16: pieces swizzled by the row; Q8_0: an odd number of pieces
    static constexpr int PITCH = Q8 ? D + 16 : 2 * D;
    static constexpr int SCALES = 16 * PITCH;  // Q8_0: scales [16][dim/32], behind the rows
    static constexpr int SLOT = SCALES + (Q8 ? D : 0);
    // (the merge of the warps' parts, up to 16 heads of D fp32 values each, reuses a warp's ring)
    static constexpr int MERGE = (D <= 128 ? 16 : 8) * D * 4;
    static constexpr int WARP = DEC_SLOTS * SLOT > MERGE ? DEC_SLOTS * SLOT : MERGE;
    static constexpr int RING = DEC_WARPS * WARP;
};

// One CTA joins the partials of CTAs i0 .. i1 of an item and writes its output (at `at`).  The
// weights 2^(m_i - m) of up to JOIN_TILE parts are laid into shared memory, then every thread adds
// up 4 neighbouring values, its loads independent of each other; where the item has few values the
// threads share its parts out.
constexpr int JOIN_TILE = 64;
template <int D, int H>
__device__ __noinline__ void join_parts(const DecodeParams& p, int i0, int i1, int heads, int dim, uint8_t* smem, float* sm_m,
                                        float* sm_l, int64_t at) {
    constexpr int T = 32 * DEC_WARPS;
    float* w = reinterpret_cast<float*>(smem);                      // [JOIN_TILE][H]
    float4* sums = reinterpret_cast<float4*>(w + JOIN_TILE * H);    // [T]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = i1 - i0 + 1, pitch = H * (D + 2);
    // the first part is in the slot of a segment that begins its item
    auto part_of = [&](int c) { return p.part + (2 * (int64_t)(i0 + c) + (c == 0)) * pitch; };
    for (int hd = warp; hd < heads; hd += DEC_WARPS) {
        float mx = -INFINITY, sum = 0.0f;
        for (int c = lane; c < n; c += 32) {
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(part_of(c) + H * D) + hd);
            const float nm = fmaxf(mx, ml.x), ms = nm == -INFINITY ? 0.0f : nm;
            sum = sum * ex2(mx - ms) + ml.y * ex2(ml.x - ms);
            mx = nm;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, mx, off), os = __shfl_xor_sync(0xffffffffu, sum, off);
            const float nm = fmaxf(mx, om), ms = nm == -INFINITY ? 0.0f : nm;
            sum = sum * ex2(mx - ms) + os * ex2(om - ms);
            mx = nm;
        }
        if (lane == 0) {
            sm_m[hd] = mx == -INFINITY ? 0.0f : mx;
            sm_l[hd] = sum;
        }
    }
    __syncthreads();
    const int nv = heads * dim >> 2, dv = dim >> 2;  // 4-value pieces of the item, of a head
    const int shares = max(1, T / nv), share = nv < T ? tid / nv : 0;
    for (int v0 = 0; v0 < nv; v0 += T) {
        const int v = nv < T ? tid - share * nv : v0 + tid;
        const bool mine = v < nv && share < shares;
        const int hd = mine ? v / dv : 0, e = (v - hd * dv) << 2;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int c0 = 0; c0 < n; c0 += JOIN_TILE) {
            const int m = min(JOIN_TILE, n - c0);
            __syncthreads();
            for (int i = tid; i < m * heads; i += T) {
                const int c = i / heads, x = i - c * heads;
                w[c * H + x] = ex2(__ldcg(part_of(c0 + c) + H * D + 2 * x) - sm_m[x]);
            }
            __syncthreads();
            if (mine) {
                for (int c = share; c < m; c += 8 * shares) {  // (the last batch repeats its last load)
                    float4 o[8];
#pragma unroll
                    for (int x = 0; x < 8; x++) {
                        const int cx = c + x * shares < m ? c + x * shares : c;
                        o[x] = __ldcg(reinterpret_cast<const float4*>(part_of(c0 + cx) + hd * D + e));
                    }
#pragma unroll
                    for (int x = 0; x < 8; x++) {
                        const float f = c + x * shares < m ? w[(c + x * shares) * H + hd] : 0.0f;
                        acc.x = fmaf(o[x].x, f, acc.x);
                        acc.y = fmaf(o[x].y, f, acc.y);
                        acc.z = fmaf(o[x].z, f, acc.z);
                        acc.w = fmaf(o[x].w, f, acc.w);
                    }
                }
            }
        }
        if (shares > 1) {
            __syncthreads();
            sums[tid] = acc;
            __syncthreads();
            if (share == 0)
                for (int x = 1; x < shares; x++) {
                    const float4 o = sums[x * nv + v];
                    acc.x += o.x;
                    acc.y += o.y;
                    acc.z += o.z;
                    acc.w += o.w;
                }
        }
        if (mine && share == 0) {
            const float sum = sm_l[hd];
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            const int64_t a = at + (int64_t)hd * dim + e;
            if (p.out_f16) {
                const __half2 x = __floats2half2_rn(acc.x * inv, acc.y * inv), y = __floats2half2_rn(acc.z * inv, acc.w * inv);
                *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + a) = make_uint2(h2u(x), h2u(y));
            } else {
                *reinterpret_cast<float4*>(static_cast<float*>(p.out) + a) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            }
        }
    }
}

// Q8_0: the scales of one row of a chunk (all of a row's at once where the row is as wide as the
// kernel's, so that they lie on an aligned boundary)
template <int D, bool EXACT>
__device__ __forceinline__ void row_scales(const uint8_t* base, int r, int dim, __half (&d)[D / 32]) {
    if (EXACT) {
        const uint8_t* q = base + r * (D / 16);
        if (D == 64) *reinterpret_cast<uint32_t*>(d) = *reinterpret_cast<const uint32_t*>(q);
        else if (D == 128) *reinterpret_cast<uint2*>(d) = *reinterpret_cast<const uint2*>(q);
        else *reinterpret_cast<uint4*>(d) = *reinterpret_cast<const uint4*>(q);
    } else {
#pragma unroll
        for (int b = 0; b < D / 32; b++) d[b] = b * 32 < dim ? reinterpret_cast<const __half*>(base)[r * (dim >> 5) + b] : __ushort_as_half(0);
    }
}

// CTAs per SM that the ring leaves room for (so many registers are a thread's)
template <int D, bool Q8>
constexpr int DEC_RESIDENT = D == 64 ? 5 : D == 128 ? 4 : 2;

// D: the row width of the kernel's layout; EXACT: rows are that wide (else narrower: dim < D)
template <int D, int NT, bool Q8, bool EXACT>
__global__ void __launch_bounds__(32 * DEC_WARPS, NT == 1 ? DEC_RESIDENT<D, Q8> : 1) k_attn_decode(const DecodeParams p) {
    using L = DecLayout<D, Q8>;
    constexpr int KSTEPS = D / 16;
    constexpr int H = 8 * NT;  // query heads of an item
    static_assert(L::WARP >= H * D * 4 && L::RING >= 4 * (JOIN_TILE * H + 4 * 32 * DEC_WARPS), "merge and join reuse the ring");
    extern __shared__ __align__(128) uint8_t smem[];
    float* sm_m = reinterpret_cast<float*>(smem + L::RING);  // [DEC_WARPS][H]
    float* sm_l = sm_m + DEC_WARPS * H;
    int* flags = reinterpret_cast<int*>(sm_l + DEC_WARPS * H);  // [0] scan carry, [1..4] warp sums, [5] last, [6] most steps
    unsigned long long* all_steps = reinterpret_cast<unsigned long long*>(flags + 8);
    int* pre = flags + 10;                                        // [n_seq + 1] blocks before each sequence, of one item

    // (the shuffle tells the compiler that the warp's index is the same for its lanes)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int r8 = lane >> 2, c4 = lane & 3;
    const int dim = EXACT ? D : p.c.dim;
    const int n_item_h = p.c.n_kv * p.n_hg;  // items of a sequence

    // pre[s + 1] = the sum of x up to sequence s (128 sequences at a time, flags[0] carries)
    auto scan = [&](int s, int x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) flags[1 + warp] = x;
        __syncthreads();
        int before = flags[0];
        for (int w = 0; w < warp; w++) before += flags[1 + w];
        if (s < p.n_seq) pre[s + 1] = before + x;
        __syncthreads();
        if (tid == 32 * DEC_WARPS - 1) flags[0] = before + x;
        __syncthreads();
    };
    griddep_release();
    griddep_wait();
    // the steps of every sequence: their sum and the most
    auto chunks_of = [&](int s) { return seq_chunks(seq_visible(p, s, seq_len(p, s))).count(); };
    if (tid == 0) flags[0] = 0, flags[6] = 0, *all_steps = 0, pre[0] = 0;
    __syncthreads();
    for (int base = 32 * warp; base < p.n_seq; base += 32 * DEC_WARPS) {
        const unsigned n = base + lane < p.n_seq ? (unsigned)(chunks_of(base + lane) + DEC_WARPS - 1) / DEC_WARPS : 0u;
        const unsigned sum = __reduce_add_sync(0xffffffffu, n), most = __reduce_max_sync(0xffffffffu, n);
        if (lane == 0) {
            atomicAdd(all_steps, (unsigned long long)sum);
            atomicMax(&flags[6], (int)most);
        }
    }
    __syncthreads();
    const int64_t steps = (int64_t)*all_steps;
    // Little work is dealt in blocks of several steps, one a CTA: 3, as a step's loads are in flight
    // together with the next ones', and more where the longest item would have so many parts that their
    // join (heads * dim values a part, by one CTA) took longer than the steps.
    // Items of 6 steps or fewer (8 where the join has many values) stay whole: 1 sequence of 400 rows in 3
    // parts / whole (us), F16 32 / 8 heads of 64 9.8 / 8.2, 16 / 1 of 128 15.4 / 11.6; of 709, 10.4 / 12.2 and 15.8 / 17.0.
    const int values = min(H, p.g) * dim, most = flags[6];
    const int few = max(most <= (values < 1024 ? 6 : 8) ? most : 3, (int)ceilf(sqrtf((float)most * (float)values * DEC_JOIN)));
    int block = !p.whole && steps * n_item_h <= (int64_t)few * gridDim.x ? few : 1;
    if (steps >> 30) block = max(block, (int)(steps >> 30) + 1);  // (the running sum has 32 bits)
    // Else an item counts DEC_ITEM steps more than it has: what its start and its end cost.
    const int extra = block == 1 && !p.whole ? DEC_ITEM : 0;
    for (int base = 0; base < p.n_seq; base += 32 * DEC_WARPS) {
        const int s = base + tid;
        int x = 0;
        if (s < p.n_seq) x = (chunks_of(s) + DEC_WARPS * block - 1) / (DEC_WARPS * block);
        scan(s, x > 0 ? x + extra : 0);
    }
    for (int s = blockIdx.x; s < p.n_seq; s += gridDim.x) {  // no key to see: zeros
        if (pre[s + 1] > pre[s]) continue;
        const int64_t row = s * p.out_stride;
        for (int i = tid; i < p.c.n_kv * p.g * dim >> 2; i += 32 * DEC_WARPS) {
            if (p.out_f16) *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + row + 4 * i) = make_uint2(0, 0);
            else *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row + 4 * i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
    }
    const int64_t total = (int64_t)pre[p.n_seq] * n_item_h;
    if (total == 0) return;
    const int64_t ctas = min((int64_t)gridDim.x, total);
    if (!p.whole && blockIdx.x >= ctas) return;
    // this CTA's range of blocks; in `whole` mode its items are blockIdx.x, + gridDim.x, ...
    int64_t at = blockIdx.x * total / ctas, stop = (blockIdx.x + 1) * total / ctas;
    int item_w = blockIdx.x;

    constexpr float LOG2E = 1.4426950408889634f;
    const float scale_log2 = p.scale * LOG2E;
    uint8_t* ring = smem + warp * L::WARP;
    const uint32_t ring_s = smem_u32(ring);
    const int row_pieces = Q8 ? dim >> 4 : dim >> 3;  // 16-byte pieces of a row
    // 16 rows lie one after the other in a page (of 16 rows or more), so lane l copies their
    // 16-byte pieces l, l + 32, ...: the places in a slot, place(i) of piece i of this lane.  Rows
    // as wide as the kernel's: with the swizzle they repeat every 8 rows, without it they are linear.
    constexpr int N_COPY = Q8 ? D / 32 : D / 16;
    constexpr int N_TO = !EXACT ? N_COPY : Q8 ? 1 : D / 32;
    uint32_t to[N_TO];
#pragma unroll
    for (int i = 0; i < N_TO; i++) {
        const int idx = i * 32 + lane, r = idx / row_pieces, j = idx - r * row_pieces;
        to[i] = r * L::PITCH + (Q8 ? 16 * j : ((j ^ (r & 7)) << 4));
    }
    auto place = [&](int i) -> uint32_t {
        if (!EXACT) return to[i % N_TO];
        return Q8 ? to[0] + i * (512 / D) * L::PITCH : to[i % N_TO] + (i / N_TO) * 16 * D;
    };
    // Where ldmatrix finds 16-byte piece 2i (+ 8 for the next four) of this lane's row.  Keys: matrices of
    // rows 0-7 and 8-15 of one piece, then of the next; values, transposed, F16 the same, Q8_0 rows
    // 0-7 of two pieces, then rows 8-15.
    uint32_t at_k[Q8 ? 1 : 4], at_v[Q8 ? 1 : 4];
    {
        const int rk = (lane & 7) + ((lane >> 3) & 1) * 8, ck = lane >> 4;
        const int rv = (lane & 7) + (lane >> 4) * 8, cv = (lane >> 3) & 1;
        if (Q8) {
            at_k[0] = rk * L::PITCH + 16 * ck;
            at_v[0] = rv * L::PITCH + 16 * cv;
        } else {
#pragma unroll
            for (int i = 0; i < (Q8 ? 1 : 4); i++) {
                at_k[i] = rk * L::PITCH + (((2 * i + ck) ^ (rk & 7)) << 4);
                at_v[i] = rv * L::PITCH + (((2 * i + cv) ^ (rv & 7)) << 4);
            }
        }
    }
    [[maybe_unused]] const int64_t pool_end = p.c.tile + (p.c.n_pages - 1) * p.c.page_stride;  // from a head's tile of page 0
    const int64_t plane = (int64_t)dim << p.c.page_shift;  // Q8_0: where a tile's scales begin
    const int page_mask = (1 << p.c.page_shift) - 1;
    [[maybe_unused]] const __half2 k1152 = __float2half2_rn(1152.0f);  // a byte u under 0x64 is the half 1024 + u

    while (true) {
        // the next segment: blocks [st0, st1) of item (s, kv head h, head group hg)
        int s, hh, st0, st1, n_blocks;
        if (p.whole) {
            if (item_w >= p.n_seq * n_item_h) break;
            s = item_w / n_item_h;
            hh = item_w - s * n_item_h;
            n_blocks = pre[s + 1] - pre[s];
            item_w += gridDim.x;
            if (n_blocks == 0) continue;
            st0 = 0;
            st1 = n_blocks;
        } else {
            if (at >= stop) break;
            int lo = 0, hi = p.n_seq - 1;  // the sequence whose blocks hold `at`
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if ((int64_t)pre[mid + 1] * n_item_h > at) hi = mid;
                else lo = mid + 1;
            }
            s = lo;
            const int n_all = pre[s + 1] - pre[s];
            n_blocks = n_all - extra;
            const int64_t rel = at - (int64_t)pre[s] * n_item_h;
            hh = (int)(rel / n_all);
            const int b0 = (int)(rel - (int64_t)hh * n_all), b1 = (int)min((int64_t)n_all, b0 + (stop - at));
            at += b1 - b0;
            st0 = max(b0 - extra, 0);
            st1 = max(b1 - extra, 0);
            if (st0 == st1) continue;
        }
        const int h = hh / p.n_hg, hg = hh - h * p.n_hg;
        const int len = seq_len(p, s);
        const Visible vis = seq_visible(p, s, len);
        const Chunks ch = seq_chunks(vis);
        const int n_chunks = ch.count();
        const int head0 = hg * H;                 // first query head of the group
        const int heads = min(H, p.g - head0);    // how many there are
        const uint8_t* kbase = p.c.k + (int64_t)h * p.c.tile;
        const uint8_t* vbase = p.c.v + (int64_t)h * p.c.tile;
        const int32_t* table = p.pages + (int64_t)s * p.max_pages;

        // q as the B operand: column (head) lane/4, k rows 2*(lane%4).. (F16), or the order in
        // which the Q8_0 codes are unpacked
        uint32_t qf[KSTEPS][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            const int hd = nt * 8 + r8;
            const __half* qr = p.q + s * p.q_stride + (int64_t)(h * p.g + head0 + hd) * dim;
#pragma unroll
            for (int ks = 0; ks < KSTEPS; ks++) {
                qf[ks][nt][0] = qf[ks][nt][1] = 0;
                if (hd < heads && ks * 16 < dim) {
                    if (Q8) {
                        const uint2 w = *reinterpret_cast<const uint2*>(qr + 16 * ks + 4 * c4);
                        qf[ks][nt][0] = w.x;
                        qf[ks][nt][1] = w.y;
                    } else {
                        qf[ks][nt][0] = *reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * c4);
                        qf[ks][nt][1] = *reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * c4 + 8);
                    }
                }
            }
        }
        float slope[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int hd = nt * 8 + 2 * c4 + j;
                slope[nt][j] = p.slopes && hd < heads ? p.slopes[h * p.g + head0 + hd] : 0.0f;
            }

        float m[NT][2], l[NT][2];
        float o[KSTEPS][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
            for (int mt = 0; mt < KSTEPS; mt++) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.0f;
        }

        // this warp's chunks of the segment, every DEC_WARPS-th below `chunk_end`
        const int chunk0 = st0 * block * DEC_WARPS + warp, chunk_end = min(n_chunks, st1 * block * DEC_WARPS);
        // chunks whose 16 rows are all seen, in the causal part, and in one page
        const int full0 = (vis.low + 15) & ~15;
        const unsigned full_n = p.c.page_shift >= 4 ? (unsigned)max(0, (vis.end & ~15) - full0) : 0u;
        auto all_seen = [&](int row) { return (unsigned)(row - full0) < full_n; };
        bool bad_page = false;
        auto page_of = [&](int row) {  // -1: past the end, or outside the pool
            if (row >= len) return -1;
            const int id = table[row >> p.c.page_shift];
            const bool ok = (unsigned)id < (unsigned)p.c.n_pages;
            bad_page |= !ok;
            return ok ? id : -1;
        };
        // The next chunk whose keys are copied, and the pages of its rows 0-7 and 8-15, looked up one
        // chunk ahead; the chunk whose values are copied next (its keys are on their way).
        int k_next = chunk0, id_lo = -1, id_hi = -1;
        int v_row = -1, v_lo = -1, v_hi = -1;
        bool v_whole = false;
        int64_t v_off = 0;  // of the chunk's first row from a head's tile of page 0
        auto look_up = [&]() {
            if (k_next < chunk_end) {
                const int row = ch.at(k_next) << 4;
                // (a chunk holds a key that is seen; half of one, a page of its own, may not)
                if (p.c.page_shift >= 4) {
                    id_lo = id_hi = page_of(row);
                } else {
                    id_lo = vis.any(row, row + 8) ? page_of(row) : -1;
                    id_hi = vis.any(row + 8, row + 16) ? page_of(row + 8) : -1;
                }
            }
        };
        look_up();
        auto copy = [&](uint32_t dst, const uint8_t* base) {
            if (v_whole) {
                const uint8_t* src = base + v_off + 16 * lane;
                if (!SYN_IN_BOUNDS(v_off >= 0 && v_off + 256 * row_pieces <= pool_end)) return;
#pragma unroll
                for (int i = 0; i < N_COPY; i++) {
                    if (2 * i >= row_pieces) break;
                    cp16_all(dst + place(i), src + 512 * i);
                }
                // Q8_0: the rows' scales, dim/16 pieces (rows of 16 * row_pieces bytes, scales of row_pieces)
                if (Q8 && lane < row_pieces)
                    cp16_all(dst + L::SCALES + 16 * lane, src + plane - (v_row & page_mask) * (15 * row_pieces));
                return;
            }
            // a chunk at an end of what is seen, or pages of 8 rows: rows that the query does not
            // see are not read but zero (a masked V row may hold anything, and 0 * inf is not 0)
            const int64_t page = (int64_t)max(v_lo, 0) * p.c.page_stride, page_hi = (int64_t)max(v_hi, 0) * p.c.page_stride;
            const int cell = v_row & page_mask, cell_hi = (v_row + 8) & page_mask;
#pragma unroll
            for (int i = 0; i < N_COPY; i++) {
                if (2 * i >= row_pieces) break;
                const uint32_t at_dst = place(i);
                const int r = (int)at_dst / L::PITCH, j = i * 32 + lane - r * row_pieces;
                const bool upper = r >= 8, ok = (upper ? v_hi : v_lo) >= 0 && vis(v_row + r);
                const int64_t off = ok ? (upper ? page_hi + (int64_t)(cell_hi + r - 8) * (row_pieces * 16)
                                                : page + (int64_t)(cell + r) * (row_pieces * 16)) + 16 * j
                                       : 0;
                if (!SYN_IN_BOUNDS(off >= 0 && off + 16 <= pool_end)) continue;
                cp16(dst + at_dst, base + off, ok ? 16u : 0u);
            }
            if (Q8 && lane < row_pieces) {  // scales: rows 0-7 and 8-15 apart
                const bool upper = 2 * lane >= row_pieces, ok = (upper ? v_hi : v_lo) >= 0;
                const int64_t off = ok ? plane + (upper ? page_hi + (int64_t)cell_hi * row_pieces + 16 * (lane - row_pieces / 2)
                                                        : page + (int64_t)cell * row_pieces + 16 * lane)
                                       : 0;
                if (SYN_IN_BOUNDS(off >= 0 && off + 16 <= pool_end)) cp16(dst + L::SCALES + 16 * lane, base + off, ok ? 16u : 0u);
            }
        };
        auto issue_k = [&](int slot) {
            v_row = -1;
            if (k_next < chunk_end) {
                v_row = ch.at(k_next) << 4;
                v_lo = id_lo;
                v_hi = id_hi;
                v_whole = v_lo >= 0 && all_seen(v_row);
                v_off = (int64_t)((uint64_t)(uint32_t)v_lo * p.stride16 + (uint32_t)((v_row & page_mask) * row_pieces)) << 4;
                copy(ring_s + slot * L::SLOT, kbase);
                k_next += DEC_WARPS;
                look_up();
            }
            cp_commit();
        };
        auto issue_v = [&](int slot) {
            if (v_row >= 0) copy(ring_s + slot * L::SLOT, vbase);
            cp_commit();
        };
        issue_k(0);
        issue_v(1);
        issue_k(2);

        int sk = 0, sv = 1;  // slots of the chunk's keys and values
        for (int ci = chunk0; ci < chunk_end; ci += DEC_WARPS) {
            const int row0 = ch.at(ci) << 4;
            const bool full = all_seen(row0);
            const uint32_t kt = ring_s + sk * L::SLOT, vt = ring_s + sv * L::SLOT;
            const uint8_t *ktp = ring + sk * L::SLOT, *vtp = ring + sv * L::SLOT;
            cp_wait<2>();
            __syncwarp();

            // S^T = K Q^T, rows lane/4 and lane/4 + 8
            float sc[NT][4];
            if (Q8) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.0f;
                alignas(16) __half da[D / 32], db[D / 32];
                row_scales<D, EXACT>(ktp + L::SCALES, r8, dim, da);
                row_scales<D, EXACT>(ktp + L::SCALES, r8 + 8, dim, db);
#pragma unroll
                for (int b = 0; b < D / 32; b++) {
                    if (b * 32 >= dim) break;
                    // codes of a 32-value block: 8 per lane and row, exact in fp16
                    uint32_t a0[4], a1[4];
                    uint32_t w[4];
                    ldsm4(kt + at_k[0] + 32 * b, w);
#pragma unroll
                    for (int u = 0; u < 4; u++) w[u] ^= 0x80808080u;
#pragma unroll
                    for (int u = 0; u < 2; u++) {  // values 4c, 4c + 1 and 4c + 2, 4c + 3 of a 16-value half
                        a0[u] = h2u(__hsub2(u2h(__byte_perm(w[u], 0x64646464u, 0x4140)), k1152));
                        a0[2 + u] = h2u(__hsub2(u2h(__byte_perm(w[u], 0x64646464u, 0x4342)), k1152));
                        a1[u] = h2u(__hsub2(u2h(__byte_perm(w[2 + u], 0x64646464u, 0x4140)), k1152));
                        a1[2 + u] = h2u(__hsub2(u2h(__byte_perm(w[2 + u], 0x64646464u, 0x4342)), k1152));
                    }
                    const float fa = __half2float(da[b]), fb = __half2float(db[b]);
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) {
                        float c[4];
                        mma16816_zero(c, a0, qf[2 * b][nt][0], qf[2 * b][nt][1]);
                        mma16816(c, a1, qf[2 * b + 1][nt][0], qf[2 * b + 1][nt][1]);
                        sc[nt][0] = fmaf(c[0], fa, sc[nt][0]);
                        sc[nt][1] = fmaf(c[1], fa, sc[nt][1]);
                        sc[nt][2] = fmaf(c[2], fb, sc[nt][2]);
                        sc[nt][3] = fmaf(c[3], fb, sc[nt][3]);
                    }
                }
            } else {
                float s1[NT][4];
#pragma unroll
                for (int ks = 0; ks < KSTEPS; ks++) {
                    if (ks * 16 >= dim) break;
                    uint32_t a[4];
                    ldsm4(kt + at_k[ks & 3] + 128 * (ks >> 2), a);
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) {
                        if (ks < 2) mma16816_zero(ks & 1 ? s1[nt] : sc[nt], a, qf[ks][nt][0], qf[ks][nt][1]);
                        else mma16816(ks & 1 ? s1[nt] : sc[nt], a, qf[ks][nt][0], qf[ks][nt][1]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int j = 0; j < 4; j++) sc[nt][j] += s1[nt][j];
            }
            __syncwarp();  // every lane has read the keys before their slot is filled again
            issue_v(sk);

            // Q8_0: a row's weight in the product is p times its value scales.  The power of two of the row's
            // largest scale, 2^e, goes into the score, so that the running maximum m is that of what the rows add
            // to o, and a row of large values that has next to no weight takes no bits from the others; the scales
            // go in relative to it, d * 2^(1 - e) in [2, 4) for the largest (an fp16 product that is exact down to
            // 2^-15 of that).  The sum l takes p * 2^(1 - e): o and l are in the same units.
            alignas(16) __half dv[Q8 ? 4 : 1][D / 32];  // scales of rows 2c, 2c + 1, 2c + 8, 2c + 9
            uint32_t down[2];                           // 2^(1 - e) of rows 2c, 2c + 1 and of 2c + 8, 2c + 9
            float row_e[2] = {0.0f, 0.0f}, row_down[2] = {1.0f, 1.0f};  // of rows lane/4, lane/4 + 8
            if constexpr (Q8) {
                cp_wait<2>();  // (the values)
                __syncwarp();
#pragma unroll
                for (int u = 0; u < 2; u++) {
                    __half2 top[2];
#pragma unroll
                    for (int x = 0; x < 2; x++) {
                        const int r = 2 * c4 + x + 8 * u;
                        row_scales<D, EXACT>(vtp + L::SCALES, r, dim, dv[2 * u + x]);
                        if (!full && !vis(row0 + r)) {
#pragma unroll
                            for (int b = 0; b < D / 32; b++) dv[2 * u + x][b] = __ushort_as_half(0);
                        }
                        top[x] = __habs2(*reinterpret_cast<const __half2*>(&dv[2 * u + x][0]));
#pragma unroll
                        for (int b = 2; b < D / 32; b += 2) top[x] = __hmax2(top[x], __habs2(*reinterpret_cast<const __half2*>(&dv[2 * u + x][b])));
                    }
                    // the larger half of either row's, its power of two between 2^-14 and 2^15
                    const __half2 both = __hmax2(u2h(__byte_perm(h2u(top[0]), h2u(top[1]), 0x5410)), u2h(__byte_perm(h2u(top[0]), h2u(top[1]), 0x7632)));
                    const __half2 power = __hmin2(__hmax2(u2h(h2u(both) & 0x7C007C00u), u2h(0x04000400u)), u2h(0x78007800u));
                    down[u] = 0x7C007C00u - h2u(power);
                }
#pragma unroll
                for (int u = 0; u < 2; u++) {
                    const uint32_t w = __shfl_sync(0xffffffffu, down[u], r8 >> 1);  // (lane c holds rows 2c, 2c + 1)
                    row_down[u] = __half2float(__ushort_as_half((unsigned short)(w >> (16 * (r8 & 1)))));
                    row_e[u] = 8388736.0f - __uint_as_float((__float_as_uint(row_down[u]) >> 23) | 0x4B000000u);  // (2^23 + 128 less 2^23 + its exponent)
                }
            }

            // softmax of the chunk, in powers of two
            uint32_t ph[NT][2], pl[NT][2];  // P^T as the B operand (heads and tails)
            float alpha[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                float pr[4];
                if (p.cap > 0.0f || p.slopes) {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        float x = sc[nt][j] * p.scale;
                        if (p.cap > 0.0f) x = p.cap * tanh_rel(x * p.inv_cap);
                        const float y = fmaf(-slope[nt][j & 1], (float)(len - 1 - row0 - r8 - (j >> 1) * 8), x);
                        sc[nt][j] = Q8 ? fmaf(y, LOG2E, row_e[j >> 1]) : y * LOG2E;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; j++) sc[nt][j] = Q8 ? fmaf(sc[nt][j], scale_log2, row_e[j >> 1]) : sc[nt][j] * scale_log2;
                }
                if (!full) {
                    if (!vis(row0 + r8)) sc[nt][0] = sc[nt][1] = -INFINITY;
                    if (!vis(row0 + r8 + 8)) sc[nt][2] = sc[nt][3] = -INFINITY;
                }
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    float mx = fmaxf(sc[nt][j], sc[nt][j + 2]);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    mx = fmaxf(mx, m[nt][j]);
                    const float ms = mx == -INFINITY ? 0.0f : mx;  // nothing seen yet
                    alpha[nt][j] = ex2(m[nt][j] - ms);
                    m[nt][j] = mx;
                    pr[j] = ex2(sc[nt][j] - (ms - DEC_P_LOG2<Q8>));
                    pr[j + 2] = ex2(sc[nt][j + 2] - (ms - DEC_P_LOG2<Q8>));
                    l[nt][j] = fmaf(l[nt][j], alpha[nt][j], Q8 ? fmaf(pr[j], row_down[0], pr[j + 2] * row_down[1]) : pr[j] + pr[j + 2]);
                }
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    uint32_t hi, lo;
                    split_pair(pr[2 * i], pr[2 * i + 1], hi, lo);
                    ph[nt][i] = transpose8(hi);
                    pl[nt][i] = transpose8(lo);
                }
            }
            if (!Q8) {
                cp_wait<2>();
                __syncwarp();
            }

            // O^T = O^T * alpha + V^T P^T
            if constexpr (Q8) {
                // with d' a relative scale, the head of p * d' is h = fp16(p_hi * d'), and its tail
                // p_lo * d' + (p_hi * d' - h), the bracket exact in one fma
#pragma unroll
                for (int b = 0; b < D / 32; b++) {
                    if (b * 32 >= dim) break;
                    uint32_t a0[4], a1[4];
                    // transposed pairs of codes: rows 2c and 2c + 1 of values 2r, 2r + 1 (r = lane / 4)
                    uint32_t w[4];
                    ldsm4t(vt + at_v[0] + 32 * b, w);
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        w[u] ^= 0x80808080u;
                        a0[u] = h2u(__hsub2(u2h(__byte_perm(w[u], 0x64646464u, 0x4240)), k1152));
                        a1[u] = h2u(__hsub2(u2h(__byte_perm(w[u], 0x64646464u, 0x4341)), k1152));
                    }
                    const __half2 d0 = __hmul2(__halves2half2(dv[0][b], dv[1][b]), u2h(down[0])), d1 = __hmul2(__halves2half2(dv[2][b], dv[3][b]), u2h(down[1]));
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) {
                        const __half2 h0 = __hmul2(u2h(ph[nt][0]), d0), h1 = __hmul2(u2h(ph[nt][1]), d1);
                        const uint32_t lo0 = h2u(__hfma2(u2h(pl[nt][0]), d0, __hfma2(u2h(ph[nt][0]), d0, __hneg2(h0))));
                        const uint32_t lo1 = h2u(__hfma2(u2h(pl[nt][1]), d1, __hfma2(u2h(ph[nt][1]), d1, __hneg2(h1))));
                        const uint32_t hi0 = h2u(h0), hi1 = h2u(h1);
#pragma unroll
                        for (int u = 0; u < 2; u++) {
                            float c[4];
                            mma16816_zero(c, u ? a1 : a0, lo0, lo1);
                            mma16816(c, u ? a1 : a0, hi0, hi1);
#pragma unroll
                            for (int j = 0; j < 4; j++) o[2 * b + u][nt][j] = fmaf(o[2 * b + u][nt][j], alpha[nt][j & 1], c[j]);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int mt = 0; mt < KSTEPS; mt++) {
                    if (mt * 16 >= dim) break;
                    uint32_t a[4];
                    ldsm4t(vt + at_v[mt & 3] + 128 * (mt >> 2), a);
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) {
                        float c[4];
                        mma16816_zero(c, a, pl[nt][0], pl[nt][1]);
                        mma16816(c, a, ph[nt][0], ph[nt][1]);
#pragma unroll
                        for (int j = 0; j < 4; j++) o[mt][nt][j] = fmaf(o[mt][nt][j], alpha[nt][j & 1], c[j]);
                    }
                }
            }
            __syncwarp();  // every lane has read the values
            issue_k(sv);
            sk = sk == 0 ? 2 : sk - 1;
            sv = sv == 0 ? 2 : sv - 1;
        }
        cp_wait<0>();
        if (bad_page) record_error(p.err, SYN_DEVERR_BOUNDS);

        // the warps' parts of the segment, joined in shared memory
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], off);
                if (r8 == 0) sm_m[warp * H + nt * 8 + 2 * c4 + j] = m[nt][j];
            }
        __syncthreads();
        float* buf = reinterpret_cast<float*>(ring);  // [H][D], this warp's
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int hd = nt * 8 + 2 * c4 + j;
                float mx = sm_m[hd];
                for (int w = 1; w < DEC_WARPS; w++) mx = fmaxf(mx, sm_m[w * H + hd]);
                const float f = ex2(m[nt][j] - (mx == -INFINITY ? 0.0f : mx));
                if (r8 == 0) sm_l[warp * H + hd] = l[nt][j] * f;  // (read after the next barrier)
                if (hd < heads) {
#pragma unroll
                    for (int mt = 0; mt < KSTEPS; mt++) {
                        if (mt * 16 >= dim) break;
                        // rows lane/4 and lane/4 + 8 of the tile; Q8_0: the codes' order
                        const int d0 = Q8 ? (mt >> 1) * 32 + 2 * r8 + (mt & 1) : mt * 16 + r8;
                        const int d1 = Q8 ? d0 + 16 : d0 + 8;
                        buf[hd * D + d0] = o[mt][nt][j] * f;
                        buf[hd * D + d1] = o[mt][nt][j + 2] * f;
                    }
                }
            }
        __syncthreads();
        const bool direct = st1 - st0 == n_blocks;
        // a partial's slot: 2*CTA + 1 where the segment begins its item, else 2*CTA
        float* part = p.part + (2 * (int64_t)blockIdx.x + (st0 == 0)) * H * (D + 2);
        for (int i = tid; i < heads * dim >> 2; i += 32 * DEC_WARPS) {
            const int hd = i / (dim >> 2), e = (i - hd * (dim >> 2)) << 2;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < DEC_WARPS; w++) {
                const float4 x = *reinterpret_cast<const float4*>(smem + w * L::WARP + 4 * (hd * D + e));
                acc.x += x.x;
                acc.y += x.y;
                acc.z += x.z;
                acc.w += x.w;
                sum += sm_l[w * H + hd];
            }
            if (direct) {
                const int64_t at_out = s * p.out_stride + (int64_t)(h * p.g + head0 + hd) * dim + e;
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                if (p.out_f16) {
                    const __half2 x = __floats2half2_rn(acc.x * inv, acc.y * inv), y = __floats2half2_rn(acc.z * inv, acc.w * inv);
                    *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + at_out) = make_uint2(h2u(x), h2u(y));
                } else {
                    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at_out) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                }
            } else {
                __stcg(reinterpret_cast<float4*>(part + hd * D + e), acc);
                if (e == 0) {
                    float mx = sm_m[hd];
                    for (int w = 1; w < DEC_WARPS; w++) mx = fmaxf(mx, sm_m[w * H + hd]);
                    __stcg(reinterpret_cast<float2*>(part + H * D) + hd, make_float2(mx, sum));
                }
            }
        }
        if (!direct) {
            // the CTAs that share the item: those whose ranges hold its first and last block
            const int64_t t0 = (int64_t)pre[s] * n_item_h + (int64_t)hh * (n_blocks + extra) + extra;
            const int i0 = (int)(((t0 + 1) * ctas - 1) / total), i1 = (int)(((t0 + n_blocks) * ctas - 1) / total);
            const int item = s * n_item_h + hh;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int before = atomicAdd(&p.count[item], 1);
                flags[5] = before == i1 - i0;
                if (before == i1 - i0) p.count[item] = 0;  // ready for the next call
            }
            __syncthreads();
            if (flags[5]) {
                __threadfence();
                join_parts<D, H>(p, i0, i1, heads, dim, smem, sm_m, sm_l, s * p.out_stride + (int64_t)(h * p.g + head0) * dim);
            }
        }
        __syncthreads();  // the ring and the flags are free for the next segment
    }
}

// ---- host side ---------------------------------------------------------------------------

template <int D, int NT, bool Q8, bool EXACT>
static cudaError_t run_decode_as(const DecodeParams& p, int sms, cudaStream_t s) {
    auto kern = k_attn_decode<D, NT, Q8, EXACT>;
    constexpr int smem = DecLayout<D, Q8>::RING + 2 * DEC_WARPS * 8 * NT * 4 + 40 + 4 * (DEC_MAX_SEQ + 1);
    static ResidentCtas resident;  // per device, looked up once
    int per_sm = 0;
    const cudaError_t e = resident.get(reinterpret_cast<const void*>(kern), 32 * DEC_WARPS, smem, &per_sm);
    if (e != cudaSuccess) return e;
    const int grid = sms * std::min(per_sm, DECODE_CTAS_PER_SM);
    return launch_overlapped(kern, grid, 32 * DEC_WARPS, smem, s, p);
}

template <int D, int NT, bool Q8>
static cudaError_t run_decode(const DecodeParams& p, int sms, cudaStream_t s) {
    return p.c.dim == D ? run_decode_as<D, NT, Q8, true>(p, sms, s) : run_decode_as<D, NT, Q8, false>(p, sms, s);
}

// heads of a group: two columns of 8 where there are more than 8 and the accumulators fit
static int decode_nt(int g, int dim) { return g > 8 && dim <= 128 ? 2 : 1; }

int64_t decode_count_words(int64_t n_seq, int n_heads, int n_kv, int dim) {
    const int g = n_heads / n_kv, h = 8 * decode_nt(g, dim);
    return std::min<int64_t>(n_seq, DEC_MAX_SEQ) * n_kv * ((g + h - 1) / h);
}
int64_t decode_part_floats(int n_heads, int n_kv, int dim, int sms) {
    const int d = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
    return (int64_t)sms * DECODE_CTAS_PER_SM * 2 * 8 * decode_nt(n_heads / n_kv, dim) * (d + 2);
}

cudaError_t launch_attn_decode(const KvCache& c, const AttnDesc& a, int64_t n_seq, const void* q, const int32_t* pages,
                               int64_t max_pages, const int32_t* lens, void* out, float* part, int* count, bool whole,
                               int* err, int sms, int* launches, cudaStream_t s) {
    for (int64_t s0 = 0; s0 < n_seq; s0 += DEC_MAX_SEQ) {
        DecodeParams p;
        p.c = c;
        p.q = static_cast<const __half*>(q) + s0 * a.q_stride;
        p.q_stride = a.q_stride;
        p.out_stride = a.out_stride;
        p.out = static_cast<uint8_t*>(out) + s0 * a.out_stride * (a.out_f16 ? 2 : 4);
        p.pages = pages + s0 * max_pages;
        p.max_pages = max_pages;
        p.lens = lens + s0;
        p.slopes = a.slopes;
        p.prefix = a.prefix ? a.prefix + s0 : nullptr;
        p.first = a.first ? a.first + s0 : nullptr;
        p.part = part;
        p.count = count;
        p.err = err;
        p.scale = a.scale;
        p.cap = a.cap;
        p.inv_cap = a.cap > 0.0f ? std::min(1.0f / a.cap, 0x1p127f) : 0.0f;  // (finite: a score of 0 stays 0)
        p.n_seq = (int)std::min<int64_t>(DEC_MAX_SEQ, n_seq - s0);
        p.g = a.n_heads / c.n_kv;
        const int nt = decode_nt(p.g, c.dim);
        p.n_hg = (p.g + 8 * nt - 1) / (8 * nt);
        p.stride16 = (uint32_t)(c.page_stride >> 4);
        p.window = a.window;
        p.out_f16 = a.out_f16;
        p.whole = whole;
        cudaError_t e;
#define SYN_DEC(D, NT) (c.q8 ? run_decode<D, NT, true>(p, sms, s) : run_decode<D, NT, false>(p, sms, s))
        if (c.dim <= 64) e = nt == 1 ? SYN_DEC(64, 1) : SYN_DEC(64, 2);
        else if (c.dim <= 128) e = nt == 1 ? SYN_DEC(128, 1) : SYN_DEC(128, 2);
        else e = SYN_DEC(256, 1);
#undef SYN_DEC
        if (e != cudaSuccess) return e;
        (*launches)++;
    }
    return cudaSuccess;
}

#ifdef SYN_DEBUG
SYN_BOUNDS_READER(debug_bounds_attn_decode)
#endif

}  // namespace syn
