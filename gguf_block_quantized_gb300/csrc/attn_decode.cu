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
//     operand and up to 8 query heads as the columns: S^T = K Q^T, then O^T += V^T P^T.  The
//     product is a small share of the time (a chunk costs about 200 issue slots of the 1400 that
//     its bytes take to arrive), so the tensor path only has to free the other pipes.
//   - p is split into two fp16 numbers (head and tail, 22 bits) and each chunk's product starts
//     from zero and is added to the fp32 sums by fma, because the tensor pipe's own additions
//     truncate.  Scores likewise come from two short chains.  So the result is as exact as fp32
//     arithmetic allows, which fp32 outputs show.
//   - Work is cut by length, not by sequence: blocks of steps (4 chunks, one per warp) of all
//     (sequence, kv head) items are dealt to the CTAs in equal contiguous ranges, found on the
//     device from the lengths (a captured graph keeps working as they grow).  A CTA whose range
//     covers an item writes the output; else it leaves a partial in the workspace, and the CTA
//     that finishes an item last (a counter) joins the partials in order.  No CTA waits.
#include <algorithm>
#include <climits>

#include "kernels.h"
#include "kv_cache.cuh"

namespace syn {

constexpr int DEC_WARPS = 4;
constexpr int DEC_STAGES = 3;
constexpr int DEC_MAX_SEQ = 1024;  // sequences of one launch (their step counts are in shared memory)
// Work is dealt in blocks of this many steps: as many as a ring holds, whose loads are in flight
// together, so cutting a short item finer would not end it sooner.
constexpr int DEC_BLOCK = 3;
constexpr float DEC_P_LOG2 = 14.0f;  // p is held as 2^14 p, in fp16: small p stay normal numbers

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
    int n_seq, g, n_hg, window, out_f16, whole;
};

// ---- primitives ------------------------------------------------------------------------

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp16_all(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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
    const int64_t most = min(p.max_pages << p.c.page_shift, (int64_t)INT_MAX - 64);
    const int len = p.lens[s];
    return len < 0 ? 0 : (int)min((int64_t)len, most);
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
    // row pitches in shared memory.  F16: 16-byte pieces swizzled by the row (ldmatrix reads 8
    // rows of one piece); Q8_0: pitches that put the rows a half-warp reads on different banks
    static constexpr int PK = Q8 ? ((D / 32) % 2 ? D : D + 32) : 2 * D;
    static constexpr int PV = Q8 ? D + 16 : 2 * D;
    static constexpr int K = 0;
    static constexpr int V = 16 * PK;
    static constexpr int KS = V + 16 * PV;  // scales [16][dim/32]
    static constexpr int VS = KS + (Q8 ? D : 0);
    static constexpr int STAGE = VS + (Q8 ? D : 0);
    static constexpr int WARP = DEC_STAGES * STAGE;
    static constexpr int RING = DEC_WARPS * WARP;
};

// CTAs per SM that the ring leaves room for (so many registers are a thread's)
template <int D, bool Q8>
constexpr int DEC_RESIDENT = D == 64 ? (Q8 ? 4 : 4) : D == 128 ? (Q8 ? 3 : 2) : (Q8 ? 1 : 1);

template <int D, int NT, bool Q8>
__global__ void __launch_bounds__(32 * DEC_WARPS, NT == 1 ? DEC_RESIDENT<D, Q8> : 1) k_attn_decode(const DecodeParams p) {
    using L = DecLayout<D, Q8>;
    constexpr int KSTEPS = D / 16;
    constexpr int H = 8 * NT;  // query heads of an item
    static_assert(L::WARP >= H * D * 4, "the merge buffer reuses the ring");
    extern __shared__ __align__(128) uint8_t smem[];
    float* sm_m = reinterpret_cast<float*>(smem + L::RING);  // [DEC_WARPS][H]
    float* sm_l = sm_m + DEC_WARPS * H;
    int* flags = reinterpret_cast<int*>(sm_l + DEC_WARPS * H);  // [0] scan carry, [1..4] warp sums, [5] last
    int* pre = flags + 8;                                        // [n_seq + 1] blocks before each sequence, of one item

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r8 = lane >> 2, c4 = lane & 3;
    const int dim = p.c.dim;
    const int n_item_h = p.c.n_kv * p.n_hg;  // items of a sequence

    // blocks of every sequence, as a running sum
    if (tid == 0) flags[0] = 0, pre[0] = 0;
    __syncthreads();
    for (int base = 0; base < p.n_seq; base += 32 * DEC_WARPS) {
        const int s = base + tid;
        int n = 0;
        if (s < p.n_seq) {
            n = (seq_chunks(seq_visible(p, s, seq_len(p, s))).count() + DEC_WARPS * DEC_BLOCK - 1) / (DEC_WARPS * DEC_BLOCK);
            if (n == 0) {  // no key to see: zeros, written by the CTAs in turn
                if (s % gridDim.x == blockIdx.x) {
                    const int64_t n_out = (int64_t)p.c.n_kv * p.g * dim;
                    for (int64_t i = 0; i < n_out; i++) {
                        if (p.out_f16) static_cast<__half*>(p.out)[s * p.out_stride + i] = __float2half_rn(0.0f);
                        else static_cast<float*>(p.out)[s * p.out_stride + i] = 0.0f;
                    }
                }
            }
        }
        int x = n;
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
    // A chunk's 16 rows lie one after the other in a page, so lane l copies the 16-byte pieces
    // l, l + 32, ...: their places in a stage
    constexpr int N_COPY = Q8 ? D / 32 : D / 16;
    uint32_t to_k[N_COPY], to_v[N_COPY];
#pragma unroll
    for (int i = 0; i < N_COPY; i++) {
        const int idx = i * 32 + lane, r = idx / row_pieces, j = idx - r * row_pieces;
        to_k[i] = L::K + r * L::PK + (Q8 ? 16 * j : ((j ^ (r & 7)) << 4));
        to_v[i] = L::V + r * L::PV + (Q8 ? 16 * j : ((j ^ (r & 7)) << 4));
    }

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
            n_blocks = pre[s + 1] - pre[s];
            const int64_t rel = at - (int64_t)pre[s] * n_item_h;
            hh = (int)(rel / n_blocks);
            st0 = (int)(rel - (int64_t)hh * n_blocks);
            st1 = (int)min((int64_t)n_blocks, st0 + (stop - at));
            at += st1 - st0;
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
                        const uint2 w = *reinterpret_cast<const uint2*>(qr + (ks >> 1) * 32 + 8 * c4 + 4 * (ks & 1));
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
        int e_run = 0;  // Q8_0: o is held relative to 2^(e_run - 15)
        float o[KSTEPS][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
            for (int mt = 0; mt < KSTEPS; mt++) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.0f;
        }

        // this warp's chunks of the segment, every DEC_WARPS-th below `chunk_end`
        const int chunk0 = st0 * (DEC_WARPS * DEC_BLOCK) + warp;
        const int chunk_end = min(n_chunks, st1 * (DEC_WARPS * DEC_BLOCK));
        int next_issue = chunk0;
        auto all_seen = [&](int row) {  // the 16 rows from `row`
            return (row >= vis.low && row + 16 <= vis.end) || (row >= vis.first && row + 16 <= vis.pre);
        };
        // the page ids of the next chunk to issue, looked up one chunk ahead (rows 0-7 and 8-15)
        auto page_of = [&](int row) {
            if (row >= len) return -1;
            const int id = table[row >> p.c.page_shift];
            if ((unsigned)id >= (unsigned long long)p.c.n_pages) {
                record_error(p.err, SYN_DEVERR_BOUNDS);
                return -1;
            }
            return id;
        };
        int id_lo = -1, id_hi = -1;
        auto look_up = [&]() {
            if (next_issue < chunk_end) {
                const int row = ch.at(next_issue) << 4;
                id_lo = page_of(row);
                id_hi = p.c.page_shift >= 4 ? id_lo : page_of(row + 8);
            }
        };
        look_up();
        [[maybe_unused]] const int64_t pool_end = p.c.tile + (p.c.n_pages - 1) * p.c.page_stride;  // from a head's tile of page 0
        const int64_t plane = (int64_t)dim << p.c.page_shift;                     // Q8_0: a tile's scales
        const int n_sp = dim >> 4;  // Q8_0: 16-byte pieces of 16 rows' scales (at most 16)
        auto issue = [&](int stage) {
            if (next_issue < chunk_end) {
                const int row0 = ch.at(next_issue) << 4;
                const uint32_t dst = ring_s + stage * L::STAGE;
                const int cell_lo = row0 & ((1 << p.c.page_shift) - 1);
                if (p.c.page_shift >= 4 && id_lo >= 0 && all_seen(row0)) {
                    const int64_t off = (int64_t)id_lo * p.c.page_stride + (int64_t)cell_lo * row_pieces * 16;
                    if (SYN_IN_BOUNDS(off >= 0 && off + 256 * row_pieces <= pool_end)) {
                        const uint8_t *ks = kbase + off + 16 * lane, *vs = vbase + off + 16 * lane;
#pragma unroll
                        for (int i = 0; i < N_COPY; i++) {
                            if (2 * i >= row_pieces) break;
                            cp16_all(dst + to_k[i], ks + 512 * i);
                            cp16_all(dst + to_v[i], vs + 512 * i);
                        }
                        if (Q8 && lane < 2 * n_sp) {
                            const int i = lane < n_sp ? lane : lane - n_sp;
                            cp16_all(dst + (lane < n_sp ? L::KS : L::VS) + 16 * i,
                                     (lane < n_sp ? kbase : vbase) + (int64_t)id_lo * p.c.page_stride + plane + (int64_t)cell_lo * n_sp + 16 * i);
                        }
                    }
                } else {
                    // a chunk at an end of what is seen, or over two pages: rows that the query does
                    // not see are not read but zero (a masked V row may hold anything, and 0 * inf is
                    // not 0)
                    const int64_t off_lo = (int64_t)max(id_lo, 0) * p.c.page_stride, off_hi = (int64_t)max(id_hi, 0) * p.c.page_stride;
                    const int cell_hi = p.c.page_shift >= 4 ? cell_lo + 8 : 0;
#pragma unroll
                    for (int i = 0; i < N_COPY; i++) {
                        if (2 * i >= row_pieces) break;
                        const int r = (int)(to_k[i] - L::K) / L::PK, j = i * 32 + lane - r * row_pieces;
                        const bool upper = r >= 8;
                        const bool ok = (upper ? id_hi : id_lo) >= 0 && vis(row0 + r);
                        const int64_t off = ok ? (upper ? off_hi + (int64_t)(cell_hi + r - 8) * row_pieces * 16
                                                        : off_lo + (int64_t)(cell_lo + r) * row_pieces * 16) + 16 * j
                                               : 0;
                        if (!SYN_IN_BOUNDS(off >= 0 && off + 16 <= pool_end)) continue;
                        cp16(dst + to_k[i], kbase + off, ok ? 16u : 0u);
                        cp16(dst + to_v[i], vbase + off, ok ? 16u : 0u);
                    }
                    if (Q8 && lane < 2 * n_sp) {  // scales: rows 0-7 and 8-15 apart
                        const int i = lane < n_sp ? lane : lane - n_sp;
                        const bool upper = 2 * i >= n_sp;
                        const bool ok = (upper ? id_hi : id_lo) >= 0;
                        const int64_t off = ok ? plane + (upper ? off_hi + (int64_t)cell_hi * n_sp + 16 * (i - n_sp / 2)
                                                                : off_lo + (int64_t)cell_lo * n_sp + 16 * i)
                                               : 0;
                        if (SYN_IN_BOUNDS(off >= 0 && off + 16 <= pool_end))
                            cp16(dst + (lane < n_sp ? L::KS : L::VS) + 16 * i, (lane < n_sp ? kbase : vbase) + off, ok ? 16u : 0u);
                    }
                }
                next_issue += DEC_WARPS;
                look_up();
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < DEC_STAGES - 1; i++) issue(i);

        int stage = 0;
        for (int ci = chunk0; ci < chunk_end; ci += DEC_WARPS) {
            cp_wait<DEC_STAGES - 2>();
            __syncwarp();
            issue(stage == 0 ? DEC_STAGES - 1 : stage - 1);
            const int row0 = ch.at(ci) << 4;
            const uint32_t st = ring_s + stage * L::STAGE;
            const uint8_t* stp = ring + stage * L::STAGE;
            const bool full = all_seen(row0);
            const bool seen_a = full || vis(row0 + r8), seen_b = full || vis(row0 + r8 + 8);

            // S^T = K Q^T
            float sc[NT][4];
            if (Q8) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.0f;
                const __half2 k1152 = __float2half2_rn(1152.0f);
#pragma unroll
                for (int b = 0; b < D / 32; b++) {
                    if (b * 32 >= dim) break;
                    // codes of a 32-value block: 8 per lane and row, exact in fp16
                    uint32_t a0[4], a1[4];
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        const uint2 w = *reinterpret_cast<const uint2*>(stp + L::K + (r8 + 8 * u) * L::PK + 32 * b + 8 * c4);
                        const uint32_t x = w.x ^ 0x80808080u, y = w.y ^ 0x80808080u;
                        a0[u] = h2u(__hsub2(u2h(__byte_perm(x, 0x64646464u, 0x4140)), k1152));
                        a0[2 + u] = h2u(__hsub2(u2h(__byte_perm(x, 0x64646464u, 0x4342)), k1152));
                        a1[u] = h2u(__hsub2(u2h(__byte_perm(y, 0x64646464u, 0x4140)), k1152));
                        a1[2 + u] = h2u(__hsub2(u2h(__byte_perm(y, 0x64646464u, 0x4342)), k1152));
                    }
                    const float da = h2f_bits(*reinterpret_cast<const uint16_t*>(stp + L::KS + 2 * (r8 * (dim >> 5) + b)));
                    const float db = h2f_bits(*reinterpret_cast<const uint16_t*>(stp + L::KS + 2 * ((r8 + 8) * (dim >> 5) + b)));
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) {
                        float c[4];
                        mma16816_zero(c, a0, qf[2 * b][nt][0], qf[2 * b][nt][1]);
                        mma16816(c, a1, qf[2 * b + 1][nt][0], qf[2 * b + 1][nt][1]);
                        sc[nt][0] = fmaf(c[0], da, sc[nt][0]);
                        sc[nt][1] = fmaf(c[1], da, sc[nt][1]);
                        sc[nt][2] = fmaf(c[2], db, sc[nt][2]);
                        sc[nt][3] = fmaf(c[3], db, sc[nt][3]);
                    }
                }
            } else {
                float s1[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int j = 0; j < 4; j++) sc[nt][j] = s1[nt][j] = 0.0f;
                const int rr = (lane & 7) + ((lane >> 3) & 1) * 8, cc = lane >> 4;
                const uint32_t rowa = st + L::K + rr * L::PK;
#pragma unroll
                for (int ks = 0; ks < KSTEPS; ks++) {
                    if (ks * 16 >= dim) break;
                    uint32_t a[4];
                    ldsm4(rowa + (((2 * ks + cc) ^ (rr & 7)) << 4), a);
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
                        mma16816(ks & 1 ? s1[nt] : sc[nt], a, qf[ks][nt][0], qf[ks][nt][1]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int j = 0; j < 4; j++) sc[nt][j] += s1[nt][j];
            }

            // softmax of the chunk, in powers of two
            uint32_t ph[NT][2], pl[NT][2];  // F16: P^T as the B operand (heads and tails)
            float pr[NT][4], alpha[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                if (p.cap > 0.0f || p.slopes) {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        float x = sc[nt][j] * p.scale;
                        if (p.cap > 0.0f) x = p.cap * tanh_rel(x * p.inv_cap);
                        sc[nt][j] = fmaf(-slope[nt][j & 1], (float)(len - 1 - row0 - r8 - (j >> 1) * 8), x) * LOG2E;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; j++) sc[nt][j] *= scale_log2;
                }
                if (!full) {
                    if (!seen_a) sc[nt][0] = sc[nt][1] = -INFINITY;
                    if (!seen_b) sc[nt][2] = sc[nt][3] = -INFINITY;
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
                    pr[nt][j] = ex2(sc[nt][j] - ms + DEC_P_LOG2);
                    pr[nt][j + 2] = ex2(sc[nt][j + 2] - ms + DEC_P_LOG2);
                    l[nt][j] = fmaf(l[nt][j], alpha[nt][j], pr[nt][j] + pr[nt][j + 2]);
                }
                if (!Q8) {
                    uint32_t hi, lo;
                    split_pair(pr[nt][0], pr[nt][1], hi, lo);
                    ph[nt][0] = transpose8(hi);
                    pl[nt][0] = transpose8(lo);
                    split_pair(pr[nt][2], pr[nt][3], hi, lo);
                    ph[nt][1] = transpose8(hi);
                    pl[nt][1] = transpose8(lo);
                }
            }

            // O^T = O^T * alpha + V^T P^T
            if (Q8) {
                // A row's value scales go into p, in fp32 and before the split, relative to 2^e, the
                // largest power of two among the scales so far: p * scale then fits fp16 whatever
                // the scales (o is kept in units of 2^e, as it is relative to 2^m).
                uint32_t dv[D / 32][2];  // scales of rows (2c, 2c+1), (2c+8, 2c+9) of each block
                uint32_t top = 0;
#pragma unroll
                for (int b = 0; b < D / 32; b++) {
                    if (b * 32 >= dim) break;
                    const uint16_t* sv = reinterpret_cast<const uint16_t*>(stp + L::VS) + 2 * c4 * (dim >> 5) + b;
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        uint32_t x = sv[8 * u * (dim >> 5)], y = sv[(8 * u + 1) * (dim >> 5)];
                        if (!full) {
                            x = vis(row0 + 2 * c4 + 8 * u) ? x : 0u;
                            y = vis(row0 + 2 * c4 + 8 * u + 1) ? y : 0u;
                        }
                        dv[b][u] = x | y << 16;
                        top = max(top, max(x, y) & 0x7FFFu);
                    }
                }
                const int e_new = max(e_run, (int)(__reduce_max_sync(0xffffffffu, top) >> 10));
                const float down = __int_as_float((127 + 15 - e_new) << 23), step = __int_as_float((127 + e_run - e_new) << 23);
                e_run = e_new;
                // p in the B operand's layout: rows 2c, 2c+1, 2c+8, 2c+9 of head lane/4, as the upper and
                // lower halves of the fp32 words
                float pb[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    alpha[nt][0] *= step;
                    alpha[nt][1] *= step;
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        const uint32_t x = __float_as_uint(pr[nt][2 * u]), y = __float_as_uint(pr[nt][2 * u + 1]);
                        const uint32_t hi = transpose8(__byte_perm(x, y, 0x7632)), lo = transpose8(__byte_perm(x, y, 0x5410));
                        pb[nt][2 * u] = __uint_as_float(__byte_perm(lo, hi, 0x5410)) * down;
                        pb[nt][2 * u + 1] = __uint_as_float(__byte_perm(lo, hi, 0x7632)) * down;
                    }
                }
                const __half2 k1152 = __float2half2_rn(1152.0f);
#pragma unroll
                for (int b = 0; b < D / 32; b++) {
                    if (b * 32 >= dim) break;
                    uint32_t a0[4], a1[4];
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        const uint8_t* vr = stp + L::V + (2 * c4 + 8 * u) * L::PV + 32 * b + 4 * r8;
                        const uint32_t x = *reinterpret_cast<const uint32_t*>(vr) ^ 0x80808080u;
                        const uint32_t y = *reinterpret_cast<const uint32_t*>(vr + L::PV) ^ 0x80808080u;
                        const uint32_t x01 = __byte_perm(x, y, 0x5140), x23 = __byte_perm(x, y, 0x7362);
                        a0[2 * u] = h2u(__hsub2(u2h(__byte_perm(x01, 0x64646464u, 0x4140)), k1152));
                        a0[2 * u + 1] = h2u(__hsub2(u2h(__byte_perm(x01, 0x64646464u, 0x4342)), k1152));
                        a1[2 * u] = h2u(__hsub2(u2h(__byte_perm(x23, 0x64646464u, 0x4140)), k1152));
                        a1[2 * u + 1] = h2u(__hsub2(u2h(__byte_perm(x23, 0x64646464u, 0x4342)), k1152));
                    }
                    const float2 d0 = __half22float2(u2h(dv[b][0])), d1 = __half22float2(u2h(dv[b][1]));
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) {
                        uint32_t hi0, lo0, hi1, lo1;
                        split_pair(pb[nt][0] * d0.x, pb[nt][1] * d0.y, hi0, lo0);
                        split_pair(pb[nt][2] * d1.x, pb[nt][3] * d1.y, hi1, lo1);
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
                const int rr = (lane & 7) + (lane >> 4) * 8, cc = (lane >> 3) & 1;
                const uint32_t rowa = st + L::V + rr * L::PV;
#pragma unroll
                for (int mt = 0; mt < KSTEPS; mt++) {
                    if (mt * 16 >= dim) break;
                    uint32_t a[4];
                    ldsm4t(rowa + (((2 * mt + cc) ^ (rr & 7)) << 4), a);
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
            stage = stage == DEC_STAGES - 1 ? 0 : stage + 1;
            __syncwarp();  // every lane has read the stage before it is filled again
        }
        cp_wait<0>();

        // the warps' parts of the segment, joined in shared memory
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], off);
                if (r8 == 0) {
                    sm_m[warp * H + nt * 8 + 2 * c4 + j] = m[nt][j];
                    sm_l[warp * H + nt * 8 + 2 * c4 + j] = l[nt][j];
                }
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
                float f = ex2(m[nt][j] - (mx == -INFINITY ? 0.0f : mx));
                if (Q8) f *= __int_as_float((127 - 15 + e_run) << 23);
                if (hd < heads) {
#pragma unroll
                    for (int mt = 0; mt < KSTEPS; mt++) {
                        if (mt * 16 >= dim) break;
                        // rows lane/4 and lane/4 + 8 of the tile; Q8_0: the codes' order
                        const int d0 = Q8 ? (mt >> 1) * 32 + 4 * r8 + 2 * (mt & 1) : mt * 16 + r8;
                        const int d1 = Q8 ? d0 + 1 : d0 + 8;
                        buf[hd * D + d0] = o[mt][nt][j] * f;
                        buf[hd * D + d1] = o[mt][nt][j + 2] * f;
                    }
                }
            }
        __syncthreads();
        const bool direct = st1 - st0 == n_blocks;
        // a partial's slot: 2*CTA + 1 where the segment begins its item, else 2*CTA
        float* part = p.part + (2 * (int64_t)blockIdx.x + (st0 == 0)) * H * (D + 2);
        for (int i = tid; i < heads * dim; i += 32 * DEC_WARPS) {
            const int hd = i / dim, e = i - hd * dim;
            float mx = sm_m[hd], acc = 0.0f, sum = 0.0f;
            for (int w = 1; w < DEC_WARPS; w++) mx = fmaxf(mx, sm_m[w * H + hd]);
            const float ms = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
            for (int w = 0; w < DEC_WARPS; w++) {
                acc += reinterpret_cast<const float*>(smem + w * L::WARP)[hd * D + e];
                sum = fmaf(sm_l[w * H + hd], ex2(sm_m[w * H + hd] - ms), sum);
            }
            if (direct) {
                const int64_t at_out = s * p.out_stride + (int64_t)(h * p.g + head0 + hd) * dim + e;
                const float y = sum == 0.0f ? 0.0f : acc / sum;
                if (p.out_f16) static_cast<__half*>(p.out)[at_out] = __float2half_rn(y);
                else static_cast<float*>(p.out)[at_out] = y;
            } else {
                __stcg(part + hd * (D + 2) + e, acc);
                if (e == 0) {
                    __stcg(part + hd * (D + 2) + D, mx);
                    __stcg(part + hd * (D + 2) + D + 1, sum);
                }
            }
        }
        if (!direct) {
            // the CTAs that share the item: those whose ranges hold its first and last block
            const int64_t t0 = (int64_t)pre[s] * n_item_h + (int64_t)hh * n_blocks;
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
                for (int i = tid; i < heads * dim; i += 32 * DEC_WARPS) {
                    const int hd = i / dim, e = i - hd * dim;
                    float mx = -INFINITY, sum = 0.0f, acc = 0.0f;
                    for (int c = i0; c <= i1; c++) {
                        const float* q = p.part + ((2 * (int64_t)c + (c == i0)) * H + hd) * (D + 2);
                        const float pm = __ldcg(q + D), pl2 = __ldcg(q + D + 1), po = __ldcg(q + e);
                        const float nm = fmaxf(mx, pm), ms = nm == -INFINITY ? 0.0f : nm;
                        const float fa = ex2(mx - ms), fb = ex2(pm - ms);
                        acc = acc * fa + po * fb;
                        sum = sum * fa + pl2 * fb;
                        mx = nm;
                    }
                    const int64_t at_out = s * p.out_stride + (int64_t)(h * p.g + head0 + hd) * dim + e;
                    const float y = sum == 0.0f ? 0.0f : acc / sum;
                    if (p.out_f16) static_cast<__half*>(p.out)[at_out] = __float2half_rn(y);
                    else static_cast<float*>(p.out)[at_out] = y;
                }
            }
        }
        __syncthreads();  // the ring and the flags are free for the next segment
    }
}

// ---- host side ---------------------------------------------------------------------------

template <int D, int NT, bool Q8>
static cudaError_t run_decode(const DecodeParams& p, int sms, cudaStream_t s) {
    auto kern = k_attn_decode<D, NT, Q8>;
    constexpr int smem = DecLayout<D, Q8>::RING + 2 * DEC_WARPS * 8 * NT * 4 + 32 + 4 * (DEC_MAX_SEQ + 1);
    static ResidentCtas resident;  // per device, looked up once
    int per_sm = 0;
    const cudaError_t e = resident.get(reinterpret_cast<const void*>(kern), 32 * DEC_WARPS, smem, &per_sm);
    if (e != cudaSuccess) return e;
    const int grid = sms * std::min(per_sm, DECODE_CTAS_PER_SM);
    kern<<<grid, 32 * DEC_WARPS, smem, s>>>(p);
    return cudaGetLastError();
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
        p.inv_cap = a.cap > 0.0f ? 1.0f / a.cap : 0.0f;
        p.n_seq = (int)std::min<int64_t>(DEC_MAX_SEQ, n_seq - s0);
        p.g = a.n_heads / c.n_kv;
        const int nt = decode_nt(p.g, c.dim);
        p.n_hg = (p.g + 8 * nt - 1) / (8 * nt);
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
