// attn_prefill.cu — attention of several new tokens of each sequence over the paged cache, on the
// 5th-generation tensor cores (tcgen05, sm_103a).
//
//   x_j = log2(e) * (cap*tanh(scale*q.k_j/cap) - slope*|p - j|),  p_j = 2^(x_j - m),
//   out = sum_j p_j v_j / sum_j p_j  over the keys the query sees, m a running maximum.
//
// An item is 128 or 256 rows of (new token, query head of one kv head), the heads of a token next to
// each other, so that all the heads of a kv head share the cached rows; its keys come in tiles of
// BN.  One persistent CTA per SM takes items until none is left, from the packed batch's end: of a sequence
// the last tokens, which see the most keys, come first.  Warp roles:
//   schedule one warp: takes the next item (a counter), works out what it needs, an item ahead of the
//            others, so that loads and products of an item begin while the one before is written;
//   softmax  4 warps per 128 rows, a thread per row: S from tensor memory, the row's maximum, p in
//            fp16 back into the columns of S, the sum in fp32; O is rescaled in tensor memory when
//            a row's maximum has grown by more than 2^8 (p stays below 2^14 in fp16: rarely);
//   MMA      one warp: S = Q K^T (Q and K from shared memory), O += P V (P from tensor memory, V as
//            an MN-major operand: cached rows are used as they lie);
//   loader   one warp: F16: tensor-map copies of page pieces into a ring of tiles (128-byte
//            swizzle); Q8_0: bulk copies of codes and scales into a ring of raw tiles, which
//   expand   (Q8_0) four warps turn into fp16 tiles of the same layout.
// Registers go where they are used (setmaxnreg): a softmax thread holds its row's 128 scores.
// All hand-offs are mbarriers with bounded waits.
//
// Rows that a mask empties give zeros.  A masked score is replaced before the maximum; V rows past
// the sequence's end are zeroed in shared memory.  A V row that only some rows of the item see may
// still hold infinities or NaN, and 0 * inf is not 0: a row whose sums come out non-finite is
// computed again from the keys it sees, in fp32, when its CTA has done its items (no other warp waits for it
// then).  With an infinite value in the first row of a prompt of 2048 tokens, 32 / 8 heads of 128, every row is:
// 3.7 ms where it takes 0.050; 8192 tokens 50 ms, not 0.39.
//
// Few rows over a long cache: an item's tiles are split between CTAs (no CTA waits: the last to
// finish, by a counter, joins the partials in order).
//
// Measured on GB300, 32 / 8 heads of 128, F16: a prompt of 8192 tokens 395 us, 1.40 PFLOP/s (71 % of
// a library matrix product's rate: a tile of 128 keys takes 2700 cycles, the products of its
// two row tiles 2048: a row tile's softmax, 1450 cycles, stands between its two products); 6 prompts of up to 1001 tokens, capped in a window of 1024, 69 us; 2 chunks of up
// to 2000 tokens over 8000 Q8_0 rows, slopes and documents, 98 us; 9 tokens over 709 rows, heads of 64, 12.2 us.
#include <algorithm>
#include <climits>

#include "kernels.h"
#include "kv_cache.cuh"
#include "tcgen05.cuh"

namespace syn {

constexpr int PRE_MAX_SEQ = 1024;     // sequences of one launch
constexpr float PRE_P_LOG2 = 6.0f;    // p is held as 2^6 p
constexpr float PRE_GROW_LOG2 = 8.0f; // the maximum's lag

// Rows to be computed again, when the CTA has done its items: a warp's rows of an item.
struct Redo {
    int s, h, row0;
    uint32_t bits;
    int next;  // of the same warp
};

struct PrefillParams {
    KvCache c;
    KvCache raw;               // where rows_by_hand reads: the user's cache and table, which are c and pages
    const int32_t* raw_pages;  // unless c is the expanded copy of a Q8_0 cache
    const __half* q;
    int64_t q_stride, out_stride;
    void* out;
    const int32_t* starts;
    const int32_t* pages;
    int64_t max_pages;
    const int32_t* lens;
    const float* slopes;
    const int32_t* prefix;
    const int32_t* first;
    float* part;
    int* count;  // per item, zero between calls
    int* turns;  // [0] items taken past the CTAs' first ones, [1] CTAs done; zero between calls
    Redo* redo;  // [n_redo] one for each warp's rows of each item
    int n_redo;
    int* err;
    float scale, cap;
    int n_seq, n_tok, g, window, out_f16, sms, split;
    int q_tma;  // Q by tensor-map copies (g divides 128: a tile's rows are whole tokens)
    uint32_t idesc_s, idesc_o;
};

template <int D, bool Q8>
struct PreShape {
    static constexpr int QT = D <= 128 ? 2 : 1;     // 128-row tiles of an item
    static constexpr int BN = D <= 128 ? 128 : 64;  // keys of a tile
    static constexpr int NS = D <= 64 ? 6 : Q8 ? 3 : 4;  // tiles (K or V) in the ring
    static constexpr int NR = Q8 ? 2 : 0;           // raw tiles (codes, then scales) ahead of it
    static constexpr int R = 128 * QT;
    static constexpr int STAGE = BN * D * 2;
    static constexpr int RAW = BN * D + BN * D / 16;
    static constexpr int Q_TILE = 128 * D * 2;
    static constexpr int Q = 0;
    static constexpr int RING = QT * Q_TILE;
    static constexpr int RAWS = RING + NS * STAGE;
    static constexpr int BARS = RAWS + NR * RAW;
    static constexpr int INFO = BARS + (8 * (2 * NS + 2 * NR + 19) + 8 + 15) / 16 * 16;
    static constexpr int BYTES = INFO + 64 + 2 * 96 + 4 * (PRE_MAX_SEQ + 1);
    static constexpr int MAX_SPLIT = NS * STAGE / (4 * R);  // parts of an item whose weights fit into the ring
    static constexpr int O_COL = QT == 2 ? 256 : 128;  // S slots below it
    static constexpr int SLOT = QT == 2 ? 128 : 64;    // columns of an S slot
    // warps: softmax, then MMA, loader, scheduler and one that idles, then (Q8_0) four that expand
    static constexpr int MMA_WARP = 4 * QT, LOAD_WARP = MMA_WARP + 1, PLAN_WARP = MMA_WARP + 2, EXPAND_WARP = MMA_WARP + 4;
    static constexpr int READERS = MMA_WARP + 2 + (Q8 ? 4 : 0);  // warps that follow the scheduler
    static constexpr int WARPS = MMA_WARP + 4 + (Q8 ? 4 : 0), THREADS = 32 * WARPS;
    // registers a thread of each kind after the hand-over (two row tiles; their sum over the warps is
    // what the launch gives them: 168 each of 12 warps, 128 each of 16)
    static constexpr int SOFTMAX_REGS = Q8 ? 136 : 208, MMA_REGS = Q8 ? 112 : 88, EXPAND_REGS = 128;
    static_assert(QT == 1 || (Q8 ? 8 * SOFTMAX_REGS + 4 * MMA_REGS + 4 * EXPAND_REGS <= 16 * 128
                                 : 8 * SOFTMAX_REGS + 4 * MMA_REGS <= 12 * 168), "more registers than the launch has");
};

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

// What the scheduler tells the other warps of an item.
struct Item {
    int nt;      // tiles of this part (0: no row sees a key; -1: no item is left)
    int t0;      // its first tile
    int n_split, sp, index;  // parts of the item, this one, the item's number
    int s, h, row0, rows, n_new, tok0, len, prefix;
    Tiles tiles;
    Visible seen;  // what some row sees lies in here
};
static_assert(sizeof(Item) <= 96, "two items' space in shared memory");
__device__ __forceinline__ Item item_of(volatile const int* w) {
    Item it;
    it.nt = w[0];
    it.t0 = w[1];
    it.n_split = w[2];
    it.sp = w[3];
    it.index = w[4];
    it.s = w[5];
    it.h = w[6];
    it.row0 = w[7];
    it.rows = w[8];
    it.n_new = w[9];
    it.tok0 = w[10];
    it.len = w[11];
    it.prefix = w[12];
    it.tiles.a0 = w[13];
    it.tiles.a1 = w[14];
    it.tiles.b0 = w[15];
    it.tiles.b1 = w[16];
    it.seen.first = w[17];
    it.seen.pre = w[18];
    it.seen.low = w[19];
    it.seen.end = w[20];
    return it;
}

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

// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (starts that run backwards or past the call's tokens count as none)
__device__ __forceinline__ int new_tokens(const int32_t* starts, int s, int n_tok) {
    const int a = starts[s], b = starts[s + 1];
    return a < 0 || b > n_tok ? 0 : max(b - a, 0);
}

__device__ __forceinline__ void store_out(const PrefillParams& p, int64_t at, float y) {
    if (p.out_f16) static_cast<__half*>(p.out)[at] = __float2half_rn(y);
    else static_cast<float*>(p.out)[at] = y;
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

// The rows row0, row0 + 1, ... of sequence s (a row: a token and a query head of kv head h) that `bits` names,
// a lane each, computed again in fp32 from the keys that they see in tiles [t0, t1) of `tiles` (t1 = 0: from all that
// they see), 8 keys' scores at a time, then their values, which all lanes read together.  The sums are held in this
// lane's row of the CTA's partial (o: R rows, D values each, then maxima and sums), which is where a part's go
// in the end; else the outputs are written.  It ends where every sum is NaN, which nothing mends.  (Q8: the
// user's cache is Q8_0.)
template <bool Q8>
__device__ __noinline__ void rows_by_hand(const PrefillParams& p, int s, int h, int row0, uint32_t bits, Tiles tiles, int t0, int t1,
                                          int BN, bool part, float* o, int R, int D) {
    const int lane = threadIdx.x & 31, dim = p.c.dim, shift = p.raw.page_shift, mask = (1 << shift) - 1;
    const int64_t scales = (int64_t)dim << shift;  // Q8_0: where a tile's scales begin
    const bool mine = (bits >> lane) & 1;
    const int t = mine ? (row0 + lane) / p.g : 0, tok = p.starts[s] + t;
    const int head = h * p.g + (mine ? row0 + lane - t * p.g : 0);
    const int len = held_rows(p.lens[s], p.max_pages, p.c.page_shift), pos = len - new_tokens(p.starts, s, p.n_tok) + t;
    const Visible vis = visible_of(len, pos, p.first ? p.first[tok] : 0, p.prefix ? p.prefix[s] : 0, p.window);
    const int32_t* table = p.raw_pages + (int64_t)s * p.max_pages;
    const __half* qrow = p.q + (int64_t)tok * p.q_stride + (int64_t)head * dim;
    const float slope = p.slopes ? p.slopes[head] : 0.0f;
    if (t1 == 0) {
        const bool early = mine && vis.pre > vis.first, late = mine && vis.end > vis.low;
        const int lo = early ? vis.first : late ? vis.low : INT_MAX, hi = max(early ? vis.pre : 0, late ? vis.end : 0);
        tiles.a0 = tiles.a1 = 0;
        tiles.b1 = (__reduce_max_sync(0xffffffffu, hi) + BN - 1) / BN;
        tiles.b0 = min(__reduce_min_sync(0xffffffffu, lo) / BN, tiles.b1);
        t0 = 0;
        t1 = tiles.count();
    }
    float m = -INFINITY, l = 0.0f;
    for (int e = 0; e < dim && mine; e++) o[(int64_t)e * R] = 0.0f;
    bool left = true;
    for (int64_t n = (int64_t)t0 * BN; n < (int64_t)t1 * BN && left; n += 8) {
        const int jb = tiles.at((int)(n / BN)) * BN + (int)(n % BN);
        uint32_t seen = mine ? (span_bits(vis.low - jb, vis.end - jb, 0) | span_bits(vis.first - jb, vis.pre - jb, 0)) & 0xffu : 0u;
        if (!__any_sync(0xffffffffu, seen != 0)) continue;
        const int id = table[jb >> shift];  // (8 keys lie in one page)
        if ((unsigned)id >= (unsigned)p.raw.n_pages) continue;
        const int64_t tile = (int64_t)id * p.raw.page_stride + (int64_t)h * p.raw.tile, row = (int64_t)(jb & mask) * dim;
        float sc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
        for (int e = 0; e < dim; e += 8) {
            float q[8];
            cached8<false>(reinterpret_cast<const uint8_t*>(qrow), 0, e, q);
#pragma unroll
            for (int c = 0; c < 8; c++) {
                float k[8];
                cached8<Q8>(p.raw.k + tile, scales, row + c * dim + e, k);
#pragma unroll
                for (int i = 0; i < 8; i++) sc[c] = fmaf(q[i], k[i], sc[c]);
            }
        }
        float nm = m;
#pragma unroll
        for (int c = 0; c < 8; c++) {
            float x = sc[c] * p.scale;
            if (p.cap > 0.0f) x = p.cap * tanhf(x / p.cap);
            x = fmaf(-slope, fabsf((float)(pos - jb - c)), x) * 1.4426950408889634f;
            sc[c] = (seen >> c) & 1 ? x : -INFINITY;
            nm = fmaxf(nm, sc[c]);
        }
        const float ms = nm == -INFINITY ? 0.0f : nm, f = ex2(m - ms);
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < 8; c++) {
            sc[c] = (seen >> c) & 1 ? ex2(sc[c] - ms + PRE_P_LOG2) : 0.0f;
            sum += sc[c];
        }
        m = nm;
        l = fmaf(l, f, sum);
        left = __any_sync(0xffffffffu, mine && l == l);
#pragma unroll 2
        for (int e = 0; e < dim; e += 8) {
            float acc[8];
#pragma unroll
            for (int i = 0; i < 8; i++) acc[i] = o[(int64_t)(e + i) * R] * f;
#pragma unroll
            for (int c = 0; c < 8; c++) {
                float v[8];
                cached8<Q8>(p.raw.v + tile, scales, row + c * dim + e, v);
#pragma unroll
                for (int i = 0; i < 8; i++) acc[i] = (seen >> c) & 1 ? fmaf(sc[c], v[i], acc[i]) : acc[i];
            }
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (mine) o[(int64_t)(e + i) * R] = acc[i];
        }
    }
    if (!mine) return;
    if (part) {
        o[(int64_t)D * R] = m;
        o[(int64_t)(D + 1) * R] = l;
    } else {
        const int64_t out0 = (int64_t)tok * p.out_stride + (int64_t)head * dim;
        for (int e = 0; e < dim; e++) store_out(p, out0 + e, l == 0.0f ? 0.0f : o[(int64_t)e * R] / l);
    }
}

template <int D, bool Q8, bool MOD>
__global__ void __launch_bounds__(PreShape<D, Q8>::THREADS, 1)
    k_attn_prefill(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ CUtensorMap qmap, const __grid_constant__ PrefillParams p) {
    using L = PreShape<D, Q8>;
    constexpr int QT = L::QT, BN = L::BN, NS = L::NS, NR = L::NR, R = L::R, THREADS = L::THREADS;
    constexpr int MMA_WARP = L::MMA_WARP, LOAD_WARP = L::LOAD_WARP, EXPAND_WARP = L::EXPAND_WARP;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BARS);
    uint64_t* kv_full = bars;
    uint64_t* kv_empty = kv_full + NS;
    uint64_t* s_full = kv_empty + NS;  // [2] S in its slot
    uint64_t* p_full = s_full + 2;     // [2] P in its slot
    uint64_t* p_half = p_full + 2;     // [2] its first half
    uint64_t* o_done = p_half + 2;     // [2] a P V product is complete
    uint64_t* q_full = o_done + 2;     // [2]
    uint64_t* raw_full = q_full + 2;       // [NR] Q8_0: codes and scales have arrived
    uint64_t* raw_empty = raw_full + NR;   // [NR]
    uint64_t* mma_idle = raw_empty + NR;
    uint64_t* q_empty = mma_idle + 1;      // [2] the item's last S is complete
    uint64_t* item_full = q_empty + 2;     // [2]
    uint64_t* item_empty = item_full + 2;  // [2]
    uint64_t* join_bar = item_empty + 2;   // the softmax warps, around a join
    uint64_t* item_want = join_bar + 1;    // the loader has nothing left to load
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(item_want + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* info = reinterpret_cast<int*>(smem + L::INFO);  // [0] carry of the scan, [1] the join's verdict
    volatile uint32_t* raw_there = reinterpret_cast<volatile uint32_t*>(info + 12);  // [NR] pieces that arrived
    volatile int* item_ints = info + 16;  // [2][24] items
    int* pre = info + 64;                 // [n_seq + 1] items (of one kv head) before each sequence

    // (the shuffle tells the compiler that the warp's index is the same for its lanes)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int dim = p.c.dim, nh = (dim + 63) >> 6;  // 64-value column chunks of a row

    // ---- set-up that touches no global memory, ahead of the kernel before this one -----------
    if (tid == 0) {
        for (int i = 0; i < NS; i++) {
            mbar_init(smem_u32(&kv_full[i]), Q8 ? 4 : 1);
            mbar_init(smem_u32(&kv_empty[i]), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_u32(&s_full[i]), 1);
            mbar_init(smem_u32(&p_full[i]), 4);
            mbar_init(smem_u32(&p_half[i]), 4);
            mbar_init(smem_u32(&o_done[i]), 1);
            mbar_init(smem_u32(&q_full[i]), p.q_tma ? 1 : 4);
            mbar_init(smem_u32(&q_empty[i]), 1);
            mbar_init(smem_u32(&item_full[i]), 1);
            mbar_init(smem_u32(&item_empty[i]), L::READERS);
        }
        for (int i = 0; i < NR; i++) {
            mbar_init(smem_u32(&raw_full[i]), 1);
            mbar_init(smem_u32(&raw_empty[i]), 4);
        }
        mbar_init(smem_u32(mma_idle), 1);
        mbar_init(smem_u32(join_bar), MMA_WARP);
        mbar_init(smem_u32(item_want), 1);
        *abort_flag = 0;
        info[0] = 0;
        pre[0] = 0;
        fence_mbar_init();
    }
    if (warp == MMA_WARP) tmem_alloc(smem_u32(tmem_slot), 512);
    griddep_release();
    griddep_wait();

    auto items_of = [&](int n_new) { return (int)(((int64_t)n_new * p.g + R - 1) / R); };
    if (p.n_seq > 32) {  // (up to 32 sequences are the scheduler's lanes)
        __syncthreads();
        for (int base = 0; base < p.n_seq; base += THREADS) {
            const int sq = base + tid;
            int x = sq < p.n_seq ? items_of(new_tokens(p.starts, sq, p.n_tok)) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            int* sums = reinterpret_cast<int*>(smem);  // (nothing else uses it yet)
            if (lane == 31) sums[warp] = x;
            __syncthreads();
            int before = info[0];
            for (int w = 0; w < warp; w++) before += sums[w];
            if (sq < p.n_seq) pre[sq + 1] = before + x;
            __syncthreads();
            if (tid == THREADS - 1) info[0] = before + x;
            __syncthreads();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // the next item, for the warps that follow the scheduler; false: none is left, or a wait gave up
    int n_items = 0;
    auto next_item = [&](Item& it) {
        const int slot = n_items & 1;
        if (!mbar_wait(smem_u32(&item_full[slot]), (n_items >> 1) & 1, p.err, abort_flag)) return false;
        it = item_of(item_ints + 24 * slot);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&item_empty[slot]));
        n_items++;
        return it.nt >= 0;
    };
    auto tiles_in_use = [&](const Item& it) { return QT == 2 && it.rows <= 128 ? 1 : QT; };  // 128-row tiles

    // The ring's order: K of the first tile, then (two row tiles) V and the next K, or (one) the
    // next K and V.  Piece i of an item's 2*nt: is it V, and of which tile.
    auto piece_v = [&](int i, int nt) { return QT == 2 ? (i & 1) : i == 2 * nt - 1 || (i > 0 && (i & 1) == 0); };
    auto piece_tile = [&](int i, int nt) { return QT == 2 ? i >> 1 : i == 2 * nt - 1 ? nt - 1 : i == 0 ? 0 : (i & 1) ? (i + 1) >> 1 : (i >> 1) - 1; };

    // An item's tiles go up, or, with a bias by distance, from the last one down: the largest scores come
    // first, and O is not rescaled tile after tile (a 4096-token prompt with slopes 154 -> 129 us;
    // without, going down costs 3 %: rows that see nothing of the last tile start late).
    auto turn_tile = [&](int i, int nt) { return MOD && p.slopes ? nt - 1 - i : i; };

    if (warp < MMA_WARP) {
        // ------------------------------------ softmax ------------------------------------------
        if (QT == 2) take_registers<L::SOFTMAX_REGS>();
        const int qt = warp >> 2;
        const int r = tid;  // row of the item
        const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t o_base = lane_base + L::O_COL + qt * D;
        const float c_log2 = p.scale * 1.4426950408889634f;
        const float cap_log2 = p.cap * 1.4426950408889634f;
        // (finite however small the cap is: a score of 0 stays 0)
        const float to_cap = p.cap > 0.0f ? fminf(fmaxf(p.scale / p.cap, -1e38f), 1e38f) : 0.0f, to_cap2 = 2.0f * 1.4426950408889634f * to_cap;
        int done = 0, q_turn = 0, joins = 0;  // tiles and Q tiles of this row tile, syncs of the softmax warps so far
        auto softmax_sync = [&]() {  // (bounded, as every wait: a warp may have given up)
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(join_bar));
            return mbar_wait(smem_u32(join_bar), joins++ & 1, p.err, abort_flag);
        };
        int redo_list = -1, split_slot = -1;  // this warp's rows to be computed again; where the split item is, if this is one's part
        uint32_t split_redo = 0;              // this warp's rows of that part
        Item it{};
        while (next_item(it)) {
            const bool row_ok = tid < it.rows;
            Visible vis;
            vis.first = vis.pre = vis.low = vis.end = 0;
            int pos = 0, my_tok = 0, my_head = 0;
            if (row_ok) {
                const int t = (it.row0 + tid) / p.g;
                my_head = it.h * p.g + (it.row0 + tid - t * p.g);
                my_tok = it.tok0 + t;
                pos = it.len - it.n_new + t;
                vis = visible_of(it.len, pos, p.first ? p.first[my_tok] : 0, it.prefix, p.window);
            }
            const int64_t out0 = (int64_t)my_tok * p.out_stride + (int64_t)my_head * dim;
            if (it.nt == 0) {  // no row of the item sees a key
                if (row_ok)
                    for (int e = 0; e < dim; e++) store_out(p, out0 + e, 0.0f);
                continue;
            }
            float* part = p.part + (int64_t)blockIdx.x * R * (D + 2);  // [D][R] values, [R] maxima, [R] sums
            if (it.n_split > 1) split_slot = (n_items - 1) & 1;  // (the CTA's only item)
            if (qt >= tiles_in_use(it)) continue;
            if (!p.q_tma) {
                // this thread's Q row into shared memory, 16-byte piece j of chunk c at j ^ (row % 8)
                if (!mbar_wait(smem_u32(&q_empty[qt]), (q_turn & 1) ^ 1, p.err, abort_flag)) break;
                uint8_t* qs = smem + L::Q + qt * L::Q_TILE + (tid & 127) * 128;
                const uint4* qrow = reinterpret_cast<const uint4*>(p.q + (int64_t)my_tok * p.q_stride + (int64_t)my_head * dim);
#pragma unroll
                for (int j0 = 0; j0 < D / 8; j0 += 8) {  // (8 loads on their way at a time)
                    uint4 w[8];
#pragma unroll
                    for (int j = 0; j < 8; j++) w[j] = row_ok && 8 * (j0 + j) < dim ? __ldg(qrow + j0 + j) : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < 8; j++) *reinterpret_cast<uint4*>(qs + (j0 >> 3) * (128 * 128) + ((j ^ (tid & 7)) << 4)) = w[j];
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&q_full[qt]));
                q_turn++;
            }
            const float slope = MOD && p.slopes && row_ok ? p.slopes[my_head] * 1.4426950408889634f : 0.0f;
            float m = -INFINITY, l = 0.0f;
            bool ok = true;
            for (int i = 0; i < it.nt; i++, done++) {
                const int slot = QT == 2 ? qt : done & 1;
                const uint32_t phase = QT == 2 ? done & 1 : (done >> 1) & 1;
                if (!mbar_wait(smem_u32(&s_full[slot]), phase, p.err, abort_flag)) { ok = false; break; }
                tc_fence_after();
                const uint32_t s_base = lane_base + slot * L::SLOT;
                const int j0 = it.tiles.at(it.t0 + turn_tile(i, it.nt)) * BN;
                const bool full = !row_ok || (j0 >= vis.low && j0 + BN <= vis.end) || (j0 >= vis.first && j0 + BN <= vis.pre);
                const bool masked = !__all_sync(0xffffffffu, full);  // (the same for the warp)
                // Scores of columns c0 .. c0 + N - 1, in powers of two where they are capped or biased, masked.
                auto finish = [&](auto& v, int c0) {
                    constexpr int N = sizeof(v) / 4;
                    if (MOD) {
                        if (p.cap > 0.0f) {
                            // Scores up to half the cap in size: tanh(y) = y times a polynomial in y^2, fitted on
                            // [0, 1/2] to 3e-7, the scale and the cap folded into its coefficients: five paired
                            // instructions for two scores, and none of the two special-function ones a score of
                            // the general form, which has to share that unit with the powers.  Each score goes
                            // by its own size, so that its bits do not depend on the others'; the vote only spares
                            // the general form where no score needs it (keys that a row does not see may vote).
                            // 4096 tokens, F16, heads of 128 (256): not capped 109 (136) us, capped with small scores
                            // 157 (150), with scores on both sides of half the cap everywhere 257 (184); there the general
                            // form for all, whose choice rows would have to share, takes 198 (172).
                            const float k = to_cap * to_cap;
                            const float a0 = 0.999999464f * c_log2, a1 = -0.333263761f * c_log2 * k, a2 = 0.131909124f * c_log2 * k * k,
                                        a3 = -0.0444185817f * c_log2 * k * k * k;
                            const uint64_t b0 = pack2(a0, a0), b1 = pack2(a1, a1), b2 = pack2(a2, a2), b3 = pack2(a3, a3);
                            // (the scale may be negative; with a cap so small that a coefficient overflows no score is small)
                            const float to_half = fabsf(a3) < INFINITY ? fabsf(to_cap) : INFINITY;
                            auto small2 = [&](uint64_t x) {
                                const uint64_t z = mul2(x, x);
                                return unpack2(mul2(x, fma2(z, fma2(z, fma2(z, b3, b2), b1), b0)));
                            };
                            float big = 0.0f;
#pragma unroll
                            for (int c = 0; c < N; c += 2)
                                big = fmaxf(fmaxf(big, fabsf(__uint_as_float(v[c]))), fabsf(__uint_as_float(v[c + 1])));
                            if (__all_sync(0xffffffffu, big * to_half <= 0.5f)) {
#pragma unroll
                                for (int c = 0; c < N; c += 2) {
                                    const float2 r2 = small2(pack2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])));
                                    v[c] = __float_as_uint(r2.x);
                                    v[c + 1] = __float_as_uint(r2.y);
                                }
                            } else {
                                // cap*tanh(x/cap) = cap - 2 cap/(1 + 2^(2 x log2(e)/cap)), all in powers of two
                                const uint64_t k2 = pack2(to_cap2, to_cap2), one2 = pack2(1.0f, 1.0f);
                                const uint64_t m2 = pack2(-2.0f * cap_log2, -2.0f * cap_log2), cap2 = pack2(cap_log2, cap_log2);
#pragma unroll
                                for (int c = 0; c < N; c += 2) {
                                    const float v0 = __uint_as_float(v[c]), v1 = __uint_as_float(v[c + 1]);
                                    const float2 r2 = small2(pack2(v0, v1)), y = unpack2(mul2(pack2(v0, v1), k2));
                                    const float2 z = unpack2(add2(pack2(ex2(y.x), ex2(y.y)), one2));
                                    const float2 x = unpack2(fma2(pack2(rcp(z.x), rcp(z.y)), m2, cap2));
                                    v[c] = __float_as_uint(fabsf(v0) * to_half <= 0.5f ? r2.x : x.x);
                                    v[c + 1] = __float_as_uint(fabsf(v1) * to_half <= 0.5f ? r2.y : x.y);
                                }
                            }
                        }
                        // (not capped: still to be scaled; c_log2 or 1)
                        const float left = p.cap > 0.0f ? 1.0f : c_log2;
                        if (p.slopes && !p.prefix) {
                            // no key after the query is seen: the distance is far - c, two scores at a time (c counts in
                            // whole numbers, exactly)
                            const float far = (float)(pos - j0 - c0);
                            uint64_t c2 = pack2(0.0f, 1.0f);
                            const uint64_t two2 = pack2(2.0f, 2.0f), s2 = pack2(slope, slope), f2 = pack2(-slope * far, -slope * far);
                            const uint64_t l2 = pack2(left, left);
#pragma unroll
                            for (int c = 0; c < N; c += 2) {
                                const float2 x = unpack2(fma2(pack2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), l2, fma2(c2, s2, f2)));
                                v[c] = __float_as_uint(x.x);
                                v[c + 1] = __float_as_uint(x.y);
                                c2 = add2(c2, two2);
                            }
                        } else if (p.slopes) {
                            const float far = (float)(pos - j0 - c0);
#pragma unroll
                            for (int c = 0; c < N; c++)
                                v[c] = __float_as_uint(fmaf(-slope, fabsf(far - (float)c), __uint_as_float(v[c]) * left));
                        } else if (!(p.cap > 0.0f)) {  // (a scale that is not positive)
#pragma unroll
                            for (int c = 0; c < N; c++) v[c] = __float_as_uint(__uint_as_float(v[c]) * left);
                        }
                    }
                    if (masked) {
#pragma unroll
                        for (int w = 0; w < N / 32; w++) {
                            const int j = j0 + c0;
                            const uint32_t bits = row_ok ? span_bits(vis.low - j, vis.end - j, w) | span_bits(vis.first - j, vis.pre - j, w)
                                                         : 0xffffffffu;
#pragma unroll
                            for (int c = 0; c < 32; c++)
                                if (!((bits >> c) & 1)) v[32 * w + c] = 0xff800000u;  // -inf
                        }
                    }
                };
                auto largest = [&](auto& v, float mx) {
                    constexpr int N = sizeof(v) / 4;
                    float m4[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < N; c += 8)
#pragma unroll
                        for (int u = 0; u < 4; u++)
                            m4[u] = fmaxf(fmaxf(m4[u], __uint_as_float(v[c + 2 * u])), __uint_as_float(v[c + 2 * u + 1]));
                    return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                };
                // The scores of an F16 cache's row are held, all BN of them.  Beside the expanding warps (Q8_0) a
                // thread has too few registers for that: they pass twice, 32 at a time: finished, searched for
                // the maximum and put back, then fetched again for the powers.  (Spilled, the expanding warps'
                // codes above all, a tile took 6800 cycles: local memory is outside what shared memory
                // leaves of L1.)
                constexpr bool HOLD = !Q8;
                constexpr int N = BN / 32;
                uint32_t held[HOLD ? BN : 32], other[32];
                float mx = -INFINITY;
                if (HOLD) {
#pragma unroll
                    for (int c = 0; c < BN; c += 32) TMEM_LD32(s_base + c, (held + (HOLD ? c : 0)));
#pragma unroll
                    for (int c = 0; c < BN; c += 32) TMEM_LD_WAIT32((held + (HOLD ? c : 0)));
                    finish(held, 0);
                    mx = largest(held, mx);
                } else {
                    TMEM_LD32(s_base, held);
                    TMEM_LD_WAIT32(held);
#pragma unroll
                    for (int w = 0; w < N; w++) {
                        uint32_t(&v)[32] = reinterpret_cast<uint32_t(&)[32]>(*((w & 1) ? other : held));
                        uint32_t(&next)[32] = reinterpret_cast<uint32_t(&)[32]>(*((w & 1) ? held : other));
                        if (w + 1 < N) TMEM_LD32(s_base + 32 * (w + 1), next);
                        finish(v, 32 * w);
                        mx = largest(v, mx);
                        if (w + 1 < N) TMEM_LD_WAIT32(next);
                        if (MOD || masked) TMEM_ST32(s_base + 32 * w, v);
                    }
                    if (MOD || masked) tmem_st_wait();
                    TMEM_LD32(s_base, held);
                }
                if (!MOD) mx *= c_log2;
                // the reference of the powers follows the maximum when that has grown by 2^8
                const bool grow = mx > m + PRE_GROW_LOG2;  // (or is the first that is not -inf)
                const float f = grow ? ex2(m - mx) : 1.0f;
                if (grow) {
                    m = mx;
                    l *= f;
                }
                if (i > 0 && __any_sync(0xffffffffu, grow)) {
                    // O holds the tiles before: wait for the last product into it, then scale
                    if (!mbar_wait(smem_u32(&o_done[qt]), (done - 1) & 1, p.err, abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    for (int c = 0; c < dim; c += 16) {
                        uint32_t o[16];
                        TMEM_LD16(o_base + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int u = 0; u < 16; u++) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
                        TMEM_ST16(o_base + c, o);
                    }
                }
                const float ms = (m == -INFINITY ? 0.0f : m) - PRE_P_LOG2;
                const uint64_t c2 = pack2(MOD ? 1.0f : c_log2, MOD ? 1.0f : c_log2), ms2 = pack2(-ms, -ms);
                uint64_t sum2[2] = {0, 0};
                if (!HOLD) TMEM_LD_WAIT32(held);
#pragma unroll
                for (int w = 0; w < N; w++) {
                    uint32_t(&v)[32] = reinterpret_cast<uint32_t(&)[32]>(*(HOLD ? held + 32 * (HOLD ? w : 0) : (w & 1) ? other : held));
                    uint32_t(&next)[32] = reinterpret_cast<uint32_t(&)[32]>(*((w & 1) ? held : other));
                    if (!HOLD && w + 1 < N) TMEM_LD32(s_base + 32 * (w + 1), next);
                    uint32_t pw[16];
#pragma unroll
                    for (int u = 0; u < 16; u++) {
                        const float2 x = unpack2(fma2(pack2(__uint_as_float(v[2 * u]), __uint_as_float(v[2 * u + 1])), c2, ms2));
                        const float a = ex2(x.x), e = ex2(x.y);
                        sum2[u & 1] = add2(sum2[u & 1], pack2(a, e));
                        const __half2 hh = __floats2half2_rn(a, e);
                        pw[u] = *reinterpret_cast<const uint32_t*>(&hh);
                    }
                    if (!HOLD && w + 1 < N) TMEM_LD_WAIT32(next);  // (before P overwrites scores)
                    TMEM_ST16(s_base + 16 * w, pw);
                    if (w == N / 2 - 1) {  // the product with the first half of the tile's keys can begin
                        tmem_st_wait();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&p_half[slot]));
                    }
                }
                const float2 sa = unpack2(add2(sum2[0], sum2[1]));
                l += sa.x + sa.y;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&p_full[slot]));
            }
            // (one row tile: S of a tile is issued before the product of the one before, so the last
            // two products may both be outstanding, and a parity tells only neighbours apart)
            if (QT == 1 && it.nt > 1) ok = ok && mbar_wait(smem_u32(&o_done[qt]), (done - 2) & 1, p.err, abort_flag);
            if (!ok || !mbar_wait(smem_u32(&o_done[qt]), (done - 1) & 1, p.err, abort_flag)) break;
            tc_fence_after();
            {
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                uint64_t odd2 = 0;  // 0 times every sum: NaN where one is not finite
                for (int c = 0; c < dim; c += 32) {
                    uint32_t o[32];
                    __syncwarp();
                    TMEM_LD32(o_base + c, o);
                    TMEM_LD_WAIT32(o);
#pragma unroll
                    for (int u = 0; u < 32; u += 2) odd2 = fma2(pack2(__uint_as_float(o[u]), __uint_as_float(o[u + 1])), 0, odd2);
                    if (!row_ok) continue;
                    if (it.n_split > 1) {
#pragma unroll
                        for (int u = 0; u < 32; u++) __stcg(part + (int64_t)(c + u) * R + r, __uint_as_float(o[u]));
                    } else if (p.out_f16) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<__half*>(p.out) + out0 + c);
#pragma unroll
                        for (int u = 0; u < 4; u++) {
                            uint32_t w[4];
#pragma unroll
                            for (int x = 0; x < 4; x++) {
                                const __half2 hh = __floats2half2_rn(__uint_as_float(o[8 * u + 2 * x]) * inv, __uint_as_float(o[8 * u + 2 * x + 1]) * inv);
                                w[x] = *reinterpret_cast<const uint32_t*>(&hh);
                            }
                            dst[u] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
                        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + out0 + c);
#pragma unroll
                        for (int u = 0; u < 8; u++)
                            dst[u] = make_float4(__uint_as_float(o[4 * u]) * inv, __uint_as_float(o[4 * u + 1]) * inv,
                                                 __uint_as_float(o[4 * u + 2]) * inv, __uint_as_float(o[4 * u + 3]) * inv);
                    }
                }
                __syncwarp();
                if (it.n_split > 1 && row_ok) {
                    __stcg(part + (int64_t)D * R + r, m);
                    __stcg(part + (int64_t)(D + 1) * R + r, l);
                }
                // Rows whose weighted values are not finite are computed again: a value that the row does
                // not see may have come in as 0 * inf.  Where the sum of the weights is not finite itself a score
                // that the row sees is not, and its outputs are NaN as they are; but over Q8_0 the key may only
                // have been past what fp16 holds.  That is slow, so it waits until no other warp waits for this one.
                const float2 odd = unpack2(odd2);
                const bool odd_l = !(l * 0.0f == 0.0f), odd_o = !(odd.x + odd.y == 0.0f);
                // (And where scores are in the millions: the powers take scores times the scale, unrounded, less a rounded
                // maximum, and what lies between the two has to stay well below 1.)
                const bool far = !MOD && fabsf(m) > 0x1p22f && fabsf(m) < INFINITY;
                const uint32_t redo = __ballot_sync(0xffffffffu, row_ok && (far || (odd_l ? p.raw.q8 : odd_o)));
                if (it.n_split > 1) {
                    split_redo = redo;
                } else if (redo) {
                    const int64_t at = (int64_t)it.index * (R / 32) + warp;
                    if (at < p.n_redo) {  // (more items than that only where starts[] does not ascend)
                        if (lane == 0) p.redo[at] = Redo{it.s, it.h, it.row0 + 32 * warp, redo, redo_list};
                        redo_list = (int)at;
                    }
                }
            }
        }
        __syncwarp();
        auto by_hand = [&](int s, int h, int row0, uint32_t bits, const Tiles& tiles, int t0, int t1, bool part) {
            float* o = p.part + (int64_t)blockIdx.x * R * (D + 2) + r;
            if (Q8 || p.raw.q8) rows_by_hand<true>(p, s, h, row0, bits, tiles, t0, t1, BN, part, o, R, D);
            else rows_by_hand<false>(p, s, h, row0, bits, tiles, t0, t1, BN, part, o, R, D);
        };
        while (redo_list >= 0) {
            const Redo x = p.redo[redo_list];
            by_hand(x.s, x.h, x.row0, x.bits, Tiles{}, 0, 0, false);
            redo_list = x.next;
        }
        // ---- the last of a split item's CTAs joins the partials ------------------------------------
        if (split_slot >= 0) do {
            it = item_of(item_ints + 24 * split_slot);
            if (split_redo)
                by_hand(it.s, it.h, it.row0 + 32 * warp, split_redo, it.tiles, it.t0, it.t0 + it.nt, true);
            __threadfence();
            const bool together = softmax_sync();
            if (tid == 0) {  // (also where a wait gave up: the counters of the calls to come start from zero)
                const int before = atomicAdd(&p.count[it.index], 1);
                info[1] = before == it.n_split - 1;
                if (before == it.n_split - 1) p.count[it.index] = 0;
            }
            if (!together || !softmax_sync() || !info[1]) break;
            const bool row_ok = tid < it.rows;
            __threadfence();
            const float* base = p.part + (int64_t)(blockIdx.x - it.sp) * R * (D + 2);
            constexpr int64_t pitch = (int64_t)R * (D + 2);
            // each row's weights of the parts (the ring is free), then the values: independent loads
            float* weight = reinterpret_cast<float*>(smem + L::RING);  // [it.n_split][R]
            if (row_ok) {
                float mx = -INFINITY, sum = 0.0f;
                for (int x0 = 0; x0 < it.n_split; x0 += 8) {  // (the last batch repeats the last part's loads)
                    float pm[8], pl[8];
#pragma unroll
                    for (int x = 0; x < 8; x++) {
                        const float* q = base + min(x0 + x, it.n_split - 1) * pitch + (int64_t)D * R + tid;
                        pm[x] = __ldcg(q);
                        pl[x] = __ldcg(q + R);
                    }
#pragma unroll
                    for (int x = 0; x < 8; x++) {
                        if (x0 + x >= it.n_split) continue;
                        const float nm = fmaxf(mx, pm[x]), ms = nm == -INFINITY ? 0.0f : nm;
                        sum = sum * ex2(mx - ms) + pl[x] * ex2(pm[x] - ms);
                        mx = nm;
                        weight[(x0 + x) * R + tid] = pm[x];
                    }
                }
                const float ms = mx == -INFINITY ? 0.0f : mx, inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                for (int x = 0; x < it.n_split; x++) weight[x * R + tid] = ex2(weight[x * R + tid] - ms) * inv;
            }
            if (!softmax_sync()) break;
            // A thread joins 4 values of 4 rows at a time, the loads of 4 parts (16 float4) in flight together; a
            // warp 16 values of 32 rows, so that its loads are whole lines and its stores whole sectors.
            const int row_blocks = (it.rows + 31) >> 5;
            for (int u = tid >> 5; u < row_blocks * (dim >> 4); u += R / 32) {
                const int e = (u / row_blocks << 4) + ((lane >> 3) << 2), r4 = (u - (u / row_blocks) * row_blocks) * 32 + ((lane & 7) << 2);
                if (r4 >= it.rows) continue;
                float acc[4][4];
#pragma unroll
                for (int i = 0; i < 4; i++) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
                for (int x0 = 0; x0 < it.n_split; x0 += 4) {  // (the last batch repeats the last part's loads)
                    float4 po[4][4];
#pragma unroll
                    for (int x = 0; x < 4; x++)
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            po[x][i] = __ldcg(reinterpret_cast<const float4*>(base + min(x0 + x, it.n_split - 1) * pitch + (int64_t)(e + i) * R + r4));
#pragma unroll
                    for (int x = 0; x < 4; x++) {
                        if (x0 + x >= it.n_split) continue;
                        const float4 w = *reinterpret_cast<const float4*>(weight + (x0 + x) * R + r4);
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            acc[0][i] = fmaf(po[x][i].x, w.x, acc[0][i]);
                            acc[1][i] = fmaf(po[x][i].y, w.y, acc[1][i]);
                            acc[2][i] = fmaf(po[x][i].z, w.z, acc[2][i]);
                            acc[3][i] = fmaf(po[x][i].w, w.w, acc[3][i]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    if (r4 + j >= it.rows) continue;
                    const int t = (it.row0 + r4 + j) / p.g;
                    const int64_t at = (int64_t)(it.tok0 + t) * p.out_stride + (int64_t)(it.h * p.g + it.row0 + r4 + j - t * p.g) * dim + e;
                    if (p.out_f16) {
                        const __half2 lo = __floats2half2_rn(acc[j][0], acc[j][1]), hi = __floats2half2_rn(acc[j][2], acc[j][3]);
                        *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + at) =
                            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                    } else {
                        *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
                    }
                }
            }
        } while (false);
    } else if (warp < EXPAND_WARP) {
      if (QT == 2) give_registers<L::MMA_REGS>();
      if (warp == MMA_WARP) {
        // ------------------------------------ MMA ----------------------------------------------
        int rc = 0;                           // ring pieces taken so far
        int done[2] = {0, 0}, q_turn[2] = {0, 0};  // tiles and Q tiles of each row tile so far
        bool ok = true;
        Item it{};
        auto take = [&](int i) {  // wait for piece i of the ring
            if (!mbar_wait(smem_u32(&kv_full[i % NS]), (i / NS) & 1, p.err, abort_flag)) return false;
            tc_fence_after();
            return true;
        };
        const uint32_t lead = elect_lane();
        const uint32_t ring_s = smem_u32(smem + L::RING), q_s = smem_u32(smem + L::Q);
        const uint64_t k_major = sdesc_sw128(0), n_major = sdesc_sw128_mn(0, BN * 128);
        auto issue_s = [&](int qt, int slot, int i) {  // S = Q K^T from piece i
            const uint64_t qd = k_major + ((q_s + qt * L::Q_TILE) >> 4), kd = k_major + ((ring_s + (i % NS) * L::STAGE) >> 4);
#pragma unroll
            for (int ks = 0; ks < D / 16; ks++)
                if (ks * 16 < dim)
                    mma_f16_lead(lead, tmem + slot * L::SLOT, qd + (((ks >> 2) * (128 * 128) + (ks & 3) * 32) >> 4),
                                 kd + (((ks >> 2) * (BN * 128) + (ks & 3) * 32) >> 4), p.idesc_s, ks > 0);
            mma_commit_lead(lead, smem_u32(&s_full[slot]));
        };
        auto issue_o = [&](int qt, int slot, int i, uint32_t phase, bool first) {  // O += P V from piece i
            const uint64_t vd = n_major + ((ring_s + (i % NS) * L::STAGE) >> 4);
#pragma unroll
            for (int half = 0; half < 2; half++) {
                if (!mbar_wait(smem_u32(half ? &p_full[slot] : &p_half[slot]), phase, p.err, abort_flag)) return false;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < BN / 32; k++) {
                    const int ks = half * (BN / 32) + k;
                    mma_f16_ts_lead(lead, tmem + L::O_COL + qt * D, tmem + slot * L::SLOT + 8 * ks, vd + (ks * 2048 >> 4), p.idesc_o,
                                    !first || ks > 0);
                }
            }
            mma_commit_lead(lead, smem_u32(&o_done[qt]));
            return true;
        };
        auto release = [&](int i) { mma_commit_lead(lead, smem_u32(&kv_empty[i % NS])); };
        // V rows past the sequence's end hold whatever the page holds: zeros
        auto clean = [&](int i, int tile) {
            const int j0 = it.tiles.at(it.t0 + turn_tile(tile, it.nt)) * BN;
            if (Q8 || j0 + BN <= it.len) return;
            uint8_t* va = smem + L::RING + (i % NS) * L::STAGE;
            const int from = max(it.len - j0, 0);
            for (int u = lane; u < (BN - from) * nh * 8; u += 32) {
                const int c = u / ((BN - from) * 8), x = u - c * (BN - from) * 8;
                *reinterpret_cast<uint4*>(va + c * (BN * 128) + from * 128 + x * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
        };
        while (ok && next_item(it)) {
            const int nt = it.nt, q_act = tiles_in_use(it);
            if (nt == 0) continue;
#pragma unroll
            for (int qt = 0; qt < QT; qt++)
                if (qt < q_act) ok = ok && mbar_wait(smem_u32(&q_full[qt]), q_turn[qt]++ & 1, p.err, abort_flag);
            if (!ok || !(ok = take(rc))) break;
            // (S of the first tile goes where P of the last item's last tile was: in order behind its product)
#pragma unroll
            for (int qt = 0; qt < QT; qt++) {
                if (qt >= q_act) continue;
                issue_s(qt, QT == 2 ? qt : done[0] & 1, rc);
                if (nt == 1) mma_commit_lead(lead, smem_u32(&q_empty[qt]));
            }
            release(rc);
            rc++;
            for (int i = 0; i < nt && ok; i++) {
                if (QT == 2) {
                    const int pv = rc, pk = rc + 1;
                    if (!(ok = take(pv))) break;
                    clean(pv, i);
                    if (i + 1 < nt && !(ok = take(pk))) break;
#pragma unroll
                    for (int qt = 0; qt < QT; qt++) {
                        if (qt >= q_act || !ok) continue;
                        if (!(ok = issue_o(qt, qt, pv, done[qt]++ & 1, i == 0))) continue;
                        if (i + 1 < nt) issue_s(qt, qt, pk);
                        if (i + 2 == nt) mma_commit_lead(lead, smem_u32(&q_empty[qt]));
                    }
                    if (!ok) break;
                    release(pv);
                    if (i + 1 < nt) release(pk);
                    rc = i + 1 < nt ? pk + 1 : pv + 1;
                } else {
                    if (i + 1 < nt) {
                        if (!(ok = take(rc))) break;
                        issue_s(0, (done[0] + 1) & 1, rc);
                        if (i + 2 == nt) mma_commit_lead(lead, smem_u32(&q_empty[0]));
                        release(rc);
                        rc++;
                    }
                    if (!(ok = take(rc))) break;
                    clean(rc, i);
                    if (!(ok = issue_o(0, done[0] & 1, rc, (done[0] >> 1) & 1, i == 0))) break;
                    done[0]++;
                    release(rc);
                    rc++;
                }
            }
        }
        // every product issued is complete before the accumulators are freed (the softmax warps
        // have seen the last one finish, except after an abort)
        mma_commit_lead(lead, smem_u32(mma_idle));
        mbar_drain(smem_u32(mma_idle), 0, p.err);
      } else if (warp == LOAD_WARP) {
        // ------------------------------------ loader -------------------------------------------
        const int box = min(BN, 1 << p.c.page_shift), n_box = BN / box;  // rows of a copy; lane l does the l-th
        int kc = 0, q_turn[2] = {0, 0};  // pieces and Q tiles so far
        bool ok = true;
        Item it{};
        for (bool first = true; ok; first = false) {
            if (!first && lane == 0) mbar_arrive(smem_u32(item_want));
            if (!next_item(it)) break;
            if (it.nt == 0) continue;
            const int q_act = tiles_in_use(it);
            if (p.q_tma) {
                // 128 / g tokens of g heads: the row order of the item.  (Tokens past the call's are zeros;
                // those of the next sequence are rows that nobody writes.)
#pragma unroll
                for (int qt = 0; qt < QT; qt++) {
                    if (qt >= q_act || !ok) continue;
                    if (!(ok = mbar_wait(smem_u32(&q_empty[qt]), (q_turn[qt] & 1) ^ 1, p.err, abort_flag))) continue;
                    q_turn[qt]++;
                    if (lane == 0) {
                        const uint32_t full = smem_u32(&q_full[qt]), dst = smem_u32(smem + L::Q + qt * L::Q_TILE);
                        mbar_arrive_expect_tx(full, (uint32_t)nh * 128 * 128);
                        for (int c = 0; c < nh; c++)
                            tma_load_3d(dst + c * (128 * 128), &qmap, 64 * c, it.h * p.g, it.tok0 + (it.row0 + 128 * qt) / p.g, full);
                    }
                    __syncwarp();
                }
            }
#ifdef SYN_TEST_STALL
            const int n_pieces = 0;  // timeout-test build: no tile is ever loaded, so the waits run out
#else
            const int n_pieces = 2 * it.nt;
#endif
            const int32_t* table = p.pages + (int64_t)it.s * p.max_pages;
            for (int i = 0; i < n_pieces && ok; i++, kc++) {
                const int st = Q8 ? kc % max(NR, 1) : kc % NS;
                const uint32_t turn = (uint32_t)(Q8 ? kc / max(NR, 1) : kc / NS);
                const bool is_v = piece_v(i, it.nt);
                const int j = it.tiles.at(it.t0 + turn_tile(piece_tile(i, it.nt), it.nt)) * BN + lane * box;
                int id = -1;  // past the end, or an id outside the pool
                if (lane < n_box && j < it.len) {
                    const int x = table[j >> p.c.page_shift];
                    if ((unsigned)x < (unsigned)p.c.n_pages) id = x;
                    else if (it.seen.any(j, j + box)) record_error(p.err, SYN_DEVERR_BOUNDS);  // (else it may be gone)
                }
                if (!(ok = mbar_wait(smem_u32(Q8 ? &raw_empty[st] : &kv_empty[st]), (turn & 1) ^ 1, p.err, abort_flag))) break;
                const int cell = j & ((1 << p.c.page_shift) - 1);
                if (!Q8) {
                    // a page that is not there becomes the page after the last: the copy fills it with zeros
                    const uint32_t full = smem_u32(&kv_full[st]);
                    if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)nh * BN * 128);
                    __syncwarp();
                    if (lane < n_box && SYN_IN_BOUNDS((lane + 1) * box * 128 + (nh - 1) * BN * 128 <= L::STAGE)) {
                        const uint32_t dst = smem_u32(smem + L::RING + st * L::STAGE) + lane * box * 128;
                        for (int c = 0; c < nh; c++)
                            tma_load_4d(dst + c * (BN * 128), is_v ? &vmap : &kmap, 64 * c, cell, it.h, id < 0 ? (int)p.c.n_pages : id, full);
                    }
                } else {
                    // (rows of pages that are not there, or past the end, are zeroed by the expanding warps)
                    const uint32_t full = smem_u32(&raw_full[st]), there = __ballot_sync(0xffffffffu, id >= 0);
                    const uint32_t codes = (uint32_t)(box * dim), scales = codes / 16;
                    if (lane == 0) {
                        raw_there[st] = there;  // (before the arrival that lets raw_full complete)
                        mbar_arrive_expect_tx(full, (uint32_t)__popc(there) * (codes + scales));
                    }
                    __syncwarp();
                    if (id >= 0 && SYN_IN_BOUNDS((uint32_t)(lane + 1) * codes <= BN * D && id < p.c.n_pages)) {
                        const uint32_t dst = smem_u32(smem + L::RAWS + st * L::RAW);
                        const uint8_t* tile = (is_v ? p.c.v : p.c.k) + (int64_t)id * p.c.page_stride + (int64_t)it.h * p.c.tile;
                        bulk_g2s(dst + lane * codes, tile + (int64_t)cell * dim, codes, full);
                        bulk_g2s(dst + BN * D + lane * scales, tile + ((int64_t)dim << p.c.page_shift) + (int64_t)cell * (dim >> 4), scales, full);
                    }
                }
                __syncwarp();
            }
        }
        // the tiles still in flight (issued, not consumed: only after an abort) land first
        if (p.q_tma)
#pragma unroll
            for (int qt = 0; qt < QT; qt++)
                if (q_turn[qt] > 0) mbar_drain(smem_u32(&q_full[qt]), (q_turn[qt] - 1) & 1, p.err);
        if (Q8) {
            for (int u = max(0, kc - NR); u < kc; u++) mbar_drain(smem_u32(&raw_full[u % max(NR, 1)]), (u / max(NR, 1)) & 1, p.err);
        } else {
            for (int u = max(0, kc - NS); u < kc; u++) mbar_drain(smem_u32(&kv_full[u % NS]), (u / NS) & 1, p.err);
        }
      } else if (warp == L::PLAN_WARP) {
        // ------------------------------------ scheduler ----------------------------------------
        // up to 32 sequences: a lane each
        const int mine = min(lane, p.n_seq - 1);
        int my_new = 0, my_sum = 0;
        if (p.n_seq <= 32) {
            my_new = lane < p.n_seq ? new_tokens(p.starts, mine, p.n_tok) : 0;
            my_sum = items_of(my_new);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, my_sum, o);
                if (lane >= o) my_sum += y;
            }
        }
        const int n_tiles_q = p.n_seq <= 32 ? __shfl_sync(0xffffffffu, my_sum, 31) : pre[p.n_seq];
        const int64_t items = (int64_t)n_tiles_q * p.c.n_kv;
        // parts of an item: as many as leave every SM one
        const int max_split = p.split && items > 0 && items < p.sms ? min((int)(p.sms / items), L::MAX_SPLIT) : 1;
        const int64_t total = items * max_split;
        int64_t w = blockIdx.x;
        for (int n = 0;;) {
            Item it{};
            it.nt = -1;
            if (w < total) {
                const int64_t b = w / max_split;
                it.index = (int)b;
                it.sp = (int)(w - b * max_split);
                // the last tiles of a sequence see the most keys: they go first (of the sequences, the last)
                const int qtile = n_tiles_q - 1 - (int)(b / p.c.n_kv);
                it.h = (int)(b % p.c.n_kv);
                int before;
                if (p.n_seq <= 32) {
                    it.s = __ffs(__ballot_sync(0xffffffffu, my_sum > qtile)) - 1;
                    before = it.s > 0 ? __shfl_sync(0xffffffffu, my_sum, max(it.s - 1, 0)) : 0;
                } else {
                    int lo = 0, hi = p.n_seq - 1;
                    while (lo < hi) {
                        const int mid = (lo + hi) >> 1;
                        if (pre[mid + 1] > qtile) hi = mid;
                        else lo = mid + 1;
                    }
                    it.s = lo;
                    before = pre[lo];
                }
                it.n_new = new_tokens(p.starts, it.s, p.n_tok);
                it.tok0 = p.starts[it.s];
                it.len = held_rows(p.lens[it.s], p.max_pages, p.c.page_shift);
                it.prefix = p.prefix ? p.prefix[it.s] : 0;
                it.row0 = (qtile - before) * R;
                it.rows = (int)min((int64_t)R, (int64_t)it.n_new * p.g - it.row0);
                // [mf, prefix) then [ml, me): every key that some row sees lies in one of them
                const int pre_end = min(max(it.prefix, 0), it.len), pos0 = it.len - it.n_new;
                const int tk0 = it.row0 / p.g, tk1 = (it.row0 + it.rows - 1) / p.g;  // first and last token
                int mf, ml, me;
                if (p.first) {
                    mf = ml = INT_MAX;
                    me = 0;
                    for (int t = tk0 + lane; t <= tk1; t += 32) {
                        const Visible v = visible_of(it.len, pos0 + t, p.first[it.tok0 + t], it.prefix, p.window);
                        if (v.pre > v.first || v.end > v.low) {
                            mf = min(mf, v.pre > v.first ? v.first : v.low);
                            ml = min(ml, v.end > v.low ? v.low : v.pre);
                            me = max(me, max(v.end, v.pre));
                        }
                    }
                    mf = __reduce_min_sync(0xffffffffu, mf);
                    ml = __reduce_min_sync(0xffffffffu, ml);
                    me = __reduce_max_sync(0xffffffffu, me);
                } else if (pos0 + tk1 >= 0) {  // positions ascend: the first and the last token tell
                    ml = p.window > 0 ? max(0, max(pos0 + tk0, 0) - p.window + 1) : 0;
                    mf = pre_end > 0 ? 0 : ml;
                    me = max(min(pos0 + tk1 + 1, it.len), pre_end);
                } else {
                    ml = me = pre_end;
                    mf = 0;
                }
                Tiles& tl = it.tiles;
                tl.a0 = tl.a1 = tl.b0 = tl.b1 = 0;
                if (me > 0) {
                    tl.b0 = ml / BN;
                    tl.b1 = me > ml ? (me + BN - 1) / BN : tl.b0;
                    tl.a0 = tl.a1 = mf / BN;
                    const int ae = min(pre_end, ml);
                    if (ae > mf) tl.a1 = (ae + BN - 1) / BN;
                    if (tl.b1 > tl.b0) tl.a1 = max(tl.a0, min(tl.a1, tl.b0));
                }
                it.seen.first = mf;
                it.seen.pre = pre_end;
                it.seen.low = ml;
                it.seen.end = me;
                const int all = tl.count();
                // Each part more shortens what a part computes and lengthens the join: sqrt(keys / 64) parts.
                // Measured, one sequence, 32 / 8 heads of 128 (us): 64 tokens over 4096 keys
                // in 16 parts 44, 8 (the rule) 39, 4 39, 2 50; 24 / 1 heads, 8 tokens over 32000 in 125 parts
                // 145, 22 (the rule) 57; heads of 256, 32 over 4096 in 32 parts 72, 8 45.
                // Up to 512 keys, or 768 where the join has many values, it does not pay: 9 tokens over 400 keys in
                // 2 parts 17.4, whole 15.2, over 709 in 3 parts 17.0, whole 18.1; 64 over 709 26.6 and 21.7.
                it.n_split = all * BN <= (it.rows * dim < 16384 ? 512 : 768) ? 1 : min(max_split, (int)sqrtf((float)all * (BN / 64)));
                it.t0 = (int)((int64_t)all * min(it.sp, it.n_split) / it.n_split);
                it.nt = it.sp < it.n_split ? (int)((int64_t)all * (it.sp + 1) / it.n_split) - it.t0 : -2;
            }
            if (it.nt != -2) {  // (-2: the item has fewer parts)
                const int slot = n & 1;
                if (!mbar_wait(smem_u32(&item_empty[slot]), ((n >> 1) & 1) ^ 1, p.err, abort_flag)) break;
                if (lane == 0) {
                    volatile int* o = item_ints + 24 * slot;
                    o[0] = it.nt;
                    o[1] = it.t0;
                    o[2] = it.n_split;
                    o[3] = it.sp;
                    o[4] = it.index;
                    o[5] = it.s;
                    o[6] = it.h;
                    o[7] = it.row0;
                    o[8] = it.rows;
                    o[9] = it.n_new;
                    o[10] = it.tok0;
                    o[11] = it.len;
                    o[12] = it.prefix;
                    o[13] = it.tiles.a0;
                    o[14] = it.tiles.a1;
                    o[15] = it.tiles.b0;
                    o[16] = it.tiles.b1;
                    o[17] = it.seen.first;
                    o[18] = it.seen.pre;
                    o[19] = it.seen.low;
                    o[20] = it.seen.end;
                    mbar_arrive(smem_u32(&item_full[slot]));
                }
                __syncwarp();
                n++;
                if (it.nt == -1) break;
            }
            // The next one: the CTAs' first items are their numbers, the rest are counted out, each when the
            // loader has the one before on its way (taken earlier, the items of a small call would be
            // dealt before it shows which CTAs are done first: 6 ragged prompts 101 us, not 79)
            if (it.nt != -2 && !mbar_wait(smem_u32(item_want), (n - 1) & 1, p.err, abort_flag)) break;
            int taken = 0;
            if (lane == 0) taken = atomicAdd(&p.turns[0], 1);
            w = (int64_t)gridDim.x + __shfl_sync(0xffffffffu, taken, 0);
        }
        // the last CTA to get here makes the counters ready for the next call
        if (lane == 0 && atomicAdd(&p.turns[1], 1) == (int)gridDim.x - 1) p.turns[0] = p.turns[1] = 0;
      }
    } else if (Q8) {
        // ------------------------------------ expand (Q8_0) -------------------------------------
        // (they keep the 128 registers of the launch)
        const int lt = tid - 32 * EXPAND_WARP;
        // 16 codes at a time.  A thread takes piece x4 of the 64-value chunks of rows lt/4, lt/4 + 32, ...;
        // neighbouring rows take the chunks in opposite order, so that the 8 lanes that a shared-memory
        // access serves at once touch all the banks, reading and storing.
        constexpr int HALVES = D / 64, UNITS = BN / 32 * HALVES;
        const int x4 = lt & 3, row_t = lt >> 2;
        const int box_shift = min(p.c.page_shift, BN == 128 ? 7 : 6), n_box = BN >> box_shift;
        const uint32_t all_there = n_box == 32 ? 0xffffffffu : (1u << n_box) - 1u;
        const __half2 k1152 = __float2half2_rn(1152.0f);
        int kc = 0;
        bool ok = true;
        Item it{};
        while (ok && next_item(it)) {
#ifdef SYN_TEST_STALL
            const int n_pieces = 0;
#else
            const int n_pieces = 2 * it.nt;
#endif
            for (int i = 0; i < n_pieces && ok; i++, kc++) {
                const int rs = kc % max(NR, 1), st = kc % NS;
                if (!(ok = mbar_wait(smem_u32(&raw_full[rs]), (kc / max(NR, 1)) & 1, p.err, abort_flag))) break;
                if (!(ok = mbar_wait(smem_u32(&kv_empty[st]), ((kc / NS) & 1) ^ 1, p.err, abort_flag))) break;
                const int left = it.len - it.tiles.at(it.t0 + turn_tile(piece_tile(i, it.nt), it.nt)) * BN;  // rows of the tile that exist
                const uint32_t there = raw_there[rs];
                const bool whole = left >= BN && there == all_there;
                const uint8_t* raw = smem + L::RAWS + rs * L::RAW;
                uint8_t* dst = smem + L::RING + st * L::STAGE + row_t * 128;
                const int swap = (((2 * x4) ^ (row_t & 7)) << 4);
                // one piece: 16 codes and their scale to 16 halves.  A byte c becomes 1024 + c by a permute with
                // 0x64; value = scale * code, the one rounding of the expansion (relative 2^-11, like that of p)
                auto put = [&](uint8_t* to, const uint4& code, uint32_t bits) {
                    const __half2 d = expand_scale(bits);
                    const uint32_t cw[4] = {code.x, code.y, code.z, code.w};
                    uint32_t w[8];
#pragma unroll
                    for (int y = 0; y < 4; y++) {
                        const uint32_t z = cw[y] ^ 0x80808080u;
                        uint32_t lo = __byte_perm(z, 0x64646464u, 0x4140), hi = __byte_perm(z, 0x64646464u, 0x4342);
                        const __half2 hl = __hmul2(__hsub2(*reinterpret_cast<__half2*>(&lo), k1152), d);
                        const __half2 hh = __hmul2(__hsub2(*reinterpret_cast<__half2*>(&hi), k1152), d);
                        w[2 * y] = *reinterpret_cast<const uint32_t*>(&hl);
                        w[2 * y + 1] = *reinterpret_cast<const uint32_t*>(&hh);
                    }
                    *reinterpret_cast<uint4*>(to + swap) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(to + (swap ^ 16)) = make_uint4(w[4], w[5], w[6], w[7]);
                };
                if (whole && dim == D) {  // (no test stands between the loads, all ahead of the stores)
                    constexpr int BATCH = UNITS < 4 ? UNITS : 4;
                    const uint8_t* codes = raw + row_t * D + 16 * x4;
                    const uint8_t* scales = raw + BN * D + row_t * (D / 16) + 2 * (x4 >> 1);
                    const int odd = row_t & 1;
#pragma unroll
                    for (int u0 = 0; u0 < UNITS; u0 += BATCH) {
                        uint4 code[BATCH];
                        uint32_t bits[BATCH];
#pragma unroll
                        for (int u = 0; u < BATCH; u++) {
                            const int ru = (u0 + u) / HALVES, half = HALVES > 1 ? ((u0 + u) % HALVES) ^ odd : 0;
                            code[u] = *reinterpret_cast<const uint4*>(codes + ru * (32 * D) + 64 * half);
                            bits[u] = *reinterpret_cast<const uint16_t*>(scales + ru * (2 * D) + 4 * half);
                        }
#pragma unroll
                        for (int u = 0; u < BATCH; u++) {
                            const int ru = (u0 + u) / HALVES, half = HALVES > 1 ? ((u0 + u) % HALVES) ^ odd : 0;
                            put(dst + half * (BN * 128) + ru * (32 * 128), code[u], bits[u]);
                        }
                    }
                } else {  // rows that are not there are zeros
                    for (int u = 0; u < UNITS; u++) {
                        const int half = HALVES > 1 ? (u % HALVES) ^ (row_t & 1) : 0, x = x4 + 4 * half, row = row_t + 32 * (u / HALVES);
                        if (half >= nh) continue;
                        uint4 code = make_uint4(0, 0, 0, 0);
                        uint32_t bits = 0;
                        if (16 * x < dim && row < left && ((there >> (row >> box_shift)) & 1)) {
                            code = *reinterpret_cast<const uint4*>(raw + row * dim + 16 * x);
                            bits = *reinterpret_cast<const uint16_t*>(raw + BN * D + 2 * (row * (dim >> 5) + (x >> 1)));
                        }
                        put(dst + half * (BN * 128) + (u / HALVES) * (32 * 128), code, bits);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&kv_full[st]));
                    mbar_arrive(smem_u32(&raw_empty[rs]));
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---- a Q8_0 cache expanded ahead of the kernel --------------------------------------------
//
// The rows of every sequence as fp16 values (scale * code, rounded once: the values the expanding warps
// make), in an F16 cache of scratch: page i of sequence s is page s * max_pages + i of it.  Bound: HBM and
// L2 (17/16 bytes read and 2 written a value).  The work is counted by what the sequences hold, 256 of them at a
// time, not by the page table's width: 8 prompts of 512 tokens, pages of 64, 75 us with the prefill itself for
// tables of 8 to 1000 pages (by the width: 74 to 183 us).
struct ExpandParams {
    KvCache c;      // Q8_0
    uint8_t* k;     // scratch pools
    uint8_t* v;
    int32_t* table; // [n_seq][max_pages]
    const int32_t* starts;
    const int32_t* pages;
    const int32_t* lens;
    int64_t max_pages;
    int n_seq, n_tok, window;
};

__global__ void __launch_bounds__(256) k_kv_expand(const ExpandParams p) {
    const int dim = p.c.dim, page = 1 << p.c.page_shift, per_row = dim >> 4, n = page * per_row;  // 16 codes at a time
    const __half2 k1152 = __float2half2_rn(1152.0f);
    auto expand = [&](int64_t sp, int id, int h, int is_v) {
        const uint8_t* src = (is_v ? p.c.v : p.c.k) + (int64_t)id * p.c.page_stride + (int64_t)h * p.c.tile;
        uint4* dst = reinterpret_cast<uint4*>((is_v ? p.v : p.k) + (sp * p.c.n_kv + h) * ((int64_t)n * 32));
#pragma unroll 2
        for (int x = threadIdx.x; x < n; x += 256) {
            const uint4 code = *reinterpret_cast<const uint4*>(src + 16 * (int64_t)x);
            const uint32_t bits = *reinterpret_cast<const uint16_t*>(src + 16 * (int64_t)n + 2 * (x >> 1));  // (2 pieces a block)
            const __half2 d = expand_scale(bits);
            const uint32_t cw[4] = {code.x, code.y, code.z, code.w};
            uint32_t w[8];
#pragma unroll
            for (int y = 0; y < 4; y++) {
                const uint32_t z = cw[y] ^ 0x80808080u;
                uint32_t lo = __byte_perm(z, 0x64646464u, 0x4140), hi = __byte_perm(z, 0x64646464u, 0x4342);
                const __half2 hl = __hmul2(__hsub2(*reinterpret_cast<__half2*>(&lo), k1152), d);
                const __half2 hh = __hmul2(__hsub2(*reinterpret_cast<__half2*>(&hi), k1152), d);
                w[2 * y] = *reinterpret_cast<const uint32_t*>(&hl);
                w[2 * y + 1] = *reinterpret_cast<const uint32_t*>(&hh);
            }
            dst[2 * x] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[2 * x + 1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    };
    griddep_release();
    griddep_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, per_page = 2 * p.c.n_kv;
    // The pages of sequence s that some query reads: [first, end).  Rows ahead of every query's window are not
    // read, but all of a tile (of up to 128 rows) that a query's window begins in is: no number that was never
    // written meets p = 0.  (Far fewer than 2^31 in all: the scratch has room for them.)
    auto pages_of = [&](int s, int& first, int& end) {
        const int len = held_rows(p.lens[s], p.max_pages, p.c.page_shift), n_new = new_tokens(p.starts, s, p.n_tok);
        const int64_t low = p.window > 0 ? ((int64_t)len - n_new - p.window) & ~int64_t(127) : 0;
        end = n_new > 0 ? (len + page - 1) >> p.c.page_shift : 0;
        first = (int)min((int64_t)end, max(low, (int64_t)0) >> p.c.page_shift);
    };
    __shared__ int before[257], sums[8];  // units (page, pool, head) ahead of each sequence
    int u = blockIdx.x;
    for (int s0 = 0; s0 < p.n_seq; s0 += 256) {
        int x = 0;
        if (s0 + tid < p.n_seq) {
            int first, end;
            pages_of(s0 + tid, first, end);
            x = (end - first) * per_page;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) sums[warp] = x;
        __syncthreads();
        for (int w = 0; w < warp; w++) x += sums[w];
        before[tid + 1] = x;
        if (tid == 0) before[0] = 0;
        __syncthreads();
        for (; u < before[256]; u += gridDim.x) {
            int lo = 0, hi = 255;  // the sequence whose units hold u
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (before[mid + 1] > u) hi = mid;
                else lo = mid + 1;
            }
            int first, end;
            pages_of(s0 + lo, first, end);
            const int i = (u - before[lo]) / per_page, hp = u - before[lo] - i * per_page, h = hp >> 1, is_v = hp & 1;
            const int64_t sp = (s0 + lo) * p.max_pages + first + i;
            const int id = p.pages[sp];
            const bool ok = (unsigned)id < (unsigned)p.c.n_pages;
            // a page outside the pool is one here too: reported if a query's tile takes it
            if (hp == 0 && tid == 0) p.table[sp] = ok ? (int32_t)sp : -1;
            if (ok) expand(sp, id, h, is_v);
        }
        u -= before[256];
        __syncthreads();
    }
}

cudaError_t launch_kv_expand(const KvCache& c, int64_t n_seq, int64_t n_tok, const int32_t* starts, const int32_t* pages, int64_t max_pages,
                             const int32_t* lens, int window, void* k, void* v, int32_t* table, int sms, cudaStream_t s) {
    ExpandParams p;
    p.c = c;
    p.k = static_cast<uint8_t*>(k);
    p.v = static_cast<uint8_t*>(v);
    p.table = table;
    p.starts = starts;
    p.pages = pages;
    p.lens = lens;
    p.max_pages = max_pages;
    p.n_seq = (int)n_seq;
    p.n_tok = (int)n_tok;
    p.window = window;
    const int64_t units = n_seq * max_pages * 2 * c.n_kv;
    return launch_overlapped(k_kv_expand, (int)std::min<int64_t>(units, (int64_t)sms * 8), 256, 0, s, p);
}

// ---- host side ---------------------------------------------------------------------------

template <int D, bool Q8, bool MOD>
static cudaError_t run_prefill(const CUtensorMap& km, const CUtensorMap& vm, const CUtensorMap& qm, const PrefillParams& p,
                               int grid, cudaStream_t s) {
    auto kern = k_attn_prefill<D, Q8, MOD>;
    constexpr int smem = 1024 + PreShape<D, Q8>::BYTES;
    static_assert(smem <= 232448, "shared memory per CTA exceeds 227 KB");
    static ResidentCtas resident;
    int n;
    cudaError_t e = resident.get(reinterpret_cast<const void*>(kern), PreShape<D, Q8>::THREADS, smem, &n);
    if (e != cudaSuccess) return e;
    if (PreShape<D, Q8>::QT == 2) {
        // the hand-over of registers deals out what the launch has: a build with fewer must not start
        static const int regs = [&] {
            cudaFuncAttributes a;
            return cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(kern)) == cudaSuccess ? a.numRegs : 0;
        }();
        if (regs < (Q8 ? 128 : 168)) return cudaErrorInvalidConfiguration;
    }
    return launch_overlapped(kern, grid, PreShape<D, Q8>::THREADS, smem, s, km, vm, qm, p);
}

static int prefill_rows(int dim) { return dim <= 128 ? 256 : 128; }

// at most one split item per SM has a counter, one CTA per SM a partial
static int64_t part_floats(int dim, int sms) {
    return (int64_t)sms * prefill_rows(dim) * ((dim <= 64 ? 64 : dim <= 128 ? 128 : 256) + 2);
}
// an entry of `redo` for each 32 rows of an item (a power of two: a growing prompt seldom needs more than the last)
static int64_t redo_entries(int64_t n_seq, int64_t n_tok, int n_heads, int n_kv, int dim) {
    const int R = prefill_rows(dim);
    const int64_t need = (n_tok * (n_heads / n_kv) / R + std::min<int64_t>({n_seq, n_tok, PRE_MAX_SEQ})) * n_kv * (R / 32);
    int64_t n = 4096;
    while (n < need) n *= 2;
    return n;
}
int64_t prefill_part_floats(int64_t n_seq, int64_t n_tok, int n_heads, int n_kv, int dim, int sms) {
    return part_floats(dim, sms) + redo_entries(n_seq, n_tok, n_heads, n_kv, dim) * (int64_t)(sizeof(Redo) / 4);
}

cudaError_t launch_attn_prefill(const KvCache& c, const KvCache& raw, const AttnDesc& a, int64_t n_seq, int64_t n_tok,
                                const void* q, const int32_t* starts, const int32_t* pages, const int32_t* raw_pages,
                                int64_t max_pages, const int32_t* lens, void* out, float* part, int* count, bool split,
                                int* err, int sms, int* launches, cudaStream_t s) {
    CUtensorMap km, vm, qm;
    const int D = c.dim <= 64 ? 64 : c.dim <= 128 ? 128 : 256, BN = D <= 128 ? 128 : 64;
    PFN_encodeTiled encode = get_encode();
    if (!encode) return cudaErrorNotSupported;
    const int g = a.n_heads / c.n_kv;
    const bool q_tma = g <= 128 && 128 % g == 0;
    if (q_tma) {
        cuuint64_t dims[3] = {(cuuint64_t)c.dim, (cuuint64_t)a.n_heads, (cuuint64_t)n_tok};
        cuuint64_t strides[2] = {(cuuint64_t)c.dim * 2, (cuuint64_t)a.q_stride * 2};
        cuuint32_t box[3] = {64, (cuuint32_t)g, (cuuint32_t)(128 / g)}, estr[3] = {1, 1, 1};
        if (encode(&qm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    } else {
        qm = CUtensorMap{};  // unused
    }
    if (!c.q8) {
        const int64_t page = int64_t(1) << c.page_shift;
        cuuint64_t dims[4] = {(cuuint64_t)c.dim, (cuuint64_t)page, (cuuint64_t)c.n_kv, (cuuint64_t)c.n_pages};
        cuuint64_t strides[3] = {(cuuint64_t)c.dim * 2, (cuuint64_t)c.tile, (cuuint64_t)c.page_stride};
        cuuint32_t box[4] = {64, (cuuint32_t)std::min<int64_t>(BN, page), 1, 1}, estr[4] = {1, 1, 1, 1};
        for (int i = 0; i < 2; i++)
            if (encode(i ? &vm : &km, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, i ? c.v : c.k, dims, strides, box, estr,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return cudaErrorInvalidValue;
    } else {
        km = vm = CUtensorMap{};  // unused
    }
    PrefillParams p;
    p.c = c;
    p.raw = raw;
    p.q = static_cast<const __half*>(q);
    p.q_stride = a.q_stride;
    p.out_stride = a.out_stride;
    p.out = out;
    p.max_pages = max_pages;
    p.slopes = a.slopes;
    p.first = a.first;
    p.part = part;
    p.redo = reinterpret_cast<Redo*>(part + part_floats(c.dim, sms));
    p.n_redo = (int)redo_entries(n_seq, n_tok, a.n_heads, c.n_kv, c.dim);
    p.count = count + 2;
    p.turns = count;
    p.err = err;
    p.scale = a.scale;
    p.cap = a.cap;
    p.n_tok = (int)n_tok;
    p.g = g;
    p.q_tma = q_tma;
    p.window = a.window;
    p.out_f16 = a.out_f16;
    p.sms = sms;
    p.split = split;
    // kind::f16: D fp32, A and B fp16, M = 128; S: B K-major, N = BN; O: B MN-major, N = dim
    p.idesc_s = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | (8u << 24);
    p.idesc_o = (1u << 4) | (1u << 16) | ((uint32_t)(c.dim >> 3) << 17) | (8u << 24);
    const int R = prefill_rows(c.dim);
    // (a scale that is not positive takes the general path: the fast one scales the maximum)
    const bool mod = a.cap > 0.0f || a.slopes || !(a.scale > 0.0f);
    for (int64_t s0 = 0; s0 < n_seq; s0 += PRE_MAX_SEQ) {
        p.n_seq = (int)std::min<int64_t>(PRE_MAX_SEQ, n_seq - s0);
        p.starts = starts + s0;
        p.pages = pages + s0 * max_pages;
        p.raw_pages = raw_pages + s0 * max_pages;
        p.lens = lens + s0;
        p.prefix = a.prefix ? a.prefix + s0 : nullptr;
        // (more items than this many have a row number past 32 bits; the parts of few items are at most
        // one per SM)
        if (((n_tok * p.g + R - 1) / R + p.n_seq) * c.n_kv > INT_MAX) return cudaErrorInvalidValue;
        const int grid = sms;
        cudaError_t e;
#define SYN_PRE(D)                                                                                              \
    (c.q8 ? (mod ? run_prefill<D, true, true>(km, vm, qm, p, grid, s) : run_prefill<D, true, false>(km, vm, qm, p, grid, s)) \
          : (mod ? run_prefill<D, false, true>(km, vm, qm, p, grid, s) : run_prefill<D, false, false>(km, vm, qm, p, grid, s)))
        e = D == 64 ? SYN_PRE(64) : D == 128 ? SYN_PRE(128) : SYN_PRE(256);
#undef SYN_PRE
        if (e != cudaSuccess) return e;
        (*launches)++;
    }
    return cudaSuccess;
}

#ifdef SYN_DEBUG
SYN_BOUNDS_READER(debug_bounds_attn_prefill)
#endif

}  // namespace syn
