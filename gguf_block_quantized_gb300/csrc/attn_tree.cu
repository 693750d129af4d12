// attn_tree.cu — attention of drafted tokens, the nodes of a tree, of each sequence over the paged cache, on the
// 5th-generation tensor cores (tcgen05, sm_103a).
//
//   x_j = log2(e) * (cap*tanh(scale*q.k_j/cap) - slope*distance),  p_j = 2^(x_j - m),
//   out = sum_j p_j v_j / sum_j p_j  over the keys the node sees, m a running maximum.
//
// Node i of a sequence's n drafts sees rows ahead of them all (the context) and, among them, its chain: itself, its
// parent, the parent's, ...; its position is the context's length plus its depth.  A row's thread walks
// the chain where a tile of keys reaches into the drafts, and only there.
//
// Bound: HBM up to some 256 rows of (node, query head) a kv head, where the products take as long.  Every cached row is
// read once for all of a kv head's rows, up to 256 (D <= 128) or 128 of them: an item.  Keys come in tiles of BN.
//   - Work is cut by length: the items' tiles, and some for an item's start and end, are dealt to the CTAs in equal
//     contiguous ranges, found on the device from the lengths.  A CTA whose range covers an item writes the
//     output; else it leaves a partial, and a second kernel joins the parts of items, all SMs at it.
//   - More than 128 rows: the two groups of softmax warps have 128 rows each.  Up to 128: both have the same
//     rows, and one half of each tile's keys, with a maximum, a sum and an accumulator of its own, which
//     meet at the item's end.  So a tile's scores are 64 a thread either way, and the next tile's product S runs
//     while they are worked on.
// Warp roles:
//   schedule one warp: cuts the CTA's range into items and parts, an item ahead of the others;
//   softmax  4 warps, or twice 4, a thread per row: S from tensor memory, its maximum, p in fp16 back into the columns of
//            S; O is rescaled in tensor memory when a row's maximum has grown by more than 2^8;
//   MMA      one warp: S = Q K^T (from shared memory), O += P V (P from tensor memory, V as it lies);
//   loader   one warp: F16: tensor-map copies of page pieces into a ring of tiles (128-byte swizzle); Q8_0:
//            bulk copies of codes and scales into a ring of raw tiles, which
//   expand   (Q8_0) eight warps turn into fp16 tiles of the same layout.
// All hand-offs are mbarriers with bounded waits.
//
// Measured on GB300 (cold L2; 32 / 8 heads of 128, pages of 64): 24 F16 sequences of 190 to 4000 rows with up to 26
// drafts 43 us (133 MB, 3.1 TB/s: 5 us to the first product, 7 us of join); 48 Q8_0 sequences of 500 to 6001 with up
// to 13 drafts, capped, 136 us (240 MB, 1.8 TB/s; 105 us without the cap: nothing is full, no scheduler's issue slots past 53 %,
// the tensor pipe 28 %, DRAM 34 %, so a tile's chain of expansion, S, softmax and P V bounds it, one and a half tiles ahead);
// 64 drafts over 120001 F16 rows 118 to 124 us (493 MB, 4.1 TB/s, and 1.0 PFLOP/s): softmax of 256 rows, 1.83 us a tile, is 90 of
// them, what does not grow with the length the rest.
//
// What is alike in attn_prefill.cu (cap, expansion, loader, rows computed again) is mended in both.
//
// A masked score is replaced before the maximum; V rows past the sequence's end are zeroed in shared memory.  A V
// row that only some rows of the item see may still hold infinities or NaN, and 0 * inf is not 0: a row whose
// sums come out non-finite is computed again from the keys it sees, in fp32, when its CTA has done its items.
#include <algorithm>
#include <climits>

#include "attn_tokens.cuh"
#include "kernels.h"

namespace syn {

// What an item's start and end cost, in tiles (1, 2, 3, 4: 24 sequences of 190 to 4000 rows 45.1, 42.8, 43.3, 44.1 us).
constexpr int TREE_ITEM = 2;
// And a part's share of the join: items no longer than the ranges by more are not split (4 sequences of 300 to 500 rows: 0: 17.9
// us, 4 and more: 12.6).
constexpr int TREE_JOIN = 4;
// Tables of at most this many tiles: whole items and no join, which costs some 5 us even where it finds nothing to do (it waits
// for the first kernel's end).  us, whole : split, up to 26 drafts, heads of 128 (F16 / Q8_0):
//    1 sequence of 700 rows 15.1 : 18.7 / 18.0 : 19.8,   1000: 17.4 : 18.2 / 21.0 : 19.9,   1300: 22.5 : 20.1 / 25.6 : 20.8
//    6 of 1000: 18.1 : 21.2 / 21.4 : 23.9,   1600: 24.9 : 22.0 / 29.6 : 24.2
//   19 of 1000: 21.9 : 27.3 / 23.5 : 28.7,   2000: 32.8 : 38.1 / 36.7 : 42.1
//   96 of 500 to 1000: 73.3 : 85.9 / 94.3 : 113.3
// Heads of 256 (tiles of 64 keys), pages of 16, 1 sequence: 300 rows 16.6 : 18.0,  600: 26.6 : 19.3;  pages of 64, 48 of 350 to
// 700: 56.2 : 66.4.  Heads of 64, pages of 16 (a tile is eight copies), 1 sequence: 600 rows 13.7 : 16.8,  900: 18.5 : 16.8;
// 24 of 450 to 900: 29.3 : 29.5,  950 to 1900: 48.8 : 38.3.
// (One long sequence among short ones would wait for itself: so not past 16 tiles.)
constexpr int tree_whole(int D, bool large_pages, bool many) {
    return large_pages ? (D <= 128 ? 8 : 6) * (many ? 2 : 1) : many ? 8 : 6;
}

struct TreeRedo {  // rows to be computed again, when the CTA has done its items: a warp's rows of an item
    int s, h, row0;
    uint32_t bits;
    Tiles tiles;
    int t0, t1, slot;  // a part's tiles and partial (-1: the item is whole)
    int next;          // of the same warp
};
struct TreeSeq {  // a sequence of the launch
    int cost_before, items_before;  // tiles (and what items cost besides) and items of those ahead of it
    int first;                      // the first key that some node sees
    int tok0, n_new, len, prefix;
};
struct TreeSplit {  // an item that several CTAs share
    int tok0, h, row0, rows, first, parts;  // first: the CTA of its first part
    int before, pad;                        // the join's tasks for the items listed before it
};

constexpr int JOIN_VALUES = 4;  // of 32 rows: a task of the join

struct TreeParams {
    KvCache c;
    const __half* q;
    int64_t q_stride, out_stride;
    void* out;
    const int32_t* starts;
    const int32_t* parents;  // of each new token, among its sequence's
    const int32_t* pages;
    int64_t max_pages;
    const int32_t* lens;
    const float* slopes;
    const int32_t* prefix;
    const int32_t* first;
    float* part;        // three partials a CTA: of an item it goes on with, of one it begins, of rows computed again
    TreeSplit* splits;
    int* n_splits;      // [0] the join's tasks and [1] how many (one 64-bit number), [2] CTAs of the join done; zero between calls
    TreeRedo* redo;     // [n_redo] one for each warp's rows of each item, then [CTAs][2][warps] of parts
    int64_t n_redo;
    int* err;
    float scale, cap;
    int n_seq, n_tok, g, window, out_f16, split;
    int q_tma;  // Q by tensor-map copies (g divides 128: a tile's rows are whole tokens)
    uint32_t idesc_s, idesc_o;
};

// Sequences of one launch: as shared memory has room.
constexpr int tree_max_seq(int D, bool q8) { return q8 && D >= 128 ? 256 : 512; }

template <int D, bool Q8>
struct TreeShape {
    static constexpr int QT = D <= 128 ? 2 : 1;     // softmax groups, and 128-row tiles of an item
    static constexpr int BN = D <= 128 ? 128 : 64;  // keys of a tile
    static constexpr int NS = D <= 64 ? 6 : Q8 ? 3 : 4;  // tiles (K or V) in the ring
    static constexpr int NR = Q8 ? 3 : 0;           // raw tiles (codes, then scales) ahead of it
    static constexpr int R = 128 * QT;
    static constexpr int STAGE = BN * D * 2;
    static constexpr int RAW = BN * D + BN * D / 16;
    static constexpr int Q_TILE = 128 * D * 2;
    static constexpr int Q = 0;
    static constexpr int RING = QT * Q_TILE;
    static constexpr int RAWS = RING + NS * STAGE;
    static constexpr int BARS = RAWS + NR * RAW;
    static constexpr int INFO = BARS + (8 * (2 * NS + 2 * NR + 20) + 8 + 15) / 16 * 16;
    // [64 bytes] flags, [2][24] items, [2][128] maxima and sums, [4] rows, the sequences
    static constexpr int SUMS = INFO + 64 + 2 * 96, SEQS = SUMS + 2 * 128 * 8 + 16;
    static constexpr int BYTES = SEQS + (int)sizeof(TreeSeq) * (tree_max_seq(D, Q8) + 1);
    static constexpr int O_COL = QT == 2 ? 256 : 128;  // S slots below it
    static constexpr int SLOT = QT == 2 ? 128 : 64;    // columns of an S slot
    // warps: softmax, then one that idles, scheduler, loader and MMA (beside the softmax warps of the last rows, which few
    // items have), then (Q8_0) eight that expand
    static constexpr int SOFTMAX = 4 * QT, PLAN_WARP = SOFTMAX + 1, LOAD_WARP = SOFTMAX + 2, MMA_WARP = SOFTMAX + 3, EXPAND_WARP = SOFTMAX + 4;
    static constexpr int EXPANDERS = Q8 ? 8 : 0;
    static constexpr int READERS = SOFTMAX + 2 + EXPANDERS;  // warps that follow the scheduler
    static constexpr int WARPS = SOFTMAX + 4 + EXPANDERS, THREADS = 32 * WARPS;
    // Registers a thread of each kind after the hand-over (their sum over the warps is what the launch gives them):
    // a softmax thread holds its row's 64 scores beside what masks, caps and biases them, and what it spills lies outside
    // what shared memory leaves of L1.
    static constexpr int LAUNCH_REGS = THREADS == 640 ? 96 : THREADS == 512 ? 128 : 168;
    static constexpr int SOFTMAX_REGS = !Q8 ? 208 : QT == 2 ? 136 : 232, MMA_REGS = !Q8 ? 88 : QT == 2 ? 80 : 88, EXPAND_REGS = QT == 2 ? 64 : 96;
    static constexpr bool HAND_OVER = QT == 2 || Q8;  // (else 8 warps, which have 255 each)
    static_assert(!HAND_OVER || SOFTMAX * SOFTMAX_REGS + 4 * MMA_REGS + EXPANDERS * EXPAND_REGS <= WARPS * LAUNCH_REGS,
                  "more registers than the launch has");
    static constexpr int64_t PART = (int64_t)R * (D + 2);  // of a partial: [D][R] values, [R] maxima, [R] sums
};

// What the scheduler tells the other warps of an item.
struct TreeItem {
    int nt;    // tiles of this part (0: no row sees a key; -1: no item is left)
    int t0;    // its first tile
    int slot;  // -1: the item is whole; else which of the CTA's partials
    int index, s, h, row0, rows, n_new, tok0, len, prefix;
    Tiles tiles;
    Visible seen;  // what some row sees lies in here
};
static_assert(sizeof(TreeItem) == 80, "read and written as 20 numbers, two items in shared memory");
__device__ __forceinline__ TreeItem tree_item(volatile const int* w) {
    TreeItem it;
    it.nt = w[0];
    it.t0 = w[1];
    it.slot = w[2];
    it.index = w[3];
    it.s = w[4];
    it.h = w[5];
    it.row0 = w[6];
    it.rows = w[7];
    it.n_new = w[8];
    it.tok0 = w[9];
    it.len = w[10];
    it.prefix = w[11];
    it.tiles.a0 = w[12];
    it.tiles.a1 = w[13];
    it.tiles.b0 = w[14];
    it.tiles.b1 = w[15];
    it.seen.first = w[16];
    it.seen.pre = w[17];
    it.seen.low = w[18];
    it.seen.end = w[19];
    return it;
}

// The parent of new token i (tok0: the sequence's first); below 0: none.  Chains end: one that does not go down is cut.
__device__ __forceinline__ int parent_of(const TreeParams& p, int tok0, int i) {
    const int a = __ldg(p.parents + tok0 + i);
    if (a >= i) {
        record_error(p.err, SYN_DEVERR_BOUNDS);
        return -1;
    }
    return a;
}
__device__ __forceinline__ int depth_of(const TreeParams& p, int tok0, int i) {
    int d = 0;
    for (int a = parent_of(p, tok0, i); a >= 0; a = parent_of(p, tok0, a)) d++;
    return d;
}
// The context's keys that a token at position pos sees.
__device__ __forceinline__ Visible visible_context(int context, int pos, int first, int prefix, int window) {
    Visible w;
    w.first = max(first, 0);
    w.end = max(context, 0);
    w.pre = min(prefix, w.end);
    w.low = w.first;
    if (window > 0) w.low = max(w.low, pos >= window ? pos - window + 1 : 0);
    return w;
}
// Calls f(key) for the keys of token i's chain that it sees and that are at least `from`, the nearest first.
template <typename F>
__device__ __forceinline__ void walk_chain(const TreeParams& p, int tok0, int i, int context, int from, F f) {
    for (int a = i, d = 0; a >= 0 && context + a >= from && (p.window == 0 || d < p.window); d++) {
        f(context + a);
        a = parent_of(p, tok0, a);
    }
}
// The tiles that some node of a sequence may see keys of: of the prefix from key `first` on, and from the widest
// window's first key to the end.
__device__ __forceinline__ Tiles tiles_of(const TreeParams& p, int len, int context, int first, int prefix, int BN) {
    const int pre = min(max(prefix, 0), max(context, 0)), from = max(first, 0);
    const int low = max(from, p.window > 0 ? max(context - p.window + 1, 0) : 0);
    Tiles t;
    t.b0 = low / BN;
    t.b1 = max(t.b0, len > low ? (len + BN - 1) / BN : t.b0);
    t.a0 = t.a1 = min(from / BN, t.b0);
    if (pre > from) t.a1 = min(max((min(pre, low) + BN - 1) / BN, t.a0), t.b0);
    return t;
}

__device__ __forceinline__ void store_out(const TreeParams& p, int64_t at, float y) {
    if (p.out_f16) static_cast<__half*>(p.out)[at] = __float2half_rn(y);
    else static_cast<float*>(p.out)[at] = y;
}

// The rows of `x`, a lane each, computed again in fp32 from the keys that they see in its tiles, 8 keys' scores at a
// time, then their values, which all lanes read together.  The sums are held in this lane's row of a partial (o: R
// rows, D values each, then maxima and sums), which is where a part's go in the end; else the outputs are written.  It
// ends where every sum is NaN, which nothing mends.
template <bool Q8>
__device__ __noinline__ void tree_rows_by_hand(const TreeParams& p, const TreeRedo& x, int BN, float* o, int R, int D) {
    const int lane = threadIdx.x & 31, dim = p.c.dim, shift = p.c.page_shift, mask = (1 << shift) - 1;
    const int64_t scales = (int64_t)dim << shift;  // Q8_0: where a tile's scales begin
    const bool mine = (x.bits >> lane) & 1;
    const int tok0 = p.starts[x.s], t = mine ? (x.row0 + lane) / p.g : 0, tok = tok0 + t;
    const int head = x.h * p.g + (mine ? x.row0 + lane - t * p.g : 0);
    const int len = held_rows(p.lens[x.s], p.max_pages, p.c.page_shift), context = len - new_tokens(p.starts, x.s, p.n_tok);
    const int pos = context + (mine && (p.window || p.slopes) ? depth_of(p, tok0, t) : 0);
    const Visible vis = visible_context(context, pos, p.first ? p.first[tok] : 0, p.prefix ? p.prefix[x.s] : 0, p.window);
    const int32_t* table = p.pages + (int64_t)x.s * p.max_pages;
    const __half* qrow = p.q + (int64_t)tok * p.q_stride + (int64_t)head * dim;
    const float slope = p.slopes ? p.slopes[head] : 0.0f;
    float m = -INFINITY, l = 0.0f;
    for (int e = 0; e < dim && mine; e++) o[(int64_t)e * R] = 0.0f;
    bool left = true;
    for (int64_t n = (int64_t)x.t0 * BN; n < (int64_t)x.t1 * BN && left; n += 8) {
        const int jb = x.tiles.at((int)(n / BN)) * BN + (int)(n % BN);
        uint32_t seen = mine ? (span_bits(vis.low - jb, vis.end - jb, 0) | span_bits(vis.first - jb, vis.pre - jb, 0)) & 0xffu : 0u;
        uint32_t chain = 0;  // those of the row's chain; nearer: keys of it past these 8
        int nearer = 0;
        if (mine && jb + 8 > context)
            walk_chain(p, tok0, t, context, max(jb, vis.first), [&](int key) {
                if (key < jb + 8) chain |= 1u << (key - jb);
                else nearer++;
            });
        seen |= chain;
        if (!__any_sync(0xffffffffu, seen != 0)) continue;
        const int id = table[jb >> shift];  // (8 keys lie in one page)
        if ((unsigned)id >= (unsigned)p.c.n_pages) continue;
        const int64_t tile = (int64_t)id * p.c.page_stride + (int64_t)x.h * p.c.tile, row = (int64_t)(jb & mask) * dim;
        float sc[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
        for (int e = 0; e < dim; e += 8) {
            float q[8];
            cached8<false>(reinterpret_cast<const uint8_t*>(qrow), 0, e, q);
#pragma unroll
            for (int c = 0; c < 8; c++) {
                float k[8];
                cached8<Q8>(p.c.k + tile, scales, row + c * dim + e, k);
#pragma unroll
                for (int i = 0; i < 8; i++) sc[c] = fmaf(q[i], k[i], sc[c]);
            }
        }
        float nm = m;
#pragma unroll
        for (int c = 0; c < 8; c++) {
            float y = sc[c] * p.scale;
            if (p.cap > 0.0f) y = p.cap * tanhf(y / p.cap);
            const int far = (chain >> c) & 1 ? nearer + __popc(chain >> (c + 1)) : pos - jb - c;
            y = fmaf(-slope, (float)far, y) * 1.4426950408889634f;
            sc[c] = (seen >> c) & 1 ? y : -INFINITY;
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
                cached8<Q8>(p.c.v + tile, scales, row + c * dim + e, v);
#pragma unroll
                for (int i = 0; i < 8; i++) acc[i] = (seen >> c) & 1 ? fmaf(sc[c], v[i], acc[i]) : acc[i];
            }
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (mine) o[(int64_t)(e + i) * R] = acc[i];
        }
    }
    if (!mine) return;
    if (x.slot >= 0) {
        o[(int64_t)D * R] = m;
        o[(int64_t)(D + 1) * R] = l;
    } else {
        const int64_t out0 = (int64_t)tok * p.out_stride + (int64_t)head * dim;
        for (int e = 0; e < dim; e++) store_out(p, out0 + e, l == 0.0f ? 0.0f : o[(int64_t)e * R] / l);
    }
}

// What happens to scores besides their scale: nothing, a cap, or all there is (biases, scales that are not positive).  A
// kernel with all of it is slower without it: the code that it jumps over (48 sequences over Q8_0, capped: 160 us,
// not 147).
enum { PLAIN = 0, CAPPED = 1, GENERAL = 2 };

template <int D, bool Q8, int MOD>
__global__ void __launch_bounds__(TreeShape<D, Q8>::THREADS, 1)
    k_attn_tree(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                const __grid_constant__ CUtensorMap qmap, const __grid_constant__ TreeParams p) {
    using L = TreeShape<D, Q8>;
    constexpr int QT = L::QT, BN = L::BN, NS = L::NS, NR = L::NR, R = L::R, THREADS = L::THREADS;
    constexpr int MMA_WARP = L::MMA_WARP, LOAD_WARP = L::LOAD_WARP, EXPAND_WARP = L::EXPAND_WARP;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BARS);
    uint64_t* kv_full = bars;
    uint64_t* kv_empty = kv_full + NS;
    uint64_t* s_full = kv_empty + NS;      // [2] S in its slot
    uint64_t* p_full = s_full + 2;         // [2][2] P of a slot's half
    uint64_t* o_done = p_full + 4;         // [2][2] a group's product P V is complete: of a tile's first half (its only one), its second
    uint64_t* q_full = o_done + 4;         // [2]
    uint64_t* q_empty = q_full + 2;        // [2] the item's last S is complete
    uint64_t* raw_full = q_empty + 2;      // [NR] Q8_0: codes and scales have arrived
    uint64_t* raw_empty = raw_full + NR;   // [NR]
    uint64_t* item_full = raw_empty + NR;  // [2]
    uint64_t* item_empty = item_full + 2;  // [2]
    uint64_t* meet_bar = item_empty + 2;   // the softmax warps
    uint64_t* mma_idle = meet_bar + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_idle + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* info = reinterpret_cast<int*>(smem + L::INFO);  // the scan's carry: [0] cost, [1] items, [2] the longest item
    volatile uint32_t* raw_there = reinterpret_cast<volatile uint32_t*>(info + 12);  // [NR] pieces that arrived
    volatile int* item_ints = info + 16;                                             // [2][24] items
    float2* sums = reinterpret_cast<float2*>(smem + L::SUMS);                        // [2][128] a group's maxima and sums
    volatile uint32_t* odd_rows = reinterpret_cast<volatile uint32_t*>(sums + 256);  // [4]
    TreeSeq* seqs = reinterpret_cast<TreeSeq*>(smem + L::SEQS);  // [n_seq], and the totals

    // (the shuffle tells the compiler that the warp's index is the same for its lanes)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int dim = p.c.dim, nh = (dim + 63) >> 6;  // 64-value column chunks of a row

    // ---- set-up that touches no global memory, ahead of the kernel before this one -----------
    if (tid == 0) {
        for (int i = 0; i < NS; i++) {
            mbar_init(smem_u32(&kv_full[i]), Q8 ? L::EXPANDERS : 1);
            mbar_init(smem_u32(&kv_empty[i]), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_u32(&s_full[i]), 1);
            mbar_init(smem_u32(&p_full[2 * i]), 4);
            mbar_init(smem_u32(&p_full[2 * i + 1]), 4);
            mbar_init(smem_u32(&o_done[2 * i]), 1);
            mbar_init(smem_u32(&o_done[2 * i + 1]), 1);
            mbar_init(smem_u32(&q_full[i]), p.q_tma ? 1 : 4);
            mbar_init(smem_u32(&q_empty[i]), 1);
            mbar_init(smem_u32(&item_full[i]), 1);
            mbar_init(smem_u32(&item_empty[i]), L::READERS);
        }
        for (int i = 0; i < NR; i++) {
            mbar_init(smem_u32(&raw_full[i]), 1);
            mbar_init(smem_u32(&raw_empty[i]), L::EXPANDERS);
        }
        mbar_init(smem_u32(mma_idle), 1);
        mbar_init(smem_u32(meet_bar), L::SOFTMAX);
        *abort_flag = 0;
        info[0] = info[1] = info[2] = 0;
        fence_mbar_init();
    }
    if (warp == MMA_WARP) tmem_alloc(smem_u32(tmem_slot), 512);
    if (warp == LOAD_WARP && lane < 3) prefetch_map(lane == 0 ? &kmap : lane == 1 ? &vmap : &qmap);
    griddep_release();
    griddep_wait();

    auto rows_tiles = [&](int n_new) { return (int)(((int64_t)n_new * p.g + R - 1) / R); };
    // Sequence s into its place: its items, what they cost (past 2^30: so much), the tiles of one.
    struct Work {
        int items, nt, cost;
    };
    auto work_of = [&](int s) {
        Work w{0, 0, 0};
        if (s >= p.n_seq) return w;
        // (all on their way together)
        const int tok0 = __ldcg(p.starts + s), tok1 = __ldcg(p.starts + s + 1), rows = __ldcg(p.lens + s);
        const int prefix = p.prefix ? __ldcg(p.prefix + s) : 0;
        const int n_new = tok0 < 0 || tok1 > p.n_tok ? 0 : max(tok1 - tok0, 0), len = held_rows(rows, p.max_pages, p.c.page_shift);
        int first = 0;
        if (p.first && n_new > 0) {
            first = INT_MAX;
            for (int t = tok0; t < tok0 + n_new; t++) first = min(first, p.first[t]);
        }
        seqs[s].first = first;
        seqs[s].tok0 = tok0;
        seqs[s].n_new = n_new;
        seqs[s].len = len;
        seqs[s].prefix = prefix;
        w.items = rows_tiles(n_new) * p.c.n_kv;
        w.nt = w.items ? tiles_of(p, len, len - n_new, first, prefix, BN).count() : 0;
        w.cost = (int)min((int64_t)w.items * (max(w.nt, 1) + TREE_ITEM), int64_t(1) << 30);
        return w;
    };
    // (sums past 2^31: no call comes to that many tiles but by sequences that share their pages; nothing is split then)
    auto add = [](int a, int b) { return (int)min((unsigned)a + (unsigned)b, 1u << 30); };
    auto scan = [&](Work& w) {  // over the warp's lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int c = __shfl_up_sync(0xffffffffu, w.cost, o), x = __shfl_up_sync(0xffffffffu, w.items, o);
            if (lane >= o) {
                w.cost = add(w.cost, c);
                w.items += x;
            }
        }
    };
    if (p.n_seq > 64) {  // (up to 64 sequences: the scheduler alone)
        __syncthreads();
        Work* of_warps = reinterpret_cast<Work*>(smem);  // (nothing else uses it yet)
        for (int base = 0; base < p.n_seq; base += THREADS) {
            const int s = base + tid;
            Work w = work_of(s);
            const int nt = __reduce_max_sync(0xffffffffu, w.nt);
            scan(w);
            if (lane == 31) of_warps[warp] = w;
            if (lane == 0) atomicMax(&info[2], nt);
            __syncthreads();
            int cost = info[0], items = info[1];
            for (int i = 0; i < warp; i++) {
                cost = add(cost, of_warps[i].cost);
                items += of_warps[i].items;
            }
            cost = add(cost, w.cost);
            items += w.items;
            if (s < p.n_seq) {
                seqs[s + 1].cost_before = cost;
                seqs[s + 1].items_before = items;
            }
            if (s == 0) seqs[0].cost_before = seqs[0].items_before = 0;
            __syncthreads();
            if (tid == THREADS - 1) {
                info[0] = cost;
                info[1] = items;
            }
            __syncthreads();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // the next item, for the warps that follow the scheduler; false: none is left, or a wait gave up
    int n_items = 0;
    auto next_item = [&](TreeItem& it) {
        const int slot = n_items & 1;
        if (!mbar_wait(smem_u32(&item_full[slot]), (n_items >> 1) & 1, p.err, abort_flag)) return false;
        it = tree_item(item_ints + 24 * slot);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&item_empty[slot]));
        n_items++;
        return it.nt >= 0;
    };
    // (what names the item's place in the call is fetched again at its end, which spares registers: the place is given
    // back then)
    auto hold_item = [&](TreeItem& it) {
        const int slot = n_items & 1;
        if (!mbar_wait(smem_u32(&item_full[slot]), (n_items >> 1) & 1, p.err, abort_flag)) return false;
        it = tree_item(item_ints + 24 * slot);
        return it.nt >= 0;
    };
    auto drop_item = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&item_empty[n_items & 1]));
        n_items++;
    };
    // two row tiles, a softmax group each; else one, and a half of each tile's keys each (D > 128: one group)
    auto two_tiles = [&](const TreeItem& it) { return QT == 2 && it.rows > 128; };
    // An item's tiles go up, or, with a bias by distance, from the last one down: the largest scores come
    // first, and O is not rescaled tile after tile.
    auto turn_tile = [&](int i, int nt) { return MOD == GENERAL && p.slopes ? nt - 1 - i : i; };

    // The ring's order: K of the first tile, then (two row tiles) V and the next K, or (one) the
    // next K and V.  Piece i of an item's 2*nt: is it V, and of which tile.
    auto piece_v = [&](int i, int nt, bool two) { return two ? (i & 1) : i == 2 * nt - 1 || (i > 0 && (i & 1) == 0); };
    auto piece_tile = [&](int i, int nt, bool two) { return two ? i >> 1 : i == 2 * nt - 1 ? nt - 1 : i == 0 ? 0 : (i & 1) ? (i + 1) >> 1 : (i >> 1) - 1; };

    if (warp < L::SOFTMAX) {
        // ------------------------------------ softmax ------------------------------------------
        if (L::HAND_OVER) take_registers<L::SOFTMAX_REGS>();
        const int st = warp >> 2;  // group
        const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t o_base = lane_base + L::O_COL + st * D;
        const float c_log2 = p.scale * 1.4426950408889634f;
        const float cap_log2 = p.cap * 1.4426950408889634f;
        // (finite however small the cap is: a score of 0 stays 0)
        const float to_cap = p.cap > 0.0f ? fminf(fmaxf(p.scale / p.cap, -1e38f), 1e38f) : 0.0f, to_cap2 = 2.0f * 1.4426950408889634f * to_cap;
        uint32_t uses = 0;                // bit x: the phase of S slot x
        int done = 0, done2 = 0;          // products P V of this group so far: of a tile's first half, of its second
        int q_turn = 0, meetings = 0;
        auto meet = [&]() {  // (bounded, as every wait: a warp may have given up)
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(meet_bar));
            return mbar_wait(smem_u32(meet_bar), meetings++ & 1, p.err, abort_flag);
        };
        int redo_list = -1;
        TreeItem it{};
        while (hold_item(it)) {
            const bool two = two_tiles(it), halves = QT == 2 && !two;  // (halves: of a tile's keys)
            const int r = two ? tid : tid & 127;                       // row of the item
            const bool row_ok = r < it.rows, idle = (r & ~31) >= it.rows;  // (idle: the whole warp has none)
            const int context = it.len - it.n_new;
            Visible vis;
            vis.first = vis.pre = vis.low = vis.end = 0;
            int pos = 0, node = 0;
            float slope = 0.0f;
            if (row_ok) {
                node = (it.row0 + r) / p.g;
                if (MOD == GENERAL && p.slopes) slope = p.slopes[it.h * p.g + (it.row0 + r - node * p.g)] * 1.4426950408889634f;
                pos = context + (p.window || (MOD == GENERAL && p.slopes) ? depth_of(p, it.tok0, node) : 0);
                vis = visible_context(context, pos, p.first ? p.first[it.tok0 + node] : 0, it.prefix, p.window);
            }
            auto place_of = [&](const TreeItem& it) {  // of this thread's row
                const int node = (it.row0 + r) / p.g;
                return make_int2(it.tok0 + node, it.h * p.g + (it.row0 + r - node * p.g));
            };
            if (it.nt == 0) {  // no row of the item sees a key
                const int2 at = place_of(it);
                if (row_ok && (two || st == 0))
                    for (int e = 0; e < dim; e++) store_out(p, (int64_t)at.x * p.out_stride + (int64_t)at.y * dim + e, 0.0f);
                drop_item();
                continue;
            }
            if (!p.q_tma && (two || st == 0)) {
                // this thread's Q row into shared memory, 16-byte piece j of chunk c at j ^ (row % 8)
                const int qt = two ? st : 0;
                if (!mbar_wait(smem_u32(&q_empty[qt]), (q_turn & 1) ^ 1, p.err, abort_flag)) break;
                uint8_t* qs = smem + L::Q + qt * L::Q_TILE + (tid & 127) * 128;
                const int2 place = place_of(it);
                const uint4* qrow = reinterpret_cast<const uint4*>(p.q + (int64_t)place.x * p.q_stride + (int64_t)place.y * dim);
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
            float m = -INFINITY, l = 0.0f;
            bool ok = true;
            for (int i = 0; i < it.nt && ok; i++) {
                const int slot = two ? st : i & 1;
                const uint32_t phase = (uses >> slot) & 1;
                uses ^= two ? 3u : 1u << slot;
                if (!(ok = mbar_wait(smem_u32(&s_full[slot]), phase, p.err, abort_flag))) break;
                tc_fence_after();
                for (int half = halves ? st : 0; half < (two ? 2 : halves ? st + 1 : 1); half++) {
                    const uint32_t s_base = lane_base + slot * L::SLOT + 64 * half;
                    const int j0 = it.tiles.at(it.t0 + turn_tile(i, it.nt)) * BN + 64 * half;
                    // the products into O so far: of the tile before, or of this one's first half
                    auto wait_o = [&]() {
                        if (two && half) return mbar_wait(smem_u32(&o_done[2 * st]), done & 1, p.err, abort_flag);
                        if (i == 0) return true;
                        return two ? mbar_wait(smem_u32(&o_done[2 * st + 1]), (done2 - 1) & 1, p.err, abort_flag)
                                   : mbar_wait(smem_u32(&o_done[2 * st]), (done - 1) & 1, p.err, abort_flag);
                    };
                    if (idle) {
                        if (!(ok = wait_o())) break;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&p_full[2 * slot + half]));
                        continue;
                    }
                    uint32_t v[64];
                    TMEM_LD32(s_base, v);
                    TMEM_LD32(s_base + 32, (v + 32));
                    const bool full = !row_ok || (j0 >= vis.low && j0 + 64 <= vis.end) || (j0 >= vis.first && j0 + 64 <= vis.pre);
                    const bool masked = !__all_sync(0xffffffffu, full);  // (the same for the warp)
                    // the keys of the row's chain, and how many of it are past these
                    uint32_t chain[2] = {0, 0};
                    int nearer = 0;
                    const bool drafts = j0 + 64 > context;
                    if (drafts && row_ok)
                        walk_chain(p, it.tok0, node, context, max(j0, vis.first), [&](int key) {
                            const int c = key - j0;
                            if (c >= 64) nearer++;
                            else if (c >= 32) chain[1] |= 1u << (c - 32);
                            else chain[0] |= 1u << c;
                        });
                    TMEM_LD_WAIT32(v);
                    TMEM_LD_WAIT32((v + 32));
                    if (MOD) {
                        if (MOD == CAPPED || p.cap > 0.0f) {
                            // Scores up to half the cap in size: tanh(y) = y times a polynomial in y^2, fitted on
                            // [0, 1/2] to 3e-7, the scale and the cap folded into its coefficients; past it the
                            // general form.  Each score goes by its own size, so that its bits do not depend on
                            // the others'; the vote only spares the general form where no score needs it.
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
                            for (int c = 0; c < 64; c += 2)
                                big = fmaxf(fmaxf(big, fabsf(__uint_as_float(v[c]))), fabsf(__uint_as_float(v[c + 1])));
                            if (__all_sync(0xffffffffu, big * to_half <= 0.5f)) {
                                // (eight pairs a step at a time: one after the other each waits for its own five)
#pragma unroll
                                for (int c = 0; c < 64; c += 16) {
                                    uint64_t x[8], z[8], y[8];
#pragma unroll
                                    for (int u = 0; u < 8; u++) x[u] = pack2(__uint_as_float(v[c + 2 * u]), __uint_as_float(v[c + 2 * u + 1]));
#pragma unroll
                                    for (int u = 0; u < 8; u++) z[u] = mul2(x[u], x[u]);
#pragma unroll
                                    for (int u = 0; u < 8; u++) y[u] = fma2(z[u], b3, b2);
#pragma unroll
                                    for (int u = 0; u < 8; u++) y[u] = fma2(z[u], y[u], b1);
#pragma unroll
                                    for (int u = 0; u < 8; u++) y[u] = fma2(z[u], y[u], b0);
#pragma unroll
                                    for (int u = 0; u < 8; u++) {
                                        const float2 r2 = unpack2(mul2(x[u], y[u]));
                                        v[c + 2 * u] = __float_as_uint(r2.x);
                                        v[c + 2 * u + 1] = __float_as_uint(r2.y);
                                    }
                                }
                            } else {
                                // cap*tanh(x/cap) = cap - 2 cap/(1 + 2^(2 x log2(e)/cap)), all in powers of two
                                const uint64_t k2 = pack2(to_cap2, to_cap2), one2 = pack2(1.0f, 1.0f);
                                const uint64_t m2 = pack2(-2.0f * cap_log2, -2.0f * cap_log2), cap2 = pack2(cap_log2, cap_log2);
#pragma unroll
                                for (int c = 0; c < 64; c += 2) {
                                    const float v0 = __uint_as_float(v[c]), v1 = __uint_as_float(v[c + 1]);
                                    const float2 r2 = small2(pack2(v0, v1)), y = unpack2(mul2(pack2(v0, v1), k2));
                                    const float2 z = unpack2(add2(pack2(ex2(y.x), ex2(y.y)), one2));
                                    const float2 x = unpack2(fma2(pack2(rcp(z.x), rcp(z.y)), m2, cap2));
                                    v[c] = __float_as_uint(fabsf(v0) * to_half <= 0.5f ? r2.x : x.x);
                                    v[c + 1] = __float_as_uint(fabsf(v1) * to_half <= 0.5f ? r2.y : x.y);
                                }
                            }
                        }
                        if (MOD == GENERAL) {
                            // (not capped: still to be scaled; c_log2 or 1)
                            const float to_scale = p.cap > 0.0f ? 1.0f : c_log2;
                            if (p.slopes && drafts) {  // (the context's keys by position, the chain's by how many of it are nearer)
#pragma unroll
                                for (int c = 0; c < 64; c++) {
                                    const int b = c & 31, of_chain = nearer + (c < 32 ? __popc(chain[1]) : 0) + (b < 31 ? __popc(chain[c >> 5] >> (b + 1)) : 0);
                                    const float by = (float)(j0 + c < context ? pos - j0 - c : of_chain);
                                    v[c] = __float_as_uint(fmaf(-slope, by, __uint_as_float(v[c]) * to_scale));
                                }
                            } else if (p.slopes) {
                                // the distance is far - c, two scores at a time (c counts in whole numbers, exactly)
                                const float far = (float)(pos - j0);
                                uint64_t c2 = pack2(0.0f, 1.0f);
                                const uint64_t two2 = pack2(2.0f, 2.0f), s2 = pack2(slope, slope), f2 = pack2(-slope * far, -slope * far);
                                const uint64_t l2 = pack2(to_scale, to_scale);
#pragma unroll
                                for (int c = 0; c < 64; c += 2) {
                                    const float2 x = unpack2(fma2(pack2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), l2, fma2(c2, s2, f2)));
                                    v[c] = __float_as_uint(x.x);
                                    v[c + 1] = __float_as_uint(x.y);
                                    c2 = add2(c2, two2);
                                }
                            } else if (!(p.cap > 0.0f)) {  // (a scale that is not positive)
#pragma unroll
                                for (int c = 0; c < 64; c++) v[c] = __float_as_uint(__uint_as_float(v[c]) * to_scale);
                            }
                        }
                    }
                    if (masked) {
#pragma unroll
                        for (int w = 0; w < 2; w++) {
                            const uint32_t bits = row_ok ? span_bits(vis.low - j0, vis.end - j0, w) | span_bits(vis.first - j0, vis.pre - j0, w) | chain[w]
                                                         : 0xffffffffu;
#pragma unroll
                            for (int c = 0; c < 32; c++)
                                if (!((bits >> c) & 1)) v[32 * w + c] = 0xff800000u;  // -inf
                        }
                    }
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 64; c += 8)
#pragma unroll
                        for (int u = 0; u < 4; u++)
                            m4[u] = fmaxf(fmaxf(m4[u], __uint_as_float(v[c + 2 * u])), __uint_as_float(v[c + 2 * u + 1]));
                    float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    if (!MOD) mx *= c_log2;
                    // the reference of the powers follows the maximum when that has grown by 2^8
                    const bool grow = mx > m + PRE_GROW_LOG2;  // (or is the first that is not -inf)
                    const float f = grow ? ex2(m - mx) : 1.0f;
                    if (grow) {
                        m = mx;
                        l *= f;
                    }
                    if ((i > 0 || (two && half)) && __any_sync(0xffffffffu, grow)) {
                        if (!(ok = wait_o())) break;
                        tc_fence_after();
                        for (int c = 0; c < dim; c += 16) {
                            uint32_t o[16];
                            TMEM_LD16(o_base + c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int u = 0; u < 16; u++) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
                            TMEM_ST16(o_base + c, o);
                        }
                        tmem_st_wait();
                    }
                    const float ms = (m == -INFINITY ? 0.0f : m) - PRE_P_LOG2;
                    const uint64_t c2 = pack2(MOD ? 1.0f : c_log2, MOD ? 1.0f : c_log2), ms2 = pack2(-ms, -ms);
                    uint64_t sum2[2] = {0, 0};
                    uint32_t pw[32];
#pragma unroll
                    for (int u = 0; u < 32; u++) {
                        const float2 x = unpack2(fma2(pack2(__uint_as_float(v[2 * u]), __uint_as_float(v[2 * u + 1])), c2, ms2));
                        const float a = ex2(x.x), e = ex2(x.y);
                        sum2[u & 1] = add2(sum2[u & 1], pack2(a, e));
                        const __half2 hh = __floats2half2_rn(a, e);
                        pw[u] = *reinterpret_cast<const uint32_t*>(&hh);
                    }
                    TMEM_ST32(s_base, pw);
                    const float2 sa = unpack2(add2(sum2[0], sum2[1]));
                    l += sa.x + sa.y;
                    // (no more than one product into O is outstanding: a parity tells neighbours apart)
                    if (!(ok = wait_o())) break;
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&p_full[2 * slot + half]));
                }
                done++;
                if (two) done2++;
            }
            if (!ok || !mbar_wait(smem_u32(two ? &o_done[2 * st + 1] : &o_done[2 * st]), (two ? done2 - 1 : done - 1) & 1, p.err, abort_flag)) break;
            tc_fence_after();
            // ---- the item's end: a row's values, from one accumulator or (halves) two ------------------
            it = tree_item(item_ints + 24 * (n_items & 1));
            drop_item();
            const int2 place = place_of(it);
            const int64_t out0 = (int64_t)place.x * p.out_stride + (int64_t)place.y * dim;
            float f0 = 1.0f, f1 = 0.0f, all_l = l, all_m = m;
            if (halves) {
                sums[st * 128 + r] = make_float2(m, l);
                if (!meet()) break;
                tc_fence_after();
                const float2 a = sums[r], b = sums[128 + r];
                all_m = fmaxf(a.x, b.x);
                const float ms = all_m == -INFINITY ? 0.0f : all_m;
                f0 = ex2(a.x - ms);
                f1 = ex2(b.x - ms);
                all_l = a.y * f0 + b.y * f1;
            }
            uint64_t odd2 = 0;  // 0 times every sum: NaN where one is not finite
            if (!idle) {
                const float inv = all_l == 0.0f ? 0.0f : 1.0f / all_l;
                float* part = p.part + ((int64_t)blockIdx.x * 3 + max(it.slot, 0)) * L::PART;
                const float scale0 = it.slot >= 0 ? f0 : f0 * inv, scale1 = it.slot >= 0 ? f1 : f1 * inv;
                for (int c = halves ? 32 * st : 0; c < dim; c += halves ? 64 : 32) {
                    uint32_t o[32];
                    __syncwarp();
                    if (halves) {
                        uint32_t o1[32];
                        TMEM_LD32(lane_base + L::O_COL + c, o);
                        TMEM_LD32(lane_base + L::O_COL + D + c, o1);
                        TMEM_LD_WAIT32(o);
                        TMEM_LD_WAIT32(o1);
#pragma unroll
                        for (int u = 0; u < 32; u += 2) {
                            const uint64_t x0 = pack2(__uint_as_float(o[u]), __uint_as_float(o[u + 1])), x1 = pack2(__uint_as_float(o1[u]), __uint_as_float(o1[u + 1]));
                            odd2 = fma2(x0, 0, odd2);
                            odd2 = fma2(x1, 0, odd2);
                            const float2 y = unpack2(fma2(x1, pack2(scale1, scale1), mul2(x0, pack2(scale0, scale0))));
                            o[u] = __float_as_uint(y.x);
                            o[u + 1] = __float_as_uint(y.y);
                        }
                    } else {
                        TMEM_LD32(o_base + c, o);
                        TMEM_LD_WAIT32(o);
#pragma unroll
                        for (int u = 0; u < 32; u += 2) {
                            const uint64_t x0 = pack2(__uint_as_float(o[u]), __uint_as_float(o[u + 1]));
                            odd2 = fma2(x0, 0, odd2);
                            const float2 y = unpack2(mul2(x0, pack2(scale0, scale0)));
                            o[u] = __float_as_uint(y.x);
                            o[u + 1] = __float_as_uint(y.y);
                        }
                    }
                    if (!row_ok) continue;
                    if (it.slot >= 0) {
#pragma unroll
                        for (int u = 0; u < 32; u++) __stcg(part + (int64_t)(c + u) * R + r, __uint_as_float(o[u]));
                    } else if (p.out_f16) {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<__half*>(p.out) + out0 + c);
#pragma unroll
                        for (int u = 0; u < 4; u++) {
                            uint32_t w[4];
#pragma unroll
                            for (int x = 0; x < 4; x++) {
                                const __half2 hh = __floats2half2_rn(__uint_as_float(o[8 * u + 2 * x]), __uint_as_float(o[8 * u + 2 * x + 1]));
                                w[x] = *reinterpret_cast<const uint32_t*>(&hh);
                            }
                            dst[u] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
                        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + out0 + c);
#pragma unroll
                        for (int u = 0; u < 8; u++)
                            dst[u] = make_float4(__uint_as_float(o[4 * u]), __uint_as_float(o[4 * u + 1]), __uint_as_float(o[4 * u + 2]),
                                                 __uint_as_float(o[4 * u + 3]));
                    }
                }
                __syncwarp();
                if (it.slot >= 0 && row_ok && (!halves || st == 0)) {
                    __stcg(part + (int64_t)D * R + r, all_m);
                    __stcg(part + (int64_t)(D + 1) * R + r, all_l);
                }
            }
            // Rows whose weighted values are not finite are computed again: a value that the row does not see may have
            // come in as 0 * inf.  Where the sum of the weights is not finite itself a score that the row sees is
            // not, and its outputs are NaN as they are; but over Q8_0 the key may only have been past what fp16
            // holds.  (And where scores are in the millions: the powers take scores times the scale, unrounded,
            // less a rounded maximum, and what lies between the two has to stay well below 1.)
            const float2 odd = unpack2(odd2);
            const bool odd_l = !(all_l * 0.0f == 0.0f), odd_o = !(odd.x + odd.y == 0.0f);
            const bool far = !MOD && fabsf(all_m) > 0x1p22f && fabsf(all_m) < INFINITY;
            uint32_t redo = __ballot_sync(0xffffffffu, row_ok && (far || (odd_l ? Q8 : odd_o)));
            tc_fence_before();
            if (halves) {
                if (st == 1 && lane == 0) odd_rows[warp & 3] = redo;
                if (!meet()) break;  // (and the next item's products may overwrite the accumulators)
                if (st == 1) continue;
                redo |= odd_rows[warp & 3];
            }
            if (redo) {
                const int64_t at = it.slot < 0 ? (int64_t)it.index * (R / 32) + warp : p.n_redo + ((int64_t)blockIdx.x * 2 + it.slot) * (R / 32) + warp;
                if (it.slot >= 0 || at < p.n_redo) {  // (more items than that only where starts[] does not ascend)
                    if (lane == 0)
                        p.redo[at] = TreeRedo{it.s, it.h, it.row0 + 32 * warp, redo, it.tiles, it.slot >= 0 ? it.t0 : 0,
                                              it.slot >= 0 ? it.t0 + it.nt : it.tiles.count(), it.slot, redo_list};
                    redo_list = (int)at;
                }
            }
        }
        __syncwarp();
        while (redo_list >= 0) {
            const TreeRedo x = p.redo[redo_list];
            // (row r of a part is row r of its partial; of a whole item the sums' place is the CTA's third)
            float* o = p.part + ((int64_t)blockIdx.x * 3 + (x.slot >= 0 ? x.slot : 2)) * L::PART + tid;
            tree_rows_by_hand<Q8>(p, x, BN, o, R, D);
            redo_list = x.next;
        }
    } else if (warp < EXPAND_WARP) {
      if (L::HAND_OVER) give_registers<L::MMA_REGS>();
      if (warp == MMA_WARP) {
        // ------------------------------------ MMA ----------------------------------------------
        int rc = 0;                        // ring pieces taken so far
        uint32_t uses = 0;                 // bit x: the phase of S slot x
        int q_turn[2] = {0, 0};
        bool ok = true;
        TreeItem it{};
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
        // a group's O += P V with the 64 keys of a slot's half, from piece i
        auto issue_o = [&](int group, int slot, int half, int i, uint32_t phase, bool first, int done) {
            const uint64_t vd = n_major + ((ring_s + (i % NS) * L::STAGE) >> 4);
            if (!mbar_wait(smem_u32(&p_full[2 * slot + half]), phase, p.err, abort_flag)) return false;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; k++)
                mma_f16_ts_lead(lead, tmem + L::O_COL + group * D, tmem + slot * L::SLOT + 64 * half + 8 * k, vd + ((4 * half + k) * 2048 >> 4), p.idesc_o,
                                !first || k > 0);
            mma_commit_lead(lead, smem_u32(&o_done[2 * group + done]));
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
            const int nt = it.nt;
            const bool two = two_tiles(it);
            if (nt == 0) continue;
            ok = mbar_wait(smem_u32(&q_full[0]), q_turn[0]++ & 1, p.err, abort_flag);
            if (two) ok = ok && mbar_wait(smem_u32(&q_full[1]), q_turn[1]++ & 1, p.err, abort_flag);
            if (!ok || !(ok = take(rc))) break;
            // (S of the first tile goes where P of the last item's last tile was: in order behind its product)
            issue_s(0, 0, rc);
            if (two) issue_s(1, 1, rc);
            if (nt == 1) {
                mma_commit_lead(lead, smem_u32(&q_empty[0]));
                if (two) mma_commit_lead(lead, smem_u32(&q_empty[1]));
            }
            release(rc);
            rc++;
            for (int i = 0; i < nt && ok; i++) {
                if (two) {
                    const int pv = rc, pk = rc + 1;
                    if (!(ok = take(pv))) break;
                    clean(pv, i);
                    if (i + 1 < nt && !(ok = take(pk))) break;
#pragma unroll
                    for (int qt = 0; qt < 2; qt++) {
                        const uint32_t phase = (uses >> qt) & 1;
                        uses ^= 1u << qt;
                        if (!ok) continue;
                        ok = issue_o(qt, qt, 0, pv, phase, i == 0, 0) && issue_o(qt, qt, 1, pv, phase, false, 1);
                        if (!ok) continue;
                        if (i + 1 < nt) issue_s(qt, qt, pk);
                        if (i + 2 == nt) mma_commit_lead(lead, smem_u32(&q_empty[qt]));
                    }
                    if (!ok) break;
                    release(pv);
                    if (i + 1 < nt) release(pk);
                    rc = i + 1 < nt ? pk + 1 : pv + 1;
                } else {
                    const int slot = i & 1;
                    if (i + 1 < nt) {
                        if (!(ok = take(rc))) break;
                        issue_s(0, slot ^ 1, rc);
                        if (i + 2 == nt) mma_commit_lead(lead, smem_u32(&q_empty[0]));
                        release(rc);
                        rc++;
                    }
                    if (!(ok = take(rc))) break;
                    clean(rc, i);
                    const uint32_t phase = (uses >> slot) & 1;
                    uses ^= 1u << slot;
                    ok = issue_o(0, slot, 0, rc, phase, i == 0, 0);
                    if (QT == 2) ok = ok && issue_o(QT - 1, slot, 1, rc, phase, i == 0, 0);
                    if (!ok) break;
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
        TreeItem it{};
        while (ok && next_item(it)) {
            if (it.nt == 0) continue;
            const bool two = two_tiles(it);
#ifdef SYN_TEST_STALL
            const int n_pieces = 0;  // timeout-test build: no tile is ever loaded, so the waits run out
#else
            const int n_pieces = 2 * it.nt;
#endif
            const int32_t* table = p.pages + (int64_t)it.s * p.max_pages;
            auto first_key = [&](int i) { return it.tiles.at(it.t0 + turn_tile(piece_tile(i, it.nt, two), it.nt)) * BN + lane * box; };  // of this lane's box
            auto look_up = [&](int i) {  // the page (asked for a piece ahead)
                const int j = i < n_pieces ? first_key(i) : INT_MAX;
                return lane < n_box && j < it.len ? __ldg(table + (j >> p.c.page_shift)) : -1;
            };
            int entry = look_up(0);
            if (p.q_tma) {
                // 128 / g tokens of g heads: the row order of the item.  (Tokens past the call's are zeros;
                // those of the next sequence are rows that nobody writes.)
#pragma unroll
                for (int qt = 0; qt < QT; qt++) {
                    if ((qt && !two) || !ok) continue;
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
            for (int i = 0; i < n_pieces && ok; i++, kc++) {
                const int st = Q8 ? kc % max(NR, 1) : kc % NS;
                const uint32_t turn = (uint32_t)(Q8 ? kc / max(NR, 1) : kc / NS);
                const bool is_v = piece_v(i, it.nt, two);
                const int j = first_key(i), after = look_up(i + 1);
                int id = -1;  // past the end, or an id outside the pool
                if (lane < n_box && j < it.len) {
                    if ((unsigned)entry < (unsigned)p.c.n_pages) id = entry;
                    else if (it.seen.any(j, j + box)) record_error(p.err, SYN_DEVERR_BOUNDS);  // (else it may be gone)
                }
                entry = after;
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
        // (Much of what a small call takes passes here, ahead of the first load, and most of that in fetching code
        // that runs once: what the first item needs comes first, without a division that a sum can spare.)
        int longest = info[2];
        if (p.n_seq <= 64) {
            int cost = 0, items = 0;
            if (lane == 0) seqs[0].cost_before = seqs[0].items_before = 0;
#pragma unroll 1
            for (int base = 0; base < p.n_seq; base += 32) {
                Work w = work_of(base + lane);
                longest = max(longest, __reduce_max_sync(0xffffffffu, w.nt));
                scan(w);
                if (base + lane < p.n_seq) {
                    seqs[base + lane + 1].cost_before = add(cost, w.cost);
                    seqs[base + lane + 1].items_before = items + w.items;
                }
                cost = add(cost, __shfl_sync(0xffffffffu, w.cost, 31));
                items += __shfl_sync(0xffffffffu, w.items, 31);
            }
            __syncwarp();
        }
        const int total = seqs[p.n_seq].cost_before, items = seqs[p.n_seq].items_before, ctas = (int)gridDim.x;
        // Ranges of `range` tiles, or whole items in turn: where nothing may be split, or splitting would not pay.
        const int range = max((total + ctas - 1) / ctas, 1);
        const bool whole = !p.split || total >= 1 << 30 || (items <= ctas && longest + TREE_ITEM <= range + TREE_JOIN);
        int64_t at = whole ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * range;  // an item's number, or a place in the work
        const int64_t to = whole ? (int64_t)items : min(at + range, (int64_t)total);
        for (int n = 0;;) {
            TreeItem it{};
            it.nt = -1;
            it.slot = -1;
            int rest = 0;  // tiles of an item that others go on with
            if (at < to) {
                int lo = 0;  // the sequence: 32 at a time
                for (uint32_t past = 0; !past; lo += past ? __ffs(past) - 1 : 32) {
                    const TreeSeq* q = &seqs[min(lo + lane, p.n_seq - 1) + 1];
                    past = __ballot_sync(0xffffffffu, (whole ? q->items_before : q->cost_before) > (int)at);
                }
                const TreeSeq q = seqs[lo];
                it.s = lo;
                it.n_new = q.n_new;
                it.tok0 = q.tok0;
                it.len = q.len;
                it.prefix = q.prefix;
                const int pos0 = it.len - it.n_new;
                it.tiles = tiles_of(p, it.len, pos0, q.first, it.prefix, BN);
                const int nt = it.tiles.count(), tiles_q = rows_tiles(it.n_new);
                const int each = max(nt, 1) + TREE_ITEM, within = whole ? (int)at - q.items_before : ((int)at - q.cost_before) / each;
                it.index = q.items_before + within;
                it.h = tiles_q == 1 ? within : within / tiles_q;
                it.row0 = (within - it.h * tiles_q) * R;
                it.rows = (int)min((int64_t)R, (int64_t)it.n_new * p.g - it.row0);
                bool mine = true;  // (else: only the cost of the item's end lies in this range)
                if (whole) {
                    it.nt = nt;
                    at += ctas;
                } else {
                    const int begin = q.cost_before + within * each, from = (int)at - begin;
                    it.t0 = min(from, nt);
                    it.nt = min(from + (int)(to - at), nt) - it.t0;
                    mine = nt > 0 ? it.nt > 0 : from == 0;
                    rest = nt - it.t0 - it.nt;
                    if (mine && (it.t0 > 0 || rest > 0)) it.slot = it.t0 > 0 ? 0 : 1;
                    at = min((int64_t)begin + each, to);
                }
                if (!mine) continue;
                if (n == 0) {  // the loader's first look at the page table, ahead of it
                    const int j = it.tiles.at(it.t0) * BN + lane * min(BN, 1 << p.c.page_shift);
                    if (it.nt > 0 && lane * min(BN, 1 << p.c.page_shift) < BN && j < it.len)
                        asm volatile("{\n\t.reg .b32 x;\n\tld.global.ca.b32 x, [%0];\n\t}" ::"l"(p.pages + (int64_t)it.s * p.max_pages + (j >> p.c.page_shift)));
                }
                // [mf, pre) and [ml, me): every key that some row sees lies in one of them
                const int pre_end = min(max(it.prefix, 0), max(pos0, 0));
                int mf = INT_MAX, ml = INT_MAX, me = 0;
                if (p.first || p.window) {
                    const int tk0 = it.row0 / p.g, tk1 = (it.row0 + it.rows - 1) / p.g;  // first and last token
                    for (int t = tk0 + lane; t <= tk1; t += 32) {
                        const Visible v = visible_context(pos0, p.window ? pos0 + depth_of(p, it.tok0, t) : pos0,
                                                          p.first ? p.first[it.tok0 + t] : 0, it.prefix, p.window);
                        const int chain = max(max(pos0, v.first), 0);  // (its chain lies between here and its own row)
                        if (v.end > v.low) {
                            ml = min(ml, v.low);
                            me = max(me, v.end);
                        }
                        if (pos0 + t >= chain) {
                            ml = min(ml, chain);
                            me = max(me, pos0 + t + 1);
                        }
                        if (v.pre > v.first) mf = min(mf, v.first);
                    }
                    mf = __reduce_min_sync(0xffffffffu, mf);
                    ml = __reduce_min_sync(0xffffffffu, ml);
                    me = __reduce_max_sync(0xffffffffu, me);
                } else {
                    ml = 0;
                    me = it.len;
                    mf = pre_end > 0 ? 0 : INT_MAX;
                }
                it.seen.first = min(mf, ml);
                it.seen.pre = mf == INT_MAX ? 0 : pre_end;
                it.seen.low = ml;
                it.seen.end = me;
            }
            const int slot = n & 1;
            if (!mbar_wait(smem_u32(&item_empty[slot]), ((n >> 1) & 1) ^ 1, p.err, abort_flag)) break;
            if (lane == 0) {
                const int o[20] = {it.nt, it.t0, it.slot, it.index, it.s, it.h, it.row0, it.rows, it.n_new, it.tok0, it.len, it.prefix,
                                   it.tiles.a0, it.tiles.a1, it.tiles.b0, it.tiles.b1, it.seen.first, it.seen.pre, it.seen.low, it.seen.end};
#pragma unroll
                for (int i = 0; i < 20; i++) item_ints[24 * slot + i] = o[i];
                mbar_arrive(smem_u32(&item_full[slot]));
            }
            if (it.slot == 1 && lane == 0) {  // (its first part)
                const unsigned long long tasks = (unsigned long long)((it.rows + 31) / 32 * (dim / JOIN_VALUES));
                const unsigned long long before = atomicAdd(reinterpret_cast<unsigned long long*>(p.n_splits), (1ull << 32) + tasks);
                const int x = (int)(before >> 32);
                if (x < ctas)  // (each end of a range splits one at most)
                    p.splits[x] = TreeSplit{it.tok0, it.h, it.row0, it.rows, (int)blockIdx.x, 1 + (rest + range - 1) / range, (int)before, 0};
            }
            __syncwarp();
            n++;
            if (it.nt == -1) break;
        }
      }
    } else if (Q8) {
        // ------------------------------------ expand (Q8_0) -------------------------------------
        if (L::EXPAND_REGS < L::LAUNCH_REGS) give_registers<L::EXPAND_REGS>();
        const int lt = tid - 32 * EXPAND_WARP;
        // 16 codes at a time.  A thread takes piece x4 of the 64-value chunks of rows lt/4, lt/4 + ROWS, ...;
        // neighbouring rows take the chunks in opposite order, so that the 8 lanes that a shared-memory
        // access serves at once touch all the banks, reading and storing.
        constexpr int ROWS = 8 * L::EXPANDERS, HALVES = D / 64, UNITS = BN / (Q8 ? ROWS : BN) * HALVES;  // (ROWS: a pass)
        const int x4 = lt & 3, row_t = lt >> 2;
        const int box_shift = min(p.c.page_shift, BN == 128 ? 7 : 6), n_box = BN >> box_shift;
        const uint32_t all_there = n_box == 32 ? 0xffffffffu : (1u << n_box) - 1u;
        const __half2 k1152 = __float2half2_rn(1152.0f);
        int kc = 0;
        bool ok = true;
        TreeItem it{};
        while (ok && next_item(it)) {
            const bool two = two_tiles(it);
#ifdef SYN_TEST_STALL
            const int n_pieces = 0;
#else
            const int n_pieces = 2 * it.nt;
#endif
            for (int i = 0; i < n_pieces && ok; i++, kc++) {
                const int rs = kc % max(NR, 1), st = kc % NS;
                if (!(ok = mbar_wait(smem_u32(&raw_full[rs]), (kc / max(NR, 1)) & 1, p.err, abort_flag))) break;
                if (!(ok = mbar_wait(smem_u32(&kv_empty[st]), ((kc / NS) & 1) ^ 1, p.err, abort_flag))) break;
                const int left = it.len - it.tiles.at(it.t0 + turn_tile(piece_tile(i, it.nt, two), it.nt)) * BN;  // rows of the tile that exist
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
                            code[u] = *reinterpret_cast<const uint4*>(codes + ru * (ROWS * D) + 64 * half);
                            bits[u] = *reinterpret_cast<const uint16_t*>(scales + ru * (ROWS * D / 16) + 4 * half);
                        }
#pragma unroll
                        for (int u = 0; u < BATCH; u++) {
                            const int ru = (u0 + u) / HALVES, half = HALVES > 1 ? ((u0 + u) % HALVES) ^ odd : 0;
                            put(dst + half * (BN * 128) + ru * (ROWS * 128), code[u], bits[u]);
                        }
                    }
                } else {  // rows that are not there are zeros
                    for (int u = 0; u < UNITS; u++) {
                        const int half = HALVES > 1 ? (u % HALVES) ^ (row_t & 1) : 0, x = x4 + 4 * half, row = row_t + ROWS * (u / HALVES);
                        if (half >= nh) continue;
                        uint4 code = make_uint4(0, 0, 0, 0);
                        uint32_t bits = 0;
                        if (16 * x < dim && row < left && ((there >> (row >> box_shift)) & 1)) {
                            code = *reinterpret_cast<const uint4*>(raw + row * dim + 16 * x);
                            bits = *reinterpret_cast<const uint16_t*>(raw + BN * D + 2 * (row * (dim >> 5) + (x >> 1)));
                        }
                        put(dst + half * (BN * 128) + (u / HALVES) * (ROWS * 128), code, bits);
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

// ---- the join of split items ---------------------------------------------------------------
//
// A warp joins 4 values of 32 rows of an item: the parts' weights from their maxima and sums, with their values, four
// parts' loads on their way together.
constexpr int JOIN_THREADS = 256, JOIN_MOST = 1024, JOIN_PARTS = 4, JOIN_CTAS = 4;

struct JoinParams {
    const float* part;
    const TreeSplit* splits;
    int* n_splits;
    void* out;
    int64_t out_stride, part_floats;  // of a partial
    int R, D, dim, g, out_f16, ctas;  // ctas: of the first kernel
};

__global__ void __launch_bounds__(JOIN_THREADS, JOIN_CTAS) k_attn_tree_join(const JoinParams p) {
    __shared__ int before[JOIN_MOST];
    griddep_release();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chunks = p.dim / JOIN_VALUES;
    const int tasks = const_cast<volatile int*>(p.n_splits)[0], n = min(const_cast<volatile int*>(p.n_splits)[1], JOIN_MOST);
    for (int i = threadIdx.x; i < n; i += JOIN_THREADS) before[i] = p.splits[i].before;
    __syncthreads();
    for (int u = blockIdx.x * (JOIN_THREADS / 32) + warp; u < tasks; u += gridDim.x * (JOIN_THREADS / 32)) {
        int lo = 0, hi = n;  // the last item whose tasks begin at u or before it
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before[mid] <= u) lo = mid;
            else hi = mid;
        }
        const TreeSplit x = p.splits[lo];
        const int row = (u - x.before) / chunks * 32 + lane, e0 = (u - x.before) % chunks * JOIN_VALUES;
        if (!SYN_IN_BOUNDS(u >= x.before && x.parts >= 1 && x.first >= 0 && x.first + x.parts <= p.ctas && row < p.R)) continue;
        // part i: what the CTA first + i went on with; of the first what it began
        auto part = [&](int i) { return p.part + ((int64_t)(x.first + i) * 3 + (i == 0)) * p.part_floats + row; };
        float mx = -INFINITY, sum = 0.0f, acc[JOIN_VALUES];
#pragma unroll
        for (int e = 0; e < JOIN_VALUES; e++) acc[e] = 0.0f;
        for (int i0 = 0; i0 < x.parts; i0 += JOIN_PARTS) {  // (the last batch repeats the last part's loads)
            float m[JOIN_PARTS], l[JOIN_PARTS], o[JOIN_PARTS][JOIN_VALUES];
#pragma unroll
            for (int i = 0; i < JOIN_PARTS; i++) {
                const float* q = part(min(i0 + i, x.parts - 1));
                m[i] = __ldcg(q + (int64_t)p.D * p.R);
                l[i] = __ldcg(q + (int64_t)(p.D + 1) * p.R);
#pragma unroll
                for (int e = 0; e < JOIN_VALUES; e++) o[i][e] = __ldcg(q + (int64_t)(e0 + e) * p.R);
            }
            float nm = mx;
#pragma unroll
            for (int i = 0; i < JOIN_PARTS; i++) {
                if (i0 + i >= x.parts) m[i] = -INFINITY;
                nm = fmaxf(nm, m[i]);
            }
            const float ms = nm == -INFINITY ? 0.0f : nm, f = ex2(mx - ms);
            mx = nm;
            sum *= f;
#pragma unroll
            for (int e = 0; e < JOIN_VALUES; e++) acc[e] *= f;
#pragma unroll
            for (int i = 0; i < JOIN_PARTS; i++) {
                if (i0 + i >= x.parts) continue;
                const float w = ex2(m[i] - ms);
                sum = fmaf(l[i], w, sum);
#pragma unroll
                for (int e = 0; e < JOIN_VALUES; e++) acc[e] = fmaf(o[i][e], w, acc[e]);
            }
        }
        if (row >= x.rows) continue;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const int t = (x.row0 + row) / p.g;
        const int64_t at = (int64_t)(x.tok0 + t) * p.out_stride + (int64_t)(x.h * p.g + x.row0 + row - t * p.g) * p.dim + e0;
        if (p.out_f16) {
            const __half2 a = __floats2half2_rn(acc[0] * inv, acc[1] * inv), b = __floats2half2_rn(acc[2] * inv, acc[3] * inv);
            *reinterpret_cast<uint2*>(static_cast<__half*>(p.out) + at) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
        } else {
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
        }
    }
    // the last CTA to get here makes the count ready for the next call
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(p.n_splits + 2, 1) == (int)gridDim.x - 1) p.n_splits[0] = p.n_splits[1] = p.n_splits[2] = 0;
}

// ---- host side ---------------------------------------------------------------------------

template <int D, bool Q8, int MOD>
static cudaError_t run_tree(const CUtensorMap& km, const CUtensorMap& vm, const CUtensorMap& qm, const TreeParams& p, int grid, cudaStream_t s) {
    auto kern = k_attn_tree<D, Q8, MOD>;
    constexpr int smem = 1024 + TreeShape<D, Q8>::BYTES;
    static_assert(smem <= 232448, "shared memory per CTA exceeds 227 KB");
    static ResidentCtas resident;
    int n;
    cudaError_t e = resident.get(reinterpret_cast<const void*>(kern), TreeShape<D, Q8>::THREADS, smem, &n);
    if (e != cudaSuccess) return e;
    if (TreeShape<D, Q8>::HAND_OVER) {
        // the hand-over of registers deals out what the launch has: a build with fewer must not start
        static const int regs = [&] {
            cudaFuncAttributes a;
            return cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(kern)) == cudaSuccess ? a.numRegs : 0;
        }();
        if (regs < TreeShape<D, Q8>::LAUNCH_REGS) return cudaErrorInvalidConfiguration;
    }
    return launch_overlapped(kern, grid, TreeShape<D, Q8>::THREADS, smem, s, km, vm, qm, p);
}

static int tree_rows(int dim) { return dim <= 128 ? 256 : 128; }
static int tree_width(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
static int64_t tree_partial(int dim) { return (int64_t)tree_rows(dim) * (tree_width(dim) + 2); }
// an entry for each 32 rows of an item (a power of two: a growing batch seldom needs more than the last)
static int64_t tree_redo(int64_t n_seq, int64_t n_tok, int n_heads, int n_kv, int dim) {
    const int R = tree_rows(dim);
    const int64_t need = (n_tok * (n_heads / n_kv) / R + std::min<int64_t>({n_seq, n_tok, 512})) * n_kv * (R / 32);
    int64_t n = 4096;
    while (n < need) n *= 2;
    return n;
}
int64_t tree_part_floats(int64_t n_seq, int64_t n_tok, int n_heads, int n_kv, int dim, int sms) {
    const int64_t redo = tree_redo(n_seq, n_tok, n_heads, n_kv, dim) + (int64_t)sms * 2 * (tree_rows(dim) / 32);
    return 3 * sms * tree_partial(dim) + redo * (int64_t)(sizeof(TreeRedo) / 4) + sms * (int64_t)(sizeof(TreeSplit) / 4);
}

cudaError_t launch_attn_tree(const KvCache& c, const AttnDesc& a, int64_t n_seq, int64_t n_tok, const void* q,
                             const int32_t* starts, const int32_t* parents, const int32_t* pages, int64_t max_pages,
                             const int32_t* lens, void* out, float* part, int* count, bool split, int* err, int sms,
                             int* launches, cudaStream_t s) {
    if (sms > JOIN_MOST) return cudaErrorInvalidConfiguration;
    CUtensorMap km, vm, qm;
    const int D = tree_width(c.dim), BN = D <= 128 ? 128 : 64, R = tree_rows(c.dim);
    PFN_encodeTiled encode = get_encode();
    if (!encode) return cudaErrorNotSupported;
    const int g = a.n_heads / c.n_kv;
    const bool q_tma = g <= 128 && 128 % g == 0;
    qm = CUtensorMap{};  // (unused else)
    if (q_tma) {
        cuuint64_t dims[3] = {(cuuint64_t)c.dim, (cuuint64_t)a.n_heads, (cuuint64_t)n_tok};
        cuuint64_t strides[2] = {(cuuint64_t)c.dim * 2, (cuuint64_t)a.q_stride * 2};
        cuuint32_t box[3] = {64, (cuuint32_t)g, (cuuint32_t)(128 / g)}, estr[3] = {1, 1, 1};
        if (encode(&qm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(q), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
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
    TreeParams p;
    p.c = c;
    p.q = static_cast<const __half*>(q);
    p.q_stride = a.q_stride;
    p.out_stride = a.out_stride;
    p.out = out;
    p.max_pages = max_pages;
    p.slopes = a.slopes;
    p.first = a.first;
    p.parents = parents;
    p.part = part;
    p.n_redo = tree_redo(n_seq, n_tok, a.n_heads, c.n_kv, c.dim);
    p.redo = reinterpret_cast<TreeRedo*>(part + 3 * sms * tree_partial(c.dim));
    p.splits = reinterpret_cast<TreeSplit*>(p.redo + p.n_redo + (int64_t)sms * 2 * (R / 32));
    p.n_splits = count;
    p.err = err;
    p.scale = a.scale;
    p.cap = a.cap;
    p.n_tok = (int)n_tok;
    p.g = g;
    p.q_tma = q_tma;
    p.window = a.window;
    p.out_f16 = a.out_f16;
    // (many: items for more than half the SMs, at least)
    p.split = split && (max_pages << c.page_shift) > (int64_t)tree_whole(D, c.page_shift >= 6, 2 * n_seq * c.n_kv > sms) * BN;
    // kind::f16: D fp32, A and B fp16, M = 128; S: B K-major, N = BN; O: B MN-major, N = dim
    p.idesc_s = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | (8u << 24);
    p.idesc_o = (1u << 4) | (1u << 16) | ((uint32_t)(c.dim >> 3) << 17) | (8u << 24);
    // (a scale that is not positive takes the general path: the fast one scales the maximum)
    const int mod = a.slopes || !(a.scale > 0.0f) ? GENERAL : a.cap > 0.0f ? CAPPED : PLAIN;
    const JoinParams j{part, p.splits, p.n_splits, out, a.out_stride, tree_partial(c.dim), R, D, c.dim, g, a.out_f16, sms};
    const int most = tree_max_seq(D, c.q8);
    for (int64_t s0 = 0; s0 < n_seq; s0 += most) {
        p.n_seq = (int)std::min<int64_t>(most, n_seq - s0);
        p.starts = starts + s0;
        p.pages = pages + s0 * max_pages;
        p.lens = lens + s0;
        p.prefix = a.prefix ? a.prefix + s0 : nullptr;
        // (more items than this many have a row number past 32 bits)
        if (((n_tok * p.g + R - 1) / R + p.n_seq) * c.n_kv > INT_MAX) return cudaErrorInvalidValue;
        cudaError_t e;
#define SYN_TREE_MOD(D, Q8)                                                    \
    (mod == PLAIN    ? run_tree<D, Q8, PLAIN>(km, vm, qm, p, sms, s)           \
     : mod == CAPPED ? run_tree<D, Q8, CAPPED>(km, vm, qm, p, sms, s)          \
                     : run_tree<D, Q8, GENERAL>(km, vm, qm, p, sms, s))
#define SYN_TREE(D) (c.q8 ? SYN_TREE_MOD(D, true) : SYN_TREE_MOD(D, false))
        e = D == 64 ? SYN_TREE(64) : D == 128 ? SYN_TREE(128) : SYN_TREE(256);
#undef SYN_TREE
#undef SYN_TREE_MOD
        if (e != cudaSuccess) return e;
        ++*launches;
        if (!p.split) continue;
        e = launch_overlapped(k_attn_tree_join, JOIN_CTAS * sms, JOIN_THREADS, 0, s, j);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    return cudaSuccess;
}

#ifdef SYN_DEBUG
SYN_BOUNDS_READER(debug_bounds_attn_tree)
#endif

}  // namespace syn
