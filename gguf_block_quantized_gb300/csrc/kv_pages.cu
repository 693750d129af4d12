// kv_pages.cu — the pages of a paged cache as sequences hold them: forked, extended, packed, given back
// and copied.
//
// refs[page] counts the page-table entries that hold the page; 0: free.  Pages are taken lowest first,
// in the order of sequences and columns, so that what a call does depends on its arguments alone,
// whatever the order of the atomics.
//
// Bound: the tables are a few KB, so fork, extend and trim are their launches' latency and a chain of dependent loads (from
// a graph on GB300: trim, fork and extend of 4 beams 10.8 us; extend, compact and trim of the drafts of 64
// sequences 13.1 us; called one after the other from Python 17 to 20 us, which is the host's three calls).  Extend lists
// free pages in one CTA, 4096 counts a turn from page 0 on: 62 us behind 200000 held pages, 11 where the first are free.
// Rows and pages are read and written once: 733 MB of pages copied in 108 us (6.8 TB/s); 254 MB of single rows of 128
// bytes packed in 56 us (4.5 TB/s).
#include <algorithm>
#include <climits>

#include "kernels.h"
#include "kv_cache.cuh"

namespace syn {

constexpr int PG_THREADS = 256;

// (for the index checks: `bytes` from byte `at` of a pool on lie in it)
__device__ __forceinline__ bool in_pool(const KvCache& c, int64_t at, int bytes) {
    return at >= 0 && at + bytes <= (c.n_pages - 1) * c.page_stride + c.n_kv * c.tile;
}

// ---- fork and trim: a thread per table entry --------------------------------------------

struct ForkParams {
    int32_t* refs;
    const int32_t* from;
    const int32_t* pages;
    const int32_t* lens;
    int32_t* new_pages;
    int32_t* new_lens;
    int* err;
    int64_t n_seq, n_new, max_pages, n_pages;
    int page_shift;
};

__global__ void __launch_bounds__(PG_THREADS) k_kv_fork(const ForkParams p) {
    griddep_release();
    griddep_wait();
    const int64_t total = p.n_new * p.max_pages, step = (int64_t)gridDim.x * PG_THREADS;
    for (int64_t u = (int64_t)blockIdx.x * PG_THREADS + threadIdx.x; u < total; u += step) {
        const int64_t i = u / p.max_pages, j = u - i * p.max_pages;
        const int s = p.from[i];
        if (s >= p.n_seq && j == 0) record_error(p.err, SYN_DEVERR_BOUNDS);
        const int len = s >= 0 && s < p.n_seq ? held_rows(p.lens[s], p.max_pages, p.page_shift) : 0;
        if (!SYN_IN_BOUNDS(i < p.n_new && j < p.max_pages)) continue;
        int id = -1;
        if (j < ((int64_t)len + (1 << p.page_shift) - 1) >> p.page_shift) {
            id = p.pages[s * p.max_pages + j];
            if ((unsigned)id < (unsigned)p.n_pages) {
                atomicAdd(p.refs + id, 1);
            } else {
                record_error(p.err, SYN_DEVERR_BOUNDS);
                id = -1;
            }
        }
        p.new_pages[u] = id;
        if (j == 0) p.new_lens[i] = len;
    }
}

struct TrimParams {
    int32_t* refs;
    int32_t* pages;
    const int32_t* lens;
    int* err;
    int64_t n_seq, max_pages, n_pages;
    int page_shift;
};

__global__ void __launch_bounds__(PG_THREADS) k_kv_trim(const TrimParams p) {
    griddep_release();
    griddep_wait();
    const int64_t total = p.n_seq * p.max_pages, step = (int64_t)gridDim.x * PG_THREADS;
    for (int64_t u = (int64_t)blockIdx.x * PG_THREADS + threadIdx.x; u < total; u += step) {
        const int64_t s = u / p.max_pages, j = u - s * p.max_pages;
        if (j < ((int64_t)max(p.lens[s], 0) + (1 << p.page_shift) - 1) >> p.page_shift) continue;
        if (!SYN_IN_BOUNDS(s < p.n_seq)) continue;
        const int id = p.pages[u];
        if (id < 0) continue;
        p.pages[u] = -1;
        if (id >= p.n_pages) {
            record_error(p.err, SYN_DEVERR_BOUNDS);
        } else if (atomicSub(p.refs + id, 1) <= 0) {  // (given back before)
            atomicAdd(p.refs + id, 1);
            record_error(p.err, SYN_DEVERR_BOUNDS);
        }
    }
}

static int table_grid(int64_t entries, int sms) {
    return (int)std::min<int64_t>((entries + PG_THREADS - 1) / PG_THREADS, (int64_t)sms * 8);
}

cudaError_t launch_kv_fork(const KvCache& c, int32_t* refs, int64_t n_seq, const int32_t* pages, int64_t max_pages,
                           const int32_t* lens, int64_t n_new, const int32_t* from, int32_t* new_pages, int32_t* new_lens,
                           int* err, int sms, cudaStream_t s) {
    const ForkParams p{refs, from, pages, lens, new_pages, new_lens, err, n_seq, n_new, max_pages, c.n_pages, c.page_shift};
    return launch_overlapped(k_kv_fork, table_grid(n_new * max_pages, sms), PG_THREADS, 0, s, p);
}

cudaError_t launch_kv_trim(const KvCache& c, int32_t* refs, int64_t n_seq, int32_t* pages, int64_t max_pages,
                           const int32_t* lens, int* err, int sms, cudaStream_t s) {
    const TrimParams p{refs, pages, lens, err, n_seq, max_pages, c.n_pages, c.page_shift};
    return launch_overlapped(k_kv_trim, table_grid(n_seq * max_pages, sms), PG_THREADS, 0, s, p);
}

// ---- extend ------------------------------------------------------------------------------
//
// The columns a sequence's new rows fall into are items, counted through over the sequences.  An item
// whose entry is empty (missing), or whose page others hold too (shared), needs a page.  One CTA plans:
//   1. each shared item takes its entry off its page's count; where a count comes to 0 every holder
//      writes, and the last of them (by a minimum over negative numbers) keeps the page;
//   2. the free pages are listed, lowest first, as many as are needed;
//   3. where they suffice the items take them in order; where they do not, nobody keeps a shared page, and
//      the sequences whose needs, summed up to them, fit, take theirs.
// A second kernel gives out the slots and copies the rows of first pages that were shared.  (One kernel, in which
// the other CTAs wait for the plan behind a flag, took longer: trim, fork and extend of 4 beams, from a graph, 14.1 us and
// not 10.8; the accepted drafts of 64 sequences 22.4 and not 18.9.)

constexpr int EXT_THREADS = 512;  // of the plan

struct ExtendParams {
    KvCache c;
    int32_t* refs;
    int32_t* pages;
    const int32_t* lens;
    int32_t* new_lens;
    const int32_t* starts;  // NULL: one row each
    int64_t* slots;
    int4* plan;      // per sequence: page copied from (-1: none), copied to, length, whether it was extended
    int32_t* need;   // [items] 0: a page of its own, 1: missing, 2: shared; then, where pages are short, sums
    int32_t* free_list;  // [items]
    int* err;
    int64_t max_pages, n_tok, max_items;
    int n_seq;
};

// (rows that run backwards or past the call's tokens count as none)
__device__ __forceinline__ int new_rows(const ExtendParams& p, int s) {
    if (!p.starts) return 1;
    const int a = p.starts[s], b = p.starts[s + 1];
    return a < 0 || b > p.n_tok ? 0 : max(b - a, 0);
}

// Two numbers up to 2^30 added, up to 2^30.
__device__ __forceinline__ int add_up_to(int a, int b) { return (int)min((unsigned)a + (unsigned)b, 1u << 30); }

// The inclusive sum over the CTA's threads, and their total, up to 2^30 (which only starts that overlap come to: a call has
// at most 2^28 pages of new rows, and some for its sequences).
__device__ __forceinline__ int block_sum(int x, int* sums, int& total) {
    constexpr int WARPS = EXT_THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x = add_up_to(x, y);
    }
    __syncthreads();  // (the sums before this one have been read)
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int w = lane < WARPS ? sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < WARPS; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w = add_up_to(w, y);
    }
    total = __shfl_sync(0xffffffffu, w, WARPS - 1);
    const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    return add_up_to(x, warp > 0 ? before : 0);
}

// Which of counts[at .. at + 8) are 0.
__device__ __forceinline__ int free_of(const int32_t* counts, int64_t at, int64_t n) {
    int bits = 0;
    if (at + 8 <= n && (reinterpret_cast<uintptr_t>(counts + at) & 15) == 0) {
        const int4 a = __ldcg(reinterpret_cast<const int4*>(counts + at)), b = __ldcg(reinterpret_cast<const int4*>(counts + at) + 1);
        const int x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; i++) bits |= x[i] == 0 ? 1 << i : 0;
    } else {
        for (int i = 0; i < 8; i++)
            if (at + i < n && __ldcg(counts + at + i) == 0) bits |= 1 << i;
    }
    return bits;
}

__device__ void plan_pages(const ExtendParams& p, int* off, int* sums) {
    const int tid = threadIdx.x, shift = p.c.page_shift, page = 1 << shift;
    // (the first counts, on their way; a page that this call takes off its holders is not free for it)
    const int bits0 = free_of(p.refs, (int64_t)tid * 8, p.c.n_pages);
    // ---- the items ---------------------------------------------------------------------------
    int items = 0;
    if (tid == 0) off[0] = 0;
    for (int s0 = 0; s0 < p.n_seq; s0 += EXT_THREADS) {
        const int s = s0 + tid;
        int columns = 0;
        if (s < p.n_seq) {
            const int len = held_rows(p.lens[s], p.max_pages, shift), n = new_rows(p, s);
            const int64_t end = ((int64_t)len + n + page - 1) >> shift;
            const bool fits = end <= p.max_pages && (int64_t)len + n <= INT_MAX - 1024;
            if (fits && n > 0) columns = (int)(end - (len >> shift));
            p.plan[s] = make_int4(-1, -1, len, fits);
        }
        int total;
        const int sum = block_sum(columns, sums, total);
        if (s < p.n_seq) off[s + 1] = add_up_to(items, sum);
        items = add_up_to(items, total);
    }
    __syncthreads();
    // (starts that overlap could name more rows than the call has)
    if (items > p.max_items) {
        if (tid == 0) record_error(p.err, SYN_DEVERR_BOUNDS);
        for (int s = tid; s < p.n_seq; s += EXT_THREADS) {
            p.new_lens[s] = p.plan[s].z;
            p.plan[s].w = 0;
        }
        return;
    }
    volatile int32_t* refs = p.refs;
    struct Item {
        int s, id;
        int64_t entry;
    };
    auto fetch = [&](int u) {
        Item x{0, -1, 0};
        if (u >= items) return x;
        int lo = 0, hi = p.n_seq - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (off[mid + 1] > u) hi = mid;
            else lo = mid + 1;
        }
        x.s = lo;
        x.entry = (int64_t)lo * p.max_pages + (p.plan[lo].z >> shift) + (u - off[lo]);
        if (!SYN_IN_BOUNDS(u >= off[lo] && x.entry < (int64_t)(lo + 1) * p.max_pages)) return x;
        x.id = p.pages[x.entry];
        return x;
    };
    // (a thread's first item, mostly its only one, stays in registers)
    const Item mine = fetch(tid);
    auto item = [&](int u) { return u == tid ? mine : fetch(u); };
    // ---- missing and shared ------------------------------------------------------------------
    int any_shared = 0;
    for (int u = tid; u < items; u += EXT_THREADS) {
        const int id = item(u).id;
        int what = 1;
        if ((unsigned)id < (unsigned)p.c.n_pages) {
            what = refs[id] > 1 ? 2 : 0;
        } else if (id >= 0) {
            record_error(p.err, SYN_DEVERR_BOUNDS);
        }
        any_shared |= what == 2;
        if (SYN_IN_BOUNDS(u < p.max_items)) p.need[u] = what;
    }
    any_shared = __syncthreads_or(any_shared);
    if (any_shared) {
        for (int u = tid; u < items; u += EXT_THREADS)
            if (p.need[u] == 2) atomicSub(p.refs + item(u).id, 1);
        __syncthreads();
        for (int u = tid; u < items; u += EXT_THREADS)
            if (p.need[u] == 2) {
                const int id = item(u).id;
                if (refs[id] <= 0) atomicMin(p.refs + id, -1 - u);
            }
        __syncthreads();
    }
    auto keeps = [&](int u, int id) { return refs[id] == -1 - u; };
    // ---- the free pages ----------------------------------------------------------------------
    int wanted = 0;
    for (int u0 = 0; u0 < items; u0 += EXT_THREADS) {
        const int u = u0 + tid, what = u < items ? p.need[u] : 0;
        wanted += __syncthreads_count(what == 1 || (what == 2 && !keeps(u, item(u).id)));
    }
    int n_free = 0;
    for (int64_t b = 0; b < p.c.n_pages && n_free < wanted; b += EXT_THREADS * 8) {
        const int64_t at = b + (int64_t)tid * 8;
        int bits = b == 0 ? bits0 : free_of(p.refs, at, p.c.n_pages);
        int total;
        int rank = n_free + block_sum(__popc(bits), sums, total) - __popc(bits);
        n_free += total;
        for (; bits; bits &= bits - 1, rank++)
            if (rank < p.max_items && SYN_IN_BOUNDS(rank >= 0 && at + __ffs(bits) <= p.c.n_pages)) p.free_list[rank] = (int)at + __ffs(bits) - 1;
    }
    __syncthreads();
    const bool enough = n_free >= wanted;
    if (!enough) {
        // ---- pages are short: who is served, and the counts as they were for the others -------------
        int base = 0;
        for (int u0 = 0; u0 < items; u0 += EXT_THREADS) {
            const int u = u0 + tid;
            int total;
            const int what = u < items ? p.need[u] : 0, sum = base + block_sum(what != 0, sums, total);
            if (what == 2) {
                const int id = item(u).id;
                if (keeps(u, id)) refs[id] = 0;
            }
            if (u < items) p.need[u] = sum << 2 | what;
            base += total;
        }
        __syncthreads();
        for (int s = tid; s < p.n_seq; s += EXT_THREADS) {
            const int before = off[s] ? p.need[off[s] - 1] >> 2 : 0, upto = off[s + 1] ? p.need[off[s + 1] - 1] >> 2 : 0;
            if (p.plan[s].w) p.plan[s].w = upto == before || upto <= n_free;
        }
        __syncthreads();
        for (int u = tid; u < items; u += EXT_THREADS) {
            const Item x = item(u);
            if ((p.need[u] & 3) == 2 && !p.plan[x.s].w) atomicAdd(p.refs + x.id, 1);
        }
        __syncthreads();
    }
    // ---- the pages dealt out -----------------------------------------------------------------
    int given = 0;
    for (int u0 = 0; u0 < items; u0 += EXT_THREADS) {
        const int u = u0 + tid;
        const Item x = item(u);
        const int what = u < items && (enough || p.plan[x.s].w) ? p.need[u] & 3 : 0;
        const bool kept = enough && what == 2 && keeps(u, x.id), take = what && !kept;
        int total;
        const int rank = given + block_sum(take, sums, total) - 1;
        given += total;
        if (kept) refs[x.id] = 1;
        if (take && SYN_IN_BOUNDS(rank >= 0 && rank < n_free && rank < p.max_items)) {
            const int got = p.free_list[rank];
            refs[got] = 1;
            p.pages[x.entry] = got;
            if (what == 2 && u == off[x.s]) {
                p.plan[x.s].x = x.id;
                p.plan[x.s].y = got;
            }
        }
    }
    __syncthreads();
    for (int s = tid; s < p.n_seq; s += EXT_THREADS) {
        const int4 a = p.plan[s];
        p.new_lens[s] = a.z + (a.w ? new_rows(p, s) : 0);
    }
}

__global__ void __launch_bounds__(EXT_THREADS) k_kv_extend_plan(const ExtendParams p) {
    __shared__ int off[KV_EXTEND_SEQS + 1];
    __shared__ int sums[32];
    griddep_release();
    griddep_wait();
    plan_pages(p, off, sums);
}
__global__ void __launch_bounds__(PG_THREADS) k_kv_extend_rows(const ExtendParams p) {
    const int shift = p.c.page_shift, page = 1 << shift, tid = threadIdx.x;
    griddep_release();
    griddep_wait();
    if (p.slots)
        for (int64_t t = (int64_t)blockIdx.x * PG_THREADS + tid; t < p.n_tok; t += (int64_t)gridDim.x * PG_THREADS) {
            int lo = 0, hi = p.n_seq;  // the last sequence that starts at t or before it
            if (p.starts) {
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (p.starts[mid] <= t) lo = mid;
                    else hi = mid;
                }
            } else {
                lo = (int)t;
            }
            const int64_t at = p.starts ? t - p.starts[lo] : 0;
            int64_t slot = -1;
            const int4 a = p.plan[lo];
            if (a.w && at >= 0 && at < new_rows(p, lo)) {
                const int row = a.z + (int)at;
                if (SYN_IN_BOUNDS((row >> shift) < p.max_pages)) slot = ((int64_t)p.pages[lo * p.max_pages + (row >> shift)] << shift) + (row & (page - 1));
            }
            p.slots[t] = slot;
        }
    // the rows of a tile (one kv head, keys or values) that move with their sequence
    const int tiles = 2 * p.c.n_kv, n16 = p.c.dim >> (p.c.q8 ? 4 : 3);  // 16-byte pieces of a row
    for (int64_t x = blockIdx.x; x < (int64_t)p.n_seq * tiles; x += gridDim.x) {
        const int s = (int)(x / tiles), h = (int)(x - (int64_t)s * tiles) >> 1;
        const int4 a = p.plan[s];
        if (a.x < 0) continue;
        uint8_t* pool = x & 1 ? p.c.v : p.c.k;
        const uint8_t* src = pool + a.x * p.c.page_stride + h * p.c.tile;
        uint8_t* dst = pool + a.y * p.c.page_stride + h * p.c.tile;
        const int rows = a.z & (page - 1);
        if (!SYN_IN_BOUNDS(in_pool(p.c, src - pool, (int)p.c.tile) && in_pool(p.c, dst - pool, (int)p.c.tile))) continue;
        for (int i = tid; i < rows * n16; i += PG_THREADS)
            reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(src)[i];
        if (p.c.q8) {
            const int64_t scales = (int64_t)p.c.dim << shift;
            for (int i = tid; i < rows * (p.c.dim >> 5); i += PG_THREADS)
                reinterpret_cast<uint16_t*>(dst + scales)[i] = reinterpret_cast<const uint16_t*>(src + scales)[i];
        }
    }
}

int64_t extend_items(const KvCache& c, int64_t n_seq, int64_t n_tok) { return (n_tok >> c.page_shift) + 2 * n_seq; }

cudaError_t launch_kv_extend(const KvCache& c, int32_t* refs, int64_t n_seq, int64_t n_tok, int32_t* pages, int64_t max_pages,
                             const int32_t* lens, const int32_t* starts, int32_t* new_lens, int64_t* slots, void* scratch,
                             int* err, int sms, int* launches, cudaStream_t s) {
    ExtendParams p;
    p.c = c;
    p.refs = refs;
    p.pages = pages;
    p.lens = lens;
    p.new_lens = new_lens;
    p.starts = starts;
    p.slots = slots;
    p.max_items = extend_items(c, n_seq, n_tok);
    p.plan = static_cast<int4*>(scratch);
    p.need = reinterpret_cast<int32_t*>(p.plan + n_seq);
    p.free_list = p.need + p.max_items;
    p.err = err;
    p.max_pages = max_pages;
    p.n_tok = n_tok;
    p.n_seq = (int)n_seq;
    cudaError_t e = launch_overlapped(k_kv_extend_plan, 1, EXT_THREADS, 0, s, p);
    if (e != cudaSuccess) return e;
    ++*launches;
    const int64_t work = std::max<int64_t>((slots ? n_tok + PG_THREADS - 1 : 0) / PG_THREADS, n_seq * 2 * c.n_kv);
    e = launch_overlapped(k_kv_extend_rows, (int)std::min<int64_t>(work, 2 * sms), PG_THREADS, 0, s, p);
    if (e == cudaSuccess) ++*launches;
    return e;
}

// ---- compact -----------------------------------------------------------------------------
//
// Rows move down in place: row base + i comes from base + rows[i] >= base + i.  A CTA has columns of a sequence's
// tiles (a tile: a kv head, keys or values; a column: some 16-byte pieces of each row) to itself and goes through
// them in passes of CMP_SHORT units a thread (a unit: a piece of a row), in the order of the rows within each tile: a pass
// is loaded whole before any of it is stored.  A unit of list row i overwrites the piece of a list row k with
// rows[k] = i, if there is one; as rows ascend k <= i, so that piece was loaded in this pass or one before, and what later
// passes load lies past every place stored so far.  (So a tile's units stay in the order of its rows.)  No CTA
// waits for another.  Short lists are a chain of dependent loads
// (starts, rows, page ids, counts, rows): what makes a call longer is the CTAs it takes to start.

constexpr int CMP_THREADS = 256;
constexpr int CMP_ROWS = 256;   // rows of a batch
// Most rows of a chunk of a long list (3 sequences of 21001 to 60001 Q8_0 rows, half kept: 16, 32, 64, 128 rows: 57.0, 55.7,
// 58.0, 68.5 us).
constexpr int CMP_CHUNK = 32;
constexpr int CMP_UNITS = 8;    // pieces a thread holds
constexpr int CMP_SHORT = 4;    // and of a short one (8: 114 registers, which leave two CTAs an SM)
constexpr int CMP_SCALES = 4;   // and pieces of scales
constexpr int CMP_CTAS = 4;     // of an SM, for long lists (2, 3, 4: 68.1, 59.4, 57.0 us)
constexpr int CMP_TARGET = 3;   // and for short ones (64 sequences, 2048 and 4096 F16 rows: 2: 5.8, 8.8 us, 3: 4.8, 7.1 us)

struct CompactParams {
    KvCache c;
    const int32_t* refs;
    const int32_t* pages;
    const int32_t* base;
    const int32_t* starts;
    const int32_t* rows;
    int32_t* new_lens;
    int* err;
    int64_t max_pages, n_rows;
    int n_seq, cut, width, group;  // columns a tile is cut into, 16-byte pieces of one; tiles of a CTA
    int apart;                     // (Q8_0) the scales are a column more, not the last one's
};

template <typename U>
__device__ __forceinline__ void move_rows(const CompactParams& p, int tile0, int n_tiles, int first, int width, const int64_t* src,
                                          const int64_t* dst, int n) {
    const int each = n * width, units = n_tiles * each;
    // unit u is piece x of row r of tile t; the next of a thread is CMP_THREADS on
    const int dt = CMP_THREADS / each, dr = (CMP_THREADS - dt * each) / width, dx = CMP_THREADS - dt * each - dr * width;
    int t = threadIdx.x / each, r = (threadIdx.x - t * each) / width, x = threadIdx.x - t * each - r * width;
    auto on = [&]() {
        x += dx, r += dr, t += dt;
        if (x >= width) x -= width, r++;
        if (r >= n) r -= n, t++;
    };
    auto at = [&](int64_t row) {
        const int tile = tile0 + t;
        return reinterpret_cast<U*>((tile & 1 ? p.c.v : p.c.k) + row + (tile >> 1) * p.c.tile) + first + x;
    };
    auto inside = [&](int64_t row) {  // (for the index checks)
        const int tile = tile0 + t;
        return r < CMP_ROWS && tile < 2 * p.c.n_kv && in_pool(p.c, row + (tile >> 1) * p.c.tile + (first + x) * (int)sizeof(U), sizeof(U));
    };
    U held[CMP_SHORT];
    for (int u0 = 0; u0 < units; u0 += CMP_THREADS * CMP_SHORT) {
        const int t0 = t, r0 = r, x0 = x;
#pragma unroll
        for (int i = 0; i < CMP_SHORT; i++, on())
            if (t < n_tiles && src[r] >= 0 && SYN_IN_BOUNDS(inside(src[r]))) held[i] = *at(src[r]);
        __syncthreads();
        t = t0, r = r0, x = x0;
#pragma unroll
        for (int i = 0; i < CMP_SHORT; i++, on())
            if (t < n_tiles && src[r] >= 0 && SYN_IN_BOUNDS(inside(src[r]) && inside(dst[r]))) *at(dst[r]) = held[i];
    }
}

__global__ void __launch_bounds__(CMP_THREADS, 4) k_kv_compact(const CompactParams p) {
    // where a row's values are in a pool's tile 0, and (Q8_0) its scales; -1: the row stays
    __shared__ int64_t src[CMP_ROWS], dst[CMP_ROWS], src_s[CMP_ROWS], dst_s[CMP_ROWS];
    const int tid = threadIdx.x, shift = p.c.page_shift, tiles = 2 * p.c.n_kv, groups = (tiles + p.group - 1) / p.group,
              per = p.cut + p.apart;
    griddep_release();
    griddep_wait();
    for (int unit = blockIdx.x; unit < p.n_seq * per * groups; unit += gridDim.x) {
        const int column = unit % per, tile0 = unit / per % groups * p.group, s = unit / (per * groups);
        const int a = p.starts[s], b = p.starts[s + 1], n = a < 0 || b > p.n_rows ? 0 : max(b - a, 0);
        const int base = max(p.base[s], 0), n_tiles = min(p.group, tiles - tile0);
        const bool tells = column == 0 && tile0 == 0;
        if (tells && tid == 0) p.new_lens[s] = (int)min((int64_t)base + n, (int64_t)INT_MAX);
        const int32_t* table = p.pages + (int64_t)s * p.max_pages;
        const int64_t held = min(p.max_pages << shift, (int64_t)INT_MAX);
        auto slot_of = [&](int64_t row) -> int64_t {
            if (row >= held) return -1;
            const int id = table[row >> shift];
            return (unsigned)id < (unsigned)p.c.n_pages ? ((int64_t)id << shift) + (row & ((1 << shift) - 1)) : -1;
        };
        for (int i0 = 0; i0 < n; i0 += CMP_ROWS) {
            const int m = min(n - i0, CMP_ROWS);
            __syncthreads();  // (the batch before is stored)
            for (int i = tid; i < m; i += CMP_THREADS) {
                const int row = p.rows[a + i0 + i];
                int64_t from = -1, to = -1;
                if (row != i0 + i) {
                    // (a row that would come from before its place, or not after the one before, may be gone already)
                    const bool ok = row > i0 + i && (i0 + i == 0 || p.rows[a + i0 + i - 1] < row);
                    if (ok) {
                        from = slot_of((int64_t)base + row);
                        to = slot_of((int64_t)base + i0 + i);
                    }
                    // (a page that others hold too is not written to)
                    if (to >= 0 && p.refs && p.refs[to >> shift] > 1) to = -1;
                    if (from < 0 || to < 0) {
                        from = -1;
                        if (tells) record_error(p.err, SYN_DEVERR_BOUNDS);
                    }
                }
                const int64_t cells = (int64_t(1) << shift) - 1, pitch = p.c.q8 ? p.c.dim : 2 * p.c.dim;
                const int64_t f = (from >> shift) * p.c.page_stride, o = (to >> shift) * p.c.page_stride;
                src[i] = from < 0 ? -1 : f + (from & cells) * pitch;
                dst[i] = o + (to & cells) * pitch;
                if (p.c.q8) {
                    src_s[i] = from < 0 ? -1 : f + ((int64_t)p.c.dim << shift) + (from & cells) * (p.c.dim >> 4);
                    dst_s[i] = o + ((int64_t)p.c.dim << shift) + (to & cells) * (p.c.dim >> 4);
                }
            }
            __syncthreads();
            const int pieces = p.c.dim >> (p.c.q8 ? 4 : 3), first = column * p.width;
            if (column < p.cut) move_rows<uint4>(p, tile0, n_tiles, first, min(p.width, pieces - first), src, dst, m);
            if (p.c.q8 && column == per - 1)
                move_rows<uint16_t>(p, tile0, n_tiles, 0, p.c.dim >> 5, src_s, dst_s, m);
        }
    }
}

// Long lists: a chunk of rows (of a group of its heads' tiles) is a CTA's.  Chunks are taken in order, by a
// counter; each loads its rows, says so, and stores them once the chunks whose rows lie where it stores (one or two,
// found by a search in the ascending list) have loaded theirs.  Those chunks are not after it, and wait for
// nothing before they say so but their CTA's chunk before: every wait ends.  What a chunk needs to know is a chain of
// dependent loads (sequence, rows, page ids, counts; the search), so a warp of its own finds it out a chunk
// ahead.  (Not two: a chunk that is taken and not loaded keeps others waiting, 87 to 109 us instead of 57.)

struct LongParams {
    CompactParams m;
    int* turn;   // [0] the next chunk to be taken, [1] CTAs done; zero between calls
    int* flags;  // [groups][chunks] 1: loaded; zero between calls
    int chunks, chunk_rows, groups, group_tiles;
};
struct LongChunk {
    int64_t src[CMP_CHUNK], dst[CMP_CHUNK];      // where a row's values are in a pool's tile 0; -1: the row stays
    int64_t src_s[CMP_CHUNK], dst_s[CMP_CHUNK];  // (Q8_0) its scales
    int chunk, group, rows, c0, c1;              // rows: 0: none moves, -1: no chunk is left; [c0, c1): chunks waited for
};

// A warp's: what the CTAs need to know of the chunk taken.
__device__ __forceinline__ void plan_chunk(const LongParams& q, int taken, LongChunk* out) {
    const CompactParams& p = q.m;
    const int lane = threadIdx.x & 31, shift = p.c.page_shift;
    if (taken >= q.chunks * q.groups) {
        if (lane == 0) out->rows = -1;
        return;
    }
    const int64_t held = min(p.max_pages << shift, (int64_t)INT_MAX), cell_mask = (int64_t(1) << shift) - 1;
    const int chunk = taken / q.groups, group = taken - chunk * q.groups, r0 = chunk * q.chunk_rows;
    const int m = min(q.chunk_rows, (int)p.n_rows - r0);
    auto sequence_of = [&](int r) {  // the last sequence that starts at r or before it
        int lo = 0, hi = p.n_seq;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.starts[mid] <= r) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    bool moves = false;
    int first_seq = 0;
#pragma unroll
    for (int k = 0; k < CMP_CHUNK / 32; k++) {
        const int i = lane + 32 * k, r = r0 + i;
        if (i >= m || !SYN_IN_BOUNDS(i < CMP_CHUNK && r < p.n_rows)) continue;
        const int lo = sequence_of(r);
        if (k == 0) first_seq = lo;
        const int a = p.starts[lo], b = p.starts[lo + 1], at = r - a;
        int64_t from = -1, to = -1;
        if (a >= 0 && at >= 0 && b <= p.n_rows && r < b) {
            const int row = p.rows[r], before = at ? p.rows[r - 1] : -1, base = max(p.base[lo], 0);
            if (row != at) {
                auto slot_of = [&](int64_t y) -> int64_t {
                    if (y >= held) return -1;
                    const int id = p.pages[(int64_t)lo * p.max_pages + (y >> shift)];
                    return (unsigned)id < (unsigned)p.c.n_pages ? ((int64_t)id << shift) + (y & cell_mask) : -1;
                };
                if (row > at && before < row) {
                    from = slot_of((int64_t)base + row);
                    to = slot_of((int64_t)base + at);
                }
                if (to >= 0 && p.refs && p.refs[to >> shift] > 1) to = -1;
                if (from < 0 || to < 0) {
                    from = -1;
                    record_error(p.err, SYN_DEVERR_BOUNDS);
                }
            }
        }
        moves |= from >= 0;
        const int64_t pitch = p.c.dim * (p.c.q8 ? 1 : 2), scales = (int64_t)p.c.dim << shift;
        const int64_t from0 = (from >> shift) * p.c.page_stride, to0 = (to >> shift) * p.c.page_stride;
        out->src[i] = from < 0 ? -1 : from0 + (from & cell_mask) * pitch;
        out->dst[i] = to0 + (to & cell_mask) * pitch;
        out->src_s[i] = from0 + scales + (from & cell_mask) * (p.c.dim >> 4);
        out->dst_s[i] = to0 + scales + (to & cell_mask) * (p.c.dim >> 4);
    }
    moves = __any_sync(0xffffffffu, moves);
    first_seq = __shfl_sync(0xffffffffu, first_seq, 0);
    // the chunks [c0, c1) that hold what lies at the places of this one's rows of its first sequence (those
    // of sequences that begin in it are its own)
    const int a = max(p.starts[first_seq], 0), b = min(max(p.starts[first_seq + 1], a), (int)p.n_rows);
    int c0 = 0, c1 = 0;
    if (moves && a < r0) {
        const int place = r0 - a;
        int lo = a, n = min(r0 + m, b) - a;  // (a row is not before its place: none after this chunk)
        while (n > 0) {  // the list's first row that is not below the first place
            const int step = (n + 31) / 32, at = lo + lane * step;
            const int below = __popc(__ballot_sync(0xffffffffu, lane * step < n && p.rows[at] < place));
            // rows lo + step * (below - 1) and before are below; row lo + step * below is not
            if (below == 0) break;
            lo += (below - 1) * step + 1;
            n = min(step - 1, max(n - ((below - 1) * step + 1), 0));
        }
        c0 = lo / q.chunk_rows;
        c1 = min((lo + m + q.chunk_rows - 1) / q.chunk_rows, chunk);  // (at most m rows lie at m places)
    }
    if (lane == 0) {
        out->chunk = chunk;
        out->group = group;
        out->rows = moves ? m : 0;
        out->c0 = c0;
        out->c1 = c1;
    }
}

constexpr int CMP_LONG_THREADS = CMP_THREADS + 32;  // the last warp plans
__device__ __forceinline__ void copiers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(CMP_THREADS) : "memory"); }

template <typename S>
__global__ void __launch_bounds__(CMP_LONG_THREADS, CMP_CTAS) k_kv_compact_long(const LongParams q) {
    const CompactParams& p = q.m;
    __shared__ LongChunk plans[2];
    __shared__ int gave_up, last;
    extern __shared__ uint4 pieces[];  // [CMP_UNITS][CMP_THREADS] on their way, each thread's its own
    const int tid = threadIdx.x;
    const bool plans_ahead = tid >= CMP_THREADS;
    griddep_release();
    griddep_wait();
    auto take = [&]() {
        int t = 0;
        if (tid == CMP_THREADS) t = atomicAdd(q.turn, 1);
        return __shfl_sync(0xffffffffu, t, 0);
    };
    if (plans_ahead) {
        plan_chunk(q, take(), &plans[0]);
    } else {
        if (tid == 0) gave_up = 0;
        // the lengths
        for (int s = blockIdx.x * CMP_THREADS + tid; s < p.n_seq; s += gridDim.x * CMP_THREADS) {
            const int a = p.starts[s], b = p.starts[s + 1], n = a < 0 || b > p.n_rows ? 0 : max(b - a, 0);
            p.new_lens[s] = (int)min((int64_t)max(p.base[s], 0) + n, (int64_t)INT_MAX);
        }
    }
    const int n16 = p.c.dim >> (p.c.q8 ? 4 : 3), ns = p.c.q8 ? (p.c.dim >> 4) / (int)sizeof(S) : 0;  // units of a row of a tile
    uint4* held16 = pieces + tid;
    for (int x = 0;; x ^= 1) {
        __syncthreads();  // (plans[x] is made, plans[x ^ 1] and the pieces have been used)
        const LongChunk& w = plans[x];
        if (w.rows < 0) break;
        if (plans_ahead) {
            plan_chunk(q, take(), &plans[x ^ 1]);
            continue;
        }
        // this thread's piece of a row (one 16 bytes of a tile), and the rows it takes: tid / u16, then every per16-th
        const int tile0 = w.group * q.group_tiles, tiles = min(q.group_tiles, 2 * p.c.n_kv - tile0);
        const int u16 = tiles * n16, us = tiles * ns, per16 = CMP_THREADS / u16, per_s = us ? CMP_THREADS / us : 1;
        const int row16 = tid / u16, t16 = (tid - row16 * u16) / n16, row_s = us ? tid / us : 0, t_s = us ? (tid - row_s * us) / ns : 0;
        uint8_t* at16 = ((tile0 + t16) & 1 ? p.c.v : p.c.k) + ((tile0 + t16) >> 1) * p.c.tile + (tid - row16 * u16 - t16 * n16) * 16;
        uint8_t* at_s = ((tile0 + t_s) & 1 ? p.c.v : p.c.k) + ((tile0 + t_s) >> 1) * p.c.tile + (tid - row_s * us - t_s * ns) * (int)sizeof(S);
        const int end16 = row16 < per16 ? w.rows : 0, end_s = us && row_s < per_s ? w.rows : 0;
        // (for the index checks: this thread's piece of 16 bytes, or of scales, of the row at `row` of tile 0)
        auto in16 = [&](int64_t row) { return in_pool(p.c, at16 - ((tile0 + t16) & 1 ? p.c.v : p.c.k) + row, 16); };
        auto in_s = [&](int64_t row) { return in_pool(p.c, at_s - ((tile0 + t_s) & 1 ? p.c.v : p.c.k) + row, sizeof(S)); };
        S ws[CMP_SCALES];
#pragma unroll
        for (int i = 0; i < CMP_UNITS; i++) {
            const int r = row16 + i * per16;
            if (r < end16 && w.src[r] >= 0 && SYN_IN_BOUNDS(r < CMP_CHUNK && in16(w.src[r]))) cp16_all(smem_u32(held16 + i * CMP_THREADS), at16 + w.src[r]);
        }
        cp_commit();
#pragma unroll
        for (int i = 0; i < CMP_SCALES; i++) {
            const int r = row_s + i * per_s;
            if (r < end_s && w.src[r] >= 0 && SYN_IN_BOUNDS(r < CMP_CHUNK && in_s(w.src_s[r]))) ws[i] = *reinterpret_cast<const S*>(at_s + w.src_s[r]);
        }
        cp_wait<0>();
        copiers_sync();  // (what was loaded is loaded)
        int* flags = q.flags + (int64_t)w.group * q.chunks;
#ifndef SYN_TEST_STALL  // (timeout-test build: no chunk says that it is loaded, so the waits for one run out)
        if (tid == 0 && SYN_IN_BOUNDS(w.chunk >= 0 && w.chunk < q.chunks && w.group < q.groups && w.c1 <= q.chunks)) {
            __threadfence();
            atomicExch(flags + w.chunk, 1);
        }
#endif
        if (w.c0 + tid < w.c1 && !gave_up) {
            const long long t0 = clock64();
            for (int j = w.c0 + tid; j < w.c1; j += CMP_THREADS)
                while (*reinterpret_cast<volatile int*>(flags + j) == 0)
                    if (clock64() - t0 > SYN_WAIT_CYCLES) {
                        record_error(p.err, SYN_DEVERR_TIMEOUT);
                        gave_up = 1;
                        break;
                    }
            __threadfence();
        }
        copiers_sync();
        if (gave_up) continue;
#pragma unroll
        for (int i = 0; i < CMP_UNITS; i++) {
            const int r = row16 + i * per16;
            if (r < end16 && w.src[r] >= 0 && SYN_IN_BOUNDS(in16(w.dst[r]))) *reinterpret_cast<uint4*>(at16 + w.dst[r]) = held16[i * CMP_THREADS];
        }
#pragma unroll
        for (int i = 0; i < CMP_SCALES; i++) {
            const int r = row_s + i * per_s;
            if (r < end_s && w.src[r] >= 0 && SYN_IN_BOUNDS(in_s(w.dst_s[r]))) *reinterpret_cast<S*>(at_s + w.dst_s[r]) = ws[i];
        }
    }
    // the last CTA to get here leaves the counters and flags as they were (behind every CTA's own: the fences
    // order each flag that was set before its CTA's count, and the last count before the zeros)
    if (tid == 0) {
        __threadfence();
        last = atomicAdd(q.turn + 1, 1) == (int)gridDim.x - 1;
        __threadfence();
    }
    __syncthreads();
    if (!last) return;
    if (tid < 2) q.turn[tid] = 0;
    for (int i = tid; i < q.chunks * q.groups; i += CMP_LONG_THREADS) q.flags[i] = 0;
}

// Which lists count as long.  The kernel of short ones goes through a sequence's rows one batch after the other, but starts
// faster, and many sequences have tiles enough for all SMs (where one of them may have most of the rows, so not
// past 8192).  us from a graph, every second row kept, 8 heads of 128, F16 / Q8_0, long : short:
//    1 sequence,   1024 rows   7.3 : 10.0 /  7.1 :  9.6     2048   8.8 : 18.7 /  7.9 : 17.9
//    4             2048        8.9 :  8.0 /  7.9 :  8.7     4096   9.7 : 14.8 /  9.7 : 15.6
//    8             4096        9.7 :  9.2 /  9.7 : 11.3     8192  18.7 : 18.2 / 10.8 : 22.3
//   16             4096        9.6 :  7.6 /  9.6 :  7.7     8192  18.9 : 16.2 / 10.8 : 14.1
//   64             4096        9.7 :  7.2 /  9.4 :  6.6     8192  18.4 : 14.6 / 10.8 :  9.4
static bool long_lists(int64_t n_seq, int64_t n_rows) { return n_rows >= std::min<int64_t>(512 * (n_seq + 1), 8192); }

// How a long list is cut: a thread for each 16 bytes of a row of a group's tiles, some rows a pass (and for each 2 to 8 bytes
// of scales).
static int64_t cut_long(const KvCache& c, int64_t n_rows, LongParams* q) {
    const int n16 = c.dim >> (c.q8 ? 4 : 3), ns = c.q8 ? (c.dim >> 4) / (c.dim % 128 == 0 ? 8 : c.dim % 64 == 0 ? 4 : 2) : 0;
    // (as few tiles as make chunks of CMP_CHUNK rows: what lies together is moved together)
    const int tiles = std::min(2 * c.n_kv, std::max(1, std::min(CMP_THREADS, CMP_THREADS * CMP_UNITS / CMP_CHUNK) / n16));
    int rows = CMP_THREADS / (tiles * n16) * CMP_UNITS;
    if (ns) rows = std::min(rows, CMP_THREADS / (tiles * ns) * CMP_SCALES);
    q->group_tiles = tiles;
    q->groups = (2 * c.n_kv + tiles - 1) / tiles;
    q->chunk_rows = std::min(rows, CMP_CHUNK);
    q->chunks = (int)((n_rows + q->chunk_rows - 1) / q->chunk_rows);
    return (int64_t)q->chunks * q->groups;
}

int64_t compact_count_words(const KvCache& c, int64_t n_seq, int64_t n_rows) {
    if (!long_lists(n_seq, n_rows)) return 0;
    LongParams q;
    const int64_t n = cut_long(c, n_rows, &q);
    // (the counter of chunks goes past the last by one for each CTA: it stays within 32 bits)
    return n <= INT_MAX - (1 << 20) ? n + 2 : -1;
}

cudaError_t launch_kv_compact(const KvCache& c, const int32_t* refs, int64_t n_seq, int64_t n_rows, const int32_t* pages,
                              int64_t max_pages, const int32_t* base, const int32_t* starts, const int32_t* rows,
                              int32_t* new_lens, int* count, int* err, int sms, int* launches, cudaStream_t s) {
    CompactParams p;
    p.c = c;
    p.refs = refs;
    p.pages = pages;
    p.base = base;
    p.starts = starts;
    p.rows = rows;
    p.new_lens = new_lens;
    p.err = err;
    p.max_pages = max_pages;
    p.n_rows = n_rows;
    p.n_seq = (int)n_seq;
    cudaError_t e;
    if (long_lists(n_seq, n_rows)) {
        LongParams q;
        q.m = p;
        const int64_t n = cut_long(c, n_rows, &q);
        q.turn = count;
        q.flags = count + 2;
        auto kern = c.dim % 128 == 0 ? k_kv_compact_long<uint2> : c.dim % 64 == 0 ? k_kv_compact_long<uint32_t> : k_kv_compact_long<uint16_t>;
        const int grid = (int)std::min<int64_t>(n, (int64_t)sms * CMP_CTAS);
        e = launch_overlapped(kern, grid, CMP_LONG_THREADS, CMP_UNITS * CMP_THREADS * 16, s, q);
    } else {
        // About CMP_TARGET CTAs an SM: several tiles to one where there are many sequences, columns of at least 32 bytes of a row
        // (a sector) where there are few.
        const int pieces = c.dim >> (c.q8 ? 4 : 3), tiles = 2 * c.n_kv;
        const int64_t want = (int64_t)CMP_TARGET * sms;
        p.group = (int)std::min<int64_t>(std::max<int64_t>(n_seq * tiles / want, 1), tiles);
        const int64_t units = n_seq * ((tiles + p.group - 1) / p.group);
        p.width = pieces;
        while (p.width > 2 && units * ((pieces + p.width - 1) / p.width) < want) p.width = (p.width + 1) / 2;
        p.cut = (pieces + p.width - 1) / p.width;
        p.apart = c.q8 && p.cut > 1;
        e = launch_overlapped(k_kv_compact, (int)std::min<int64_t>(units * (p.cut + p.apart), (int64_t)sms * 8), CMP_THREADS, 0, s, p);
    }
    if (e == cudaSuccess) ++*launches;
    return e;
}

// ---- copy --------------------------------------------------------------------------------
//
// Whole pages, 16 KB a turn of a CTA, eight 16-byte loads of a thread on their way together.

struct CopyParams {
    KvCache from, to;
    const int32_t* src;
    const int32_t* dst;
    int* err;
    int64_t n, bytes;  // bytes of a page in one pool
};

constexpr int COPY_UNITS = 8;

__global__ void __launch_bounds__(PG_THREADS) k_kv_copy(const CopyParams p) {
    griddep_release();
    griddep_wait();
    constexpr int64_t CHUNK = (int64_t)PG_THREADS * COPY_UNITS * 16;
    const int64_t chunks = (p.bytes + CHUNK - 1) / CHUNK, total = 2 * p.n * chunks;
    for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
        const int64_t i = u / (2 * chunks), at = u - i * 2 * chunks, is_v = at >= chunks, off = (at - is_v * chunks) * CHUNK;
        const int from = p.src[i], to = p.dst[i];
        if ((unsigned)from >= (unsigned)p.from.n_pages || (unsigned)to >= (unsigned)p.to.n_pages) {
            if (at == 0 && threadIdx.x == 0) record_error(p.err, SYN_DEVERR_BOUNDS);
            continue;
        }
        const uint8_t* a = (is_v ? p.from.v : p.from.k) + from * p.from.page_stride;
        uint8_t* b = (is_v ? p.to.v : p.to.k) + to * p.to.page_stride;
        uint4 held[COPY_UNITS];
#pragma unroll
        for (int x = 0; x < COPY_UNITS; x++) {
            const int64_t o = off + (x * PG_THREADS + threadIdx.x) * 16;
            if (o < p.bytes && SYN_IN_BOUNDS(in_pool(p.from, a + o - (is_v ? p.from.v : p.from.k), 16))) held[x] = *reinterpret_cast<const uint4*>(a + o);
        }
#pragma unroll
        for (int x = 0; x < COPY_UNITS; x++) {
            const int64_t o = off + (x * PG_THREADS + threadIdx.x) * 16;
            if (o < p.bytes && SYN_IN_BOUNDS(in_pool(p.to, b + o - (is_v ? p.to.v : p.to.k), 16))) *reinterpret_cast<uint4*>(b + o) = held[x];
        }
    }
}

cudaError_t launch_kv_copy(const KvCache& from, const KvCache& to, int64_t n, const int32_t* src, const int32_t* dst, int* err,
                           int sms, cudaStream_t s) {
    const CopyParams p{from, to, src, dst, err, n, from.tile * from.n_kv};
    const int64_t chunk = (int64_t)PG_THREADS * COPY_UNITS * 16, total = 2 * n * ((p.bytes + chunk - 1) / chunk);
    return launch_overlapped(k_kv_copy, (int)std::min<int64_t>(total, (int64_t)sms * 16), PG_THREADS, 0, s, p);
}

#ifdef SYN_DEBUG
SYN_BOUNDS_READER(debug_bounds_kv_pages)
#endif

}  // namespace syn
