// attn_prefill.cu — attention of several new tokens of each sequence (the kernel is in attn_prefill.cuh), and
// the expansion of a Q8_0 cache ahead of it.
#include "attn_prefill.cuh"

namespace syn {

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

int64_t prefill_part_floats(int64_t n_seq, int64_t n_tok, int n_heads, int n_kv, int dim, int sms) {
    return part_floats(dim, sms) + redo_entries(n_seq, n_tok, n_heads, n_kv, dim) * (int64_t)(sizeof(Redo) / 4);
}

cudaError_t launch_attn_prefill(const KvCache& c, const KvCache& raw, const AttnDesc& a, int64_t n_seq, int64_t n_tok,
                                const void* q, const int32_t* starts, const int32_t* pages, const int32_t* raw_pages,
                                int64_t max_pages, const int32_t* lens, void* out, float* part, int* count, bool split,
                                int* err, int sms, int* launches, cudaStream_t s) {
    return launch_attn_tokens<false>(c, raw, a, n_seq, n_tok, q, starts, nullptr, pages, raw_pages, max_pages, lens, out, part,
                                     count, split, err, sms, launches, s);
}

#ifdef SYN_DEBUG
SYN_BOUNDS_READER(debug_bounds_attn_prefill)
#endif

}  // namespace syn
