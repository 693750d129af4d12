// api_attn.cu — the C entry points of the paged key-value cache, its pages and its attention, and of the
// log probabilities (declared in include/syn.h): argument checks, workspaces, dispatch to kv_append.cu,
// kv_pages.cu, attn_decode.cu, attn_prefill.cu, attn_tree.cu and logprobs.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "kv_cache.cuh"
#include "syn.h"

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxHeads = 1024;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Checks a cache descriptor and turns it into what the kernels take.
int cache_of(const syn_kv_cache* c, syn::KvCache* out) {
    if (!c) return SYN_ERR_NULL;
    if (c->type != SYN_TYPE_F16 && c->type != SYN_TYPE_Q8_0) return SYN_ERR_TYPE;
    const int64_t tile = syn_kv_tile_bytes(c->type, c->head_dim, c->page_size);
    if (tile < 0 || c->n_kv_heads < 1 || c->n_kv_heads > kMaxHeads || c->n_pages < 1 || c->n_pages > INT32_MAX)
        return SYN_ERR_SHAPE;
    const int64_t packed = tile * c->n_kv_heads;
    const int64_t stride = c->page_stride ? c->page_stride : packed;
    if (stride < packed || stride % 16 || stride > kMaxElems / c->n_pages || stride >= (int64_t(1) << 35))
        return SYN_ERR_SHAPE;
    if (!c->k || !c->v) return SYN_ERR_NULL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return SYN_ERR_ALIGN;
    out->k = static_cast<uint8_t*>(c->k);
    out->v = static_cast<uint8_t*>(c->v);
    out->n_pages = c->n_pages;
    out->page_stride = stride;
    out->tile = tile;
    out->n_kv = c->n_kv_heads;
    out->dim = c->head_dim;
    out->page_shift = __builtin_ctz((unsigned)c->page_size);
    out->q8 = c->type == SYN_TYPE_Q8_0;
    return SYN_OK;
}

// Checks the attention's options and, where there are rows, q / out against the cache.
int attn_of(const syn_attn* a, const syn::KvCache& c, int64_t rows, const void* q, const void* out, syn::AttnDesc* d) {
    if (!a) return SYN_ERR_NULL;
    if (a->out_type != SYN_OUT_F32 && a->out_type != SYN_OUT_F16) return SYN_ERR_TYPE;
    if (a->n_heads < 1 || a->n_heads > kMaxHeads || a->n_heads % c.n_kv || a->window < 0 || !std::isfinite(a->scale) ||
        !std::isfinite(a->cap) || a->cap < 0.0f)
        return SYN_ERR_SHAPE;
    const int64_t row = (int64_t)a->n_heads * c.dim;
    const int64_t qs = a->q_stride ? a->q_stride : row, os = a->out_stride ? a->out_stride : row;
    const int64_t most = kMaxElems / (rows ? rows : 1);
    if (qs < row || os < row || qs % 8 || os % 8 || qs > most || os > most) return SYN_ERR_SHAPE;
    if (rows && (!q || !out)) return SYN_ERR_NULL;
    if (!aligned(q, 16) || !aligned(out, 16)) return SYN_ERR_ALIGN;
    if (!aligned(a->slopes, 4) || !aligned(a->prefix, 4) || !aligned(a->first, 4)) return SYN_ERR_ALIGN;
    d->slopes = a->slopes;
    d->prefix = a->prefix;
    d->first = a->first;
    d->q_stride = qs;
    d->out_stride = os;
    d->n_heads = a->n_heads;
    d->window = a->window;
    d->out_f16 = a->out_type == SYN_OUT_F16;
    // (past 2^80 the largest score alone counts, as products are multiples of 2^-48; they are below 2^47, with Q8_0
    // keys of the largest scale, so that a score times log2(e) stays finite)
    d->scale = std::min(std::max(a->scale, -0x1p80f), 0x1p80f);
    d->cap = a->cap;
    return SYN_OK;
}

int check_cuda(cudaError_t e) { return e == cudaSuccess ? SYN_OK : SYN_ERR_CUDA; }

// The attention scratch of a stream: counters first (zero between calls), then the partials.
constexpr size_t kCountBytes = size_t(1) << 20;

// A Q8_0 prefill expands its cache to fp16 ahead of the kernel, once, where the kernel would expand each
// row many times: once for every 256 (token, head) rows of a sequence that see it.  It does so from this
// many such tiles a sequence on average on, and up to kExpandBytes of scratch in all.  Measured on GB300,
// 32 / 8 heads, one call at a time over a cold L2, expanded in the kernel / ahead (us).  8 sequences of 256, 512,
// 1024 and 2048 tokens, all new (4, 8, 16 and 32 tiles each):
//   slopes, heads of 64:   31 / 33,  56 / 54,  128 / 109,  378 / 279
//   slopes, heads of 128:  40 / 41,  68 / 66,  156 / 128,  453 / 316
//   slopes, heads of 256:  44 / 50,  93 / 95,  253 / 220,  828 / 657
//   none, heads of 64:     24 / 28,  42 / 47,   89 / 88,   236 / 219
//   none, heads of 128:    29 / 36,  50 / 58,  113 / 111,  322 / 279
//   none, heads of 256:    42 / 45,  87 / 82,  234 / 203,  760 / 607
// One sequence of 16384 rows, the last 512, 1024 and 2048 new (8, 16 and 32 tiles): slopes, heads of 128
// 240 / 164, 416 / 259, 746 / 456; none, heads of 128 162 / 144, 283 / 227, 515 / 394.
// (So 32 is late where there are no slopes and many cached rows, and for heads of 256.)
int64_t expand_tiles(const syn::KvCache& c, const syn::AttnDesc& a) {
    return (a.slopes || a.cap > 0.0f) && c.dim <= 128 ? 8 : 32;
}
constexpr int64_t kExpandBytes = int64_t(1) << 31;  // (a power of two: so is what the workspace is rounded up to)

int scratch_for(cudaStream_t s, int64_t count_words, int64_t part_floats, int** count, float** part) {
    // a multiple of a fixed step, so that a growing batch does not reallocate at every call
    const size_t cb = ((size_t)count_words * 4 + kCountBytes - 1) / kCountBytes * kCountBytes;
    const size_t pb = ((size_t)part_floats * 4 + kCountBytes - 1) / kCountBytes * kCountBytes;
    void* p;
    size_t at;
    const int rc = syn::attn_workspace(s, cb, pb, &at, &p);
    if (rc) return rc;
    *count = static_cast<int*>(p);
    *part = reinterpret_cast<float*>(static_cast<uint8_t*>(p) + at);
    return SYN_OK;
}

}  // namespace

extern "C" {

int64_t syn_kv_tile_bytes(int type, int head_dim, int page_size) {
    if ((type != SYN_TYPE_F16 && type != SYN_TYPE_Q8_0) || head_dim < 32 || head_dim > 256 || head_dim % 32 ||
        page_size < 8 || page_size > 65536 || (page_size & (page_size - 1)))
        return -1;
    const int64_t n = (int64_t)page_size * head_dim;
    return type == SYN_TYPE_F16 ? 2 * n : n + n / 16;
}

int syn_rope_turns(int n_rot, double base, double scale, const float* factors, uint64_t* out) {
    if (n_rot < 0 || n_rot > 256 || n_rot % 8 || !(base > 0.0) || !std::isfinite(base) || !std::isfinite(scale))
        return SYN_ERR_SHAPE;
    if (n_rot == 0) return SYN_OK;
    if (!out) return SYN_ERR_NULL;
    for (int i = 0; i < n_rot / 2; i++) {
        const double f = factors ? (double)factors[i] : 1.0;
        if (!(std::fabs(f) > 0.0) || !std::isfinite(f)) return SYN_ERR_RANGE;
    }
    for (int i = 0; i < n_rot / 2; i++) {
        const double f = factors ? (double)factors[i] : 1.0;
        const double turns = scale * std::pow(base, -2.0 * i / n_rot) / f / 6.283185307179586476925286766559;
        const double frac = turns - std::floor(turns);  // whole turns per position do nothing
        const double scaled = std::ldexp(frac, 64);
        out[i] = scaled >= 18446744073709551616.0 ? 0 : (uint64_t)scaled;
    }
    return SYN_OK;
}

int syn_kv_append(const syn_kv_cache* cache, const syn_rope* rope, int64_t n_tok, const float* q, int64_t q_stride,
                  int n_heads, void* q_out, const float* k, int64_t k_stride, const float* v, int64_t v_stride,
                  const int32_t* pos, const int64_t* slots, syn_stream_t stream) {
    syn::KvCache c;
    int rc = cache_of(cache, &c);
    if (rc) return rc;
    if (!rope) return SYN_ERR_NULL;
    if (rope->layout != SYN_ROPE_ADJACENT && rope->layout != SYN_ROPE_HALVES) return SYN_ERR_TYPE;
    if (rope->n_rot < 0 || rope->n_rot > c.dim || rope->n_rot % 8 || rope->n_axes < 1 || rope->n_axes > 8 ||
        !std::isfinite(rope->magnitude))
        return SYN_ERR_SHAPE;
    const int64_t kv_row = (int64_t)c.n_kv * c.dim, q_row = (int64_t)n_heads * c.dim;
    if (!k_stride) k_stride = kv_row;
    if (!v_stride) v_stride = kv_row;
    if (!q_stride) q_stride = q_row;
    if (n_tok < 0 || n_tok > INT32_MAX || n_heads < 0 || n_heads > kMaxHeads || k_stride < kv_row || v_stride < kv_row ||
        k_stride % 4 || v_stride % 4 || (n_heads && (q_stride < q_row || q_stride % 4)))
        return SYN_ERR_SHAPE;
    if (n_tok == 0) return SYN_OK;
    if (k_stride > kMaxElems / n_tok || v_stride > kMaxElems / n_tok || q_stride > kMaxElems / n_tok) return SYN_ERR_SHAPE;
    if (!k || !v || !slots || (n_heads && (!q || !q_out)) || (rope->n_rot && (!pos || !rope->turns))) return SYN_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8) || !aligned(pos, 4) || !aligned(rope->turns, 8) ||
        (n_heads && (!aligned(q, 16) || !aligned(q_out, 16))))
        return SYN_ERR_ALIGN;
    int sms, *words;
    rc = syn::call_state(&sms, &words);
    if (rc) return rc;
    syn::RopeDesc r;
    r.turns = rope->turns;
    r.axis = rope->axis;
    r.n_rot = rope->n_rot;
    r.n_axes = rope->n_axes;
    r.halves = rope->layout == SYN_ROPE_HALVES;
    r.magnitude = rope->magnitude;
    rc = check_cuda(syn::launch_kv_append(c, r, n_tok, q, q_stride, n_heads, q_out, k, k_stride, v, v_stride, pos, slots,
                                          words, sms, reinterpret_cast<cudaStream_t>(stream)));
    if (rc == SYN_OK) syn::note_launches(1);
    return rc;
}

int syn_kv_read(const syn_kv_cache* cache, int64_t n, const int64_t* slots, void* k, void* v, syn_stream_t stream) {
    syn::KvCache c;
    int rc = cache_of(cache, &c);
    if (rc) return rc;
    if (n < 0 || n > kMaxElems / ((int64_t)c.n_kv * c.dim)) return SYN_ERR_SHAPE;
    if (n == 0) return SYN_OK;
    if (!slots || !k || !v) return SYN_ERR_NULL;
    if (!aligned(slots, 8) || !aligned(k, 16) || !aligned(v, 16)) return SYN_ERR_ALIGN;
    int sms, *words;
    rc = syn::call_state(&sms, &words);
    if (rc) return rc;
    rc = check_cuda(syn::launch_kv_read(c, n, slots, k, v, words, sms, reinterpret_cast<cudaStream_t>(stream)));
    if (rc == SYN_OK) syn::note_launches(1);
    return rc;
}

int syn_attn_decode(const syn_kv_cache* cache, const syn_attn* attn, int64_t n_seq, const void* q, const int32_t* pages,
                    int64_t max_pages, const int32_t* lens, void* out, syn_stream_t stream) {
    syn::KvCache c;
    int rc = cache_of(cache, &c);
    if (rc) return rc;
    if (n_seq < 0 || n_seq > INT32_MAX || max_pages < (n_seq > 0) || max_pages > INT32_MAX) return SYN_ERR_SHAPE;
    syn::AttnDesc a;
    rc = attn_of(attn, c, n_seq, q, out, &a);
    if (rc) return rc;
    if (n_seq == 0) return SYN_OK;
    if (!pages || !lens) return SYN_ERR_NULL;
    if (!aligned(pages, 4) || !aligned(lens, 4)) return SYN_ERR_ALIGN;
    int sms, *words;
    rc = syn::call_state(&sms, &words);
    if (rc) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int* count;
    float* part;
    rc = scratch_for(s, syn::decode_count_words(n_seq, a.n_heads, c.n_kv, c.dim),
                     syn::decode_part_floats(a.n_heads, c.n_kv, c.dim, sms), &count, &part);
    if (rc) return rc;
    int launches = 0;
    rc = check_cuda(syn::launch_attn_decode(c, a, n_seq, q, pages, max_pages, lens, out, part, count,
                                            syn::deterministic(), words, sms, &launches, s));
    syn::note_launches(launches);
    return rc;
}

int syn_attn_prefill(const syn_kv_cache* cache, const syn_attn* attn, int64_t n_seq, int64_t n_tok, const void* q,
                     const int32_t* starts, const int32_t* pages, int64_t max_pages, const int32_t* lens, void* out,
                     syn_stream_t stream) {
    syn::KvCache c;
    int rc = cache_of(cache, &c);
    if (rc) return rc;
    if (n_seq < 0 || n_seq > INT32_MAX || n_tok < 0 || max_pages < (n_seq > 0 && n_tok > 0) || max_pages > INT32_MAX)
        return SYN_ERR_SHAPE;
    syn::AttnDesc a;
    rc = attn_of(attn, c, n_seq ? n_tok : 0, q, out, &a);
    if (rc) return rc;
    if (n_tok > (INT32_MAX - 1024) / a.n_heads) return SYN_ERR_SHAPE;  // 32-bit row numbers
    if (n_seq == 0 || n_tok == 0) return SYN_OK;
    if (!starts || !pages || !lens) return SYN_ERR_NULL;
    if (!aligned(starts, 4) || !aligned(pages, 4) || !aligned(lens, 4)) return SYN_ERR_ALIGN;
    int sms, *words;
    rc = syn::call_state(&sms, &words);
    if (rc) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int* count;
    float* part;
    rc = scratch_for(s, sms + 2, syn::prefill_part_floats(n_seq, n_tok, a.n_heads, c.n_kv, c.dim, sms), &count, &part);
    if (rc) return rc;
    const syn::KvCache raw = c;
    const int32_t* raw_pages = pages;
    int launches = 0;
    // bytes of a page, as fp16, in one of the two scratch pools
    const int64_t page = (int64_t(2) * c.dim * c.n_kv) << c.page_shift;
    if (c.q8 && !syn::deterministic() && n_tok * (a.n_heads / c.n_kv) >= expand_tiles(c, a) * 256 * n_seq &&
        n_seq * max_pages <= kExpandBytes / (2 * page + 4)) {
        const int64_t pool = n_seq * max_pages * page;
        void* ws;
        rc = syn::attn_rows_workspace(s, (size_t)(2 * pool + n_seq * max_pages * 4), &ws);
        if (rc && rc != SYN_ERR_NOMEM) return rc;
        if (rc == SYN_OK) {  // (no room: expanded in the kernel)
            uint8_t* k = static_cast<uint8_t*>(ws);
            int32_t* table = reinterpret_cast<int32_t*>(k + 2 * pool);
            rc = check_cuda(syn::launch_kv_expand(c, n_seq, n_tok, starts, pages, max_pages, lens, a.prefix ? 0 : a.window, k, k + pool,
                                                  table, sms, s));
            if (rc) return rc;
            launches = 1;
            c.q8 = 0;
            c.k = k;
            c.v = k + pool;
            c.page_stride = page;
            c.tile = page / c.n_kv;
            c.n_pages = n_seq * max_pages;
            pages = table;
        }
    }
    rc = check_cuda(syn::launch_attn_prefill(c, raw, a, n_seq, n_tok, q, starts, pages, raw_pages, max_pages, lens, out, part, count,
                                             !syn::deterministic(), words, sms, &launches, s));
    syn::note_launches(launches);
    return rc;
}

int syn_attn_tree(const syn_kv_cache* cache, const syn_attn* attn, int64_t n_seq, int64_t n_tok, const void* q,
                  const int32_t* starts, const int32_t* parents, const int32_t* pages, int64_t max_pages, const int32_t* lens,
                  void* out, syn_stream_t stream) {
    syn::KvCache c;
    int rc = cache_of(cache, &c);
    if (rc) return rc;
    if (n_seq < 0 || n_seq > INT32_MAX || n_tok < 0 || max_pages < (n_seq > 0 && n_tok > 0) || max_pages > INT32_MAX)
        return SYN_ERR_SHAPE;
    syn::AttnDesc a;
    rc = attn_of(attn, c, n_seq ? n_tok : 0, q, out, &a);
    if (rc) return rc;
    if (n_tok > (INT32_MAX - 1024) / a.n_heads) return SYN_ERR_SHAPE;  // 32-bit row numbers
    if (n_seq == 0 || n_tok == 0) return SYN_OK;
    if (!starts || !parents || !pages || !lens) return SYN_ERR_NULL;
    if (!aligned(starts, 4) || !aligned(parents, 4) || !aligned(pages, 4) || !aligned(lens, 4)) return SYN_ERR_ALIGN;
    int sms, *words;
    rc = syn::call_state(&sms, &words);
    if (rc) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int* count;
    float* part;
    rc = scratch_for(s, 4, syn::tree_part_floats(n_seq, n_tok, a.n_heads, c.n_kv, c.dim, sms), &count, &part);
    if (rc) return rc;
    int launches = 0;
    rc = check_cuda(syn::launch_attn_tree(c, a, n_seq, n_tok, q, starts, parents, pages, max_pages, lens, out, part, count,
                                          !syn::deterministic(), words, sms, &launches, s));
    syn::note_launches(launches);
    return rc;
}

int syn_kv_fork(const syn_kv_cache* cache, int32_t* refs, int64_t n_seq, const int32_t* pages, int64_t max_pages,
                const int32_t* lens, int64_t n_new, const int32_t* from, int32_t* new_pages, int32_t* new_lens,
                syn_stream_t stream) {
    syn::KvCache c;
    int rc = cache_of(cache, &c);
    if (rc) return rc;
    if (n_seq < 0 || n_seq > INT32_MAX || n_new < 0 || n_new > INT32_MAX || max_pages < (n_new > 0) || max_pages > INT32_MAX)
        return SYN_ERR_SHAPE;
    if (n_new == 0) return SYN_OK;
    if (!refs || !from || !new_pages || !new_lens || (n_seq && (!pages || !lens))) return SYN_ERR_NULL;
    if (!aligned(refs, 4) || !aligned(from, 4) || !aligned(new_pages, 4) || !aligned(new_lens, 4) || !aligned(pages, 4) ||
        !aligned(lens, 4))
        return SYN_ERR_ALIGN;
    int sms, *words;
    rc = syn::call_state(&sms, &words);
    if (rc) return rc;
    rc = check_cuda(syn::launch_kv_fork(c, refs, n_seq, pages, max_pages, lens, n_new, from, new_pages, new_lens, words, sms,
                                        reinterpret_cast<cudaStream_t>(stream)));
    if (rc == SYN_OK) syn::note_launches(1);
    return rc;
}

int syn_kv_extend(const syn_kv_cache* cache, int32_t* refs, int64_t n_seq, int64_t n_tok, int32_t* pages, int64_t max_pages,
                  const int32_t* lens, const int32_t* starts, int32_t* new_lens, int64_t* slots, syn_stream_t stream) {
    syn::KvCache c;
    int rc = cache_of(cache, &c);
    if (rc) return rc;
    if (n_seq < 0 || n_seq > syn::KV_EXTEND_SEQS || n_tok < 0 || n_tok > INT32_MAX - 1024 || (!starts && n_tok != n_seq) ||
        max_pages < (n_seq > 0) || max_pages > INT32_MAX)
        return SYN_ERR_SHAPE;
    if (n_seq == 0) return SYN_OK;
    if (!refs || !pages || !lens || !new_lens) return SYN_ERR_NULL;
    if (!aligned(refs, 4) || !aligned(pages, 4) || !aligned(lens, 4) || !aligned(starts, 4) || !aligned(new_lens, 4) ||
        !aligned(slots, 8))
        return SYN_ERR_ALIGN;
    int sms, *words;
    rc = syn::call_state(&sms, &words);
    if (rc) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int* count;
    float* scratch;
    rc = scratch_for(s, 1, 4 * n_seq + 2 * syn::extend_items(c, n_seq, n_tok), &count, &scratch);
    if (rc) return rc;
    int launches = 0;
    rc = check_cuda(syn::launch_kv_extend(c, refs, n_seq, n_tok, pages, max_pages, lens, starts, new_lens, slots, scratch, words,
                                          sms, &launches, s));
    syn::note_launches(launches);
    return rc;
}

int syn_kv_compact(const syn_kv_cache* cache, const int32_t* refs, int64_t n_seq, int64_t n_rows, const int32_t* pages,
                   int64_t max_pages, const int32_t* base, const int32_t* starts, const int32_t* rows, int32_t* new_lens,
                   syn_stream_t stream) {
    syn::KvCache c;
    int rc = cache_of(cache, &c);
    if (rc) return rc;
    // (a CTA for each column of a tile: at most 17 of them)
    if (n_seq < 0 || n_seq > INT32_MAX / (34 * (int64_t)c.n_kv) || n_rows < 0 || n_rows > INT32_MAX - 1024 ||
        max_pages < (n_seq > 0) || max_pages > INT32_MAX)
        return SYN_ERR_SHAPE;
    if (n_seq == 0) return SYN_OK;
    if (!pages || !base || !starts || !new_lens || (n_rows && !rows)) return SYN_ERR_NULL;
    if (!aligned(refs, 4) || !aligned(pages, 4) || !aligned(base, 4) || !aligned(starts, 4) || !aligned(rows, 4) ||
        !aligned(new_lens, 4))
        return SYN_ERR_ALIGN;
    const int64_t count_words = syn::compact_count_words(c, n_seq, n_rows);
    if (count_words < 0) return SYN_ERR_SHAPE;
    int sms, *words;
    rc = syn::call_state(&sms, &words);
    if (rc) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int* count = nullptr;
    float* part;
    if (count_words) {
        rc = scratch_for(s, count_words, 1, &count, &part);
        if (rc) return rc;
    }
    int launches = 0;
    rc = check_cuda(syn::launch_kv_compact(c, refs, n_seq, n_rows, pages, max_pages, base, starts, rows, new_lens,
                                           count, words, sms, &launches, s));
    syn::note_launches(launches);
    return rc;
}

int syn_kv_trim(const syn_kv_cache* cache, int32_t* refs, int64_t n_seq, int32_t* pages, int64_t max_pages,
                const int32_t* lens, syn_stream_t stream) {
    syn::KvCache c;
    int rc = cache_of(cache, &c);
    if (rc) return rc;
    if (n_seq < 0 || n_seq > INT32_MAX || max_pages < (n_seq > 0) || max_pages > INT32_MAX) return SYN_ERR_SHAPE;
    if (n_seq == 0) return SYN_OK;
    if (!refs || !pages || !lens) return SYN_ERR_NULL;
    if (!aligned(refs, 4) || !aligned(pages, 4) || !aligned(lens, 4)) return SYN_ERR_ALIGN;
    int sms, *words;
    rc = syn::call_state(&sms, &words);
    if (rc) return rc;
    rc = check_cuda(syn::launch_kv_trim(c, refs, n_seq, pages, max_pages, lens, words, sms,
                                        reinterpret_cast<cudaStream_t>(stream)));
    if (rc == SYN_OK) syn::note_launches(1);
    return rc;
}

int syn_kv_copy(const syn_kv_cache* from, const syn_kv_cache* to, int64_t n, const int32_t* src, const int32_t* dst,
                syn_stream_t stream) {
    syn::KvCache a, b;
    int rc = cache_of(from, &a);
    if (rc == SYN_OK) rc = cache_of(to, &b);
    if (rc) return rc;
    if (a.q8 != b.q8) return SYN_ERR_TYPE;
    if (a.dim != b.dim || a.n_kv != b.n_kv || a.page_shift != b.page_shift || n < 0 || n > INT32_MAX) return SYN_ERR_SHAPE;
    if (n == 0) return SYN_OK;
    if (!src || !dst) return SYN_ERR_NULL;
    if (!aligned(src, 4) || !aligned(dst, 4)) return SYN_ERR_ALIGN;
    int sms, *words;
    rc = syn::call_state(&sms, &words);
    if (rc) return rc;
    rc = check_cuda(syn::launch_kv_copy(a, b, n, src, dst, words, sms, reinterpret_cast<cudaStream_t>(stream)));
    if (rc == SYN_OK) syn::note_launches(1);
    return rc;
}

int syn_logprobs(const syn_logits* opt, int64_t n_rows, int64_t n_vocab, const void* logits, int64_t n_ids, const int32_t* ids,
                 float* logprob, float* entropy, int64_t n_top, int32_t* top, float* top_logprob, syn_stream_t stream) {
    if (!opt) return SYN_ERR_NULL;
    if (opt->type != SYN_OUT_F32 && opt->type != SYN_OUT_F16) return SYN_ERR_TYPE;
    const int64_t words_of = (n_vocab + 31) / 32;
    const int64_t stride = opt->stride ? opt->stride : n_vocab, mask_stride = opt->mask_stride ? opt->mask_stride : words_of;
    if (n_rows < 0 || n_rows > INT32_MAX / 8 || n_vocab < 1 || n_vocab > (1 << 30) || stride < n_vocab || mask_stride < words_of ||
        n_ids < 0 || n_ids > 65536 || n_top < 0 || n_top > syn::LOGPROBS_TOP || !std::isfinite(opt->scale) ||
        !(opt->scale > 0.0f) || !std::isfinite(opt->cap) || opt->cap < 0.0f)
        return SYN_ERR_SHAPE;
    if (n_rows == 0) return SYN_OK;
    if (stride > kMaxElems / n_rows || mask_stride > kMaxElems / n_rows) return SYN_ERR_SHAPE;
    if (!logits || (n_ids && (!ids || !logprob)) || (n_top && (!top || !top_logprob))) return SYN_ERR_NULL;
    const bool f16 = opt->type == SYN_OUT_F16;
    if (!aligned(logits, f16 ? 2 : 4) || !aligned(opt->scales, 4) || !aligned(opt->mask, 4) || !aligned(ids, 4) ||
        !aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(top, 4) || !aligned(top_logprob, 4))
        return SYN_ERR_ALIGN;
    int sms, *words;
    const int rc = syn::call_state(&sms, &words);
    if (rc) return rc;
    syn::LogitsDesc d;
    d.stride = stride;
    d.scales = opt->scales;
    d.mask = opt->mask;
    d.mask_stride = mask_stride;
    d.f16 = f16;
    d.scale = opt->scale;
    d.cap = opt->cap;
    const int e = check_cuda(syn::launch_logprobs(d, n_rows, (int)n_vocab, logits, ids, (int)n_ids, logprob, entropy, (int)n_top,
                                                  top, top_logprob, syn::deterministic(), words, sms,
                                                  reinterpret_cast<cudaStream_t>(stream)));
    if (e == SYN_OK) syn::note_launches(1);
    return e;
}

}  // extern "C"
