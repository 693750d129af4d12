// attn_tree.cu — attention of drafted tokens, the nodes of a tree, of each sequence: a node sees the context and
// its own ancestors (the kernel is in attn_prefill.cuh).
#include "attn_prefill.cuh"

namespace syn {

cudaError_t launch_attn_tree(const KvCache& c, const AttnDesc& a, int64_t n_seq, int64_t n_tok, const void* q,
                             const int32_t* starts, const int32_t* parents, const int32_t* pages, int64_t max_pages,
                             const int32_t* lens, void* out, float* part, int* count, bool split, int* err, int sms,
                             int* launches, cudaStream_t s) {
    return launch_attn_tokens<true>(c, c, a, n_seq, n_tok, q, starts, parents, pages, pages, max_pages, lens, out, part, count,
                                    split, err, sms, launches, s);
}

#ifdef SYN_DEBUG
SYN_BOUNDS_READER(debug_bounds_attn_tree)
#endif

}  // namespace syn
