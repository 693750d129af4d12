// kernels.h — host-side launchers of the libsyn kernels (internal to the library).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace syn {

cudaError_t launch_quantize(int type, const float* src, void* dst, int64_t n_blocks, int* range_err,
                            int sms, cudaStream_t s);
cudaError_t launch_dequantize(int type, const void* src, float* dst, int64_t n_blocks, int sms,
                              cudaStream_t s);
cudaError_t launch_quantize_act(int xtype, const float* X, int64_t n_blocks, int8_t* qs, float* d,
                                int16_t* bsums, int sms, cudaStream_t s);
cudaError_t launch_act_half(int xtype, const float* X, int64_t n_blocks, void* xh, int sms,
                            cudaStream_t s);
// Q4_K / Q6_K weights -> fp16 values (n_blocks blocks, 256 halves each, row-major like W),
// each the fp32 dequantization rounded once to fp16.
cudaError_t launch_deq_half(int type, const void* src, void* dst, int64_t n_blocks, int sms, cudaStream_t s);
cudaError_t launch_block_sums(int type, const void* W, int64_t n_out, int64_t nb, const void* Xq,
                              int64_t n_tok, int32_t* S, cudaStream_t s);

// Decode products of up to GEMV_MAX_JOBS independent matrices in one launch.
constexpr int GEMV_MAX_JOBS = 16;
struct GemvDesc {
    int type;
    const void* W;
    int64_t n_out, n_in;
    const float* X;
    float* Y;
};
// Decode products: Y = W * Xq for few tokens.  Two launches: the activation conversion into
// the workspace ws (gemv_workspace_bytes), then the decode kernel as its programmatic
// dependent (it streams weights before waiting for the conversion).  no_split: every output
// row is computed by one warp (the deterministic mode), else long rows may be split.
cudaError_t launch_gemv_batch(int n, const GemvDesc* d, int64_t n_tok, void* ws, int* err, int sms, bool no_split,
                              cudaStream_t s);
int64_t gemv_workspace_bytes(int n, const GemvDesc* d, int64_t n_tok);

// Shared memory one token of a matrix's converted activations takes in the decode kernel;
// a launch holds at most gemv_act_limit() bytes of them (all matrices, one token).
int64_t gemv_act_bytes(int type, int64_t n_in);
int64_t gemv_act_limit();

// The SM limit set by syn_set_sm_limit (0: none).
int sm_limit();

// Prefill product on the tensor cores.  xh: n_tok x n_in fp16 activations, written by
// launch_act_half immediately before on the same stream (the product kernel is its
// programmatic dependent).  Y is overwritten, except where the product splits along K: those
// columns are added into, so the caller enqueues gemm_zero_y() before launch_act_half.
cudaError_t launch_gemm(int type, const void* W, int64_t n_out, int64_t n_in, const void* xh,
                        int64_t n_tok, float* Y, int* err, int sms, cudaStream_t s);
cudaError_t gemm_zero_y(float* Y, int64_t n_out, int64_t n_in, int64_t n_tok, int sms, cudaStream_t s);
// The prefill schedule of a product (host only): {S, m_full, stream-K, tiles}.
void gemm_plan(int64_t n_out, int64_t n_in, int64_t n_tok, int sms, int out[4]);

// F16 weights (n_in % 8 == 0): X -> fp16 (round to nearest even) into xh, and the decode
// product reading W and the fp16 activations from ws (n_tok * n_in halves).
cudaError_t launch_x_to_half(const float* X, int64_t n, void* xh, int sms, cudaStream_t s);
cudaError_t launch_gemv_f16(const void* W, int64_t n_out, int64_t n_in, const float* X, int64_t n_tok, float* Y,
                            void* ws, int sms, cudaStream_t s);

// ---- paged key-value cache and attention (kv_append.cu, attn_decode.cu, attn_prefill.cu) ----

struct KvCache;  // kv_cache.cuh

struct RopeDesc {
    const uint64_t* turns;  // n_rot / 2 turns per position, as 64-bit fractions
    const uint8_t* axis;    // n_rot / 2 position axes, or NULL (all 0)
    int n_rot, n_axes, halves;
    float magnitude;
};
struct AttnDesc {
    const float* slopes;    // n_heads, or NULL
    const int32_t* prefix;  // per sequence, or NULL
    const int32_t* first;   // per query, or NULL
    int64_t q_stride, out_stride;
    int n_heads, window, out_f16;
    float scale, cap;
};

cudaError_t launch_kv_append(const KvCache& c, const RopeDesc& r, int64_t n_tok, const float* q, int64_t q_stride,
                             int n_heads, void* q_out, const float* k, int64_t k_stride, const float* v,
                             int64_t v_stride, const int32_t* pos, const int64_t* slots, int* err, int sms,
                             cudaStream_t s);
cudaError_t launch_kv_read(const KvCache& c, int64_t n, const int64_t* slots, void* k, void* v, int* err, int sms,
                           cudaStream_t s);

// One token of each sequence.  part (decode_part_floats) and count (decode_count_words, zero
// before the first call and left zero by every call) are the launch's scratch.  whole: no item
// is split between CTAs.  *launches gets the number of kernels.
constexpr int DECODE_CTAS_PER_SM = 5;
cudaError_t launch_attn_decode(const KvCache& c, const AttnDesc& a, int64_t n_seq, const void* q, const int32_t* pages,
                               int64_t max_pages, const int32_t* lens, void* out, float* part, int* count, bool whole,
                               int* err, int sms, int* launches, cudaStream_t s);
int64_t decode_count_words(int64_t n_seq, int n_heads, int n_kv, int dim);
int64_t decode_part_floats(int n_heads, int n_kv, int dim, int sms);

// Several new tokens of each sequence (packed, starts[s] .. starts[s+1]).  part:
// prefill_part_floats (partials, then the list of rows to be computed again); count: at least `sms` + 2 words, as above.  split: items may be split
// between CTAs.
cudaError_t launch_attn_prefill(const KvCache& c, const KvCache& raw, const AttnDesc& a, int64_t n_seq, int64_t n_tok,
                                const void* q, const int32_t* starts, const int32_t* pages, const int32_t* raw_pages,
                                int64_t max_pages, const int32_t* lens, void* out, float* part, int* count, bool split,
                                int* err, int sms, int* launches, cudaStream_t s);
int64_t prefill_part_floats(int64_t n_seq, int64_t n_tok, int n_heads, int n_kv, int dim, int sms);
// The rows of a Q8_0 cache that the sequences hold as the pages of an F16 cache of scratch (k, v: n_seq *
// max_pages pages of n_kv tiles each; table: its page table, n_seq x max_pages, -1 for a page outside the
// pool).  window > 0: rows ahead of every query's window are left out.
cudaError_t launch_kv_expand(const KvCache& c, int64_t n_seq, int64_t n_tok, const int32_t* starts, const int32_t* pages, int64_t max_pages,
                             const int32_t* lens, int window, void* k, void* v, int32_t* table, int sms, cudaStream_t s);

// What the C entry points of api_attn.cu share with api.cu: the SMs of this call and the
// status words ([0]) of the current device; the attention's workspace of (device, stream), at
// least `zeroed` bytes that were zero when it was allocated, then (from byte *zeroed_at on) at
// least `rest` bytes; the deterministic mode.
int call_state(int* sms, int** words);
int attn_workspace(cudaStream_t s, size_t zeroed, size_t rest, size_t* zeroed_at, void** out);
// The workspace of (current device, stream) for the expanded rows of a Q8_0 cache.
int attn_rows_workspace(cudaStream_t s, size_t bytes, void** out);
bool deterministic();

// Shared-memory limit and resident CTAs per SM of a kernel, looked up once per device.
class ResidentCtas {
    std::atomic<int> n_[64] = {};

  public:
    cudaError_t get(const void* kern, int threads, int smem, int* out) {
        int dev;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64 && n_[dev].load() > 0) {
            *out = n_[dev].load();
            return cudaSuccess;
        }
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        int n = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        if (dev >= 0 && dev < 64) n_[dev].store(n);
        *out = n;
        return cudaSuccess;
    }
};

// Launches a kernel that may start before the one ahead of it on the stream has finished
// (programmatic stream serialization).  The kernel runs griddep_wait() (common.cuh) before it
// touches global memory; only its launch and set-up overlap.
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kern)(P...), int grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Adds n to the count syn_launch_count reports.
void note_launches(int n);

// The status word of syn_mul_mat_prefill_static's fixed array on device dev: *word gets it
// (0 when that entry point has not run on dev); clear != 0 resets it.  Allocates nothing;
// the caller synchronizes the device first.
int static_status(int dev, int clear, int* word);

#ifdef SYN_DEBUG
// SYN_DEBUG build: the index-check status word of each kernel file on the current device
// (SYN_DEVERR_BOUNDS when a check failed; -1 if unreadable), reset when clear != 0, and a
// launch whose one check is given an out-of-range index on purpose (the access it guards,
// into a shared array twice the checked size, is skipped).
int debug_bounds_quant(int clear);
int debug_bounds_gemv(int clear);
int debug_bounds_gemv_f16(int clear);
int debug_bounds_gemm(int clear);
int debug_bounds_kv_append(int clear);
int debug_bounds_attn_decode(int clear);
int debug_bounds_attn_prefill(int clear);
cudaError_t launch_bounds_selftest(cudaStream_t s);
#endif

}  // namespace syn
