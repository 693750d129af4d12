// logprobs.cu — log probabilities of given tokens, the entropy and the most likely tokens of rows of
// logits, in one pass over the logits.
//
//   z = scale * (cap > 0 ? cap*tanh(x/cap) : x) over the allowed tokens, d = z - z(largest x)
//   S = sum e^d, T = sum d e^d;  logp(v) = d_v - ln S,  entropy = ln S - T/S
// Both sums follow a running maximum: when it moves by r, S' = S e^r and T' = (T + r S) e^r.
//
// Bound: HBM (or L2, where the product that made the logits has just written them): every logit is read
// once, into the registers of the thread that keeps them, 32 at a time.
//   - A row is cut between the CTAs of a cluster (1 to 8, as many as the rows leave room for), which
//     send what they found to the first through its shared memory.  No CTA waits for another row's.
//   - The n_top largest: the 512 threads' own maxima are counted against a threshold, which is halved
//     in until between n_top and 2 n_top of them reach it; every logit below it is beaten by n_top others, so only the few
//     threads above it look through their 32 logits.  What they find is ordered by counting, for
//     each, the larger ones (ties: the lower token first).  Later pieces of a row start from the
//     n_top-th largest found so far.
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "kv_cache.cuh"

namespace cg = cooperative_groups;

namespace syn {

constexpr int LP_THREADS = 512;
constexpr int LP_HOLD = 32;      // logits in a thread's registers
constexpr int LP_TOP = LOGPROBS_TOP;
constexpr int LP_CLUSTER = 8;
constexpr uint32_t LP_NONE = 0x007FFFFFu;  // order_of(-inf)

struct LogprobParams {
    const void* x;
    int64_t stride;  // values between rows
    const float* scales;
    const uint32_t* mask;
    int64_t mask_stride;  // words between rows
    const int32_t* ids;
    float* logprob;
    float* entropy;
    int32_t* top;
    float* top_logprob;
    int* err;
    int64_t n_rows;
    int n_vocab, n_ids, n_top, cut;  // cut: CTAs of a row
    float scale, cap;
};

// A number that grows with the value (no NaN), and back.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_order(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ uint4 load_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// What a thread, a CTA and a row know of the sums: the largest logit x (NaN where there is one), S and T.
struct Sums {
    float x, s, t;
};

template <bool F16>
__device__ __forceinline__ float logit_at(const void* row, int64_t i) {
    return F16 ? __half2float(static_cast<const __half*>(row)[i]) : static_cast<const float*>(row)[i];
}

template <bool F16>
__global__ void __launch_bounds__(LP_THREADS, 2) k_logprobs(const LogprobParams p) {
    constexpr int E = F16 ? 8 : 4, V = LP_HOLD / E;  // logits of a 16-byte piece, pieces a thread holds
    constexpr int WARPS = LP_THREADS / 32;
    __shared__ uint64_t found[LP_TOP + 2 * LP_TOP * LP_HOLD], best[LP_TOP];
    __shared__ uint64_t sent[LP_CLUSTER * LP_TOP];  // (the first CTA's) the others' largest
    __shared__ Sums sent_sums[LP_CLUSTER], warp_sums[WARPS];
    __shared__ int sent_n[LP_CLUSTER], n_found;
    __shared__ uint32_t warp_lo[WARPS], warp_hi[WARPS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int part = p.cut > 1 ? (int)cg::this_cluster().block_rank() : 0;
    griddep_release();
    if (p.cut > 1) cg::this_cluster().barrier_arrive();  // (waited for before a row's stores: all have begun, and read the row before)
    griddep_wait();

    const int64_t rows_at_once = gridDim.x / p.cut;
    for (int64_t r = blockIdx.x / p.cut; r < p.n_rows; r += rows_at_once) {
        const uint8_t* row = static_cast<const uint8_t*>(p.x) + r * p.stride * (F16 ? 2 : 4);
        const uint32_t* mask = p.mask ? p.mask + r * p.mask_stride : nullptr;
        const float scale = p.scales ? p.scale * p.scales[r] : p.scale;
        const bool scale_ok = scale > 0.0f && scale < INFINITY;
        // pieces start on 16-byte boundaries: the first may begin before the row, the last end behind it
        const int head = (int)(reinterpret_cast<uintptr_t>(row) & 15) / (F16 ? 2 : 4);
        const int pieces = (head + p.n_vocab + E - 1) / E;
        const int per = (pieces + p.cut - 1) / p.cut, end = min(pieces, per * (part + 1));
        // (the larger logit's d is 0 exactly; a logit of -inf counts as a token that is not allowed)
        auto from = [&](float x, float x0) {
            return p.cap > 0.0f ? scale * (p.cap * tanhf(x / p.cap) - p.cap * tanhf(x0 / p.cap)) : scale * (x - x0);
        };
        auto join = [&](Sums a, const Sums& b) {
            const float x = max_nan(a.x, b.x), x0 = x == -INFINITY ? 0.0f : x;
            const float ra = a.x == -INFINITY ? 0.0f : from(a.x, x0), rb = b.x == -INFINITY ? 0.0f : from(b.x, x0);
            // (e^-200 is 0; 0 times infinity stays out)
            const float fa = expf(fmaxf(ra, -200.0f)), fb = expf(fmaxf(rb, -200.0f));
            Sums y;
            y.x = x;
            y.s = a.s * fa + b.s * fb;
            y.t = (a.t + fmaxf(ra, -200.0f) * a.s) * fa + (b.t + fmaxf(rb, -200.0f) * b.s) * fb;
            return y;
        };
        auto key_of = [&](float x, int token) { return ((uint64_t)order_of(x) << 32) | (uint32_t)~token; };
        // the n_top largest of the n keys in `found`, in order, into `best`; both stay as they are till the next barrier
        auto rank_found = [&](int n) {
            for (int i = tid; i < n; i += LP_THREADS) {
                const uint64_t mine = found[i];
                int rank = 0;
                for (int j = 0; j < n; j++) rank += found[j] > mine;
                if (rank < p.n_top) best[rank] = mine;
            }
        };

        Sums mine{-INFINITY, 0.0f, 0.0f};
        int n_best = 0;
        uint32_t floor_at = LP_NONE;  // logits up to here are out
        for (int base = per * part; base < end; base += LP_THREADS * V) {
            float v[LP_HOLD];
#pragma unroll
            for (int i = 0; i < V; i++) {
                const int at = base + i * LP_THREADS + tid, e0 = at * E - head;
                if (at < end && e0 >= 0 && e0 + E <= p.n_vocab) {
                    const uint4 w = load_once(row + (int64_t)e0 * (F16 ? 2 : 4));
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        if (F16) {
                            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
                            v[i * E + 2 * j % E] = y.x;
                            v[i * E + (2 * j + 1) % E] = y.y;
                        } else {
                            v[i * E + j] = __uint_as_float(u[j]);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < E; j++)
                        v[i * E + j] = at < end && e0 + j >= 0 && e0 + j < p.n_vocab ? logit_at<F16>(row, e0 + j) : -INFINITY;
                }
            }
            if (mask) {
                const int words = (p.n_vocab + 31) >> 5;
#pragma unroll
                for (int i = 0; i < V; i++) {
                    const int at = base + i * LP_THREADS + tid, e0 = at * E - head, w = max(e0, 0) >> 5;
                    const uint32_t lo = at < end ? __ldg(mask + w) : 0u;
                    const uint32_t hi = at < end && (e0 & 31) + E > 32 && e0 >= 0 && w + 1 < words ? __ldg(mask + w + 1) : 0u;
                    const uint32_t bits = e0 < 0 ? lo << -e0 : __funnelshift_r(lo, hi, e0 & 31);
#pragma unroll
                    for (int j = 0; j < E; j++)
                        if (!((bits >> j) & 1)) v[i * E + j] = -INFINITY;
                }
            }
            float x = -INFINITY;
#pragma unroll
            for (int j = 0; j < LP_HOLD; j++) x = max_nan(x, v[j]);
            // ---- the sums -----------------------------------------------------------------------
            if (x != -INFINITY) {
                if (!(x <= mine.x)) {
                    if (mine.x != -INFINITY) mine = join(mine, Sums{x, 0.0f, 0.0f});
                    mine.x = max_nan(mine.x, x);
                }
                float s[2] = {0.0f, 0.0f}, t[2] = {0.0f, 0.0f};
                if (p.cap > 0.0f) {
                    const float z0 = p.cap * tanhf(mine.x / p.cap);
#pragma unroll
                    for (int j = 0; j < LP_HOLD; j++) {
                        float d = scale * (p.cap * tanhf(v[j] / p.cap) - z0);
                        d = v[j] == -INFINITY ? -200.0f : fmaxf(d, -200.0f);
                        const float e = ex2(d * 1.4426950408889634f);
                        s[j & 1] += e;
                        t[j & 1] = fmaf(e, d, t[j & 1]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < LP_HOLD; j++) {
                        const float d = fmaxf(scale * (v[j] - mine.x), -200.0f);  // (2^-288 is 0)
                        const float e = ex2(d * 1.4426950408889634f);
                        s[j & 1] += e;
                        t[j & 1] = fmaf(e, d, t[j & 1]);
                    }
                }
                mine.s += s[0] + s[1];
                mine.t += t[0] + t[1];
            }
            // ---- the largest --------------------------------------------------------------------
            if (p.n_top > 0) {
                const int k = p.n_top;
                const uint32_t u = x == x ? order_of(x + 0.0f) : 0u;  // (-0 is 0)
                int n = __syncthreads_count(u > floor_at);
                if (n == 0) continue;
                uint32_t at_least = floor_at + 1;
                int tie = 0x7fffffff;  // of the logits at the threshold, those up to this token
                if (n > 2 * k) {
                    const uint32_t wl = __reduce_min_sync(0xffffffffu, u > floor_at ? u : 0xffffffffu), wh = __reduce_max_sync(0xffffffffu, u);
                    if (lane == 0) {
                        warp_lo[warp] = wl;
                        warp_hi[warp] = wh;
                    }
                    __syncthreads();
                    uint32_t lo = warp_lo[lane % WARPS], hi = warp_hi[lane % WARPS];
                    lo = __reduce_min_sync(0xffffffffu, lo);
                    hi = __reduce_max_sync(0xffffffffu, hi);
                    while (lo < hi && n > 2 * k) {  // (n: how many reach lo; fewer than k reach hi + 1)
                        const uint32_t mid = lo + (hi - lo) / 2 + 1;
                        const int c = __syncthreads_count(u >= mid);
                        if (c >= k) {
                            lo = mid;
                            n = c;
                        } else {
                            hi = mid - 1;
                        }
                    }
                    at_least = lo;
                    if (n > 2 * k) {  // many maxima are the same: the same again over the first tokens that have it
                        const float same = of_order(lo);
                        int first = 0x7fffffff;
#pragma unroll
                        for (int j = LP_HOLD - 1; j >= 0; j--)
                            if (v[j] == same) first = (base + j / E * LP_THREADS + tid) * E - head + j % E;
                        if (u > lo) first = -1;
                        int a = -1, b = p.n_vocab - 1;  // (fewer than k are at most a; more than 2k at most b)
                        while (n > 2 * k) {
                            const int mid = a + (b - a) / 2;
                            const int c = __syncthreads_count(first <= mid);
                            if (c >= k) {
                                b = mid;
                                n = c;
                            } else {
                                a = mid;
                            }
                        }
                        tie = b;
                    }
                }
                if (tid == 0) n_found = n_best;
                if (tid < n_best) found[tid] = best[tid];
                __syncthreads();
                if (u >= at_least) {
                    const float least = of_order(at_least);
#pragma unroll
                    for (int j = 0; j < LP_HOLD; j++) {
                        const int token = (base + j / E * LP_THREADS + tid) * E - head + j % E;
                        if (v[j] > least || (v[j] == least && token <= tie)) {
                            const int at = atomicAdd(&n_found, 1);
                            found[min(at, LP_TOP + 2 * LP_TOP * LP_HOLD - 1)] = key_of(v[j] + 0.0f, token);
                        }
                    }
                }
                __syncthreads();
                const int m = n_found;
                rank_found(m);
                __syncthreads();
                n_best = min(m, k);
                if (n_best == k) floor_at = (uint32_t)(best[k - 1] >> 32);
            }
        }

        // ---- the CTA's, then the row's -----------------------------------------------------------
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const Sums other{__shfl_xor_sync(0xffffffffu, mine.x, o), __shfl_xor_sync(0xffffffffu, mine.s, o),
                             __shfl_xor_sync(0xffffffffu, mine.t, o)};
            mine = lane & o ? join(other, mine) : join(mine, other);  // (the same order in both)
        }
        if (lane == 0) warp_sums[warp] = mine;
        __syncthreads();
        if (warp == 0) {
            mine = warp_sums[lane % WARPS];
#pragma unroll
            for (int o = WARPS / 2; o > 0; o >>= 1) {
                const Sums other{__shfl_xor_sync(0xffffffffu, mine.x, o), __shfl_xor_sync(0xffffffffu, mine.s, o),
                                 __shfl_xor_sync(0xffffffffu, mine.t, o)};
                mine = lane & o ? join(other, mine) : join(mine, other);
            }
        }
        if (p.cut > 1) {
            auto cluster = cg::this_cluster();
            cluster.barrier_wait();
            Sums* to_sums = cluster.map_shared_rank(sent_sums, 0);
            int* to_n = cluster.map_shared_rank(sent_n, 0);
            uint64_t* to = cluster.map_shared_rank(sent, 0);
            if (tid == 0) {
                to_sums[part] = mine;
                to_n[part] = n_best;
            }
            if (tid < n_best) to[part * LP_TOP + tid] = best[tid];
            cluster.sync();
            if (part == 0) {
                int at = 0;
                for (int c = 0; c < p.cut; c++) {
                    if (tid < sent_n[c]) found[at + tid] = sent[c * LP_TOP + tid];
                    at += sent_n[c];
                }
                mine = sent_sums[0];
                for (int c = 1; c < p.cut; c++) mine = join(mine, sent_sums[c]);
                if (r + rows_at_once < p.n_rows) cluster.barrier_arrive();  // (what was sent has been read)
                __syncthreads();
                rank_found(at);
                n_best = min(at, p.n_top);
            } else {
                if (r + rows_at_once < p.n_rows) cluster.barrier_arrive();
                continue;
            }
        }
        if (tid == 0) warp_sums[0] = mine;
        __syncthreads();
        mine = warp_sums[0];
        const bool bad = !(mine.x < INFINITY) || !scale_ok;  // NaN or infinite logits, a scale that is none
        const float nan = __int_as_float(0x7fffffff);
        const float log_s = mine.s > 0.0f ? logf(mine.s) : 0.0f;
        if (tid == 0 && p.entropy) p.entropy[r] = bad ? nan : mine.s > 0.0f ? log_s - mine.t / mine.s : 0.0f;
        for (int i = tid; i < p.n_ids; i += LP_THREADS) {
            const int token = p.ids[r * p.n_ids + i];
            float y = 0.0f;
            if (token >= p.n_vocab) record_error(p.err, SYN_DEVERR_BOUNDS);
            else if (token >= 0) {
                const float x = logit_at<F16>(row, token);
                const bool on = (!mask || ((mask[token >> 5] >> (token & 31)) & 1)) && x > -INFINITY;
                y = bad ? nan : on ? from(x, mine.x) - log_s : -INFINITY;
            }
            p.logprob[r * p.n_ids + i] = y;
        }
        for (int i = tid; i < p.n_top; i += LP_THREADS) {
            const bool there = i < n_best && !bad;
            p.top[r * p.n_top + i] = there ? (int32_t)~(uint32_t)best[i] : -1;
            p.top_logprob[r * p.n_top + i] = bad ? nan : there ? from(of_order((uint32_t)(best[i] >> 32)), mine.x) - log_s : -INFINITY;
        }
        __syncthreads();  // (the next row uses the same shared memory)
    }
}

cudaError_t launch_logprobs(const LogitsDesc& d, int64_t n_rows, int n_vocab, const void* x, const int32_t* ids, int n_ids,
                            float* logprob, float* entropy, int n_top, int32_t* top, float* top_logprob, bool whole,
                            int* err, int sms, cudaStream_t s) {
    LogprobParams p;
    p.x = x;
    p.stride = d.stride;
    p.scales = d.scales;
    p.mask = d.mask;
    p.mask_stride = d.mask_stride;
    p.ids = ids;
    p.logprob = logprob;
    p.entropy = entropy;
    p.top = top;
    p.top_logprob = top_logprob;
    p.err = err;
    p.n_rows = n_rows;
    p.n_vocab = n_vocab;
    p.n_ids = n_ids;
    p.n_top = n_top;
    p.scale = d.scale;
    p.cap = d.cap;
    // As many CTAs a row as the rows leave room for (two CTAs an SM), and each still has a thread's worth
    // for all of its threads; whole: what a row's sums are does not depend on how many rows there are.
    int cut = 1;
    const int64_t hold = (int64_t)LP_THREADS * LP_HOLD;
    while (cut < LP_CLUSTER && n_vocab > hold * cut && (whole || 2 * cut * n_rows <= 2 * (int64_t)sms)) cut *= 2;
    p.cut = cut;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(n_rows * cut, std::max(2 * sms / cut, 1) * cut));
    cfg.blockDim = dim3(LP_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cut;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cut > 1 ? 2 : 1;
    return d.f16 ? cudaLaunchKernelEx(&cfg, k_logprobs<true>, p) : cudaLaunchKernelEx(&cfg, k_logprobs<false>, p);
}

}  // namespace syn
