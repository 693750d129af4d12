// logprobs.cu — log probabilities of given tokens, the entropy and the most likely tokens of rows of
// logits, in one pass over the logits.
//
//   z = cap > 0 ? cap*tanh(x/cap) : x,  y = scale log2(e) (z - the largest z)
//   S = sum 2^y, T = sum y 2^y;  logp(v) = ln2 (y_v - log2 S),  entropy = ln2 (log2 S - T/S)
// Both sums follow a running maximum: when it grows by g (as y counts), S' = S 2^-g and T' = (T - g S) 2^-g.
//
// Bound: HBM (or L2, where the product that made the logits has just written them): every logit is read
// once; a thread holds four 16-byte pieces while the next four are on their way.  fp16 logits come close to
// the issue slots (5 instructions a logit).
//   - A row is cut between the CTAs of a cluster (1 to 8, as many as the rows leave room for), which
//     send what they found to the first through its shared memory.  No CTA waits for another row's.
//   - The n_top largest: a thread notes the largest of each eighth of its logits (a unit).  At the row's end the
//     threads' own maxima are counted against a threshold, which is halved in until between n_top and 2 n_top of
//     them reach it; every logit below it is beaten by n_top others, so only the units that reach it are read
//     again (from L2).  What they hold is ordered by counting, for each, the larger ones (ties: the lower token first).
//
// Measured on GB300 (cold L2): one fp32 row of 128256 logits, top 20, 8.8 us; 61 masked, capped rows of 50257 15.5 us; 600 rows of
// 128256, top 8, 52 us (5.9 TB/s); 4095 fp16 rows of 128256 202 to 205 us (5.1 TB/s).
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "kv_cache.cuh"

namespace cg = cooperative_groups;

namespace syn {

constexpr int LP_TOP = LOGPROBS_TOP;
constexpr int LP_CLUSTER = 8;
constexpr int LP_UNITS = 8;      // of a thread
constexpr int LP_PIECES = 4;     // 16-byte pieces a thread holds
constexpr float LP_LN2 = 0.693147180559945309f, LP_LOG2E = 1.44269504088896341f;

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
    float scale, cap, inv_cap;
};

// A number that grows with the value (no NaN), and back.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_order(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u); }
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
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

// A row's logits: 16-byte pieces from the boundary at or below its first, so that the first piece may begin before the
// row and the last end behind it (those are read logit by logit).
template <bool F16>
struct Row {
    static constexpr int E = F16 ? 8 : 4;  // logits of a piece
    const uint8_t* at;
    const uint32_t* mask;
    int n, head, pieces;

    __device__ __forceinline__ Row(const LogprobParams& p, int64_t r)
        : at(static_cast<const uint8_t*>(p.x) + r * p.stride * (F16 ? 2 : 4)), mask(p.mask ? p.mask + r * p.mask_stride : nullptr),
          n(p.n_vocab), head((int)(reinterpret_cast<uintptr_t>(at) & 15) / (F16 ? 2 : 4)), pieces((head + n + E - 1) / E) {}
    __device__ __forceinline__ float one(int64_t i) const {
        return F16 ? __half2float(reinterpret_cast<const __half*>(at)[i]) : reinterpret_cast<const float*>(at)[i];
    }
    __device__ __forceinline__ int token(int piece, int j) const { return piece * E - head + j; }
    // A piece's bits; in those of logits that are not the row's, -inf.
    __device__ __forceinline__ uint4 load(int piece, int end) const {
        const int e0 = token(piece, 0);
        if (piece < end && e0 >= 0 && e0 + E <= n && SYN_IN_BOUNDS(piece >= 0 && piece < pieces && (reinterpret_cast<uintptr_t>(at + (int64_t)e0 * (F16 ? 2 : 4)) & 15) == 0))
            return load_once(at + (int64_t)e0 * (F16 ? 2 : 4));
        uint32_t w[4] = {F16 ? 0xFC00FC00u : 0xFF800000u, F16 ? 0xFC00FC00u : 0xFF800000u, F16 ? 0xFC00FC00u : 0xFF800000u,
                         F16 ? 0xFC00FC00u : 0xFF800000u};
        if (piece < end) {
#pragma unroll
            for (int j = 0; j < E; j++)
                if (e0 + j >= 0 && e0 + j < n) {
                    if (F16) {
                        const uint32_t h = reinterpret_cast<const uint16_t*>(at)[e0 + j];
                        w[j / 2] = j & 1 ? (w[j / 2] & 0xFFFFu) | h << 16 : (w[j / 2] & 0xFFFF0000u) | h;
                    } else {
                        w[j % 4] = reinterpret_cast<const uint32_t*>(at)[e0 + j];
                    }
                }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // The piece with -inf where the mask does not allow the token.
    __device__ __forceinline__ uint4 allowed(const uint4& piece, int index) const {
        const int e0 = token(index, 0), w = max(e0, 0) >> 5;
        const bool any = e0 < n;
        const uint32_t lo = any && SYN_IN_BOUNDS(w <= (n - 1) >> 5) ? __ldg(mask + w) : 0u;
        const uint32_t hi = any && (e0 & 31) + E > 32 && e0 >= 0 && w < (n - 1) >> 5 ? __ldg(mask + w + 1) : 0u;
        const uint32_t bits = e0 < 0 ? lo << -e0 : __funnelshift_r(lo, hi, e0 & 31);
        uint32_t u[4] = {piece.x, piece.y, piece.z, piece.w};
#pragma unroll
        for (int j = 0; j < E; j++)
            if (!((bits >> j) & 1)) {
                if (F16) u[j / 2] = j & 1 ? (u[j / 2] & 0xFFFFu) | 0xFC000000u : (u[j / 2] & 0xFFFF0000u) | 0xFC00u;
                else u[j % 4] = 0xFF800000u;
            }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};

template <bool F16>
__device__ __forceinline__ void values_of(const uint4& piece, float (&v)[F16 ? 8 : 4]) {
    const uint32_t u[4] = {piece.x, piece.y, piece.z, piece.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
        if (F16) {
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
            v[F16 ? 2 * j : j] = y.x;
            v[F16 ? 2 * j + 1 : j] = y.y;
        } else {
            v[j] = __uint_as_float(u[j]);
        }
    }
}
// The largest value of a thread's pieces (NaN where there is one).
template <bool F16>
__device__ __forceinline__ float largest_of(const uint4 (&piece)[LP_PIECES]) {
    if (F16) {
        __half2 m = __float2half2_rn(-INFINITY);
#pragma unroll
        for (int i = 0; i < LP_PIECES; i++) {
            const uint32_t u[4] = {piece[i].x, piece[i].y, piece[i].z, piece[i].w};
#pragma unroll
            for (int j = 0; j < 4; j++) m = __hmax2_nan(m, *reinterpret_cast<const __half2*>(&u[j]));
        }
        return max_nan(__low2float(m), __high2float(m));
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < LP_PIECES; i++) {
        m = max_nan(m, __uint_as_float(piece[i].x), __uint_as_float(piece[i].y));
        m = max_nan(m, __uint_as_float(piece[i].z), __uint_as_float(piece[i].w));
    }
    return m;
}

template <bool F16, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) k_logprobs(const LogprobParams p) {
    constexpr int E = Row<F16>::E, WARPS = THREADS / 32, MOST = LP_TOP + THREADS * E;
    static_assert(MOST * 8 >= LP_UNITS * THREADS * 4, "the units' maxima lie where the found keys will");
    __shared__ uint64_t found[MOST], best[LP_TOP];
    float* unit_max = reinterpret_cast<float*>(found);
    __shared__ uint64_t sent[LP_CLUSTER * LP_TOP];  // (the first CTA's) the others' largest
    __shared__ int units[LP_UNITS * 2 * LP_TOP];
    __shared__ Sums sent_sums[LP_CLUSTER], warp_sums[WARPS];
    __shared__ int sent_n[LP_CLUSTER], n_found, n_units;
    __shared__ uint32_t warp_lo[WARPS], warp_hi[WARPS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int part = p.cut > 1 ? (int)cg::this_cluster().block_rank() : 0;
    griddep_release();
    if (p.cut > 1) cg::this_cluster().barrier_arrive();  // (waited for before a row's stores: all have begun, and read the row before)
    griddep_wait();

    const int64_t rows_at_once = gridDim.x / p.cut;
    for (int64_t r = blockIdx.x / p.cut; r < p.n_rows; r += rows_at_once) {
        const Row<F16> row(p, r);
        const int per = (row.pieces + p.cut - 1) / p.cut, begin = per * part, end = min(row.pieces, begin + per);
        // a turn: the CTA's next LP_PIECES * THREADS pieces; group: turns of a unit
        const int turns = max(0, (end - begin + LP_PIECES * THREADS - 1) / (LP_PIECES * THREADS)), group = (turns + LP_UNITS - 1) / LP_UNITS;
        auto piece_of = [&](int turn, int i) { return begin + (turn * LP_PIECES + i) * THREADS + tid; };
        uint4 next[LP_PIECES];
#pragma unroll
        for (int i = 0; i < LP_PIECES; i++) next[i] = row.load(piece_of(0, i), end);
        const float scale = p.scales ? p.scale * p.scales[r] : p.scale;
        const bool scale_ok = scale > 0.0f && scale < INFINITY;
        const float c = fminf(scale * LP_LOG2E, 0x1.fffffep127f);  // (finite: the largest logit's y is 0)
        // cap*tanh(x/cap): up to half the cap x times a polynomial in (x/cap)^2, fitted on [0, 1/2] to 1e-7, past it
        // cap - 2 cap/(1 + 2^(2 x log2(e)/cap)), which is off by 2e-7 cap at most (CUDA's tanhf: 15.9 us, not 15.5, for 61
        // masked rows of 50257)
        auto capped = [&](float x) {
            if (!(p.cap > 0.0f)) return x;
            const float y = x * p.inv_cap, q = y * y;
            const float small = x * fmaf(q, fmaf(q, fmaf(q, fmaf(q, 0.0171413198f, -0.0529892407f), 0.133248284f), -0.333330721f), 1.0f);
            const float large = fmaf(-2.0f * p.cap, rcp(1.0f + ex2(y * (2.0f * LP_LOG2E))), p.cap);
            return fabsf(y) <= 0.5f ? small : large;
        };
        // sums over a maximum of x0, as they are over one of x, which is not smaller (z: its capped value)
        auto move_to = [&](float x0, float z, float& s, float& t) {
            const float g = s > 0.0f ? fminf(c * (z - capped(x0)), 300.0f) : 0.0f, f = ex2(-g);  // (2^-300 is 0, which keeps infinities out)
            t = (t - g * s) * f;
            s *= f;
        };
        // a logit that is asked for, on its way while the row streams
        const int asked = part == 0 && tid < p.n_ids ? p.ids[r * p.n_ids + tid] : -1;
        const bool asked_on = asked >= 0 && asked < p.n_vocab && (!row.mask || ((row.mask[asked >> 5] >> (asked & 31)) & 1));
        const float asked_x = asked_on ? row.one(asked) : -INFINITY;

        Sums mine{-INFINITY, 0.0f, 0.0f};
        float z0 = 0.0f, unit = -INFINITY;  // z0: that of mine.x
        for (int turn = 0, left = group, u = 0; turn < turns; turn++) {
            uint4 now[LP_PIECES];
#pragma unroll
            for (int i = 0; i < LP_PIECES; i++) now[i] = next[i];
#pragma unroll
            for (int i = 0; i < LP_PIECES; i++) next[i] = row.load(piece_of(turn + 1, i), turn + 1 < turns ? end : 0);
            if (row.mask)
#pragma unroll
                for (int i = 0; i < LP_PIECES; i++) now[i] = row.allowed(now[i], piece_of(turn, i));
            const float x = largest_of<F16>(now);
            unit = max_nan(unit, x);
            if (--left == 0 || turn + 1 == turns) {
                if (p.n_top > 0 && SYN_IN_BOUNDS(u < LP_UNITS)) unit_max[u++ * THREADS + tid] = unit;
                left = group;
                unit = -INFINITY;
            }
            if (x == -INFINITY) continue;
            if (!(x <= mine.x)) {
                mine.x = max_nan(mine.x, x);
                const float z = capped(mine.x), g = mine.s > 0.0f ? fminf(c * (z - z0), 300.0f) : 0.0f, f = ex2(-g);
                mine.t = (mine.t - g * mine.s) * f;
                mine.s *= f;
                z0 = z;
            }
            uint64_t s2 = 0, t2 = 0;
            const uint64_t c2 = pack2(c, c), z2 = pack2(-z0, -z0);
#pragma unroll
            for (int i = 0; i < LP_PIECES; i++) {
                float v[E];
                values_of<F16>(now[i], v);
                if (p.cap > 0.0f) {
#pragma unroll
                    for (int j = 0; j < E; j++) v[j] = v[j] == -INFINITY ? -INFINITY : capped(v[j]);
                }
#pragma unroll
                for (int j = 0; j < E; j += 2) {
                    float2 y = unpack2(mul2(add2(pack2(v[j], v[j + 1]), z2), c2));
                    y.x = fmaxf(y.x, -300.0f);
                    y.y = fmaxf(y.y, -300.0f);
                    const uint64_t e2 = pack2(ex2(y.x), ex2(y.y));
                    s2 = add2(s2, e2);
                    t2 = fma2(e2, pack2(y.x, y.y), t2);
                }
            }
            const float2 s = unpack2(s2), t = unpack2(t2);
            mine.s += s.x + s.y;
            mine.t += t.x + t.y;
        }

        // ---- the sums of the CTA ---------------------------------------------------------------
        const uint32_t none = order_of(-INFINITY), nan_order = 0xffffffffu;
        const uint32_t u = mine.x == mine.x ? order_of(mine.x + 0.0f) : nan_order;  // (-0 is 0)
        {
            const uint32_t wl = __reduce_min_sync(0xffffffffu, u > none ? u : nan_order), wh = __reduce_max_sync(0xffffffffu, u);
            if (lane == 0) {
                warp_lo[warp] = wl;
                warp_hi[warp] = wh;
            }
            if (tid == 0) n_found = n_units = 0;
        }
        int n = __syncthreads_count(u > none);
        uint32_t lo = __reduce_min_sync(0xffffffffu, warp_lo[lane % WARPS]), hi = __reduce_max_sync(0xffffffffu, warp_hi[lane % WARPS]);
        Sums sums{hi == nan_order ? __int_as_float(0x7fffffff) : of_order(hi), mine.s, mine.t};
        move_to(mine.x, capped(sums.x), sums.s, sums.t);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            sums.s += __shfl_xor_sync(0xffffffffu, sums.s, o);
            sums.t += __shfl_xor_sync(0xffffffffu, sums.t, o);
        }
        if (lane == 0) warp_sums[warp] = sums;
        // ---- the CTA's largest -----------------------------------------------------------------
        // the n_top largest of the n keys in `found`, in order, into `best`
        auto rank_found = [&](int n) {
            for (int i = tid; i < n; i += THREADS) {
                const uint64_t key = found[i];
                int rank = 0;
#pragma unroll 8
                for (int j = 0; j < n; j++) rank += found[j] > key;
                if (rank < p.n_top && SYN_IN_BOUNDS(rank < LP_TOP && n <= MOST)) best[rank] = key;
            }
        };
        int n_best = 0;
        if (p.n_top > 0 && hi != nan_order) {
            const int k = p.n_top;
            while (lo < hi && n > 2 * k) {  // (n: how many reach lo; fewer than k reach hi + 1)
                const uint32_t mid = lo + (hi - lo) / 2 + 1;
                const int reach = __syncthreads_count(u >= mid);
                if (reach >= k) {
                    lo = mid;
                    n = reach;
                } else {
                    hi = mid - 1;
                }
            }
            if (n < k) lo = none + 1;  // (fewer threads have a logit than are wanted: all their logits count)
            const float least = of_order(lo);
            int tie = 0x7fffffff, first = -1;  // of the logits at the threshold those up to token `tie` count; this thread's first
            if (n > 2 * k) {  // many maxima are the same: the same search over the tokens that have it
                first = u > lo ? -1 : 0x7fffffff;
                for (int turn = 0; turn < turns && u == lo && first > p.n_vocab; turn++)
#pragma unroll
                    for (int i = LP_PIECES - 1; i >= 0; i--) {
                        float v[E];
                        const uint4 piece = row.load(piece_of(turn, i), end);
                        values_of<F16>(row.mask ? row.allowed(piece, piece_of(turn, i)) : piece, v);
#pragma unroll
                        for (int j = E - 1; j >= 0; j--)
                            if (v[j] == least) first = row.token(piece_of(turn, i), j);
                    }
                int a = -1, b = p.n_vocab - 1;  // (fewer than k are at most a; more than 2k at most b)
                while (n > 2 * k && a + 1 < b) {
                    const int mid = a + (b - a) / 2;
                    const int reach = __syncthreads_count(first <= mid);
                    if (reach >= k) {
                        b = mid;
                        n = reach;
                    } else {
                        a = mid;
                    }
                }
                tie = b;
            }
            if (n > 0 && u >= lo && first <= tie)  // (at most 2k threads)
                for (int i = 0; i < LP_UNITS && i * group < turns; i++)
                    if (unit_max[i * THREADS + tid] >= least) {
                        const int slot = atomicAdd(&n_units, 1);
                        if (SYN_IN_BOUNDS(slot < LP_UNITS * 2 * LP_TOP)) units[slot] = i * THREADS + tid;
                    }
            __syncthreads();
            const int per_unit = group * LP_PIECES, loads = n_units * per_unit;
            uint64_t above = 0;  // what is not above this key is out
            for (int l0 = 0; l0 < loads; l0 += THREADS) {
                if (l0 > 0) {
                    __syncthreads();
                    const int m = n_found;
                    __syncthreads();  // (every thread goes by the same count: none has added to it since)
                    if (m + THREADS * E > MOST) {  // (rows whose large logits crowd in few threads)
                        rank_found(m);
                        __syncthreads();
                        if (tid < min(m, k)) found[tid] = best[tid];
                        if (m >= k) above = best[k - 1];
                        if (tid == 0) n_found = min(m, k);
                        __syncthreads();
                    }
                }
                const int l = l0 + tid;
                if (l < loads) {
                    const int which = units[l / per_unit], x = l % per_unit, of = which % THREADS;
                    const int turn = which / THREADS * group + x / LP_PIECES;
                    const int piece = begin + (turn * LP_PIECES + x % LP_PIECES) * THREADS + of;
                    float v[E];
                    const uint4 raw = row.load(piece, turn < turns ? end : 0);
                    values_of<F16>(row.mask ? row.allowed(raw, piece) : raw, v);
#pragma unroll
                    for (int j = 0; j < E; j++) {
                        const int token = row.token(piece, j);
                        const uint64_t key = ((uint64_t)order_of(v[j] + 0.0f) << 32) | (uint32_t)~token;
                        if ((v[j] > least || (v[j] == least && token <= tie)) && key > above) {
                            const int slot = atomicAdd(&n_found, 1);
                            if (SYN_IN_BOUNDS(slot < MOST)) found[slot] = key;
                        }
                    }
                }
            }
            __syncthreads();
            n_best = min(n_found, k);
            rank_found(n_found);
        }
        __syncthreads();
        // (each warp for itself, in the same order)
        sums = warp_sums[lane % WARPS];
#pragma unroll
        for (int o = WARPS / 2; o > 0; o >>= 1) {
            sums.s += __shfl_xor_sync(0xffffffffu, sums.s, o);
            sums.t += __shfl_xor_sync(0xffffffffu, sums.t, o);
        }
        // ---- the row's -------------------------------------------------------------------------
        if (p.cut > 1) {
            auto cluster = cg::this_cluster();
            cluster.barrier_wait();
            if (tid == 0) {
                cluster.map_shared_rank(sent_sums, 0)[part] = sums;
                cluster.map_shared_rank(sent_n, 0)[part] = n_best;
            }
            if (tid < n_best && SYN_IN_BOUNDS(part < LP_CLUSTER && n_best <= LP_TOP)) cluster.map_shared_rank(sent, 0)[part * LP_TOP + tid] = best[tid];
            cluster.sync();
            if (part > 0) {
                if (r + rows_at_once < p.n_rows) cluster.barrier_arrive();
                continue;
            }
            sums = sent_sums[lane % p.cut];
            float x = sums.x;
            for (int o = p.cut / 2; o > 0; o >>= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
            move_to(sums.x, capped(x), sums.s, sums.t);
            sums.x = x;
            for (int o = p.cut / 2; o > 0; o >>= 1) {
                sums.s += __shfl_xor_sync(0xffffffffu, sums.s, o);
                sums.t += __shfl_xor_sync(0xffffffffu, sums.t, o);
            }
            if (p.n_top > 0) {
                int at = 0;
                for (int i = 0; i < p.cut; i++) {
                    const int m = sent_n[i];
                    if (tid < m && SYN_IN_BOUNDS(m <= LP_TOP && at + m <= MOST)) found[at + tid] = sent[i * LP_TOP + tid];
                    at += m;
                }
                __syncthreads();
                rank_found(at);
                n_best = min(at, p.n_top);
                __syncthreads();
            }
            if (r + rows_at_once < p.n_rows) cluster.barrier_arrive();  // (what was sent has been read)
        }
        const bool bad = !(sums.x < INFINITY) || !scale_ok;  // NaN or infinite logits, a scale that is none
        const float nan = __int_as_float(0x7fffffff), row_z = capped(sums.x), log_s = sums.s > 0.0f ? log2f(sums.s) : 0.0f;
        // (by the scale itself: 2^y of a logit of the type's lowest value is 0, its log probability need not be -inf)
        auto logp = [&](float x) {
            const float z = capped(x), d = z - row_z;
            return fmaf(-LP_LN2, log_s, d > -INFINITY ? scale * d : scale * z - scale * row_z);
        };
        if (tid == 0 && p.entropy) p.entropy[r] = bad ? nan : sums.s > 0.0f ? LP_LN2 * (log_s - sums.t / sums.s) : 0.0f;
        auto tell = [&](int i, int token, float x) {
            if (token >= p.n_vocab) record_error(p.err, SYN_DEVERR_BOUNDS);
            p.logprob[r * p.n_ids + i] = token < 0 || token >= p.n_vocab ? 0.0f : bad ? nan : x == -INFINITY ? -INFINITY : logp(x);
        };
        if (tid < p.n_ids) tell(tid, asked, asked_x);
        for (int i = tid + THREADS; i < p.n_ids; i += THREADS) {
            const int token = p.ids[r * p.n_ids + i];
            const bool on = token >= 0 && token < p.n_vocab && (!row.mask || ((row.mask[token >> 5] >> (token & 31)) & 1));
            tell(i, token, on ? row.one(token) : -INFINITY);
        }
        for (int i = tid; i < p.n_top; i += THREADS) {
            const bool there = i < n_best && !bad;
            p.top[r * p.n_top + i] = there ? (int32_t)~(uint32_t)best[i] : -1;
            p.top_logprob[r * p.n_top + i] = bad ? nan : there ? logp(of_order((uint32_t)(best[i] >> 32))) : -INFINITY;
        }
        __syncthreads();  // (the next row uses the same shared memory)
    }
}

template <bool F16, int THREADS>
static cudaError_t run_logprobs(const LogprobParams& p, int sms, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    // (no more CTAs than run at once: a row's end costs a CTA what its start costs the next)
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(p.n_rows * p.cut, std::max(1024 / THREADS * sms / p.cut, 1) * p.cut));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cut;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cut > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_logprobs<F16, THREADS>, p);
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
    p.inv_cap = d.cap > 0.0f ? std::min(1.0f / d.cap, 1e38f) : 0.0f;  // (finite: a logit of 0 stays 0)
    // An SM holds 1024 threads: four CTAs of 256, so that others stream while one is at a row's end (600 rows of
    // 128256 fp32 logits 52.4 us, with two of 512 56.0, with eight of 128 54.7; 4095 fp16 rows 202, 240 and 204), eight of 128
    // for short rows, one of 512 where a few rows leave SMs idle (one row 8.8 us, with 256 9.4, with 128 13.2).  As many CTAs a
    // row as the rows leave room for, while each still has a turn for all of its threads.  (whole: what a row's sums are does not
    // depend on how many rows there are.)
    const int e = d.f16 ? 8 : 4, threads = n_vocab <= 128 * LP_PIECES * e * 4 ? 128 : !whole && LP_CLUSTER * n_rows <= sms ? 512 : 256;
    const int64_t turn = (int64_t)threads * LP_PIECES * e;
    int cut = 1;
    while (cut < LP_CLUSTER && n_vocab > turn * cut && (whole || 2 * cut * n_rows <= 1024 / threads * (int64_t)sms)) cut *= 2;
    p.cut = cut;
    if (threads == 256) return d.f16 ? run_logprobs<true, 256>(p, sms, s) : run_logprobs<false, 256>(p, sms, s);
    if (threads == 128) return d.f16 ? run_logprobs<true, 128>(p, sms, s) : run_logprobs<false, 128>(p, sms, s);
    return d.f16 ? run_logprobs<true, 512>(p, sms, s) : run_logprobs<false, 512>(p, sms, s);
}

#ifdef SYN_DEBUG
SYN_BOUNDS_READER(debug_bounds_logprobs)
#endif

}  // namespace syn
