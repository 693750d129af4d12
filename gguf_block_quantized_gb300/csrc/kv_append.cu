// kv_append.cu — rows into and out of the paged key-value cache.
//
// k_kv_append: for each token, q and k rows rotated by the token's position, q rounded to
// fp16, k and v written to their slot of the cache.  For pair i of a row (values (2i, 2i+1) or
// (i, i + n_rot/2)) at position p of the pair's axis, with f_i turns per position:
//   (a, b) -> magnitude * (a cos t - b sin t, a sin t + b cos t),  t = 2 pi p f_i
// f_i is a 64-bit fraction of a turn, so p * f_i wraps at whole turns in integer arithmetic:
// the reduced angle is as exact at position 10^6 as at 1 (an fp32 product p * f loses
// p * 2^-24 radians).  32 bits of the fraction go to sincospif.
//
// Bound: HBM (4 B read and about 2 B written per value).  Persistent CTAs: one warp runs ahead,
// computing each token's n_rot/2 sines once for all heads and copying its rows (cp.async.bulk, in
// pieces of up to 16 KB) into a ring in shared memory; eight warps take 4 consecutive values a
// thread from there, rotate, and store them as 8 bytes (a warp's stores are contiguous).  So about
// 150 KB of loads are in flight on an SM whatever the threads wait for.  A Q8_0 block is 8
// neighbouring lanes, its amax three shuffles.  Measured on GB300: 8192 tokens of 32 / 8 heads of 128 into
// F16 47.9 us, 6.3 TB/s (93 % of a copy's rate; every thread loading for itself 66 us); one token
// 3.8 us; 4095 tokens into F16 26.5 us (84 %), into Q8_0 31.3 (68 %), there instructions bound it: 68 % of the
// issue slots, the integer and conversion pipe at 50 %.  Read back (k_kv_read) 10.7 us either way: its loads wait
// for the slot they go by, and start and end are most of it.
#include <algorithm>

#include "kernels.h"
#include "kv_cache.cuh"

namespace syn {

constexpr int APPEND_WARPS = 8;                          // that rotate and store
constexpr int APPEND_THREADS = 32 * (APPEND_WARPS + 1);  // and the one that loads
constexpr int APPEND_STAGE = 16384;                      // a piece: whole rows
constexpr int APPEND_STAGES = 4;
constexpr int APPEND_CTAS_PER_SM = 3;                    // what the rings leave room for

struct AppendParams {
    KvCache c;
    const float *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    __half* q_out;
    const int32_t* pos;  // n_axes x n_tok
    const int64_t* slots;
    const uint64_t* turns;
    const uint8_t* axis;
    int64_t n_tok, n_items;  // an item: the pieces of one of `parts` parts of a token
    int* err;
    int n_heads, n_rot, n_axes, halves;
    int piece_rows, q_pieces, kv_pieces, parts;
    float magnitude;
};

__device__ __forceinline__ uint2 pack_half4(const float4& x) {
    const __half2 a = __floats2half2_rn(x.x, x.y), b = __floats2half2_rn(x.z, x.w);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// 4 values of a Q8_0 block held by 8 neighbouring lanes: codes (packed) and the block's scale.
// A block with a non-finite value, or whose scale overflows fp16, gets a NaN scale: it reads
// back as NaN, never as something finite.
__device__ __forceinline__ uint32_t q8_codes(const float4& x, unsigned short& scale) {
    float a = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
    if (!(fabsf(x.x) + fabsf(x.y) + fabsf(x.z) + fabsf(x.w) < INFINITY)) a = INFINITY;  // (NaN as well)
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    const __half d = __float2half_rn(a / 127.0f);
    const float df = __half2float(d);
    const bool fine = df < INFINITY;
    scale = fine ? __half_as_ushort(d) : (unsigned short)0x7FFF;
    if (!fine || df == 0.0f) return 0u;
    // The code is x / d rounded half away from zero.  x times the reciprocal is off by less than 2^-21
    // of itself (2^-14 below 128): nearest-even rounding of it, by adding 1.5 * 2^23, gives that
    // code unless it lies that near a tie; then the four are divided.
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(df));
    constexpr float BIAS = 12582912.0f;
    float y[4] = {x.x * inv, x.y * inv, x.z * inv, x.w * inv};
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++) far = fmaxf(far, fabsf(y[i] - ((y[i] + BIAS) - BIAS)));
    if (far > 0.5f - 6.2e-5f) {
        const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; i++) y[i] = copysignf(floorf(fabsf(v[i]) / df + 0.5f), v[i]);
    }
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; i++) c[i] = __float_as_uint(fminf(fmaxf(y[i], -127.0f), 127.0f) + BIAS);  // (the stored scale can lie below amax/127)
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}

struct AppendSmem {
    uint8_t ring[APPEND_STAGES][APPEND_STAGE];
    float2 cs[2][128];  // (cos, sin) of each pair, times the magnitude, of two items; n_rot <= 256
    uint64_t full[APPEND_STAGES], empty[APPEND_STAGES], cs_full[2], cs_empty[2];
    int abort;
};

// The pieces of a token, in order: q rows, k rows, v rows, piece_rows at a time.
struct Piece {
    int kind, row, rows;  // kind 0 q, 1 k, 2 v
};
__device__ __forceinline__ Piece piece_of(const AppendParams& p, int i) {
    Piece x;
    x.kind = i < p.q_pieces ? 0 : i < p.q_pieces + p.kv_pieces ? 1 : 2;
    x.row = (i - (x.kind == 0 ? 0 : x.kind == 1 ? p.q_pieces : p.q_pieces + p.kv_pieces)) * p.piece_rows;
    x.rows = min(p.piece_rows, (x.kind == 0 ? p.n_heads : p.c.n_kv) - x.row);
    return x;
}

// DIM: head_dim, or 0 for a width without a kernel of its own.  With a width of 64, 128 or 256 a
// lane's place in a row is the same for every row, so its sines stay in registers.
template <bool Q8, int DIM>
__global__ void __launch_bounds__(APPEND_THREADS, APPEND_CTAS_PER_SM) k_kv_append(const AppendParams p) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    AppendSmem& sm = *reinterpret_cast<AppendSmem*>(smem_raw);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int dim = DIM ? DIM : p.c.dim, per_row = dim >> 2;  // 4-value units per row
    const int half_rot = p.n_rot >> 1, pieces = p.q_pieces + 2 * p.kv_pieces;
    volatile int* abort_flag = &sm.abort;
    if (tid == 0) {
        for (int i = 0; i < APPEND_STAGES; i++) {
            mbar_init(smem_u32(&sm.full[i]), 1);
            mbar_init(smem_u32(&sm.empty[i]), APPEND_WARPS);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_u32(&sm.cs_full[i]), 1);
            mbar_init(smem_u32(&sm.cs_empty[i]), APPEND_WARPS);
        }
        sm.abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    griddep_release();
    griddep_wait();

    int n = 0, it = 0;  // pieces and items of this CTA so far
    if (warp == APPEND_WARPS) {
        // ---- loads and sines, ahead of the others ------------------------------------------
        bool ok = true;
        for (int64_t w = blockIdx.x; w < p.n_items && ok; w += gridDim.x, it++) {
            const int64_t t = w / p.parts;
            const int part = (int)(w - t * p.parts);
            const int i0 = pieces * part / p.parts, i1 = pieces * (part + 1) / p.parts;
            int i = i0;
            auto copy = [&]() {  // piece i, whose stage is free
                if (lane == 0) {
                    const Piece x = piece_of(p, i);
                    const float* src = x.kind == 0 ? p.q + t * p.q_stride : x.kind == 1 ? p.k + t * p.k_stride : p.v + t * p.v_stride;
                    const uint32_t bytes = (uint32_t)(x.rows * dim * 4), full = smem_u32(&sm.full[n % APPEND_STAGES]);
                    const bool in = SYN_IN_BOUNDS(bytes > 0 && bytes <= APPEND_STAGE && t < p.n_tok);
                    mbar_arrive_expect_tx(full, in ? bytes : 0u);
                    if (in) bulk_g2s(smem_u32(sm.ring[n % APPEND_STAGES]), src + (int64_t)x.row * dim, bytes, full);
                }
                __syncwarp();
                n++;
                i++;
            };
#ifndef SYN_TEST_STALL  // (timeout-test build: no piece is ever loaded, so the waits for one run out)
            // the ring is empty at the start: its loads need not wait for the sines
            while (n < APPEND_STAGES && i < i1) copy();
#endif
            const int b = it & 1;
            if (!mbar_wait(smem_u32(&sm.cs_empty[b]), ((it >> 1) & 1) ^ 1, p.err, abort_flag)) break;
            for (int j = lane; j < half_rot; j += 32) {
                const int ax = p.axis ? min((int)p.axis[j], p.n_axes - 1) : 0;
                const int64_t pos = p.pos[(int64_t)ax * p.n_tok + t];
                const uint64_t phase = (uint64_t)pos * p.turns[j];
                float s, c;
                sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f /* 2^-31: half turns */, &s, &c);
                sm.cs[b][j] = make_float2(c * p.magnitude, s * p.magnitude);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.cs_full[b]));
#ifndef SYN_TEST_STALL
            while (i < i1) {
                if (!mbar_wait(smem_u32(&sm.empty[n % APPEND_STAGES]), ((n / APPEND_STAGES) & 1) ^ 1, p.err, abort_flag)) {
                    ok = false;
                    break;
                }
                copy();
            }
#endif
        }
        // the pieces still in flight (issued, not consumed: only after an abort) land first
        for (int i = max(0, n - APPEND_STAGES); i < n; i++)
            mbar_drain(smem_u32(&sm.full[i % APPEND_STAGES]), (i / APPEND_STAGES) & 1, p.err);
        return;
    }
    // ---- rotate and store --------------------------------------------------------------------
    for (int64_t w = blockIdx.x; w < p.n_items; w += gridDim.x, it++) {
        const int64_t t = w / p.parts;
        const int part = (int)(w - t * p.parts);
        const int i0 = pieces * part / p.parts, i1 = pieces * (part + 1) / p.parts;
        const int64_t slot = p.slots[t], page = slot >> p.c.page_shift;
        const int cell = (int)(slot & (((int64_t)1 << p.c.page_shift) - 1));
        bool store = slot >= 0;
        if (store && page >= p.c.n_pages) {
            if (tid == 0) record_error(p.err, SYN_DEVERR_BOUNDS);
            store = false;
        }
        const int b = it & 1;
        if (!mbar_wait(smem_u32(&sm.cs_full[b]), (it >> 1) & 1, p.err, abort_flag)) return;
        const float2* cs = sm.cs[b];
        // a unit's rotation: values e .. e + 3 of a row, the other halves of their pairs at e + other
        struct Turn {
            float4 c0, c1;
            int other;
            bool on;
        };
        auto turn_of = [&](int e) {
            Turn k;
            k.on = e < p.n_rot;
            k.other = 0;
            k.c0 = k.c1 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (k.on) {
                if (p.halves) {  // cosines in c0; sines, signed, in c1
                    const bool lower = e < half_rot;
                    const float4* c = reinterpret_cast<const float4*>(cs + (lower ? e : e - half_rot));
                    const float4 x = c[0], y = c[1];
                    const float sg = lower ? -1.0f : 1.0f;
                    k.other = lower ? half_rot : -half_rot;
                    k.c0 = make_float4(x.x, x.z, y.x, y.z);
                    k.c1 = make_float4(sg * x.y, sg * x.w, sg * y.y, sg * y.w);
                } else {
                    k.c0 = *reinterpret_cast<const float4*>(cs + (e >> 1));  // (cos, sin) of two pairs
                }
            }
            return k;
        };
        auto turned = [&](const Turn& k, const float* src) {
            const float4 a = *reinterpret_cast<const float4*>(src);
            if (!k.on) return a;
            float4 r;
            if (p.halves) {
                const float4 y = *reinterpret_cast<const float4*>(src + k.other);
                r.x = fmaf(a.x, k.c0.x, y.x * k.c1.x);
                r.y = fmaf(a.y, k.c0.y, y.y * k.c1.y);
                r.z = fmaf(a.z, k.c0.z, y.z * k.c1.z);
                r.w = fmaf(a.w, k.c0.w, y.w * k.c1.w);
            } else {
                r.x = fmaf(a.x, k.c0.x, -a.y * k.c0.y);
                r.y = fmaf(a.x, k.c0.y, a.y * k.c0.x);
                r.z = fmaf(a.z, k.c0.z, -a.w * k.c0.w);
                r.w = fmaf(a.z, k.c0.w, a.w * k.c0.z);
            }
            return r;
        };
        auto put = [&](uint8_t* tile, const float4& r, int e, bool in) {  // 4 values of a cached row
            if (Q8) {
                unsigned short scale;
                const uint32_t codes = q8_codes(r, scale);
                if (in) {
                    *reinterpret_cast<uint32_t*>(tile + cell * dim + e) = codes;
                    if ((e & 31) == 0)
                        *reinterpret_cast<unsigned short*>(tile + ((int64_t)dim << p.c.page_shift) + 2 * (cell * (dim >> 5) + (e >> 5))) = scale;
                }
            } else if (in) {
                *reinterpret_cast<uint2*>(tile + 2 * (cell * dim + e)) = pack_half4(r);
            }
        };
        const int e_mine = DIM ? (32 * warp + lane) % (DIM ? DIM / 4 : 1) * 4 : 0;
        const Turn mine = turn_of(e_mine);
        for (int i = i0; i < i1; i++, n++) {
            const Piece x = piece_of(p, i);
            const int st = n % APPEND_STAGES;
            if (!mbar_wait(smem_u32(&sm.full[st]), (n / APPEND_STAGES) & 1, p.err, abort_flag)) return;
            const float* src = reinterpret_cast<const float*>(sm.ring[st]);
            uint8_t* pool = (x.kind == 2 ? p.c.v : p.c.k) + page * p.c.page_stride + (int64_t)x.row * p.c.tile;
            __half* qo = p.q_out + (t * p.n_heads + x.row) * dim;
            const int units = x.rows * per_row;
            // (units is a multiple of 8: the 8 lanes of a Q8_0 block stay together)
            if (DIM) {
                const int u = 32 * warp + lane;
                constexpr int ROWS = DIM ? 1024 / DIM : 1;  // rows that the eight warps take at a time
                const int row = u / (DIM ? DIM / 4 : 1);
                const bool there = SYN_IN_BOUNDS(x.row + x.rows <= (x.kind == 0 ? p.n_heads : p.c.n_kv) && (x.kind == 0 || !store || page < p.c.n_pages));
                if (x.kind == 0) {
#pragma unroll 4
                    for (int k = 0; k < x.rows; k += ROWS)
                        if (row + k < x.rows && there) *reinterpret_cast<uint2*>(qo + 4 * u + k * DIM) = pack_half4(turned(mine, src + 4 * u + k * DIM));
                } else {
                    uint8_t* tile = pool + row * p.c.tile;
#pragma unroll 2
                    for (int k = 0; k < x.rows; k += ROWS) {
                        const float* s4 = src + 4 * min(u + k * (DIM / 4), units - 1);
                        const float4 r = x.kind == 1 ? turned(mine, s4) : *reinterpret_cast<const float4*>(s4);
                        put(tile, r, e_mine, row + k < x.rows && store && there);
                        tile += ROWS * p.c.tile;
                    }
                }
            } else {
                for (int u0 = 32 * warp; u0 < units; u0 += 32 * APPEND_WARPS) {
                    const int u = min(u0 + lane, units - 1), row = u / per_row, e = (u - row * per_row) << 2;
                    const bool live = u0 + lane < units;
                    const float4 r = x.kind < 2 ? turned(turn_of(e), src + 4 * u) : *reinterpret_cast<const float4*>(src + 4 * u);
                    if (x.kind == 0) {
                        if (live) *reinterpret_cast<uint2*>(qo + 4 * u) = pack_half4(r);
                    } else {
                        put(pool + row * p.c.tile, r, e, live && store && SYN_IN_BOUNDS(x.row + row < p.c.n_kv && page < p.c.n_pages && e + 4 <= dim));
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.empty[st]));
        }
        if (lane == 0) mbar_arrive(smem_u32(&sm.cs_empty[b]));
    }
}

// k_kv_read: the cached rows at the given slots as fp16 values (Q8_0: code * scale, one rounding),
// n x n_kv x dim; rows of negative slots read as zeros.
struct ReadParams {
    KvCache c;
    const int64_t* slots;
    __half* k;
    __half* v;
    int64_t n;
    int* err;
};

__global__ void __launch_bounds__(256) k_kv_read(const ReadParams p) {
    const int dim = p.c.dim, per_row = dim >> 3, per_tok = p.c.n_kv * per_row;  // 8-value units
    griddep_release();
    griddep_wait();
    for (int64_t t = blockIdx.x; t < p.n; t += gridDim.x) {
        const int64_t slot = p.slots[t], page = slot >> p.c.page_shift;
        const int cell = (int)(slot & (((int64_t)1 << p.c.page_shift) - 1));
        const bool there = slot >= 0 && page < p.c.n_pages;
        if (slot >= 0 && !there && threadIdx.x == 0) record_error(p.err, SYN_DEVERR_BOUNDS);
        for (int u = threadIdx.x; u < 2 * per_tok; u += 256) {  // keys, then values
            const bool is_v = u >= per_tok;
            const int at = is_v ? u - per_tok : u, h = at / per_row, e = (at - h * per_row) << 3;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (there) {
                const uint8_t* tile = (is_v ? p.c.v : p.c.k) + page * p.c.page_stride + (int64_t)h * p.c.tile;
                if (p.c.q8) {
                    const uint2 q = *reinterpret_cast<const uint2*>(tile + (int64_t)cell * dim + e);
                    const float d = h2f_bits(*reinterpret_cast<const unsigned short*>(
                        tile + ((int64_t)dim << p.c.page_shift) + 2 * ((int64_t)cell * (dim >> 5) + (e >> 5))));
                    auto four = [&](uint32_t x) {
                        return pack_half4(make_float4(d * (float)(int8_t)x, d * (float)(int8_t)(x >> 8), d * (float)(int8_t)(x >> 16),
                                                      d * (float)(int8_t)(x >> 24)));
                    };
                    const uint2 a = four(q.x), b = four(q.y);
                    w = make_uint4(a.x, a.y, b.x, b.y);
                } else {
                    w = *reinterpret_cast<const uint4*>(tile + 2 * ((int64_t)cell * dim + e));
                }
            }
            *reinterpret_cast<uint4*>((is_v ? p.v : p.k) + (t * per_tok + at) * 8) = w;
        }
    }
}

cudaError_t launch_kv_append(const KvCache& c, const RopeDesc& r, int64_t n_tok, const float* q, int64_t q_stride,
                             int n_heads, void* q_out, const float* k, int64_t k_stride, const float* v,
                             int64_t v_stride, const int32_t* pos, const int64_t* slots, int* err, int sms,
                             cudaStream_t s) {
    AppendParams p;
    p.c = c;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out = static_cast<__half*>(q_out);
    p.pos = pos;
    p.slots = slots;
    p.turns = r.turns;
    p.axis = r.axis;
    p.n_tok = n_tok;
    p.err = err;
    p.n_heads = n_heads;
    p.n_rot = r.n_rot;
    p.n_axes = r.n_axes;
    p.halves = r.halves;
    p.magnitude = r.magnitude;
    p.piece_rows = APPEND_STAGE / (4 * c.dim);
    p.q_pieces = (n_heads + p.piece_rows - 1) / p.piece_rows;
    p.kv_pieces = (c.n_kv + p.piece_rows - 1) / p.piece_rows;
    // few tokens: each token's pieces are dealt to several CTAs
    const int64_t ctas = (int64_t)sms * APPEND_CTAS_PER_SM;
    p.parts = (int)std::max<int64_t>(1, std::min<int64_t>(p.q_pieces + 2 * p.kv_pieces, ctas / n_tok));
    p.n_items = n_tok * p.parts;
    const int grid = (int)std::min<int64_t>(p.n_items, ctas);
    auto run = [&](auto kern, ResidentCtas& resident) {
        int per_sm;
        const cudaError_t e = resident.get(reinterpret_cast<const void*>(kern), APPEND_THREADS, sizeof(AppendSmem), &per_sm);
        return e != cudaSuccess ? e : launch_overlapped(kern, grid, APPEND_THREADS, sizeof(AppendSmem), s, p);
    };
    static ResidentCtas resident[2][4];
    switch (c.dim) {
    case 64: return c.q8 ? run(k_kv_append<true, 64>, resident[1][0]) : run(k_kv_append<false, 64>, resident[0][0]);
    case 128: return c.q8 ? run(k_kv_append<true, 128>, resident[1][1]) : run(k_kv_append<false, 128>, resident[0][1]);
    case 256: return c.q8 ? run(k_kv_append<true, 256>, resident[1][2]) : run(k_kv_append<false, 256>, resident[0][2]);
    default: return c.q8 ? run(k_kv_append<true, 0>, resident[1][3]) : run(k_kv_append<false, 0>, resident[0][3]);
    }
}

cudaError_t launch_kv_read(const KvCache& c, int64_t n, const int64_t* slots, void* k, void* v, int* err, int sms,
                           cudaStream_t s) {
    ReadParams p;
    p.c = c;
    p.slots = slots;
    p.k = static_cast<__half*>(k);
    p.v = static_cast<__half*>(v);
    p.n = n;
    p.err = err;
    return launch_overlapped(k_kv_read, (int)std::min<int64_t>(n, (int64_t)sms * 8), 256, 0, s, p);
}

#ifdef SYN_DEBUG
SYN_BOUNDS_READER(debug_bounds_kv_append)
#endif

}  // namespace syn
