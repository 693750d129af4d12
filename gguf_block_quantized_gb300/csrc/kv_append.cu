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
// Bound: HBM (4 B read and about 2 B written per value).  One CTA per token: the n_rot/2 sines
// are computed once for all heads (a thread per pair), while the rows' loads are in flight.  A
// thread takes 4 consecutive values (16-byte loads, 8-byte stores, both coalesced); where the
// other half of a pair lies n_rot/2 values away it is loaded again, from L1.  A Q8_0 block is 8
// neighbouring lanes, its amax three shuffles.
#include "kernels.h"
#include "kv_cache.cuh"

namespace syn {

constexpr int APPEND_THREADS = 256;
constexpr int APPEND_DEEP = 4;  // units whose loads a thread has in flight

struct AppendParams {
    KvCache c;
    const float *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    __half* q_out;
    const int32_t* pos;  // n_axes x n_tok
    const int64_t* slots;
    const uint64_t* turns;
    const uint8_t* axis;
    int64_t n_tok;
    int* err;
    int n_heads, n_rot, n_axes, halves;
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
    scale = df < INFINITY ? __half_as_ushort(d) : (unsigned short)0x7FFF;
    const float v[4] = {x.x, x.y, x.z, x.w};
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        // round half away from zero (roundf), as the format's encoder does; the stored scale
        // can lie below amax/127, so the code is clamped
        float r = df > 0.0f && df < INFINITY ? roundf(v[i] / df) : 0.0f;
        r = fminf(fmaxf(r, -127.0f), 127.0f);
        w |= (uint32_t)(uint8_t)(int8_t)(int)r << (8 * i);
    }
    return w;
}

__global__ void __launch_bounds__(APPEND_THREADS) k_kv_append(const AppendParams p) {
    __shared__ float2 cs[128];  // (cos, sin) of each pair, times the magnitude; n_rot <= 256
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x;
    const int dim = p.c.dim, per_row = dim >> 2;  // 4-value units per row
    const int rows = p.n_heads + 2 * p.c.n_kv, total = rows * per_row;
    const int half_rot = p.n_rot >> 1;
    const int64_t slot = p.slots[t];
    const int64_t page = slot >> p.c.page_shift;
    const int cell = (int)(slot & (((int64_t)1 << p.c.page_shift) - 1));
    bool store = slot >= 0;
    if (store && page >= p.c.n_pages) {
        if (tid == 0) record_error(p.err, SYN_DEVERR_BOUNDS);
        store = false;
    }
    const float* qrow = p.n_heads ? p.q + t * p.q_stride : nullptr;
    const float* krow = p.k + t * p.k_stride;
    const float* vrow = p.v + t * p.v_stride;

    // (lanes past the end repeat the last unit's loads and take part in the shuffles)
    for (int base = 0; base < total; base += APPEND_THREADS * APPEND_DEEP) {
        float4 x[APPEND_DEEP], y[APPEND_DEEP];
        int row[APPEND_DEEP], e[APPEND_DEEP];
#pragma unroll
        for (int i = 0; i < APPEND_DEEP; i++) {
            const int u = min(base + i * APPEND_THREADS + tid, total - 1);
            row[i] = u / per_row;
            e[i] = (u - row[i] * per_row) << 2;
            const bool is_q = row[i] < p.n_heads, is_v = row[i] >= p.n_heads + p.c.n_kv;
            const float* src = is_q ? qrow + (int64_t)row[i] * dim
                             : is_v ? vrow + (int64_t)(row[i] - p.n_heads - p.c.n_kv) * dim
                                    : krow + (int64_t)(row[i] - p.n_heads) * dim;
            if (base + i * APPEND_THREADS >= total) continue;  // (the same for the whole CTA)
            x[i] = *reinterpret_cast<const float4*>(src + e[i]);
            y[i] = x[i];
            if (p.halves && !is_v && e[i] < p.n_rot)
                y[i] = *reinterpret_cast<const float4*>(src + (e[i] < half_rot ? e[i] + half_rot : e[i] - half_rot));
        }
        if (base == 0) {
            for (int i = tid; i < half_rot; i += APPEND_THREADS) {
                const int ax = p.axis ? min((int)p.axis[i], p.n_axes - 1) : 0;
                const int64_t pos = p.pos[(int64_t)ax * p.n_tok + t];
                const uint64_t phase = (uint64_t)pos * p.turns[i];
                float s, c;
                sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f /* 2^-31: half turns */, &s, &c);
                cs[i] = make_float2(c * p.magnitude, s * p.magnitude);
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < APPEND_DEEP; i++) {
            if (base + i * APPEND_THREADS >= total) break;
            const bool live = base + i * APPEND_THREADS + tid < total;
            const bool is_q = row[i] < p.n_heads, is_v = row[i] >= p.n_heads + p.c.n_kv;
            float4 r = x[i];
            if (!is_v && e[i] < p.n_rot) {
                if (p.halves) {
                    const bool lower = e[i] < half_rot;
                    const float2* c = cs + (lower ? e[i] : e[i] - half_rot);
                    const float sg = lower ? -1.0f : 1.0f;
                    r.x = fmaf(x[i].x, c[0].x, sg * y[i].x * c[0].y);
                    r.y = fmaf(x[i].y, c[1].x, sg * y[i].y * c[1].y);
                    r.z = fmaf(x[i].z, c[2].x, sg * y[i].z * c[2].y);
                    r.w = fmaf(x[i].w, c[3].x, sg * y[i].w * c[3].y);
                } else {
                    const float2 c0 = cs[e[i] >> 1], c1 = cs[(e[i] >> 1) + 1];
                    r.x = fmaf(x[i].x, c0.x, -x[i].y * c0.y);
                    r.y = fmaf(x[i].x, c0.y, x[i].y * c0.x);
                    r.z = fmaf(x[i].z, c1.x, -x[i].w * c1.y);
                    r.w = fmaf(x[i].z, c1.y, x[i].w * c1.x);
                }
            }
            uint32_t codes = 0;
            unsigned short scale = 0;
            if (p.c.q8) codes = q8_codes(r, scale);
            if (!live) continue;
            if (is_q) {
                *reinterpret_cast<uint2*>(p.q_out + (t * p.n_heads + row[i]) * dim + e[i]) = pack_half4(r);
            } else if (store) {
                const int h = row[i] - p.n_heads - (is_v ? p.c.n_kv : 0);
                uint8_t* tile = (is_v ? p.c.v : p.c.k) + page * p.c.page_stride + (int64_t)h * p.c.tile;
                if (!SYN_IN_BOUNDS(h >= 0 && h < p.c.n_kv && page >= 0 && page < p.c.n_pages && e[i] + 4 <= dim)) continue;
                if (p.c.q8) {
                    *reinterpret_cast<uint32_t*>(tile + (int64_t)cell * dim + e[i]) = codes;
                    if ((e[i] & 31) == 0)
                        *reinterpret_cast<unsigned short*>(tile + ((int64_t)dim << p.c.page_shift) +
                                                           2 * ((int64_t)cell * (dim >> 5) + (e[i] >> 5))) = scale;
                } else {
                    *reinterpret_cast<uint2*>(tile + 2 * ((int64_t)cell * dim + e[i])) = pack_half4(r);
                }
            }
        }
    }
}

// k_kv_read: the cached rows at the given slots as fp16 values (Q8_0: code * scale, one rounding),
// n x n_kv x dim; rows of negative slots read as zeros.
struct ReadParams {
    KvCache c;
    const int64_t* slots;
    __half* k;
    __half* v;
    int64_t n_units;
    int* err;
};

__global__ void __launch_bounds__(256) k_kv_read(const ReadParams p) {
    const int dim = p.c.dim, per_tok = (p.c.n_kv * dim) >> 2;  // 4-value units of one tensor
    for (int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; u < p.n_units; u += (int64_t)gridDim.x * blockDim.x) {
        const int64_t tt = u / per_tok;  // token, keys and values in turn
        const int at = (int)(u - tt * per_tok) << 2;
        const int64_t t = tt >> 1;
        const bool is_v = tt & 1;
        const int h = at / dim, e = at - h * dim;
        const int64_t slot = p.slots[t], page = slot >> p.c.page_shift;
        const int cell = (int)(slot & (((int64_t)1 << p.c.page_shift) - 1));
        uint2 w = make_uint2(0, 0);
        if (slot >= 0 && page < p.c.n_pages) {
            const uint8_t* tile = (is_v ? p.c.v : p.c.k) + page * p.c.page_stride + (int64_t)h * p.c.tile;
            if (p.c.q8) {
                const uint32_t q = *reinterpret_cast<const uint32_t*>(tile + (int64_t)cell * dim + e);
                const float d = h2f_bits(*reinterpret_cast<const unsigned short*>(
                    tile + ((int64_t)dim << p.c.page_shift) + 2 * ((int64_t)cell * (dim >> 5) + (e >> 5))));
                w = pack_half4(make_float4(d * (float)(int8_t)q, d * (float)(int8_t)(q >> 8),
                                           d * (float)(int8_t)(q >> 16), d * (float)(int8_t)(q >> 24)));
            } else {
                w = *reinterpret_cast<const uint2*>(tile + 2 * ((int64_t)cell * dim + e));
            }
        } else if (slot >= 0) {
            record_error(p.err, SYN_DEVERR_BOUNDS);
        }
        *reinterpret_cast<uint2*>((is_v ? p.v : p.k) + t * ((int64_t)per_tok << 2) + at) = w;
    }
}

cudaError_t launch_kv_append(const KvCache& c, const RopeDesc& r, int64_t n_tok, const float* q, int64_t q_stride,
                             int n_heads, void* q_out, const float* k, int64_t k_stride, const float* v,
                             int64_t v_stride, const int32_t* pos, const int64_t* slots, int* err, cudaStream_t s) {
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
    k_kv_append<<<(unsigned)n_tok, APPEND_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvCache& c, int64_t n, const int64_t* slots, void* k, void* v, int* err, int sms,
                           cudaStream_t s) {
    ReadParams p;
    p.c = c;
    p.slots = slots;
    p.k = static_cast<__half*>(k);
    p.v = static_cast<__half*>(v);
    p.n_units = n * 2 * ((int64_t)c.n_kv * c.dim / 4);
    p.err = err;
    const int64_t blocks = (p.n_units + 255) / 256, most = (int64_t)sms * 8;
    k_kv_read<<<(unsigned)(blocks < most ? blocks : most), 256, 0, s>>>(p);
    return cudaGetLastError();
}

#ifdef SYN_DEBUG
SYN_BOUNDS_READER(debug_bounds_kv_append)
#endif

}  // namespace syn
