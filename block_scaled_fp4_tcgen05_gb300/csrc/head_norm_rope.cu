// head_norm_rope.cu -- norms of the query and key heads with the position
// rotation in one pass over the QKV projection's output, written as BF16 or,
// for keys and values, quantised into the paged cache; the gradient; and the
// cache's plain write and read.
//
// Per head vector x of D elements, in fp32:
//   z = x * 1/sqrt(mean(x^2) + eps) * w                 (w == NULL: z = x)
//   y_a = z_a c_j - z_b s_j,  y_b = z_b c_j + z_a s_j    for the pairs (a, b) of
// the first R elements, (j, j + R/2) or, interleaved, (2j, 2j + 1), with cos c
// and sin s of the token's position from a table.  Gradient, with r the
// reciprocal root, h = x r and dz = dy turned back:
//   dw = sum dz h,   dx = r (dz w - h mean(dz w h)).
//
// HBM-bound.  8, 16 or 32 lanes hold a vector, 16 bytes each, so every access
// is a whole 16-byte piece of a row; a warp takes one token and four vectors per
// group of lanes, so that their loads are in flight together and the angles and
// weights are read once for all of them.  A pair's other element comes from a
// lane R/16 away, as the packed BF16 words that were loaded (half the exchanges
// of fp32 values); w is folded into the cosines and sines.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qfp4_common.cuh"
#include "qfp4_fp4_codes.cuh"
#include "qfp4_kv_cache.cuh"

namespace qfp4 {

__device__ uint32_t g_status_heads = 0;

int status_word_heads(uint32_t **word) { return status_word(g_status_heads, word); }

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kNoCache = -1;
constexpr float kFloor = 0x1p-100f;     // least magnitude that an E4M3 vector's scale is taken from

enum { kQuery = 0, kKey = 1, kValue = 2 };

struct CacheParams {
    uint8_t *cache;
    const int32_t *slots;       // [T]
    const float *gs[2];         // NVFP4's global scales of K and V
    int64_t slot_count;         // pages * page_size
    int32_t page_size, kv_heads;
};

struct HeadParams {
    const __nv_bfloat16 *x[3];  // queries, keys, values: head 0 of token 0
    int64_t ldx[3];             // elements from token to token
    __nv_bfloat16 *out[2];      // queries, keys
    int64_t ldo[2];
    const __nv_bfloat16 *w[2];  // [D] or NULL
    const float *table;         // [table_rows, R]: cos, then sin
    const int32_t *positions;   // [T] or NULL
    int64_t T, table_rows;
    int32_t heads[3], blocks[3];
    int32_t D, R, interleaved, norm;
    float eps;
    CacheParams c;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint4 pack8(const float (&y)[8])
{
    return make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int LANES>
__device__ __forceinline__ float group_max(float v)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// What the rotation does to a lane's eight elements: y = a x + b x', with x' the
// pairs' other elements.
struct Turn {
    int partner;        // lane that holds x'
    bool in;            // these elements turn (all eight or none: R is a multiple of 16)
    float c[8], s[8];   // s with the sign that x' gets

    template <int LANES>
    __device__ __forceinline__ void load(const HeadParams &p, int64_t position, int lane)
    {
        const int g = lane % LANES, i0 = 8 * g, half = p.R / 2;
        in = i0 < p.R;
        partner = lane;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            c[e] = 1.0f;
            s[e] = 0.0f;
        }
        if (in && !p.interleaved) partner = i0 < half ? lane + half / 8 : lane - half / 8;
        if (!in) return;
        const float *row = p.table + position * p.R;
        if (p.interleaved) {
            const float4 cv = __ldg(reinterpret_cast<const float4 *>(row + i0 / 2));
            const float4 sv = __ldg(reinterpret_cast<const float4 *>(row + half + i0 / 2));
            const float cc[4] = {cv.x, cv.y, cv.z, cv.w}, ss[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                c[2 * e] = c[2 * e + 1] = cc[e];
                s[2 * e] = -ss[e];
                s[2 * e + 1] = ss[e];
            }
        } else {
            const int j = i0 < half ? i0 : i0 - half;
            const float sign = i0 < half ? -1.0f : 1.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 cv = __ldg(reinterpret_cast<const float4 *>(row + j) + h);
                const float4 sv = __ldg(reinterpret_cast<const float4 *>(row + half + j) + h);
                c[4 * h] = cv.x, c[4 * h + 1] = cv.y, c[4 * h + 2] = cv.z, c[4 * h + 3] = cv.w;
                s[4 * h] = sign * sv.x, s[4 * h + 1] = sign * sv.y, s[4 * h + 2] = sign * sv.z, s[4 * h + 3] = sign * sv.w;
            }
        }
    }
    // The other elements of the pairs, from the words as they were loaded; zero
    // where nothing turns (there 0 times an infinity would be NaN).
    __device__ __forceinline__ uint4 others(const HeadParams &p, const uint4 &v) const
    {
        uint4 o;
        if (p.interleaved) {
            o = make_uint4(__byte_perm(v.x, 0, 0x1032), __byte_perm(v.y, 0, 0x1032), __byte_perm(v.z, 0, 0x1032),
                           __byte_perm(v.w, 0, 0x1032));
        } else {
            o.x = __shfl_sync(0xffffffffu, v.x, partner);
            o.y = __shfl_sync(0xffffffffu, v.y, partner);
            o.z = __shfl_sync(0xffffffffu, v.z, partner);
            o.w = __shfl_sync(0xffffffffu, v.w, partner);
        }
        return in ? o : make_uint4(0, 0, 0, 0);
    }
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Writes a lane's eight elements of a key (half 0) or value (half 1) to the
// cache: the quantisers' rules, with one scale per vector (E4M3) or per 16
// elements (NVFP4).  Every lane of the group takes part.
template <int TYPE, int LANES>
__device__ __forceinline__ void store_cached(const HeadParams &p, int half, int64_t slot, int head, int lane,
                                             const float (&y)[8], bool live, float gs, float inv_gs)
{
    const CacheParams &c = p.c;
    const CacheUnit u(TYPE, LANES * 8);
    const int g = lane % LANES;
    const int64_t page = slot / c.page_size;
    const int in_page = static_cast<int>(slot - page * c.page_size), j = in_page & 15;
    uint8_t *unit = c.cache + ((page * c.kv_heads + head) * (c.page_size / 16) + in_page / 16) * u.bytes;
    const int x = g * (u.row / LANES);
    uint8_t *at = unit + (half == 0 ? u.k_code(j, x) : u.v_code(j, x));
    if (TYPE == QFP4_CACHE_BF16) {
        if (live) *reinterpret_cast<uint4 *>(at) = pack8(y);
        return;
    }
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[e]));
    if (TYPE == QFP4_CACHE_E4M3) {
        const float a = fmaxf(group_max<LANES>(amax), kFloor);
        const float inv = __fdiv_rn(448.0f, a);
        uint2 q;
        q.x = e4m3x2(y[0] * inv, y[1] * inv) | (e4m3x2(y[2] * inv, y[3] * inv) << 16);
        q.y = e4m3x2(y[4] * inv, y[5] * inv) | (e4m3x2(y[6] * inv, y[7] * inv) << 16);
        if (live) {
            *reinterpret_cast<uint2 *>(at) = q;
            if (g == 0)
                *reinterpret_cast<float *>(unit + (half == 0 ? u.k_token_scale(j) : u.v_token_scale(j))) =
                    __fdiv_rn(a, 448.0f);
        }
    } else {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        const BlockScale b = block_scale<QFP4_NVFP4>(amax, gs, inv_gs);
        const uint32_t q = encode8_f32<QFP4_NVFP4>(y, b);
        if (live) {
            *reinterpret_cast<uint32_t *>(at) = q;
            if ((g & 1) == 0)
                unit[half == 0 ? u.k_block_scale(j, g / 2) : u.v_block_scale(j, g / 2)] = static_cast<uint8_t>(b.code);
        }
    }
}

// Vectors per group of lanes: four 16-byte loads in flight per lane.
constexpr int kVectors = 4;

template <int LANES, int CACHE>
__global__ void __launch_bounds__(kThreads) head_kernel(const HeadParams p)
{
    constexpr int GROUPS = 32 / LANES, BLOCK = GROUPS * kVectors;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, g = lane % LANES, sub = lane / LANES;
    const int per_token = p.blocks[0] + p.blocks[1] + p.blocks[2];
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t t = item / per_token;
    if (t >= p.T) return;
    int block = static_cast<int>(item - t * per_token), kind = kQuery;
    if (block >= p.blocks[0]) {
        block -= p.blocks[0];
        kind = kKey;
        if (block >= p.blocks[1]) {
            block -= p.blocks[1];
            kind = kValue;
        }
    }
    const bool lane_in = 8 * g < p.D;
    const __nv_bfloat16 *x = p.x[kind] + t * p.ldx[kind] + 8 * g;
    const int heads = p.heads[kind];
    uint4 v[kVectors];      // not through the read-only path: the output may take the input's place
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
        const int head = block * BLOCK + i * GROUPS + sub;
        v[i] = make_uint4(0, 0, 0, 0);
        if (lane_in && head < heads) v[i] = *reinterpret_cast<const uint4 *>(x + static_cast<int64_t>(head) * p.D);
    }
    // tokens without a position are padding: nothing of theirs is written
    const int64_t position = p.positions ? p.positions[t] : 0;
    const bool far = p.R > 0 && position >= p.table_rows;
    int64_t slot = 0;
    bool bad = far;
    if (CACHE != kNoCache) {
        slot = p.c.slots[t];
        bad |= slot >= p.c.slot_count;
    }
    if (bad && lane == 0) atomicOr(&g_status_heads, kStatusBadGroup);
    if (position < 0 || far) return;
    if (CACHE != kNoCache && kind != kQuery && (slot < 0 || slot >= p.c.slot_count)) return;

    Turn turn;
    float a[8], b[8];
    if (kind != kValue) {
        turn.load<LANES>(p, position, lane);
        uint4 w = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);      // ones
        if (p.w[kind] && lane_in) w = __ldg(reinterpret_cast<const uint4 *>(p.w[kind] + 8 * g));
        const uint4 wo = turn.others(p, w);
        unpack8(w, a);
        unpack8(wo, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            a[e] *= turn.c[e];
            b[e] *= turn.s[e];
        }
    }
    float gs = 1.0f, inv_gs = 1.0f;
    if (CACHE == QFP4_CACHE_NVFP4 && kind != kQuery) {
        gs = *p.c.gs[kind == kValue];
        inv_gs = __frcp_rn(gs);
    }
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
        const int head = block * BLOCK + i * GROUPS + sub;
        const bool live = lane_in && head < heads;
        float y[8];
        unpack8(v[i], y);
        if (kind != kValue) {
            float r = 1.0f;
            if (p.norm) {
                float ss = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
                r = rsqrtf(group_sum<LANES>(ss) / static_cast<float>(p.D) + p.eps);
            }
            float o[8];
            unpack8(turn.others(p, v[i]), o);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = fmaf(b[e], o[e], a[e] * y[e]) * r;
        }
        if (CACHE == kNoCache || kind == kQuery) {
            if (live)
                *reinterpret_cast<uint4 *>(p.out[kind] + t * p.ldo[kind] + static_cast<int64_t>(head) * p.D + 8 * g) =
                    pack8(y);
        } else {
            store_cached<CACHE, LANES>(p, kind == kValue, slot, min(head, heads - 1), lane, y, live, gs, inv_gs);
        }
    }
}

// ---------------------------------------------------------------- gradient

struct BackParams {
    HeadParams f;                       // x, w, table, positions, sizes as in the forward pass
    const __nv_bfloat16 *dy[2];
    int64_t ldy[2];
    __nv_bfloat16 *dx[2];
    int64_t lddx[2];
    float *partial;                     // [gridDim.x][2][D]
};

// Vectors per group of lanes in the gradient: two loads each.
constexpr int kBackVectors = 2;

template <int LANES>
__global__ void __launch_bounds__(kThreads) head_backward_kernel(const BackParams q)
{
    constexpr int GROUPS = 32 / LANES, BLOCK = GROUPS * kBackVectors;
    __shared__ float s_dw[kWarps][2][LANES * 8];
    const HeadParams &p = q.f;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, g = lane % LANES, sub = lane / LANES, warp = threadIdx.x >> 5;
    const int per_token = p.blocks[0] + p.blocks[1];
    const int64_t items = p.T * per_token;
    const bool lane_in = 8 * g < p.D;
    float dw[2][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.0f;
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp; item < items;
         item += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t t = item / per_token;
        int block = static_cast<int>(item - t * per_token);
        const int kind = block >= p.blocks[0] ? kKey : kQuery;
        if (kind == kKey) block -= p.blocks[0];
        const int heads = p.heads[kind];
        const __nv_bfloat16 *x = p.x[kind] + t * p.ldx[kind] + 8 * g;
        const __nv_bfloat16 *dy = q.dy[kind] + t * q.ldy[kind] + 8 * g;
        __nv_bfloat16 *dx = q.dx[kind] + t * q.lddx[kind] + 8 * g;
        const int64_t position = p.positions ? p.positions[t] : 0;
        const bool far = p.R > 0 && position >= p.table_rows;
        if (far && lane == 0) atomicOr(&g_status_heads, kStatusBadGroup);
        const bool alive = position >= 0 && !far;
        uint4 xv[kBackVectors], dv[kBackVectors];
#pragma unroll
        for (int i = 0; i < kBackVectors; ++i) {
            const int64_t head = block * BLOCK + i * GROUPS + sub;
            xv[i] = dv[i] = make_uint4(0, 0, 0, 0);
            if (alive && lane_in && head < heads) {
                // not through the read-only path: dx may take the place of either
                dv[i] = *reinterpret_cast<const uint4 *>(dy + head * p.D);
                if (p.norm) xv[i] = *reinterpret_cast<const uint4 *>(x + head * p.D);
            }
        }
        Turn turn;
        if (alive) turn.load<LANES>(p, position, lane);
        float w[8];
        uint4 wv = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
        if (p.w[kind] && lane_in) wv = __ldg(reinterpret_cast<const uint4 *>(p.w[kind] + 8 * g));
        unpack8(wv, w);
#pragma unroll
        for (int i = 0; i < kBackVectors; ++i) {
            const int64_t head = block * BLOCK + i * GROUPS + sub;
            float dz[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (alive) {        // uniform over the warp
                float o[8];
                unpack8(dv[i], dz);
                unpack8(turn.others(p, dv[i]), o);
#pragma unroll
                for (int e = 0; e < 8; ++e) dz[e] = fmaf(-turn.s[e], o[e], turn.c[e] * dz[e]);
                if (p.norm) {
                    float h[8], ss = 0.0f, dot = 0.0f;
                    unpack8(xv[i], h);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        ss = fmaf(h[e], h[e], ss);
                        dot = fmaf(dz[e] * w[e], h[e], dot);
                    }
                    const float n = static_cast<float>(p.D);
                    const float r = rsqrtf(group_sum<LANES>(ss) / n + p.eps);
                    const float mean = group_sum<LANES>(dot) * r / n;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        h[e] *= r;
                        const float d = dz[e] * h[e];
                        dw[0][e] += kind == kQuery ? d : 0.0f;
                        dw[1][e] += kind == kKey ? d : 0.0f;
                        dz[e] = r * fmaf(-h[e], mean, dz[e] * w[e]);
                    }
                }
            }
            if (lane_in && head < heads) *reinterpret_cast<uint4 *>(dx + head * p.D) = pack8(dz);
        }
    }
    if (!p.norm) return;
    // the groups of a warp hold the same elements: added up in a fixed order
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = dw[k][e];
#pragma unroll
            for (int o = 16; o >= LANES; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (sub == 0) s_dw[warp][k][8 * g + e] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.D; i += kThreads) {
        const int k = i >= p.D, d = i - k * p.D;
        float v = 0.0f;
#pragma unroll
        for (int wi = 0; wi < kWarps; ++wi) v += s_dw[wi][k][d];
        q.partial[static_cast<int64_t>(blockIdx.x) * 2 * p.D + i] = v;
    }
}

// Weight gradients from the CTAs' partial sums, in 64 bits: 32 columns per CTA.
__global__ void __launch_bounds__(1024) head_weight_kernel(const float *partial, int rows, int D, float *dq, float *dk)
{
    __shared__ double s_sum[32][33];
    pdl_wait();
    pdl_launch_dependents();
    const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + c;
    double v = 0.0;
    if (i < 2 * D)
        for (int k = r; k < rows; k += 32) v += static_cast<double>(partial[static_cast<int64_t>(k) * 2 * D + i]);
    s_sum[r][c] = v;
    __syncthreads();
    if (r != 0 || i >= 2 * D) return;
    v = 0.0;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += s_sum[k][c];
    float *out = i < D ? dq : dk;
    if (out) out[i < D ? i : i - D] = static_cast<float>(v);
}

// ------------------------------------------------------------- cache's read

struct ReadParams {
    CacheParams c;
    int64_t T;
    int32_t heads;
    __nv_bfloat16 *out[2];      // K, V
    int64_t ldo[2];
};

// A warp takes eight tokens of one head: where their slots follow one another
// (a prefix), every 32-byte sector that it reads is used whole.
constexpr int kReadTokens = 8;

template <int TYPE, int LANES>
__device__ __forceinline__ uint4 cached8(const uint8_t *unit, int half, int j, int g, float gs)
{
    const CacheUnit u(TYPE, LANES * 8);
    const int x = g * (u.row / LANES);
    const uint8_t *at = unit + (half == 0 ? u.k_code(j, x) : u.v_code(j, x));
    if (TYPE == QFP4_CACHE_BF16) return __ldg(reinterpret_cast<const uint4 *>(at));
    float y[8];
    if (TYPE == QFP4_CACHE_E4M3) {
        const uint2 q = __ldg(reinterpret_cast<const uint2 *>(at));
        const float s = __ldg(reinterpret_cast<const float *>(unit + (half == 0 ? u.k_token_scale(j) : u.v_token_scale(j))));
        const uint32_t w[2] = {q.x, q.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)))));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            y[2 * i] = f.x * s;
            y[2 * i + 1] = f.y * s;
        }
    } else {
        const uint32_t q = __ldg(reinterpret_cast<const uint32_t *>(at));
        const float s = ue4m3_decode(__ldg(unit + (half == 0 ? u.k_block_scale(j, g / 2) : u.v_block_scale(j, g / 2)))) * gs;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h;
            asm("{\n.reg .b8 x0, x1, x2, x3;\nmov.b32 {x0, x1, x2, x3}, %1;\ncvt.rn.f16x2.e2m1x2 %0, x0;\n}"
                : "=r"(h) : "r"(q >> (8 * i)));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            y[2 * i] = f.x * s;
            y[2 * i + 1] = f.y * s;
        }
    }
    return pack8(y);
}

template <int TYPE, int LANES>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const ReadParams p)
{
    constexpr int GROUPS = 32 / LANES, N = kReadTokens / GROUPS;
    constexpr int D = 8 * LANES, UNIT = cache_unit_bytes(TYPE, D);
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, g = lane % LANES, sub = lane / LANES;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t t0 = item / p.heads * kReadTokens;
    const int head = static_cast<int>(item % p.heads);
    if (t0 >= p.T) return;
    float gs[2] = {1.0f, 1.0f};
    if (TYPE == QFP4_CACHE_NVFP4) {
        gs[0] = *p.c.gs[0];
        gs[1] = *p.c.gs[1];
    }
    int64_t slot[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t t = t0 + i * GROUPS + sub;
        slot[i] = t < p.T ? p.c.slots[t] : -1;
        if (slot[i] >= p.c.slot_count) {
            atomicOr(&g_status_heads, kStatusBadGroup);
            slot[i] = -1;
        }
    }
    uint4 v[2][N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[0][i] = v[1][i] = make_uint4(0, 0, 0, 0);
        if (slot[i] < 0) continue;
        const int64_t page = slot[i] / p.c.page_size;
        const int in_page = static_cast<int>(slot[i] - page * p.c.page_size);
        const uint8_t *unit = p.c.cache + ((page * p.heads + head) * (p.c.page_size / 16) + in_page / 16) * UNIT;
        v[0][i] = cached8<TYPE, LANES>(unit, 0, in_page & 15, g, gs[0]);
        v[1][i] = cached8<TYPE, LANES>(unit, 1, in_page & 15, g, gs[1]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t t = t0 + i * GROUPS + sub;
        if (t >= p.T) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (p.out[h])
                *reinterpret_cast<uint4 *>(p.out[h] + t * p.ldo[h] + static_cast<int64_t>(head) * D + 8 * g) = v[h][i];
    }
}

// ------------------------------------------------------------------ launches

int lanes_of(int64_t D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }

template <int LANES>
int launch_heads(HeadParams &p, int cache, cudaStream_t s)
{
    constexpr int BLOCK = 32 / LANES * kVectors;
    int64_t per_token = 0;
    for (int k = 0; k < 3; ++k) per_token += p.blocks[k] = (p.heads[k] + BLOCK - 1) / BLOCK;
    const int64_t grid = (p.T * per_token + kWarps - 1) / kWarps;
    if (grid > INT32_MAX) return QFP4_ERR_UNSUPPORTED;
    auto kernel = cache == kNoCache ? head_kernel<LANES, kNoCache>
                : cache == QFP4_CACHE_BF16 ? head_kernel<LANES, QFP4_CACHE_BF16>
                : cache == QFP4_CACHE_E4M3 ? head_kernel<LANES, QFP4_CACHE_E4M3>
                                           : head_kernel<LANES, QFP4_CACHE_NVFP4>;
    return launch_status(launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, p));
}

int launch_heads_any(HeadParams &p, int cache, cudaStream_t s)
{
    switch (lanes_of(p.D)) {
    case 8: return launch_heads<8>(p, cache, s);
    case 16: return launch_heads<16>(p, cache, s);
    default: return launch_heads<32>(p, cache, s);
    }
}

// CTAs of the gradient's grid, whose partial sums of the weights' gradients
// the workspace holds: four per SM, no more than there is work for.
int64_t back_grid(int64_t T, int64_t q_heads, int64_t kv_heads, int64_t D)
{
    const int block = 32 / lanes_of(D) * kBackVectors;
    const int64_t items = T * ((q_heads + block - 1) / block + (kv_heads + block - 1) / block);
    const int64_t want = (items + kWarps - 1) / kWarps, most = 4 * 152;
    return want < most ? want : most;
}

constexpr int64_t kMaxTokens = int64_t{1} << 30, kMaxHeads = 4096;

bool head_sizes_ok(int64_t T, int64_t q_heads, int64_t kv_heads, int64_t D, int64_t R)
{
    return T <= kMaxTokens && q_heads <= kMaxHeads && kv_heads <= kMaxHeads && D % 16 == 0 && D >= 16 && D <= 256 &&
           R % 16 == 0 && R <= D;
}

int check_cache(int type, int64_t kv_heads, int64_t D, int64_t pages, int64_t page_size)
{
    if (!cache_type_ok(type) || kv_heads < 1 || D < 1 || pages < 0 || page_size < 1) return QFP4_ERR_INVALID_ARG;
    if ((D != 64 && D != 128 && D != 256) || page_size % 16 != 0 || page_size > 65536 || kv_heads > kMaxHeads ||
        pages > INT32_MAX || pages * page_size > INT32_MAX)
        return QFP4_ERR_UNSUPPORTED;
    return QFP4_OK;
}

// What the forward calls and the gradient share: sizes, table and weights.
int fill_common(HeadParams &p, const void *QKV, int64_t ld, int64_t T, int64_t q_heads, int64_t kv_heads, int64_t D,
                const void *q_weight, const void *k_weight, float eps, const float *table, int64_t table_rows,
                int64_t R, int interleaved, const int32_t *positions, int64_t least_ld)
{
    if (T < 0 || q_heads < 1 || kv_heads < 1 || D < 1 || R < 0 || table_rows < 0 || (interleaved & ~1) ||
        !(eps >= 0.0f) || eps > 3.0e38f || ld < least_ld)
        return QFP4_ERR_INVALID_ARG;
    if ((q_weight == nullptr) != (k_weight == nullptr) || (R > 0 && (!table || !positions || table_rows < 1)))
        return QFP4_ERR_INVALID_ARG;
    if (!head_sizes_ok(T, q_heads, kv_heads, D, R) || ld % 8 != 0) return QFP4_ERR_UNSUPPORTED;
    if (T == 0) return QFP4_OK;
    if (!QKV) return QFP4_ERR_INVALID_ARG;
    if (!aligned16(QKV) || !aligned16(q_weight) || !aligned16(k_weight) || !aligned16(table) || !aligned4(positions))
        return QFP4_ERR_MISALIGNED;
    const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(QKV);
    for (int k = 0; k < 3; ++k) p.ldx[k] = ld;
    p.x[0] = x;
    p.x[1] = x + q_heads * D;
    p.x[2] = x + (q_heads + kv_heads) * D;
    p.w[0] = static_cast<const __nv_bfloat16 *>(q_weight);
    p.w[1] = static_cast<const __nv_bfloat16 *>(k_weight);
    p.table = table;
    p.positions = positions;
    p.T = T;
    p.table_rows = table_rows;
    p.heads[0] = static_cast<int32_t>(q_heads);
    p.heads[1] = static_cast<int32_t>(kv_heads);
    p.D = static_cast<int32_t>(D);
    p.R = static_cast<int32_t>(R);
    p.interleaved = interleaved;
    p.norm = q_weight != nullptr;
    p.eps = eps;
    return QFP4_OK;
}

int fill_cache(CacheParams &c, int type, void *cache, int64_t kv_heads, int64_t pages, int64_t page_size,
               const int32_t *slots, const float *gs_k, const float *gs_v)
{
    if (!slots || (!cache && pages > 0) || (type == QFP4_CACHE_NVFP4 && (!gs_k || !gs_v))) return QFP4_ERR_INVALID_ARG;
    if (!aligned16(cache) || !aligned4(slots) || !aligned4(gs_k) || !aligned4(gs_v)) return QFP4_ERR_MISALIGNED;
    c.cache = static_cast<uint8_t *>(cache);
    c.slots = slots;
    c.gs[0] = gs_k;
    c.gs[1] = gs_v;
    c.slot_count = pages * page_size;
    c.page_size = static_cast<int32_t>(page_size);
    c.kv_heads = static_cast<int32_t>(kv_heads);
    return QFP4_OK;
}

}  // namespace
}  // namespace qfp4

using namespace qfp4;

extern "C" size_t qfp4_kv_cache_page_bytes(int type, int64_t kv_heads, int64_t head_dim, int64_t page_size)
{
    if (check_cache(type, kv_heads, head_dim, 0, page_size) != QFP4_OK) return 0;
    return static_cast<size_t>(kv_heads) * (page_size / 16) * cache_unit_bytes(type, static_cast<int>(head_dim));
}

extern "C" int qfp4_qk_norm_rope(const void *QKV_bf16, int64_t ld, int64_t T, int64_t q_heads, int64_t kv_heads,
                                 int64_t head_dim, const void *q_weight, const void *k_weight, float eps,
                                 const float *cos_sin, int64_t table_rows, int64_t rotary_dim, int interleaved,
                                 const int32_t *positions, void *Q_out, int64_t ldq, void *K_out, int64_t ldk,
                                 void *stream)
{
    HeadParams p = {};
    const int rc = fill_common(p, QKV_bf16, ld, T, q_heads, kv_heads, head_dim, q_weight, k_weight, eps, cos_sin,
                               table_rows, rotary_dim, interleaved, positions, (q_heads + kv_heads) * head_dim);
    if (rc != QFP4_OK) return rc;
    if (ldq < q_heads * head_dim || ldk < kv_heads * head_dim) return QFP4_ERR_INVALID_ARG;
    if (ldq % 8 != 0 || ldk % 8 != 0) return QFP4_ERR_UNSUPPORTED;
    if (T == 0) return QFP4_OK;
    if (!Q_out || !K_out) return QFP4_ERR_INVALID_ARG;
    if (!aligned16(Q_out) || !aligned16(K_out)) return QFP4_ERR_MISALIGNED;
    p.out[0] = static_cast<__nv_bfloat16 *>(Q_out);
    p.out[1] = static_cast<__nv_bfloat16 *>(K_out);
    p.ldo[0] = ldq;
    p.ldo[1] = ldk;
    return launch_heads_any(p, kNoCache, static_cast<cudaStream_t>(stream));
}

extern "C" int qfp4_qk_norm_rope_cache(const void *QKV_bf16, int64_t ld, int64_t T, int64_t q_heads, int64_t kv_heads,
                                       int64_t head_dim, const void *q_weight, const void *k_weight, float eps,
                                       const float *cos_sin, int64_t table_rows, int64_t rotary_dim, int interleaved,
                                       const int32_t *positions, void *Q_out, int64_t ldq, int type, void *cache,
                                       int64_t pages, int64_t page_size, const int32_t *slots, const float *gs_k,
                                       const float *gs_v, void *stream)
{
    HeadParams p = {};
    int rc = fill_common(p, QKV_bf16, ld, T, q_heads, kv_heads, head_dim, q_weight, k_weight, eps, cos_sin, table_rows,
                         rotary_dim, interleaved, positions, (q_heads + 2 * kv_heads) * head_dim);
    if (rc == QFP4_OK) rc = check_cache(type, kv_heads, head_dim, pages, page_size);
    if (rc != QFP4_OK) return rc;
    if (ldq < q_heads * head_dim) return QFP4_ERR_INVALID_ARG;
    if (ldq % 8 != 0) return QFP4_ERR_UNSUPPORTED;
    if (T == 0) return QFP4_OK;
    if (!Q_out) return QFP4_ERR_INVALID_ARG;
    rc = fill_cache(p.c, type, cache, kv_heads, pages, page_size, slots, gs_k, gs_v);
    if (rc != QFP4_OK) return rc;
    if (!aligned16(Q_out)) return QFP4_ERR_MISALIGNED;
    p.heads[2] = p.heads[1];
    p.out[0] = static_cast<__nv_bfloat16 *>(Q_out);
    p.ldo[0] = ldq;
    return launch_heads_any(p, type, static_cast<cudaStream_t>(stream));
}

extern "C" int qfp4_kv_cache_write(int type, const void *K_bf16, int64_t ldk, const void *V_bf16, int64_t ldv,
                                   int64_t T, int64_t kv_heads, int64_t head_dim, const int32_t *slots,
                                   const float *gs_k, const float *gs_v, void *cache, int64_t pages,
                                   int64_t page_size, void *stream)
{
    int rc = check_cache(type, kv_heads, head_dim, pages, page_size);
    if (rc == QFP4_ERR_INVALID_ARG || T < 0 || ldk < kv_heads * head_dim || ldv < kv_heads * head_dim)
        return QFP4_ERR_INVALID_ARG;
    if (rc != QFP4_OK || T > kMaxTokens || ldk % 8 != 0 || ldv % 8 != 0) return QFP4_ERR_UNSUPPORTED;
    if (T == 0) return QFP4_OK;
    if (!K_bf16 || !V_bf16) return QFP4_ERR_INVALID_ARG;
    HeadParams p = {};
    rc = fill_cache(p.c, type, cache, kv_heads, pages, page_size, slots, gs_k, gs_v);
    if (rc != QFP4_OK) return rc;
    if (!aligned16(K_bf16) || !aligned16(V_bf16)) return QFP4_ERR_MISALIGNED;
    p.x[1] = static_cast<const __nv_bfloat16 *>(K_bf16);
    p.x[2] = static_cast<const __nv_bfloat16 *>(V_bf16);
    p.ldx[1] = ldk;
    p.ldx[2] = ldv;
    p.T = T;
    p.heads[1] = p.heads[2] = static_cast<int32_t>(kv_heads);
    p.D = static_cast<int32_t>(head_dim);
    return launch_heads_any(p, type, static_cast<cudaStream_t>(stream));
}

namespace {

template <int LANES>
int launch_read(const ReadParams &p, int type, cudaStream_t s)
{
    const int64_t items = (p.T + kReadTokens - 1) / kReadTokens * p.heads, grid = (items + kWarps - 1) / kWarps;
    if (grid > INT32_MAX) return QFP4_ERR_UNSUPPORTED;
    auto kernel = type == QFP4_CACHE_BF16 ? cache_read_kernel<QFP4_CACHE_BF16, LANES>
                : type == QFP4_CACHE_E4M3 ? cache_read_kernel<QFP4_CACHE_E4M3, LANES>
                                          : cache_read_kernel<QFP4_CACHE_NVFP4, LANES>;
    return launch_status(launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, p));
}

}  // namespace

extern "C" int qfp4_kv_cache_read(int type, const void *cache, int64_t pages, int64_t page_size, int64_t kv_heads,
                                  int64_t head_dim, const int32_t *slots, int64_t T, const float *gs_k,
                                  const float *gs_v, void *K_out, int64_t ldk, void *V_out, int64_t ldv, void *stream)
{
    int rc = check_cache(type, kv_heads, head_dim, pages, page_size);
    if (rc == QFP4_ERR_INVALID_ARG || T < 0 || (K_out && ldk < kv_heads * head_dim) ||
        (V_out && ldv < kv_heads * head_dim))
        return QFP4_ERR_INVALID_ARG;
    if (rc != QFP4_OK || T > kMaxTokens || (K_out && ldk % 8 != 0) || (V_out && ldv % 8 != 0))
        return QFP4_ERR_UNSUPPORTED;
    if (T == 0) return QFP4_OK;
    if (!K_out && !V_out) return QFP4_ERR_INVALID_ARG;
    ReadParams p = {};
    rc = fill_cache(p.c, type, const_cast<void *>(cache), kv_heads, pages, page_size, slots, gs_k, gs_v);
    if (rc != QFP4_OK) return rc;
    if (!aligned16(K_out) || !aligned16(V_out)) return QFP4_ERR_MISALIGNED;
    p.T = T;
    p.heads = static_cast<int32_t>(kv_heads);
    p.out[0] = static_cast<__nv_bfloat16 *>(K_out);
    p.out[1] = static_cast<__nv_bfloat16 *>(V_out);
    p.ldo[0] = ldk;
    p.ldo[1] = ldv;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (head_dim) {
    case 64: return launch_read<8>(p, type, s);
    case 128: return launch_read<16>(p, type, s);
    default: return launch_read<32>(p, type, s);
    }
}

extern "C" size_t qfp4_qk_norm_rope_backward_workspace_bytes(int64_t T, int64_t q_heads, int64_t kv_heads,
                                                             int64_t head_dim)
{
    if (T < 0 || q_heads < 1 || kv_heads < 1 || !head_sizes_ok(T, q_heads, kv_heads, head_dim, 0)) return 0;
    return static_cast<size_t>(back_grid(T, q_heads, kv_heads, head_dim)) * 2 * head_dim * sizeof(float);
}

extern "C" int qfp4_qk_norm_rope_backward(const void *QKV_bf16, int64_t ld, int64_t T, int64_t q_heads,
                                          int64_t kv_heads, int64_t head_dim, const void *q_weight,
                                          const void *k_weight, float eps, const float *cos_sin, int64_t table_rows,
                                          int64_t rotary_dim, int interleaved, const int32_t *positions,
                                          const void *dQ, int64_t lddq, const void *dK, int64_t lddk, void *dQKV,
                                          int64_t lddqkv, float *dq_weight, float *dk_weight, void *workspace,
                                          size_t ws_bytes, void *stream)
{
    BackParams b = {};
    const int64_t width = (q_heads + kv_heads) * head_dim;
    const int rc = fill_common(b.f, QKV_bf16, ld, T, q_heads, kv_heads, head_dim, q_weight, k_weight, eps, cos_sin,
                               table_rows, rotary_dim, interleaved, positions, width);
    if (rc != QFP4_OK) return rc;
    if (lddq < q_heads * head_dim || lddk < kv_heads * head_dim || lddqkv < width) return QFP4_ERR_INVALID_ARG;
    if (lddq % 8 != 0 || lddk % 8 != 0 || lddqkv % 8 != 0) return QFP4_ERR_UNSUPPORTED;
    const bool norm = q_weight != nullptr;
    if (norm && (!dq_weight || !dk_weight)) return QFP4_ERR_INVALID_ARG;
    if (!aligned4(dq_weight) || !aligned4(dk_weight)) return QFP4_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned columns = static_cast<unsigned>((2 * head_dim + 31) / 32);
    const int D = static_cast<int>(head_dim);
    if (T > 0) {
        if (!dQ || !dK || !dQKV) return QFP4_ERR_INVALID_ARG;
        if (!aligned16(dQ) || !aligned16(dK) || !aligned16(dQKV) || !aligned16(workspace)) return QFP4_ERR_MISALIGNED;
        if (norm && (!workspace ||
                     ws_bytes < qfp4_qk_norm_rope_backward_workspace_bytes(T, q_heads, kv_heads, head_dim)))
            return QFP4_ERR_WORKSPACE;
        b.dy[0] = static_cast<const __nv_bfloat16 *>(dQ);
        b.dy[1] = static_cast<const __nv_bfloat16 *>(dK);
        b.ldy[0] = lddq;
        b.ldy[1] = lddk;
        b.dx[0] = static_cast<__nv_bfloat16 *>(dQKV);
        b.dx[1] = b.dx[0] + q_heads * head_dim;
        b.lddx[0] = b.lddx[1] = lddqkv;
        b.partial = static_cast<float *>(workspace);
        const int lanes = lanes_of(head_dim), block = 32 / lanes * kBackVectors;
        for (int k = 0; k < 2; ++k) b.f.blocks[k] = (b.f.heads[k] + block - 1) / block;
        const dim3 grid(static_cast<unsigned>(back_grid(T, q_heads, kv_heads, head_dim)));
        auto kernel = lanes == 8 ? head_backward_kernel<8>
                    : lanes == 16 ? head_backward_kernel<16> : head_backward_kernel<32>;
        const int st = launch_status(launch_pdl(kernel, grid, dim3(kThreads), 0, s, b));
        if (st != QFP4_OK || !norm) return st;
        return launch_status(launch_pdl(head_weight_kernel, dim3(columns), dim3(1024), 0, s, b.partial,
                                        static_cast<int>(grid.x), D, dq_weight, dk_weight));
    }
    // no token: zero gradients
    if (!norm) return QFP4_OK;
    return launch_status(launch_pdl(head_weight_kernel, dim3(columns), dim3(1024), 0, s,
                                    static_cast<const float *>(nullptr), 0, D, dq_weight, dk_weight));
}
