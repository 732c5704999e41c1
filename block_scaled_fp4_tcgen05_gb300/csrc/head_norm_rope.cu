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
// HBM-bound, with the instructions per element close behind, so they are few:
// 8, 16 or 32 lanes hold a vector, eight elements each, in two pieces of four
// that hold both elements of their pairs (4 g .. and R/2 + 4 g .., or eight
// neighbours): no lane needs another's elements but for the sums.  The arithmetic
// is on packed pairs of fp32.  Every warp of one wave walks an equal piece of the
// line of (token, heads), the next heads' loads ahead, with the angles and weights in
// registers.  16384 tokens x 40 heads x 128 take 58 us (5.9 TB/s, 0.87 of the copy
// bandwidth); with a warp for every eight heads that reads them once 74, with the
// pairs' elements exchanged between lanes 63, through a ring of bulk copies 70.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qfp4_common.cuh"
#include "qfp4_fp4_codes.cuh"
#include "qfp4_kv_cache.cuh"
#include "qfp4_lane_ops.cuh"
#include "sm103_ptx.cuh"

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
    uint64_t page_magic;        // ceil(2^37 / page_units): what a division by it is done with
    int32_t page_units, kv_heads;       // page_units: page_size / 16

    // Number of the unit of a slot for key head 0; head h's lies h page_units on.
    __device__ __forceinline__ int64_t unit_of(int slot) const
    {
        const uint32_t n = static_cast<uint32_t>(slot) >> 4, page = static_cast<uint32_t>(n * page_magic >> 37);
        return static_cast<int64_t>(page) * kv_heads * page_units + (n - page * page_units);
    }
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
    int32_t heads[3];
    int32_t blocks[3];          // of each kind in a token; a block is what a warp works on at a time
    uint32_t share, more;       // blocks of a warp; so many first warps have one more
    int32_t D, R, interleaved, norm;
    float eps, inv_D;
    CacheParams c;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

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

// A lane's eight elements of a vector: two pieces of four, as packed pairs that
// the rotation mixes, (a[i], b[i]) -> (a c - b s, b c + a s).
struct Eight {
    uint64_t a[2], b[2];
};

struct Raw {
    uint2 v[2];     // the pieces as they lie in memory
};

// Interleaved pairs are the low and high halves of a piece's words, the others
// the two pieces' elements in the same place.
template <bool INTER>
__device__ __forceinline__ Eight unpack(const Raw &r)
{
    const uint64_t lo0 = f2_pack(bf16_lo(r.v[0].x), bf16_lo(r.v[0].y)), hi0 = f2_pack(bf16_hi(r.v[0].x), bf16_hi(r.v[0].y));
    const uint64_t lo1 = f2_pack(bf16_lo(r.v[1].x), bf16_lo(r.v[1].y)), hi1 = f2_pack(bf16_hi(r.v[1].x), bf16_hi(r.v[1].y));
    return INTER ? Eight{{lo0, lo1}, {hi0, hi1}} : Eight{{lo0, hi0}, {lo1, hi1}};
}

// Back to the pieces' elements in memory's order.
template <bool INTER>
__device__ __forceinline__ void elements(const Eight &y, float (&e)[8])
{
    f2_unpack(y.a[0], e[0], e[2]);
    f2_unpack(INTER ? y.b[0] : y.a[1], e[1], e[3]);
    f2_unpack(INTER ? y.a[1] : y.b[0], e[4], e[6]);
    f2_unpack(y.b[1], e[5], e[7]);
}

template <bool INTER>
__device__ __forceinline__ Raw pack(const Eight &y)
{
    float e[8];
    elements<INTER>(y, e);
    Raw r;
    r.v[0] = make_uint2(pack2(e[0], e[1]), pack2(e[2], e[3]));
    r.v[1] = make_uint2(pack2(e[4], e[5]), pack2(e[6], e[7]));
    return r;
}

// Where a lane's pieces lie in a vector, and whether they turn.
struct Place {
    int at[2];
    bool turns;

    template <int LANES, bool INTER>
    __device__ __forceinline__ static Place of(const HeadParams &p, int g, bool value)
    {
        const bool turns = !value && 8 * g < p.R, apart = turns && !INTER;
        return {{apart ? 4 * g : 8 * g, apart ? p.R / 2 + 4 * g : 8 * g + 4}, turns};
    }
    __device__ __forceinline__ Raw load(const __nv_bfloat16 *x) const
    {
        // not through the read-only path: an output may take its input's place
        return {{*reinterpret_cast<const uint2 *>(x + at[0]), *reinterpret_cast<const uint2 *>(x + at[1])}};
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *y, const Raw &r) const
    {
        *reinterpret_cast<uint2 *>(y + at[0]) = r.v[0];
        *reinterpret_cast<uint2 *>(y + at[1]) = r.v[1];
    }
};

// Cosines and sines of a lane's pairs.
struct Turn {
    uint64_t c[2], s[2];

    template <bool INTER>
    __device__ __forceinline__ static Turn of(const HeadParams &p, const Place &pl, int64_t position, int g)
    {
        float4 cv = make_float4(1.0f, 1.0f, 1.0f, 1.0f), sv = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (pl.turns) {
            const float *row = p.table + position * p.R + 4 * g;
            cv = __ldg(reinterpret_cast<const float4 *>(row));
            sv = __ldg(reinterpret_cast<const float4 *>(row + p.R / 2));
        }
        return INTER ? Turn{{f2_pack(cv.x, cv.y), f2_pack(cv.z, cv.w)}, {f2_pack(sv.x, sv.y), f2_pack(sv.z, sv.w)}}
                     : Turn{{f2_pack(cv.x, cv.z), f2_pack(cv.y, cv.w)}, {f2_pack(sv.x, sv.z), f2_pack(sv.y, sv.w)}};
    }
};

__device__ __forceinline__ uint64_t f2_neg(uint64_t v) { return v ^ 0x8000000080000000ull; }

__device__ __forceinline__ float f2_sum(uint64_t v)
{
    float lo, hi;
    f2_unpack(v, lo, hi);
    return lo + hi;
}

__device__ __forceinline__ Raw ones()
{
    return {{make_uint2(0x3F803F80u, 0x3F803F80u), make_uint2(0x3F803F80u, 0x3F803F80u)}};
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Where a lane's eight elements of a token's keys (half 0) or values (half 1) lie
// in a unit, and their scale.
template <int TYPE, int LANES>
struct CachePlace {
    static constexpr int UNIT = cache_unit_bytes(TYPE, LANES * 8);
    int code, scale;

    __device__ __forceinline__ CachePlace(int half, int j, int g)
    {
        constexpr CacheUnit U(TYPE, LANES * 8);
        const int x = g * (U.row / LANES);
        code = half == 0 ? U.k_code(j, x) : U.v_code(j, x);
        scale = TYPE == QFP4_CACHE_E4M3 ? (half == 0 ? U.k_token_scale(j) : U.v_token_scale(j))
                                        : (half == 0 ? U.k_block_scale(j, g / 2) : U.v_block_scale(j, g / 2));
    }
};

// Where the eight neighbouring elements 8 g .. of a vector lie whose pieces are apart:
// its first four in lane `from`, the others in the next, in the pieces of the same place.
struct Gather {
    int from;
    bool moves, second;

    template <int LANES>
    __device__ __forceinline__ static Gather of(const HeadParams &p, const Place &pl, int lane)
    {
        const int g = lane % LANES, i = 8 * g;
        const bool second = i >= p.R / 2;
        return {pl.turns ? lane - g + (second ? i - p.R / 2 : i) / 4 : lane, pl.turns, second};
    }
    // N words of two pieces
    template <int N>
    __device__ __forceinline__ void words(uint32_t (&w)[N]) const
    {
        uint32_t o[N];
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
            const uint32_t a0 = __shfl_sync(0xffffffffu, w[k], from), b0 = __shfl_sync(0xffffffffu, w[N / 2 + k], from);
            const uint32_t a1 = __shfl_sync(0xffffffffu, w[k], from + 1), b1 = __shfl_sync(0xffffffffu, w[N / 2 + k], from + 1);
            o[k] = second ? b0 : a0;
            o[N / 2 + k] = second ? b1 : a1;
        }
#pragma unroll
        for (int k = 0; k < N; ++k) w[k] = moves ? o[k] : w[k];
    }
};

// Writes a lane's eight elements to the cache: the quantisers' rules, with one
// scale per vector (E4M3) or per 16 elements (NVFP4).  Every lane of the group takes
// part.  Elements that lie apart are brought together as narrow as the scale allows.
template <int TYPE, int LANES>
__device__ __forceinline__ void store_cached(uint8_t *unit, const CachePlace<TYPE, LANES> &place, int lane,
                                             float (&y)[8], bool live, float gs, float inv_gs, bool apart,
                                             const Gather &gather)
{
    const int g = lane % LANES;
    uint8_t *at = unit + place.code;
    if constexpr (TYPE == QFP4_CACHE_BF16) {
        uint32_t w[4] = {pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7])};
        if (apart) gather.words(w);
        if (live) *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
        return;
    }
    if constexpr (TYPE == QFP4_CACHE_NVFP4) {
        if (apart) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(y[e]);
            gather.words(w);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(w[e]);
        }
    }
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[e]));
    if constexpr (TYPE == QFP4_CACHE_E4M3) {
        const float a = fmaxf(group_max<LANES>(amax), kFloor);
        const float inv = __fdiv_rn(448.0f, a);
        uint32_t w[2] = {e4m3x2(y[0] * inv, y[1] * inv) | (e4m3x2(y[2] * inv, y[3] * inv) << 16),
                         e4m3x2(y[4] * inv, y[5] * inv) | (e4m3x2(y[6] * inv, y[7] * inv) << 16)};
        if (apart) gather.words(w);
        if (live) {
            *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
            if (g == 0) *reinterpret_cast<float *>(unit + place.scale) = __fdiv_rn(a, 448.0f);
        }
    } else if constexpr (TYPE == QFP4_CACHE_NVFP4) {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        const BlockScale b = block_scale<QFP4_NVFP4>(amax, gs, inv_gs);
        const uint32_t q = encode8_f32<QFP4_NVFP4>(y, b);
        if (live) {
            *reinterpret_cast<uint32_t *>(at) = q;
            if ((g & 1) == 0) unit[place.scale] = static_cast<uint8_t>(b.code);
        }
    }
}

// Vectors that a group of lanes works on at a time, with as many loads ahead.
constexpr int kVectors = 2;

// CTAs per SM that the kernels' registers are sized for (with an E4M3 cache, 16384 tokens
// x (32 + 8 + 8) heads x 128: three 79 us, two 91, four 84; floor 56).
constexpr int kHeadCtas = 4, kCacheCtas = 3, kBackCtas = 2;
constexpr int head_ctas(int cache) { return cache == kNoCache ? kHeadCtas : kCacheCtas; }

// Piece of the line of (token, block of heads of a kind) that a warp takes: as
// many blocks for each, whatever the tokens and heads.  In 32 bits, and divided on the
// host: three 64-bit divisions per warp cost 0.6 us of a short call.
struct Piece {
    uint32_t begin;
    int count;

    __device__ __forceinline__ explicit Piece(const HeadParams &p)
    {
        const uint32_t w = blockIdx.x * kWarps + (threadIdx.x >> 5);
        begin = w * p.share + min(w, p.more);
        count = static_cast<int>(p.share + (w < p.more));
    }
};

template <int LANES, int CACHE, bool INTER>
__global__ void __launch_bounds__(kThreads, head_ctas(CACHE)) head_kernel(const HeadParams p)
{
    constexpr int GROUPS = 32 / LANES, BLOCK = GROUPS * kVectors;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, g = lane % LANES, sub = lane / LANES;
    const uint32_t per_token = p.blocks[0] + p.blocks[1] + p.blocks[2];
    const Piece piece(p);
    if (piece.count == 0) return;
    const bool lane_in = 8 * g < p.D;
    const uint32_t t_first = piece.begin / per_token;
    int64_t t = t_first;
    int block = static_cast<int>(piece.begin - t_first * per_token);
    int position_next = p.positions ? p.positions[t] : 0;
    int slot_next = CACHE != kNoCache ? p.c.slots[t] : 0;
    float gs[2] = {1.0f, 1.0f}, inv_gs[2] = {1.0f, 1.0f};
    if (CACHE == QFP4_CACHE_NVFP4) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            gs[h] = *p.c.gs[h];
            inv_gs[h] = __frcp_rn(gs[h]);
        }
    }
#pragma unroll 1
    for (int left = piece.count, run = 0; left > 0; left -= run) {
        int c = block, kind = kQuery;
        if (c >= p.blocks[0]) {
            c -= p.blocks[0];
            kind = kKey;
            if (c >= p.blocks[1]) {
                c -= p.blocks[1];
                kind = kValue;
            }
        }
        run = min(left, p.blocks[kind] - c);        // blocks of this token and kind
        const int head_end = min(p.heads[kind], (c + run) * BLOCK), head0 = c * BLOCK + sub;
        const Place pl = Place::of<LANES, INTER>(p, g, kind == kValue);
        const __nv_bfloat16 *x = p.x[kind] + t * p.ldx[kind] + static_cast<int64_t>(head0) * p.D;
        Raw next[kVectors] = {};
#pragma unroll
        for (int i = 0; i < kVectors; ++i)
            if (lane_in && head0 + i * GROUPS < head_end) next[i] = pl.load(x + i * GROUPS * p.D);
        int position = position_next, slot = slot_next;
        const int64_t tok = t;
        block += run;
        if (block == static_cast<int>(per_token)) {
            block = 0;
            if (++t < p.T) {
                position_next = p.positions ? p.positions[t] : 0;
                slot_next = CACHE != kNoCache ? p.c.slots[t] : 0;
            }
        }
        // tokens without a position are padding: nothing of theirs is written
        bool bad = p.R > 0 && position >= p.table_rows;
        if (bad) position = -1;
        if (CACHE != kNoCache && slot >= p.c.slot_count) {
            bad = true;
            slot = -1;
        }
        if (bad && lane == 0) atomicOr(&g_status_heads, kStatusBadGroup);
        if (position < 0 || (CACHE != kNoCache && kind != kQuery && slot < 0)) continue;      // uniform over the warp

        constexpr int TYPE = CACHE == kNoCache ? 0 : CACHE;
        const CachePlace<TYPE, LANES> place(kind == kValue, slot & 15, g);
        const Gather gather = Gather::of<LANES>(p, pl, lane);
        uint8_t *units = nullptr;       // of head 0
        if (CACHE != kNoCache && kind != kQuery)
            units = p.c.cache + p.c.unit_of(slot) * CachePlace<TYPE, LANES>::UNIT;

        // y = r (a ac + b bs, b bc + a as), the weights in the cosines and sines
        uint64_t ac[2], as[2], bc[2], bs[2];
        if (kind != kValue) {
            const Turn turn = Turn::of<INTER>(p, pl, position, g);
            Raw wr = ones();
            if (p.w[kind] && lane_in) wr = pl.load(p.w[kind]);
            const Eight w = unpack<INTER>(wr);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ac[i] = f2_mul(w.a[i], turn.c[i]);
                as[i] = f2_mul(w.a[i], turn.s[i]);
                bc[i] = f2_mul(w.b[i], turn.c[i]);
                bs[i] = f2_neg(f2_mul(w.b[i], turn.s[i]));
            }
        }
#pragma unroll 1
        for (int head = head0; head - sub < head_end; head += BLOCK) {
            Raw now[kVectors];
            x += BLOCK * p.D;
#pragma unroll
            for (int i = 0; i < kVectors; ++i) {
                now[i] = next[i];
                if (lane_in && head + (kVectors + i) * GROUPS < head_end) next[i] = pl.load(x + i * GROUPS * p.D);
            }
#pragma unroll
            for (int i = 0; i < kVectors; ++i) {
                const int h = head + i * GROUPS;
                const bool live = lane_in && h < head_end;
                Eight v = unpack<INTER>(now[i]);
                if (kind != kValue) {
                    float r = 1.0f;
                    if (p.norm) {
                        const uint64_t ss = f2_fma(v.b[1], v.b[1], f2_fma(v.b[0], v.b[0], f2_fma(v.a[1], v.a[1], f2_mul(v.a[0], v.a[0]))));
                        r = rsqrtf(group_sum<LANES>(f2_sum(ss)) * p.inv_D + p.eps);
                    }
                    const uint64_t r2 = f2_pack(r, r);
                    Eight o = v;        // the pairs' other elements
                    if (p.R < p.D && !pl.turns) o = Eight{{0, 0}, {0, 0}};     // 0 times an infinity would be NaN
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint64_t ya = f2_fma(o.b[k], bs[k], f2_mul(v.a[k], ac[k]));
                        v.b[k] = f2_mul(f2_fma(o.a[k], as[k], f2_mul(v.b[k], bc[k])), r2);
                        v.a[k] = f2_mul(ya, r2);
                    }
                }
                if (CACHE == kNoCache || kind == kQuery) {
                    if (live) pl.store(p.out[kind] + tok * p.ldo[kind] + static_cast<int64_t>(h) * p.D, pack<INTER>(v));
                } else {
                    float e[8];
                    elements<INTER>(v, e);
                    const int half = kind == kValue;
                    uint8_t *unit = units + static_cast<int64_t>(min(h, head_end - 1)) * p.c.page_units * place.UNIT;
                    store_cached<TYPE, LANES>(unit, place, lane, e, live, gs[half], inv_gs[half], !INTER && kind == kKey, gather);
                }
            }
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
#ifdef QFP4_FAULT_INJECTION
    bool skip_copy;
#endif
};

// The gradient's vectors per group of lanes, and a warp's ring of stages in shared
// memory, filled by bulk copies: a block of x and one of dy each, 16 bytes per lane,
// vector and tensor.
constexpr int kBackVectors = 4, kStages = 2, kHalfStage = 512 * kBackVectors, kStage = 2 * kHalfStage;
constexpr int kRing = kWarps * kStages * kStage;

// As head_kernel, but the queries of all tokens come before the keys, so that
// nearly every warp sums the weights' gradient of one kind; and with the loads
// through a ring.  What bounds it is the chain of each vector's sums and roots: four
// vectors at a time with two CTAs per SM take 93 us for 16384 tokens x 40 heads x
// 128 (5.5 TB/s, 0.81 of the copy bandwidth); before a step that took 2 us off, two at
// a time 112, eight 114, 143 with three CTAs, whose registers do not suffice, and 116
// with loads into registers instead of the ring.
template <int LANES, bool INTER>
__global__ void __launch_bounds__(kThreads, kBackCtas) head_backward_kernel(const BackParams q)
{
    constexpr int GROUPS = 32 / LANES, BLOCK = GROUPS * kBackVectors;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_bar[kWarps * kStages];
    __shared__ float s_dw[kWarps][2][LANES * 8];
    const HeadParams &p = q.f;
    const int lane = threadIdx.x & 31, g = lane % LANES, sub = lane / LANES, warp = threadIdx.x >> 5;
    const uint32_t bars = smem_u32(s_bar + warp * kStages);
    uint8_t *ring = smem + warp * kStages * kStage;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) mbar_init(bars + 8 * i, 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t items_q = static_cast<uint32_t>(p.T * p.blocks[0]);
    const Piece piece(p);
    const bool lane_in = 8 * g < p.D;
    const Place pl = Place::of<LANES, INTER>(p, g, false);
    if (p.norm && sub == 0) {       // by the lanes that add the warp's sums later
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) s_dw[warp][k][8 * g + e] = 0.0f;
    }
    int kind = piece.begin >= items_q ? kKey : kQuery;
    const uint32_t in_kind = kind == kKey ? piece.begin - items_q : piece.begin, t_first = in_kind / p.blocks[kind];
    int64_t t = t_first;
    int block = static_cast<int>(in_kind - t_first * p.blocks[kind]);

    // ---- the ring's producer: the same walk, ahead
    int64_t ahead_t = t;
    int ahead_block = block, ahead_kind = kind, to_issue = piece.count;
    auto issue = [&](int stage) {
        if (lane == 0) {
            const int k = ahead_kind, head = ahead_block * BLOCK;
            const uint32_t bytes = static_cast<uint32_t>(min(BLOCK, p.heads[k] - head) * p.D) * 2u;
            const uint32_t bar = bars + 8 * stage, dst = smem_u32(ring) + stage * kStage;
            const int64_t from = static_cast<int64_t>(head) * p.D;
            mbar_arrive_expect_tx(bar, p.norm ? 2 * bytes : bytes);
#ifdef QFP4_FAULT_INJECTION
            if (!(q.skip_copy && blockIdx.x == 0 && warp == 0))
#endif
            bulk_load(dst, q.dy[k] + ahead_t * q.ldy[k] + from, bytes, bar);
            if (p.norm) bulk_load(dst + kHalfStage, p.x[k] + ahead_t * p.ldx[k] + from, bytes, bar);
        }
        --to_issue;
        if (++ahead_block == p.blocks[ahead_kind]) {
            ahead_block = 0;
            if (++ahead_t == p.T && ahead_kind == kQuery) {
                ahead_t = 0;
                ahead_kind = kKey;
            }
        }
    };
    int position_next = piece.count > 0 && p.positions ? p.positions[t] : 0;
#pragma unroll
    for (int i = 0; i < kStages; ++i)
        if (to_issue > 0) issue(i);

    Eight w, dw = {{0, 0}, {0, 0}};
    // the groups of a warp hold the same elements: added up in a fixed order
    auto flush = [&](int k) {
        float e[8];
        elements<INTER>(dw, e);
        dw = Eight{{0, 0}, {0, 0}};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int o = 16; o >= LANES; o >>= 1) e[i] += __shfl_xor_sync(0xffffffffu, e[i], o);
            if (sub == 0) s_dw[warp][k][8 * g + i] += e[i];
        }
    };
    int stage = 0;
    uint32_t phase = 0;
    bool new_kind = true, dead = false;
#pragma unroll 1
    for (int left = piece.count, run = 0; left > 0; left -= run) {
        run = min(left, p.blocks[kind] - block);        // blocks of this token and kind
        const int heads = p.heads[kind], head0 = block * BLOCK + sub;
        __nv_bfloat16 *dx = q.dx[kind] + t * q.lddx[kind] + static_cast<int64_t>(head0) * p.D;
        int position = position_next;
        const int was = kind;
        block += run;
        if (block == p.blocks[kind]) {
            block = 0;
            if (++t == p.T && kind == kQuery) {
                t = 0;
                kind = kKey;
            }
        }
        if (left > run && p.positions) position_next = p.positions[t];
        if (new_kind) {
            Raw wr = ones();
            if (p.w[was] && lane_in) wr = pl.load(p.w[was]);
            w = unpack<INTER>(wr);
        }
        if (p.R > 0 && position >= p.table_rows) {
            position = -1;
            if (lane == 0) atomicOr(&g_status_heads, kStatusBadGroup);
        }
        const bool alive = position >= 0;       // uniform over the warp
        const Turn turn = Turn::of<INTER>(p, pl, max(position, 0), g);      // not used without a position
        const uint64_t back[2] = {f2_neg(turn.s[0]), f2_neg(turn.s[1])};
#pragma unroll 1
        for (int n = 0; n < run; ++n) {
            if (!dead && !mbar_wait(bars + 8 * stage, phase)) {     // what comes out is undefined, but it ends
                if (lane == 0) atomicOr(&g_status_heads, kStatusTimeout);
                dead = true;
                to_issue = 0;
            }
            const uint8_t *buf = ring + stage * kStage + sub * p.D * 2;
            Raw xv[kBackVectors], dv[kBackVectors];
#pragma unroll
            for (int i = 0; i < kBackVectors; ++i) {
                const __nv_bfloat16 *src = reinterpret_cast<const __nv_bfloat16 *>(buf + i * GROUPS * p.D * 2);
                dv[i] = pl.load(src);
                if (p.norm) xv[i] = pl.load(src + kHalfStage / 2);
            }
            __syncwarp();
            if (to_issue > 0) issue(stage);
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
#pragma unroll
            for (int i = 0; i < kBackVectors; ++i) {
                const bool live = lane_in && head0 + n * BLOCK + i * GROUPS < heads;
                if (!live) xv[i] = dv[i] = Raw{};       // other vectors' elements, or none
                Eight d = {{0, 0}, {0, 0}};
                if (alive) {
                    const Eight v = unpack<INTER>(dv[i]);
                    Eight o = v;
                    if (p.R < p.D && !pl.turns) o = Eight{{0, 0}, {0, 0}};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        d.a[k] = f2_fma(o.b[k], turn.s[k], f2_mul(v.a[k], turn.c[k]));
                        d.b[k] = f2_fma(o.a[k], back[k], f2_mul(v.b[k], turn.c[k]));
                    }
                    if (p.norm) {
                        Eight h = unpack<INTER>(xv[i]), gw;
                        uint64_t ss = 0, dot = 0;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            gw.a[k] = f2_mul(d.a[k], w.a[k]);
                            gw.b[k] = f2_mul(d.b[k], w.b[k]);
                            ss = f2_fma(h.b[k], h.b[k], f2_fma(h.a[k], h.a[k], ss));
                            dot = f2_fma(gw.b[k], h.b[k], f2_fma(gw.a[k], h.a[k], dot));
                        }
                        // no vector: with eps = 0 its root would be that of 0, and the weights' sums NaN
                        const float sum = group_sum<LANES>(f2_sum(ss)), r = live ? rsqrtf(sum * p.inv_D + p.eps) : 0.0f;
                        const float mean = group_sum<LANES>(f2_sum(dot)) * r * p.inv_D;
                        const uint64_t r2 = f2_pack(r, r), m2 = f2_pack(-mean * r, -mean * r);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            h.a[k] = f2_mul(h.a[k], r2);
                            h.b[k] = f2_mul(h.b[k], r2);
                            dw.a[k] = f2_fma(d.a[k], h.a[k], dw.a[k]);
                            dw.b[k] = f2_fma(d.b[k], h.b[k], dw.b[k]);
                            d.a[k] = f2_fma(h.a[k], m2, f2_mul(gw.a[k], r2));
                            d.b[k] = f2_fma(h.b[k], m2, f2_mul(gw.b[k], r2));
                        }
                    }
                }
                if (live) pl.store(dx + i * GROUPS * p.D, pack<INTER>(d));
            }
            dx += BLOCK * p.D;
        }
        new_kind = kind != was;
        if (p.norm && (new_kind || left == run)) flush(was);
    }
    if (dead) {     // copies in flight have time to land before the shared memory goes to another CTA
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) {
        }
    }
    if (!p.norm) return;
    __syncthreads();
    // place i of a lane's eight back to the element that it holds
    for (int i = threadIdx.x; i < 2 * LANES * 8; i += kThreads) {
        const int k = i >= LANES * 8, in = i - k * LANES * 8, gi = in / 8, e = in % 8;
        if (8 * gi >= p.D) continue;
        const Place at = Place::of<LANES, INTER>(p, gi, false);
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < kWarps; ++j) v += s_dw[j][k][in];
        q.partial[static_cast<int64_t>(blockIdx.x) * 2 * p.D + k * p.D + (e < 4 ? at.at[0] + e : at.at[1] + e - 4)] = v;
    }
}

// Weight gradients from the CTAs' partial sums: 32 columns per CTA, each added up
// by 32 threads side by side and then by a tree (sums of 64 bits take 14 us here).
__global__ void __launch_bounds__(1024) head_weight_kernel(const float *partial, int rows, int D, float *dq, float *dk)
{
    __shared__ float s_sum[32][33];
    pdl_wait();
    pdl_launch_dependents();
    const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + c;
    float v = 0.0f;
    if (i < 2 * D) {
#pragma unroll 8
        for (int k = r; k < rows; k += 32) v += partial[static_cast<int64_t>(k) * 2 * D + i];
    }
    s_sum[r][c] = v;
    __syncthreads();
    v = s_sum[c][r];        // lane c of warp r: part c of column r
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int column = blockIdx.x * 32 + r;
    if (c != 0 || column >= 2 * D) return;
    float *out = column < D ? dq : dk;
    if (out) out[column < D ? column : column - D] = v;
}

// ------------------------------------------------------------ cache's write

struct WriteParams {
    CacheParams c;
    const __nv_bfloat16 *in[2];     // K, V
    int64_t ld[2];
    uint32_t vectors, heads;        // vectors: tokens * heads
};

// N neighbouring bytes of codes, N = 4, 8 or 16, from the registers that hold them.
template <int N>
__device__ __forceinline__ void store_codes(uint8_t *at, const uint32_t *w)
{
    if constexpr (N == 4) *reinterpret_cast<uint32_t *>(at) = w[0];
    else if constexpr (N == 8) *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A lane takes 16 elements of a token's key and value vector of a head: a block of
// NVFP4 whole, so that its scale, as much work as its codes, is found once: 32768 tokens
// x 8 heads x 128 take 40 us in NVFP4 (floor 25; bound by the quotients' instructions),
// 32 in E4M3 (30) and 55 in BF16 (40; the pieces of 16 and 64 bytes); head_kernel, whose
// lanes hold eight elements, took 99, 71 and 75.
template <int TYPE, int LANES>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const WriteParams p)
{
    constexpr int D = 16 * LANES, GROUPS = 32 / LANES;
    constexpr CacheUnit U(TYPE, D);
    constexpr int CODES = U.row / LANES, WORDS = CODES / 4;         // of a lane
    constexpr int V_RUN = CODES < 16 ? (U.row / 8 < CODES ? U.row / 8 : CODES) : (U.row / 8 < 16 ? U.row / 8 : 16);
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, g = lane % LANES;
    const uint32_t first = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * GROUPS, mine = first + lane / LANES;
    if (first >= p.vectors) return;
    const uint32_t v = min(mine, p.vectors - 1), t = v / p.heads, head = v - t * p.heads;
    int slot = p.c.slots[t];
    uint4 x[2][2];
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            x[half][i] = reinterpret_cast<const uint4 *>(p.in[half] + t * p.ld[half] + static_cast<int64_t>(head) * D + 16 * g)[i];
    float gs[2] = {1.0f, 1.0f};
    if (TYPE == QFP4_CACHE_NVFP4) {
        gs[0] = *p.c.gs[0];
        gs[1] = *p.c.gs[1];
    }
    if (slot >= p.c.slot_count) {
        if (g == 0) atomicOr(&g_status_heads, kStatusBadGroup);
        slot = -1;
    }
    const bool live = mine < p.vectors && slot >= 0;
    slot = max(slot, 0);
    uint8_t *unit = p.c.cache + (p.c.unit_of(slot) + static_cast<int64_t>(head) * p.c.page_units) * U.bytes;
    const int j = slot & 15;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint32_t w[8] = {x[half][0].x, x[half][0].y, x[half][0].z, x[half][0].w,
                               x[half][1].x, x[half][1].y, x[half][1].z, x[half][1].w};
        uint32_t code[WORDS];
        uint8_t *const k_at = unit + U.k_code(j, g * CODES);
        if constexpr (TYPE == QFP4_CACHE_BF16) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) code[i] = w[i];
        } else {
            float y[16], amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[2 * i] = bf16_lo(w[i]);
                y[2 * i + 1] = bf16_hi(w[i]);
                amax = fmaxf(amax, fmaxf(fabsf(y[2 * i]), fabsf(y[2 * i + 1])));
            }
            if constexpr (TYPE == QFP4_CACHE_E4M3) {
                const float a = fmaxf(group_max<LANES>(amax), kFloor), inv = __fdiv_rn(448.0f, a);
#pragma unroll
                for (int i = 0; i < WORDS; ++i)
                    code[i] = e4m3x2(y[4 * i] * inv, y[4 * i + 1] * inv) | (e4m3x2(y[4 * i + 2] * inv, y[4 * i + 3] * inv) << 16);
                if (live && g == 0) *reinterpret_cast<float *>(unit + (half == 0 ? U.k_token_scale(j) : U.v_token_scale(j))) = __fdiv_rn(a, 448.0f);
            } else {
                const BlockScale b = block_scale<QFP4_NVFP4>(amax, gs[half], __frcp_rn(gs[half]));
#pragma unroll
                for (int i = 0; i < WORDS; ++i) code[i] = encode8_f32<QFP4_NVFP4>(y + 8 * i, b);
                if (live) unit[half == 0 ? U.k_block_scale(j, g) : U.v_block_scale(j, g)] = static_cast<uint8_t>(b.code);
            }
        }
        if (!live) continue;
        if (half == 0) {
            constexpr int RUN = CODES < 16 ? CODES : 16;
#pragma unroll
            for (int i = 0; i < CODES; i += RUN) store_codes<RUN>(k_at + i, code + i / 4);
        } else {
#pragma unroll
            for (int i = 0; i < CODES; i += V_RUN) store_codes<V_RUN>(unit + U.v_code(j, g * CODES + i), code + i / 4);
        }
    }
}

// ------------------------------------------------------------- cache's read

struct ReadParams {
    CacheParams c;
    int64_t T;
    uint32_t heads, warp_heads, parts;      // heads that a warp takes, and how many such parts there are
    __nv_bfloat16 *out[2];      // K, V
    int64_t ldo[2];
};

// A warp takes four tokens and as many heads as leave 48 warps for each SM: what a
// token's place costs is paid once for them (32768 tokens x 8 heads x 128 in NVFP4:
// 31 us, floor 25; a warp for each head, without the next head's loads ahead, 36; as many
// registers as five CTAs per SM have 40).  Where the tokens' slots follow one
// another (a prefix), every 32-byte sector of codes that it reads is used whole.
constexpr int kReadVectors = 2, kReadWarps = 48 * 152, kReadCtas = 4;

// Tokens of a warp: two for each group of lanes that holds a vector.
__host__ __device__ constexpr int read_tokens(int lanes) { return 32 / lanes * kReadVectors; }

// The places of a token's codes and scales in a unit are those of token 0, which a
// lane knows, plus what depends on the token alone.
template <int TYPE, int LANES>
struct TokenPlace {
    int code[2], scale[2];      // keys, values

    __device__ __forceinline__ explicit TokenPlace(int j)
    {
        constexpr CacheUnit U(TYPE, LANES * 8);
        constexpr int PIECE = U.row < 64 ? U.row : 64, W = U.row / 8;
        const int quad = (j >> 3) * 2 + (j & 1), t = (j >> 1) & 3;
        code[0] = (j >> 3) * (U.row / PIECE * 8 * PIECE) + (j & 7) * PIECE;
        code[1] = W >= 16 ? quad * (W / 16 * 512) + t * 16 : (quad * W >> 4) * 512 + t * 16 + (quad * W & 15);
        scale[0] = j * U.scale;
        scale[1] = TYPE == QFP4_CACHE_E4M3 ? 4 * j : 4 * t + quad;
    }
};

// Eight elements of a vector as they lie in the cache.
template <int TYPE>
struct Cached {
    uint32_t code[TYPE == QFP4_CACHE_BF16 ? 4 : TYPE == QFP4_CACHE_E4M3 ? 2 : 1], scale;

    __device__ __forceinline__ void load(const uint8_t *at, const uint8_t *s)
    {
        if constexpr (TYPE == QFP4_CACHE_BF16) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(at));
            code[0] = v.x, code[1] = v.y, code[2] = v.z, code[3] = v.w;
        } else if constexpr (TYPE == QFP4_CACHE_E4M3) {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(at));
            code[0] = v.x, code[1] = v.y;
            scale = __ldg(reinterpret_cast<const uint32_t *>(s));
        } else {
            code[0] = __ldg(reinterpret_cast<const uint32_t *>(at));
            scale = __ldg(s);
        }
    }
    __device__ __forceinline__ uint4 bf16(float gs) const
    {
        if constexpr (TYPE == QFP4_CACHE_BF16) {
            return make_uint4(code[0], code[1], code[2], code[3]);
        } else {
            uint32_t h[4];      // FP16 holds E2M1 and E4M3 values as they are
            float f;
            if constexpr (TYPE == QFP4_CACHE_E4M3) {
                f = __uint_as_float(scale);
                h[0] = lane_ops::fp8x2<0>(code[0]), h[1] = lane_ops::fp8x2<1>(code[0]);
                h[2] = lane_ops::fp8x2<0>(code[1]), h[3] = lane_ops::fp8x2<1>(code[1]);
            } else {
                const uint32_t sh = lane_ops::fp8x2<0>(scale);
                f = __low2float(*reinterpret_cast<const __half2 *>(&sh)) * gs;
                h[0] = lane_ops::fp4x2<0>(code[0]), h[1] = lane_ops::fp4x2<1>(code[0]);
                h[2] = lane_ops::fp4x2<2>(code[0]), h[3] = lane_ops::fp4x2<3>(code[0]);
            }
            const uint64_t f2 = f2_pack(f, f);
            float y[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 c = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
                f2_unpack(f2_mul(f2_pack(c.x, c.y), f2), y[2 * i], y[2 * i + 1]);
            }
            return pack8(y);
        }
    }
};

template <int TYPE, int LANES>
__global__ void __launch_bounds__(kThreads, kReadCtas) cache_read_kernel(const ReadParams p)
{
    constexpr int GROUPS = 32 / LANES, N = kReadVectors;
    constexpr int D = 8 * LANES, UNIT = cache_unit_bytes(TYPE, D);
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, g = lane % LANES, sub = lane / LANES;
    const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5), block = item / p.parts;
    const int64_t t0 = static_cast<int64_t>(block) * read_tokens(LANES);
    if (t0 >= p.T) return;
    const uint32_t head0 = (item - block * p.parts) * p.warp_heads;
    int heads = static_cast<int>(min(p.heads - head0, p.warp_heads));
    float gs[2] = {1.0f, 1.0f};
    if (TYPE == QFP4_CACHE_NVFP4) {
        gs[0] = *p.c.gs[0];
        gs[1] = *p.c.gs[1];
    }
    const CachePlace<TYPE, LANES> k0(0, 0, g), v0(1, 0, g);
    const uint8_t *unit[N];     // NULL: none
    int code[2][N], scale[2][N];
    __nv_bfloat16 *out[2][N];   // NULL: not wanted
    Cached<TYPE> next[2][N] = {};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t t = t0 + i * GROUPS + sub;
        int slot = t < p.T ? p.c.slots[t] : -1;
        if (slot >= p.c.slot_count) {
            atomicOr(&g_status_heads, kStatusBadGroup);
            slot = -1;
        }
        unit[i] = slot < 0 ? nullptr : p.c.cache + (p.c.unit_of(slot) + static_cast<int64_t>(head0) * p.c.page_units) * UNIT;
        const TokenPlace<TYPE, LANES> tp(slot & 15);
        code[0][i] = k0.code + tp.code[0], scale[0][i] = k0.scale + tp.scale[0];
        code[1][i] = v0.code + tp.code[1], scale[1][i] = v0.scale + tp.scale[1];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            out[h][i] = t < p.T && p.out[h] ? p.out[h] + t * p.ldo[h] + static_cast<int64_t>(head0) * D + 8 * g : nullptr;
            if (unit[i]) next[h][i].load(unit[i] + code[h][i], unit[i] + scale[h][i]);
        }
    }
    const int64_t step = static_cast<int64_t>(p.c.page_units) * UNIT;
#pragma unroll 1
    for (; heads > 0; --heads) {
        Cached<TYPE> now[2][N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            now[0][i] = next[0][i];
            now[1][i] = next[1][i];
            if (unit[i] && heads > 1) {
                unit[i] += step;
#pragma unroll
                for (int h = 0; h < 2; ++h) next[h][i].load(unit[i] + code[h][i], unit[i] + scale[h][i]);
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (out[h][i]) {
                    *reinterpret_cast<uint4 *>(out[h][i]) = now[h][i].bf16(gs[h]);
                    out[h][i] += D;
                }
    }
}

// ------------------------------------------------------------------ launches

int lanes_of(int64_t D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }

// Cuts the tokens' heads into blocks and these into the warps' pieces; CTAs of the
// grid: one wave at most, -1 for more blocks than 32 bits count.
int64_t plan_blocks(HeadParams &p, int lanes, int vectors, int per_sm)
{
    const int block = 32 / lanes * vectors;
    int64_t per_token = 0;
    for (int k = 0; k < 3; ++k) per_token += p.blocks[k] = (p.heads[k] + block - 1) / block;
    const int64_t items = p.T * per_token;
    if (items > UINT32_MAX) return -1;
    const int64_t want = (items + kWarps - 1) / kWarps, grid = want < per_sm * 152 ? want : per_sm * 152;
    if (grid > 0) {
        p.share = static_cast<uint32_t>(items / (grid * kWarps));
        p.more = static_cast<uint32_t>(items % (grid * kWarps));
    }
    return grid;
}

template <int LANES, bool INTER>
int launch_heads(HeadParams &p, int cache, cudaStream_t s)
{
    const int64_t grid = plan_blocks(p, LANES, kVectors, head_ctas(cache));
    if (grid < 0) return QFP4_ERR_UNSUPPORTED;
    auto kernel = cache == kNoCache ? head_kernel<LANES, kNoCache, INTER>
                : cache == QFP4_CACHE_BF16 ? head_kernel<LANES, QFP4_CACHE_BF16, INTER>
                : cache == QFP4_CACHE_E4M3 ? head_kernel<LANES, QFP4_CACHE_E4M3, INTER>
                                           : head_kernel<LANES, QFP4_CACHE_NVFP4, INTER>;
    return launch_status(launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, p));
}

int launch_heads_any(HeadParams &p, int cache, cudaStream_t s)
{
    switch (lanes_of(p.D)) {
    case 8: return p.interleaved ? launch_heads<8, true>(p, cache, s) : launch_heads<8, false>(p, cache, s);
    case 16: return p.interleaved ? launch_heads<16, true>(p, cache, s) : launch_heads<16, false>(p, cache, s);
    default: return p.interleaved ? launch_heads<32, true>(p, cache, s) : launch_heads<32, false>(p, cache, s);
    }
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
    if ((D != 64 && D != 128 && D != 256) || page_size % 16 != 0 || page_size > 16384 || kv_heads > kMaxHeads ||
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
    p.inv_D = 1.0f / static_cast<float>(D);
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
    c.page_units = static_cast<int32_t>(page_size / 16);
    // exact for every unit number below 2^27, at most 2^10 units in a page
    c.page_magic = ((uint64_t{1} << 37) + c.page_units - 1) / c.page_units;
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

namespace {

template <int LANES>
int launch_write(const WriteParams &p, int type, cudaStream_t s)
{
    constexpr uint32_t CTA = kWarps * 32 / LANES;
    auto kernel = type == QFP4_CACHE_BF16 ? cache_write_kernel<QFP4_CACHE_BF16, LANES>
                : type == QFP4_CACHE_E4M3 ? cache_write_kernel<QFP4_CACHE_E4M3, LANES>
                                          : cache_write_kernel<QFP4_CACHE_NVFP4, LANES>;
    return launch_status(launch_pdl(kernel, dim3((p.vectors + CTA - 1) / CTA), dim3(kThreads), 0, s, p));
}

}  // namespace

extern "C" int qfp4_kv_cache_write(int type, const void *K_bf16, int64_t ldk, const void *V_bf16, int64_t ldv,
                                   int64_t T, int64_t kv_heads, int64_t head_dim, const int32_t *slots,
                                   const float *gs_k, const float *gs_v, void *cache, int64_t pages,
                                   int64_t page_size, void *stream)
{
    int rc = check_cache(type, kv_heads, head_dim, pages, page_size);
    if (rc == QFP4_ERR_INVALID_ARG || T < 0 || ldk < kv_heads * head_dim || ldv < kv_heads * head_dim)
        return QFP4_ERR_INVALID_ARG;
    if (rc != QFP4_OK || T > kMaxTokens || T * kv_heads > INT32_MAX || ldk % 8 != 0 || ldv % 8 != 0)
        return QFP4_ERR_UNSUPPORTED;
    if (T == 0) return QFP4_OK;
    if (!K_bf16 || !V_bf16) return QFP4_ERR_INVALID_ARG;
    WriteParams p = {};
    rc = fill_cache(p.c, type, cache, kv_heads, pages, page_size, slots, gs_k, gs_v);
    if (rc != QFP4_OK) return rc;
    if (!aligned16(K_bf16) || !aligned16(V_bf16)) return QFP4_ERR_MISALIGNED;
    p.in[0] = static_cast<const __nv_bfloat16 *>(K_bf16);
    p.in[1] = static_cast<const __nv_bfloat16 *>(V_bf16);
    p.ld[0] = ldk;
    p.ld[1] = ldv;
    p.vectors = static_cast<uint32_t>(T * kv_heads);
    p.heads = static_cast<uint32_t>(kv_heads);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (head_dim) {
    case 64: return launch_write<4>(p, type, s);
    case 128: return launch_write<8>(p, type, s);
    default: return launch_write<16>(p, type, s);
    }
}

namespace {

template <int LANES>
int launch_read(ReadParams &p, int type, cudaStream_t s)
{
    const int64_t blocks = (p.T + read_tokens(LANES) - 1) / read_tokens(LANES), share = blocks * p.heads / kReadWarps;
    p.warp_heads = share < 1 ? 1 : share < p.heads ? static_cast<uint32_t>(share) : p.heads;
    p.parts = (p.heads + p.warp_heads - 1) / p.warp_heads;
    const int64_t grid = (blocks * p.parts + kWarps - 1) / kWarps;
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
    if (rc != QFP4_OK || T > kMaxTokens || T * kv_heads > INT32_MAX || (K_out && ldk % 8 != 0) || (V_out && ldv % 8 != 0))
        return QFP4_ERR_UNSUPPORTED;
    if (T == 0) return QFP4_OK;
    if (!K_out && !V_out) return QFP4_ERR_INVALID_ARG;
    ReadParams p = {};
    rc = fill_cache(p.c, type, const_cast<void *>(cache), kv_heads, pages, page_size, slots, gs_k, gs_v);
    if (rc != QFP4_OK) return rc;
    if (!aligned16(K_out) || !aligned16(V_out)) return QFP4_ERR_MISALIGNED;
    p.T = T;
    p.heads = static_cast<uint32_t>(kv_heads);
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
    HeadParams p = {};
    p.T = T;
    p.heads[0] = static_cast<int32_t>(q_heads);
    p.heads[1] = static_cast<int32_t>(kv_heads);
    // partial sums of the weights' gradients, a pair of vectors per CTA
    const int64_t ctas = plan_blocks(p, lanes_of(head_dim), kBackVectors, kBackCtas);
    return ctas < 0 ? 0 : static_cast<size_t>(ctas) * 2 * head_dim * sizeof(float);
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
        const int lanes = lanes_of(head_dim);
        const int64_t ctas = plan_blocks(b.f, lanes, kBackVectors, kBackCtas);
        if (ctas < 0) return QFP4_ERR_UNSUPPORTED;
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
#ifdef QFP4_FAULT_INJECTION
        b.skip_copy = inject_skip_copy();
#endif
        const dim3 grid(static_cast<unsigned>(ctas));
        auto kernel = lanes == 8 ? (interleaved ? head_backward_kernel<8, true> : head_backward_kernel<8, false>)
                    : lanes == 16 ? (interleaved ? head_backward_kernel<16, true> : head_backward_kernel<16, false>)
                                  : (interleaved ? head_backward_kernel<32, true> : head_backward_kernel<32, false>);
        int st = ensure_smem_attr(reinterpret_cast<const void *>(kernel), kRing);
        if (st == QFP4_OK) st = launch_status(launch_pdl(kernel, grid, dim3(kThreads), kRing, s, b));
        if (st != QFP4_OK || !norm) return st;
        return launch_status(launch_pdl(head_weight_kernel, dim3(columns), dim3(1024), 0, s, b.partial,
                                        static_cast<int>(grid.x), D, dq_weight, dk_weight));
    }
    // no token: zero gradients
    if (!norm) return QFP4_OK;
    return launch_status(launch_pdl(head_weight_kernel, dim3(columns), dim3(1024), 0, s,
                                    static_cast<const float *>(nullptr), 0, D, dq_weight, dk_weight));
}
