// qfp4_attention.cuh -- attention of one new token per sequence over the paged
// cache (see qfp4_kv_cache.cuh for the cache's layout).  One translation unit
// per cache type instantiates the kernel.
//
//   x_j = scale q . k_j (in units of log 2),  p_j = 2^(x_j - m),
//   o = sum p_j v_j / sum p_j,  lse = ln 2 (m + log2 sum p_j)
// in one pass over the cache, with m, the sums and o in fp32 registers.  m follows the
// largest x_j (attn_headroom below it, and up to kSlack more).
//
// Bound by the cache's bytes.  A warp takes 16 tokens as the rows of a tensor
// core product with up to 8 (or 16) query heads that share the key head as its
// columns: S^T = K Q^T, then O^T = V^T P^T, so a group of 8 heads fills the
// columns and the cache is read once for all of them.  The codes go from shared
// memory to the operand registers as they lie, 16 bytes per lane and free of bank
// conflicts, and become FP16 there: E2M1 and E4M3 values and their products with
// UE4M3 scales have at most 6 significant bits and are exact in FP16.  Queries
// become FP16 too, each multiplied by the power of two that takes its largest
// element to [2^14, 2^15): what lies 2^28 below that loses bits, 2^-39 of the
// largest at most.  p is rounded to FP16: 2^-11 of it, or 2^-25, 2^-32 of the largest
// p at most, which lies between 2^7 and 2^15.  An E4M3 token's value scale s joins it as
// 2^(x + log2 s - m'), m' the like of m for that exponent, so that no range of scales
// is lost.  With a BF16 cache the operands are BF16 and p is the
// sum of two (2^-16).
//
// The tokens of all sequences and heads are one line of tiles; each CTA takes an
// equal piece of it, whatever the lengths, and the pieces of a head that lies
// across CTAs are joined by the one that finishes last (many pieces in groups, and then
// the groups), in the order of the pieces: results repeat bit for bit.  Each warp brings its own tokens with bulk
// copies into a ring of stages of its own, ahead of the tile that it works on and
// across the heads' borders; no other warp waits for it until a head ends.
//
// Measured (of the copy bandwidth, head_dim 128): BF16 64 ragged sequences of up to
// 8192 x 8 heads 181 us (0.93), E4M3 103 us (0.84); NVFP4 4 x 131072 x 8 heads 123 us
// (0.73).  What is left of NVFP4 are instructions: a unit of 16 tokens takes about 330,
// 64 conversions and 64 multiplications by scales among them, at 2.4 a cycle.  Its 16
// warps per SM of 128 registers beat 12 of 168 (131 us against 159 at that time); stages
// of 64 tokens, which halve the work around each, leave room for 12 warps only (147 us).
// With up to 16 queries per key head it has 8 warps of 232 registers (104 us for 16 x
// 16384 x 8 heads, floor 45).
// Short calls are a chain of latencies: length, page number, tokens, first products,
// warps' join, pieces' join; 1 x 4096 tokens x 8 heads take 10.5 us, 3 of them the
// pieces'.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qfp4_common.cuh"
#include "qfp4_kv_cache.cuh"
#include "qfp4_lane_ops.cuh"
#include "sm103_ptx.cuh"

namespace qfp4 {

struct AttnParams {
    const __nv_bfloat16 *q;     // [B, q_heads, D], ldq elements from sequence to sequence
    int64_t ldq;
    int32_t B, kv_heads, group; // group: query heads of a key head
    int32_t blocks;             // blocks of query heads in a group
    const uint8_t *cache;
    int64_t pages;
    int32_t page_units, max_pages, window;      // page_units: page_size / 16
    uint64_t page_magic;        // ceil(2^36 / page_units): what a division by it is done with
    const int32_t *page_table, *lengths;
    float scale_log2;           // scale * log2(e)
    const float *gs_k, *gs_v;
    __nv_bfloat16 *out;         // [B, q_heads, D]
    float *lse;                 // [B, q_heads] or NULL
    uint32_t *counters;         // [3][kAttnMaxCtas], zero before and after
    float *partial;             // [grid][2] pieces
    uint32_t *status;
#ifdef QFP4_FAULT_INJECTION
    bool skip_copy;
#endif
};

// CTAs that the workspace is sized for at most: 152 SMs, eight on each.
constexpr int kAttnMaxCtas = 152 * 8;

// Pieces that are joined at a time: an item's all, or groups of them whose joined pieces
// are joined in turn (one sequence of 131072 tokens with one key head, 304 to 608 pieces:
// NVFP4 16 us, 38 all at once; BF16 26, 78).
__device__ __forceinline__ int attn_join_group(int pieces) { return pieces <= 24 ? pieces : pieces <= 256 ? 16 : 32; }

// Space of a piece in the workspace: o, then m and l of each query.
__host__ __device__ constexpr int attn_piece_floats(int queries, int D) { return queries * (D + 2); }

// Tokens of a warp's stage, stages of its ring, and CTAs per SM that the registers
// are sized for.  Shared memory holds fewer of some: of four warps three in E4M3 and BF16
// (one in BF16 with 256 elements), of two warps five in E4M3 and six in BF16.  That those
// forms would gain by registers for what fits is not measured.
constexpr int attn_stage_tokens(int type, int D)
{
    return type == QFP4_CACHE_BF16 ? (D == 64 ? 32 : 16) : D == 64 ? 64 : D == 128 ? 32 : 16;
}
constexpr int kAttnStages = 2;
// How far the largest exponent lies above its base when that moves, and how much further
// it may rise before it moves again: weights of 2^7 to 2^15 leave FP16 the range below for
// the small ones.  A BF16 cache's weights have BF16's range.
constexpr float kSlack = 8.0f;
constexpr float attn_headroom(int type) { return type == QFP4_CACHE_BF16 ? 0.0f : 7.0f; }
constexpr int attn_ctas(int type, int D, int nt, int warps)
{
    return (D == 256 ? (type == QFP4_CACHE_NVFP4 ? 12 : 8) : nt == 2 ? 8 : 16) / warps;
}

template <int TYPE, int D, int NT, int WARPS_>
struct AttnCfg {
    static constexpr int TOKENS = attn_stage_tokens(TYPE, D), STAGES = kAttnStages, UNITS = TOKENS / 16;
    static constexpr int UNIT = cache_unit_bytes(TYPE, D), STAGE = UNITS * UNIT;
    static constexpr int WARPS = WARPS_, THREADS = 32 * WARPS;
    static constexpr int TILE = TOKENS * WARPS;
    static constexpr int QUERIES = 8 * NT;
    static constexpr float HEADROOM = attn_headroom(TYPE);
    static constexpr int RING = WARPS * STAGES * STAGE;
    // Where the warps' results meet: half of them side by side, or one after the
    // other where more would cost a CTA per SM.
    static constexpr int SUMS = TYPE == QFP4_CACHE_NVFP4 && D <= 128 ? WARPS / 2 : 1, SUM = QUERIES * (D + 4);
    static constexpr int JOIN = SUMS * SUM * 4 + WARPS * QUERIES * 8;
    static constexpr int BARS = WARPS * STAGES * 8;
    static constexpr int SMEM = RING + JOIN + BARS;
};

namespace attn {

using namespace lane_ops;

template <int TYPE>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (TYPE == QFP4_CACHE_BF16) mma_bf16(c, a, b0, b1);
    else mma_f16(c, a, b0, b1);
}

// How the line of tiles is dealt out.  Evenly where there are more than two for each CTA
// of the grid.  Else one for each, so that as many as can load, or two: where there are
// more than CTAs, where an item has at least 32 (half as many pieces to join: BF16, 1 x
// 4096 tokens x 8 heads 13.4 us, 15.9 with one), and where it has two (none to join:
// NVFP4, 512 tokens 7.5 us, 8.9).  Three and four were slower.
struct Shares {
    int64_t total, ctas;
    int fixed;          // tiles of a CTA; 0: evenly

    __device__ __forceinline__ Shares(const AttnParams &p, int64_t tiles) : total(tiles)
    {
        const int64_t grid = gridDim.x, items = static_cast<int64_t>(p.B) * p.kv_heads * p.blocks;
        const bool two = total > grid || total >= 32 * items || (total > items && total <= 2 * items);
        fixed = total > 2 * grid ? 0 : two ? 2 : 1;
        ctas = fixed ? (total + fixed - 1) >> (fixed - 1) : grid;
    }
    __device__ __forceinline__ int64_t begin_of(int64_t cta) const
    {
        return fixed ? min(cta * fixed, total) : cta * total / ctas;
    }
    __device__ __forceinline__ int64_t cta_of(int64_t tile) const
    {
        return fixed ? tile >> (fixed - 1) : ((tile + 1) * ctas - 1) / total;
    }
};

// Where a CTA stands on the line of tiles: sequence, (key head, query block) and tile.
struct Cursor {
    int b, head, block, tile, tiles;
    int first, len;             // tokens that the sequence's tiles begin at (a multiple of 16) and end before

    template <int TILE>
    __device__ __forceinline__ void load(const AttnParams &p)
    {
        first = tiles = len = 0;
        if (b >= p.B) return;
        extent(p, p.lengths[b], first, len);
        tiles = count<TILE>(first, len);
    }
    __device__ static __forceinline__ void extent(const AttnParams &p, int length, int &first, int &len)
    {
        const int64_t most = static_cast<int64_t>(p.max_pages) * p.page_units * 16;
        len = length < 0 ? 0 : length > most ? static_cast<int>(most) : length;
        first = p.window > 0 && len > p.window ? (len - p.window) & ~15 : 0;
    }
    // an empty sequence has one tile, which writes its zeros
    template <int TILE>
    __device__ static __forceinline__ int count(int first, int len)
    {
        const int n = (len - first + TILE - 1) / TILE;
        return n > 0 ? n : 1;
    }
    template <int TILE>
    __device__ __forceinline__ void next(const AttnParams &p)
    {
        skip<TILE>(p, 1);
    }
    // n tiles on, to the next item at most
    template <int TILE>
    __device__ __forceinline__ void skip(const AttnParams &p, int n)
    {
        if ((tile += n) < tiles) return;
        tile = 0;
        if (++block < p.blocks) return;
        block = 0;
        if (++head < p.kv_heads) return;
        head = 0;
        ++b;
        load<TILE>(p);
    }
};

}  // namespace attn

template <int TYPE, int D, int NT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, attn_ctas(TYPE, D, NT, WARPS)) attention_decode_kernel(const AttnParams p)
{
    using namespace attn;
    using C = AttnCfg<TYPE, D, NT, WARPS>;
    constexpr CacheUnit U(TYPE, D);
    constexpr int UNITS = C::UNITS, STAGES = C::STAGES, TILE = C::TILE, QUERIES = C::QUERIES;
    constexpr int KSTEPS = D / 16, MTILES = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_sum[C::WARPS];
    __shared__ int64_t s_start[2];      // the CTA's first tile: sequence, tile within it
    __shared__ int64_t s_total;         // tiles of the whole line
    __shared__ uint32_t s_last;
    // items that lie across CTAs and a group of whose pieces this CTA completed: CTAs of the
    // pieces, and the first of the group; n = 0 for none
    struct Late {
        int b, head, block, c0, n, first;
    };
    __shared__ Late s_late[2];
    float *s_o = reinterpret_cast<float *>(smem + C::RING);                     // [QUERIES][D + 4]
    float2 *s_ml = reinterpret_cast<float2 *>(s_o + C::SUMS * C::SUM);         // [warps][QUERIES]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const uint32_t bars = smem_u32(smem + C::RING + C::JOIN) + warp * STAGES * 8;
    uint8_t *ring = smem + warp * STAGES * C::STAGE;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i) mbar_init(bars + 8 * i, 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_launch_dependents();

    // ---- the CTA's piece of the line of tiles
    const int items = p.kv_heads * p.blocks;
    // `per` neighbouring sequences for each thread: its tiles, and where they begin in its warp's
    const int per = (p.B + C::THREADS - 1) / C::THREADS;
    int64_t mine = 0;
    bool bad = false;
#pragma unroll 4
    for (int b = tid * per; b < min(p.B, (tid + 1) * per); ++b) {
        int first, len;
        const int length = __ldg(p.lengths + b);
        Cursor::extent(p, length, first, len);
        bad |= length != len;
        mine += static_cast<int64_t>(items) * Cursor::count<TILE>(first, len);
    }
    if (bad && blockIdx.x == 0) atomicOr(p.status, kStatusBadGroup);
    auto sums_up_to = [lane](int64_t v) {       // of the warp's lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        return v;
    };
    const int64_t mine_upto = sums_up_to(mine);
    if (lane == 31) s_sum[warp] = mine_upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int i = 0; i < C::WARPS; ++i) total += s_sum[i];
    int64_t lo, hi;
    {
        const Shares shares(p, total);
        if (blockIdx.x >= shares.ctas) return;
        lo = shares.begin_of(blockIdx.x);
        hi = shares.begin_of(blockIdx.x + 1);
        if (tid == 0) s_total = total;
        if (tid < 2) s_late[tid].n = 0;
    }
    // the thread whose sequences hold the first tile; then the sequence, by its warp
    int64_t from = mine_upto - mine;
    for (int i = 0; i < warp; ++i) from += s_sum[i];
    const bool here = lo >= from && lo < from + mine;
    const uint32_t holds = __ballot_sync(0xffffffffu, here);
    if (here && per == 1) {
        s_start[0] = tid;
        s_start[1] = lo - from;
    }
    if (holds && per > 1) {
        const int which = __ffs(static_cast<int>(holds)) - 1, b1 = min(p.B, (warp * 32 + which + 1) * per);
        from = __shfl_sync(0xffffffffu, from, which);
        for (int b0 = (warp * 32 + which) * per; b0 < b1; b0 += 32) {
            const int b = b0 + lane;
            int64_t n = 0;
            if (b < b1) {
                int first, len;
                Cursor::extent(p, __ldg(p.lengths + b), first, len);
                n = static_cast<int64_t>(items) * Cursor::count<TILE>(first, len);
            }
            const int64_t upto = from + sums_up_to(n);
            if (n > 0 && lo >= upto - n && lo < upto) {
                s_start[0] = b;
                s_start[1] = lo - (upto - n);
            }
            from = __shfl_sync(0xffffffffu, upto, 31);
            if (from > lo) break;
        }
    }
    __syncthreads();
    Cursor cur;
    cur.b = static_cast<int>(s_start[0]);
    cur.load<TILE>(p);
    const int item0 = s_start[1] <= UINT32_MAX ? static_cast<uint32_t>(s_start[1]) / static_cast<uint32_t>(cur.tiles) : static_cast<int>(s_start[1] / cur.tiles);
    cur.head = item0 / p.blocks;
    cur.block = item0 - cur.head * p.blocks;
    cur.tile = static_cast<int>(s_start[1] - static_cast<int64_t>(item0) * cur.tiles);

    // ---- the warp's ring
    Cursor ahead = cur;
    int64_t to_issue = hi - lo;
    // This lane's unit of the tile that a cursor stands at: its page (-1: none) and
    // place there.
    struct Unit {
        int page, place;
    };
    const int lane_token = warp * C::TOKENS + 16 * lane;
    auto unit_of = [&](const Cursor &c) {
        const int token = c.first + c.tile * TILE + lane_token;
        Unit u{-1, -1};
        if (lane < UNITS && token < c.len) {        // a stage has room for UNITS
            const uint32_t n = static_cast<uint32_t>(token) / 16;
            const uint32_t page = static_cast<uint32_t>(n * p.page_magic >> 36);
            u.page = p.page_table[static_cast<int64_t>(c.b) * p.max_pages + page];
            u.place = static_cast<int>(n - page * p.page_units);
        }
        return u;
    };
    auto issue = [&](int head, Unit u, int stage) {
        const bool has = u.place >= 0;
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, has));
        if (has && static_cast<uint32_t>(u.page) >= static_cast<uint32_t>(p.pages)) {
            atomicOr(p.status, kStatusBadGroup);
            u.page = 0;
        }
        if (lane == 0) mbar_arrive_expect_tx(bars + 8 * stage, n * C::UNIT);
        __syncwarp();
#ifdef QFP4_FAULT_INJECTION
        if (p.skip_copy && blockIdx.x == 0 && warp == 0 && lane == 0) return;
#endif
        if (has) {
            const int64_t unit = (static_cast<int64_t>(u.page) * p.kv_heads + head) * p.page_units + u.place;
            bulk_load(smem_u32(ring + stage * C::STAGE + lane * C::UNIT), p.cache + unit * C::UNIT, C::UNIT, bars + 8 * stage);
        }
    };
    {       // the first stages: all page numbers are on their way before the first is waited for
        int head[STAGES], n = 0;
        Unit u[STAGES];
#pragma unroll
        for (int i = 0; i < STAGES; ++i) {
            head[i] = ahead.head;
            if (i < to_issue) {
                u[i] = unit_of(ahead);
                ahead.next<TILE>(p);
                n = i + 1;
            }
        }
#pragma unroll
        for (int i = 0; i < STAGES; ++i)
            if (i < n) issue(head[i], u[i], i);
        to_issue -= n;
    }
    Unit next{-1, -1};
    if (to_issue > 0) next = unit_of(ahead);

    int stage = 0;
    uint32_t phase = 0;
    bool dead = false;
    const float gs_k = TYPE == QFP4_CACHE_NVFP4 ? *p.gs_k : 1.0f, gs_v = TYPE == QFP4_CACHE_NVFP4 ? *p.gs_v : 1.0f;
    int64_t at = lo;

    // The queries of the cursor's head as they are in memory: on their way while the
    // segment before is joined.
    uint32_t qf[NT][KSTEPS][2];
    auto load_q = [&] {
        const int queries = min(QUERIES, p.group - cur.block * QUERIES);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bool has = 8 * n + g < queries;
            const __nv_bfloat16 *src = p.q + cur.b * p.ldq + (static_cast<int64_t>(cur.head) * p.group + cur.block * QUERIES + 8 * n + g) * D;
            // k step (chunk i, u): lane t's dims are four of chunk 4 i + t of the row
            constexpr int EC = U.row / 4 >= 16 ? 16 * D / U.row : D / 4;    // elements of a chunk
#pragma unroll
            for (int ks = 0; ks < KSTEPS; ++ks) {
                const int i = ks / (EC / 4), u = ks % (EC / 4);
                uint2 v = make_uint2(0, 0);
                if (has) v = *reinterpret_cast<const uint2 *>(src + (4 * i + t) * EC + 4 * u);
                qf[n][ks][0] = v.x;
                qf[n][ks][1] = v.y;
            }
        }
    };
    load_q();
    while (at < hi) {
        // ---- a segment: the CTA's tiles of one (sequence, key head, query block)
        const int b = cur.b, head = cur.head, qblock = cur.block, seg_first = cur.tile, seg_tiles = cur.tiles, len = cur.len, first = cur.first;
        const int visible = p.window > 0 && len > p.window ? len - p.window : 0;      // first token that counts

        float qmul[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float back = 1.0f;      // what the products of this lane's query are multiplied by
            if (TYPE != QFP4_CACHE_BF16) {
                float amax = 0.0f;
#pragma unroll
                for (int ks = 0; ks < KSTEPS; ++ks)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(qf[n][ks][r] << 16)), fabsf(__uint_as_float(qf[n][ks][r] & 0xFFFF0000u))));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // the exponent that takes amax to [2^14, 2^15); an infinity takes everything
                // beside it into FP16's range, so that it alone counts
                const int e = min(126, 14 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127));
                const float up = pow2(e);
                back = pow2(-e);
#pragma unroll
                for (int ks = 0; ks < KSTEPS; ++ks)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t v = qf[n][ks][r];
                        qf[n][ks][r] = pack_f16(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xFFFF0000u) * up);
                    }
            }
            back *= p.scale_log2 * gs_k;
            // the products' columns 2t, 2t + 1
            qmul[n][0] = __shfl_sync(0xffffffffu, back, 8 * t);
            qmul[n][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
        }

        // m, mw: what l and o are relative to, base and base_w the same or 0 for none
        float o[NT][MTILES][4], m[NT][2], mw[NT][2], base[NT][2], base_w[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < MTILES; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[n][i][k] = 0.0f;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                m[n][k] = mw[n][k] = -INFINITY;
                base[n][k] = base_w[n][k] = l[n][k] = 0.0f;
            }
        }

        const int seg_n = static_cast<int>(hi - at < seg_tiles - seg_first ? hi - at : seg_tiles - seg_first);
        int token0 = first + seg_first * TILE + warp * C::TOKENS;
#pragma unroll 1
        for (int n_tile = 0; n_tile < seg_n; ++n_tile, token0 += TILE) {
            if (!dead && !mbar_wait(bars + 8 * stage, phase)) {     // what comes out is undefined, but it ends
                if (lane == 0) atomicOr(p.status, kStatusTimeout);
                dead = true;
                to_issue = 0;
            }
            const uint8_t *buf = ring + stage * C::STAGE;
            const int units = min(UNITS, max(0, (len - token0 + 15) >> 4));
            if (units > 0) {
                // ---- logits: rows are tokens g and g + 8 of each unit, columns the queries 2t and 2t + 1
                float x[UNITS][NT][4];
                float ls[UNITS][2];     // E4M3: log2 of the value scales
#pragma unroll
                for (int un = 0; un < UNITS; ++un) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[un][n][k] = 0.0f;
                    ls[un][0] = ls[un][1] = 0.0f;
                    if (un < units) {
                        const uint8_t *unit = buf + un * C::UNIT;
                        constexpr int CB = U.row / 4 >= 16 ? 16 : U.row / 4;    // bytes of a chunk
                        constexpr int CHUNKS = U.row / (4 * CB), KPC = KSTEPS / CHUNKS;
#pragma unroll
                        for (int i = 0; i < CHUNKS; ++i) {
                            uint32_t w[2][4];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint8_t *src = unit + U.k_code(8 * h, (4 * i) * CB) + g * (4 * CB) + t * CB;
                                if constexpr (CB == 16) {
                                    const uint4 v = *reinterpret_cast<const uint4 *>(src);
                                    w[h][0] = v.x, w[h][1] = v.y, w[h][2] = v.z, w[h][3] = v.w;
                                } else {
                                    const uint2 v = *reinterpret_cast<const uint2 *>(src);
                                    w[h][0] = v.x, w[h][1] = v.y, w[h][2] = w[h][3] = 0;
                                }
                            }
                            uint32_t sc[2][2] = {};     // NVFP4: a block's scale, twice
                            if constexpr (TYPE == QFP4_CACHE_NVFP4) {
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    if constexpr (CB == 16) {
                                        const uint32_t v = fp8x2<0>(*reinterpret_cast<const uint16_t *>(
                                            unit + U.k_scales + (8 * h + g) * U.scale + 2 * (4 * i + t)));
                                        sc[h][0] = __byte_perm(v, 0, 0x1010);
                                        sc[h][1] = __byte_perm(v, 0, 0x3232);
                                    } else {
                                        const uint32_t v = fp8x2<0>(unit[U.k_scales + (8 * h + g) * U.scale + t]);
                                        sc[h][0] = __byte_perm(v, 0, 0x1010);
                                    }
                                }
                            }
#pragma unroll
                            for (int u = 0; u < KPC; ++u) {
                                uint32_t a[4];
                                if constexpr (TYPE == QFP4_CACHE_NVFP4) {
                                    const int word = u / 2;
                                    const uint32_t s0 = sc[0][u / 4], s1 = sc[1][u / 4];
                                    if (u & 1) {
                                        a[0] = mul_f16x2(fp4x2<2>(w[0][word]), s0);
                                        a[1] = mul_f16x2(fp4x2<2>(w[1][word]), s1);
                                        a[2] = mul_f16x2(fp4x2<3>(w[0][word]), s0);
                                        a[3] = mul_f16x2(fp4x2<3>(w[1][word]), s1);
                                    } else {
                                        a[0] = mul_f16x2(fp4x2<0>(w[0][word]), s0);
                                        a[1] = mul_f16x2(fp4x2<0>(w[1][word]), s1);
                                        a[2] = mul_f16x2(fp4x2<1>(w[0][word]), s0);
                                        a[3] = mul_f16x2(fp4x2<1>(w[1][word]), s1);
                                    }
                                } else if constexpr (TYPE == QFP4_CACHE_E4M3) {
                                    a[0] = fp8x2<0>(w[0][u]);
                                    a[1] = fp8x2<0>(w[1][u]);
                                    a[2] = fp8x2<1>(w[0][u]);
                                    a[3] = fp8x2<1>(w[1][u]);
                                } else {
                                    a[0] = w[0][2 * u];
                                    a[1] = w[1][2 * u];
                                    a[2] = w[0][2 * u + 1];
                                    a[3] = w[1][2 * u + 1];
                                }
#pragma unroll
                                for (int n = 0; n < NT; ++n) mma<TYPE>(x[un][n], a, qf[n][i * KPC + u][0], qf[n][i * KPC + u][1]);
                            }
                        }
                        float ks0 = 1.0f, ks1 = 1.0f;
                        if constexpr (TYPE == QFP4_CACHE_E4M3) {
                            ks0 = *reinterpret_cast<const float *>(unit + U.k_token_scale(0) + 4 * g);
                            ks1 = *reinterpret_cast<const float *>(unit + U.k_token_scale(8) + 4 * g);
                            ls[un][0] = log2_fast(*reinterpret_cast<const float *>(unit + U.v_token_scale(0) + 4 * g));
                            ls[un][1] = log2_fast(*reinterpret_cast<const float *>(unit + U.v_token_scale(8) + 4 * g));
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            x[un][n][0] *= qmul[n][0] * ks0;
                            x[un][n][1] *= qmul[n][1] * ks0;
                            x[un][n][2] *= qmul[n][0] * ks1;
                            x[un][n][3] *= qmul[n][1] * ks1;
                        }
                    }
                }
                // tokens outside the sequence or its window: whatever lies there does not count
                if (token0 < visible || token0 + C::TOKENS > len) {
#pragma unroll
                    for (int un = 0; un < UNITS; ++un)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int token = token0 + 16 * un + 8 * h + g;
                            if (token < visible || token >= len) {
#pragma unroll
                                for (int n = 0; n < NT; ++n) x[un][n][2 * h] = x[un][n][2 * h + 1] = -INFINITY;
                                ls[un][h] = 0.0f;
                            }
                        }
                }
                // ---- what the exponents are taken relative to.  It moves only when a logit
                // lies more than the headroom and kSlack above it (the weights are as exact in
                // FP16 there), to the headroom below the maximum of the logits so far; with
                // value scales it is that of x + log2 s which matters for FP16, and moves so.  A
                // NaN moves it too.  The limit is rounded down: at logits whose last bit is 16 it
                // would be 16 above, beyond FP16.
                constexpr float HEAD_W = C::HEADROOM, HEAD = TYPE == QFP4_CACHE_E4M3 ? 0.0f : HEAD_W;
                bool above = false;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int un = 0; un < UNITS; ++un)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                above |= !(x[un][n][2 * h + k] <= __fadd_rd(m[n][k], HEAD + kSlack));
                                if (TYPE == QFP4_CACHE_E4M3) above |= !(x[un][n][2 * h + k] + ls[un][h] <= __fadd_rd(mw[n][k], HEAD_W + kSlack));
                            }
                if (__any_sync(0xffffffffu, above)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float alpha[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float top = -INFINITY, top_w = -INFINITY;
#pragma unroll
                            for (int un = 0; un < UNITS; ++un) {
                                top = max_nan(top, max_nan(x[un][n][k], x[un][n][2 + k]));
                                if (TYPE == QFP4_CACHE_E4M3)
                                    top_w = max_nan(top_w, max_nan(x[un][n][k] + ls[un][0], x[un][n][2 + k] + ls[un][1]));
                            }
#pragma unroll
                            for (int s = 4; s < 32; s <<= 1) {
                                top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, s));
                                if (TYPE == QFP4_CACHE_E4M3) top_w = max_nan(top_w, __shfl_xor_sync(0xffffffffu, top_w, s));
                            }
                            const float m_new = max_nan(m[n][k], top - HEAD);
                            base[n][k] = m_new == -INFINITY ? 0.0f : m_new;
                            alpha[k] = exp2_fast(m[n][k] - base[n][k]);
                            l[n][k] *= alpha[k];
                            m[n][k] = m_new;
                            if (TYPE == QFP4_CACHE_E4M3) {
                                const float w_new = max_nan(mw[n][k], top_w - HEAD_W);
                                base_w[n][k] = w_new == -INFINITY ? 0.0f : w_new;
                                alpha[k] = exp2_fast(mw[n][k] - base_w[n][k]);
                                mw[n][k] = w_new;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < MTILES; ++i) {
                            o[n][i][0] *= alpha[0];
                            o[n][i][1] *= alpha[1];
                            o[n][i][2] *= alpha[0];
                            o[n][i][3] *= alpha[1];
                        }
                    }
                }
                // ---- weights and their products with the values
#pragma unroll
                for (int un = 0; un < UNITS; ++un) {
                    if (un >= units) continue;
                    const uint8_t *unit = buf + un * C::UNIT;
                    uint32_t pf[NT][2], pl[NT][2];      // operand P^T, and what BF16 leaves of it
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float x0 = x[un][n][2 * h], x1 = x[un][n][2 * h + 1];
                            const float p0 = exp2_fast(x0 - base[n][0]), p1 = exp2_fast(x1 - base[n][1]);
                            l[n][0] += p0;
                            l[n][1] += p1;
                            pl[n][h] = 0;
                            if constexpr (TYPE == QFP4_CACHE_BF16) {
                                const uint32_t v = pack_bf16(p0, p1);
                                pf[n][h] = transpose8x8(v);
                                pl[n][h] = transpose8x8(pack_bf16(p0 - __uint_as_float(v << 16), p1 - __uint_as_float(v & 0xFFFF0000u)));
                            } else if constexpr (TYPE == QFP4_CACHE_E4M3) {
                                pf[n][h] = transpose8x8(pack_f16(exp2_fast(x0 + ls[un][h] - base_w[n][0]),
                                                                 exp2_fast(x1 + ls[un][h] - base_w[n][1])));
                            } else {
                                pf[n][h] = transpose8x8(pack_f16(p0, p1));
                            }
                        }
                    // this lane's tokens s = 2 h + e: 8 h + 2 t + e
                    const int tok = token0 + 16 * un + 2 * t;
                    const bool part = token0 + 16 * un < visible || token0 + 16 * un + 16 > len;
                    uint32_t live = 0xF;
                    if (part) {
                        live = 0;
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            const int token = tok + 8 * (s >> 1) + (s & 1);
                            if (token >= visible && token < len) live |= 1u << s;
                        }
                    }
                    constexpr int W = U.row / 8;                        // bytes of a token that a lane holds
                    constexpr int STEP = W >= 16 ? 4 : W / 4;           // words of a token per round
#pragma unroll
                    for (int y0 = 0; y0 < W / 4; y0 += STEP) {
                        uint32_t w[4][STEP];
                        const uint4 *src = reinterpret_cast<const uint4 *>(unit + U.v_codes) + lane;
                        if constexpr (W >= 16) {
#pragma unroll
                            for (int s = 0; s < 4; ++s) {
                                const uint4 v = src[(s * (W / 16) + y0 / 4) * 32];
                                w[s][0] = v.x, w[s][1] = v.y, w[s][2] = v.z, w[s][3] = v.w;
                            }
                        } else if constexpr (W == 8) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint4 v = src[h * 32];
                                w[2 * h][0] = v.x, w[2 * h][1] = v.y, w[2 * h + 1][0] = v.z, w[2 * h + 1][1] = v.w;
                            }
                        } else {
                            const uint4 v = src[0];
                            w[0][0] = v.x, w[1][0] = v.y, w[2][0] = v.z, w[3][0] = v.w;
                        }
                        if (part) {
#pragma unroll
                            for (int s = 0; s < 4; ++s)
#pragma unroll
                                for (int y = 0; y < STEP; ++y) w[s][y] = live >> s & 1 ? w[s][y] : 0u;
                        }
#pragma unroll
                        for (int y = 0; y < STEP; ++y) {
                            if constexpr (TYPE == QFP4_CACHE_NVFP4) {
                                // block of these eight dims; the scales of the lane's four tokens lie together
                                const int blk = (g * (D / 8) + 8 * (y0 + y)) / 16;
                                uint32_t sw = *reinterpret_cast<const uint32_t *>(unit + U.v_scales + blk * 16 + 4 * t);
                                if (part) sw &= __byte_perm(0x0000FF00u, 0, (live & 1) | (live & 2) << 3 | (live & 4) << 6 | (live & 8) << 9);
                                const uint32_t s01 = fp8x2<0>(sw), s23 = fp8x2<1>(sw);
                                // a byte of two tokens' codes of a dim: the even dims, the odd ones
                                constexpr uint32_t LOW = 0x0F0F0F0Fu;
                                const uint32_t e01 = (w[0][y] & LOW) | (w[1][y] << 4 & ~LOW), o01 = (w[0][y] >> 4 & LOW) | (w[1][y] & ~LOW);
                                const uint32_t e23 = (w[2][y] & LOW) | (w[3][y] << 4 & ~LOW), o23 = (w[2][y] >> 4 & LOW) | (w[3][y] & ~LOW);
                                const uint32_t a[4][4] = {
                                    {mul_f16x2(fp4x2<0>(e01), s01), mul_f16x2(fp4x2<0>(o01), s01), mul_f16x2(fp4x2<0>(e23), s23), mul_f16x2(fp4x2<0>(o23), s23)},
                                    {mul_f16x2(fp4x2<1>(e01), s01), mul_f16x2(fp4x2<1>(o01), s01), mul_f16x2(fp4x2<1>(e23), s23), mul_f16x2(fp4x2<1>(o23), s23)},
                                    {mul_f16x2(fp4x2<2>(e01), s01), mul_f16x2(fp4x2<2>(o01), s01), mul_f16x2(fp4x2<2>(e23), s23), mul_f16x2(fp4x2<2>(o23), s23)},
                                    {mul_f16x2(fp4x2<3>(e01), s01), mul_f16x2(fp4x2<3>(o01), s01), mul_f16x2(fp4x2<3>(e23), s23), mul_f16x2(fp4x2<3>(o23), s23)}};
#pragma unroll
                                for (int k = 0; k < 4; ++k)
#pragma unroll
                                    for (int n = 0; n < NT; ++n) mma_f16(o[n][4 * (y0 + y) + k], a[k], pf[n][0], pf[n][1]);
                            } else if constexpr (TYPE == QFP4_CACHE_E4M3) {
                                const uint32_t lo0 = __byte_perm(w[0][y], w[1][y], 0x5140), hi0 = __byte_perm(w[0][y], w[1][y], 0x7362);
                                const uint32_t lo1 = __byte_perm(w[2][y], w[3][y], 0x5140), hi1 = __byte_perm(w[2][y], w[3][y], 0x7362);
                                const uint32_t a0[4] = {fp8x2<0>(lo0), fp8x2<1>(lo0), fp8x2<0>(lo1), fp8x2<1>(lo1)};
                                const uint32_t a1[4] = {fp8x2<0>(hi0), fp8x2<1>(hi0), fp8x2<0>(hi1), fp8x2<1>(hi1)};
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    mma_f16(o[n][2 * (y0 + y)], a0, pf[n][0], pf[n][1]);
                                    mma_f16(o[n][2 * (y0 + y) + 1], a1, pf[n][0], pf[n][1]);
                                }
                            } else {
                                const uint32_t a[4] = {__byte_perm(w[0][y], w[1][y], 0x5410), __byte_perm(w[0][y], w[1][y], 0x7632),
                                                       __byte_perm(w[2][y], w[3][y], 0x5410), __byte_perm(w[2][y], w[3][y], 0x7632)};
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    mma_bf16(o[n][y0 + y], a, pf[n][0], pf[n][1]);
                                    mma_bf16(o[n][y0 + y], a, pl[n][0], pl[n][1]);
                                }
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (to_issue > 0) {
                issue(ahead.head, next, stage);
                ahead.next<TILE>(p);
                if (--to_issue > 0) next = unit_of(ahead);
            }
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1;
            }
        }
        at += seg_n;
        cur.skip<TILE>(p, seg_n);
        if (at < hi) load_q();

        // ---- the warps' results joined: o relative to the CTA's maximum, added up in the warps' order
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], s);
                if (g == 0) s_ml[warp * QUERIES + 8 * n + 2 * t + k] = make_float2(m[n][k], l[n][k]);
            }
        __syncthreads();
        constexpr int TURNS = C::WARPS / C::SUMS;
#pragma unroll
        for (int turn = 0; turn < TURNS; ++turn) {
            if (turn == warp / C::SUMS) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int q = 8 * n + 2 * t + k;
                        float top = -INFINITY;
#pragma unroll
                        for (int w = 0; w < C::WARPS; ++w) top = max_nan(top, s_ml[w * QUERIES + q].x);
                        const float own = TYPE == QFP4_CACHE_E4M3 ? mw[n][k] : m[n][k];
                        const float f = own == -INFINITY ? 0.0f : exp2_fast(own - top);
                        // dims g D / 8 + 2 i and the next
                        float *dst = s_o + (warp % C::SUMS) * C::SUM + q * (D + 4) + g * (D / 8);
#pragma unroll
                        for (int i = 0; i < MTILES; ++i) {
                            float2 v = make_float2(o[n][i][k] * f, o[n][i][2 + k] * f);
                            if (turn > 0) {
                                const float2 old = *reinterpret_cast<const float2 *>(dst + 2 * i);
                                v.x += old.x;
                                v.y += old.y;
                            }
                            *reinterpret_cast<float2 *>(dst + 2 * i) = v;
                        }
                    }
            }
            __syncthreads();
        }
        const bool whole = seg_first == 0 && seg_n == seg_tiles;
        constexpr int PIECE = attn_piece_floats(QUERIES, D);
        float *piece = p.partial + (2 * static_cast<int64_t>(blockIdx.x) + (seg_first == 0)) * PIECE;
        // a thread's query and dims
        constexpr int ALL = C::THREADS / QUERIES, PER = ALL < D / 4 ? ALL : D / 4, DIMS = D / PER;
        static_assert(DIMS % 4 == 0 && PER * QUERIES <= C::THREADS, "a thread has whole fours of one query's dims");
        const bool mine = tid < PER * QUERIES;
        const int q = mine ? tid / PER : 0, d0 = (tid % PER) * 4;
        float m_all = -INFINITY, l_all = 0.0f;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) m_all = max_nan(m_all, s_ml[w * QUERIES + q].x);
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
            const float2 v = s_ml[w * QUERIES + q];
            if (v.x != -INFINITY) l_all += v.y * exp2_fast(v.x - m_all);
        }
        float acc[DIMS];
#pragma unroll
        for (int i = 0; i < DIMS / 4; ++i) {
            const float *src = s_o + q * (D + 4) + d0 + 4 * PER * i;
            float4 v = *reinterpret_cast<const float4 *>(src);
#pragma unroll
            for (int k = 1; k < C::SUMS; ++k) {
                const float4 u = *reinterpret_cast<const float4 *>(src + k * C::SUM);
                v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
            }
            acc[4 * i] = v.x, acc[4 * i + 1] = v.y, acc[4 * i + 2] = v.z, acc[4 * i + 3] = v.w;
        }
        auto write_out = [&](int seq, int hd, int block, float m_, float l_) {
            if (!mine || q >= min(QUERIES, p.group - block * QUERIES)) return;
            // no token: zeros
            const float inv = m_ == -INFINITY ? 0.0f : gs_v / l_;
            const int64_t row = (static_cast<int64_t>(seq) * p.kv_heads + hd) * p.group + block * QUERIES + q;
#pragma unroll
            for (int i = 0; i < DIMS / 4; ++i)
                *reinterpret_cast<uint2 *>(p.out + row * D + d0 + 4 * PER * i) =
                    make_uint2(pack_bf16(acc[4 * i] * inv, acc[4 * i + 1] * inv), pack_bf16(acc[4 * i + 2] * inv, acc[4 * i + 3] * inv));
            if (p.lse && tid % PER == 0) p.lse[row] = m_ == -INFINITY ? -INFINITY : (m_ + log2f(l_)) * 0.693147180559945309f;
        };
        auto write_piece = [&](float *to, float m_, float l_) {
            if (!mine) return;
#pragma unroll
            for (int i = 0; i < DIMS / 4; ++i)
                *reinterpret_cast<float4 *>(to + q * D + d0 + 4 * PER * i) =
                    make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
            if (tid % PER == 0) *reinterpret_cast<float2 *>(to + QUERIES * D + 2 * q) = make_float2(m_, l_);
        };
        if (whole) {
            write_out(b, head, qblock, m_all, l_all);
        } else {
            write_piece(piece, m_all, l_all);
            // CTAs that hold the item's first and last tile
            const int64_t i0 = at - seg_n - seg_first, i1 = i0 + seg_tiles - 1;
            const Shares shares(p, s_total);
            const int64_t c0 = shares.cta_of(i0), c1 = shares.cta_of(i1);
            const int pieces = static_cast<int>(c1 - c0) + 1, size = attn_join_group(pieces);
            const int group = static_cast<int>(blockIdx.x - c0) / size, first = static_cast<int>(c0) + group * size;
            // an item's first group has the counter of its first CTA, the others one of the
            // second row: the last CTA of an item may be the first of the next
            uint32_t *counter = p.counters + (group > 0 ? kAttnMaxCtas : 0) + first;
            // one thread releases the piece for all, who have met at the barrier, and
            // acquires the others' for all who meet at the next
            __syncthreads();
            if (tid == 0) s_last = atom_add_acq_rel_gpu(counter, 1u) + 1 == static_cast<uint32_t>(min(size, pieces - group * size));
            __syncthreads();
            if (s_last && tid == 0) {       // the group's pieces are there: joined when this CTA's own tiles are done
                *counter = 0;
                // a CTA has two items in pieces at most
                s_late[seg_first == 0] = Late{b, head, qblock, static_cast<int>(c0), pieces, first};
            }
        }
        __syncthreads();
        if (at < hi) continue;

        // ---- joins: the pieces come to the rings' place, so many at a time that their
        // loads do not wait for one another
        constexpr int CHUNKS = PIECE / 4, BATCH = C::RING / (PIECE * 4);
        static_assert(PIECE % 4 == 0 && BATCH >= 1, "pieces are copied 16 bytes at a time");
        float *s_pieces = reinterpret_cast<float *>(smem);
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
            const Late w = s_late[which];
            if (w.n == 0) continue;
            const int size = attn_join_group(w.n), groups = (w.n + size - 1) / size;
            // a group's pieces; then, by the CTA that finishes last, the groups'
            int first = w.first, count = min(size, w.c0 + w.n - w.first), step = 1;
#pragma unroll 1
            for (;;) {
                float m_ = -INFINITY, l_ = 0.0f;
#pragma unroll
                for (int i = 0; i < DIMS; ++i) acc[i] = 0.0f;
#pragma unroll 1
                for (int done = 0; done < count; done += BATCH) {
                    const int n = min(BATCH, count - done);
                    for (int i = tid; i < n * CHUNKS; i += C::THREADS) {
                        const int c = i / CHUNKS, cta = first + (done + c) * step;
                        cp_async16(smem_u32(s_pieces + i * 4),
                                   p.partial + (2 * static_cast<int64_t>(cta) + (cta == w.c0)) * PIECE + (i - c * CHUNKS) * 4);
                    }
                    cp_async_wait_all();
                    __syncthreads();
                    float top = m_;
#pragma unroll 8
                    for (int c = 0; c < n; ++c) top = max_nan(top, s_pieces[c * PIECE + QUERIES * D + 2 * q]);
                    const float f0 = m_ == -INFINITY ? 0.0f : exp2_fast(m_ - top);
                    m_ = top;
                    l_ *= f0;
#pragma unroll
                    for (int i = 0; i < DIMS; ++i) acc[i] *= f0;
#pragma unroll 4
                    for (int c = 0; c < n; ++c) {
                        const float *pc = s_pieces + c * PIECE;
                        const float2 ml = *reinterpret_cast<const float2 *>(pc + QUERIES * D + 2 * q);
                        const float f = ml.x == -INFINITY ? 0.0f : exp2_fast(ml.x - top);
                        l_ += ml.y * f;
#pragma unroll
                        for (int i = 0; i < DIMS / 4; ++i) {
                            const float4 v = *reinterpret_cast<const float4 *>(pc + q * D + d0 + 4 * PER * i);
                            acc[4 * i] += v.x * f;
                            acc[4 * i + 1] += v.y * f;
                            acc[4 * i + 2] += v.z * f;
                            acc[4 * i + 3] += v.w * f;
                        }
                    }
                    __syncthreads();
                }
                if (step > 1 || groups == 1) {
                    write_out(w.b, w.head, w.block, m_, l_);
                    break;
                }
                // in the place of the group's first piece, which has been read
                write_piece(p.partial + (2 * static_cast<int64_t>(first) + (first == w.c0)) * PIECE, m_, l_);
                uint32_t *counter = p.counters + 2 * kAttnMaxCtas + w.c0;
                __syncthreads();
                if (tid == 0) s_last = atom_add_acq_rel_gpu(counter, 1u) + 1 == static_cast<uint32_t>(groups);
                __syncthreads();
                if (!s_last) break;
                if (tid == 0) *counter = 0;
                first = w.c0, count = groups, step = size;
            }
        }
    }
    if (dead) {     // copies in flight have time to land before the shared memory goes to another CTA
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) {
        }
    }
}

// CTAs of this kernel that an SM holds, no more than `most`; asked once.
template <int TYPE, int D, int NT, int WARPS>
int attn_per_sm(int most)
{
    static std::atomic<int> known{0};
    int n = known.load(std::memory_order_relaxed);
    if (n == 0) {
        using C = AttnCfg<TYPE, D, NT, WARPS>;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attention_decode_kernel<TYPE, D, NT, WARPS>, C::THREADS,
                                                          C::SMEM) != cudaSuccess ||
            n < 1)
            return 0;
        known.store(n, std::memory_order_relaxed);
    }
    return n < most ? n : most;
}

// The grid is what the GPU holds at once, whatever the lengths, which only the
// device knows: 152 SMs times the CTAs of each, as many as `most` at most.
template <int TYPE, int D, int NT, int WARPS>
int attn_launch_one(const AttnParams &p, int most, cudaStream_t s)
{
    using C = AttnCfg<TYPE, D, NT, WARPS>;
    auto kernel = attention_decode_kernel<TYPE, D, NT, WARPS>;
    const int rc = ensure_smem_attr(reinterpret_cast<const void *>(kernel), C::SMEM);
    if (rc != QFP4_OK) return rc;
    const int n = attn_per_sm<TYPE, D, NT, WARPS>(most);
    if (n == 0) return QFP4_ERR_CUDA;
    return launch_status(launch_pdl(kernel, dim3(152 * n), dim3(C::THREADS), C::SMEM, s, p));
}

// CTAs that an SM takes at most: twice as many, of two warps, for many items (sequences
// x key heads x blocks of queries).
inline bool attn_many(int64_t items, int nt) { return items > (nt == 2 ? 2 : 4) * 152; }
inline int attn_most_per_sm(int64_t items, int nt) { return attn_many(items, nt) ? 8 : 4; }

// Four warps a CTA, up to four CTAs on an SM (three in E4M3 and BF16).  Many items: two
// warps and up to twice as many CTAs, which hide one another's joins (256 ragged sequences up to 300 tokens x 8 heads: NVFP4
// 26.4 us, 29.2 with four; E4M3 32.3, 36.2; up to 2000 tokens 81, 86 and 105, 109; one
// warp 28, 36, 83, 109; 512 items up to 300 tokens 14.4, 13.5; 512 items of 16 query heads
// up to 1000 tokens E4M3 30, 41, and 128 of up to 16384 as long with either).  Few items in NVFP4: eight
// warps, two CTAs on an SM, half as many pieces to join (1 x 4096 tokens x 8 heads 11 us, 16
// with four warps; 1 x 131072 48, 55).
template <int TYPE, int D, int NT>
int attn_launch(const AttnParams &p, cudaStream_t s)
{
    const int64_t items = static_cast<int64_t>(p.B) * p.kv_heads * p.blocks;
    const int most = attn_most_per_sm(items, NT);
    if (attn_many(items, NT)) return attn_launch_one<TYPE, D, NT, 2>(p, most, s);
    if constexpr (TYPE == QFP4_CACHE_NVFP4 && D <= 128) {
        if (items <= 2 * 152) return attn_launch_one<TYPE, D, NT, 8>(p, most, s);
    }
    return attn_launch_one<TYPE, D, NT, 4>(p, most, s);
}

// Of attention_decode_<type>.cu.
int attn_launch_bf16(const AttnParams &p, int D, int nt, cudaStream_t s);
int attn_launch_e4m3(const AttnParams &p, int D, int nt, cudaStream_t s);
int attn_launch_nvfp4(const AttnParams &p, int D, int nt, cudaStream_t s);

// Query heads of a block: those of a group, 8 or 16; 8 where 16 would not fit
// in the registers (D = 256).
inline int attn_tiles(int64_t group, int D) { return group > 8 && D <= 128 ? 2 : 1; }

template <int TYPE>
int attn_launch_type(const AttnParams &p, int D, int nt, cudaStream_t s)
{
    if (D == 64) return nt == 1 ? attn_launch<TYPE, 64, 1>(p, s) : attn_launch<TYPE, 64, 2>(p, s);
    if (D == 128) return nt == 1 ? attn_launch<TYPE, 128, 1>(p, s) : attn_launch<TYPE, 128, 2>(p, s);
    return attn_launch<TYPE, 256, 1>(p, s);
}

}  // namespace qfp4
