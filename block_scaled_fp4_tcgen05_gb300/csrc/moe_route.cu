// moe_route.cu -- expert router: top-k choice, gates, per-expert counts, the
// row order of the experts' product, the balance loss, and its gradient.
//
// With p = softmax(l) per token, c_e the pairs that chose expert e, n the valid
// tokens, P_e = sum_t p_te / n:
//   loss = E / (k n) sum_e c_e P_e
// and, choices held fixed, with s_e = dloss E c_e / (k n^2):
//   dl_i = p_i (s_i - sum_e p_e s_e) + gates' part,
//   gates' part, g = p / sum of the chosen p: g_i (dg_i - sum_j g_j dg_j) at the
//   chosen experts; g = p: [chosen] p_i dg_i - p_i sum_j p_j dg_j.
//
// Forward, two launches (one for few tokens).  route_rows_kernel: CTA c takes a
// contiguous range of tokens.  Instructions bound it, most of them in the k
// rounds of top-k, so where experts are few a round serves several tokens: G
// lanes (4, 8 or 32) share a token, each with up to 16 of its logits in
// registers.  Keys are integers in the order of the logits; a lane keeps its
// best and second best, so a round is a maximum over the G lanes, a vote for
// the lane that holds it and that lane's next best.  A lane adds up its
// experts' p over its tokens in registers.  The CTA's counts and its sum of p
// go to the workspace.
// route_place_kernel: each CTA adds up the counts of all ranges, so it knows
// where each expert's rows begin and how many of them come from earlier
// ranges, and ranks its own pairs in order; one more CTA writes the totals and
// the loss.  All sums run in a fixed order: results repeat bit for bit.
//
// 16384 tokens x 256 experts, top 8, take 21 us (58 with keys searched anew in
// every round and the ranges' counts added one after another), about 12 of
// them in the first kernel at 0.75 of the issue slots; the second is a chain of
// latencies (8 us together for 512 tokens).  64 tokens x 8 experts: 3.9 us in
// one launch.  The gradient reads the logits once more and writes as much:
// 16384 x 256 in 8.5 us (3.9 TB/s), 16384 x 64 BF16 in 4.2 (12.6 and 8.0 with a
// warp per token); its instructions bound it likewise.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "qfp4_common.cuh"

namespace qfp4 {
namespace {

constexpr int kMaxExperts = 256;
constexpr int kMaxTopk = 16;
constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kBackThreads = 256;
constexpr int kMaxRowWarps = 32;            // of the CTAs that read the logits: 16, or 32 where a warp has one token
constexpr int kMaxChunks = 152;             // one CTA on each SM
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;

struct RouteParams {
    const void *logits;         // [T, E] BF16 or fp32
    const uint8_t *valid;       // [T] or NULL
    int64_t T;
    int32_t E, topk, renorm;
    int64_t chunk;              // tokens per CTA
    int32_t *ids;
    float *gates;
    int32_t *counts, *row_offsets, *dest, *src, *n_valid;
    float *mean_prob, *loss;
    // workspace: per chunk, counts [E] (int32), sums of p [E] (fp32); then
    // valid tokens per chunk
    int32_t *ws_counts;         // rows of E4 = E rounded up to 4
    float *ws_prob;             // the same
    int32_t *ws_valid;
};

// Order-preserving key: larger float, larger key.  Adding +0 turns -0 into +0
// and every NaN into the one whose key is above all others.
__device__ __forceinline__ uint32_t sort_key(float v)
{
    const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// The larger one; NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float load_logit(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16 *p) { return __bfloat162float(__ldg(p)); }
__device__ __forceinline__ void store_logit(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v)
{
    for (int d = 16; d > 0; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kFull, v, d));
    return v;
}

// base of exp(l - base): the row's largest logit, 0 for a row with no open
// expert.  A NaN or +inf logit makes base, or a difference with it, and so the
// row's sum, NaN.  exp is 2^(x log2 e) by the hardware's exponential: the
// rounded product costs |x| 2^-24 relative, the exponential 2^-22.
__device__ __forceinline__ float softmax_base(uint32_t top) { return top <= kKeyNegInf ? 0.0f : key_value(top); }

struct RouteShared {
    alignas(16) int32_t counts[kMaxExperts];        // of this range
    int32_t start[kMaxExperts];                     // first row of each expert, all ranges
    int32_t before[kMaxExperts];                    // rows of it that earlier ranges fill
    int32_t total[kMaxExperts];
    union {
        float prob[kMaxRowWarps][kMaxExperts];      // sums of p per warp
        struct {
            int32_t row[kWarps][kMaxExperts];       // counts, then next row, of each warp's pairs
            union {
                int4 part[2][kThreads];             // partial sums over ranges, four experts each
                float4 ppart[kThreads];
            };
        };
    };
    int32_t valid;
    int32_t rows;                                   // rows of all experts
};

// Choices, gates and counts of tokens [t0, t1), and the warps' sums of p; by
// WARPS warps.  G lanes per token, V experts per lane: lane l of the G has
// experts l, l + G, ...
template <typename L, int G, int V, int WARPS>
__device__ __forceinline__ void route_rows(const RouteParams &p, int64_t t0, int64_t t1, RouteShared &sh)
{
    constexpr int kTokens = 32 / G;                     // tokens of a warp at a time
    constexpr int kHold = (kMaxTopk + G - 1) / G;       // choices that a lane keeps: l, l + G, ...
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane % G, first = lane - l;
    float psum[V], ahead[V];
#pragma unroll
    for (int v = 0; v < V; ++v) psum[v] = 0.0f;
    int nvalid = 0;
    auto load_row = [&](int64_t t) {
        const L *row = static_cast<const L *>(p.logits) + t * p.E + l;
#pragma unroll
        for (int v = 0; v < V; ++v) ahead[v] = t < t1 && l + G * v < p.E ? load_logit(row + G * v) : -INFINITY;
    };
    auto group_sum = [](float x) {
#pragma unroll
        for (int d = G / 2; d > 0; d >>= 1) x = __fadd_rn(x, __shfl_xor_sync(kFull, x, d));
        return x;
    };
    load_row(t0 + warp * kTokens + lane / G);
    for (int64_t tw = t0 + warp * kTokens; tw < t1; tw += WARPS * kTokens) {
        const int64_t t = tw + lane / G;
        const bool here = t < t1;
        const bool valid = here && (!p.valid || p.valid[t] != 0);
        if (valid && l == 0) ++nvalid;
        float x[V];
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = __fadd_rn(ahead[v], 0.0f);
        load_row(t + WARPS * kTokens);      // the next tokens' logits come while these are worked on
        // the lane's best and second best key and their places (equal keys: the lowest expert first)
        uint32_t best = 0u, second = 0u;
        int at = 0, then = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t key = sort_key(x[v]);
            const bool b = key > best, c = key > second;
            second = b ? best : c ? key : second;
            then = b ? at : c ? v : then;
            best = b ? key : best;
            at = b ? v : at;
        }
        bool known = true;                      // second is the lane's next best
        auto group_max = [](uint32_t k) {
            if constexpr (G == 32) {
                k = __reduce_max_sync(kFull, k);
            } else {
#pragma unroll
                for (int d = G / 2; d > 0; d >>= 1) k = max(k, __shfl_xor_sync(kFull, k, d));
            }
            return k;
        };
        uint32_t top = group_max(best);
        const float base = softmax_base(top);
        float sum = 0.0f;
        {
            float e[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                e[v] = __expf(x[v] - base);     // (0 where there is no expert: its logit is -inf)
                sum += e[v];
            }
            sum = group_sum(sum);
            // tokens that are not valid add nothing, whatever their logits hold
            const float inv = !valid || sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
#pragma unroll
            for (int v = 0; v < V; ++v) psum[v] = valid ? fmaf(e[v], inv, psum[v]) : psum[v];
            sum = inv;
        }
        int32_t my_id[kHold];
        uint32_t my_key[kHold];
#pragma unroll
        for (int h = 0; h < kHold; ++h) {
            my_id[h] = -1;
            my_key[h] = 0u;
#pragma unroll 1
            for (int i = 0; i < G; ++i) {
                if (h * G + i >= p.topk) break;
                if (h + i > 0) top = group_max(best);
                const bool open = valid && top > kKeyNegInf;
                if (G == 32 && !open) break;        // (the whole warp's token)
                uint32_t who = __ballot_sync(kFull, best == top) >> first & (kFull >> (32 - G));
                uint32_t e = l + G * at;
                const bool several = open && (who & (who - 1u)) != 0;
                if (G == 32 ? several : __any_sync(kFull, several)) {
                    // equal keys on several lanes: the lowest expert
                    uint32_t low = best == top ? e : 0xFFFFFFFFu;
#pragma unroll
                    for (int d = G / 2; d > 0; d >>= 1) low = min(low, __shfl_xor_sync(kFull, low, d));
                    who = 1u << (low % G);
                }
                const int src = __ffs(who) - 1;
                e = __shfl_sync(kFull, e, src, G);
                if (l == i && open) {
                    my_id[h] = static_cast<int32_t>(e);
                    my_key[h] = top;
                }
                const bool mine = l == src;
                if (mine && !known) {           // the lane's third and later: the largest after (best, at)
                    second = 0u;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const uint32_t key = sort_key(x[v]);
                        if ((key < best || (key == best && v > at)) && key > second) {
                            second = key;
                            then = v;
                        }
                    }
                }
                best = mine ? second : best;
                at = mine ? then : at;
                known = known && !mine;
            }
        }
        // the chosen experts' terms, and their sum where the gates are shares of it
        float my_x[kHold], scale = 0.0f;
#pragma unroll
        for (int h = 0; h < kHold; ++h) {
            my_x[h] = my_id[h] >= 0 ? __expf(key_value(my_key[h]) - base) : 0.0f;
            scale = __fadd_rn(scale, my_x[h]);
        }
        scale = p.renorm ? group_sum(scale) : 0.0f;
        scale = !p.renorm ? sum : scale == 0.0f ? 0.0f : __fdiv_rn(1.0f, scale);
#pragma unroll
        for (int h = 0; h < kHold; ++h) {
            const int j = h * G + l;
            if (here && j < p.topk) {
                p.ids[t * p.topk + j] = my_id[h];
                p.gates[t * p.topk + j] = my_x[h] * scale;
                if (my_id[h] >= 0) atomicAdd(&sh.counts[my_id[h]], 1);
            }
        }
    }
    // the warp's tokens side by side, in order
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int d = G; d < 32; d <<= 1) psum[v] = __fadd_rn(psum[v], __shfl_xor_sync(kFull, psum[v], d));
        if (lane < G && l + G * v < kMaxExperts) sh.prob[warp][l + G * v] = psum[v];
    }
    nvalid = __reduce_add_sync(kFull, nvalid);
    if (lane == 0) atomicAdd(&sh.valid, nvalid);
}

// Sum of expert e's p over the warps of this CTA.
template <int WARPS>
__device__ __forceinline__ float route_prob(const RouteShared &sh, int e)
{
    float s = sh.prob[0][e];
#pragma unroll 8
    for (int w = 1; w < WARPS; ++w) s = __fadd_rn(s, sh.prob[w][e]);
    return s;
}

// First row of each expert from the totals; by the first warp.
__device__ __forceinline__ void route_starts(const RouteParams &p, RouteShared &sh)
{
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < 32) {
        int32_t n[kMaxExperts / 32], mine = 0;
#pragma unroll
        for (int i = 0; i < kMaxExperts / 32; ++i) {
            const int e = lane * (kMaxExperts / 32) + i;
            n[i] = mine;
            mine += e < p.E ? sh.total[e] : 0;
        }
        int32_t up = mine;
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(kFull, up, d);
            if (lane >= d) up += o;
        }
#pragma unroll
        for (int i = 0; i < kMaxExperts / 32; ++i) {
            const int e = lane * (kMaxExperts / 32) + i;
            if (e < p.E) sh.start[e] = up - mine + n[i];
        }
        if (lane == 31) sh.rows = up;
    }
}

// Rows of the pairs of tokens [t0, t1): after the experts' starts and the rows
// that earlier ranges fill, in the pairs' order.  All threads; sh.row is zero.
__device__ __forceinline__ void route_place(const RouteParams &p, int64_t t0, int64_t t1, RouteShared &sh)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t f0 = t0 * p.topk, f1 = t1 * p.topk;
    const int64_t per_warp = ((f1 - f0 + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int64_t w0 = min(f1, f0 + warp * per_warp), w1 = min(f1, w0 + per_warp);
    // the first pairs' experts stay in registers for the second pass
    constexpr int kKeep = 4;
    int32_t kept[kKeep];
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
        const int64_t f = w0 + 32 * i + lane;
        kept[i] = f < w1 ? __ldcg(p.ids + f) : -1;
    }
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
        if (kept[i] >= 0) atomicAdd(&sh.row[warp][kept[i]], 1);
    for (int64_t f = w0 + 32 * kKeep + lane; f < w1; f += 32) {
        const int32_t e = __ldcg(p.ids + f);
        if (e >= 0) atomicAdd(&sh.row[warp][e], 1);
    }
    __syncthreads();
    for (int e = tid; e < p.E; e += kThreads) {
        int32_t at = sh.start[e] + sh.before[e];
#pragma unroll 8
        for (int w = 0; w < kWarps; ++w) {
            const int32_t n = sh.row[w][e];
            sh.row[w][e] = at;
            at += n;
        }
    }
    __syncthreads();
    auto place = [&](int64_t f, int32_t e) {
        const uint32_t same = __match_any_sync(kFull, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        int32_t row = -1;
        if (e >= 0) row = sh.row[warp][e] + rank;
        __syncwarp();
        if (e >= 0 && rank == 0) sh.row[warp][e] += __popc(same);
        __syncwarp();
        if (f + lane < w1) {
            p.dest[f + lane] = row;
            if (row >= 0) p.src[row] = static_cast<int32_t>(static_cast<uint32_t>(f + lane) / static_cast<uint32_t>(p.topk));
        }
    };
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
        if (w0 + 32 * i < w1) place(w0 + 32 * i, kept[i]);
    for (int64_t f = w0 + 32 * kKeep; f < w1; f += 32) place(f, f + lane < w1 ? __ldcg(p.ids + f + lane) : -1);
}

// Totals, offsets, mean p and loss; prob = sum of expert tid's p over all tokens.
__device__ __forceinline__ void route_totals(const RouteParams &p, RouteShared &sh, int32_t valid, float prob)
{
    const int tid = threadIdx.x;
    const float n = static_cast<float>(max(valid, 1));
    float s = 0.0f;
    if (tid < p.E) {
        const float mean = __fdiv_rn(prob, n);
        p.mean_prob[tid] = mean;
        p.counts[tid] = sh.total[tid];
        p.row_offsets[tid] = sh.start[tid];
        s = mean * static_cast<float>(sh.total[tid]);
    }
    __shared__ float part[kMaxExperts / 32];
    if (tid < kMaxExperts) {
        s = warp_sum(s);
        if ((tid & 31) == 0) part[tid >> 5] = s;
    }
    __syncthreads();
    if (tid == 0) {
        float sum = part[0];
#pragma unroll
        for (int w = 1; w < kMaxExperts / 32; ++w) sum = __fadd_rn(sum, part[w]);
        p.loss[0] = sum * __fdiv_rn(static_cast<float>(p.E), static_cast<float>(p.topk) * n);
        p.row_offsets[p.E] = sh.rows;
        p.n_valid[0] = valid;
    }
}

template <typename L, int G, int V, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 1)
route_rows_kernel(const RouteParams p)
{
    __shared__ RouteShared sh;
    const int tid = threadIdx.x;
    if (tid < kMaxExperts) sh.counts[tid] = 0;
    if (tid == 0) sh.valid = 0;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t0 = min(p.T, blockIdx.x * p.chunk), t1 = min(p.T, t0 + p.chunk);
    route_rows<L, G, V, WARPS>(p, t0, t1, sh);
    __syncthreads();
    if (tid < p.E) p.ws_prob[blockIdx.x * ((p.E + 3) / 4 * 4) + tid] = route_prob<WARPS>(sh, tid);
    if (tid < (p.E + 3) / 4)
        reinterpret_cast<int4 *>(p.ws_counts)[blockIdx.x * ((p.E + 3) / 4) + tid] = reinterpret_cast<const int4 *>(sh.counts)[tid];
    if (tid == 0) p.ws_valid[blockIdx.x] = sh.valid;
}

// CTA c < chunks places range c; the last one writes the totals.
__global__ void __launch_bounds__(kThreads)
route_place_kernel(const RouteParams p, int chunks)
{
    __shared__ RouteShared sh;
    const int tid = threadIdx.x;
    const bool totals = static_cast<int>(blockIdx.x) == chunks;
    // four experts' counts are added up by `parts` threads, up to 19 ranges each (E > 128; fewer experts, fewer)
    const int e4 = (p.E + 3) / 4;
    const int width = e4 <= 8 ? 8 : e4 <= 16 ? 16 : e4 <= 32 ? 32 : 64;
    const int parts = kThreads / width, part = tid / width, e = tid % width;
    for (int f = tid; f < kWarps * kMaxExperts; f += kThreads) (&sh.row[0][0])[f] = 0;
    pdl_wait();
    pdl_launch_dependents();
    int4 before = make_int4(0, 0, 0, 0), total = make_int4(0, 0, 0, 0);
    float4 prob = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    constexpr int kLoads = (kMaxChunks + 7) / 8;                // (8 parts at 64 threads of width)
    if (totals && e < e4) {
        float4 n[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int c = part + i * parts;
            n[i] = c < chunks ? __ldcg(reinterpret_cast<const float4 *>(p.ws_prob) + c * e4 + e)
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            prob.x = __fadd_rn(prob.x, n[i].x);
            prob.y = __fadd_rn(prob.y, n[i].y);
            prob.z = __fadd_rn(prob.z, n[i].z);
            prob.w = __fadd_rn(prob.w, n[i].w);
        }
    }
    if (e < e4) {
        int4 n[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int c = part + i * parts;
            n[i] = c < chunks ? __ldcg(reinterpret_cast<const int4 *>(p.ws_counts) + c * e4 + e) : make_int4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (part + i * parts < static_cast<int>(blockIdx.x)) {
                before.x += n[i].x; before.y += n[i].y; before.z += n[i].z; before.w += n[i].w;
            }
            total.x += n[i].x; total.y += n[i].y; total.z += n[i].z; total.w += n[i].w;
        }
    }
    sh.part[0][tid] = before;
    sh.part[1][tid] = total;
    __syncthreads();
    if (tid < p.E) {
        int32_t b = 0, n = 0;
        const int32_t *pb = reinterpret_cast<const int32_t *>(sh.part[0]) + tid;
        const int32_t *pn = reinterpret_cast<const int32_t *>(sh.part[1]) + tid;
#pragma unroll 16
        for (int i = 0; i < parts; ++i) {
            b += pb[i * width * 4];
            n += pn[i * width * 4];
        }
        sh.before[tid] = b;
        sh.total[tid] = n;
    }
    __syncthreads();
    route_starts(p, sh);
    __syncthreads();
    // rows that no pair takes
    const int64_t pairs = p.T * p.topk;
    for (int64_t r = sh.rows + static_cast<int64_t>(blockIdx.x) * kThreads + tid; r < pairs;
         r += static_cast<int64_t>(gridDim.x) * kThreads)
        p.src[r] = -1;
    if (!totals) {
        const int64_t t0 = min(p.T, blockIdx.x * p.chunk);
        route_place(p, t0, min(p.T, t0 + p.chunk), sh);
        return;
    }
    __syncthreads();
    sh.ppart[tid] = prob;
    if (tid < 32) {
        int32_t n = 0;
        for (int c = tid; c < chunks; c += 32) n += __ldcg(p.ws_valid + c);
        n = __reduce_add_sync(kFull, n);
        if (tid == 0) sh.valid = n;
    }
    __syncthreads();
    float s = 0.0f;
    if (tid < p.E) {
        const float *pp = reinterpret_cast<const float *>(sh.ppart) + tid;
#pragma unroll 8
        for (int i = 0; i < parts; ++i) s = __fadd_rn(s, pp[i * width * 4]);
    }
    route_totals(p, sh, sh.valid, s);
}

// Few tokens: the whole of it in one CTA.
template <typename L, int G, int V>
__global__ void __launch_bounds__(kThreads, 1)
route_one_kernel(const RouteParams p)
{
    __shared__ RouteShared sh;
    const int tid = threadIdx.x;
    if (tid < kMaxExperts) {
        sh.counts[tid] = 0;
        sh.before[tid] = 0;
    }
    if (tid == 0) sh.valid = 0;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    route_rows<L, G, V, kWarps>(p, 0, p.T, sh);
    __syncthreads();
    float prob = 0.0f;
    if (tid < p.E) {
        prob = route_prob<kWarps>(sh, tid);
        sh.total[tid] = sh.counts[tid];
    }
    __syncthreads();
    for (int f = tid; f < kWarps * kMaxExperts; f += kThreads) (&sh.row[0][0])[f] = 0;
    route_starts(p, sh);
    __syncthreads();
    for (int64_t r = sh.rows + tid; r < p.T * p.topk; r += kThreads) p.src[r] = -1;
    route_place(p, 0, p.T, sh);     // (the ids it reads were written before the barriers above)
    route_totals(p, sh, sh.valid, prob);
}

struct BackParams {
    const void *logits;
    const uint8_t *valid;
    int64_t T;
    int32_t E, topk, renorm;
    const int32_t *ids, *counts, *n_valid;
    const float *dgates, *dloss;
    void *dlogits;
};

// G lanes per token, V experts per lane, in runs of P (pairs of BF16 logits
// move as one word: 16384 x 64 in 4.2 us, 4.6 one by one; not for an odd E,
// whose rows are not aligned to them).  The chosen experts' elements are
// written twice: with the others, then by the lane that holds the choice and
// knows its p.  Adding the gates' part to the owner's register instead takes
// top-k rounds of V comparisons.
template <typename L, int G, int V, int P>
__global__ void __launch_bounds__(kBackThreads)
route_backward_kernel(const BackParams p)
{
    constexpr int kTokens = 32 / G;
    constexpr int kHold = (kMaxTopk + G - 1) / G;
    __shared__ float share[kMaxExperts];        // s_e
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane % G;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kBackThreads / 32) * kTokens;
    int64_t tw = (static_cast<int64_t>(blockIdx.x) * (kBackThreads / 32) + warp) * kTokens;
    pdl_wait();
    pdl_launch_dependents();
    float x[V];
    bool here, valid;
    int64_t t;
    auto load_row = [&]() {
        t = tw + lane / G;
        here = t < p.T;
        valid = here && (!p.valid || p.valid[t] != 0);
        const L *row = static_cast<const L *>(p.logits) + t * p.E + l * P;
#pragma unroll
        for (int v = 0; v < V; v += P) {
            const bool open = valid && l * P + G * v < p.E;
            if constexpr (P == 2) {
                const float2 two = open ? __bfloat1622float2(__ldg(reinterpret_cast<const __nv_bfloat162 *>(row + G * v)))
                                        : make_float2(-INFINITY, -INFINITY);
                x[v] = two.x;
                x[v + 1] = two.y;
            } else {
                x[v] = open ? load_logit(row + G * v) : -INFINITY;
            }
        }
    };
    load_row();
    {
        // s_e = dloss E c_e / (k n^2)
        const float n = static_cast<float>(max(p.n_valid[0], 1));
        const float f = p.dloss ? __fdiv_rn(__fdiv_rn(p.dloss[0] * static_cast<float>(p.E), n), static_cast<float>(p.topk) * n) : 0.0f;
        for (int e = threadIdx.x; e < kMaxExperts; e += kBackThreads)
            share[e] = e < p.E ? f * static_cast<float>(p.counts[e]) : 0.0f;
    }
    __syncthreads();
    float s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = share[l * P + G * (v / P * P) + v % P];
    auto group_sum = [](float a) {
#pragma unroll
        for (int d = G / 2; d > 0; d >>= 1) a = __fadd_rn(a, __shfl_xor_sync(kFull, a, d));
        return a;
    };
    for (; tw < p.T; tw += stride, load_row()) {
        // choices l, l + G, ... of the token
        int32_t id[kHold];
        float dg[kHold], chosen[kHold];
#pragma unroll
        for (int h = 0; h < kHold; ++h) {
            const int j = h * G + l;
            id[h] = valid && p.dgates && j < p.topk ? p.ids[t * p.topk + j] : -1;
            if (id[h] >= p.E) id[h] = -1;
            dg[h] = id[h] >= 0 ? p.dgates[t * p.topk + j] : 0.0f;
            chosen[h] = id[h] >= 0 ? load_logit(static_cast<const L *>(p.logits) + t * p.E + id[h]) : -INFINITY;
        }
        float top = x[0];
#pragma unroll
        for (int v = 1; v < V; ++v) top = max_nan(top, x[v]);
        uint32_t best = sort_key(top);
        if constexpr (G == 32) {
            best = __reduce_max_sync(kFull, best);
        } else {
#pragma unroll
            for (int d = G / 2; d > 0; d >>= 1) best = max(best, __shfl_xor_sync(kFull, best, d));
        }
        const float base = softmax_base(best);
        float sum = 0.0f, dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] = __expf(x[v] - base);         // (0 where there is no expert)
            sum += x[v];
        }
        sum = group_sum(sum);
        const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] *= inv;
            dot = fmaf(x[v], s[v], dot);
        }
        dot = group_sum(dot);
        if (p.dgates) {
            float total = 0.0f, gd = 0.0f, g[kHold];
#pragma unroll
            for (int h = 0; h < kHold; ++h) {
                chosen[h] = __expf(chosen[h] - base) * inv;
                total = __fadd_rn(total, id[h] >= 0 ? chosen[h] : 0.0f);
            }
            if (p.renorm) total = group_sum(total);
#pragma unroll
            for (int h = 0; h < kHold; ++h) {
                g[h] = id[h] < 0 ? 0.0f : !p.renorm ? chosen[h] : total == 0.0f ? 0.0f : __fdiv_rn(chosen[h], total);
                gd = fmaf(g[h], dg[h], gd);
            }
            gd = group_sum(gd);
            if (!p.renorm) dot += gd;
#pragma unroll
            for (int h = 0; h < kHold; ++h) dg[h] = p.renorm ? g[h] * (dg[h] - gd) : g[h] * dg[h];
        }
        L *out = static_cast<L *>(p.dlogits) + t * p.E;
#pragma unroll
        for (int v = 0; v < V; v += P) {
            if (!here || l * P + G * v >= p.E) continue;
            const float a = valid ? fmaf(x[v], s[v] - dot, 0.0f) : 0.0f;
            if constexpr (P == 2)
                *reinterpret_cast<__nv_bfloat162 *>(out + l * P + G * v) =
                    __floats2bfloat162_rn(a, valid ? fmaf(x[v + 1], s[v + 1] - dot, 0.0f) : 0.0f);
            else
                store_logit(out + l + G * v, a);
        }
        if (p.dgates) {
            __syncwarp();
#pragma unroll
            for (int h = 0; h < kHold; ++h)
                if (id[h] >= 0) store_logit(out + id[h], fmaf(chosen[h], share[id[h]] - dot, dg[h]));
        }
    }
}

template <typename L, int G, int V>
int launch_route(const RouteParams &p, int chunks, cudaStream_t s)
{
    constexpr int W = G == 32 ? 32 : 16;
    // one CTA while each warp has two rounds of tokens at most
    if (p.T <= 2 * kWarps * (32 / G)) return launch_status(launch_pdl(route_one_kernel<L, G, V>, dim3(1), dim3(kThreads), 0, s, p));
    const int rc = launch_status(launch_pdl(route_rows_kernel<L, G, V, W>, dim3(chunks), dim3(32 * W), 0, s, p));
    if (rc != QFP4_OK) return rc;
    return launch_status(launch_pdl(route_place_kernel, dim3(chunks + 1), dim3(kThreads), 0, s, p, chunks));
}

template <typename L>
int launch_forward(const RouteParams &p, int chunks, cudaStream_t s)
{
    if (p.E <= 16) return launch_route<L, 4, 4>(p, chunks, s);
    if (p.E <= 32) return launch_route<L, 4, 8>(p, chunks, s);
    if (p.E <= 64) return launch_route<L, 4, 16>(p, chunks, s);
    if (p.E <= 128) return launch_route<L, 8, 16>(p, chunks, s);
    return launch_route<L, 32, 8>(p, chunks, s);
}

template <typename L, int G, int V>
int launch_back_width(const BackParams &p, cudaStream_t s)
{
    const int64_t tokens = kBackThreads / G;
    const int64_t want = (p.T + tokens - 1) / tokens, most = static_cast<int64_t>(kMaxChunks) * (2048 / kBackThreads);
    const dim3 g(static_cast<unsigned>(want < most ? want : most)), b(kBackThreads);
    if constexpr (sizeof(L) == 2)
        if (p.E % 2 == 0) return launch_status(launch_pdl(route_backward_kernel<L, G, V, 2>, g, b, 0, s, p));
    return launch_status(launch_pdl(route_backward_kernel<L, G, V, 1>, g, b, 0, s, p));
}

template <typename L>
int launch_back(const BackParams &p, cudaStream_t s)
{
    if (p.E <= 16) return launch_back_width<L, 4, 4>(p, s);
    if (p.E <= 32) return launch_back_width<L, 4, 8>(p, s);
    if (p.E <= 64) return launch_back_width<L, 8, 8>(p, s);
    if (p.E <= 128) return launch_back_width<L, 16, 8>(p, s);
    return launch_back_width<L, 32, 8>(p, s);
}

bool sizes_ok(int64_t T, int64_t E, int64_t topk)
{
    return E <= kMaxExperts && topk <= kMaxTopk && topk <= E && T <= INT32_MAX / topk;
}

// Ranges of tokens: 16 each, or more where that would make over kMaxChunks of them.
int64_t chunk_count(int64_t T)
{
    const int64_t n = (T + kWarps - 1) / kWarps;
    return n < 1 ? 1 : n > kMaxChunks ? kMaxChunks : n;
}

}  // namespace
}  // namespace qfp4

using namespace qfp4;

extern "C" size_t qfp4_moe_route_workspace_bytes(int64_t T, int64_t E, int64_t topk)
{
    if (T < 0 || E < 1 || topk < 1 || !sizes_ok(T, E, topk)) return 0;
    const size_t chunks = static_cast<size_t>(chunk_count(T));
    const size_t E4 = static_cast<size_t>((E + 3) / 4 * 4);
    return chunks * E4 * 8 + chunks * 4;
}

extern "C" int qfp4_moe_route(int logits_type, const void *logits, int64_t T, int64_t E, int64_t topk,
                              const uint8_t *valid, int renorm, int32_t *ids, float *gates, int32_t *counts,
                              int32_t *row_offsets, int32_t *dest, int32_t *src, int32_t *n_valid, float *mean_prob,
                              float *loss, void *workspace, size_t ws_bytes, void *stream)
{
    if ((logits_type != QFP4_BF16 && logits_type != QFP4_FP32) || T < 0 || E < 1 || topk < 1)
        return QFP4_ERR_INVALID_ARG;
    if (!sizes_ok(T, E, topk)) return QFP4_ERR_UNSUPPORTED;
    if (!counts || !row_offsets || !n_valid || !mean_prob || !loss || !workspace) return QFP4_ERR_INVALID_ARG;
    if (T > 0 && (!logits || !ids || !gates || !dest || !src)) return QFP4_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned4(ids) || !aligned4(gates) || !aligned4(counts) || !aligned4(row_offsets) ||
        !aligned4(dest) || !aligned4(src) || !aligned4(n_valid) || !aligned4(mean_prob) || !aligned4(loss) ||
        !aligned16(workspace))
        return QFP4_ERR_MISALIGNED;
    if (ws_bytes < qfp4_moe_route_workspace_bytes(T, E, topk)) return QFP4_ERR_WORKSPACE;
    const int64_t chunks = chunk_count(T);
    RouteParams p{logits, valid, T, static_cast<int32_t>(E), static_cast<int32_t>(topk), renorm ? 1 : 0,
                  (T + chunks - 1) / chunks, ids, gates, counts, row_offsets, dest, src, n_valid, mean_prob, loss};
    p.ws_counts = static_cast<int32_t *>(workspace);
    p.ws_prob = reinterpret_cast<float *>(p.ws_counts + chunks * ((E + 3) / 4 * 4));
    p.ws_valid = reinterpret_cast<int32_t *>(p.ws_prob + chunks * ((E + 3) / 4 * 4));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return logits_type == QFP4_BF16 ? launch_forward<__nv_bfloat16>(p, static_cast<int>(chunks), s)
                                    : launch_forward<float>(p, static_cast<int>(chunks), s);
}

extern "C" int qfp4_moe_route_backward(int logits_type, const void *logits, int64_t T, int64_t E, int64_t topk,
                                       const uint8_t *valid, int renorm, const int32_t *ids, const int32_t *counts,
                                       const int32_t *n_valid, const float *dgates, const float *dloss,
                                       void *dlogits, void *stream)
{
    if ((logits_type != QFP4_BF16 && logits_type != QFP4_FP32) || T < 0 || E < 1 || topk < 1)
        return QFP4_ERR_INVALID_ARG;
    if (!sizes_ok(T, E, topk)) return QFP4_ERR_UNSUPPORTED;
    if (T == 0) return QFP4_OK;
    if (!logits || !ids || !counts || !n_valid || !dlogits) return QFP4_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned4(ids) || !aligned4(counts) || !aligned4(n_valid) || !aligned4(dgates) ||
        !aligned4(dloss) || !aligned16(dlogits))
        return QFP4_ERR_MISALIGNED;
    const BackParams p{logits, valid, T, static_cast<int32_t>(E), static_cast<int32_t>(topk), renorm ? 1 : 0,
                       ids, counts, n_valid, dgates, dloss, dlogits};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return logits_type == QFP4_BF16 ? launch_back<__nv_bfloat16>(p, s) : launch_back<float>(p, s);
}
