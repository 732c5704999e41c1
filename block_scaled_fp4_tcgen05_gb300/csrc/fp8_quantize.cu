// fp8_quantize.cu -- BF16 -> 8-bit floating point codes (E4M3 / E5M2) with one
// fp32 scale per 128 elements: along the rows (the operand of a forward
// product), along the columns and transposed (the operand of a weight
// gradient), gathered into expert order, and per 128 x 128 block (weights).
//
// Per block, with top the type's largest magnitude and a = max(max|x|, 2^-100):
//   s = a / top (or the smallest power of two not below it),
//   code = RNE(x * top / a) (or x / s), saturating.
// 2^-100 keeps both quotients and the scale normal numbers, so a block of
// zeros needs no case of its own.
//
// One CTA takes a tile of 128 rows x 128 columns (rows alone: 32 rows, so that
// few rows still spread over the SMs).  A thread holds R consecutive rows of
// eight columns in registers: X is read once however many outputs are asked
// for.  A row's amax is exchanged over the 16 threads of the row, a column's
// taken over the rows a thread holds, then over the CTA through shared memory,
// and each scale is computed once or twice, not by every thread that needs it.
// The transposed codes go through a shared-memory tile so that both outputs
// leave in whole 128-byte lines.
//
// HBM-bound: 2 bytes read and 1 written per element and direction.  16384 x
// 4096 in both directions takes 49 us (5.5 TB/s, 0.82 of the copy bandwidth;
// 90 with every thread computing its scales, 60 without packed BF16 maxima and
// with two CTAs per SM instead of three), a 14336 x 4096 weight with its
// transpose 37 us (6.3 TB/s, 0.93).  Tiles of 512 threads with four rows each
// are slower (53 and 41 us), grouped ones too: 8 groups of 1024 rows x 4096 take
// 34 us in both directions and 21 along the columns alone (52 and 27).  16384 x
// 4096 takes 34 us along the rows alone (6.1 TB/s) and 39 along the columns (5.3).
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "qfp4_common.cuh"
#include "sm103_ptx.cuh"

namespace qfp4 {

__device__ uint32_t g_status_fp8_quant = 0;

int status_word_fp8_quant(uint32_t **word) { return status_word(g_status_fp8_quant, word); }

namespace {

constexpr float kFloor = 0x1p-100f;

struct QuantParams {
    const uint4 *X;             // [X_rows, K] BF16, 8 per uint4
    const int32_t *row_index;   // [M] or NULL
    int64_t X_rows;
    int32_t M, K;
    int32_t Mt;                 // ceil16(M): row length of Q_t
    int32_t tiles_k;            // 128-column tiles: ceil(K / 128)
    uint8_t *Q, *Q_t;
    float *SF, *SF_t;
    const int32_t *row_offsets; // grouped: DEVICE [groups + 1]
    int32_t groups;
};

constexpr int kMaxGroups = 256;

template <int TYPE> struct Fp8;
template <> struct Fp8<QFP4_E4M3> { static constexpr float top = 448.0f; };
template <> struct Fp8<QFP4_E5M2> { static constexpr float top = 57344.0f; };

// codes of lo (low byte) and hi (high byte), nearest even, saturating, NaN kept
template <int TYPE>
__device__ __forceinline__ uint32_t encode2(float lo, float hi)
{
    uint16_t r;
    if (TYPE == QFP4_E4M3) asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

struct Scale {
    float s;        // what a code stands for
    float inv;      // what an element is multiplied by
};

template <int TYPE, bool POW2>
__device__ __forceinline__ Scale block_scale(float amax)
{
    const float a = fmaxf(amax, kFloor);
    const float t = __fdiv_rn(a, Fp8<TYPE>::top);
    if (!POW2) return {t, __fdiv_rn(Fp8<TYPE>::top, a)};
    // t is normal (or inf): the power of two not below it by its exponent field
    const uint32_t u = __float_as_uint(t);
    const uint32_t e = (u >> 23) + ((u & 0x7FFFFFu) != 0 ? 1u : 0u);
    return {__uint_as_float(e << 23), e >= 254u ? 0.0f : __uint_as_float((254u - e) << 23)};
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

enum { kRows = 1, kCols = 2, kBlock = 4 };

// R rows per thread.  Thread 16 i + c holds rows R i .. R i + R - 1 and columns
// 8 c .. 8 c + 7 of the tile: 128 rows, or the 16 R of 256 threads for rows alone.
// WHAT: kRows and / or kCols, or kBlock with or without kCols.
template <int WHAT, int R>
struct QuantCfg {
    static constexpr int ROWS = WHAT == kRows ? 16 * R : 128;
    static constexpr int THREADS = 16 * (ROWS / R);
    // resident CTAs per SM that the registers are sized for
    static constexpr int CTAS = (WHAT == kRows ? 1536 : 768) / THREADS;
};

// GROUPED: every group's rows begin a row tile of their own (WHAT has kCols).
template <int TYPE, bool POW2, int WHAT, int R, bool GROUPED>
__global__ void __launch_bounds__(QuantCfg<WHAT, R>::THREADS, QuantCfg<WHAT, R>::CTAS)
fp8_quantize_kernel(const QuantParams p)
{
    constexpr bool ROWS = (WHAT & kRows) != 0, COLS = (WHAT & kCols) != 0, BLOCK = (WHAT & kBlock) != 0;
    constexpr int TR = QuantCfg<WHAT, R>::ROWS, THREADS = QuantCfg<WHAT, R>::THREADS, WARPS = THREADS / 32;
    static_assert(R == 2 || R == 8, "the exchange between rows halves them");
    static_assert(!GROUPED || (COLS && !BLOCK), "groups matter to blocks of rows only");
    __shared__ int32_t s_rows[GROUPED ? 2 : 1];
    // transposed tile: 128 columns of 32 words of four rows' codes.  Word u of
    // column 8 c + j lies at u ^ 2 c: the writes of a warp (16 values of c, two
    // neighbouring words) and the reads (16 bytes of four columns) then spread
    // over all banks.
    __shared__ __align__(16) uint32_t s_t[COLS ? 128 * 32 : 4];
    __shared__ __align__(16) float s_amax[COLS && !BLOCK ? WARPS * 128 : WARPS];

    const int tid = threadIdx.x;
    const int c = tid & 15, i = tid >> 4, warp = tid >> 5, lane = tid & 31;
    const int32_t mtile = blockIdx.x / p.tiles_k, kblock = blockIdx.x - mtile * p.tiles_k;
    int32_t m0 = mtile * TR, m_end = p.M;
    const int32_t col = kblock * 128 + 8 * c;
    const bool col_ok = col < p.K;          // K % 16 == 0: all eight or none
    const int64_t group = blockIdx.y;       // kBlock: one matrix per group
    const int64_t mat = BLOCK ? group * p.M * static_cast<int64_t>(p.K) : 0;

    pdl_wait();
    pdl_launch_dependents();

    if (GROUPED) {
        // the group whose row tiles this one is among: a thread per group, and
        // a running sum over the CTA's warps
        __shared__ int32_t s_sum[WARPS];
        static_assert(!GROUPED || THREADS >= kMaxGroups, "a thread per group");
        const bool mine = tid < p.groups;
        const int32_t lo = mine ? p.row_offsets[tid] : 0, hi = mine ? p.row_offsets[tid + 1] : 0;
        const bool bad = __syncthreads_or(mine && ((tid == 0 && lo != 0) || hi < lo || (tid == p.groups - 1 && hi > p.M)));
        if (bad) {
            if (blockIdx.x == 0 && tid == 0) atomicOr(&g_status_fp8_quant, static_cast<uint32_t>(kStatusBadGroup));
            return;
        }
        const int32_t n = (hi - lo + 127) / 128;
        int32_t up = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, up, d);
            if (lane >= d) up += o;
        }
        if (lane == 31) s_sum[warp] = up;
        if (tid == 0) s_rows[0] = s_rows[1] = 0;
        __syncthreads();
        for (int w = 0; w < warp; ++w) up += s_sum[w];
        if (mtile >= up - n && mtile < up) {
            s_rows[0] = lo + (mtile - (up - n)) * 128;
            s_rows[1] = hi;
        }
        __syncthreads();
        m0 = s_rows[0];
        m_end = s_rows[1];
        if (m0 >= m_end) return;        // beyond the last group's tiles
    }
    m0 += R * i;

    uint4 x[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int32_t m = m0 + r;
        int64_t row = m;
        bool ok = col_ok && m < m_end;
        if (!BLOCK && p.row_index && ok) {
            row = p.row_index[m];
            if (row >= p.X_rows) {
                if (c == 0) atomicOr(&g_status_fp8_quant, static_cast<uint32_t>(kStatusBadGroup));
                ok = false;
            }
            if (row < 0) ok = false;
        }
        x[r] = make_uint4(0, 0, 0, 0);
        if (ok) x[r] = ld_nc_v4(p.X + (mat + row * p.K + col) / 8);
    }

    // amax of this thread's part of each row and, two columns per word, of each
    // column; BF16 maxima are exact (a NaN gives way to the other operand)
    float ra[R];
    uint32_t cw[4] = {0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < R; ++r) {
        uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[j] &= 0x7FFF7FFFu;
            if (COLS && !BLOCK) cw[j] = max_bf16x2(cw[j], w[j]);
        }
        const uint32_t a = max_bf16x2(max_bf16x2(w[0], w[1]), max_bf16x2(w[2], w[3]));
        ra[r] = fmaxf(fmaxf(bf16_lo(a), bf16_hi(a)), 0.0f);
    }

    Scale block{};
    if (BLOCK) {
        float a = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) a = fmaxf(a, ra[r]);
        for (int d = 16; d > 0; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
        if (lane == 0) s_amax[warp] = a;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WARPS; ++w) a = fmaxf(a, s_amax[w]);
        block = block_scale<TYPE, POW2>(a);
        const int32_t tiles_m = gridDim.x / p.tiles_k;
        if (tid == 0) {
            p.SF[(group * tiles_m + mtile) * p.tiles_k + kblock] = block.s;
            if (COLS) p.SF_t[(group * p.tiles_k + kblock) * tiles_m + mtile] = block.s;
        }
    }

    if (ROWS || BLOCK) {
        // Row scales.  Each halving exchange leaves a thread half as many rows
        // and the maximum over twice as many threads, so that in the end 16 / R
        // of the 16 threads that share R rows hold each row's maximum, and a
        // scale is computed that often, not sixteen times; the threads then
        // fetch theirs back.
        Scale s = block;
        if (ROWS) {
#pragma unroll
            for (int n = R / 2, d = 8; d > 0; d >>= 1, n /= 2) {
                if (n > 0) {
                    const bool up = (c & d) != 0;
#pragma unroll
                    for (int r = 0; r < n; ++r)
                        ra[r] = fmaxf(up ? ra[r + n] : ra[r], __shfl_xor_sync(0xffffffffu, up ? ra[r] : ra[r + n], d));
                } else {
                    ra[0] = fmaxf(ra[0], __shfl_xor_sync(0xffffffffu, ra[0], d));
                }
            }
            const float mine = ra[0];
            s = block_scale<TYPE, POW2>(mine);
            constexpr int kPer = 16 / R;            // lanes that hold one row's scale
            const int32_t m = m0 + c / kPer;
            if (c % kPer == 0 && m < m_end) p.SF[static_cast<int64_t>(kblock) * p.M + m] = s.s;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float inv = ROWS ? __shfl_sync(0xffffffffu, s.inv, (lane & 16) + r * (16 / R)) : s.inv;
            const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
            uint32_t q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = encode2<TYPE>(__fmul_rn(bf16_lo(w[j]), inv), __fmul_rn(bf16_hi(w[j]), inv));
            const int32_t m = m0 + r;
            if (col_ok && m < m_end)
                *reinterpret_cast<uint2 *>(p.Q + mat + static_cast<int64_t>(m) * p.K + col) =
                    make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
        }
    }

    if (COLS) {
        float inv[8];
        if (BLOCK) {
#pragma unroll
            for (int j = 0; j < 8; ++j) inv[j] = block.inv;
        } else {
            float ca[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ca[2 * j] = bf16_lo(cw[j]);
                ca[2 * j + 1] = bf16_hi(cw[j]);
            }
            // the warp's two row groups: each lane keeps four of the columns
            float4 half;
            {
                const bool up = (lane & 16) != 0;
                float *h = &half.x;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    h[j] = fmaxf(up ? ca[j + 4] : ca[j], __shfl_xor_sync(0xffffffffu, up ? ca[j] : ca[j + 4], 16));
                reinterpret_cast<float4 *>(s_amax + warp * 128)[2 * c + (up ? 1 : 0)] = half;
            }
            __syncthreads();
            // one column per thread of the first half: its scale, its factor for the others
            if (tid < 128) {
                float a = 0.0f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) a = fmaxf(a, s_amax[w * 128 + tid]);
                const Scale s = block_scale<TYPE, POW2>(a);
                s_amax[tid] = s.inv;            // (only this thread read it: warp 0's row of the table)
                const int32_t k = kblock * 128 + tid;
                if (k < p.K) p.SF_t[static_cast<int64_t>(mtile) * p.K + k] = s.s;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 f = reinterpret_cast<const float4 *>(s_amax)[2 * c + j];
                inv[4 * j] = f.x; inv[4 * j + 1] = f.y; inv[4 * j + 2] = f.z; inv[4 * j + 3] = f.w;
            }
        }
        // codes of column 8 c + j, four rows to a word of the transposed tile
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int u = 0; u < R / 4; ++u) {
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint4 &q = x[(4 * u + r) % R];
                    const uint32_t w = j < 2 ? q.x : j < 4 ? q.y : j < 6 ? q.z : q.w;
                    v[r] = __fmul_rn((j & 1) ? bf16_hi(w) : bf16_lo(w), inv[j]);
                }
                s_t[(8 * c + j) * 32 + ((R / 4 * i + u) ^ (2 * c))] =
                    encode2<TYPE>(v[0], v[1]) | encode2<TYPE>(v[2], v[3]) << 16;
            }
        __syncthreads();
        const int64_t mat_t = BLOCK ? group * p.K * static_cast<int64_t>(p.Mt) : 0;
#pragma unroll
        for (int f = tid; f < 128 * 8; f += THREADS) {
            const int tc = f >> 3, part = f & 7, tcc = tc >> 3;
            const int32_t k = kblock * 128 + tc, m = mtile * 128 + 16 * part;
            uint4 q = reinterpret_cast<const uint4 *>(s_t)[tc * 8 + (part ^ (tcc >> 1))];
            if (tcc & 1) q = make_uint4(q.z, q.w, q.x, q.y);
            if (k < p.K && m < p.Mt)
                *reinterpret_cast<uint4 *>(p.Q_t + mat_t + static_cast<int64_t>(k) * p.Mt + m) = q;
        }
    }
}

template <int TYPE, bool POW2, int WHAT, int R, bool GROUPED = false>
int launch(const QuantParams &p, int64_t groups, cudaStream_t s)
{
    using C = QuantCfg<WHAT, R>;
    const int64_t tiles =
        ((static_cast<int64_t>(p.M) + C::ROWS - 1) / C::ROWS + (GROUPED ? p.groups : 0)) * p.tiles_k;
    if (tiles > INT32_MAX) return QFP4_ERR_UNSUPPORTED;
    return launch_status(launch_pdl(fp8_quantize_kernel<TYPE, POW2, WHAT, R, GROUPED>,
                                    dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(groups)), dim3(C::THREADS),
                                    0, s, p));
}

template <int TYPE, bool POW2>
int launch_what(const QuantParams &p, int what, int64_t groups, cudaStream_t s)
{
    if (p.groups)
        return what & kRows ? launch<TYPE, POW2, kRows | kCols, 8, true>(p, groups, s)
                            : launch<TYPE, POW2, kCols, 8, true>(p, groups, s);
    switch (what) {
    case kRows: return launch<TYPE, POW2, kRows, 2>(p, groups, s);
    case kCols: return launch<TYPE, POW2, kCols, 8>(p, groups, s);
    case kRows | kCols: return launch<TYPE, POW2, kRows | kCols, 8>(p, groups, s);
    case kBlock: return launch<TYPE, POW2, kBlock, 8>(p, groups, s);
    default: return launch<TYPE, POW2, kBlock | kCols, 8>(p, groups, s);
    }
}

int launch_any(int type, int scale, const QuantParams &p, int what, int64_t groups, cudaStream_t s)
{
    const bool pow2 = scale == QFP4_SCALE_POW2;
    if (type == QFP4_E4M3)
        return pow2 ? launch_what<QFP4_E4M3, true>(p, what, groups, s)
                    : launch_what<QFP4_E4M3, false>(p, what, groups, s);
    return pow2 ? launch_what<QFP4_E5M2, true>(p, what, groups, s)
                : launch_what<QFP4_E5M2, false>(p, what, groups, s);
}

bool types_ok(int type, int scale)
{
    return (type == QFP4_E4M3 || type == QFP4_E5M2) && (scale == QFP4_SCALE_FP32 || scale == QFP4_SCALE_POW2);
}

constexpr int64_t kMaxSize = int64_t{1} << 30;

}  // namespace
}  // namespace qfp4

using namespace qfp4;

extern "C" int qfp4_fp8_quantize(int type, int scale, const void *X_bf16, int64_t X_rows, const int32_t *row_index,
                                 int64_t M, int64_t K, void *Q, float *SF, void *Q_t, float *SF_t, void *stream)
{
    if (!types_ok(type, scale) || M < 0 || K < 0 || X_rows < 0) return QFP4_ERR_INVALID_ARG;
    if (!row_index && X_rows != M) return QFP4_ERR_INVALID_ARG;
    if (K % 16 != 0 || M > kMaxSize || K > kMaxSize) return QFP4_ERR_UNSUPPORTED;
    if (M == 0 || K == 0) return QFP4_OK;
    if ((Q == nullptr) != (SF == nullptr) || (Q_t == nullptr) != (SF_t == nullptr) || (!Q && !Q_t) ||
        (!X_bf16 && X_rows > 0))
        return QFP4_ERR_INVALID_ARG;
    if (!aligned16(X_bf16) || !aligned16(Q) || !aligned16(Q_t) || !aligned4(SF) || !aligned4(SF_t) ||
        !aligned4(row_index))
        return QFP4_ERR_MISALIGNED;
    const QuantParams p{static_cast<const uint4 *>(X_bf16), row_index, X_rows, static_cast<int32_t>(M),
                        static_cast<int32_t>(K), static_cast<int32_t>((M + 15) / 16 * 16), static_cast<int32_t>((K + 127) / 128),
                        static_cast<uint8_t *>(Q), static_cast<uint8_t *>(Q_t), SF, SF_t, nullptr, 0};
    return launch_any(type, scale, p, (Q ? kRows : 0) | (Q_t ? kCols : 0), 1, static_cast<cudaStream_t>(stream));
}

extern "C" int qfp4_fp8_quantize_weight(int type, int scale, int64_t groups, const void *W_bf16, int64_t N, int64_t K,
                                        void *Q, float *SF, void *Q_t, float *SF_t, void *stream)
{
    if (!types_ok(type, scale) || groups < 1 || N < 0 || K < 0) return QFP4_ERR_INVALID_ARG;
    if (K % 16 != 0 || N > kMaxSize || K > kMaxSize || groups > 65535) return QFP4_ERR_UNSUPPORTED;
    if (N == 0 || K == 0) return QFP4_OK;
    if (!W_bf16 || !Q || !SF || (Q_t == nullptr) != (SF_t == nullptr)) return QFP4_ERR_INVALID_ARG;
    if (!aligned16(W_bf16) || !aligned16(Q) || !aligned16(Q_t) || !aligned4(SF) || !aligned4(SF_t))
        return QFP4_ERR_MISALIGNED;
    const QuantParams p{static_cast<const uint4 *>(W_bf16), nullptr, N, static_cast<int32_t>(N),
                        static_cast<int32_t>(K), static_cast<int32_t>((N + 15) / 16 * 16), static_cast<int32_t>((K + 127) / 128),
                        static_cast<uint8_t *>(Q), static_cast<uint8_t *>(Q_t), SF, SF_t, nullptr, 0};
    return launch_any(type, scale, p, kBlock | (Q_t ? kCols : 0), groups, static_cast<cudaStream_t>(stream));
}

extern "C" size_t qfp4_fp8_grouped_cols(int64_t total_rows, int64_t groups)
{
    if (total_rows < 0 || groups < 1) return 0;
    return 128 * (static_cast<size_t>((total_rows + 127) / 128) + static_cast<size_t>(groups));
}

extern "C" int qfp4_fp8_quantize_grouped(int type, int scale, const void *X_bf16, int64_t X_rows,
                                         const int32_t *row_index, int64_t groups, const int32_t *row_offsets,
                                         int64_t total_rows, int64_t K, void *Q, float *SF, void *Q_t, float *SF_t,
                                         void *stream)
{
    if (!types_ok(type, scale) || total_rows < 0 || K < 0 || X_rows < 0 || groups < 1 || !row_offsets)
        return QFP4_ERR_INVALID_ARG;
    if (!row_index && X_rows != total_rows) return QFP4_ERR_INVALID_ARG;
    if (K % 16 != 0 || total_rows > kMaxSize || K > kMaxSize || groups > kMaxGroups) return QFP4_ERR_UNSUPPORTED;
    if (total_rows == 0 || K == 0) return QFP4_OK;
    if ((Q == nullptr) != (SF == nullptr) || !Q_t || !SF_t || (!X_bf16 && X_rows > 0)) return QFP4_ERR_INVALID_ARG;
    if (!aligned16(X_bf16) || !aligned16(Q) || !aligned16(Q_t) || !aligned4(SF) || !aligned4(SF_t) ||
        !aligned4(row_index) || !aligned4(row_offsets))
        return QFP4_ERR_MISALIGNED;
    const QuantParams p{static_cast<const uint4 *>(X_bf16), row_index, X_rows, static_cast<int32_t>(total_rows),
                        static_cast<int32_t>(K), static_cast<int32_t>(qfp4_fp8_grouped_cols(total_rows, groups)),
                        static_cast<int32_t>((K + 127) / 128), static_cast<uint8_t *>(Q), static_cast<uint8_t *>(Q_t),
                        SF, SF_t, row_offsets, static_cast<int32_t>(groups)};
    return launch_any(type, scale, p, (Q ? kRows : 0) | kCols, 1, static_cast<cudaStream_t>(stream));
}
