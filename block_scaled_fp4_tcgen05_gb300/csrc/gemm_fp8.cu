// gemm_fp8.cu -- product of 8-bit floating point operands with one fp32 scale
// per 128 elements of K (see qfp4_gemm_nt_fp8), on CTA pairs.
//
// D[m,n] = sum_j sa[j][m] sb(j,n) sum_{k in block j} a b: the tensor cores
// (tcgen05 kind::f8f6f4) sum one block of 128, and because its scale differs
// from the next one's, each block's sum leaves tensor memory for registers,
// where it is added under the fp32 product of its two scales.
//
// A cluster of two CTAs computes a tile of 256 rows x TN = 256 columns (128
// where that fills the last round of tiles better).  CTA r holds 128 rows of A
// and TN / 2 rows of B per K block (a ring of four stages of 32 KB, or seven of
// 24); the leader issues four M=256 N=TN K=32 MMAs per K block into one of 512 /
// TN accumulator slots, so that one is summed while another is drained.  Two
// warps issue them, for even and odd K blocks, so that one looks at its
// barriers while the other's MMAs run (experts' product 490 -> 474 us).
// Eight epilogue warps per CTA each keep 32 rows x TN / 2 columns of D in
// registers (128 per thread; the producer warps give theirs up with
// setmaxnreg).  A thread owns one row and its columns lie in one block of B's
// scales, so the scale is one number per thread and K block (COLSCALE: one per
// column).  D is staged in shared memory behind one fence and leaves by TMA.
//
// What bounds it is the epilogue's chain per K block (about 870 cycles at TN =
// 256, where the MMAs take 512) and, on long products, the power limit: 4096 x
// 4096 x 14336 takes 207 us (2.33 PFLOP/s; 1.36 kW); with the multiply-adds
// left out 180, and with all of K summed in tensor memory, so without any
// epilogue per block, 173 (at 1.75 GHz, the same power).  An SM's 32768
// multiply-adds per K block are 128 packed instructions per scheduler, beside
// four tensor-memory loads per warp (72 cycles each alone) and the hand-overs
// (about 95 cycles for a look at an mbarrier that is already complete).  So:
// the second half's loads run under the first half's additions; the next slot
// is looked at before the last additions and judged after them; slots are given
// back with relaxed arrivals straight at the leader; scales come through shared
// memory from a warp of their own, eight K blocks at a time (loading them in
// the epilogue warps themselves cost a global latency per K block); the
// multiply-adds are packed in pairs (212 us with single ones).  Slower, at the
// same product: the next block's first load ahead of the last additions (214
// against 207), sixteen epilogue warps of 64 columns (230 against 216), two
// slots of 128 columns per K block (281 where one of 256 took 241).
//
// COLSCALE adds a multiply per element and reads of the columns' scales from
// shared memory.  With a thread per row those reads alone, a wavefront's worth
// of returned data per column and warp, take longer than the MMAs; reading
// tensor memory 16 rows x 64 columns at a time a thread needs the scales of a
// quarter of the columns, and packed arithmetic then pays (fewer
// instructions): 14336 x 4096 x 4096 with fp32 output takes 280 us (314 with a
// thread per row, 296 with plain multiply-adds, 251 without the stores).
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "qfp4_common.cuh"
#include "qfp4_gemm_fp8.cuh"
#include "qfp4_gemm_internal.cuh"
#include "sm103_ptx.cuh"

namespace qfp4 {

__device__ uint32_t g_status_gemm_fp8 = 0;

#ifdef QFP4_FAULT_INJECTION
// Test build only: when set, one epilogue warp of the first pair's leader never
// gives back the slot of its first K block, so that the issuer's next wait for
// that slot runs out.  No copy completes on that barrier.
__device__ int g_inject_fp8_pair = 0;
__device__ __forceinline__ bool inject_skip(bool here) { return here && g_inject_fp8_pair != 0; }
#else
__device__ __forceinline__ bool inject_skip(bool) { return false; }
#endif

int status_word_gemm_fp8(uint32_t **word) { return status_word(g_status_gemm_fp8, word); }

namespace {

constexpr int64_t kMaxSize = int64_t{1} << 30;

// ---------------------------------------------------------------- CTA pairs, 256 x TN tiles

constexpr int kPairThreads = 384;       // 12 warps
constexpr int kEpiWarps = 8;
constexpr int kBatch = 8;               // K blocks per hand-over of scales
constexpr int kABytes = 128 * 128;      // a CTA's 128 rows of A x 128 elements of K
constexpr int kBoxBytes = 32 * 128;     // output staging box: 32 rows x 128 bytes

template <int TN>
struct PairCfg {
    static constexpr int STAGES = TN == 256 ? 4 : 7;
    static constexpr int STAGE = kABytes + TN / 2 * 128;        // and TN / 2 rows of B
    static constexpr int SLOTS = 512 / TN;                      // accumulator slots of TN columns
    static constexpr int COLS = TN / 2;                         // columns per epilogue warp
    static constexpr int SCALES = 128 + TN;                     // floats per K block: the CTA's rows, then the tile's
                                                                // columns (or its blocks of 128)
    static constexpr int BOXES = TN / 128;                      // staging boxes per epilogue warp
    static constexpr int OFF_SCALE = STAGES * STAGE;            // two batches
    static constexpr int OFF_OUT = OFF_SCALE + 2 * kBatch * SCALES * 4;
    static constexpr int OFF_BAR = OFF_OUT + kEpiWarps * BOXES * kBoxBytes;
    // full, empty [stage]; acc_full, acc_empty [slot]; sc_full, sc_empty [2]
    static constexpr int NBAR = 2 * STAGES + 2 * SLOTS + 4;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
    static_assert(SMEM + 4096 <= 232448, "shared memory overflow");
    static_assert(OFF_OUT % 1024 == 0, "swizzled boxes start on 1 KB");
};

__device__ __forceinline__ void record_timeout()
{
    atomicOr(&g_status_gemm_fp8, static_cast<uint32_t>(kStatusTimeout));
}



// Writes a warp's 32 rows x COLS columns of D.  Lane i holds row i, or with
// PAIRS what tmem_ld_16x256b_x8 gives it: acc[32 (2 c + h) ..] are columns 64 c
// .. 64 c + 63 of rows 16 h .. 16 h + 15.  The rows are staged as boxes of 128
// bytes x 32 rows in the 128-byte swizzle of the store map (16-byte piece c of
// row r at c ^ (r % 8)), up to BOXES of them at a time, and leave together
// behind one fence.
template <bool FP32, int COLS, int BOXES, bool PAIRS>
__device__ __forceinline__ void store_tile(const float (&acc)[COLS], uint8_t *out, const CUtensorMap &map,
                                           const Fp8Params &p, bool by_tma, int32_t row0, int32_t rows, int32_t c0,
                                           int lane)
{
    constexpr int kCols = FP32 ? 32 : 64;       // columns of a box
#pragma unroll
    for (int q0 = 0; q0 < COLS / kCols; q0 += BOXES) {
        if (c0 + q0 * kCols >= p.N) break;
        // the boxes are free once the copy engine has read what left them last
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
        if constexpr (PAIRS) {
#pragma unroll
            for (int q = 0; q < BOXES; ++q)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int g = 0; g < kCols / 8; ++g)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            // two neighbouring columns of row r: eight or four bytes of a piece
                            const int r = 16 * h + 8 * u + (lane >> 2);
                            const int a = FP32 ? ((q0 + q) / 2 * 2 + h) * 32 + ((q0 + q) % 2 * 4 + g) * 4 + 2 * u
                                               : ((q0 + q) * 2 + h) * 32 + g * 4 + 2 * u;
                            uint8_t *row = out + q * kBoxBytes + r * 128;
                            if (FP32) {
                                *reinterpret_cast<float2 *>(row + 16 * ((2 * g + ((lane >> 1) & 1)) ^ (r & 7)) +
                                                            8 * (lane & 1)) = make_float2(acc[a], acc[a + 1]);
                            } else {
                                *reinterpret_cast<__nv_bfloat162 *>(row + 16 * (g ^ (r & 7)) + 4 * (lane & 3)) =
                                    __floats2bfloat162_rn(acc[a], acc[a + 1]);
                            }
                        }
        } else {
#pragma unroll
        for (int q = 0; q < BOXES; ++q)
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (FP32) {
                        w[i] = __float_as_uint(acc[(q0 + q) * 32 + 4 * c + i]);
                    } else {
                        const int a = (q0 + q) * 64 + 8 * c + 2 * i;
                        __nv_bfloat162 pr = __floats2bfloat162_rn(acc[a], acc[a + 1]);
                        w[i] = *reinterpret_cast<uint32_t *>(&pr);
                    }
                }
                *reinterpret_cast<uint4 *>(out + q * kBoxBytes + lane * 128 + 16 * (c ^ (lane & 7))) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        if (by_tma) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
#pragma unroll
                for (int q = 0; q < BOXES; ++q) {
                    const int32_t col = c0 + (q0 + q) * kCols;
                    if (col >= p.N) break;
                    // (one fp32 addition per element, by the copy engine; numbers below 2^-126 keep their bits)
                    if (p.accumulate) tma_reduce_add_2d(&map, smem_u32(out + q * kBoxBytes), col, row0);
                    else tma_store_2d(&map, smem_u32(out + q * kBoxBytes), col, row0);
                }
                bulk_commit_group();
            }
            continue;
        }
        __syncwarp();
        // a row's 128 bytes of a box at a time, a word per lane
#pragma unroll
        for (int q = 0; q < BOXES; ++q) {
            const int32_t col = c0 + (q0 + q) * kCols + (FP32 ? lane : 2 * lane);
#pragma unroll 4
            for (int r = 0; r < rows; ++r) {
                const uint32_t v = *reinterpret_cast<const uint32_t *>(
                    out + q * kBoxBytes + r * 128 + 16 * ((lane >> 2) ^ (r & 7)) + 4 * (lane & 3));
                const int64_t at = static_cast<int64_t>(row0 + r) * p.N + col;
                if (FP32) {
                    float *d = static_cast<float *>(p.D) + at;
                    if (col < p.N) *d = p.accumulate ? *d + __uint_as_float(v) : __uint_as_float(v);
                } else {
                    uint16_t *d = static_cast<uint16_t *>(p.D) + at;
                    if (p.N % 2 == 0) {
                        if (col < p.N) *reinterpret_cast<uint32_t *>(d) = v;
                    } else {
                        if (col < p.N) d[0] = static_cast<uint16_t>(v);
                        if (col + 1 < p.N) d[1] = static_cast<uint16_t>(v >> 16);
                    }
                }
            }
        }
        __syncwarp();
    }
}

struct Tile {
    int32_t row0, row_end;      // rows of A and D: the tile's first, the end of its product's
    int32_t n0, group;
    int32_t kb0, kblocks;       // K blocks of its product
};

// kRowGroups: the groups' rows of A and D, each with its own B.
// kBlockGroups: the groups' K blocks, each with its own D (weight gradients per expert).
enum Grouping { kDense, kRowGroups, kBlockGroups };

// COLSCALE: B has one scale per row (b_rows = 1), else one per 128 rows.
template <Grouping GROUPING, bool COLSCALE, int TN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmD, const Fp8Params p)
{
    using C = PairCfg<TN>;
    constexpr bool GROUPED = GROUPING != kDense;
    // rows of one of s_ptile's tiles: row tiles of D, or blocks of K
    constexpr int kTileRows = GROUPING == kBlockGroups ? 128 : 256;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);   // leader: bytes of both CTAs
    uint64_t *empty = full + C::STAGES;                                // stage free again (MMA commit, both CTAs)
    uint64_t *acc_full = empty + C::STAGES;                            // slot's sum complete (both CTAs)
    uint64_t *acc_empty = acc_full + C::SLOTS;                         // leader: slot drained by both CTAs
    uint64_t *sc_full = acc_empty + C::SLOTS;                          // [2] batch of scales written
    uint64_t *sc_empty = sc_full + 2;                                // [2] batch of scales read
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sc_empty + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    __shared__ int32_t s_offs[GROUPED ? kMaxGroups + 1 : 1];
    __shared__ int32_t s_ptile[GROUPED ? kMaxGroups + 1 : 1];        // running sum of the groups' tiles

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int32_t kblocks = (p.K + 127) / 128;
    const int32_t ntiles_n = (p.N + TN - 1) / TN;
    const int32_t pair_id = blockIdx.x >> 1;
    const int32_t npairs = gridDim.x >> 1;

    if (GROUPED) pdl_wait();
    int32_t total_tiles;
    if (GROUPED) {
        for (int i = threadIdx.x; i <= p.groups; i += blockDim.x) s_offs[i] = p.row_offsets[i];
        __syncthreads();
        const bool bad = __syncthreads_or(threadIdx.x < p.groups &&
                                          !fp8_offsets_valid(s_offs, threadIdx.x, p.groups, p.total_rows, p.max_group_rows));
        if (bad && threadIdx.x == 0 && blockIdx.x == 0)
            atomicOr(&g_status_gemm_fp8, static_cast<uint32_t>(kStatusBadGroup));
        // running sum of the groups' tiles, eight groups a lane
        if (warp == 0) {
            constexpr int kPer = kMaxGroups / 32;
            int32_t before[kPer], sum = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int e = lane * kPer + i;
                before[i] = sum;
                sum += !bad && e < p.groups ? (s_offs[e + 1] - s_offs[e] + kTileRows - 1) / kTileRows : 0;
            }
            int32_t up = sum;
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t o = __shfl_up_sync(0xffffffffu, up, d);
                if (lane >= d) up += o;
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int e = lane * kPer + i;
                if (e < p.groups) s_ptile[e] = up - sum + before[i];
            }
            if (lane == 31) s_ptile[p.groups] = up;
        }
        __syncthreads();
        total_tiles = GROUPING == kRowGroups ? s_ptile[p.groups] * ntiles_n
                      : bad                ? 0
                                             : p.groups * ((p.M + 255) / 256) * ntiles_n;
    } else {
        total_tiles = ((p.M + 255) / 256) * ntiles_n;
    }

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < C::SLOTS; ++b) {
            mbar_init(smem_u32(&acc_full[b]), 1);
            mbar_init(smem_u32(&acc_empty[b]), 2 * kEpiWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&sc_full[b]), 32);
            mbar_init(smem_u32(&sc_empty[b]), kEpiWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmD);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    if (!GROUPED) pdl_wait();
    pdl_launch_dependents();

    auto tile_info = [&](int32_t t) {
        Tile ti;
        ti.group = 0;
        int32_t lt = t, mtiles = (p.M + 255) / 256, base = 0;
        ti.row_end = p.M;
        ti.kb0 = 0;
        ti.kblocks = kblocks;
        if (GROUPING == kBlockGroups) {
            ti.group = t / (mtiles * ntiles_n);
            lt = t - ti.group * mtiles * ntiles_n;
            base = ti.group * p.M;
            ti.row_end = base + p.M;
            ti.kb0 = s_ptile[ti.group];
            ti.kblocks = s_ptile[ti.group + 1] - ti.kb0;
        }
        if (GROUPING == kRowGroups) {
            const int32_t mt_all = t / ntiles_n;
            int lo = 0, hi = p.groups - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_ptile[mid] <= mt_all) lo = mid; else hi = mid - 1;
            }
            lt = t - s_ptile[lo] * ntiles_n;
            mtiles = s_ptile[lo + 1] - s_ptile[lo];
            base = s_offs[lo];
            ti.group = lo;
            ti.row_end = s_offs[lo + 1];
        }
        // groups of up to eight row tiles walk the column tiles together, so
        // that the pairs of one round share operand tiles in L2
        constexpr int32_t GM = 8;
        const int32_t per_group = GM * ntiles_n;
        const int32_t first_m = (lt / per_group) * GM;
        const int32_t rows_here = min(GM, mtiles - first_m);
        const int32_t idx = lt % per_group;
        ti.row0 = base + (first_m + idx % rows_here) * 256;
        ti.n0 = (idx / rows_here) * TN;
        return ti;
    };

    if (warp < 4) {
        setmaxnreg_dec<40>();
        if (warp == 0) {
            // ------------------------------------------------ TMA producer
            if (lane == 0) {
                const uint32_t full0_leader = mapa_shared(smem_u32(&full[0]), 0);
                uint32_t s = 0, phase = 1;
                bool ok = true;
                for (int32_t t = pair_id; t < total_tiles && ok; t += npairs) {
                    const Tile ti = tile_info(t);
                    const int32_t arow = ti.row0 - (GROUPING == kBlockGroups ? ti.group * p.M : 0) +
                                         128 * static_cast<int32_t>(rank);
                    const int32_t brow = (GROUPING == kRowGroups ? ti.group * p.N : 0) + ti.n0 +
                                         TN / 2 * static_cast<int32_t>(rank);
                    for (int32_t kb = ti.kb0; kb < ti.kb0 + ti.kblocks; ++kb) {
                        if (!mbar_wait(smem_u32(&empty[s]), phase)) { ok = false; break; }
                        if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full[s]), 2 * C::STAGE);
                        tma_load_2d_pair(smem_u32(smem + s * C::STAGE), &tmA, full0_leader + s * 8, kb * 128, arow);
                        tma_load_2d_pair(smem_u32(smem + s * C::STAGE + kABytes), &tmB, full0_leader + s * 8, kb * 128, brow);
                        if (++s == C::STAGES) { s = 0; phase ^= 1; }
                    }
                }
                if (!ok) { record_timeout(); *abort_flag = 1; }
            }
        } else if (warp == 3) {
            // ------------------------------------------------ scales: kBatch K blocks at a time, copied
            // straight into one of two halves (4-byte copies: a row of scales need not be aligned)
            uint32_t b = 0, phase = 1;
            bool ok = true;
            const int32_t nb = (p.N + 127) / 128;
            for (int32_t t = pair_id; t < total_tiles && ok; t += npairs) {
                const Tile ti = tile_info(t);
                const int32_t row = ti.row0 - (GROUPING == kBlockGroups ? ti.group * p.M : 0) +
                                    128 * static_cast<int32_t>(rank) + lane;
                const int32_t kb_end = ti.kb0 + ti.kblocks;
                for (int32_t kb0 = ti.kb0; kb0 < kb_end; kb0 += kBatch) {
                    if (!mbar_wait_warp(smem_u32(&sc_empty[b]), phase)) { ok = false; break; }
                    uint32_t dst = smem_u32(smem + C::OFF_SCALE) + b * (kBatch * C::SCALES * 4);
                    if (!COLSCALE && lane < 2 * kBatch && kb0 + (lane >> 1) < kb_end) {
                        // lane 2 u + h: the h-th block of 128 columns at K block u
                        cp_async4(dst + ((lane >> 1) * C::SCALES + 128 + (lane & 1)) * 4,
                                  p.B_sf + (static_cast<int64_t>(ti.group) * nb + min(ti.n0 / 128 + (lane & 1), nb - 1)) * kblocks +
                                      kb0 + (lane >> 1));
                    }
                    dst += lane * 4;
                    for (int32_t kb = kb0; kb < min(kb0 + kBatch, kb_end); ++kb, dst += C::SCALES * 4) {
                        const float *a = p.A_sf + static_cast<int64_t>(kb) * p.M;
#pragma unroll
                        for (int i = 0; i < 4; ++i) cp_async4(dst + i * 128, a + min(row + 32 * i, p.M - 1));
                        if (COLSCALE) {
                            const float *c = p.B_sf + static_cast<int64_t>(kb) * p.N;
#pragma unroll
                            for (int i = 0; i < TN / 32; ++i)
                                cp_async4(dst + 512 + i * 128, c + min(ti.n0 + lane + 32 * i, p.N - 1));
                        }
                    }
                    cp_async_arrive(smem_u32(&sc_full[b]));     // every lane, once its copies have landed
                    b ^= 1;
                    if (b == 0) phase ^= 1;
                }
            }
            if (!ok && lane == 0) { record_timeout(); *abort_flag = 1; }
        } else if (rank == 0) {
            // ------------------------------------------------ MMA issuers (leader): warp 1 takes the even K
            // blocks of the whole sequence, warp 2 the odd ones, the slots in turn, so that one looks at
            // its barriers while the other's MMAs run.  The whole warp keeps count and one lane issues:
            // descriptors stay in uniform registers.
            const uint32_t first = warp - 1;
            const uint64_t a_desc0 = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
            const uint64_t b_desc0 = smem_desc(smem_u32(smem) + kABytes, 16, 1024, kSwizzle128B);
            const uint32_t idesc = idesc_f8(256, TN, p.a_type, p.b_type);
            uint32_t s = first, phase = 0, slot = first, acc_phase = 1;
            bool ok = true;
            int64_t count = 0;
            if (GROUPING == kBlockGroups) {
                for (int32_t t = pair_id; t < total_tiles; t += npairs) count += tile_info(t).kblocks;
            } else if (pair_id < total_tiles) {
                count = static_cast<int64_t>((total_tiles - pair_id + npairs - 1) / npairs) * kblocks;
            }
            for (int64_t j = first; j < count; j += 2) {
                if (!mbar_wait_warp(smem_u32(&full[s]), phase) ||
                    !mbar_wait_warp(smem_u32(&acc_empty[slot]), acc_phase)) { ok = false; break; }
                tc_fence_after();
                if (elect_one_sync()) {
                    const uint64_t ad = a_desc0 + s * static_cast<uint64_t>(C::STAGE >> 4);
                    const uint64_t bd = b_desc0 + s * static_cast<uint64_t>(C::STAGE >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_f8_pair(tmem_base + slot * TN, ad + 2 * kk, bd + 2 * kk, idesc, kk > 0 ? 1u : 0u);
                    tc_commit_pair(smem_u32(&acc_full[slot]), 0x3);
                    tc_commit_pair(smem_u32(&empty[s]), 0x3);
                }
                __syncwarp();
                slot += 2;
                if (slot >= C::SLOTS) { slot = first; acc_phase ^= 1; }
                s += 2;
                if (s >= C::STAGES) { s -= C::STAGES; phase ^= 1; }
            }
            if (!ok && lane == 0) { record_timeout(); *abort_flag = 1; }
        }
    } else {
        setmaxnreg_inc<232>();
        // ------------------------------------------------ epilogue: eight warps, each 32 rows x TN / 2 columns
        const int quad = warp & 3;
        const int half = (warp - 4) >> 2;
        const uint32_t release = mapa_shared(smem_u32(&acc_empty[0]), 0);
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + half * C::COLS;
        uint8_t *out = smem + C::OFF_OUT + (warp - 4) * C::BOXES * kBoxBytes;
        const float *s_scale = reinterpret_cast<const float *>(smem + C::OFF_SCALE);
        uint32_t slot = 0, phase = 0, b = 0, sc_phase = 0;
        bool ok = true;
        for (int32_t t = pair_id; t < total_tiles && ok; t += npairs) {
            const Tile ti = tile_info(t);
            const int32_t c0 = ti.n0 + half * C::COLS;
            float acc[C::COLS];
#pragma unroll
            for (int i = 0; i < C::COLS; ++i) acc[i] = 0.0f;
            bool ready = false;         // the next slot's sum is known to be complete
            int u = 0;
            for (int32_t kb = 0; kb < ti.kblocks; ++kb) {
                if (u == 0 && !mbar_wait_warp(smem_u32(&sc_full[b]), sc_phase)) { ok = false; break; }
                if (!ready && !mbar_wait_warp(smem_u32(&acc_full[slot]), phase)) { ok = false; break; }
                tc_fence_after();
                const uint32_t src = taddr + slot * TN;
                bool done = false;
                const float *sc = s_scale + (b * kBatch + u) * C::SCALES;
                auto give_back = [&]() {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0 && !inject_skip(blockIdx.x == 0 && warp == 4 && t == pair_id && kb == 0))
                        mbar_arrive_cluster_relaxed(release + slot * 8);
                    if (++slot == C::SLOTS) { slot = 0; phase ^= 1; }
                    done = mbar_test(smem_u32(&acc_full[slot]), phase);
                };
                uint32_t v[2][32];
                if constexpr (COLSCALE) {
                    // 64 columns of 16 rows at a time: a thread then needs the scales of four rows and of a
                    // quarter of the columns (all of them, for one row: the reads of shared memory alone
                    // take longer than the MMAs)
                    const uint32_t upper = src + (16u << 16);
                    tmem_ld_16x256b_x8(src, v[0]);
                    tmem_ld_16x256b_x8(upper, v[1]);
                    const float *sr = sc + quad * 32 + (lane >> 2);
                    const float rs[4] = {sr[0], sr[8], sr[16], sr[24]};
                    uint64_t cs[8];             // scales of column pairs of 64 columns
                    auto columns = [&](int c) {
#pragma unroll
                        for (int g = 0; g < 8; ++g)
                            cs[g] = *reinterpret_cast<const uint64_t *>(sc + 128 + half * C::COLS + c * 64 + 8 * g +
                                                                        2 * (lane & 3));
                    };
                    auto add64 = [&](const uint32_t (&x)[32], int c, int h) {
#pragma unroll
                        for (int g = 0; g < 8; ++g)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int a = (2 * c + h) * 32 + 4 * g + 2 * u;
                                const uint64_t t = mul_f32x2(pack_b32x2(x[4 * g + 2 * u], x[4 * g + 2 * u + 1]), cs[g]);
                                const uint64_t r = pack_f32x2(rs[2 * h + u], rs[2 * h + u]);
                                unpack_f32x2(fma_f32x2(r, t, pack_f32x2(acc[a], acc[a + 1])), acc[a], acc[a + 1]);
                            }
                    };
                    columns(0);
                    tmem_ld_wait();
                    tmem_regs_after_wait(v[0]);
                    tmem_regs_after_wait(v[1]);
                    if constexpr (TN == 256) {
                        add64(v[0], 0, 0);
                        tmem_ld_16x256b_x8(src + 64, v[0]);
                        add64(v[1], 0, 1);
                        tmem_ld_16x256b_x8(upper + 64, v[1]);
                        columns(1);
                        tmem_ld_wait();
                        tmem_regs_after_wait(v[0]);
                        tmem_regs_after_wait(v[1]);
                    }
                    give_back();
                    add64(v[0], TN == 256 ? 1 : 0, 0);
                    add64(v[1], TN == 256 ? 1 : 0, 1);
                } else {
                    tmem_ld_32x32b_x32(src, v[0]);
                    tmem_ld_32x32b_x32(src + 32, v[1]);
                    // The product of the scales has to be a normal number (the header says so).  Taking them
                    // one after the other costs a multiply per element; to do so only where the product is
                    // none, decided by a vote per K block here or by the scales' warp, 3 to 5% of the time of
                    // every product (4096 x 4096 x 14336: 207 us where, in the same run, it took 201)
                    const float sm = sc[quad * 32 + lane] * sc[128 + (TN == 256 ? half : 0)];
                    const uint64_t sm2 = pack_f32x2(sm, sm);
                    auto add32 = [&](const uint32_t (&x)[32], int c) {
                        float *d = acc + c * 32;
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            unpack_f32x2(fma_f32x2(sm2, pack_b32x2(x[i], x[i + 1]), pack_f32x2(d[i], d[i + 1])), d[i], d[i + 1]);
                    };
                    tmem_ld_wait();
                    tmem_regs_after_wait(v[0]);
                    tmem_regs_after_wait(v[1]);
                    if constexpr (TN == 256) {
                        // the second half's loads run under the first half's additions
                        add32(v[0], 0);
                        tmem_ld_32x32b_x32(src + 64, v[0]);
                        add32(v[1], 1);
                        tmem_ld_32x32b_x32(src + 96, v[1]);
                        tmem_ld_wait();
                        tmem_regs_after_wait(v[0]);
                        tmem_regs_after_wait(v[1]);
                    }
                    give_back();
                    add32(v[0], TN == 256 ? 2 : 0);
                    add32(v[1], TN == 256 ? 3 : 1);
                }
                ready = __all_sync(0xffffffffu, done) && kb + 1 < ti.kblocks;
                if (++u == kBatch || kb == ti.kblocks - 1) {
                    u = 0;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sc_empty[b]));
                    b ^= 1;
                    if (b == 0) sc_phase ^= 1;
                }
            }
            if (!ok) break;
            // D leaves by TMA where its rows are 16-byte aligned and the warp's 32 rows are all this
            // tile's (rows beyond M are clipped by the map), else in four-byte or single pieces
            const int32_t wrow0 = ti.row0 + 128 * static_cast<int32_t>(rank) + quad * 32;
            const int32_t rows = ti.row_end - wrow0;
            // (a group without rows adds nothing: its D is not even read, and a -0 in it stays)
            const bool nothing = GROUPING == kBlockGroups && p.accumulate && ti.kblocks == 0;
            if (rows > 0 && c0 < p.N && !nothing) {
                const bool by_tma = p.store_map && (!GROUPED || rows >= 32);
                if (p.fp32) store_tile<true, C::COLS, C::BOXES, COLSCALE>(acc, out, tmD, p, by_tma, wrow0, min(rows, 32), c0, lane);
                else store_tile<false, C::COLS, C::BOXES, COLSCALE>(acc, out, tmD, p, by_tma, wrow0, min(rows, 32), c0, lane);
            }
            __syncwarp();
        }
        if (!ok && lane == 0) { record_timeout(); *abort_flag = 1; }
        // the staging boxes must outlive the stores issued from them
        if (lane == 0) bulk_wait_group<0>();
    }

    // teardown: lanes that skipped a single-lane role wait for their warp
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (*abort_flag) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) { }
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

bool types_ok(int a_type, int b_type, int out_type)
{
    return (a_type == QFP4_E4M3 || a_type == QFP4_E5M2) && (b_type == QFP4_E4M3 || b_type == QFP4_E5M2) &&
           (out_type == QFP4_BF16 || out_type == QFP4_FP32);
}

template <Grouping GROUPING, bool COLSCALE, int TN>
int launch_pair(Fp8Params p, int64_t tiles, cudaStream_t s)
{
    using C = PairCfg<TN>;
    auto kern = gemm_fp8_pair_kernel<GROUPING, COLSCALE, TN>;
    CUtensorMap ma, mb, md;
    int rc = ensure_smem_attr(reinterpret_cast<const void *>(kern), C::SMEM);
    if (rc == QFP4_OK) rc = make_map_direct(&ma, p.A, p.K, p.M, 128, 128);
    const uint64_t b_groups = GROUPING == kRowGroups ? p.groups : 1, d_groups = GROUPING == kBlockGroups ? p.groups : 1;
    if (rc == QFP4_OK) rc = make_map_direct(&mb, p.B, p.K, b_groups * p.N, 128, TN / 2);
    p.store_map = p.N % (p.fp32 ? 4 : 8) == 0;
    if (rc == QFP4_OK && p.store_map) rc = make_map_store(&md, p.D, p.fp32 != 0, p.N, d_groups * p.M, p.fp32 ? 32 : 64, 32);
    else md = ma;       // never used
    if (rc != QFP4_OK) return rc;
    const int sms = sm_count();
    if (sms < 2) return QFP4_ERR_CUDA;
    const int64_t pairs = tiles < sms / 2 ? tiles : sms / 2;
    return launch_status(launch_pdl(kern, dim3(static_cast<unsigned>(2 * pairs)), dim3(kPairThreads), C::SMEM, s,
                                    ma, mb, md, p));
}

template <int TN>
int launch_width(const Fp8Params &p, int64_t tiles, cudaStream_t s)
{
    if (p.groups) return p.b_rows == 1 ? launch_pair<kBlockGroups, true, TN>(p, tiles, s)
                                       : launch_pair<kRowGroups, false, TN>(p, tiles, s);
    return p.b_rows == 1 ? launch_pair<kDense, true, TN>(p, tiles, s) : launch_pair<kDense, false, TN>(p, tiles, s);
}

int launch_gemm_fp8(const Fp8Params &p, cudaStream_t s)
{
    if (!(p.groups && p.b_rows == 1) && gemm_fp8_small_pays(p)) return launch_gemm_fp8_small(p, s);
    int64_t tiles_m = (static_cast<int64_t>(p.M) + 255) / 256;
    if (p.groups && p.b_rows == 1) {
        tiles_m *= p.groups;
    } else if (p.groups) {
        // every group may add one partial tile, and none has more than max_group_rows rows
        tiles_m += p.groups;
        const int64_t by_max = static_cast<int64_t>(p.groups) * ((p.max_group_rows + 255) / 256);
        if (p.max_group_rows > 0 && by_max < tiles_m) tiles_m = by_max;
    }
    const int64_t wide = tiles_m * ((static_cast<int64_t>(p.N) + 255) / 256);
    const int64_t narrow = tiles_m * ((static_cast<int64_t>(p.N) + 127) / 128);
    if (narrow > INT32_MAX / 2) return QFP4_ERR_UNSUPPORTED;
    const int64_t pairs = sm_count() / 2;
    if (pairs < 1) return QFP4_ERR_CUDA;
    // Tiles 128 columns wide cost 0.65 of the time of one 256 wide, with either
    // form of B's scales (4096 x 4864 x 4096: 78.8 us in eight rounds of narrow
    // tiles, 62.6 in four of wide ones; fp32 with column scales 123.6 and 96.5),
    // so they pay where they fill the last round better: 1536 x 4864 x 4096 takes
    // 32.2 us in three rounds of narrow tiles and 33.0 in two of wide ones (49.0
    // and 50.1), 768 x 4864 x 4096 22.6 in two and 18.8 in one (33.7 and 27.4).
    const int64_t narrow_cost = (narrow + pairs - 1) / pairs * 13;
    return narrow_cost < (wide + pairs - 1) / pairs * 20 ? launch_width<128>(p, narrow, s)
                                                         : launch_width<256>(p, wide, s);
}

}  // namespace
}  // namespace qfp4

using namespace qfp4;

extern "C" int qfp4_gemm_nt_fp8(int a_type, int b_type, int64_t M, int64_t N, int64_t K, const void *A,
                                const float *A_sf, const void *B, const float *B_sf, int b_rows, int out_type,
                                int accumulate, void *D, void *stream)
{
    if (!types_ok(a_type, b_type, out_type) || (b_rows != 1 && b_rows != 128)) return QFP4_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 0 || (accumulate && out_type != QFP4_FP32)) return QFP4_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return QFP4_OK;            // empty D: nothing to do, nothing launched
    if (!D) return QFP4_ERR_INVALID_ARG;
    if (K % 16 != 0 || M > kMaxSize || N > kMaxSize || K > kMaxSize) return QFP4_ERR_UNSUPPORTED;
    if (!aligned16(D)) return QFP4_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) {
        // an empty sum: nothing is added, or D = 0 (+0 is all-zero bits)
        if (accumulate) return QFP4_OK;
        return launch_status(cudaMemsetAsync(D, 0, static_cast<size_t>(M) * static_cast<size_t>(N) *
                                                       (out_type == QFP4_FP32 ? 4 : 2), s));
    }
    if (!A || !A_sf || !B || !B_sf) return QFP4_ERR_INVALID_ARG;
    if (!aligned16(A) || !aligned16(B) || !aligned4(A_sf) || !aligned4(B_sf)) return QFP4_ERR_MISALIGNED;
    const Fp8Params p{static_cast<const uint8_t *>(A), static_cast<const uint8_t *>(B), A_sf, B_sf, D, nullptr,
                      static_cast<int32_t>(M), static_cast<int32_t>(N), static_cast<int32_t>(K), 0, 0,
                      a_type, b_type, b_rows, out_type == QFP4_FP32, accumulate ? 1 : 0};
    return launch_gemm_fp8(p, s);
}

extern "C" int qfp4_gemm_nt_fp8_grouped(int a_type, int b_type, int64_t groups, const int32_t *row_offsets,
                                        int64_t total_rows, int64_t max_group_rows, int64_t N, int64_t K,
                                        const void *A, const float *A_sf, const void *B, const float *B_sf,
                                        int out_type, void *D, void *stream)
{
    if (!types_ok(a_type, b_type, out_type)) return QFP4_ERR_INVALID_ARG;
    if (groups < 1 || !row_offsets || total_rows < 0 || max_group_rows < 0 || N < 1 || K < 1)
        return QFP4_ERR_INVALID_ARG;
    if (!A || !A_sf || !B || !B_sf || !D) return QFP4_ERR_INVALID_ARG;
    if (groups > kMaxGroups || K % 16 != 0 || total_rows > kMaxSize || N > kMaxSize || groups * N > kMaxSize ||
        K > kMaxSize)
        return QFP4_ERR_UNSUPPORTED;
    if (!aligned16(A) || !aligned16(B) || !aligned16(D) || !aligned4(A_sf) || !aligned4(B_sf) ||
        !aligned4(row_offsets))
        return QFP4_ERR_MISALIGNED;
    if (total_rows == 0) return QFP4_OK;
    if (max_group_rows > total_rows) max_group_rows = 0;        // no bound worth checking
    const Fp8Params p{static_cast<const uint8_t *>(A), static_cast<const uint8_t *>(B), A_sf, B_sf, D, row_offsets,
                      static_cast<int32_t>(total_rows), static_cast<int32_t>(N), static_cast<int32_t>(K),
                      static_cast<int32_t>(groups), static_cast<int32_t>(max_group_rows),
                      a_type, b_type, 128, out_type == QFP4_FP32, 0, 0, static_cast<int32_t>(total_rows)};
    return launch_gemm_fp8(p, static_cast<cudaStream_t>(stream));
}

extern "C" int qfp4_gemm_nt_fp8_kgrouped(int a_type, int b_type, int64_t groups, const int32_t *row_offsets,
                                         int64_t total_rows, int64_t M, int64_t N, const void *A, const float *A_sf,
                                         const void *B, const float *B_sf, int accumulate, float *D, void *stream)
{
    if (!types_ok(a_type, b_type, QFP4_FP32)) return QFP4_ERR_INVALID_ARG;
    if (groups < 1 || !row_offsets || total_rows < 0 || M < 0 || N < 0) return QFP4_ERR_INVALID_ARG;
    if (groups > kMaxGroups || total_rows > kMaxSize || M > kMaxSize || N > kMaxSize || groups * M > kMaxSize)
        return QFP4_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return QFP4_OK;            // empty D: nothing to do, nothing launched
    if (!D || !A || !A_sf || !B || !B_sf) return QFP4_ERR_INVALID_ARG;
    if (!aligned16(A) || !aligned16(B) || !aligned16(D) || !aligned4(A_sf) || !aligned4(B_sf) ||
        !aligned4(row_offsets))
        return QFP4_ERR_MISALIGNED;
    // K of the operands: every group's rows from a block of 128 of their own
    const int64_t K = static_cast<int64_t>(qfp4_fp8_grouped_cols(total_rows, groups));
    const Fp8Params p{static_cast<const uint8_t *>(A), static_cast<const uint8_t *>(B), A_sf, B_sf, D, row_offsets,
                      static_cast<int32_t>(M), static_cast<int32_t>(N), static_cast<int32_t>(K),
                      static_cast<int32_t>(groups), 0, a_type, b_type, 1, 1, accumulate ? 1 : 0, 0,
                      static_cast<int32_t>(total_rows)};
    return launch_gemm_fp8(p, static_cast<cudaStream_t>(stream));
}

#ifdef QFP4_FAULT_INJECTION
// Test build only (not declared in the public header): arm (1) or disarm (0)
// the missing releases of the 8-bit products.
extern "C" int qfp4_test_inject_fp8_skip_release(int on)
{
    if (cudaMemcpyToSymbol(qfp4::g_inject_fp8_pair, &on, sizeof(int)) != cudaSuccess) return QFP4_ERR_CUDA;
    return qfp4::set_inject_fp8_small(on);
}
#endif
