// gemm_fp8_small.cu -- the product of gemm_fp8.cu for few rows of A (decoding
// tokens, short prompts), where 256 x 256 tiles would leave most SMs idle and
// the weights' bytes bound the time.
//
// A CTA (tcgen05 cta_group::1) takes one tile.  Up to 32 rows of A (NT): swap
// AB, 128 rows of B in the MMA's M slot and the tokens in its N slot, D^T.
// More: 128 rows of A in the M slot and 128 of B in the N slot; a thread's
// block sums then share one scale, where the swapped form needs one per token
// from shared memory, whose bandwidth the wider MMAs use up (128 tokens x
// 14336 x 4096: 1500 cycles per K block swapped, twice the streaming time).
// K is split over the S CTAs of a cluster, each streaming its own K blocks
// through a ring; as in gemm_fp8.cu the block sums leave tensor memory (two
// slots) for registers.  At the end every CTA leaves its sums in its shared
// memory, the cluster meets, and CTA r adds up tokens r, r + S, ... over the S
// CTAs in order (the results repeat bit for bit, and no scratch in global
// memory is needed).
//
// The weights' bytes are the floor.  One token x 14336 x 4096 takes 11.8 us
// (4.9 TB/s) and 4096 x 4096 5.8 (5.1 from L2); 128 tokens x 14336 x 4096 15.7
// (4.0 TB/s; 14.2 with the weights in L2).  There a CTA's pace, about 0.31 us
// per K block, and the 112 CTAs on 152 SMs bound it: 152 of them (N = 19456)
// take the same time.  Grouped, 8 experts x 14336 x 4096, with a bound on the
// groups' rows: 72 us with 2 rows each (6.5 TB/s), 73 with 16, 98 with 48 (and
// with 16 where no bound says so).
//
// Warps: 0 TMA producer, 1 and 3 MMA issuers (1 owns tensor memory), 2 scales,
// 4.. epilogue (four of all columns, or sixteen of 32 each).
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "qfp4_common.cuh"
#include "qfp4_gemm_fp8.cuh"
#include "qfp4_gemm_internal.cuh"
#include "sm103_ptx.cuh"

namespace qfp4 {

__device__ uint32_t g_status_gemm_fp8_small = 0;

#ifdef QFP4_FAULT_INJECTION
// Test build only: one epilogue warp of the first CTA never gives back the
// slot of its first K block.
__device__ int g_inject_fp8_small = 0;
__device__ __forceinline__ bool inject_skip(bool here) { return here && g_inject_fp8_small != 0; }
int set_inject_fp8_small(int on)
{
    return cudaMemcpyToSymbol(g_inject_fp8_small, &on, sizeof(int)) == cudaSuccess ? QFP4_OK : QFP4_ERR_CUDA;
}
#else
__device__ __forceinline__ bool inject_skip(bool) { return false; }
#endif

int status_word_gemm_fp8_small(uint32_t **word) { return status_word(g_status_gemm_fp8_small, word); }

namespace {

constexpr int kMaxSplits = 8;       // CTAs of a cluster (the portable limit)
constexpr int kBatch = 8;           // K blocks per hand-over of scales

template <int NT>
struct SmallCfg {
    static constexpr bool SWAP = NT < 128;                      // rows of B in the MMA's M slot
    static constexpr int GROUPS = SWAP ? 1 : NT / 32;           // column groups of the epilogue
    static constexpr int EPI = 4 * GROUPS;                      // epilogue warps
    static constexpr int THREADS = 128 + 32 * EPI;
    static constexpr int COLS = NT / GROUPS;                    // columns per epilogue warp
    static constexpr int CTAS = SWAP ? 2 : 1;                   // resident CTAs per SM that the ring is sized for
    static constexpr int M_BYTES = 128 * 128;                   // the M slot's 128 rows x 128 elements of K
    static constexpr int STAGE = M_BYTES + NT * 128;
    static constexpr int STAGES = 5;
    static constexpr int SCALES = 128 + NT;                     // floats per K block: the M slot's rows, then the N slot's
    static constexpr int OFF_SCALE = STAGES * STAGE;
    static constexpr int OFF_BAR = OFF_SCALE + 2 * kBatch * SCALES * 4;
    static constexpr int NBAR = 2 * STAGES + 4 + 4;             // full, empty; acc_full, acc_empty [2]; sc_full, sc_empty [2]
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
    static constexpr int TMEM_COLS = 2 * NT < 32 ? 32 : 2 * NT;
    static_assert(NT * 128 * 4 <= OFF_SCALE, "the sums must fit in the ring");
    static_assert(CTAS * (SMEM + 1024) <= 233472, "shared memory overflow");
};

__device__ __forceinline__ void record_timeout()
{
    atomicOr(&g_status_gemm_fp8_small, static_cast<uint32_t>(kStatusTimeout));
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// PER_ROW: B has one scale per row (b_rows = 1), else one per 128 rows.
// GROUPED: one product per expert, each with its own tiles of up to max_rows
// rows; a CTA (a whole cluster) whose tile its expert does not reach leaves at
// once.
// tmM, tmN: maps of the operands in the MMA's M and N slots.
template <int NT, bool PER_ROW, bool GROUPED>
__global__ void __launch_bounds__(SmallCfg<NT>::THREADS, SmallCfg<NT>::CTAS)
gemm_fp8_small_kernel(const __grid_constant__ CUtensorMap tmM, const __grid_constant__ CUtensorMap tmN,
                      const Fp8Params p, const int splits, const int32_t max_rows)
{
    using C = SmallCfg<NT>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *empty = full + C::STAGES;
    uint64_t *acc_full = empty + C::STAGES;
    uint64_t *acc_empty = acc_full + 2;
    uint64_t *sc_full = acc_empty + 2;
    uint64_t *sc_empty = sc_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sc_empty + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int32_t tiles_n = (p.N + 127) / 128;
    const int32_t tile = blockIdx.x / splits;
    const int32_t n0 = (tile % tiles_n) * 128;
    // rows [m0, m_end) of A, and where B's row and block n0 lie
    int32_t m0 = (tile / tiles_n) * NT, m_end = p.M, group = 0;
    if (GROUPED) {
        const int32_t tiles_m = (max_rows + NT - 1) / NT;
        group = tile / (tiles_n * tiles_m);
        m0 = (tile / tiles_n % tiles_m) * NT;
        pdl_wait();
        const bool bad = __syncthreads_or(threadIdx.x < p.groups &&
                                          !fp8_offsets_valid(p.row_offsets, threadIdx.x, p.groups, p.total_rows, p.max_group_rows));
        if (bad && threadIdx.x == 0 && blockIdx.x == 0)
            atomicOr(&g_status_gemm_fp8_small, static_cast<uint32_t>(kStatusBadGroup));
        m0 += p.row_offsets[group];
        m_end = p.row_offsets[group + 1];
        if (bad || m0 >= m_end) return;
    }
    const int32_t wrow = group * p.N + n0;
    const float *b_sf = p.B_sf + (PER_ROW ? 0 : (static_cast<int64_t>(group) * tiles_n + n0 / 128) * ((p.K + 127) / 128));
    const int32_t kblocks = (p.K + 127) / 128;
    const int32_t kb0 = static_cast<int32_t>(static_cast<int64_t>(rank) * kblocks / splits);
    const int32_t nkb = static_cast<int32_t>(static_cast<int64_t>(rank + 1) * kblocks / splits) - kb0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&acc_full[b]), 1);
            mbar_init(smem_u32(&acc_empty[b]), C::EPI);
            mbar_init(smem_u32(&sc_full[b]), 32);
            mbar_init(smem_u32(&sc_empty[b]), C::EPI);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmM);
        prefetch_tensormap(&tmN);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    if (!GROUPED) pdl_wait();
    pdl_launch_dependents();

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            uint32_t s = 0, phase = 1;
            bool ok = true;
            for (int32_t j = 0; j < nkb; ++j) {
                if (!mbar_wait(smem_u32(&empty[s]), phase)) { ok = false; break; }
                const uint32_t bar = smem_u32(&full[s]), dst = smem_u32(smem + s * C::STAGE);
                mbar_arrive_expect_tx(bar, C::STAGE);
                tma_load_2d(dst, &tmM, bar, (kb0 + j) * 128, C::SWAP ? wrow : m0);
                tma_load_2d(dst + C::M_BYTES, &tmN, bar, (kb0 + j) * 128, C::SWAP ? m0 : wrow);
                if (++s == C::STAGES) { s = 0; phase ^= 1; }
            }
            if (!ok) { record_timeout(); *abort_flag = 1; }
        }
    } else if (warp == 1 || warp == 3) {
        // ------------------------------------------------ MMA issuers: warp 1 sums the even K blocks into slot
        // 0, warp 3 the odd ones into slot 1, so that one looks at its barriers while the other's MMAs run
        const uint32_t slot = warp >> 1;
        const uint64_t m_desc0 = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
        const uint64_t n_desc0 = smem_desc(smem_u32(smem) + C::M_BYTES, 16, 1024, kSwizzle128B);
        const uint32_t idesc = C::SWAP ? idesc_f8(128, NT, p.b_type, p.a_type) : idesc_f8(128, NT, p.a_type, p.b_type);
        uint32_t s = slot, phase = 0, acc_phase = 1;
        bool ok = true;
        for (int32_t j = slot; j < nkb; j += 2) {
            if (!mbar_wait_warp(smem_u32(&full[s]), phase) || !mbar_wait_warp(smem_u32(&acc_empty[slot]), acc_phase)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (elect_one_sync()) {
                const uint64_t md = m_desc0 + s * static_cast<uint64_t>(C::STAGE >> 4);
                const uint64_t nd = n_desc0 + s * static_cast<uint64_t>(C::STAGE >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc_mma_f8(tmem_base + slot * NT, md + 2 * kk, nd + 2 * kk, idesc, kk > 0 ? 1u : 0u);
                tc_commit(smem_u32(&acc_full[slot]));
                tc_commit(smem_u32(&empty[s]));
            }
            __syncwarp();
            acc_phase ^= 1;
            s += 2;
            if (s >= C::STAGES) { s -= C::STAGES; phase ^= 1; }
        }
        if (!ok && lane == 0) { record_timeout(); *abort_flag = 1; }
    } else if (warp == 2) {
        // ------------------------------------------------ scales, kBatch K blocks at a time: A's rows and B's
        // rows (or B's one block) where the slot that holds them expects its own
        constexpr int kAt = C::SWAP ? 512 : 0, kBt = C::SWAP ? 0 : 512;      // byte offsets in a K block's scales
        constexpr int kArows = C::SWAP ? NT : 128, kBrows = C::SWAP ? 128 : NT;
        uint32_t b = 0, phase = 1;
        bool ok = true;
        for (int32_t j0 = 0; j0 < nkb; j0 += kBatch) {
            if (!mbar_wait_warp(smem_u32(&sc_empty[b]), phase)) { ok = false; break; }
            const uint32_t dst0 = smem_u32(smem + C::OFF_SCALE) + b * (kBatch * C::SCALES * 4);
            for (int u = 0; u < kBatch && j0 + u < nkb; ++u) {
                const int64_t kb = kb0 + j0 + u;
                const uint32_t dst = dst0 + u * (C::SCALES * 4) + lane * 4;
#pragma unroll
                for (int i = 0; i < (kArows + 31) / 32; ++i)
                    if (32 * i + lane < kArows)
                        cp_async4(dst + kAt + 128 * i, p.A_sf + kb * p.M + min(m0 + lane + 32 * i, p.M - 1));
                if (PER_ROW) {
#pragma unroll
                    for (int i = 0; i < kBrows / 32; ++i)
                        cp_async4(dst + kBt + 128 * i, p.B_sf + kb * p.N + min(n0 + lane + 32 * i, p.N - 1));
                } else if (lane == 0) {
                    cp_async4(dst + kBt, b_sf + kb);
                }
            }
            cp_async_arrive(smem_u32(&sc_full[b]));
            b ^= 1;
            if (b == 0) phase ^= 1;
        }
        if (!ok && lane == 0) { record_timeout(); *abort_flag = 1; }
    } else if (warp >= 4) {
        // ------------------------------------------------ epilogue: 32 rows of the M slot x COLS columns per warp
        const int quad = warp & 3, c0 = ((warp - 4) >> 2) * C::COLS;
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + c0;
        constexpr int kLd = C::COLS < 32 ? 16 : 32;             // columns per load
        constexpr bool kColumns = C::SWAP || PER_ROW;           // the N slot has a scale per column
        float acc[C::COLS];
#pragma unroll
        for (int i = 0; i < C::COLS; ++i) acc[i] = 0.0f;
        uint32_t slot = 0, phase = 0, b = 0, sc_phase = 0;
        int u = 0;
        bool ok = true, ready = false;      // ready: the next slot's sum is known to be complete
        for (int32_t j = 0; j < nkb; ++j) {
            if (u == 0 && !mbar_wait_warp(smem_u32(&sc_full[b]), sc_phase)) { ok = false; break; }
            const float *sc = reinterpret_cast<const float *>(smem + C::OFF_SCALE) + (b * kBatch + u) * C::SCALES;
            if (!ready && !mbar_wait_warp(smem_u32(&acc_full[slot]), phase)) { ok = false; break; }
            tc_fence_after();
            uint32_t v[C::COLS / kLd][kLd];
#pragma unroll
            for (int c = 0; c < C::COLS / kLd; ++c) {
                if constexpr (kLd == 16) tmem_ld_32x32b_x16(taddr + slot * NT, v[c]);
                else tmem_ld_32x32b_x32(taddr + slot * NT + c * 32, v[c]);
            }
            float row = sc[C::SWAP && !PER_ROW ? 0 : quad * 32 + lane];
            if (!kColumns) row = row * sc[128];
            bool done = false;
#pragma unroll
            for (int c = 0; c < C::COLS / kLd; ++c) {
                // the columns' scales (the first ones while the loads are under way)
                float q[kLd];
                if constexpr (kColumns) {
#pragma unroll
                    for (int i = 0; i < kLd; i += 4) {
                        const float4 four = *reinterpret_cast<const float4 *>(sc + 128 + c0 + c * kLd + i);
                        q[i] = four.x; q[i + 1] = four.y; q[i + 2] = four.z; q[i + 3] = four.w;
                    }
                }
                if (c == 0) {
                    tmem_ld_wait();
#pragma unroll
                    for (int d = 0; d < C::COLS / kLd; ++d) tmem_regs_after_wait(v[d]);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0 && !inject_skip(blockIdx.x == 0 && warp == 4 && j == 0))
                        mbar_arrive(smem_u32(&acc_empty[slot]));
                    slot ^= 1;
                    if (slot == 0) phase ^= 1;
                    done = mbar_test(smem_u32(&acc_full[slot]), phase);
                }
                if constexpr (kColumns) {
                    // the column's scale meets the sum first, the row's the result: their product alone need
                    // not be a normal number where the term is one.  It costs nothing (100 rows x 4096 x 4096
                    // with a scale per row 9.7 us, 11.0 with the scales multiplied ahead of the loads' end)
#pragma unroll
                    for (int i = 0; i < kLd; i += 2) {
                        float lo, hi;
                        unpack_f32x2(mul_f32x2(pack_b32x2(v[c][i], v[c][i + 1]), pack_f32x2(q[i], q[i + 1])), lo, hi);
                        v[c][i] = __float_as_uint(lo);
                        v[c][i + 1] = __float_as_uint(hi);
                    }
                }
#pragma unroll
                for (int i = 0; i < kLd; ++i) acc[c * kLd + i] = fmaf(row, __uint_as_float(v[c][i]), acc[c * kLd + i]);
            }
            ready = __all_sync(0xffffffffu, done);
            if (++u == kBatch || j == nkb - 1) {
                u = 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sc_empty[b]));
                b ^= 1;
                if (b == 0) sc_phase ^= 1;
            }
        }
        if (!ok && lane == 0) { record_timeout(); *abort_flag = 1; }
        // The last block's MMAs have read the ring and every copy into it was
        // waited for by one of them: it now takes the sums, 128 columns of D
        // per token.  Swapped, a thread holds one column of every token;
        // else a part of one token's row, in 16-byte pieces whose place is
        // turned by the token so that a warp's pieces do not collide.
        if (ok) {
            if (C::SWAP) {
                float *red = reinterpret_cast<float *>(smem) + quad * 32 + lane;
#pragma unroll
                for (int i = 0; i < C::COLS; ++i) red[i * 128] = acc[i];
            } else {
                float4 *red = reinterpret_cast<float4 *>(smem) + (quad * 32 + lane) * 32;
#pragma unroll
                for (int i = 0; i < C::COLS / 4; ++i)
                    red[(c0 / 4 + i) ^ lane] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    if (splits > 1) cluster_sync_all(); else __syncthreads();
    if (*abort_flag) {
        // let copies and MMAs already in flight drain before the memory goes
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) { }
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
    // a CTA that gave up leaves undefined sums; the status word says so
    const int32_t tokens = min(NT, m_end - m0);
    const int32_t n = n0 + 4 * lane;
    for (int32_t t = rank + splits * warp; t < tokens; t += splits * (C::THREADS / 32)) {
        const uint32_t piece = (t * 32 + (C::SWAP ? lane : lane ^ (t & 31))) * 16;
        float4 a;
        if (splits == 1) {
            a = *reinterpret_cast<const float4 *>(smem + piece);
        } else {
            // all CTAs' pieces on their way, then added in order
            float4 o[kMaxSplits];
#pragma unroll
            for (int q = 0; q < kMaxSplits; ++q)
                if (q < splits) o[q] = ld_cluster_v4(mapa_shared(smem_u32(smem) + piece, q));
            a = o[0];
#pragma unroll
            for (int q = 1; q < kMaxSplits; ++q)
                if (q < splits) a = make_float4(a.x + o[q].x, a.y + o[q].y, a.z + o[q].z, a.w + o[q].w);
        }
        const float o[4] = {a.x, a.y, a.z, a.w};
        const int64_t at = static_cast<int64_t>(m0 + t) * p.N + n;
        if (p.fp32) {
            float *d = static_cast<float *>(p.D) + at;
            if (p.N % 4 == 0) {
                if (n < p.N) {
                    if (p.accumulate) {
                        const float4 old = *reinterpret_cast<const float4 *>(d);
                        a = make_float4(a.x + old.x, a.y + old.y, a.z + old.z, a.w + old.w);
                    }
                    *reinterpret_cast<float4 *>(d) = a;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < p.N) d[i] = p.accumulate ? o[i] + d[i] : o[i];
            }
        } else {
            __nv_bfloat16 *d = static_cast<__nv_bfloat16 *>(p.D) + at;
            if (p.N % 4 == 0) {
                if (n < p.N) {
                    __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y), hi = __floats2bfloat162_rn(a.z, a.w);
                    *reinterpret_cast<uint2 *>(d) = make_uint2(*reinterpret_cast<uint32_t *>(&lo),
                                                               *reinterpret_cast<uint32_t *>(&hi));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < p.N) d[i] = __float2bfloat16_rn(o[i]);
            }
        }
    }
    // no CTA may leave while another still reads its sums
    __syncwarp();
    if (splits > 1) cluster_sync_all();
}

template <int NT, bool PER_ROW, bool GROUPED>
int launch(const Fp8Params &p, int64_t tiles, int splits, int32_t max_rows, cudaStream_t s)
{
    using C = SmallCfg<NT>;
    auto kern = gemm_fp8_small_kernel<NT, PER_ROW, GROUPED>;
    CUtensorMap mm, mn;
    int rc = ensure_smem_attr(reinterpret_cast<const void *>(kern), C::SMEM);
    const uint64_t b_rows = static_cast<uint64_t>(GROUPED ? p.groups : 1) * p.N;
    if (rc == QFP4_OK) rc = make_map_direct(C::SWAP ? &mm : &mn, p.B, p.K, b_rows, 128, 128);
    if (rc == QFP4_OK) rc = make_map_direct(C::SWAP ? &mn : &mm, p.A, p.K, p.M, 128, NT);
    if (rc != QFP4_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    return launch_status(cudaLaunchKernelEx(&cfg, kern, mm, mn, p, splits, max_rows));
}

template <int NT>
int launch_nt(const Fp8Params &p, int64_t tiles, int splits, int32_t max_rows, cudaStream_t s)
{
    if (p.groups) return launch<NT, false, true>(p, tiles, splits, max_rows, s);
    return p.b_rows == 1 ? launch<NT, true, false>(p, tiles, splits, max_rows, s)
                         : launch<NT, false, false>(p, tiles, splits, max_rows, s);
}

// Rows of A (of any group) that the launch has to cover.
int64_t most_rows(const Fp8Params &p)
{
    return p.groups && p.max_group_rows > 0 && p.max_group_rows < p.M ? p.max_group_rows : p.M;
}

// Clusters of `splits` CTAs of the 128 x 128 form that the current device holds
// at once (0 where it cannot say), asked once per device and size.
int clusters_at_once(int splits)
{
    static std::atomic<int> known[64][kMaxSplits + 1];      // the answer + 1
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    const int seen = known[dev][splits].load(std::memory_order_relaxed);
    if (seen > 0) return seen - 1;
    using C = SmallCfg<128>;
    const void *kern = reinterpret_cast<const void *>(gemm_fp8_small_kernel<128, false, false>);
    int n = 0;
    if (ensure_smem_attr(kern, C::SMEM) == QFP4_OK) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(splits);
        cfg.blockDim = dim3(C::THREADS);
        cfg.dynamicSmemBytes = C::SMEM;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = static_cast<unsigned>(splits);
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
            n = 0;
            cudaGetLastError();
        }
    }
    known[dev][splits].store(n + 1, std::memory_order_relaxed);
    return n;
}

struct Plan {
    int nt, splits;
    int64_t tiles;
};

// K is split while each CTA keeps two K blocks or more and the CTAs run at
// once.  128 x 128: one per SM, and the clusters have to fit as such (16 of
// eight do not: 128 x 2048 x 2048 took 12.8 us with eight splits, 6.4 with
// four).  Few rows: a second CTA per SM pays with eight K blocks for each (1 x
// 7168 x 4096 6.4 us in 224 CTAs, 6.9 in 112; 1 x 4096 x 4096 5.4 us in 256, 5.1
// in 128).
Plan plan(const Fp8Params &p)
{
    const int64_t rows = most_rows(p), sms = sm_count();
    Plan r;
    r.nt = rows <= 16 ? 16 : rows <= 32 ? 32 : 128;
    r.tiles = static_cast<int64_t>((p.N + 127) / 128) * ((rows + r.nt - 1) / r.nt) * (p.groups ? p.groups : 1);
    r.splits = 1;
    const int64_t kblocks = (static_cast<int64_t>(p.K) + 127) / 128;
    while (r.splits < kMaxSplits && kblocks >= 4 * r.splits) {
        const int64_t ctas = r.tiles * 2 * r.splits;
        if (r.nt == 128 ? ctas > sms || r.tiles > clusters_at_once(2 * r.splits)
                        : ctas > (kblocks >= 16 * r.splits ? 2 * sms : sms))
            break;
        r.splits *= 2;
    }
    return r;
}

}  // namespace

// Up to 32 rows always (per group, as far as the host can tell).  Up to 128 but
// for many tiles of a short K, whose beginnings and ends the pairs' persistent
// loop hides; with a longer K the pairs' tiles, half of them padding, lose.  Both
// forms over K = 512, 1024, 1536, 2048, 2560, 4096 (us, here / pairs):
//   128 x 40960 (2.1 rounds)   13.9/12.3  18.2/17.9  22.0/22.6  25.9/27.9  33.9/35.8  46.4/52.3
//   128 x 65536 (3.4)          18.7/15.4  25.1/22.8  34.4/32.4  39.9/39.5  46.4/47.5  63.3/68.5
//   128 x 98304 (5.1)          27.8/20.9  42.1/33.8  50.0/45.3  57.7/55.7  67.7/67.8  92.8/99.8
//   64 groups of 128 x 2048    44.5/31.6  56.8/46.2  66.9/61.0  76.9/75.6  89.3/92.3  121/141
//   64 groups of 48 x 2048     36.8/33.1  51.9/48.4  61.7/62.4  71.5/75.9  82.9/91.4  114/139
//   8 groups of 128 x 8192     22.1/18.8  28.7/26.4             43.9/44.7  50.4/53.1  67.6/76.1
// The two are even near K = 2048 from three rounds on (fewer rows a little
// earlier); with two rounds the pairs gain little anywhere.
// More than 128 where K is split: a CTA then has half the K blocks of a pair's
// 256 x 128 tile (256 x 4096 x 14336 takes 23 us here and 34 there).  Unsplit the
// pair is as fast or faster (512 x 4096 x 14336 39 us here, 35 there; fp32 with
// column scales 76 and 54).
bool gemm_fp8_small_pays(const Fp8Params &p)
{
    const int64_t rows = most_rows(p);
    if (rows <= 32) return true;
    const Plan r = plan(p);
    if (rows <= 128) return r.tiles <= 3 * sm_count() || p.K > 16 * 128;
    return !p.groups && r.splits > 1;
}

int launch_gemm_fp8_small(const Fp8Params &p, cudaStream_t s)
{
    const Plan plan = qfp4::plan(p);
    if (plan.tiles > INT32_MAX / kMaxSplits) return QFP4_ERR_UNSUPPORTED;
    const int64_t rows = most_rows(p), tiles = plan.tiles;
    const int nt = plan.nt, splits = plan.splits;
    const int32_t max_rows = static_cast<int32_t>(rows);
    switch (nt) {
    case 16: return launch_nt<16>(p, tiles, splits, max_rows, s);
    case 32: return launch_nt<32>(p, tiles, splits, max_rows, s);
    default: return launch_nt<128>(p, tiles, splits, max_rows, s);
    }
}

}  // namespace qfp4
