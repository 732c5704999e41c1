// gemv.cu -- up to 16 BF16 rows times 4-bit weights with block scales:
//   D[m,n] = gs_w * sum_k x[m,k] * w[n,k],  w = E2M1(W) * SF,
// the weights packed and their scales in the MMA layout as qfp4_gemm_nt's B.
//
// Bound by the weights' bytes.  A CTA takes 128 rows of W (one tile of the
// scales' layout), each of its eight warps 16 of them as the rows of a tensor
// core product (m16n8k16) whose columns are the rows of x.  The codes become
// FP16 exactly; NVFP4's scales join them there (a product of E2M1 and UE4M3 has
// at most 6 significant bits), MXFP4's powers of two multiply the fp32 sums of a
// block, so that their whole range counts.  x becomes FP16 in shared memory,
// each row of a slice of K multiplied by the power of two that takes its largest
// element there to [2^8, 2^9): an element loses bits only 2^22 below that,
// 2^-34 of the largest at most.
//
// A warp brings its own rows and scales with 16-byte asynchronous copies into a
// ring of stages of its own, 128 elements of K per stage, and waits for no other
// warp but where a slice of x ends.  ldmatrix gives a lane eight neighbouring
// codes of a block.  K is split over the CTAs of a cluster, whose sums are added
// through distributed shared memory in a fixed order: results repeat bit for bit.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qfp4_attention.cuh"
#include "qfp4_common.cuh"
#include "sm103_ptx.cuh"

namespace qfp4 {

namespace {

using namespace attn;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kRows = 128;              // rows of W per CTA
constexpr int kStep = 128;              // elements of K per stage
constexpr int kStages = 8;
constexpr int kSlice = 1024;            // elements of K of x in shared memory at once
constexpr int kMaxRowsX = 16, kMaxSplits = 8;

struct GemvParams {
    const __nv_bfloat16 *x;     // [M, K]
    int64_t ldx;
    const uint8_t *w;           // [N, K / 2]
    const uint8_t *sf;          // MMA layout
    const float *gs;            // or NULL
    __nv_bfloat16 *d;           // [M, N]
    int64_t ldd;
    int32_t M, N, K;
};

template <int FMT, int NT>
struct GemvCfg {
    static constexpr int SF = FMT == QFP4_NVFP4 ? 128 : 64;         // scale bytes of a warp's stage
    static constexpr int STAGE = 16 * kStep / 2 + SF;
    static constexpr int PITCH = (kSlice + 32) * 2;                 // bytes of a row of x: two rows fall on different halves of the banks
    static constexpr int RING = kWarps * kStages * STAGE;
    static constexpr int X = 8 * NT * PITCH;
    static constexpr int OUT = 8 * NT * (kRows + 4) * 4;            // the CTA's sums, over the ring
    static constexpr int SMEM = RING + X + 8 * NT * 4;
    static_assert(OUT <= RING, "the sums take the ring's place");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// 2^(c - 127); NaN for 255
__device__ __forceinline__ float ue8m0(uint32_t c)
{
    return __uint_as_float(c == 255u ? 0x7FFFFFFFu : c == 0u ? 0x00400000u : c << 23);
}

template <int FMT, int NT>
__global__ void __launch_bounds__(kThreads) gemv_kernel(const GemvParams p, const int splits)
{
    using C = GemvCfg<FMT, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rank = blockIdx.x % splits, tile = blockIdx.x / splits;
    const int row0 = tile * kRows;
    const int steps_all = p.K / kStep;
    const int step0 = static_cast<int>(static_cast<int64_t>(rank) * steps_all / splits);
    const int steps = static_cast<int>(static_cast<int64_t>(rank + 1) * steps_all / splits) - step0;
    const uint32_t ring = smem_u32(smem) + warp * kStages * C::STAGE;
    uint8_t *xs = smem + C::RING;
    float *s_back = reinterpret_cast<float *>(smem + C::RING + C::X);

    // A warp's row lr is row 4 warp + lr % 4 + 32 (lr / 4) of the tile: its scales
    // then lie together, 64 bytes per tile of four columns.  Lane copies rows
    // lane / 4 and 8 more, chunk lane % 4 of each; chunk c of row r goes to place
    // c ^ (r / 2 % 4), so that the eight rows of an ldmatrix fall on all banks.
    const uint8_t *src[2];
    uint32_t dst[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int lr = 8 * h + g;
        const int row = min(row0 + 4 * warp + (lr & 3) + 32 * (lr >> 2), p.N - 1);
        src[h] = p.w + (static_cast<int64_t>(row) * p.K + static_cast<int64_t>(step0) * kStep) / 2 + 16 * t;
        dst[h] = ring + lr * 64 + ((t ^ (lr >> 1 & 3)) << 4);
    }
    constexpr int COLS4 = FMT == QFP4_NVFP4 ? 2 : 1;        // tiles of four scale columns per step
    const uint8_t *sf = p.sf + (static_cast<int64_t>(tile) * steps_all + step0) * (512 * COLS4) + 64 * warp + (lane >> 2) * 512 + (lane & 3) * 16;
    const bool sf_lane = lane < 4 * COLS4;
    const uint32_t sf_dst = ring + 1024 + lane * 16;
    auto issue = [&](int step, int stage) {
        if (step < steps) {
#pragma unroll
            for (int h = 0; h < 2; ++h) cp_async16(dst[h] + stage * C::STAGE, src[h] + step * (kStep / 2));
            if (sf_lane) cp_async16(sf_dst + stage * C::STAGE, sf + static_cast<int64_t>(step) * (512 * COLS4));
        }
        cp_async_commit();
    };
    pdl_wait();
    pdl_launch_dependents();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i, i);

    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[n][k] = 0.0f;

    int stage = 0;
    for (int s0 = 0; s0 < steps; s0 += kSlice / kStep) {
        const int n_steps = min(kSlice / kStep, steps - s0), width = n_steps * kStep;
        // ---- this slice of x: a warp converts rows warp and warp + 8
        if (s0 > 0) __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int m = 8 * n + warp;
            uint4 v[kSlice / 256];
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < kSlice / 256; ++i) {
                const int k = 256 * i + 8 * lane;
                v[i] = make_uint4(0, 0, 0, 0);
                if (m < p.M && k < width)
                    v[i] = __ldg(reinterpret_cast<const uint4 *>(p.x + m * p.ldx + static_cast<int64_t>(step0 + s0) * kStep + k));
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xFFFF0000u))));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            int e = 8 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127);
            e = amax == 0.0f || !(amax < 3.4e38f) ? 0 : max(-126, min(126, e));
            const float up = pow2(e);
            if (lane == 0) s_back[m] = pow2(-e);
#pragma unroll
            for (int i = 0; i < kSlice / 256; ++i) {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) h[j] = pack_f16(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xFFFF0000u) * up);
                *reinterpret_cast<uint4 *>(xs + m * C::PITCH + (256 * i + 8 * lane) * 2) = make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
        __syncthreads();
        float part[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) part[n][k] = 0.0f;
#pragma unroll 1
        for (int s = 0; s < n_steps; ++s) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            const uint32_t buf = ring + stage * C::STAGE;
            const int next = stage == 0 ? kStages - 1 : stage - 1;
            uint32_t code[2][4];        // [pair of chunks][rows 0..7 and 8..15 of the first, of the second]
#pragma unroll
            for (int c2 = 0; c2 < 2; ++c2) {
                const int lr = lane & 15, c = 2 * c2 + (lane >> 4);
                ldmatrix_x4(code[c2], buf + lr * 64 + ((c ^ (lr >> 1 & 3)) << 4));
            }
            uint32_t sw[COLS4][2];      // four columns' scales of rows g and g + 8
#pragma unroll
            for (int c4 = 0; c4 < COLS4; ++c4)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    sw[c4][h] = *reinterpret_cast<const uint32_t *>(smem + (buf - smem_u32(smem)) + 1024 + c4 * 64 + (g & 3) * 16 + ((g >> 2) + 2 * h) * 4);
            uint4 xb[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    xb[n][c] = *reinterpret_cast<const uint4 *>(xs + (8 * n + g) * C::PITCH + (s * kStep + 32 * c + 8 * t) * 2);
            __syncwarp();
            // the stage read last time round is free: its loads were waited for above
            issue(s0 + s + kStages - 1, next);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t w0 = code[c >> 1][2 * (c & 1)], w1 = code[c >> 1][2 * (c & 1) + 1];
                uint32_t a[2][4] = {{fp4x2<0>(w0), fp4x2<0>(w1), fp4x2<1>(w0), fp4x2<1>(w1)},
                                    {fp4x2<2>(w0), fp4x2<2>(w1), fp4x2<3>(w0), fp4x2<3>(w1)}};
                if constexpr (FMT == QFP4_NVFP4) {
                    // this lane's codes belong to block 2 c + t / 2: its scales of rows g and g + 8
                    const uint32_t sel = 2 * (c & 1) + (t >> 1);
                    const uint32_t both = fp8x2<0>(__byte_perm(sw[c >> 1][0], sw[c >> 1][1], sel | (sel + 4) << 4));
                    const uint32_t sg = __byte_perm(both, 0, 0x1010), sh = __byte_perm(both, 0, 0x3232);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        a[u][0] = mul_f16x2(a[u][0], sg);
                        a[u][1] = mul_f16x2(a[u][1], sh);
                        a[u][2] = mul_f16x2(a[u][2], sg);
                        a[u][3] = mul_f16x2(a[u][3], sh);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_f16(part[n], a[0], xb[n][c].x, xb[n][c].y);
                        mma_f16(part[n], a[1], xb[n][c].z, xb[n][c].w);
                    }
                } else {
                    const float sg = ue8m0(sw[0][0] >> (8 * c) & 255u), sh = ue8m0(sw[0][1] >> (8 * c) & 255u);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma_f16(sum, a[0], xb[n][c].x, xb[n][c].y);
                        mma_f16(sum, a[1], xb[n][c].z, xb[n][c].w);
                        part[n][0] = fmaf(sg, sum[0], part[n][0]);
                        part[n][1] = fmaf(sg, sum[1], part[n][1]);
                        part[n][2] = fmaf(sh, sum[2], part[n][2]);
                        part[n][3] = fmaf(sh, sum[3], part[n][3]);
                    }
                }
            }
            if (++stage == kStages) stage = 0;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float b0 = s_back[8 * n + 2 * t], b1 = s_back[8 * n + 2 * t + 1];
            acc[n][0] = fmaf(part[n][0], b0, acc[n][0]);
            acc[n][1] = fmaf(part[n][1], b1, acc[n][1]);
            acc[n][2] = fmaf(part[n][2], b0, acc[n][2]);
            acc[n][3] = fmaf(part[n][3], b1, acc[n][3]);
        }
    }
    // ---- the CTA's sums by row of x, then the cluster's
    cp_async_wait<0>();
    __syncthreads();
    constexpr int PITCH = kRows + 4;
    float *out = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int lr = g + 8 * (k >> 1), r = 4 * warp + (lr & 3) + 32 * (lr >> 2);
            out[(8 * n + 2 * t + (k & 1)) * PITCH + r] = acc[n][k];
        }
    if (splits > 1) cluster_sync_all();
    else __syncthreads();
    const float gs = p.gs ? *p.gs : 1.0f;
    // rank takes its share of the rows of W
    const int share = kRows / splits, first = rank * share;
    for (int i = tid; i < p.M * share; i += kThreads) {
        const int m = i / share, r = first + i % share;
        if (row0 + r >= p.N) continue;
        float v = 0.0f;
        if (splits == 1) {
            v = out[m * PITCH + r];
        } else {
            const uint32_t at = smem_u32(out + m * PITCH + r);
            for (int q = 0; q < splits; ++q) v += ld_cluster_f32(mapa_shared(at, q));
        }
        p.d[m * p.ldd + row0 + r] = __float2bfloat16_rn(v * gs);
    }
    if (splits > 1) cluster_sync_all();     // a CTA's sums stay until the others have read them
}

template <int FMT, int NT>
int launch(const GemvParams &p, int64_t tiles, int splits, cudaStream_t s)
{
    using C = GemvCfg<FMT, NT>;
    auto kernel = gemv_kernel<FMT, NT>;
    const int rc = ensure_smem_attr(reinterpret_cast<const void *>(kernel), C::SMEM);
    if (rc != QFP4_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits));
    cfg.blockDim = dim3(kThreads);
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
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, p, splits));
}

// K is split while the CTAs do not fill the GPU three times over and each keeps
// two steps.
int plan_splits(int64_t tiles, int64_t steps)
{
    int splits = 1;
    while (splits < kMaxSplits && tiles * splits < 3 * sm_count() && steps >= 4 * splits) splits *= 2;
    return splits;
}

}  // namespace
}  // namespace qfp4

using namespace qfp4;

extern "C" int qfp4_gemv_nt(int fmt, int64_t M, int64_t N, int64_t K, const void *X_bf16, int64_t ldx,
                            const void *W_packed, const void *W_sf, const float *gs_w, void *D_bf16, int64_t ldd,
                            void *stream)
{
    if ((fmt != QFP4_MXFP4 && fmt != QFP4_NVFP4) || M < 0 || N < 0 || K < 0 || ldx < K || ldd < N)
        return QFP4_ERR_INVALID_ARG;
    if (M > kMaxRowsX || K % 128 != 0 || ldx % 8 != 0 || N > (int64_t{1} << 30) || K > (int64_t{1} << 30))
        return QFP4_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return QFP4_OK;
    if (!D_bf16 || (K > 0 && (!X_bf16 || !W_packed || !W_sf))) return QFP4_ERR_INVALID_ARG;
    if (!aligned16(X_bf16) || !aligned16(W_packed) || !aligned16(W_sf) || !aligned4(gs_w) ||
        (reinterpret_cast<uintptr_t>(D_bf16) & 1u))
        return QFP4_ERR_MISALIGNED;
    const GemvParams p{static_cast<const __nv_bfloat16 *>(X_bf16), ldx, static_cast<const uint8_t *>(W_packed),
                       static_cast<const uint8_t *>(W_sf), fmt == QFP4_NVFP4 ? gs_w : nullptr,
                       static_cast<__nv_bfloat16 *>(D_bf16), ldd, static_cast<int32_t>(M), static_cast<int32_t>(N),
                       static_cast<int32_t>(K)};
    const int64_t tiles = (N + kRows - 1) / kRows;
    const int splits = plan_splits(tiles, K / kStep);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (fmt == QFP4_NVFP4) return M <= 8 ? launch<QFP4_NVFP4, 1>(p, tiles, splits, s) : launch<QFP4_NVFP4, 2>(p, tiles, splits, s);
    return M <= 8 ? launch<QFP4_MXFP4, 1>(p, tiles, splits, s) : launch<QFP4_MXFP4, 2>(p, tiles, splits, s);
}
