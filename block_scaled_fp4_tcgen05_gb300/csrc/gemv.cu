// gemv.cu -- up to 16 BF16 rows times 4-bit weights with block scales:
//   D[m,n] = gs_w * sum_k x[m,k] * w[n,k],  w = E2M1(W) * SF,
// the weights packed and their scales in the MMA layout as qfp4_gemm_nt's B.
//
// Bound by the weights' bytes.  A warp takes 16 rows of W as the rows of tensor
// core products (m16n8k16) whose columns are the rows of x.  The codes become FP16
// exactly; NVFP4's scales join them there (a product of E2M1 and UE4M3 has at most
// 6 significant bits), MXFP4's powers of two multiply the fp32 sums of a block, so
// that their whole range counts.  x becomes FP16 in shared memory, each row of a
// slice of K multiplied by the power of two that takes its largest element there to
// [2^8, 2^9): an element loses bits only 2^22 below that, 2^-33 of the largest at
// most.
//
// One CTA of 16 warps per SM, and one wave of them: the groups of 16 rows are dealt
// out over the clusters, K over the CTAs of a cluster, so that a CTA converts its
// part of x once and its warps stream their rows without a pause: each brings its own
// rows and scales with 16-byte asynchronous copies into a ring of stages, 256 elements
// of K per stage, across the groups' borders.  ldmatrix gives a lane eight
// neighbouring codes of a block.  The cluster's sums are added through distributed
// shared memory in a fixed order: results repeat bit for bit.
//
// Measured with the weights in HBM: 1 x 14336 x 4096 10.1 us (floor 4.9), 1 x 28672 x
// 8192 27 us (19.5); more weights add 0.9 of the copy bandwidth, so what is above the
// floor is the call's beginning and end, about 5 us.  Nine rows of x and more double
// the products and bind it by instructions: 16 x 28672 x 8192 41 us (NVFP4), 43 us
// (MXFP4), 1.9 a cycle.  Other forms, 16 and 1 rows of that size (MXFP4): CTAs of eight
// warps and 128 rows with the CTA's slice of x converted for each 52 and 38 us; the
// weights by TMA in stages of 128 rows 56 and 43; the line of groups and K shared
// evenly between the warps 47 and 30 (more work around each stage); a group's K shared
// by several warps 51 and 31.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qfp4_common.cuh"
#include "qfp4_fp4_codes.cuh"
#include "qfp4_lane_ops.cuh"
#include "sm103_ptx.cuh"

namespace qfp4 {

namespace {

using namespace lane_ops;

constexpr int kStep = 128;              // elements of K that the scales' layout and K go by
constexpr int kUnit = 256, kUnitSteps = 2;              // elements of K of a stage
constexpr int kSlice = 512, kSliceUnits = 2;            // of x with a scale of their own
constexpr int kRowSlices = 64;          // slices of rows of x in shared memory at once
constexpr int kGroups = 48;             // groups of 16 rows whose sums are
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

// NT: blocks of eight rows of x
template <int FMT, int NT>
struct GemvCfg {
    static constexpr int COLS4 = FMT == QFP4_NVFP4 ? 2 : 1;         // tiles of four scale columns per step
    static constexpr int ROWS = 16 * kUnit / 2, STAGE = ROWS + kUnitSteps * COLS4 * 64;
    // 24 warps of 80 registers are no faster than 16 (1 x 28672 x 8192: 32 us, 29 at that
    // time), nor 12 of 168 (16 x 28672 x 8192 MXFP4: 46 us, 44)
    static constexpr int WARPS = 16, THREADS = 32 * WARPS, STAGES = 3;
    static constexpr int PITCH = (kSlice + 32) * 2;                 // bytes of a row of x: two rows fall on different halves of the banks
    static constexpr int RING = WARPS * STAGES * STAGE;
    static constexpr int X = kRowSlices * PITCH, BACK = (kRowSlices + 8 * NT) * 4;
    static constexpr int SUMS = 8 * NT * 16;                        // of a group: [row of x][row of W]
    static constexpr int OUT = kGroups * SUMS * 4;
    static constexpr int SMEM = RING + X + BACK + OUT;
    static_assert(SMEM <= 227 * 1024, "one CTA per SM");
};

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

__device__ __forceinline__ void mma_f16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Whether the bytes of a and b all lie in 64..191 (their two top bits differ).
__device__ __forceinline__ bool all_middling(uint32_t a, uint32_t b)
{
    return ((a ^ a << 1) & (b ^ b << 1) & 0x80808080u) == 0x80808080u;
}

template <int FMT, int NT>
__global__ void __launch_bounds__(GemvCfg<FMT, NT>::THREADS, 1) gemv_kernel(const GemvParams p, const int splits)
{
    using C = GemvCfg<FMT, NT>;
    constexpr int STAGES = C::STAGES, COLS4 = C::COLS4, SUMS = C::SUMS, WARPS = C::WARPS, THREADS = C::THREADS;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rank = blockIdx.x % splits, cluster = blockIdx.x / splits, clusters = gridDim.x / splits;
    // this CTA's part of K, in units
    const int steps_all = p.K / kStep, units_all = (steps_all + 1) / 2;
    const int unit0 = static_cast<int>(static_cast<int64_t>(rank) * units_all / splits);
    const int units = static_cast<int>(static_cast<int64_t>(rank + 1) * units_all / splits) - unit0;
    uint8_t *xs = smem + C::RING;
    float *s_back = reinterpret_cast<float *>(xs + C::X);           // [slice][row of x]
    float *s_out = reinterpret_cast<float *>(xs + C::X + C::BACK);  // [group][row of x][row of W]

    // The cluster's groups of 16 rows.  Group q is part q % 8 of the scales' tile
    // q / 8, its row lr row 4 (q % 8) + lr % 4 + 32 (lr / 4) there: its scales then
    // lie together, 64 bytes per tile of four columns.
    const int all = (p.N + 127) / 128 * 8;
    const int q0 = static_cast<int>(static_cast<int64_t>(cluster) * all / clusters);
    const int q1 = static_cast<int>(static_cast<int64_t>(cluster + 1) * all / clusters);

    // a pass over K: what of x lies in shared memory at once
    const int most = kRowSlices / p.M * kSliceUnits;
    auto pass_units = [&](int u0) { return min(most, units - u0); };

    // ---- the ring's producer.  Lane copies chunk lane % 8 of rows lane / 8 + 4 j;
    // chunk c of row r goes to place c ^ r % 8, so that the eight rows of an ldmatrix
    // fall on all banks.
    const int64_t row_bytes = p.K / 2;
    // It stands at a unit of group in_q, in the pass over K from
    // in_u0 and over kGroups groups from in_base; in_left units of the group are left.
    int in_base = q0, in_u0 = 0, in_q = q0 + warp, in_left = 0, in_last = 0, stage_in = 0;
    const uint8_t *src[4] = {}, *sf = nullptr;
    auto open = [&] {       // the group in_q, or the next that there is for this warp
        while (in_q >= min(q1, in_base + kGroups)) {
            if ((in_u0 += most) >= units) {
                in_u0 = 0;
                if ((in_base += kGroups) >= q1) return;
            }
            in_q = in_base + warp;
        }
        const int tile = in_q >> 3, part = in_q & 7, unit = unit0 + in_u0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = min(tile * 128 + 4 * part + (lane >> 3) + 32 * j, p.N - 1);
            src[j] = p.w + row * row_bytes + static_cast<int64_t>(unit) * (kUnit / 2) + 16 * (lane & 7);
        }
        sf = p.sf + (static_cast<int64_t>(tile) * steps_all + 2 * unit) * (512 * COLS4) + 64 * part + (lane >> 2) * 512 + (lane & 3) * 16;
        in_left = pass_units(in_u0);
        // steps of the group's last unit: one where K ends in the middle of it
        in_last = min(2, steps_all - 2 * (unit + in_left - 1));
    };
    const uint32_t ring = smem_u32(smem) + warp * STAGES * C::STAGE;
    const uint32_t dst = ring + (lane >> 3) * 128;
    const uint32_t place0 = ((lane & 7) ^ (lane >> 3)) << 4, place1 = ((lane & 7) ^ ((lane >> 3) + 4)) << 4;
    auto issue = [&] {
        if (in_left > 0) {
            const uint32_t off = stage_in * C::STAGE;
            const bool both = in_left > 1 || in_last > 1;
            if (both || (lane & 7) < 4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) cp_async16(dst + off + j * 512 + (j & 1 ? place1 : place0), src[j]);
            }
            if (lane < (both ? 8 : 4) * COLS4) cp_async16(ring + off + C::ROWS + lane * 16, sf);
#pragma unroll
            for (int j = 0; j < 4; ++j) src[j] += kUnit / 2;
            sf += 2 * 512 * COLS4;
            if (--in_left == 0) {
                in_q += WARPS;
                open();
            }
        }
        if (++stage_in == STAGES) stage_in = 0;
        cp_async_commit();
    };
    pdl_wait();
    pdl_launch_dependents();
    if (units > 0) open();
#pragma unroll 1
    for (int i = 0; i < STAGES - 1; ++i) issue();

    // ---- x, [slice][row]: a warp converts a slice of a row at a time
    auto convert = [&](int u0, int n) {
#pragma unroll 1
        for (int i = warp; i < p.M * n; i += WARPS) {
            const int m = i % p.M, sl = i / p.M;
            const int64_t k0 = static_cast<int64_t>(unit0 + u0) * kUnit + sl * kSlice;
            const int64_t end = min(static_cast<int64_t>(p.K), static_cast<int64_t>(unit0 + units) * kUnit);
            uint4 v[kSlice / 256];
            float amax = 0.0f;
#pragma unroll
            for (int j = 0; j < kSlice / 256; ++j) {
                const int64_t k = k0 + 256 * j + 8 * lane;
                v[j] = make_uint4(0, 0, 0, 0);
                if (k < end) v[j] = __ldg(reinterpret_cast<const uint4 *>(p.x + m * p.ldx + k));
            }
#pragma unroll
            for (int j = 0; j < kSlice / 256; ++j) {
                const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[u] << 16)), fabsf(__uint_as_float(w[u] & 0xFFFF0000u))));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            // an infinity takes everything beside it into FP16's range, so that it alone counts
            const int e = min(126, 8 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127));
            const float up = pow2(e);
            if (lane == 0) s_back[sl * p.M + m] = pow2(-e);
#pragma unroll
            for (int j = 0; j < kSlice / 256; ++j) {
                const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
                uint32_t h[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) h[u] = pack_f16(__uint_as_float(w[u] << 16) * up, __uint_as_float(w[u] & 0xFFFF0000u) * up);
                *reinterpret_cast<uint4 *>(xs + (sl * p.M + m) * C::PITCH + (256 * j + 8 * lane) * 2) = make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
    };

    // this lane's row of an ldmatrix and the chunk that it starts from, swizzled
    const uint32_t rows_at = ring + (lane & 15) * 128, chunk_x = static_cast<uint32_t>((lane >> 4) ^ (lane & 7)) << 4;
    const uint8_t *sf_at = smem + warp * STAGES * C::STAGE + C::ROWS + (g & 3) * 16 + (g >> 2) * 4;
    const float gs = p.gs ? *p.gs : 1.0f;
    int stage = 0;
#pragma unroll 1
    for (int base = q0; base < q1; base += kGroups) {
        const int groups = min(kGroups, q1 - base);
#pragma unroll 1
        for (int u0 = 0; u0 < units; u0 += most) {
            const int n_units = pass_units(u0);
            if (base == q0 || units > most) {        // else x is there from the groups before
                if (u0 > 0) __syncthreads();
                convert(u0, (n_units + 1) / 2);
                __syncthreads();
            }
#pragma unroll 1
            for (int group = warp; group < groups; group += WARPS) {
                // pairs of sums: columns 2t and 2t + 1 of rows g (0) and g + 8 (1)
                uint64_t acc[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = 0;
#pragma unroll 1
                for (int slice = 0; slice * kSliceUnits < n_units; ++slice) {
                    // of the slice, whose x has one scale: for NVFP4 a chain of products for
                    // each step of a unit; MXFP4's blocks are chains of their own (one sum
                    // and packed fp32 44 us for 16 x 28672 x 8192, two sums 46)
                    constexpr int SUMS_OF = FMT == QFP4_NVFP4 ? 2 : 1;
                    float sum[SUMS_OF][NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) sum[0][n][k] = sum[SUMS_OF - 1][n][k] = 0.0f;
                    const uint8_t *xb = xs + (slice * p.M + g) * C::PITCH + 16 * t;      // rows that x does not have: columns that nobody reads
                    const int last = min(kSliceUnits, n_units - slice * kSliceUnits);
#pragma unroll 1
                    for (int unit = 0; unit < last; ++unit, xb += 2 * kUnit) {
                        cp_async_wait<STAGES - 2>();
                        __syncwarp();
                        const uint32_t rows = rows_at + stage * C::STAGE;
                        const uint8_t *sfs = sf_at + stage * C::STAGE;
                        const bool both = 2 * (unit0 + u0 + slice * kSliceUnits + unit) + 1 < steps_all;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            if (s == 1 && !both) break;
                            uint32_t code[2][4];        // [pair of chunks][rows 0..7 and 8..15 of the first, of the second]
                            uint32_t sw[COLS4][2];      // four columns' scales of rows g and g + 8
#pragma unroll
                            for (int c2 = 0; c2 < 2; ++c2) ldmatrix_x4(code[c2], rows + (chunk_x ^ ((4 * s + 2 * c2) << 4)));
#pragma unroll
                            for (int c4 = 0; c4 < COLS4; ++c4)
#pragma unroll
                                for (int h = 0; h < 2; ++h) sw[c4][h] = *reinterpret_cast<const uint32_t *>(sfs + (s * COLS4 + c4) * 64 + h * 8);
                            float f[4][2];      // MXFP4: the chunks' scales of rows g and g + 8
                            if (FMT == QFP4_MXFP4) {
                                // the exponent field of 2^(byte - 127); 0 and 255 are not that, and are
                                // looked for beyond 2^-63 and 2^64 only
#pragma unroll
                                for (int c = 0; c < 4; ++c)
#pragma unroll
                                    for (int h = 0; h < 2; ++h)
                                        f[c][h] = __uint_as_float((c == 3 ? sw[0][h] >> 1 : sw[0][h] << (23 - 8 * c)) & 0x7F800000u);
                                if (!__all_sync(0xffffffffu, all_middling(sw[0][0], sw[0][1]))) {
#pragma unroll
                                    for (int c = 0; c < 4; ++c)
#pragma unroll
                                        for (int h = 0; h < 2; ++h) f[c][h] = ue8m0(sw[0][h] >> (8 * c) & 255u);
                                }
                            }
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                uint4 x[NT];
#pragma unroll
                                for (int n = 0; n < NT; ++n) x[n] = *reinterpret_cast<const uint4 *>(xb + n * 8 * C::PITCH + (s * kStep + 32 * c) * 2);
                                const uint32_t w0 = code[c >> 1][2 * (c & 1)], w1 = code[c >> 1][2 * (c & 1) + 1];
                                uint32_t a[2][4] = {{fp4x2<0>(w0), fp4x2<0>(w1), fp4x2<1>(w0), fp4x2<1>(w1)},
                                                    {fp4x2<2>(w0), fp4x2<2>(w1), fp4x2<3>(w0), fp4x2<3>(w1)}};
                                if constexpr (FMT == QFP4_NVFP4) {
                                    // this lane's codes belong to block 2 c + t / 2: its scales of rows g and g + 8
                                    const uint32_t sel = 2 * (c & 1) + (t >> 1);
                                    const uint32_t two = fp8x2<0>(__byte_perm(sw[c >> 1][0], sw[c >> 1][1], sel | (sel + 4) << 4));
                                    const uint32_t sg = __byte_perm(two, 0, 0x1010), sh = __byte_perm(two, 0, 0x3232);
#pragma unroll
                                    for (int u = 0; u < 2; ++u) {
                                        a[u][0] = mul_f16x2(a[u][0], sg);
                                        a[u][1] = mul_f16x2(a[u][1], sh);
                                        a[u][2] = mul_f16x2(a[u][2], sg);
                                        a[u][3] = mul_f16x2(a[u][3], sh);
                                    }
#pragma unroll
                                    for (int n = 0; n < NT; ++n) {
                                        mma_f16(sum[s % SUMS_OF][n], a[0], x[n].x, x[n].y);
                                        mma_f16(sum[s % SUMS_OF][n], a[1], x[n].z, x[n].w);
                                    }
                                } else {
#pragma unroll
                                    for (int n = 0; n < NT; ++n) {
                                        float block[4];
                                        mma_f16_zero(block, a[0], x[n].x, x[n].y);
                                        mma_f16(block, a[1], x[n].z, x[n].w);
                                        float *d = sum[0][n];
                                        const uint64_t lo = f2_fma(f2_pack(f[c][0], f[c][0]), f2_pack(block[0], block[1]), f2_pack(d[0], d[1]));
                                        const uint64_t hi = f2_fma(f2_pack(f[c][1], f[c][1]), f2_pack(block[2], block[3]), f2_pack(d[2], d[3]));
                                        f2_unpack(lo, d[0], d[1]);
                                        f2_unpack(hi, d[2], d[3]);
                                    }
                                }
                            }
                        }
                        __syncwarp();
                        issue();        // into the stage that was read last time round
                        if (++stage == STAGES) stage = 0;
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float *b = s_back + slice * p.M + 8 * n + 2 * t;
                        const uint64_t b2 = f2_pack(b[0], b[1]);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint64_t v = f2_pack(sum[0][n][2 * h], sum[0][n][2 * h + 1]);
                            if constexpr (SUMS_OF == 2) v = f2_add(v, f2_pack(sum[1][n][2 * h], sum[1][n][2 * h + 1]));
                            acc[n][h] = f2_fma(v, b2, acc[n][h]);
                        }
                    }
                }
                // this lane's places of the group's sums: its own in every pass over K
                float *out = s_out + group * SUMS + 2 * t * 16 + g;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float v0, v1;
                        f2_unpack(acc[n][h], v0, v1);
                        float *there = out + n * 8 * 16 + 8 * h;
                        there[0] = u0 > 0 ? there[0] + v0 : v0;
                        there[16] = u0 > 0 ? there[16] + v1 : v1;
                    }
            }
        }
        if (units == 0)
            for (int i = tid; i < groups * SUMS; i += THREADS) s_out[i] = 0.0f;
        // ---- the cluster's sums: row by row of the scales' tiles
        if (splits > 1) cluster_sync_all();
        else __syncthreads();
        const int tile0 = base >> 3, tiles = ((base + groups - 1) >> 3) - tile0 + 1;
        for (int i = tid + rank * THREADS; i < p.M * tiles * 128; i += THREADS * splits) {
            const int r = i & 127, rest = i >> 7, tile = tile0 + rest % tiles, m = rest / tiles;
            const int q = tile * 8 + (r & 31) / 4 - base, lr = (r & 3) + 4 * (r >> 5), row = tile * 128 + r;
            if (q < 0 || q >= groups || row >= p.N) continue;
            const float *there = s_out + q * SUMS + m * 16 + lr;
            float v = 0.0f;
            if (splits == 1) {
                v = *there;
            } else {
                // NVFP4: all on their way before the first is added (16 x 14336 x 4096 15.4 us,
                // 15.9 one at a time); MXFP4's loop has no registers left for that (16 x 28672
                // x 8192 45 us, 43.4 one at a time)
                if constexpr (FMT == QFP4_NVFP4) {
                    float part[kMaxSplits];
#pragma unroll
                    for (int k = 0; k < kMaxSplits; ++k) part[k] = k < splits ? ld_cluster_f32(mapa_shared(smem_u32(there), k)) : 0.0f;
#pragma unroll
                    for (int k = 0; k < kMaxSplits; ++k) v += part[k];
                } else {
                    for (int k = 0; k < splits; ++k) v += ld_cluster_f32(mapa_shared(smem_u32(there), k));
                }
            }
            p.d[m * p.ldd + row] = __float2bfloat16_rn(v * gs);
        }
        if (splits > 1) cluster_sync_all();     // a CTA's sums stay until the others have read them
        else __syncthreads();
    }
    cp_async_wait<0>();
}

// Clusters of so many CTAs that the GPU holds at once, asked once; 0: none.
template <int FMT, int NT>
int clusters_at_once(int splits)
{
    static std::atomic<int> known[kMaxSplits + 1];
    int n = known[splits].load(std::memory_order_relaxed);
    if (n > 0) return n - 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(152 / splits * splits);
    cfg.blockDim = dim3(GemvCfg<FMT, NT>::THREADS);
    cfg.dynamicSmemBytes = GemvCfg<FMT, NT>::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (splits == 1) {
        n = sm_count();
    } else if (cudaOccupancyMaxActiveClusters(&n, gemv_kernel<FMT, NT>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    known[splits].store(n + 1, std::memory_order_relaxed);
    return n;
}

template <int FMT, int NT>
int launch(const GemvParams &p, cudaStream_t s)
{
    using C = GemvCfg<FMT, NT>;
    auto kernel = gemv_kernel<FMT, NT>;
    const int rc = ensure_smem_attr(reinterpret_cast<const void *>(kernel), C::SMEM);
    if (rc != QFP4_OK) return rc;
    // The split of K whose busiest CTA has the least to do, counted in units: a
    // group's part of K, the chain of the busiest warp (four times as long each), the
    // join (as long as 12), and a pause for x (24).
    const int64_t groups = (static_cast<int64_t>(p.N) + 127) / 128 * 8, units = (p.K + kUnit - 1) / kUnit;
    const int64_t most = kRowSlices / p.M * kSliceUnits;
    int splits = 0, clusters = 0;
    int64_t best = 0;
    for (int n = 1; n <= kMaxSplits && (n == 1 || units >= n); ++n) {
        const int64_t c = std::min<int64_t>(clusters_at_once<FMT, NT>(n), groups);
        if (c < 1) continue;
        const int64_t per = (groups + c - 1) / c, part = (units + n - 1) / n;
        const int64_t joins = (per + kGroups - 1) / kGroups, passes = part > most ? joins * ((part + most - 1) / most) : 1;
        const int64_t cost = per * part + (per + C::WARPS - 1) / C::WARPS * part * 4 + 12 * joins * (n > 1) + 24 * (passes - 1);
        if (splits == 0 || cost < best) {
            best = cost;
            splits = n;
            clusters = static_cast<int>(c);
        }
    }
    if (splits == 0) return QFP4_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * splits));
    cfg.blockDim = dim3(GemvCfg<FMT, NT>::THREADS);
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

template <int FMT>
int launch_any(const GemvParams &p, cudaStream_t s)
{
    return p.M <= 8 ? launch<FMT, 1>(p, s) : launch<FMT, 2>(p, s);
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
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return fmt == QFP4_NVFP4 ? launch_any<QFP4_NVFP4>(p, s) : launch_any<QFP4_MXFP4>(p, s);
}
