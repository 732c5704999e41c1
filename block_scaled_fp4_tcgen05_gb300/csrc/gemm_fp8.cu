// gemm_fp8.cu -- product of 8-bit floating point operands with one fp32 scale
// per 128 elements of K (see qfp4_gemm_nt_fp8).
//
// First form: 64 x 64 tiles on the CUDA cores, codes decoded to fp32 in shared
// memory, one block of 128 accumulated at a time and added under its scales.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "qfp4_common.cuh"
#include "sm103_ptx.cuh"

namespace qfp4 {

__device__ uint32_t g_status_gemm_fp8 = 0;

int read_clear_status_gemm_fp8(cudaStream_t s, uint32_t *out)
{
    uint32_t zero = 0;
    if (cudaMemcpyFromSymbolAsync(out, g_status_gemm_fp8, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, s) !=
        cudaSuccess)
        return QFP4_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return QFP4_ERR_CUDA;
    if (cudaMemcpyToSymbolAsync(g_status_gemm_fp8, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, s) !=
        cudaSuccess)
        return QFP4_ERR_CUDA;
    return cudaStreamSynchronize(s) == cudaSuccess ? QFP4_OK : QFP4_ERR_CUDA;
}

namespace {

constexpr int kMaxGroups = 256;
constexpr int64_t kMaxSize = int64_t{1} << 30;

struct Fp8Params {
    const uint8_t *A, *B;
    const float *A_sf, *B_sf;
    void *D;
    const int32_t *row_offsets;     // grouped: DEVICE [groups + 1]
    int32_t M, N, K;                // grouped: M = total_rows
    int32_t groups;                 // 0: dense
    int32_t max_group_rows;         // grouped: 0 = no bound
    int32_t a_type, b_type, b_rows;
    int32_t fp32, accumulate;
};

// Row offsets a grouped product can use: from 0, never decreasing, at most
// total_rows, no group above max_rows (0 = no bound).
__device__ __forceinline__ bool fp8_offsets_valid(const int32_t *offs, int groups, int32_t total_rows,
                                                  int32_t max_rows)
{
    if (offs[0] != 0 || offs[groups] > total_rows) return false;
    for (int e = 0; e < groups; ++e) {
        const int64_t rows = static_cast<int64_t>(offs[e + 1]) - offs[e];
        if (rows < 0 || (max_rows > 0 && rows > max_rows)) return false;
    }
    return true;
}

__device__ __forceinline__ float decode(uint8_t c, int type)
{
    __nv_fp8_storage_t v = c;
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, type == QFP4_E4M3 ? __NV_E4M3 : __NV_E5M2)));
}

__global__ void __launch_bounds__(256)
gemm_fp8_simple_kernel(const Fp8Params p)
{
    __shared__ float sa[32][65], sb[32][65];
    __shared__ int32_t s_row[3];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    if (tid == 0) {
        int32_t t = blockIdx.x, e = 0, lo = 0, hi = p.M;
        if (p.groups) {
            lo = hi = 0;
            if (!fp8_offsets_valid(p.row_offsets, p.groups, p.M, p.max_group_rows)) {
                if (blockIdx.x == 0 && blockIdx.y == 0)
                    atomicOr(&g_status_gemm_fp8, static_cast<uint32_t>(kStatusBadGroup));
            } else {
                for (; e < p.groups; ++e) {
                    const int32_t tiles = (p.row_offsets[e + 1] - p.row_offsets[e] + 63) / 64;
                    if (t < tiles) {
                        lo = p.row_offsets[e];
                        hi = p.row_offsets[e + 1];
                        break;
                    }
                    t -= tiles;
                }
            }
        }
        s_row[0] = lo + t * 64;
        s_row[1] = hi;
        s_row[2] = e;
    }
    __syncthreads();
    const int32_t m0 = s_row[0], m_end = s_row[1], e = s_row[2], n0 = blockIdx.y * 64;
    if (m0 >= m_end) return;
    const uint8_t *B = p.B + static_cast<int64_t>(e) * p.N * p.K;
    const int32_t kb = (p.K + 127) / 128;
    const float *B_sf = p.B_sf + static_cast<int64_t>(e) * ((p.N + 127) / 128) * kb;
    float acc[4][4] = {};
    for (int32_t b = 0; b < kb; ++b) {
        float part[4][4] = {};
        for (int k0 = b * 128; k0 < min(p.K, b * 128 + 128); k0 += 32) {
            __syncthreads();
            for (int f = tid; f < 64 * 32; f += 256) {
                const int r = f >> 5, k = k0 + (f & 31);
                sa[f & 31][r] = m0 + r < m_end && k < p.K ? decode(p.A[static_cast<int64_t>(m0 + r) * p.K + k], p.a_type) : 0.0f;
                sb[f & 31][r] = n0 + r < p.N && k < p.K ? decode(B[static_cast<int64_t>(n0 + r) * p.K + k], p.b_type) : 0.0f;
            }
            __syncthreads();
            for (int k = 0; k < 32; ++k)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j) part[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], part[i][j]);
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int32_t m = min(m0 + ty * 4 + i, p.M - 1), n = min(n0 + tx * 4 + j, p.N - 1);
                const float s = p.A_sf[static_cast<int64_t>(b) * p.M + m] *
                                (p.b_rows == 1 ? B_sf[static_cast<int64_t>(b) * p.N + n]
                                               : B_sf[static_cast<int64_t>(n / 128) * kb + b]);
                acc[i][j] = fmaf(s, part[i][j], acc[i][j]);
            }
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int32_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m >= m_end || n >= p.N) continue;
            const int64_t at = static_cast<int64_t>(m) * p.N + n;
            if (p.fp32) {
                float *d = static_cast<float *>(p.D) + at;
                *d = p.accumulate ? *d + acc[i][j] : acc[i][j];
            } else {
                static_cast<__nv_bfloat16 *>(p.D)[at] = __float2bfloat16_rn(acc[i][j]);
            }
        }
}

bool types_ok(int a_type, int b_type, int out_type)
{
    return (a_type == QFP4_E4M3 || a_type == QFP4_E5M2) && (b_type == QFP4_E4M3 || b_type == QFP4_E5M2) &&
           (out_type == QFP4_BF16 || out_type == QFP4_FP32);
}

int launch_gemm_fp8(const Fp8Params &p, cudaStream_t s)
{
    const int64_t tiles = (static_cast<int64_t>(p.M) + 63) / 64 + p.groups;
    const int64_t tiles_n = (static_cast<int64_t>(p.N) + 63) / 64;
    if (tiles_n > 65535) return QFP4_ERR_UNSUPPORTED;
    return launch_status(launch_pdl(gemm_fp8_simple_kernel,
                                    dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(tiles_n)), dim3(256), 0, s, p));
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
                      a_type, b_type, 128, out_type == QFP4_FP32, 0};
    return launch_gemm_fp8(p, static_cast<cudaStream_t>(stream));
}
