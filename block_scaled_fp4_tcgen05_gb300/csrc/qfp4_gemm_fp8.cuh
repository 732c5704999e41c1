// qfp4_gemm_fp8.cuh -- what the 8-bit products' translation units share (not ABI).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace qfp4 {

constexpr int kMaxGroups = 256;

struct Fp8Params {
    const uint8_t *A, *B;
    const float *A_sf, *B_sf;
    void *D;
    const int32_t *row_offsets;     // grouped: DEVICE [groups + 1]
    int32_t M, N, K;                // grouped by rows: M = total_rows
    int32_t groups;                 // 0: dense; with b_rows = 1, grouped by blocks of K
    int32_t max_group_rows;         // grouped: 0 = no bound
    int32_t a_type, b_type, b_rows;
    int32_t fp32, accumulate;
    int32_t store_map;              // D can be written by TMA (rows 16-byte aligned)
    int32_t total_rows;             // grouped: what row_offsets may reach
};

// Row offsets a grouped product can use: from 0, never decreasing, at most
// total_rows, no group above max_rows (0 = no bound).  Group e's part of that.
__device__ __forceinline__ bool fp8_offsets_valid(const int32_t *offs, int e, int groups, int32_t total_rows,
                                                  int32_t max_rows)
{
    const int64_t rows = static_cast<int64_t>(offs[e + 1]) - offs[e];
    return (e > 0 || offs[0] == 0) && (e < groups - 1 || offs[groups] <= total_rows) && rows >= 0 &&
           (max_rows == 0 || rows <= max_rows);
}

// Small products (few tiles of 256 x 256): tiles of 128 rows of B x up to 128
// rows of A, K split over the CTAs of a cluster.
bool gemm_fp8_small_pays(const Fp8Params &p);
int launch_gemm_fp8_small(const Fp8Params &p, cudaStream_t s);
int status_word_gemm_fp8_small(uint32_t **word);
#ifdef QFP4_FAULT_INJECTION
int set_inject_fp8_small(int on);
#endif

}  // namespace qfp4
