// qfp4_gemm_fp8.cuh -- what the 8-bit products' translation units share (not ABI).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace qfp4 {

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
    int32_t store_map;              // D can be written by TMA (rows 16-byte aligned)
};

// Small products (few tiles of 256 x 256): tiles of 128 rows of B x up to 128
// rows of A, K split over the CTAs of a cluster.  Dense only.
bool gemm_fp8_small_pays(const Fp8Params &p);
int launch_gemm_fp8_small(const Fp8Params &p, cudaStream_t s);
int read_clear_status_gemm_fp8_small(cudaStream_t s, uint32_t *out);

}  // namespace qfp4
