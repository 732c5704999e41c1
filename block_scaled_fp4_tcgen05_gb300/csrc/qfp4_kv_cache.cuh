// qfp4_kv_cache.cuh -- the paged key-value cache's layout, shared by the kernels
// that write, read and attend over it (not ABI; the layout is, see qfp4.h).
//
// The cache is [pages][kv_heads][page_size / 16] units.  A unit holds 16 tokens
// of one head, one piece of memory that a single bulk copy brings to shared
// memory: K codes, K scales, V codes, V scales.  Codes lie in the order in
// which the lanes of a warp hold them as tensor-core operands (mma m16n8k16,
// lane = 4 g + t): token j of the unit is row j of the K operand (g = j % 8,
// two halves h = j / 8) and column j of V's (t = j % 8 / 2, e = j % 2).
#pragma once

#include <cstdint>

#include "qfp4_common.cuh"

namespace qfp4 {

constexpr int kUnitTokens = 16;

inline bool cache_type_ok(int type) { return type >= QFP4_CACHE_BF16 && type <= QFP4_CACHE_NVFP4; }

__host__ __device__ constexpr int cache_row_bytes(int type, int D)
{
    return type == QFP4_CACHE_BF16 ? 2 * D : type == QFP4_CACHE_E4M3 ? D : D / 2;
}

// scale bytes of one token
__host__ __device__ constexpr int cache_scale_bytes(int type, int D)
{
    return type == QFP4_CACHE_BF16 ? 0 : type == QFP4_CACHE_E4M3 ? 4 : D / 16;
}

__host__ __device__ constexpr int cache_unit_bytes(int type, int D)
{
    return 2 * kUnitTokens * (cache_row_bytes(type, D) + cache_scale_bytes(type, D));
}

struct CacheUnit {
    int row, scale, k_scales, v_codes, v_scales, bytes;

    __host__ __device__ constexpr CacheUnit(int type, int D)
        : row(cache_row_bytes(type, D)), scale(cache_scale_bytes(type, D)), k_scales(kUnitTokens * row),
          v_codes(kUnitTokens * (row + scale)), v_scales(kUnitTokens * (2 * row + scale)),
          bytes(cache_unit_bytes(type, D))
    {
    }
    // Byte x of token j's K row: pieces of 64 bytes (the row, where that is
    // shorter), those of eight tokens side by side.
    __host__ __device__ constexpr int k_code(int j, int x) const
    {
        const int piece = row < 64 ? row : 64;
        return ((j >> 3) * (row / piece) + x / piece) * 8 * piece + (j & 7) * piece + x % piece;
    }
    // Byte x of token j's V row: an eighth p of the row goes to the lanes with
    // g = p; lane (p, t) holds its four tokens' eighths one after the other, in
    // sixteens that lie side by side over the warp.
    __host__ __device__ constexpr int v_code(int j, int x) const
    {
        const int w = row / 8, at = ((j >> 3) * 2 + (j & 1)) * w + x % w;
        return v_codes + ((at >> 4) * 32 + 4 * (x / w) + ((j >> 1) & 3)) * 16 + (at & 15);
    }
    // NVFP4's scale byte of block b of token j
    __host__ __device__ constexpr int k_block_scale(int j, int b) const { return k_scales + j * scale + b; }
    __host__ __device__ constexpr int v_block_scale(int j, int b) const
    {
        return v_scales + b * 16 + ((j >> 1) & 3) * 4 + (j >> 3) * 2 + (j & 1);
    }
    // E4M3's fp32 scale of token j
    __host__ __device__ constexpr int k_token_scale(int j) const { return k_scales + 4 * j; }
    __host__ __device__ constexpr int v_token_scale(int j) const { return v_scales + 4 * j; }
};

}  // namespace qfp4
