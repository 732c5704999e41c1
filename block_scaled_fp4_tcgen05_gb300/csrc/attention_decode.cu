// attention_decode.cu -- entry points of the attention of one new token per
// sequence over the paged cache (kernel: qfp4_attention.cuh).
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "qfp4_attention.cuh"

namespace qfp4 {

__device__ uint32_t g_status_attention = 0;

int status_word_attention(uint32_t **word) { return status_word(g_status_attention, word); }

namespace {

constexpr size_t kCounterBytes = 16384;     // at the same place for all sizes
static_assert(3 * kAttnMaxCtas * sizeof(uint32_t) <= kCounterBytes, "three counters per CTA");

constexpr int64_t kMaxHeads = 4096, kMaxBatch = 1 << 20, kMaxLength = int64_t{1} << 30;

bool sizes_ok(int64_t B, int64_t q_heads, int64_t kv_heads, int64_t D)
{
    return (D == 64 || D == 128 || D == 256) && q_heads <= kMaxHeads && B <= kMaxBatch && q_heads % kv_heads == 0;
}

// Counters and two pieces for each CTA that the GPU holds at once.
size_t workspace_bytes(int64_t B, int64_t kv_heads, int64_t group, int D)
{
    const int nt = attn_tiles(group, D), queries = 8 * nt;
    const int ctas = 152 * attn_most_per_sm(B * kv_heads * ((group + queries - 1) / queries), nt);
    return kCounterBytes + static_cast<size_t>(ctas) * 2 * attn_piece_floats(queries, D) * sizeof(float);
}

}  // namespace
}  // namespace qfp4

using namespace qfp4;

extern "C" size_t qfp4_attention_decode_workspace_bytes(int64_t B, int64_t q_heads, int64_t kv_heads, int64_t head_dim)
{
    if (B < 0 || q_heads < 1 || kv_heads < 1 || !sizes_ok(B, q_heads, kv_heads, head_dim)) return 0;
    return workspace_bytes(B, kv_heads, q_heads / kv_heads, static_cast<int>(head_dim));
}

extern "C" int qfp4_attention_decode(int type, const void *Q_bf16, int64_t ldq, int64_t B, int64_t q_heads,
                                     int64_t kv_heads, int64_t head_dim, const void *cache, int64_t pages,
                                     int64_t page_size, const int32_t *page_table, int64_t max_pages,
                                     const int32_t *lengths, int64_t window, float scale, const float *gs_k,
                                     const float *gs_v, void *O_bf16, float *lse, void *workspace, size_t ws_bytes,
                                     void *stream)
{
    const float scale_log2 = scale * 1.44269504088896341f;
    if (!cache_type_ok(type) || B < 0 || q_heads < 1 || kv_heads < 1 || head_dim < 1 || pages < 0 || page_size < 1 ||
        max_pages < 0 || window < 0 || ldq < q_heads * head_dim || !std::isfinite(scale_log2))
        return QFP4_ERR_INVALID_ARG;
    if (!sizes_ok(B, q_heads, kv_heads, head_dim) || page_size % 16 != 0 || page_size > 16384 || pages > INT32_MAX ||
        max_pages > kMaxLength / page_size || ldq % 8 != 0)
        return QFP4_ERR_UNSUPPORTED;
    if (B == 0) return QFP4_OK;
    if (!Q_bf16 || !lengths || !O_bf16 || (max_pages > 0 && (!page_table || !cache || pages < 1)) ||
        (type == QFP4_CACHE_NVFP4 && (!gs_k || !gs_v)))
        return QFP4_ERR_INVALID_ARG;
    if (!aligned16(Q_bf16) || !aligned16(cache) || !aligned16(O_bf16) || !aligned16(workspace) ||
        !aligned4(page_table) || !aligned4(lengths) || !aligned4(gs_k) || !aligned4(gs_v) || !aligned4(lse))
        return QFP4_ERR_MISALIGNED;
    const int D = static_cast<int>(head_dim), nt = attn_tiles(q_heads / kv_heads, D);
    if (!workspace || ws_bytes < workspace_bytes(B, kv_heads, q_heads / kv_heads, D)) return QFP4_ERR_WORKSPACE;
    AttnParams p = {};
    p.q = static_cast<const __nv_bfloat16 *>(Q_bf16);
    p.ldq = ldq;
    p.B = static_cast<int32_t>(B);
    p.kv_heads = static_cast<int32_t>(kv_heads);
    p.group = static_cast<int32_t>(q_heads / kv_heads);
    p.blocks = (p.group + 8 * nt - 1) / (8 * nt);
    p.cache = static_cast<const uint8_t *>(cache);
    p.pages = pages;
    p.page_units = static_cast<int32_t>(page_size / 16);
    // exact for every unit of a sequence: fewer than 2^26 of them, at most 2^10 in a page
    p.page_magic = ((uint64_t{1} << 36) + p.page_units - 1) / p.page_units;
    p.max_pages = static_cast<int32_t>(max_pages);
    p.window = static_cast<int32_t>(window < kMaxLength ? window : 0);
    p.page_table = page_table;
    p.lengths = lengths;
    p.scale_log2 = scale_log2;
    p.gs_k = gs_k;
    p.gs_v = gs_v;
    p.out = static_cast<__nv_bfloat16 *>(O_bf16);
    p.lse = lse;
    p.counters = static_cast<uint32_t *>(workspace);
    p.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kCounterBytes);
    if (status_word_attention(&p.status) != QFP4_OK) return QFP4_ERR_CUDA;
#ifdef QFP4_FAULT_INJECTION
    p.skip_copy = inject_skip_copy();
#endif
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (type) {
    case QFP4_CACHE_BF16: return attn_launch_bf16(p, D, nt, s);
    case QFP4_CACHE_E4M3: return attn_launch_e4m3(p, D, nt, s);
    default: return attn_launch_nvfp4(p, D, nt, s);
    }
}

#ifdef QFP4_FAULT_INJECTION
namespace qfp4 {
static std::atomic<int> g_skip_copy{0};
bool inject_skip_copy() { return g_skip_copy.load() != 0; }
}  // namespace qfp4

extern "C" int qfp4_test_inject_skip_copy(int on)
{
    qfp4::g_skip_copy.store(on);
    return QFP4_OK;
}
#endif
