// attention_decode_bf16.cu -- the attention of one new token over a cache of this
// type (see qfp4_attention.cuh), in a translation unit of its own.
#include "qfp4_attention.cuh"

namespace qfp4 {

int attn_launch_bf16(const AttnParams &p, int D, int nt, cudaStream_t s)
{
    return attn_launch_type<QFP4_CACHE_BF16>(p, D, nt, s);
}

}  // namespace qfp4
