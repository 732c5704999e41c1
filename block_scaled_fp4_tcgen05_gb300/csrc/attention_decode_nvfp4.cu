// attention_decode_nvfp4.cu -- the attention of one new token over a cache of this
// type (see qfp4_attention.cuh), in a translation unit of its own.
#include "qfp4_attention.cuh"

namespace qfp4 {

int attn_launch_nvfp4(const AttnParams &p, int D, int nt, cudaStream_t s)
{
    return attn_launch_type<QFP4_CACHE_NVFP4>(p, D, nt, s);
}

}  // namespace qfp4
