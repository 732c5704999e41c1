// attention_decode_e4m3.cu -- the attention of one new token over a cache of this
// type (see qfp4_attention.cuh), in a translation unit of its own.
#include "qfp4_attention.cuh"

namespace qfp4 {

int attn_launch_e4m3(const AttnParams &p, int D, int nt, cudaStream_t s)
{
    return attn_launch_type<QFP4_CACHE_E4M3>(p, D, nt, s);
}

}  // namespace qfp4
