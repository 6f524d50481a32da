// Paged attention over FP32 caches.
#include "attn_decode.cuh"

namespace rssm {

cudaError_t attn_launch_f32(const AttnArgs& a, int D, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
    return attn::launch_dim<attn::kF32>(a, D, rows, k, v, s);
}

}  // namespace rssm
