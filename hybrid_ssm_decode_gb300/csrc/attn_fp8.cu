// Paged attention over FP8 (E4M3) caches.
#include "attn_decode.cuh"

namespace rssm {

cudaError_t attn_launch_fp8(const AttnArgs& a, int D, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
    return attn::launch_dim<attn::kFP8>(a, D, rows, k, v, s);
}

}  // namespace rssm
