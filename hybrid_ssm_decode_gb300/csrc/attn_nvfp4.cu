// Paged attention over NVFP4 caches.
#include "attn_nvfp4.cuh"

namespace rssm {
namespace {

template <int D>
cudaError_t launch4(const AttnArgs& a, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
    using namespace attn;
    switch (rows) {
        case 8: return launch_shape<kNVFP4, Shape4<D, 1, 1>>(a, k, v, s);
        case 16: return launch_shape<kNVFP4, Shape4<D, 2, 1>>(a, k, v, s);
        case 32: return launch_shape<kNVFP4, Shape4<D, 2, 2>>(a, k, v, s);
        default:
            if constexpr (D == 256) return cudaErrorInvalidValue;
            else return launch_shape<kNVFP4, Shape4<D, 2, 4>>(a, k, v, s);
    }
}

}  // namespace

cudaError_t attn_launch_nvfp4(const AttnArgs& a, int D, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
    return D == 64 ? launch4<64>(a, rows, k, v, s) : D == 128 ? launch4<128>(a, rows, k, v, s) : launch4<256>(a, rows, k, v, s);
}

}  // namespace rssm
