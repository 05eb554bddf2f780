// Attention of drafted rows over an FP8 cache.
#include "attn_draft.cuh"

namespace ci {
namespace draft {
cudaError_t launch_fp8(const CUtensorMap& kmap, const CUtensorMap& vmap, const Args& k, cudaStream_t stream) {
  const int d = k.a.c.head_dim;
  return d == 64    ? launch_config<Config<64, true>>(kmap, vmap, k, stream)
         : d == 128 ? launch_config<Config<128, true>>(kmap, vmap, k, stream)
                    : launch_config<Config<256, true>>(kmap, vmap, k, stream);
}
}  // namespace draft
}  // namespace ci
