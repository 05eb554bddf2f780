// The attention kernel's instances for FP8 pages.
#include "attn.cuh"

namespace ci {
namespace attn {
cudaError_t launch_fp8(const CUtensorMap& kmap, const CUtensorMap& vmap, const Args& k, cudaStream_t s) {
  return launch_format<true>(kmap, vmap, k, s);
}
}  // namespace attn
}  // namespace ci
