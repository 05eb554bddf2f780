// The attention kernel's instances for bf16 pages.
#include "attn.cuh"

namespace ci {
namespace attn {
cudaError_t launch_bf16(const CUtensorMap& kmap, const CUtensorMap& vmap, const Args& k, cudaStream_t s) {
  return launch_format<false>(kmap, vmap, k, s);
}
}  // namespace attn
}  // namespace ci
