// Attention of few new rows over the paged cache (paged_decode.cuh).
#include "paged_decode.cuh"

namespace skl {

cudaError_t launch_paged_decode(const PagedAttnArgs& a, int ctas, cudaStream_t stream) {
  return launch_decode<false>(a, ctas, stream);
}

}  // namespace skl
