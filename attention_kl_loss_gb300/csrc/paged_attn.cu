// Attention of chunks of new tokens over the paged cache (paged_attn.cuh).
#include "paged_attn.cuh"

namespace skl {

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t stream) { return launch_attn<false>(a, stream); }

}  // namespace skl
