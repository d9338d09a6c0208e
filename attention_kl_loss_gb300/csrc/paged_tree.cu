// Attention of drafted tokens over the paged cache: each row sees the keys before
// the drafted ones and those of them whose bits its mask has (its own branch of a
// tree). The kernels are those of chunks and of few rows; a tile that holds
// drafted keys takes its visibility from the masks' bits.
#include "paged_attn.cuh"
#include "paged_decode.cuh"

namespace skl {

cudaError_t launch_tree_decode(const PagedAttnArgs& a, int ctas, cudaStream_t stream) {
  return launch_decode<true>(a, ctas, stream);
}

cudaError_t launch_tree_attn(const PagedAttnArgs& a, cudaStream_t stream) { return launch_attn<true>(a, stream); }

}  // namespace skl
