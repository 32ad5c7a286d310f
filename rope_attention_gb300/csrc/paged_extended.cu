// The paged attention calls with a window or a shared prefix: the choice of the kernel.
#include "paged_rows.cuh"

namespace ra {

cudaError_t launch_paged_extended(const PagedLaunch& L, cudaStream_t stream, const char** why) {
  if (paged_tile_serves(L)) return launch_paged_tile_extended(L, stream, why);
  if (paged_tokens_serves(L)) return launch_paged_tokens(L, stream, why);
  return launch_rows<true>(L, stream, why);
}

}  // namespace ra
