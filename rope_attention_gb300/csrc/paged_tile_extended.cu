// The paged attention calls with a window or a shared prefix, for many rows per sequence and kv
// head (paged_tile.cuh).
#include "paged_tile.cuh"

namespace ra {

cudaError_t launch_paged_tile_extended(const PagedLaunch& L, cudaStream_t stream, const char** why) {
  return launch_tile_over_pages<true>(L, stream, why);
}

}  // namespace ra
