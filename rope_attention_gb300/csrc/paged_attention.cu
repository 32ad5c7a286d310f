// paged_attention: the choice of its kernel (paged_rows.cuh, or paged_tile.cu's for many rows
// per sequence and kv head) and its workspace.
#include "paged_rows.cuh"

namespace ra {

size_t paged_attention_workspace(const PagedLaunch& L) {
  if (paged_tile_serves(L)) return kAttnHeader + paged_tile_workspace(L);
  Plan pl;
  if (!plan(L, &pl)) return 0;
  return kAttnHeader + join_bytes(pl.room, pl.NR, L.Dv);
}

cudaError_t launch_paged_attention(const PagedLaunch& L, cudaStream_t stream, const char** why) {
  if (paged_tile_serves(L)) return launch_paged_tile(L, stream, why);
  return launch_rows<false>(L, stream, why);
}

}  // namespace ra
