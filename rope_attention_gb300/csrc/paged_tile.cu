// paged_attention for many rows per sequence and kv head: the rule that chooses paged_tile.cuh's
// kernel, and its workspace.
#include "paged_tile.cuh"

namespace ra {

// V2 rows that one key tile can be wide enough for, a group of heads that fits a row tile,
// both caches of one sort, and more rows per sequence and kv head than kRows: below that the
// kernel in paged_rows.cuh, whose products cost what the rows there are need.  (4 sequences
// of 4096 positions, 8 kv heads, keys of 192: 32 rows take 35 us here and 33 there, 64 rows 34
// and 36; int8 46 and 43, 45 and 48.)
bool paged_tile_serves(const PagedLaunch& L) {
  constexpr int64_t kRows = 32;
  const int64_t g = L.heads / L.N;
  return L.variant == 2 && L.Dkv <= 192 && L.Dv <= 128 && g <= kTileRows && (L.kq != 0) == (L.vq != 0) &&
         L.total_q * g > kRows * L.B;
}

int64_t paged_tile_tokens(const PagedLaunch& L) { return 2 * (kTileRows / (L.heads / static_cast<int32_t>(L.N))); }
int paged_tile_keys(const PagedLaunch& L) { return keys_per_tile(L); }

size_t paged_tile_workspace(const PagedLaunch& L) { return join_bytes(most_blocks(L), 2 * kTileRows, L.Dv); }

cudaError_t launch_paged_tile(const PagedLaunch& L, cudaStream_t stream, const char** why) {
  return launch_tile_over_pages<false>(L, stream, why);
}

}  // namespace ra
