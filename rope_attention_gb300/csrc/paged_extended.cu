// The paged attention calls with a window or a shared prefix: the choice of the kernel.
#include "paged_tokens.cuh"

namespace ra {

cudaError_t launch_paged_extended(const PagedLaunch& L, cudaStream_t stream, const char** why) {
  if (paged_tile_serves(L)) return launch_paged_tile_extended(L, stream, why);
  if (paged_tokens_serves(L)) return launch_paged_tokens(L, stream, why);
  return launch_rows<true>(L, stream, why);
}

int paged_extended_blocks(const PagedLaunch& L) {
  if (paged_tile_serves(L)) return paged_tile_blocks(L);
  if (paged_tokens_serves(L)) return paged_tokens_blocks(L);
  Plan pl{};
  return plan(L, &pl) ? std::min(pl.G, launch_blocks(L)) : 0;
}

namespace {
// Cycles of a call's blocks for `keys` keys of every sequence, roughly: the tiles shared out, at what one of
// its kernel takes (measured over prefixes of 2000 to 20000 positions).
double call_cycles(const PagedLaunch& L, int64_t keys) {
  double tiles, each;
  if (paged_tile_serves(L)) {
    const int kt = paged_tile_keys(L);
    tiles = static_cast<double>(paged_tile_items(L)) * ((keys + kt - 1) / kt);
    each = 3500;
  } else {
    Plan pl{};
    const bool tokens = paged_tokens_serves(L);
    if (tokens) plan_tokens(L, &pl);
    else if (!plan(L, &pl)) return 0;
    tiles = static_cast<double>(pl.items) * ((keys + kKeys - 1) / kKeys);
    each = tokens ? 1150 : L.variant == 1 ? 4000 : 3300;
  }
  return std::ceil(tiles / device_sm_count()) * each;
}
}  // namespace

// Sharing the prefix's reads takes a second call (its start, its join, and the fp32 rows on their way from
// one to the other), and pays where that many tiles need not be read again.  (64 heads over 8, int8,
// sequences of 512, one call and two: 16 of them behind 2000 positions 31 and 43 us, 32 of them 53 and 53,
// behind 8192 141 and 66, 61 of them 258 and 106; the latent under 16 heads, 32 sequences: 2000 40 and
// 52, 8192 78 and 72; under 128 heads, whose tiles one sequence fills, 20000 304 and 335.)
bool prefix_is_shared(const PagedLaunch& over, const PagedLaunch& behind) {
  const double second = paged_tokens_serves(over) ? 22000 : 40000;
  const double rows = static_cast<double>(over.total_q) * over.heads * over.Dv * sizeof(float) / 620;  // bytes a cycle, there and back
  return call_cycles(behind, behind.max_prefix_len) > call_cycles(over, over.max_seq_len) + second + rows;
}

}  // namespace ra
