// The paged attention calls with a window or a shared prefix: the choice of the kernel.
#include "paged_tokens.cuh"

namespace ra {

cudaError_t launch_paged_extended(const PagedLaunch& L, cudaStream_t stream, const char** why) {
  if (paged_tile_serves(L)) return launch_paged_tile_extended(L, stream, why);
  if (paged_tokens_serves(L)) return launch_paged_tokens(L, stream, why);
  return launch_rows<true>(L, stream, why);
}

namespace {
// blocks that a call launches
int paged_extended_blocks(const PagedLaunch& L) {
  if (paged_tile_serves(L)) return paged_tile_blocks(L);
  if (paged_tokens_serves(L)) return paged_tokens_blocks(L);
  Plan pl{};
  return plan(L, &pl) ? std::min(pl.G, launch_blocks(L)) : 0;
}

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
// sequences of 512, one call and two: 16 of them behind 2000 positions 31 and 40 us, 32 of them 53 and 45,
// behind 8192 141 and 59, 61 of them 258 and 91; the latent under 16 heads, 32 sequences: 500 27 and
// 28, 2000 37 and 34, 8192 76 and 46; under 128 heads, whose tiles one sequence fills, 20000 300 and 488.)
bool prefix_is_shared(const PagedLaunch& over, const PagedLaunch& behind) {
  const double second = over.variant == 1 ? 14000 : paged_tokens_serves(over) ? 16000 : 26000;
  const double rows = static_cast<double>(over.total_q) * over.heads * over.Dv * sizeof(float) / 700;  // bytes a cycle, there and back
  return call_cycles(behind, behind.max_prefix_len) > call_cycles(over, over.max_seq_len) + second + rows;
}

// Blocks for the call over the prefix, 0 for all: the SMs that the sequences' own call leaves, where those take
// less longer over it than waiting for the others would (its start and its end beside its tiles).
int prefix_blocks(const PagedLaunch& own, const PagedLaunch& over) {
  constexpr double kStartAndEnd = 25000;
  const int sms = device_sm_count(), taken = paged_extended_blocks(own);
  if (taken >= sms) return 0;
  const double later = call_cycles(own, own.max_seq_len) + kStartAndEnd;
  return call_cycles(over, over.max_seq_len) * taken / (sms - taken) < later && 2 * taken <= sms ? sms - taken : 0;
}

}  // namespace ra
