// The paged attention calls with a window or a shared prefix: the choice of the kernel.
#include "paged_tokens.cuh"

namespace ra {

cudaError_t launch_paged_extended(const PagedLaunch& L, cudaStream_t stream, const char** why) {
  if (paged_tile_serves(L)) return launch_paged_tile_extended(L, stream, why);
  if (paged_tokens_serves(L)) return launch_paged_tokens(L, stream, why);
  return launch_rows<true>(L, stream, why);
}

namespace {
// What a call over `keys` keys of every sequence takes, roughly, in cycles: items of so many tiles, whole or
// shared out and joined, what a tile of its kernel takes, an item's beginning and end, and a block's start (launch
// included).  Fitted to calls over 500 to 20000 positions on 8 to 152 SMs.
constexpr double kJoinCycles = 15000;
struct CallCost {
  double items, each, start, end, tiles;
  bool whole;
  double cycles(int blocks) const {
    const double most = std::ceil(items / blocks);
    return start + most * end + (whole ? most * tiles * each : std::ceil(items * tiles / blocks) * each + kJoinCycles);
  }
};
CallCost call_cost(const PagedLaunch& L, int64_t keys) {
  CallCost c{};
  int kt = kKeys;
  const int64_t mean = (L.total_q + L.B - 1) / L.B;     // tokens of a sequence
  const auto items = [&](const Plan& pl) {
    return static_cast<double>((pl.hblocks > 1 ? L.total_q * pl.hblocks : L.B * ((mean + pl.tb - 1) / pl.tb)) * L.N);
  };
  if (paged_tile_serves(L)) {
    kt = paged_tile_keys(L);
    const int64_t tokens = paged_tile_tokens(L);
    const bool half = 2 * mean <= tokens;     // one of an item's two row tiles
    c = CallCost{static_cast<double>(L.B * ((mean + tokens - 1) / tokens) * L.N), half ? 2700. : 3500., half ? 20000. : 30000.,
                 half ? 12000. : 17000., 0, false};
  } else {
    Plan pl{};
    if (paged_tokens_serves(L)) {
      plan_tokens(L, &pl);
      c = CallCost{items(pl), 1150, 17000, 3000, 0, pl.whole != 0};
    } else if (plan(L, &pl)) {
      c = CallCost{items(pl), L.variant == 1 ? 4000. : 3300., 30000, L.kq || L.vq ? 16000. : 4000., 0, pl.whole != 0};
    }
  }
  c.tiles = static_cast<double>((keys + kt - 1) / kt);
  return c;
}

// Two calls of paged_rows.cuh's kernel in one launch: the own positions' items whole on `mine` blocks, the prefix's
// in parts on the others; a join behind both.
cudaError_t launch_rows_beside(const PagedLaunch& own, const PagedLaunch& over, int mine, cudaStream_t stream, const char** why) {
  Plan a, b;
  Calls<true> calls{};
  if (!prepare_rows(own, &a, &calls.a, why) || !prepare_rows(over, &b, &calls.b, why)) return cudaErrorInvalidValue;
  const int rest = std::min(b.G, device_sm_count() - mine);
  calls.a.whole = 1;
  calls.b.whole = 0;
  calls.b.join_all = 1;
  calls.split = mine;
  const cudaError_t e = launch_calls<true>(over, calls, mine + rest, std::max(a.smem, b.smem), stream);
  return e != cudaSuccess ? e : launch_join<true>(calls.b.join, over.f16, rest, b.items, stream);
}

// The blocks for the first of two calls in one launch, 0 where that is later than `best` cycles: both have
// one kernel, and the second has more blocks than items, so that each of its blocks has to do with two at most.
int beside_blocks(const PagedLaunch& own, const PagedLaunch& over, const CallCost& a, const CallCost& b, double best) {
  Plan pl{}, pl_own{};
  if (paged_tile_serves(own) || paged_tokens_serves(own) || paged_tile_serves(over) || paged_tokens_serves(over)) return 0;
  if (!plan(own, &pl_own) || !plan(over, &pl)) return 0;
  CallCost first = a, second = b;
  first.whole = true;
  second.whole = false;
  const int sms = device_sm_count(), most = std::min(pl_own.G, sms - 8);
  int mine = 0;
  for (int x = 4; x < most + 4; x += 4) {
    const int blocks = std::min(x, most), rest = std::min(pl.G, sms - blocks);
    const double t = std::max(first.cycles(blocks) + kJoinCycles, second.cycles(rest));
    if (rest <= pl.items || rest < 2 || t >= best) continue;
    best = t;
    mine = blocks;
  }
  return mine;
}
}  // namespace

// The second call costs a launch, a start, a join and the fp32 rows on their way to it, and pays where that many
// tiles need not be read again; in one launch with the first its start, its tiles and its end are beside the
// first's.  (us in one call and in two: 64 heads over 8, int8, sequences of 512: 16 of them behind
// 1500 positions 27 and 44, behind 8192 78 and 49; 32 of them behind 1500 47 and 50, behind 20000 312 and 94.  Chunks of
// up to 64 tokens, 32 heads over 4, 32 sequences behind 4000 143 and 168, 20000 493 and 439.  In one call, in two, and in
// two in one launch: the latent under 16 heads, 16 sequences behind 1500 29, 40 and 29, 8192 50, 47 and 29; 32 behind 8192
// 76, 64 and 40, 16384 128, 76 and 60; under 128 heads, whose tiles one sequence fills, behind 16384 251, 271 and more.)
cudaError_t launch_paged_prefix(const PagedLaunch& own, const PagedLaunch& over, const PagedLaunch& behind, cudaStream_t stream,
                                const char** why) {
  const int sms = device_sm_count();
  const double rows = static_cast<double>(over.total_q) * over.heads * over.Dv * sizeof(float) / 700;  // bytes a cycle, there and back
  const CallCost a = call_cost(own, own.max_seq_len), b = call_cost(over, over.max_seq_len);
  const double one = call_cost(behind, behind.max_prefix_len + own.max_seq_len).cycles(sms) - rows, two = a.cycles(sms) + b.cycles(sms);
  const int mine = beside_blocks(own, over, a, b, std::min(one, two));
  if (mine > 0) return launch_rows_beside(own, over, mine, stream, why);
  if (one <= two) return launch_paged_extended(behind, stream, why);
  const cudaError_t e = launch_paged_extended(own, stream, why);
  return e != cudaSuccess ? e : launch_paged_extended(over, stream, why);
}

}  // namespace ra
