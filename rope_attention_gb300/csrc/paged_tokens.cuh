// The plan of paged_tokens.cu's kernel, and what its warps hand each other.
#pragma once

#include "paged_rows.cuh"

namespace ra {
namespace {

// Two teams of four warps compute; of a third warpgroup, whose registers they take (2 x 208 + 88 = 3 x 168),
// one warp loads tiles and one prepares pieces.  (Three teams, for 8 rows: no gain.)
constexpr int kTokenWarps = 8, kTileWarps = 4, kTeams = kTokenWarps / kTileWarps, kTokenThreads = 32 * kTokenWarps + 128;
constexpr int kTokenLoad = kTokenWarps, kTokenPieces = kTokenWarps + 1;
constexpr int kRegsCompute = 208, kRegsOther = 88;
constexpr int kTokenStages = 12;          // at most
constexpr int kTokenRow = 132;            // floats of a row where the warps' results meet
constexpr int kTokenDk = 192, kTokenDv = 128;

// A piece as its warp hands it over.
struct TokenPiece {
  int32_t end;                            // there is no further piece
  int32_t rows, kv_head, ta, n, whole;
  int32_t ahead, skip, prefix;            // as in Piece
  int32_t slot;                           // of its part
  int32_t seen_least, from_most;
  int32_t seen[16], from[16];             // what each row sees: positions below, and from its window on
  int2 row[16];                           // token and head
  float row_scale[16], row_const[16];     // of the scores; the lse's share of the key offsets
};
struct TokenMisc {
  uint64_t full[kTokenStages], empty[kTokenStages];
  uint64_t piece_full[2], piece_empty[2];
  uint64_t valid[kValidRing];
  RunScan<kTokenThreads> run;
  float2 stats[kTokenWarps][16];          // (max, sum) of each warp's rows
  TokenPiece pieces[2];
  int32_t abort;
};

inline void plan_tokens(const PagedLaunch& L, Plan* pl) {
  const int g = L.heads / static_cast<int32_t>(L.N);
  pl->NR = (L.total_q + L.B - 1) / L.B * g <= 8 ? 8 : 16;
  // a stage: the value rows, then the key rows, each on 1024 bytes (the swizzle's period); codes count as one slab
  const auto bytes = [](int quant, int width) { return quant ? (kKeys * width + 1023) / 1024 * 1024 : (width + 63) / 64 * kSlab; };
  pl->vslabs = L.vq ? 1 : (L.Dv + 63) / 64;
  pl->kslabs = L.kq ? 1 : (L.Dkv + 63) / 64;
  pl->kslab0 = L.kq && L.Dkv == 128;            // whether codes of keys are swizzled
  pl->off_staging = bytes(L.vq, L.Dv);          // of the keys in a stage
  pl->stage = pl->off_staging + bytes(L.kq, L.Dkv);
  // where the warps' results meet, and two pieces' queries
  const int meet = kTokenWarps * pl->NR * kTokenRow * 4 + 2 * pl->NR / 8 * 24 * 32 * 4;
  const int fixed = meet + ((static_cast<int>(sizeof(TokenMisc)) + 15) & ~15);
  // As many for each team: within a piece a stage then is always one team's, which waits for its uses one after the
  // other.  (A wait knows a use of a stage from the one before by a parity alone.  With an odd number the teams take
  // turns on a stage, and one could come to it while the copy of the other's tile, issued earlier, had still not
  // landed, and take that for its own.)  From one piece to the next the teams may change places, as the team goes
  // by the tile's number in its piece and the stage by the running one: behind a piece with an odd number of
  // tiles they do.  Both teams meet at the end of a piece (bar_or), where every copy of it has landed and been used; a team
  // that went on without that would bring the fault back.
  pl->ns = std::min(kTokenStages, (kSmemMax - fixed) / pl->stage) / kTeams * kTeams;
  pl->off_p = pl->ns * pl->stage;
  pl->off_misc = pl->off_p + meet;
  pl->smem = pl->off_misc + ((static_cast<int>(sizeof(TokenMisc)) + 15) & ~15);
  // Items are cut where that saves a block more tiles than the join costs, 5 to 17 of this kernel's.  (int8, in a
  // window: 8 items of 9 tiles 14.1 us whole and 14.4 cut, of 15 16.4 and 14.4; 64 items of 15 18.5 and 22.0, of 28
  // 24.6 and 24.6; 256 items of 28 43 and 48, of 53 70 and 70.)
  share_out(L, pl, [&](int64_t T) {
    const double share = static_cast<double>(pl->items) / device_sm_count(), rounds = std::ceil(share);
    return (rounds - share) * static_cast<double>(T) <= 5 + 12 * std::min(4 * share, 1.0);
  });
  // the workspace is sized for paged_attention's kernel, whose row tiles hold more rows
  const size_t have = paged_attention_workspace(L) - kAttnHeader;
  while (pl->G > 1 && join_bytes(pl->G, pl->NR, L.Dv) > have) --pl->G;
}

}  // namespace
}  // namespace ra
