// paged_attention for many rows per sequence and kv head (chunks of new tokens): the caches
// behind tile_attention.cuh's kernel.  Measured: 512 new tokens a sequence
// over 4 bf16 sequences of up to 16384 positions, 32 heads over 8, 400 us (1090 TFLOP/s); an fp16 one over an FP8 cache of 2 x 8192 positions,
// 777 tokens and 32 heads, 335 us (590 TFLOP/s; 265 without the second half of P, whose
// results are 1.8 times as far off as fp16's own rounding).
#include "paged_maps.cuh"
#include "tile_attention.cuh"

namespace ra {
namespace {

// keys per tile: what two row tiles of queries leave room for
constexpr int kKeysWide = 96, kKeysWideCodes = 64, kKeys = 128;

int keys_per_tile(const PagedLaunch& L) { return L.Dkv <= 128 ? kKeys : L.kq ? kKeysWideCodes : kKeysWide; }

int64_t most_items(const PagedLaunch& L) {
  const int64_t tokens = 2 * (kTileRows / (L.heads / static_cast<int32_t>(L.N)));
  return std::min(L.total_q, L.total_q / tokens + L.B) * L.N;
}
int most_blocks(const PagedLaunch& L) {
  const int keys = keys_per_tile(L);
  return tile_blocks(most_items(L), std::max<int64_t>(1, (L.max_seq_len + keys - 1) / keys));
}

}  // namespace

// V2 rows that one key tile can be wide enough for, a group of heads that fits a row tile,
// both caches of one sort, and more rows per sequence and kv head than kRows: below that the
// kernel in paged_attention.cu, whose products cost what the rows there are need.  (4 sequences
// of 4096 positions, 8 kv heads, keys of 192: 32 rows take 35 us here and 33 there, 64 rows 34
// and 36; int8 46 and 43, 45 and 48.)
bool paged_tile_serves(const PagedLaunch& L) {
  constexpr int64_t kRows = 32;
  const int64_t g = L.heads / L.N;
  return L.variant == 2 && L.Dkv <= 192 && L.Dv <= 128 && g <= kTileRows && (L.kq != 0) == (L.vq != 0) &&
         L.total_q * g > kRows * L.B;
}

size_t paged_tile_workspace(const PagedLaunch& L) { return join_bytes(most_blocks(L), 2 * kTileRows, L.Dv); }

cudaError_t launch_paged_tile(const PagedLaunch& L, cudaStream_t stream, const char** why) {
  TileParams p{};
  const int g = L.heads / static_cast<int32_t>(L.N), keys = keys_per_tile(L), blocks = most_blocks(L);
  p.join.NR = 2 * kTileRows;
  p.join.sub = kTileRows;
  join_place(&p.join, L.partials, blocks);
  p.join.out = L.out;
  p.join.lse = L.lse;
  p.join.v_scale = L.v_scale;
  p.join.v_offset = L.v_offset;
  p.join.o_hs = L.Dv;
  p.join.o_ts = static_cast<int64_t>(L.Dv) * L.heads;
  p.join.heads = L.heads;
  p.join.hb = g;
  p.join.tb = kTileRows / g;
  p.join.Dv = L.Dv;
  p.join.per_head = 1;
  p.cu_q = L.cu_q;
  p.cu_k = L.seq_lens;
  p.table = L.table;
  p.err_count = L.err_count;
  p.status = L.status;
  p.k_scale = L.k_scale;
  p.k_offset = L.k_offset;
  p.table_stride = L.table_stride;
  p.cap = std::min<int64_t>(L.mode == kModeNorm ? L.cache_seq : L.table_stride * L.block_size, L.max_seq_len);
  p.block_num = L.block_num;
  p.cache_seq = L.cache_seq;
  p.B = static_cast<int32_t>(L.B);
  p.total_q = static_cast<int32_t>(L.total_q);
  p.items = static_cast<int32_t>(L.N);
  p.g = g;
  p.Dk = L.Dkv;
  p.ksteps = L.Dkv / 16;
  p.causal = L.causal;
  p.mode = L.mode;
  p.block_size = static_cast<int32_t>(L.block_size);
  p.bs_shift = -1;
  for (int s = 0; s < 31; ++s)
    if ((int64_t(1) << s) == L.block_size) p.bs_shift = s;
  // the largest box that divides a page and a key tile
  p.box_shift = 4;
  while (p.box_shift < 7 && keys % (2 << p.box_shift) == 0 && (L.mode == kModeNorm || L.block_size % (2 << p.box_shift) == 0))
    ++p.box_shift;
  p.box_rows = 1 << p.box_shift;
  p.kq = L.kq;
  p.vq = L.vq;
  p.out32 = (reinterpret_cast<uintptr_t>(L.out) & 31u) == 0 && p.join.o_ts % 16 == 0 && p.join.o_hs % 16 == 0;
  p.scale = L.scale;
  p.sl2 = static_cast<float>(static_cast<double>(L.scale) * 1.4426950408889634);
  p.wait_ns = static_cast<uint64_t>(L.wait_ns);
  p.stall_loads = L.stall_loads;
  if (!encode_maps([&] {
        return make_q_map(&p.tq, L, p.join.hb, p.join.tb) && make_map(&p.tv, L.v_cache, L, L.Dv, L.vq, p.box_rows) &&
               make_map(&p.tk, L.k_cache, L, L.Dkv, L.kq, p.box_rows);
      })) {
    *why = "cuTensorMapEncodeTiled failed or is unavailable";
    return cudaErrorInvalidValue;
  }
  const int n = std::min(blocks, device_sm_count());
  const int64_t items = most_items(L);
  if (L.kq) {
    if (L.Dkv <= 128)
      return L.f16 ? launch_tile<2, 2, kKeys, true, true, true>(p, n, items, true, stream)
                   : launch_tile<2, 2, kKeys, false, true, true>(p, n, items, true, stream);
    return L.f16 ? launch_tile<3, 2, kKeysWideCodes, true, true, true>(p, n, items, true, stream)
                 : launch_tile<3, 2, kKeysWideCodes, false, true, true>(p, n, items, true, stream);
  }
  if (L.Dkv <= 128)
    return L.f16 ? launch_tile<2, 2, kKeys, true, false, true>(p, n, items, true, stream)
                 : launch_tile<2, 2, kKeys, false, false, true>(p, n, items, true, stream);
  return L.f16 ? launch_tile<3, 2, kKeysWide, true, false, true>(p, n, items, true, stream)
               : launch_tile<3, 2, kKeysWide, false, false, true>(p, n, items, true, stream);
}

}  // namespace ra
