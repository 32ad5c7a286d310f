// Attention over packed prompts: softmax(scale q k^T) v on the projection's own output.
//
//   out[i, h] = sum_j p[i, j] v[j, h / g] / sum_j p[i, j],
//   p[i, j]   = exp(scale * q[i, h] . k[j, h / g] - m_i)   over the keys j that i sees:
//   those of its own sequence, and with `causal` those with j <= i + Lk - Lq
// (g = num_heads / num_kv_heads).  A row that sees no key is zero, its lse -inf.
//
// The kernel is tile_attention.cuh's, with 128 tokens of one head to a row tile and 128 keys
// to a key tile, all loaded by TMA straight from the strided views (channels beyond
// head_dim read as zeros).  Bound by the tensor core: 16 products of 128 x 128 x 16 per row
// tile and 128 keys.  Measured: 32760 tokens, 40 heads of 128 (the 480p latent grid against
// itself) 14.3 ms, 1540 TFLOP/s of 1720 that a library GEMM sustains under the power limit;
// against 512 text tokens 327 us (1050 TFLOP/s: four key tiles an item, whose start and end
// show); 9001 tokens in 7 causal prompts, 32 heads over 8, 157 us (840 TFLOP/s, 147 us of it
// this kernel at 47 % of the tensor pipe, the rest the join).
#include "tile_attention.cuh"

namespace ra {
namespace {

constexpr int64_t kKeysInL2 = 48 << 20;     // of the 129 MB

// [tokens, heads, d] with any strides as a 3-D map of 64 x 128-token boxes; the axis with
// the smaller stride comes second
bool make_view_map(CUtensorMap* m, const uint16_t* base, int64_t tokens, int64_t heads, int32_t d, int64_t ts, int64_t hs,
                   int32_t* swap) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  // an axis of one element is never stepped along: give it a stride the encoder accepts
  if (heads == 1) hs = std::max<int64_t>(ts * tokens, d);
  if (tokens == 1) ts = std::max<int64_t>(hs * heads, d);
  *swap = ts < hs;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(*swap ? tokens : heads),
                        static_cast<cuuint64_t>(*swap ? heads : tokens)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(*swap ? ts : hs) * 2, static_cast<cuuint64_t>(*swap ? hs : ts) * 2};
  cuuint32_t box[3] = {64, *swap ? 128u : 1u, *swap ? 1u : 128u};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<uint16_t*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t most_items(const PackedLaunch& L) {
  const int64_t block = 2 * kTileRows;
  const int64_t blocks = L.cu_q ? std::min(L.total_q, L.total_q / block + L.B) : L.B * ((L.total_q / L.B + block - 1) / block);
  return blocks * L.nq;
}
// (cu_q and cu_k are not known when the workspace is sized: the larger of both ways)
int most_blocks(const PackedLaunch& L) {
  const int64_t items = std::min(L.total_q, L.total_q / (2 * kTileRows) + L.B) * L.nq;
  return tile_blocks(items, (L.total_k + kTileRows - 1) / kTileRows);
}

}  // namespace

size_t packed_attention_workspace(const PackedLaunch& L) { return kAttnHeader + join_bytes(most_blocks(L), 2 * kTileRows, L.d); }

cudaError_t launch_packed_attention(const PackedLaunch& L, cudaStream_t stream, const char** why) {
  TileParams p{};
  if (!encode_maps([&] {
        return make_view_map(&p.tq, L.q, L.total_q, L.nq, L.d, L.q_ts, L.q_hs, &p.q_swap) &&
               make_view_map(&p.tk, L.k, L.total_k, L.nkv, L.d, L.k_ts, L.k_hs, &p.k_swap) &&
               make_view_map(&p.tv, L.v, L.total_k, L.nkv, L.d, L.v_ts, L.v_hs, &p.v_swap);
      })) {
    *why = "cuTensorMapEncodeTiled failed or is unavailable";
    return cudaErrorInvalidValue;
  }
  const int blocks = most_blocks(L);
  p.join.NR = 2 * kTileRows;
  p.join.sub = kTileRows;
  join_place(&p.join, L.partials, blocks);
  p.join.out = L.out;
  p.join.lse = L.lse;
  p.join.o_ts = L.o_ts;
  p.join.o_hs = L.o_hs;
  p.join.heads = L.nq;
  p.join.hb = 1;
  p.join.tb = kTileRows;
  p.join.Dv = L.d;
  p.cu_q = L.cu_q;
  p.cu_k = L.cu_k;
  p.status = L.status;
  p.B = static_cast<int32_t>(L.B);
  p.total_q = static_cast<int32_t>(L.total_q);
  p.total_k = static_cast<int32_t>(L.total_k);
  p.items = L.nq;
  // Keys and values that stay in L2: the heads of a row block one after another, so that its
  // rows of q and out, a token's heads side by side, pass HBM in long stretches.  Otherwise
  // the row blocks of a head, which share its keys.
  p.heads_first = L.total_k * L.nkv * L.d * 4 <= kKeysInL2;
  p.g = L.nq / L.nkv;
  p.Dk = L.d;
  p.ksteps = L.d / 16;
  p.causal = L.causal;
  p.out32 = (reinterpret_cast<uintptr_t>(L.out) & 31u) == 0 && p.join.o_ts % 16 == 0 && p.join.o_hs % 16 == 0;
  p.scale = L.scale;
  p.sl2 = static_cast<float>(static_cast<double>(L.scale) * 1.4426950408889634);
  p.wait_ns = static_cast<uint64_t>(L.wait_ns);
  p.stall_loads = L.stall_loads;
  const int n = std::min(blocks, device_sm_count());
  const int64_t items = most_items(L);
  // equal lengths without a mask: all items count alike, and whether one is cut is known here
  const bool cuts = L.cu_q || L.cu_k || L.causal ||
                    tile_runs_cut(items, kTileExtra + std::max<int64_t>(1, (L.total_k / L.B + kTileRows - 1) / kTileRows), n);
  if (L.d <= 64)
    return L.f16 ? launch_tile<1, 1, 128, true, false, false>(p, n, items, cuts, stream)
                 : launch_tile<1, 1, 128, false, false, false>(p, n, items, cuts, stream);
  return L.f16 ? launch_tile<2, 2, 128, true, false, false>(p, n, items, cuts, stream)
               : launch_tile<2, 2, 128, false, false, false>(p, n, items, cuts, stream);
}

}  // namespace ra
