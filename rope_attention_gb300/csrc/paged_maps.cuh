// Tensor maps of paged_attention's operands.
#pragma once

#include "attention.h"
#include "internal.h"
#include "kv_cache.h"

namespace ra {
namespace {

// A cache's rows as a 3-D map: PA (channels, heads, slots), the others (channels, 1, rows);
// boxes of 64 channels x box_rows rows, swizzled like an MMA operand unless they are codes
inline bool make_map(CUtensorMap* m, const void* base, const PagedLaunch& L, int32_t width, int32_t quant, int32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const uint64_t row = static_cast<uint64_t>(width) * (quant ? 1 : 2);
  const bool pa = L.mode == kModePa;
  const uint64_t slots = L.mode == kModeNorm ? static_cast<uint64_t>(L.B) * L.cache_seq
                                             : static_cast<uint64_t>(L.block_num) * L.block_size;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), pa ? static_cast<cuuint64_t>(L.N) : 1, pa ? slots : slots * L.N};
  cuuint64_t strides[2] = {row, pa ? row * L.N : row};
  cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, quant ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             quant ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q as (channels, heads, tokens), boxes of one row tile's 64 channels
inline bool make_q_map(CUtensorMap* m, const PagedLaunch& L, int32_t hb, int32_t tb) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(L.Dkv), static_cast<cuuint64_t>(L.heads), static_cast<cuuint64_t>(L.total_q)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(L.Dkv) * 2, static_cast<cuuint64_t>(L.Dkv) * 2 * L.heads};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(hb), static_cast<cuuint32_t>(tb)};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<uint16_t*>(L.q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace ra
