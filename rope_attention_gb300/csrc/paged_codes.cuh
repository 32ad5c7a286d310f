// Cache codes as fp16 operands.
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "attn_ptx.cuh"
#include "kv_cache.h"

namespace ra {
namespace {

// four codes -> four fp16 values, exactly
template <int KIND>
__device__ __forceinline__ uint2 codes_to_half(uint32_t c) {
  uint2 r;
  if constexpr (KIND == kQuantInt8) {
    // 0x6400 | u is the fp16 number 1024 + u; with u = code + 128, subtract 1152
    c ^= 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    uint32_t lo = __byte_perm(c, 0x64646464u, 0x4140), hi = __byte_perm(c, 0x64646464u, 0x4342);
    __half2 a = __hsub2(*reinterpret_cast<__half2*>(&lo), off), b = __hsub2(*reinterpret_cast<__half2*>(&hi), off);
    r.x = *reinterpret_cast<uint32_t*>(&a);
    r.y = *reinterpret_cast<uint32_t*>(&b);
  } else if constexpr (KIND == kQuantE5m2) {  // the upper byte of an fp16 number
    r.x = __byte_perm(c, 0, 0x1404);
    r.y = __byte_perm(c, 0, 0x3424);
  } else {
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c & 0xFFFFu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c >> 16), __NV_E4M3);
    r.x = a.x | (static_cast<uint32_t>(a.y) << 16);
    r.y = b.x | (static_cast<uint32_t>(b.y) << 16);
  }
  return r;
}

// 16 codes -> 32 bytes of a swizzled row: chunks 2 c and 2 c + 1 of row `key`
template <int KIND>
__device__ __forceinline__ void store_codes(uint8_t* row, int key, int c, uint4 x) {
  const uint2 a = codes_to_half<KIND>(x.x), b = codes_to_half<KIND>(x.y), d = codes_to_half<KIND>(x.z), e = codes_to_half<KIND>(x.w);
  *reinterpret_cast<uint4*>(row + (((2 * c) ^ (key & 7)) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
  *reinterpret_cast<uint4*>(row + (((2 * c + 1) ^ (key & 7)) << 4)) = make_uint4(d.x, d.y, e.x, e.y);
}
// f with the kind as a constant: a choice inside the conversion would cut a warp's chunks apart,
// and a lone warp lives from running several at once
template <class F>
__device__ __forceinline__ void with_kind(int32_t kind, F&& f) {
  if (kind == kQuantInt8) f(std::integral_constant<int, kQuantInt8>());
  else if (kind == kQuantE4m3) f(std::integral_constant<int, kQuantE4m3>());
  else f(std::integral_constant<int, kQuantE5m2>());
}
}  // namespace
}  // namespace ra
