// Rows of the paged caches gathered by slot and dequantised: the inverse of
// kv_rms_norm_rope_cache's scatter,
//   out[b, n, s, c] = (code - offset[c]) / scale[c]   (16-bit caches: the element itself).
//
// An HBM stream of short scattered rows (1 or 2 bytes read, 2 written per element), so the
// mapping spends few instructions per byte and keeps loads in flight:
//  * a block serves one head, whose quantisation it turns once into a table in shared
//    memory: x = code * r + t, r = 1 / scale, t = -offset * r, one fused multiply-add an
//    element (fp32; at most 2^-24 (2 |x| + 3 |offset / scale|) off, far below the rounding
//    to 16 bits);
//  * a warp takes 4 tokens at once and spreads their rows' 8-channel units (8 or 16 bytes
//    in, 16 out) over its lanes: four rows fill them where one would not (72 units in a
//    576-channel row: 9 rounds of 32 instead of 12), and the slot lookups and the index
//    arithmetic, done by one lane per token, are a small part;
//  * the loads of kBatch rounds are in flight together.
#include <cuda_fp8.h>

#include <algorithm>

#include "attention.h"
#include "attn_ptx.cuh"
#include "internal.h"
#include "kv_cache.h"

namespace ra {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTokens = 4;      // tokens a warp takes at once
constexpr int kBatch = 3;

struct Side {                   // one of the two caches
  const uint8_t* cache;
  const float *scale, *offset;
  uint16_t* out;
  int32_t width, kind, scalar, units;  // units of 8 channels per row
};

// the cache row of token (b, s) of head n; -1: none, -2: outside the cache
__device__ __forceinline__ int64_t row_of(const ReadLaunch& L, int64_t b, int64_t n, int64_t s) {
  const int64_t bs = L.block_size;
  if (L.mode == kModeNorm) {
    const int64_t i = __ldg(L.index + b * L.S + s);
    if (i == -1) return -1;
    return i < 0 || i >= L.cache_seq ? -2 : (b * L.N + n) * L.cache_seq + i;
  }
  int64_t slot;
  if (L.mode == kModePaBlkBnsd) {
    const int64_t first = __ldg(L.index + b * ((L.S + bs - 1) / bs) + s / bs);
    if (first == -1) return -1;
    if (first < 0 || first >= L.block_num * bs) return -2;
    slot = first + s % bs;
  } else {
    slot = __ldg(L.index + b * L.S + s);
    if (slot == -1) return -1;
  }
  if (slot < 0 || slot >= L.block_num * bs) return -2;
  const int64_t page = slot / bs, in = slot - page * bs;
  return L.mode == kModePa ? slot * L.N + n : (page * L.N + n) * bs + in;
}

// 8 codes -> 8 floats
__device__ __forceinline__ void codes_to_float(uint2 w, int32_t kind, float (&x)[8]) {
  const uint32_t v[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (kind == kQuantInt8) {
      // the byte code + 128 below the exponent of 2^23 is the float 2^23 + code + 128
      const uint32_t u = v[i] ^ 0x80808080u;
      x[4 * i] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)) - 8388736.f;
      x[4 * i + 1] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441)) - 8388736.f;
      x[4 * i + 2] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)) - 8388736.f;
      x[4 * i + 3] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443)) - 8388736.f;
    } else {
      const __nv_fp8_interpretation_t f = kind == kQuantE4m3 ? __NV_E4M3 : __NV_E5M2;
      const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v[i] & 0xFFFFu), f);
      const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v[i] >> 16), f);
      x[4 * i] = __half2float(__ushort_as_half(lo.x));
      x[4 * i + 1] = __half2float(__ushort_as_half(lo.y));
      x[4 * i + 2] = __half2float(__ushort_as_half(hi.x));
      x[4 * i + 3] = __half2float(__ushort_as_half(hi.y));
    }
  }
}

template <bool F16>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ ReadLaunch L,
                                                              const __grid_constant__ Side k,
                                                              const __grid_constant__ Side v) {
  extern __shared__ float4 table[];          // r, then t, of the k units and the v units: 2 + 2 float4 a unit
  const int64_t n = blockIdx.y;
  const int units = k.units + v.units, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < units * 8; i += kThreads) {
    const bool is_k = i < k.units * 8;
    const Side& side = is_k ? k : v;
    if (side.kind == kQuantNone) continue;
    const int c = is_k ? i : i - k.units * 8;
    const int at = side.scalar ? 0 : (L.variant == 2 ? static_cast<int>(n) * side.width : 0) + c;
    const float r = __frcp_rn(__ldg(side.scale + at));
    float* row = reinterpret_cast<float*>(table) + (i >> 3) * 16;
    row[i & 7] = r;
    row[8 + (i & 7)] = side.offset ? -__ldg(side.offset + at) * r : 0.f;
  }
  __syncthreads();
  const int64_t tokens = L.B * L.S, step = static_cast<int64_t>(gridDim.x) * kWarps * kTokens;
  const int rounds = (kTokens * units + 31) / 32;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kTokens; t0 < tokens; t0 += step) {
    // one lane per token: its cache row and its row of the output
    int64_t row = -1, out = -1;
    if (lane < kTokens && t0 + lane < tokens) {
      const int64_t t = t0 + lane, b = t / L.S, s = t - b * L.S;
      row = row_of(L, b, n, s);
      out = (b * L.N + n) * L.S + s;
      if (row == -2 && n == 0 && L.err_count) atomicAdd(L.err_count, 1);
    }
    for (int r0 = 0; r0 < rounds; r0 += kBatch) {
      uint4 in[kBatch];
      int64_t to[kBatch];
      int32_t unit[kBatch];
      bool have[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        const int i = (r0 + e) * 32 + lane, token = min(i / units, kTokens - 1);
        unit[e] = i - token * units;
        const int64_t from = __shfl_sync(0xffffffffu, row, token);
        to[e] = __shfl_sync(0xffffffffu, out, token);
        if (i >= kTokens * units) to[e] = -1;
        in[e] = make_uint4(0, 0, 0, 0);
        have[e] = to[e] >= 0 && from >= 0;
        if (have[e]) {
          const bool is_k = unit[e] < k.units;
          const Side& side = is_k ? k : v;
          const int64_t at = from * side.width + (is_k ? unit[e] : unit[e] - k.units) * 8;
          if (side.kind == kQuantNone) {
            in[e] = __ldcs(reinterpret_cast<const uint4*>(side.cache + at * 2));
          } else {
            const uint2 x = __ldcs(reinterpret_cast<const uint2*>(side.cache + at));
            in[e].x = x.x;
            in[e].y = x.y;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < kBatch; ++e) {
        if (to[e] < 0) continue;
        const bool is_k = unit[e] < k.units;
        const Side& side = is_k ? k : v;
        if (have[e] && side.kind != kQuantNone) {
          float x[8];
          codes_to_float(make_uint2(in[e].x, in[e].y), side.kind, x);
          const float4* tab = table + unit[e] * 4;
          const float4 ra = tab[0], rb = tab[1], ta = tab[2], tb = tab[3];
          in[e].x = pack_half2<!F16>(fmaf(x[0], ra.x, ta.x), fmaf(x[1], ra.y, ta.y));
          in[e].y = pack_half2<!F16>(fmaf(x[2], ra.z, ta.z), fmaf(x[3], ra.w, ta.w));
          in[e].z = pack_half2<!F16>(fmaf(x[4], rb.x, tb.x), fmaf(x[5], rb.y, tb.y));
          in[e].w = pack_half2<!F16>(fmaf(x[6], rb.z, tb.z), fmaf(x[7], rb.w, tb.w));
        }
        __stcs(reinterpret_cast<uint4*>(side.out + to[e] * side.width + (is_k ? unit[e] : unit[e] - k.units) * 8), in[e]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_cache_read(const ReadLaunch& L, cudaStream_t stream) {
  Side k{static_cast<const uint8_t*>(L.k_cache), L.k_scale, L.k_offset, L.k_out, L.kw, L.kq, L.k_scalar,
         L.k_out ? L.kw / 8 : 0};
  Side v{static_cast<const uint8_t*>(L.v_cache), L.v_scale, L.v_offset, L.v_out, L.vw, L.vq, L.v_scalar,
         L.v_out ? L.vw / 8 : 0};
  const int smem = (k.units + v.units) * 64;  // at most 16 KB
  const int64_t groups = (L.B * L.S + kWarps * kTokens - 1) / (kWarps * kTokens);
  // four blocks an SM, or fewer than that where there is less to do
  const int64_t blocks = std::min(groups, std::max<int64_t>(1, 4 * static_cast<int64_t>(device_sm_count()) / L.N));
  auto kernel = L.f16 ? cache_read_kernel<true> : cache_read_kernel<false>;
  kernel<<<dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(L.N)), kThreads, smem, stream>>>(L, k, v);
  return cudaGetLastError();
}

}  // namespace ra
