// Rows of the paged caches gathered by slot and dequantised: the inverse of
// kv_rms_norm_rope_cache's scatter,
//   out[b, n, s, c] = (code - offset[c]) / scale[c]   (16-bit caches: the element itself).
//
// An HBM stream of short scattered rows (1 or 2 bytes read, 2 written per element), so
// the mapping keeps loads in flight: a thread takes 8 channels (8 or 16 bytes in, 16 out)
// of kUnroll rows at once, with neighbouring threads on neighbouring channels.  The
// quantisation of its channels is the same in every row of a head and comes from L1.  The
// quotient is (code - offset) times the reciprocal of the scale, both fp32: within two
// units of fp32's last place, far below the rounding to 16 bits.
#include <cuda_fp8.h>

#include <algorithm>

#include "attention.h"
#include "attn_ptx.cuh"
#include "internal.h"
#include "kv_cache.h"

namespace ra {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

struct Side {                   // one of the two caches
  const uint8_t* cache;
  const float *scale, *offset;
  uint16_t* out;
  int32_t width, kind, scalar, chunks;  // chunks of 8 channels per row
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

template <bool F16>
__device__ __forceinline__ uint32_t half_pair(float a, float b) {
  return F16 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
}

template <bool F16>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ ReadLaunch L,
                                                              const __grid_constant__ Side k,
                                                              const __grid_constant__ Side v, int64_t rows) {
  const int per_row = k.chunks + v.chunks;
  const int64_t units = rows * per_row;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t u0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; u0 < units; u0 += step * kUnroll) {
    uint4 in[kUnroll];
    int64_t row[kUnroll];
    uint16_t* dst[kUnroll];
    int32_t chunk[kUnroll];
    int32_t head[kUnroll];
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
      const int64_t u = u0 + e * step;
      row[e] = -1;
      dst[e] = nullptr;
      in[e] = make_uint4(0, 0, 0, 0);
      if (u >= units) continue;
      const int64_t r = u / per_row;              // (b, n, s), s fastest
      const int32_t c = static_cast<int32_t>(u - r * per_row);
      const int64_t bn = r / L.S, s = r - bn * L.S, b = bn / L.N, n = bn - b * L.N;
      const bool is_k = c < k.chunks;
      const Side& side = is_k ? k : v;
      chunk[e] = is_k ? c : c - k.chunks;
      head[e] = static_cast<int32_t>(n);
      row[e] = row_of(L, b, n, s);
      dst[e] = side.out + r * side.width + chunk[e] * 8;
      if (row[e] == -2 && c == 0 && n == 0 && L.err_count) atomicAdd(L.err_count, 1);
      if (row[e] >= 0) {
        const int64_t at = row[e] * side.width + chunk[e] * 8;
        if (side.kind == kQuantNone) {
          in[e] = __ldg(reinterpret_cast<const uint4*>(side.cache + at * 2));
        } else {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(side.cache + at));
          in[e].x = x.x;
          in[e].y = x.y;
        }
      }
      chunk[e] = is_k ? chunk[e] : ~chunk[e];     // the sign says which cache
    }
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
      if (dst[e] == nullptr) continue;
      const bool is_k = chunk[e] >= 0;
      const Side& side = is_k ? k : v;
      if (row[e] >= 0 && side.kind != kQuantNone) {
        const int32_t c = (is_k ? chunk[e] : ~chunk[e]) * 8;
        float x[8];
        const uint32_t w[2] = {in[e].x, in[e].y};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t byte = (w[i >> 2] >> (8 * (i & 3))) & 0xFFu;
          if (side.kind == kQuantInt8)
            x[i] = static_cast<float>(static_cast<int32_t>(byte ^ 0x80u) - 128);
          else
            x[i] = __half2float(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte),
                                                        side.kind == kQuantE4m3 ? __NV_E4M3 : __NV_E5M2));
        }
        const int32_t base = (L.variant == 2 ? head[e] * side.width : 0) + c;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int32_t q = side.scalar ? 0 : base + i;
          x[i] = (x[i] - (side.offset ? __ldg(side.offset + q) : 0.f)) * __frcp_rn(__ldg(side.scale + q));
        }
        in[e] = make_uint4(half_pair<F16>(x[0], x[1]), half_pair<F16>(x[2], x[3]), half_pair<F16>(x[4], x[5]),
                           half_pair<F16>(x[6], x[7]));
      }
      *reinterpret_cast<uint4*>(dst[e]) = in[e];
    }
  }
}

}  // namespace

cudaError_t launch_cache_read(const ReadLaunch& L, cudaStream_t stream) {
  Side k{static_cast<const uint8_t*>(L.k_cache), L.k_scale, L.k_offset, L.k_out, L.kw, L.kq, L.k_scalar,
         L.k_out ? L.kw / 8 : 0};
  Side v{static_cast<const uint8_t*>(L.v_cache), L.v_scale, L.v_offset, L.v_out, L.vw, L.vq, L.v_scalar,
         L.v_out ? L.vw / 8 : 0};
  const int64_t rows = L.B * L.N * L.S, units = rows * (k.chunks + v.chunks);
  const int64_t blocks = std::min<int64_t>((units + kThreads - 1) / kThreads, static_cast<int64_t>(device_sm_count()) * 8);
  auto kernel = L.f16 ? cache_read_kernel<true> : cache_read_kernel<false>;
  kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(L, k, v, rows);
  return cudaGetLastError();
}

}  // namespace ra
