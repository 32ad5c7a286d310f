// Rows of the paged caches gathered by slot and dequantised: the inverse of
// kv_rms_norm_rope_cache's scatter,
//   out[b, n, s, c] = (code - offset[c]) / scale[c]   (16-bit caches: the element itself).
//
// An HBM stream of short scattered rows (1 or 2 bytes read, 2 written per element), so the
// mapping spends few instructions per byte and keeps loads in flight:
//  * a block serves one head, whose quantisation it turns once into a table in shared
//    memory: x = (code - offset) * r, r = 1 / scale.  The difference, r and the product are each
//    rounded to fp32, at most 3 * 2^-24 of x in all, and a code equal to its offset is 0.
//    (code * r - offset * r as one multiply-add is off by 2^-24 of offset / scale, however
//    small x is, and takes as long: 53 us both);
//  * a warp takes 4 tokens at once and spreads their rows' 8-channel units (8 or 16 bytes
//    in, 16 out) over its lanes: four rows fill them where one would not (64 + 8 units in a
//    latent and its rope part: 8 + 1 rounds of 32 lanes for four tokens, not 4 x 3), and the
//    slot lookups and the index arithmetic, done by one lane per token a turn ahead, are a
//    small part;
//  * the loads of kBatch rounds are in flight together.
// Measured (131072 rows of 512 + 64 int8 channels, 228 MB in all): 53 us, 4.3 TB/s, 63 %
// of a plain copy's rate; a mapping of one row per warp took 86 us.  Half of the issue slots
// are busy and DRAM at 40 % of its nominal rate: the latency of two dependent loads (slot,
// then row) at four blocks an SM bounds it.  Five blocks spill and are no faster (53 us).
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
constexpr int kBatch = 4;
constexpr uint32_t kNowhere = 0xFFFFFFFFu;

struct Side {                   // one of the two caches
  const uint8_t* cache;
  const float *scale, *offset;
  uint16_t* out;
  int32_t width, kind, scalar, units;  // units of 8 channels per row
};

// quotient of two numbers that are not negative: a 64-bit division is a hundred instructions,
// and few of these need it
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// A token's index entry, and the cache row of head n that it stands for (-1: none, -2:
// outside the cache).
struct Token {
  int64_t b, s, entry;
};
__device__ __forceinline__ Token load_token(const ReadLaunch& L, int64_t t) {
  Token k;
  k.b = quotient(t, L.S);
  k.s = t - k.b * L.S;
  k.entry = __ldg(L.index + (L.mode == kModePaBlkBnsd ? k.b * quotient(L.S + L.block_size - 1, L.block_size) + quotient(k.s, L.block_size)
                                                      : t));
  return k;
}
__device__ __forceinline__ int64_t row_of(const ReadLaunch& L, const Token& k, int64_t n) {
  const int64_t bs = L.block_size;
  if (k.entry == -1) return -1;
  if (L.mode == kModeNorm) return k.entry < 0 || k.entry >= L.cache_seq ? -2 : (k.b * L.N + n) * L.cache_seq + k.entry;
  const int64_t slots = L.block_num * bs;
  if (k.entry < 0 || k.entry >= slots) return -2;
  const int64_t slot = k.entry + (L.mode == kModePaBlkBnsd ? k.s - quotient(k.s, bs) * bs : 0);
  if (slot >= slots) return -2;
  const int64_t page = quotient(slot, bs);
  return L.mode == kModePa ? slot * L.N + n : (page * L.N + n) * bs + (slot - page * bs);
}

// 8 codes -> 8 floats
__device__ __forceinline__ void codes_to_float(uint2 w, int32_t kind, float2 (&x)[4]) {
  const uint32_t v[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (kind == kQuantInt8) {
      // the byte code + 128 below the exponent of 2^23 is the float 2^23 + code + 128
      const uint32_t u = v[i] ^ 0x80808080u;
      const float2 bias = make_float2(-8388736.f, -8388736.f);
      x[2 * i] = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)),
                                        __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441))), bias);
      x[2 * i + 1] = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)),
                                            __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443))), bias);
    } else {
      const __nv_fp8_interpretation_t f = kind == kQuantE4m3 ? __NV_E4M3 : __NV_E5M2;
      const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v[i] & 0xFFFFu), f);
      const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v[i] >> 16), f);
      x[2 * i] = make_float2(__half2float(__ushort_as_half(lo.x)), __half2float(__ushort_as_half(lo.y)));
      x[2 * i + 1] = make_float2(__half2float(__ushort_as_half(hi.x)), __half2float(__ushort_as_half(hi.y)));
    }
  }
}

// One cache's rows of a warp's tokens.  rows: per token its cache row and its row of the
// output; place: for every (round, lane) its token (upper half) and unit; tab: the side's
// quantisation, four arrays of a float4 per unit: 1 / scale (two), -offset (two).
template <bool F16>
__device__ __forceinline__ void read_side(const Side& side, const int64_t (*rows)[2], const uint32_t* place,
                                          const float4* tab, int lane) {
  const int rounds = (kTokens * side.units + 31) / 32;
  const bool codes = side.kind != kQuantNone;
  for (int r0 = 0; r0 < rounds; r0 += kBatch) {
    uint4 in[kBatch];
    uint4* to[kBatch];
    int32_t unit[kBatch];
    bool have[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const uint32_t at = r0 + e < rounds ? place[(r0 + e) * 32 + lane] : kNowhere;
      unit[e] = at & 0xFFFFu;
      to[e] = nullptr;
      have[e] = false;
      in[e] = make_uint4(0, 0, 0, 0);
      if (at == kNowhere) continue;
      const longlong2 row = *reinterpret_cast<const longlong2*>(rows[at >> 16]);
      if (row.y < 0) continue;
      to[e] = reinterpret_cast<uint4*>(side.out + row.y * side.width) + unit[e];
      have[e] = row.x >= 0;
      if (!have[e]) continue;
      if (codes) {
        const uint2 x = __ldcs(reinterpret_cast<const uint2*>(side.cache + row.x * side.width) + unit[e]);
        in[e].x = x.x;
        in[e].y = x.y;
      } else {
        in[e] = __ldcs(reinterpret_cast<const uint4*>(side.cache + row.x * side.width * 2) + unit[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      if (to[e] == nullptr) continue;
      if (have[e] && codes) {
        float2 x[4];
        codes_to_float(make_uint2(in[e].x, in[e].y), side.kind, x);
        const float4* t = tab + unit[e];
        const float4 ra = t[0], rb = t[side.units], ta = t[2 * side.units], tb = t[3 * side.units];
        x[0] = __fmul2_rn(make_float2(x[0].x + ta.x, x[0].y + ta.y), make_float2(ra.x, ra.y));
        x[1] = __fmul2_rn(make_float2(x[1].x + ta.z, x[1].y + ta.w), make_float2(ra.z, ra.w));
        x[2] = __fmul2_rn(make_float2(x[2].x + tb.x, x[2].y + tb.y), make_float2(rb.x, rb.y));
        x[3] = __fmul2_rn(make_float2(x[3].x + tb.z, x[3].y + tb.w), make_float2(rb.z, rb.w));
        in[e] = make_uint4(pack_half2<!F16>(x[0].x, x[0].y), pack_half2<!F16>(x[1].x, x[1].y),
                           pack_half2<!F16>(x[2].x, x[2].y), pack_half2<!F16>(x[3].x, x[3].y));
      }
      __stcs(to[e], in[e]);
    }
  }
}

// the side's table of head n, and its places
__device__ __forceinline__ void set_up(const Side& side, int32_t head, bool per_head, float4* tab, uint32_t* place) {
  for (int i = threadIdx.x; side.kind != kQuantNone && i < side.width; i += kThreads) {
    const int at = side.scalar ? 0 : (per_head ? head * side.width : 0) + i;
    float* const t = reinterpret_cast<float*>(tab + ((i >> 2) & 1) * side.units + (i >> 3)) + (i & 3);
    t[0] = __frcp_rn(__ldg(side.scale + at));
    t[8 * side.units] = side.offset ? -__ldg(side.offset + at) : 0.f;
  }
  for (int i = threadIdx.x; i < (kTokens * side.units + 31) / 32 * 32; i += kThreads) {
    const int token = i / side.units;
    place[i] = token < kTokens ? (token << 16) | (i - token * side.units) : kNowhere;
  }
}

template <bool F16>
__global__ void __launch_bounds__(kThreads, 4) cache_read_kernel(const __grid_constant__ ReadLaunch L,
                                                              const __grid_constant__ Side k,
                                                              const __grid_constant__ Side v) {
  extern __shared__ float4 shared[];
  __shared__ __align__(16) int64_t rows[kWarps][kTokens][2];
  const int64_t n = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float4 *const k_tab = shared, *const v_tab = k_tab + 4 * k.units;
  uint32_t* const k_place = reinterpret_cast<uint32_t*>(v_tab + 4 * v.units);
  uint32_t* const v_place = k_place + (kTokens * k.units + 31) / 32 * 32;
  if (k.units) set_up(k, static_cast<int32_t>(n), L.variant == 2, k_tab, k_place);
  if (v.units) set_up(v, static_cast<int32_t>(n), L.variant == 2, v_tab, v_place);
  __syncthreads();
  const int64_t tokens = L.B * L.S, step = static_cast<int64_t>(gridDim.x) * kWarps * kTokens;
  int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kTokens;
  Token next{0, 0, -1};                      // one lane per token; its entry is on the way a turn ahead
  if (lane < kTokens && t0 + lane < tokens) next = load_token(L, t0 + lane);
  for (; t0 < tokens; t0 += step) {
    if (lane < kTokens) {
      const Token token = next;
      const bool real = t0 + lane < tokens;
      const int64_t row = real ? row_of(L, token, n) : -1;
      if (row == -2 && n == 0 && L.err_count) atomicAdd(L.err_count, 1);
      rows[warp][lane][0] = row;
      rows[warp][lane][1] = real ? (token.b * L.N + n) * L.S + token.s : -1;
      if (t0 + step + lane < tokens) next = load_token(L, t0 + step + lane);
    }
    __syncwarp();
    if (v.units) read_side<F16>(v, rows[warp], v_place, v_tab, lane);
    if (k.units) read_side<F16>(k, rows[warp], k_place, k_tab, lane);
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_cache_read(const ReadLaunch& L, cudaStream_t stream) {
  Side k{static_cast<const uint8_t*>(L.k_cache), L.k_scale, L.k_offset, L.k_out, L.kw, L.kq, L.k_scalar,
         L.k_out ? L.kw / 8 : 0};
  Side v{static_cast<const uint8_t*>(L.v_cache), L.v_scale, L.v_offset, L.v_out, L.vw, L.vq, L.v_scalar,
         L.v_out ? L.vw / 8 : 0};
  const int units = k.units + v.units;
  const int smem = units * 64 + ((kTokens * k.units + 31) / 32 + (kTokens * v.units + 31) / 32) * 128;  // at most 20 KB
  const int64_t groups = (L.B * L.S + kWarps * kTokens - 1) / (kWarps * kTokens);
  // four blocks an SM, or fewer where there is less to do
  const int64_t blocks = std::min(groups, std::max<int64_t>(1, 4 * static_cast<int64_t>(device_sm_count()) / L.N));
  auto kernel = L.f16 ? cache_read_kernel<true> : cache_read_kernel<false>;
  kernel<<<dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(L.N)), kThreads, smem, stream>>>(L, k, v);
  return cudaGetLastError();
}

}  // namespace ra
