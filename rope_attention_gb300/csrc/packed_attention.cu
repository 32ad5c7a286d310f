// Attention over packed prompts: softmax(scale q k^T) v on the projection's own output.
//
//   out[i, h] = sum_j p[i, j] v[j, h / g] / sum_j p[i, j],
//   p[i, j]   = exp(scale * q[i, h] . k[j, h / g] - m_i)   over the keys j that i sees:
//   those of its own sequence, and with `causal` those with j <= i + Lk - Lq
// (g = num_heads / num_kv_heads).  A row that sees no key is zero, its lse -inf.
//
// One pass over the keys with a running maximum and sum.  The maximum only has to keep
// the exponentials in range, so a row keeps the one it has until a tile exceeds it by
// 2^kLazy; only then is its accumulator rescaled (the exact result is unchanged: the
// factor exp(-m) cancels between the sum over v and the sum of p).
//
// GB300 mapping: a block owns two 128-row query tiles of one head and streams 128-key
// tiles of K and V through a shared-memory ring (TMA, 128-byte swizzle).  Both products
// run on tcgen05: S = Q K^T from shared memory, O += P V with P read from TMEM, where
// the softmax left it in place of S.  While one tile's softmax runs, the tensor core
// works on the other's products.  Tensor memory: S/P of the two tiles, then their O.
// Warps 0-3 and 4-7: softmax of the two tiles, one row per thread, which also rescale and
// write O; warp 8: TMA; warp 9: MMA (10 and 11 only give up registers).  P is rounded to the input's 16-bit type for the
// tensor core (half a step, 2^-9 for bf16, of each weight); S, m, l and O are fp32.
//
// Every wait is bounded in time (status word, as in the projection).
#include <algorithm>
#include <atomic>
#include <cmath>

#include "attention.h"
#include "attn_ptx.cuh"
#include "internal.h"

namespace ra {
namespace {

constexpr int kRows = 128;                  // query rows per tile
constexpr int kKeys = 128;                  // keys per tile
constexpr int kThreads = 384;                // three warpgroups
// Registers per thread: launched with 168 each (384 x 168 of the SM's 65536), then moved
// from the third warpgroup to the softmax: 2 x 224 + 56 = 3 x 168
constexpr int kRegsSoftmax = 224, kRegsRest = 56;
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr float kLazy = 8.f;                // log2 of how far a tile may exceed the running maximum
constexpr uint64_t kDrainNs = 200000000ull;

struct Params {
  CUtensorMap tq, tk, tv;                   // 3-D: (d, heads, tokens) or (d, tokens, heads)
  uint16_t* out;
  float* lse;
  const int32_t *cu_q, *cu_k;
  int32_t B, total_q, total_k, nq, g, d, causal;
  int32_t q_swap, k_swap, v_swap;           // the map's axis order is (d, tokens, heads)
  int64_t o_ts, o_hs;
  float scale, sl2;                         // softmax scale, and with log2(e)
  int32_t out16;                            // out rows are 16-byte aligned
  int32_t* status;
  uint64_t wait_ns;
  int32_t stall_loads;
};

template <int DP>
struct Shape {
  static constexpr int kSlabs = DP / 64;    // 64-channel slabs of a tile
  static constexpr int kSlabBytes = kRows * 128;
  static constexpr int kTileBytes = kSlabs * kSlabBytes;
  static constexpr int kStages = DP == 128 ? 5 : 8;
  static constexpr int kRing = 2 * kTileBytes;
  static constexpr int kBar = kRing + kStages * kTileBytes;
  static constexpr int kNumBars = 2 * kStages + 2 + 2 + 2 + 2 + 1;
  static constexpr int kMisc = kBar + 8 * kNumBars;
  static constexpr int kSmem = kMisc + 16 + 1024;
  static_assert(kSmem <= 232448, "shared memory budget");
};

// start and length of sequence b, clamped to the tokens that exist
__device__ __forceinline__ void seq_span(const int32_t* cu, int32_t b, int32_t B, int32_t total, int32_t& start,
                                         int32_t& len) {
  if (cu == nullptr) {
    len = total / B;
    start = b * len;
    return;
  }
  const int32_t lo = min(max(__ldg(cu + b), 0), total), hi = min(max(__ldg(cu + b + 1), lo), total);
  start = lo;
  len = hi - lo;
}

// The sequence that holds work item `item` (blocks of 256 query rows, sequence after
// sequence) and the block's number in it; false when there is no such item.  Whole warp.
__device__ __forceinline__ bool find_item(const Params& p, int32_t item, int32_t& b, int32_t& blk) {
  const int lane = threadIdx.x & 31;
  int32_t before = 0;
  for (int32_t base = 0; base < p.B; base += 32) {
    int32_t start, len = 0;
    if (base + lane < p.B) seq_span(p.cu_q, base + lane, p.B, p.total_q, start, len);
    const int32_t n = (len + 2 * kRows - 1) / (2 * kRows);
    int32_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, item < before + incl);
    if (hit) {
      const int src = __ffs(hit) - 1;
      b = base + src;
      blk = item - before - __shfl_sync(0xffffffffu, incl - n, src);
      return true;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

template <int DP, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) packed_attention_kernel(const __grid_constant__ Params p) {
  using SH = Shape<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t s0 = smem_u32(smem);
  const uint32_t bars = s0 + SH::kBar;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (SH::kStages + s); };
  auto q_full = [&](int i) { return bars + 8u * (2 * SH::kStages + i); };
  auto s_full = [&](int i) { return bars + 8u * (2 * SH::kStages + 2 + i); };
  auto p_ready = [&](int i) { return bars + 8u * (2 * SH::kStages + 4 + i); };
  auto o_done = [&](int i) { return bars + 8u * (2 * SH::kStages + 6 + i); };
  const uint32_t drain_bar = bars + 8u * (2 * SH::kStages + 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SH::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SH::kMisc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t b, blk;
  if (!find_item(p, static_cast<int32_t>(blockIdx.x), b, blk)) return;  // the same answer in every warp
  const int32_t head = static_cast<int32_t>(blockIdx.y), kv_head = head / p.g;
  int32_t q_start, Lq, k_start, Lk;
  seq_span(p.cu_q, b, p.B, p.total_q, q_start, Lq);
  seq_span(p.cu_k, b, p.B, p.total_k, k_start, Lk);
  // keys seen by the last row of each tile, and the tiles of keys that takes
  int32_t n_tiles[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int32_t first = (2 * blk + i) * kRows, last = min(Lq, first + kRows) - 1;
    const int32_t seen = p.causal ? min(Lk, max(0, last + 1 + Lk - Lq)) : Lk;
    n_tiles[i] = last < first ? 0 : (seen + kKeys - 1) / kKeys;
  }
  const int32_t n_max = max(n_tiles[0], n_tiles[1]);

  if (threadIdx.x == 0) {
    for (int s = 0; s < SH::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(s_full(i), 1);
      mbar_init(p_ready(i), 128);
      mbar_init(o_done(i), 1);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto s_col = [&](int i) { return tmem + 128u * i; };
  auto o_col = [&](int i) { return tmem + 256u + 128u * i; };

  if (warp >= 8) {
    set_max_regs_dec<kRegsRest>();
  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ loads
    if (lane == 0 && !p.stall_loads && n_max > 0) {
      uint32_t armed = 0, armed_parity = 0;
      auto load_tile = [&](const CUtensorMap* m, int swap, uint32_t dst, uint32_t bar, int32_t token, int32_t h) {
#pragma unroll
        for (int c = 0; c < SH::kSlabs; ++c)
          tma_load_3d(dst + c * SH::kSlabBytes, m, bar, 64 * c, swap ? token : h, swap ? h : token);
      };
      auto load_q = [&](int i) {
        if (n_tiles[i] == 0) return;
        mbar_arrive_expect_tx(q_full(i), SH::kTileBytes);
        load_tile(&p.tq, p.q_swap, s0 + i * SH::kTileBytes, q_full(i), q_start + (2 * blk + i) * kRows, head);
      };
      bool ok = true;
      load_q(0);
      for (int32_t u = 0; ok && u < 2 * n_max; ++u) {  // K 0, V 0, K 1, V 1, ...
        const int st = u % SH::kStages;
        const uint32_t par = (u / SH::kStages) & 1;
        if (!bounded_wait_one(empty(st), par ^ 1u, p.wait_ns, abort_flag)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(full(st), SH::kTileBytes);
        if (u & 1)
          load_tile(&p.tv, p.v_swap, s0 + SH::kRing + st * SH::kTileBytes, full(st), k_start + (u >> 1) * kKeys, kv_head);
        else
          load_tile(&p.tk, p.k_swap, s0 + SH::kRing + st * SH::kTileBytes, full(st), k_start + (u >> 1) * kKeys, kv_head);
        armed |= 1u << st;
        armed_parity = (armed_parity & ~(1u << st)) | (par << st);
        if (u == 0) load_q(1);
      }
      if (!ok || *abort_flag) {  // let every copy in flight land before the block leaves
        for (int s = 0; s < SH::kStages; ++s)
          if (armed & (1u << s)) bounded_drain(full(s), (armed_parity >> s) & 1u, kDrainNs);
        for (int i = 0; i < 2; ++i)
          if (n_tiles[i]) bounded_drain(q_full(i), 0, kDrainNs);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    if (n_max > 0) {
      constexpr uint32_t id_s = idesc_f16(BF16, false, false, kRows, kKeys);
      constexpr uint32_t id_o = idesc_f16(BF16, false, true, kRows, DP);
      const uint64_t ring_k = sdesc_kmajor_sw128(s0 + SH::kRing);
      const uint64_t ring_v = sdesc_mnmajor_sw128(s0 + SH::kRing, SH::kSlabBytes);
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t par) {
        if (ok) ok = bounded_wait_warp(bar, par, p.wait_ns, abort_flag);
        return ok;
      };
      auto issue_s = [&](int i, int st) {  // one lane
        const uint64_t a = sdesc_kmajor_sw128(s0 + i * SH::kTileBytes);
        const uint64_t bd = ring_k + static_cast<uint64_t>(st * (SH::kTileBytes >> 4));
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint32_t off = (k >> 2) * (SH::kSlabBytes >> 4) + (k & 3) * 2;
          mma_f16_ss(s_col(i), a + off, bd + off, id_s, k > 0);
        }
        tc_commit(s_full(i));
      };
      if (wait(full(0), 0)) {
        for (int i = 0; i < 2; ++i)
          if (n_tiles[i] > 0 && wait(q_full(i), 0)) {
            tc_fence_after();
            if (elect_one()) issue_s(i, 0);
            __syncwarp();
          }
        if (ok && elect_one()) tc_commit(empty(0));
        __syncwarp();
      }
      int sv = 1, sk = 2;                        // ring stages of V j and K j + 1
      uint32_t par_v = 0, par_k = 0;
      for (int32_t j = 0; ok && j < n_max; ++j) {
        if (!wait(full(sv), par_v)) break;
        if (j + 1 < n_max && !wait(full(sk), par_k)) break;
        for (int i = 0; i < 2; ++i) {
          if (j >= n_tiles[i]) continue;
          if (!wait(p_ready(i), j & 1)) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t bd = ring_v + static_cast<uint64_t>(sv * (SH::kTileBytes >> 4));
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              mma_f16_ts(o_col(i), s_col(i) + 8 * k, bd + 128 * k, id_o, j > 0 || k > 0);
            if (j + 1 < n_tiles[i]) issue_s(i, sk);
            else tc_commit(o_done(i));
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) {
          tc_commit(empty(sv));
          if (j + 1 < n_max) tc_commit(empty(sk));
        }
        __syncwarp();
        if ((sv += 2) >= SH::kStages) sv -= SH::kStages, par_v ^= 1u;
        if ((sk += 2) >= SH::kStages) sk -= SH::kStages, par_k ^= 1u;
      }
      if (elect_one()) tc_commit(drain_bar);  // every product must finish before TMEM is released
      __syncwarp();
      bounded_drain(drain_bar, 0, kDrainNs);
    }
    __syncwarp();
  }
  } else {
    // ------------------------------------------------------------ softmax, one row per thread
    set_max_regs_inc<kRegsSoftmax>();
    const int i = warp >> 2, row = threadIdx.x & 127;
    const int32_t tile_row = (2 * blk + i) * kRows + row;  // row in the sequence
    const bool real = tile_row < Lq;
    const int32_t seen = !p.causal ? Lk : min(Lk, max(0, tile_row + 1 + Lk - Lq));
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_addr = s_col(i) + lane_base, o_addr = o_col(i) + lane_base;
    float m = neg_inf(), l = 0.f;
    bool ok = true;
    const float lazy = kLazy / p.sl2;
    for (int32_t j = 0; j < n_tiles[i]; ++j) {
      if (!bounded_wait_warp(s_full(i), j & 1, p.wait_ns, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t s[kKeys];
#pragma unroll
      for (int c = 0; c < kKeys; c += 32) tmem_ld_x32(s_addr + c, s + c);
      tmem_ld_wait();
      const int32_t nv = seen - j * kKeys;  // keys of this tile that the row sees
      if (__any_sync(0xffffffffu, nv < kKeys)) {
#pragma unroll
        for (int c = 0; c < kKeys; ++c)
          if (c >= nv) s[c] = __float_as_uint(neg_inf());
      }
      float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
      for (int c = 0; c < kKeys; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mx[e] = fmaxf(mx[e], fmaxf(__uint_as_float(s[c + e]), __uint_as_float(s[c + 4 + e])));
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (__any_sync(0xffffffffu, top > m + lazy)) {
        const float m_new = fmaxf(m, top);
        const float f = m_new == neg_inf() ? 1.f : ex2((m - m_new) * p.sl2);
        m = m_new;
        l *= f;
        if (j > 0) {  // S(j) was issued behind O += P V of tile j - 1, so O is complete here
#pragma unroll
          for (int c = 0; c < DP; c += 32) {
            uint32_t o[32];
            tmem_ld_x32(o_addr + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st_x32(o_addr + c, o);
          }
        }
      }
      const float neg = m == neg_inf() ? 0.f : -m * p.sl2;
      const float2 sl = make_float2(p.sl2, p.sl2), ng = make_float2(neg, neg);
      float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t w[16];
        exp_batch<BF16>(s + 32 * h, sl, ng, acc, w);
        tmem_st_x16(s_addr + 16 * h, w);  // P takes the place of S: 64 columns of pairs
      }
      const float2 sum = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
      l += sum.x + sum.y;
      if ((j + 1) * kKeys > Lk) {
        // V rows behind the sequence's end meet P = 0, but 0 times a stray NaN or
        // infinity is NaN: zero them in shared memory
        const int32_t u = 2 * j + 1;
        const int st = u % SH::kStages;
        if (!bounded_wait_warp(full(st), (u / SH::kStages) & 1, p.wait_ns, abort_flag)) {
          ok = false;
          break;
        }
        if (row >= Lk - j * kKeys) {
#pragma unroll
          for (int c = 0; c < SH::kSlabs; ++c) {
            uint4* dst = reinterpret_cast<uint4*>(smem + SH::kRing + st * SH::kTileBytes + c * SH::kSlabBytes + row * 128);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(p_ready(i));
    }
    if (ok && n_tiles[i] > 0) ok = bounded_wait_warp(o_done(i), 0, p.wait_ns, abort_flag);
    if (ok) {
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : 0.f;
      uint16_t* dst = p.out + static_cast<int64_t>(q_start + tile_row) * p.o_ts + static_cast<int64_t>(head) * p.o_hs;
#pragma unroll
      for (int c = 0; c < DP; c += 32) {
        uint32_t o[32];
        if (n_tiles[i] > 0) {
          tmem_ld_x32(o_addr + c, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (real) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            if (c + e < p.d) {
              // a row that sees nothing is zero whatever its accumulator holds
              uint4 w = make_uint4(0, 0, 0, 0);
              if (l > 0.f) {
                w.x = pack_half2<BF16>(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                w.y = pack_half2<BF16>(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                w.z = pack_half2<BF16>(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
                w.w = pack_half2<BF16>(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
              }
              *reinterpret_cast<uint4*>(dst + c + e) = w;
            }
          }
        }
      }
      if (real && p.lse)
        p.lse[static_cast<int64_t>(q_start + tile_row) * p.nq + head] =
            l > 0.f ? m * p.scale + logf(l) : neg_inf();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && *abort_flag) *p.status = 1;
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// [tokens, heads, d] with any strides as a 3-D map of 64 x 128-token boxes; the axis with
// the smaller stride comes second
bool make_map(CUtensorMap* m, const uint16_t* base, int64_t tokens, int64_t heads, int32_t d, int64_t ts, int64_t hs,
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

template <int DP, bool BF16>
cudaError_t launch(const Params& p, int64_t items, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto kernel = packed_attention_kernel<DP, BF16>;
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<DP>::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev);
  }
  const dim3 grid(static_cast<unsigned>(items), static_cast<unsigned>(p.nq));
  kernel<<<grid, kThreads, Shape<DP>::kSmem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_packed_attention(const PackedLaunch& L, cudaStream_t stream, const char** why) {
  Params p{};
  if (!make_map(&p.tq, L.q, L.total_q, L.nq, L.d, L.q_ts, L.q_hs, &p.q_swap) ||
      !make_map(&p.tk, L.k, L.total_k, L.nkv, L.d, L.k_ts, L.k_hs, &p.k_swap) ||
      !make_map(&p.tv, L.v, L.total_k, L.nkv, L.d, L.v_ts, L.v_hs, &p.v_swap)) {
    *why = "cuTensorMapEncodeTiled failed or is unavailable";
    return cudaErrorInvalidValue;
  }
  p.out = L.out;
  p.lse = L.lse;
  p.cu_q = L.cu_q;
  p.cu_k = L.cu_k;
  p.B = static_cast<int32_t>(L.B);
  p.total_q = static_cast<int32_t>(L.total_q);
  p.total_k = static_cast<int32_t>(L.total_k);
  p.nq = L.nq;
  p.g = L.nq / L.nkv;
  p.d = L.d;
  p.causal = L.causal;
  p.o_ts = L.o_ts;
  p.o_hs = L.o_hs;
  p.scale = L.scale;
  p.sl2 = static_cast<float>(static_cast<double>(L.scale) * 1.4426950408889634);
  p.status = L.status;
  p.wait_ns = static_cast<uint64_t>(L.wait_ns);
  p.stall_loads = L.stall_loads;
  // at most this many blocks of 256 rows over the sequences; those beyond find no work
  const int64_t block = 2 * kRows;
  const int64_t items = L.cu_q ? std::min(L.total_q, L.total_q / block + L.B)
                               : L.B * ((L.total_q / L.B + block - 1) / block);
  if (L.d <= 64) return L.f16 ? launch<64, false>(p, items, stream) : launch<64, true>(p, items, stream);
  return L.f16 ? launch<128, false>(p, items, stream) : launch<128, true>(p, items, stream);
}

}  // namespace ra
