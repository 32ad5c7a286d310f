// Work shared out in runs of key tiles, and the joining of what a run cuts in two.
//
// Both attention kernels lay the key tiles of all their work items end to end and give
// each block an equal run, so blocks finish together whatever the lengths (or, where items are
// many or a cut would save too little, runs of whole items).  A block that
// gets a part of an item stores the part's (max, sum, accumulator) in the workspace; the
// second kernel here joins an item's parts in the order of the blocks, so results do not
// depend on which block finished first.
//
// The join is bound by latency: a chain of dependent loads (the cut, the statistics, the parts)
// behind a launch, 7 to 13 us of 44 to 160 where every item is cut (40 MB of parts, mostly from
// L2).  Where the host knows that nothing is cut it is not launched.
#pragma once

#include <algorithm>

#include "attention.h"
#include "attn_ptx.cuh"
#include "internal.h"

namespace ra {
namespace {

constexpr int kMaxBlocks = 160;           // blocks that a workspace has room for (a GB300 has 152 SMs)

// a position in a ring of stages: the stage, and the parity of its barriers' phase.  (A
// division by the number of stages costs a lone warp 150 cycles or more.)
struct Ring {
  int32_t stage = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next(int32_t stages) {
    if (++stage == stages) {
      stage = 0;
      parity ^= 1u;
    }
  }
};

// What a query sees of the keys up to its own position: the last `window` of them and the first
// `sinks`.  Key tiles that no row of a row tile sees are left out of the line: its tiles are the
// sink tiles, then those from the first row's window on (`skip` tiles further).
struct Window {
  int32_t window, sinks;                    // window 0: every key
  int32_t tiles;                            // tiles that the sinks take
  int32_t most;                             // tiles that a row tile's rows can see
};
// the first position of the window that ends at `pos` (negative: there is none)
__device__ __forceinline__ int32_t window_from(const Window& w, int32_t pos) {
  return w.window > 0 && pos >= w.window ? pos - w.window + 1 : 0;
}
// For rows of `tokens` tokens and key tiles of `keys`: seen positions from window_from(first) to the
// last token's are window + tokens - 1 at most, anywhere in their first tile.
inline Window make_window(int64_t window, int64_t sinks, int64_t tokens, int64_t keys) {
  Window w{};
  if (window <= 0) {
    w.most = 0x7fffffff;
    return w;
  }
  w.window = static_cast<int32_t>(std::min<int64_t>(window, kMostPositions));
  w.sinks = static_cast<int32_t>(std::min<int64_t>(sinks, kMostPositions));
  w.tiles = static_cast<int32_t>((w.sinks + keys - 1) / keys);
  w.most = static_cast<int32_t>(std::min<int64_t>(0x7fffffff, w.tiles + (w.window + tokens + 2 * keys - 3) / keys));
  return w;
}

// A prefix whose positions stand before every sequence's own, in tiles of their own: the other way to
// serve one, in a single call without sharing its reads.
struct SharedPrefix {
  const int32_t *len, *table;               // null: none
  int32_t cap;                              // positions that it can have
};
__device__ __forceinline__ int32_t prefix_length(const SharedPrefix& x) { return x.len ? min(max(__ldg(x.len), 0), x.cap) : 0; }

// Rows that another call's rows join (attention.h, PagedLaunch): its results in fp32, with their
// statistics.
struct Prior {
  float* rows_out;
  float4* stats_out;
  const float* rows;
  const float4* stats;
};

// The end of row `at`: m (log2) and l its statistics, k0 the lse's share of the key offsets (0 where
// l is).  They go out, or the prior's are weighed with them: share.x is the row's own, share.y the prior's.
// The maxima go from one call to the other by themselves: their difference is exact, where log2 of a whole sum,
// m + log2 l, is rounded by up to |m| 2^-24, which for large scores is more than the rows' own rounding.
// A side that saw nothing has l = 0 (and counts for nothing whatever its m); a NaN on either side makes the row NaN.
__device__ __forceinline__ void prior_end(const Prior& p, int64_t at, float m, float l, float k0, bool writes, float* lse,
                                          float2& share, const float4* have = nullptr) {
  if (p.stats_out) {
    if (writes) p.stats_out[at] = make_float4(m, l, k0, 0.f);
    return;
  }
  const float4 o = have ? *have : p.stats[at];
  const float own_m = l != 0.f ? m : neg_inf(), prior_m = o.y != 0.f ? o.x : neg_inf(), top = fmaxf(own_m, prior_m);
  const float own = l != 0.f ? l * ex2(own_m - top) : 0.f, prior = o.y != 0.f ? o.y * ex2(prior_m - top) : 0.f, sum = own + prior;
  share = sum != 0.f ? make_float2(own / sum, prior / sum) : make_float2(0.f, 0.f);
  if (writes && lse) lse[at] = sum != 0.f ? top * 0.6931471805599453f + logf(sum) + (l != 0.f ? k0 : o.z) : neg_inf();
}

// A part of block c is its first piece (slot 2 c) where the item began before the block's
// run, else its last (2 c + 1).
struct JoinParams {
  float4* stats;                // [2 G][NR] (max in log2 units, sum, the lse's share of the key offsets, -)
  float* parts;                 // [2 G][NR][Dv] unscaled accumulators
  int32_t* meta;                // [G][8]: an item to join (0 / 1), its first and last block, rows of its one or
                                // two subtiles, first token (of all), first head, kv head
  uint16_t* out;
  float* lse;
  const float *v_scale, *v_offset;
  int64_t o_ts, o_hs;           // strides of out
  int32_t heads, hb, tb;        // a subtile: tb tokens x hb heads
  int32_t Dv, NR, sub;          // rows of a part, rows of a subtile (NR or NR / 2)
  int32_t per_head, v_scalar;   // the value's quantisation: [N, Dv], or [Dv] ([1])
  Prior prior;
  int32_t split;                // EXT: warps that share a row's many pieces
};

template <bool F16>
__device__ __forceinline__ uint16_t to_half(float x) {
  return F16 ? __half_as_ushort(__float2half_rn(x)) : __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
// scale and offset of one channel of a cache row (1 and 0 for a 16-bit cache)
__device__ __forceinline__ float2 channel_quant(const float* scale, const float* offset, int32_t at, int32_t scalar) {
  if (scale == nullptr) return make_float2(1.f, 0.f);
  const int32_t i = scalar ? 0 : at;
  return make_float2(__ldg(scale + i), offset ? __ldg(offset + i) : 0.f);
}

// Blocks (x, *) join the item whose first cut lies before block x of the main kernel, where its
// `meta` says that there is one; where few blocks can have one, before the x-th that has.  An item of few pieces: a warp takes four
// rows' 128 channels at once, the rows' statistics side by side in its lanes, so that the
// loads of four rows are in flight.  One with many: the block's eight warps take every
// eighth piece of one row's 128 channels, and their sums are added in a fixed order.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kJoinFew = 8, kJoinFewItems = 4;  // pieces up to which a warp takes rows alone; where few items are cut
constexpr int kJoinLoads = (kMaxBlocks + 31) / 32;

struct JoinRow {
  int32_t part;                             // row of a part
  int64_t token, head;
};
__device__ __forceinline__ JoinRow join_row(const JoinParams& p, int32_t rows0, int32_t tok0, int32_t head0, int32_t r) {
  const int32_t in = r < rows0 ? r : r - rows0;                     // row of its subtile
  const int32_t t = static_cast<int32_t>(static_cast<uint32_t>(in) / static_cast<uint32_t>(p.hb));
  return JoinRow{r < rows0 ? r : p.sub + in, tok0 + (r < rows0 ? 0 : p.tb) + t, head0 + in - t * p.hb};
}
// share: of the row's own result and of the prior's (EXT); have: the prior's, where it has been fetched
template <bool F16, bool EXT>
__device__ __forceinline__ void join_store(const JoinParams& p, const JoinRow& row, int32_t kv_head, int32_t ch, float4 acc,
                                           float l, float2 share, const float4* have = nullptr) {
  const float inv = l != 0.f ? rcp(l) : 0.f;
  float y[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
  if (p.v_scale) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 so = channel_quant(p.v_scale, p.v_offset, (p.per_head ? kv_head * p.Dv : 0) + ch + e, p.v_scalar);
      y[e] = l != 0.f ? (y[e] - so.y) * rcp(so.x) : 0.f;
    }
  }
  if constexpr (EXT) {
    const int64_t at = (row.token * p.heads + row.head) * p.Dv + ch;
    if (p.prior.rows_out) {
      *reinterpret_cast<float4*>(p.prior.rows_out + at) = make_float4(y[0], y[1], y[2], y[3]);
      return;
    }
    if (p.prior.rows) {
      const float4 o = have ? *have : *reinterpret_cast<const float4*>(p.prior.rows + at);
      y[0] = fmaf(y[0], share.x, o.x * share.y);
      y[1] = fmaf(y[1], share.x, o.y * share.y);
      y[2] = fmaf(y[2], share.x, o.z * share.y);
      y[3] = fmaf(y[3], share.x, o.w * share.y);
    }
  }
  *reinterpret_cast<uint2*>(p.out + row.token * p.o_ts + row.head * p.o_hs + ch) =
      make_uint2(pack_half2<!F16>(y[0], y[1]), pack_half2<!F16>(y[2], y[3]));
}
__device__ __forceinline__ void join_lse(const JoinParams& p, const JoinRow& row, float m, float l, float k0) {
  p.lse[row.token * p.heads + row.head] = l != 0.f ? m * 0.6931471805599453f + logf(l) + k0 : neg_inf();
}
// The end of a row's statistics: m and k0 as in the parts, l their sum.  EXT: what joins it is
// looked up and weighed (share); `writes` in the thread that writes them.
template <bool EXT>
__device__ __forceinline__ float2 join_row_end(const JoinParams& p, const JoinRow& row, float m, float l, float k0, bool writes,
                                               const float4* have = nullptr) {
  float2 share = make_float2(1.f, 0.f);
  if constexpr (EXT) {
    if (p.prior.stats_out || p.prior.stats) {
      prior_end(p.prior, row.token * p.heads + row.head, m, l, l != 0.f ? k0 : 0.f, writes, p.lse, share, have);
      return share;
    }
  }
  if (writes && p.lse) join_lse(p, row, m, l, k0);
  return share;
}

// RESIDENT blocks an SM: four for few pieces (64 registers), two for many, whose statistics the
// block holds in registers.
// EXT: the rows go to another call, or join another's (Prior).
template <bool F16, int RESIDENT, bool EXT>
__global__ void __launch_bounds__(kJoinThreads, RESIDENT) attention_join_kernel(const __grid_constant__ JoinParams p, int32_t search) {
  __shared__ float4 sum[kJoinWarps][32];
  grid_dependency_wait();                   // launched while the main kernel's last blocks still run
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int NR = p.NR, slices = (p.Dv + 127) / 128;
  int32_t c = blockIdx.x;
  if (search > 0) {                         // the x-th of the main kernel's `search` blocks that has one
    int32_t skip = c;
    c = -1;
    uint32_t has[kJoinLoads];
#pragma unroll
    for (int i = 0; i < kJoinLoads; ++i) has[i] = 32 * i + lane < search && p.meta[8 * (32 * i + lane)] != 0;
#pragma unroll
    for (int i = 0; i < kJoinLoads; ++i) {
      uint32_t set = __ballot_sync(0xffffffffu, has[i]);
      const int32_t here = __popc(set);
      if (c < 0 && skip < here) {
        for (; skip > 0; --skip) set &= set - 1;
        c = 32 * i + __ffs(set) - 1;
      }
      skip -= here;
    }
    if (c < 0) return;
  }
  const int4 m0 = *reinterpret_cast<const int4*>(p.meta + 8 * c);
  const int4 m1 = *reinterpret_cast<const int4*>(p.meta + 8 * c + 4);
  if (m0.x == 0) return;                    // no item whose first cut lies before block x
  const int32_t first = m0.y, n = m0.z - first + 1, rows0 = m0.w, rows = m0.w + m1.x, tok0 = m1.y, head0 = m1.z, kv_head = m1.w;
  auto slot = [&](int32_t i) { return 2 * static_cast<int64_t>(first + i) + (i == 0 ? 1 : 0); };
  if (n <= (RESIDENT == 2 ? kJoinFewItems : kJoinFew)) {
    const int32_t units = (rows + 3) / 4 * slices;
    for (int32_t unit = blockIdx.y * kJoinWarps + warp; unit < units; unit += gridDim.y * kJoinWarps) {
      const int32_t r0 = unit / slices * 4, ch = (unit % slices) * 128 + lane * 4;
      const int32_t mine = r0 + (lane >> 3), piece = lane & 7;
      float4 st = make_float4(neg_inf(), 0.f, neg_inf(), 0.f);
      JoinRow row = join_row(p, rows0, tok0, head0, min(mine, rows - 1));
      if (mine < rows && piece < n) st = p.stats[slot(piece) * NR + row.part];
      float m = st.x, k0 = st.y != 0.f ? st.z : neg_inf();  // the same in every piece that saw a key
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        k0 = fmaxf(k0, __shfl_xor_sync(0xffffffffu, k0, o));
      }
      const float wt = st.y != 0.f ? ex2(st.x - m) : 0.f;
      float l = st.y * wt;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      const float2 share = join_row_end<EXT>(p, row, m, l, k0, piece == 0 && mine < rows && unit % slices == 0);
      float4 acc[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[t] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int32_t i = 0; i < n; ++i) {
        float4 v[4];
        float w[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          w[t] = __shfl_sync(0xffffffffu, wt, 8 * t + i);
          const int32_t part = __shfl_sync(0xffffffffu, row.part, 8 * t);
          v[t] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (w[t] != 0.f && ch < p.Dv)   // a piece that saw nothing stored no accumulator
            v[t] = *reinterpret_cast<const float4*>(p.parts + (slot(i) * NR + part) * p.Dv + ch);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          acc[t].x = fmaf(v[t].x, w[t], acc[t].x);
          acc[t].y = fmaf(v[t].y, w[t], acc[t].y);
          acc[t].z = fmaf(v[t].z, w[t], acc[t].z);
          acc[t].w = fmaf(v[t].w, w[t], acc[t].w);
        }
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float lt = __shfl_sync(0xffffffffu, l, 8 * t);
        JoinRow rt;
        rt.token = __shfl_sync(0xffffffffu, row.token, 8 * t);
        rt.head = __shfl_sync(0xffffffffu, row.head, 8 * t);
        float2 st = share;
        if constexpr (EXT) {
          st.x = __shfl_sync(0xffffffffu, share.x, 8 * t);
          st.y = __shfl_sync(0xffffffffu, share.y, 8 * t);
        }
        if (r0 + t < rows && ch < p.Dv) join_store<F16, EXT>(p, rt, kv_head, ch, acc[t], lt, st);
      }
    }
    return;
  }
  if constexpr (EXT) {
    // `split` warps to a row's 128 channels, so that few rows fill the SMs as well as many.  (8 kv
    // heads of 256 rows in 20 pieces each: 18.4 us with eight warps to a row, 10.3 with one.)
    __shared__ float weights[kJoinWarps][kMaxBlocks];
    const int S = p.split, part = warp & (S - 1), group = warp / S, groups = kJoinWarps / S;
    constexpr int kBatch = RESIDENT == 2 ? 8 : 4;
    for (int32_t unit0 = blockIdx.y * groups; unit0 < rows * slices; unit0 += gridDim.y * groups) {
      const int32_t unit = min(unit0 + group, rows * slices - 1);
      const bool mine = unit0 + group < rows * slices;
      const int32_t ch = (unit % slices) * 128 + lane * 4;
      const JoinRow row = join_row(p, rows0, tok0, head0, unit / slices);
      float m = neg_inf(), l = 0.f, k0 = neg_inf();
      float2 st[kJoinLoads];
#pragma unroll
      for (int i = 0; i < kJoinLoads; ++i) {
        st[i] = make_float2(neg_inf(), 0.f);
        if (32 * i + lane < n) {
          const float4 x = p.stats[slot(32 * i + lane) * NR + row.part];
          st[i] = make_float2(x.x, x.y);
          if (x.y != 0.f) k0 = x.z;
          m = fmaxf(m, x.x);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        k0 = fmaxf(k0, __shfl_xor_sync(0xffffffffu, k0, o));
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kJoinLoads; ++i) {
        const float w = st[i].y != 0.f ? ex2(st[i].x - m) : 0.f;
        if (32 * i + lane < n) weights[warp][32 * i + lane] = w;
        l = fmaf(st[i].y, w, l);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      __syncwarp();
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int32_t i0 = part; i0 < n; i0 += kBatch * S) {
        float4 v[kBatch];
        float w[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int32_t i = i0 + k * S;
          w[k] = i < n ? weights[warp][i] : 0.f;
          v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (w[k] != 0.f && ch < p.Dv)   // a piece that saw nothing stored no accumulator
            v[k] = *reinterpret_cast<const float4*>(p.parts + (slot(i) * NR + row.part) * p.Dv + ch);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          acc.x = fmaf(v[k].x, w[k], acc.x);
          acc.y = fmaf(v[k].y, w[k], acc.y);
          acc.z = fmaf(v[k].z, w[k], acc.z);
          acc.w = fmaf(v[k].w, w[k], acc.w);
        }
      }
      if (S > 1) {
        sum[warp][lane] = acc;
        __syncthreads();
        if (part == 0) {
          for (int i = 1; i < S; ++i) {
            const float4 v = sum[warp + i][lane];
            acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
          }
        }
      }
      if (part == 0 && mine) {
        const float2 share = join_row_end<EXT>(p, row, m, l, k0, lane == 0 && ch < 128);
        if (ch < p.Dv) join_store<F16, EXT>(p, row, kv_head, ch, acc, l, share);
      }
      if (S > 1) __syncthreads();
    }
  } else {
  for (int32_t unit = blockIdx.y; unit < rows * slices; unit += gridDim.y) {
    const int32_t ch = (unit % slices) * 128 + lane * 4;
    const JoinRow row = join_row(p, rows0, tok0, head0, unit / slices);
    // every lane holds the statistics of pieces lane, lane + 32, ...
    float m = neg_inf(), l = 0.f, k0 = neg_inf(), wt[kJoinLoads];
    float4 st[kJoinLoads];
#pragma unroll
    for (int i = 0; i < kJoinLoads; ++i) {
      st[i] = make_float4(neg_inf(), 0.f, neg_inf(), 0.f);
      if (32 * i + lane < n) st[i] = p.stats[slot(32 * i + lane) * NR + row.part];
    }
#pragma unroll
    for (int i = 0; i < kJoinLoads; ++i) {
      m = fmaxf(m, st[i].x);
      if (st[i].y != 0.f) k0 = st[i].z;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      k0 = fmaxf(k0, __shfl_xor_sync(0xffffffffu, k0, o));
    }
#pragma unroll
    for (int i = 0; i < kJoinLoads; ++i) {
      wt[i] = st[i].y != 0.f ? ex2(st[i].x - m) : 0.f;
      l = fmaf(st[i].y, wt[i], l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kJoinLoads; ++i) {
      if (32 * i >= n) break;
      float4 v[4];
      float w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int e = warp + kJoinWarps * k;
        w[k] = __shfl_sync(0xffffffffu, wt[i], e);
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (w[k] != 0.f && ch < p.Dv)
          v[k] = *reinterpret_cast<const float4*>(p.parts + (slot(32 * i + e) * NR + row.part) * p.Dv + ch);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        acc.x = fmaf(v[k].x, w[k], acc.x);
        acc.y = fmaf(v[k].y, w[k], acc.y);
        acc.z = fmaf(v[k].z, w[k], acc.z);
        acc.w = fmaf(v[k].w, w[k], acc.w);
      }
    }
    sum[warp][lane] = acc;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int i = 1; i < kJoinWarps; ++i) {
        const float4 v = sum[i][lane];
        acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
      }
      const float2 share = join_row_end<EXT>(p, row, m, l, k0, lane == 0 && ch < 128);
      if (ch < p.Dv) join_store<F16, EXT>(p, row, kv_head, ch, acc, l, share);
    }
    __syncthreads();
  }
  }
}

// The join behind a main kernel of `blocks` blocks over at most `items` items; it is put in
// place while that kernel still runs (programmatic stream serialisation).
template <bool EXT = false>
cudaError_t launch_join(const JoinParams& given, bool f16, int blocks, int64_t items, cudaStream_t stream) {
  if (blocks < 2) return cudaSuccess;
  JoinParams p = given;
  const int cuts = static_cast<int>(std::min<int64_t>(blocks - 1, items)), slices = (p.Dv + 127) / 128;
  // (MLA decode, 8 items over 152 blocks: 59 us with the search, 74 with 144 empty blocks a row;
  // 151 cuts: 159 us without it, 168 with)
  const bool search = cuts * 4 < blocks;
  // blocks for each cut that there can be, as many as fill the SMs, four on each, once, and have
  // something to do: of few pieces a warp joins four rows, of many the block one.  (Without the
  // search the grid is that of joins of few pieces: one long item among many short ones, cut into
  // many, has its rows joined by the same few blocks.)
  const int units = search ? p.NR * slices : ((p.NR + 3) / 4 * slices + kJoinWarps - 1) / kJoinWarps;
  int y = std::max(1, std::min(units, (4 * device_sm_count() + cuts - 1) / cuts));
  if (EXT) {
    // warps that fill the SMs twice over, 16 on each; and one round of blocks
    const int64_t rows = static_cast<int64_t>(cuts) * p.NR * slices, warps = 32 * static_cast<int64_t>(device_sm_count());
    p.split = kJoinWarps;
    while (p.split > 1 && search && p.split * rows > warps) p.split /= 2;
    y = search ? std::max(1, std::min(static_cast<int>((p.NR * slices * p.split + kJoinWarps - 1) / kJoinWarps), (4 * device_sm_count() + cuts - 1) / cuts))
               : std::max(1, std::min(units, 4 * device_sm_count() / blocks));
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(search ? cuts : blocks, y);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (search)
    return f16 ? cudaLaunchKernelEx(&cfg, attention_join_kernel<true, 2, EXT>, p, blocks)
               : cudaLaunchKernelEx(&cfg, attention_join_kernel<false, 2, EXT>, p, blocks);
  return f16 ? cudaLaunchKernelEx(&cfg, attention_join_kernel<true, 4, EXT>, p, 0)
             : cudaLaunchKernelEx(&cfg, attention_join_kernel<false, 4, EXT>, p, 0);
}

// Parts leave the tile kernel as 32-byte stores, and a workspace may start on any 16 bytes: a join
// is placed on the next 32, in room that is sized for the step there.
constexpr size_t kJoinAlign = 32, kJoinSlack = kJoinAlign - 16;
inline size_t join_meta_bytes(int G) { return (static_cast<size_t>(G) * 32 + 255) / 256 * 256; }
inline size_t join_stats_bytes(int G, int NR) { return static_cast<size_t>(G) * 2 * NR * sizeof(float4); }
inline size_t join_bytes(int G, int NR, int Dv) {
  return kJoinSlack + join_meta_bytes(G) + join_stats_bytes(G, NR) + static_cast<size_t>(G) * 2 * NR * Dv * sizeof(float);
}
// sets the pointers of a join whose workspace was sized for G blocks
inline void join_place(JoinParams* j, uint8_t* at, int G) {
  at += (0 - reinterpret_cast<uintptr_t>(at)) % kJoinAlign;
  j->meta = reinterpret_cast<int32_t*>(at);
  j->stats = reinterpret_cast<float4*>(at + join_meta_bytes(G));
  j->parts = reinterpret_cast<float*>(at + join_meta_bytes(G) + join_stats_bytes(G, j->NR));
}

}  // namespace
}  // namespace ra
