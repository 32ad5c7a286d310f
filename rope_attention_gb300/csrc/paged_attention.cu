// Attention of new tokens over the paged caches of kv_rms_norm_rope_cache.
//
//   out[i, h] = sum_j softmax_j(scale q[i, h] . k_j) v_j   over the cached positions j <
//   seq_len (causal: j <= seq_len - Lq + i), k_j / v_j read through the block table.
//
// Quantised caches.  An element is x = (code - o) / s per channel, so
//   q . k_j = sum_c (q_c / s_c) code_jc - sum_c q_c o_c / s_c:
// the second sum does not depend on j and leaves the softmax (it enters the lse), and
//   out_c = (sum_j p_j code_jc / sum_j p_j - o_c) / s_c.
// The codes themselves (int8, E4M3, E5M2: all exact in fp16) are the tensor core's
// operands; q / s is rounded to fp16 behind a power of two per row that keeps the row's
// elements below 2^15, counted from its largest |q| and the head's largest 1 / s.  Elements
// down to 2^-29 of that bound keep 11 bits.
//
// GB300 mapping.  A work item is one row tile of a sequence and kv head: NR rows, a row
// being (token, head of the group), against all the sequence's keys in 64-key tiles.
// The tiles of all items, laid end to end, are cut into equal runs, one per block, so
// blocks finish together whatever the lengths; an item cut in two or more has its pieces'
// (max, sum, accumulator) joined by a second kernel, in a fixed order.  Where a cut would save
// less than its join costs, counted at the largest length (plan()), blocks take runs of whole
// items instead; those are equal in items, not in tiles, so there they finish together only if
// the lengths are alike.
//  * The rows are few (one token: 1..128 heads), so the second product is transposed:
//    O^T[channel, row] += V^T P^T puts the channels on the MMA's 128 rows and the NR rows
//    on its N, which costs tensor time and TMEM for NR columns instead of 128.  The
//    first, S = Q K^T, keeps rows on TMEM lanes so that a softmax row is one thread's;
//    its A operand is addressed as 128 rows although only NR are stored: the other lanes
//    of S come from whatever follows in shared memory and are never read.
//  * V1's value row is the first part of its key row: one tile in shared memory serves
//    both products (K-major for S, MN-major for O^T).
//  * Warp 13 reads the block table and issues TMA boxes of 16, 32 or 64 rows (what divides
//    a page), 64 channels wide: straight into the swizzled operand tile for 16-bit caches,
//    or as codes into a staging ring that warps 8-11 convert from.  Rows behind a
//    sequence's end and rows of absent pages are zeroed in shared memory (0 times a
//    stray NaN is NaN) and masked in S.  Warps 0-7 are the softmax, the rescaling and the
//    epilogue, two threads to a row of S with 32 of its 64 columns each (with one thread
//    a 64-key tile took 1740 cycles, more than its products); warp 12 issues the MMAs,
//    taking whichever of the next S = Q K^T and the next O^T += V^T P^T is ready first.
// What bounds it: neither HBM nor the tensor core but the chain load - (conversion) - S -
// softmax - O of one tile, of which shared memory has room for one or two beside Q: 2150 cycles
// a 64-key tile for V2 int8 (TMA issue 700, conversion 1400, softmax 1600, overlapped), 4900 for
// V1 (74 KB a tile; 36 + 16 products).  Measured: 8 sequences of 4096 positions, 64 heads over 8,
// int8: 43 us (55 MB, 1.3 TB/s); 32 sequences of the 576-wide latent, 128 heads, bf16: 77 us (296
// TFLOP/s); one of 333 positions, 8 heads over 2: 12 us, of which 5 are the block's start.
// Every wait is bounded in time (status word).
#include <algorithm>
#include <atomic>
#include <cmath>

#include "attention.h"
#include "attn_join.cuh"
#include "attn_ptx.cuh"
#include "internal.h"
#include "kv_cache.h"
#include "paged_codes.cuh"
#include "paged_maps.cuh"

namespace ra {
namespace {

constexpr int kKeys = 64;                 // keys per tile: one 128-byte swizzled row of P
constexpr int kSlab = kKeys * 128;        // 64 keys x 64 channels of 16 bits
constexpr int kCodeSlab = kKeys * 64;      // the same of codes
constexpr int kThreads = 512;              // four warpgroups
// Registers per thread: launched with 128 each, then moved to the softmax:
// 2 x 160 + 120 + 72 = 4 x 128
constexpr int kRegsSoftmax = 160, kRegsConvert = 120, kRegsRest = 72;
constexpr int kSoftmax = 256, kSoftmaxWarps = kSoftmax / 32, kConvertWarps = 4;
constexpr int kMmaWarp = 12, kLoadWarp = 13;
constexpr int kValidRing = 16;            // > tiles between the loads and the softmax
constexpr int kMaxStages = 6;
// Items are cut where that saves a block more tiles than the join costs: kJoinTiles, and up to
// kJoinAll more the more blocks have a cut.  (V2, one sequence, 2 kv heads: 200 positions 12.6 us
// whole and 14.5 cut, 333 15.6 and 12.6, 450 18.6 and 12.6; 64 items: 600 positions 20.7 whole and
// 25.1 cut, 1000 26.3 and 29.0.  V1, 4 items: 333 positions 27.0 and 22.9.)
// Rounds are counted over kMaxBlocks, the blocks that the workspace has room for.
constexpr int kJoinTiles = 4, kJoinAll = 10;
constexpr float kLazy = 8.f;              // log2 of how far a tile may exceed the running maximum
constexpr uint64_t kDrainNs = 200000000ull;
constexpr int kSmemMax = 232448;
constexpr int kSCols = 2 * kKeys;         // TMEM: two S buffers, then O^T

struct Params {
  CUtensorMap tk, tv;           // the caches' rows: 64 channels x 1 x box_rows boxes
  CUtensorMap tq;               // (channels, heads, tokens): boxes of 64 x hb x tb, a row tile
  uint16_t* out;
  float* lse;
  const float *k_scale, *k_offset, *v_scale, *v_offset;
  const int32_t *cu_q, *seq_lens, *table;
  int32_t* err_count;
  int32_t* status;
  JoinParams join;
  int64_t table_stride, cap;    // cap: positions that a sequence can have
  int64_t block_num, cache_seq;
  int32_t B, total_q, N, heads, g, NR, block_size, bs_shift;
  int32_t Dk, Dv, Dko;          // key width, value width, width of a k_cache row
  int32_t v1, mode, f16, kq, vq, k_scalar, v_scalar, causal;
  int32_t box_rows, box_shift;
  int32_t hb, tb, hblocks;      // a row tile: tb tokens x hb heads; tiles that a token's heads take
  int32_t vslabs, kslabs, qslabs, kslab0;
  int32_t ns, nsg;              // operand stages, staging stages (0: 16-bit caches)
  int32_t stage_bytes, staging_bytes;
  int32_t off_p, off_ring, off_staging, off_misc;
  float sl2, scale;
  uint64_t wait_ns;
  int32_t whole;                // blocks take whole items
  int32_t stall_loads;
};

struct Misc {                   // behind the tiles in shared memory
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
  uint64_t code_full[kMaxStages], code_empty[kMaxStages];
  uint64_t s_full[2], p_ready, pv_done, q_full, q_ready, q_empty, drain;
  uint64_t valid[kValidRing];
  int64_t scan[kThreads / 32];
  int64_t start_off;
  int32_t start_b;
  uint32_t tmem;
  int32_t abort;
  // followed by per-row arrays of NR: int32 out_row, float row_scale, row_const, xch[2], inv_sum
};
__host__ __device__ constexpr int row_arrays_bytes(int nr) { return nr * (4 + 5 * 4); }

__device__ __forceinline__ int32_t seq_len_of(const Params& p, int32_t b) {
  return static_cast<int32_t>(min(static_cast<int64_t>(max(__ldg(p.seq_lens + b), 0)), p.cap));
}
__device__ __forceinline__ void q_span(const Params& p, int32_t b, int32_t& start, int32_t& len) {
  if (p.cu_q == nullptr) {
    len = p.total_q / p.B;
    start = b * len;
    return;
  }
  const int32_t lo = min(max(__ldg(p.cu_q + b), 0), p.total_q), hi = min(max(__ldg(p.cu_q + b + 1), lo), p.total_q);
  start = lo;
  len = hi - lo;
}
__device__ __forceinline__ int32_t tiles_of(int32_t len) { return max(1, (len + kKeys - 1) / kKeys); }
// row tiles of lq tokens and one kv head (lq * heads < 2^31)
__device__ __forceinline__ int32_t row_tiles_of(const Params& p, int32_t lq) {
  return p.hblocks > 1 ? lq * p.hblocks : static_cast<int32_t>(static_cast<uint32_t>(lq + p.tb - 1) / static_cast<uint32_t>(p.tb));
}
// what a sequence counts for in the line: its items' tiles, or its items
__device__ __forceinline__ int64_t seq_work(const Params& p, int32_t lq, int32_t len) {
  return static_cast<int64_t>(row_tiles_of(p, lq)) * p.N * (p.whole ? 1 : tiles_of(len));
}

// The spans of 32 sequences, one to a lane: a walk over them waits for memory once.
struct Spans {
  int32_t base, start, lq, len;
  __device__ __forceinline__ void load(const Params& p, int32_t from) {
    base = from;
    const int32_t b = from + static_cast<int32_t>(threadIdx.x & 31);
    start = lq = len = 0;
    if (b < p.B) {
      q_span(p, b, start, lq);
      len = seq_len_of(p, b);
    }
  }
};

// One block's share of an item: key tiles [ta, tb) of row tile rt of (b, n).
struct Piece {
  int32_t b, n, tok, head, rows, q_start, Lq, len;  // the tile's first token (of its sequence) and head
  int32_t t0, take, T;          // nominal tiles: [t0, t0 + take) of T
  int32_t ta, tb;               // those that any of its rows sees
  __device__ bool whole() const { return take == T; }
};
// Walks the pieces of a run of tiles (p.whole: of items), a whole warp at once.
struct Walker {
  int32_t b;
  int64_t off, rem;             // position inside sequence b, tiles left
  Spans spans;
  __device__ bool next(const Params& p, Piece& w) {
    while (rem > 0 && b < p.B) {
      if (b >= spans.base + 32) spans.load(p, b);
      const int32_t qs = __shfl_sync(0xffffffffu, spans.start, b - spans.base);
      const int32_t lq = __shfl_sync(0xffffffffu, spans.lq, b - spans.base);
      const int32_t len = __shfl_sync(0xffffffffu, spans.len, b - spans.base);
      const int32_t T = tiles_of(len), each = p.whole ? 1 : T;
      const int32_t rts = row_tiles_of(p, lq);
      const int64_t work = static_cast<int64_t>(rts) * p.N * each;
      if (off >= work) {
        off -= work;
        ++b;
        continue;
      }
      // (a 64-bit division is a hundred instructions: only for what needs it)
      const int64_t item = work >> 32 ? off / each : static_cast<int64_t>(static_cast<uint32_t>(off) / static_cast<uint32_t>(each));
      w.b = b;
      w.t0 = static_cast<int32_t>(off - item * each);
      w.T = T;
      w.take = p.whole ? T : static_cast<int32_t>(min(static_cast<int64_t>(T - w.t0), rem));
      w.n = static_cast<int32_t>(static_cast<uint32_t>(item) / static_cast<uint32_t>(rts));  // item < rts * N <= 2^31
      const int32_t rt = static_cast<int32_t>(item - static_cast<int64_t>(w.n) * rts);
      if (p.hblocks > 1) {
        w.tok = rt / p.hblocks;
        const int32_t h = (rt - w.tok * p.hblocks) * p.hb;
        w.head = w.n * p.g + h;
        w.rows = min(p.hb, p.g - h);
      } else {
        w.tok = rt * p.tb;
        w.head = w.n * p.g;
        w.rows = min(p.tb, lq - w.tok) * p.g;
      }
      w.q_start = qs;
      w.Lq = lq;
      w.len = len;
      const int32_t last = p.hblocks > 1 ? w.tok : min(w.tok + p.tb, lq) - 1;
      const int32_t seen = p.causal ? min(len, max(0, len - lq + last + 1)) : len;
      const int32_t vt = (seen + kKeys - 1) / kKeys;
      w.ta = min(w.t0, vt);
      w.tb = min(w.t0 + w.take, vt);
      off += p.whole ? 1 : w.take;
      rem -= p.whole ? 1 : w.take;
      return true;
    }
    return false;
  }
};

// over the softmax warps
__device__ __forceinline__ uint32_t bar_or(uint32_t pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(pred)
      : "memory");
  return r;
}
__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <bool F16>
__device__ __forceinline__ float half_to_float(uint32_t u) {
  return F16 ? __half2float(__ushort_as_half(static_cast<uint16_t>(u))) : __uint_as_float(u << 16);
}
// the scales of key channels c..c+7 of head n: V1's key is the ckv row, then the k row
__device__ __forceinline__ void key_scales(const Params& p, int32_t n, int32_t c, float (&s)[8]) {
  const bool latent = p.v1 && c < p.Dv;
  const float* scale = latent ? p.v_scale : p.k_scale;
  const bool one = latent ? p.v_scalar : p.k_scalar;
  const int32_t at = latent ? c : p.v1 ? c - p.Dv : n * p.Dk + c;
  if (scale == nullptr || one || c >= p.Dk) {
    const float x = scale != nullptr && one ? __ldg(scale) : 1.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = x;
    return;
  }
  const float4 a = __ldg(reinterpret_cast<const float4*>(scale + at)), b = __ldg(reinterpret_cast<const float4*>(scale + at) + 1);
  s[0] = a.x, s[1] = a.y, s[2] = a.z, s[3] = a.w, s[4] = b.x, s[5] = b.y, s[6] = b.z, s[7] = b.w;
}
__device__ __forceinline__ float key_offset(const Params& p, int32_t n, int32_t c) {
  if (p.v1 && c < p.Dv) return channel_quant(p.v_scale, p.v_offset, c, p.v_scalar).y;
  return channel_quant(p.k_scale, p.k_offset, p.v1 ? c - p.Dv : n * p.Dk + c, p.k_scalar).y;
}
__device__ __forceinline__ float2 value_quant(const Params& p, int32_t n, int32_t c) {
  return channel_quant(p.v_scale, p.v_offset, p.v1 ? c : n * p.Dv + c, p.v_scalar);
}

// Where the key is codes: the piece's rows of q, in their swizzled operand, over the key's
// scales and behind a power of two that keeps the row's elements below 2^15: 2^29 above
// fp16's subnormals, so that a bound on the largest element (the largest |q| times the
// largest 1 / s) serves as well as the element itself.  row_scale gets the softmax scale
// that undoes the power, row_const the lse's share of the offsets.  A warp takes a row, a
// lane the 8-channel chunks lane, lane + 32, lane + 64.  Rolled loops: at the start of a
// block each line of code comes from L2, at several hundred cycles.
template <bool F16>
__device__ __forceinline__ bool scale_q(const Params& p, int32_t n, int32_t rows, uint8_t* smem, float* row_scale,
                                        float* row_const, int warp, int lane, uint32_t q_full, uint32_t parity,
                                        volatile int* abort_flag) {
  const int nck = p.Dk / 8;
  float inv_s[3][8], top = 0.f;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int c = (lane + 32 * i) * 8;
    key_scales(p, n, c, inv_s[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      inv_s[i][e] = c < p.Dk ? rcp(inv_s[i][e]) : 0.f;
      top = fmaxf(top, fabsf(inv_s[i][e]));
    }
  }
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));  // not negative: bits order like values
  if (!bounded_wait_warp(q_full, parity, p.wait_ns, abort_flag)) return false;
#pragma unroll 1
  for (int r = warp; r < rows; r += kSoftmaxWarps) {
    uint8_t* row = smem + r * 128;
    uint4 x[3];
    uint32_t big = 0;  // |q| as bits orders like the value in either type
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int c = lane + 32 * i;
      x[i] = c < nck ? *reinterpret_cast<const uint4*>(row + (c >> 3) * p.NR * 128 + (((c & 7) ^ (r & 7)) << 4))
                     : make_uint4(0, 0, 0, 0);
      big = __vmaxu2(__vmaxu2(big, x[i].x & 0x7FFF7FFFu), x[i].y & 0x7FFF7FFFu);
      big = __vmaxu2(__vmaxu2(big, x[i].z & 0x7FFF7FFFu), x[i].w & 0x7FFF7FFFu);
    }
    big = __reduce_max_sync(0xffffffffu, max(big & 0xFFFFu, big >> 16));
    // |q| < 2^(e + 15), 1 / s < 2^(f + 15) with e, f the exponents below: |q| / s * up < 2^15
    const int k = max(-100, min(100, -(scale_exponent(half_to_float<F16>(big)) + scale_exponent(top) + 15)));
    const float up = exp2_int(k);
    if (lane == 0) {
      row_scale[r] = p.sl2 * exp2_int(-k);
      row_const[r] = 0.f;
    }
    if (p.lse) {
      float shift = 0.f;
#pragma unroll 1
      for (int c = lane; c < nck; c += 32) {
        const uint4 z = *reinterpret_cast<const uint4*>(row + (c >> 3) * p.NR * 128 + (((c & 7) ^ (r & 7)) << 4));
        const uint32_t u[4] = {z.x, z.y, z.z, z.w};
        float sc[8];
        key_scales(p, n, c * 8, sc);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          shift += half_to_float<F16>((u[e >> 1] >> (16 * (e & 1))) & 0xFFFFu) / sc[e] * key_offset(p, n, c * 8 + e);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) shift += __shfl_xor_sync(0xffffffffu, shift, o);
      if (lane == 0) row_const[r] = -shift * p.scale;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int c = lane + 32 * i;
      // V1's key can be codes in one part and 16-bit values in the other
      const bool f16 = F16 || ((p.v1 && c * 8 < p.Dv) ? p.vq != 0 : p.kq != 0);
      const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t y[4];
      float a[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        a[e] = half_to_float<F16>((u[e >> 1] >> (16 * (e & 1))) & 0xFFFFu) * (inv_s[i][e] * up);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = pack_f16x2(a[2 * e], a[2 * e + 1]);
      if (!f16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = pack_bf16x2(a[2 * e], a[2 * e + 1]);
      }
      if (c < nck)
        *reinterpret_cast<uint4*>(row + (c >> 3) * p.NR * 128 + (((c & 7) ^ (r & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
  return true;
}

// F16: q, out and 16-bit caches are fp16, not bf16; P16: P is fp16 (V's operand is)
// PLO: fp16 results over codes.  q / s is rounded to 11 bits, like the result; so that P's
// rounding does not add a third error of that size, P goes in as two fp16 numbers (hi + lo).
template <bool F16, bool P16, bool PLO>
__global__ void __launch_bounds__(kThreads, 1) paged_attention_kernel(const __grid_constant__ Params p) {
  constexpr float kLift = P16 ? kHalfLift : 0.f;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc& ms = *reinterpret_cast<Misc*>(smem + p.off_misc);
  const int NR = p.NR;
  int32_t* out_row = reinterpret_cast<int32_t*>(&ms + 1);  // row of q and out, -1: none
  float* row_scale = reinterpret_cast<float*>(out_row + NR);
  float* row_const = row_scale + NR;
  float* xch = row_const + NR;              // [2][NR] what the two threads of a row exchange
  float* inv_sum = xch + 2 * NR;
  const uint32_t s0 = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&ms.tmem), 512);
    tmem_relinquish();
  } else if (threadIdx.x == kSoftmax) {
    for (int s = 0; s < p.ns; ++s) {
      // one arrival with the bytes of a 16-bit cache, one from each warp that converts codes
      mbar_init(smem_u32(&ms.kv_full[s]), (p.vq == 0 || p.kq == 0 ? 1 : 0) + (p.nsg != 0 ? kConvertWarps : 0));
      mbar_init(smem_u32(&ms.kv_empty[s]), 1);
    }
    for (int s = 0; s < p.nsg; ++s) {
      mbar_init(smem_u32(&ms.code_full[s]), 1);
      mbar_init(smem_u32(&ms.code_empty[s]), kConvertWarps);
    }
    mbar_init(smem_u32(&ms.s_full[0]), 1);
    mbar_init(smem_u32(&ms.s_full[1]), 1);
    mbar_init(smem_u32(&ms.p_ready), kSoftmaxWarps);
    mbar_init(smem_u32(&ms.pv_done), 1);
    mbar_init(smem_u32(&ms.q_full), 1);
    mbar_init(smem_u32(&ms.q_ready), kSoftmaxWarps);
    mbar_init(smem_u32(&ms.q_empty), 1);
    mbar_init(smem_u32(&ms.drain), 1);
    ms.abort = 0;
    fence_mbar_init();
    p.join.meta[8 * blockIdx.x] = 0;         // nothing to join, unless the first piece says so below
  } else if (threadIdx.x == 32 * kLoadWarp) {
    prefetch_tensormap(&p.tq);
    prefetch_tensormap(&p.tk);
    prefetch_tensormap(&p.tv);
  }
  grid_launch_dependents();

  // ---- this block's run of tiles.  Up to 32 sequences every warp finds it for itself, beside
  // the set-up above (a block-wide scan behind it cost a short decode step 2.5k cycles more).
  Walker walk;
  walk.b = p.B;
  walk.off = 0;
  walk.spans.load(p, 0);
  const bool few = p.B <= 32;
  int64_t mine = 0;
  int32_t b_lo = lane, b_hi = lane;
  if (few) {
    mine = seq_work(p, walk.spans.lq, walk.spans.len);
  } else {
    const int32_t chunk = (p.B + kThreads - 1) / kThreads;
    b_lo = min(p.B, static_cast<int32_t>(threadIdx.x) * chunk);
    b_hi = min(p.B, b_lo + chunk);
    for (int32_t b = b_lo; b < b_hi; ++b) {
      int32_t qs, lq;
      q_span(p, b, qs, lq);
      mine += seq_work(p, lq, seq_len_of(p, b));
    }
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  int64_t before = incl - mine, W = 0;
  if (few) {
    W = __shfl_sync(0xffffffffu, incl, 31);
  } else {
    if (lane == 31) ms.scan[warp] = incl;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int64_t t = ms.scan[w];
      if (w < warp) before += t;
      W += t;
    }
  }
  const int64_t G = gridDim.x;
  const int64_t even = W >> 31 ? (W + G - 1) / G : static_cast<int64_t>((static_cast<uint32_t>(W) + static_cast<uint32_t>(G) - 1) / static_cast<uint32_t>(G));
  const int64_t per = max(even, static_cast<int64_t>(1)), start = per * blockIdx.x;
  walk.rem = max(static_cast<int64_t>(0), min(per, W - start));  // none: the block has nothing to do
  const bool here = before <= start && start < before + mine;
  if (few) {
    const uint32_t at = __ballot_sync(0xffffffffu, here);
    if (at) {
      walk.b = __ffs(at) - 1;
      walk.off = start - __shfl_sync(0xffffffffu, before, walk.b);
    }
  } else if (here) {
    int32_t b = b_lo;
    int64_t off = start - before;
    for (; b < b_hi; ++b) {
      int32_t qs, lq;
      q_span(p, b, qs, lq);
      const int64_t w = seq_work(p, lq, seq_len_of(p, b));
      if (off < w) break;
      off -= w;
    }
    ms.start_b = b;
    ms.start_off = off;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!few && walk.rem > 0) {
    walk.b = ms.start_b;
    walk.off = ms.start_off;
    walk.spans.load(p, walk.b);
  }
  const uint32_t tmem = ms.tmem;
  const bool k_quant = p.kq != 0 || (p.v1 && p.vq != 0);
  volatile int* abort_flag = &ms.abort;
  Piece w{};

  if (warp >= kMmaWarp) {
    set_max_regs_dec<kRegsRest>();
  if (warp == kLoadWarp) {
    // ------------------------------------------------------------ loads
    const int groups = kKeys >> p.box_shift;
    const bool direct = p.vq == 0 || p.kq == 0, staged = p.vq != 0 || p.kq != 0;
    const uint32_t direct_bytes = ((p.vq ? 0 : p.vslabs) + (p.kq ? 0 : p.kslabs)) * p.box_rows * 128;
    const uint32_t staged_bytes = ((p.vq ? p.vslabs : 0) + (p.kq ? p.kslabs : 0)) * p.box_rows * 64;
    uint32_t armed[3] = {0, 0, 0}, armed_parity[3] = {0, 0, 0};   // copies in flight: operands, codes, Q
    int32_t u = 0, pieces = 0;
    Ring kv, code;
    bool ok = !p.stall_loads;
    while (ok && walk.next(p, w)) {
      if (w.ta >= w.tb) continue;
      // Cache rows.  Lane i holds where group `base + i` of the piece starts: 32 groups of
      // box_rows keys per trip to the block table.
      const int32_t g_end = w.tb * groups, head = p.mode == kModePa ? w.n : 0;
      int64_t row = -1;
      int32_t base = w.ta * groups - 32;
      for (int32_t t = w.ta; t < w.tb; ++t, ++u) {
        if (t * groups >= base + 32) {
          base += 32;
          const int32_t pos = (base + lane) << p.box_shift;
          row = -1;
          if (base + lane < g_end && pos < w.len) {
            if (p.mode == kModeNorm) {
              row = (static_cast<int64_t>(w.b) * p.N + w.n) * p.cache_seq + pos;
            } else {
              const int32_t pg = p.bs_shift >= 0 ? pos >> p.bs_shift : pos / p.block_size;
              const int32_t in = pos - pg * p.block_size;
              const int64_t page = __ldg(p.table + w.b * p.table_stride + pg);
              if (page >= 0 && page < p.block_num)
                row = p.mode == kModePa ? page * p.block_size + in : (page * p.N + w.n) * p.block_size + in;
              else if (p.err_count)
                atomicAdd(p.err_count, 1);
            }
          }
        }
        if (t == w.ta) {  // the row tile of Q, once the products of the last one are through with it
          ok = bounded_wait_warp(smem_u32(&ms.q_empty), (pieces & 1) ^ 1u, p.wait_ns, abort_flag);
          if (!ok) break;
          if (elect_one()) {
            const uint32_t bar = smem_u32(&ms.q_full);
            mbar_arrive_expect_tx(bar, p.qslabs * p.hb * p.tb * 128);
            for (int c = 0; c < p.qslabs; ++c) tma_load_3d(s0 + c * NR * 128, &p.tq, bar, 64 * c, w.head, w.q_start + w.tok);
          }
          __syncwarp();
          armed[2] = 1;
          armed_parity[2] = pieces & 1;
          ++pieces;
        }
        const int st = kv.stage, sg = code.stage;
        const uint32_t par_d = kv.parity, par_s = code.parity;
        if (direct) ok = bounded_wait_warp(smem_u32(&ms.kv_empty[st]), par_d ^ 1u, p.wait_ns, abort_flag);
        if (ok && staged) ok = bounded_wait_warp(smem_u32(&ms.code_empty[sg]), par_s ^ 1u, p.wait_ns, abort_flag);
        if (!ok) break;
        // the starts of this tile's groups (at most four), and which of its keys exist
        int32_t at[4];
        uint64_t bits = 0;
        uint32_t live = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          at[i] = -1;
          if (i < groups) {
            at[i] = __shfl_sync(0xffffffffu, static_cast<int32_t>(row), t * groups - base + i);
            const int32_t have = min(p.box_rows, w.len - (t * kKeys + (i << p.box_shift)));
            if (at[i] >= 0) {
              bits |= (~0ull >> (64 - have)) << (i << p.box_shift);
              ++live;
            }
          }
        }
        if (elect_one()) {
          const uint32_t bar_d = smem_u32(&ms.kv_full[st]), bar_s = smem_u32(&ms.code_full[sg]);
          ms.valid[u % kValidRing] = bits;
          if (direct) mbar_arrive_expect_tx(bar_d, live * direct_bytes);
          if (staged) mbar_arrive_expect_tx(bar_s, live * staged_bytes);
          const uint32_t operand = s0 + p.off_ring + st * p.stage_bytes, codes = s0 + p.off_staging + sg * p.staging_bytes;
          // (lean loops: the copies of a tile go out one after the other from here)
          const uint32_t to_v = p.vq ? codes : operand, to_k = p.kq ? codes + (p.vq ? p.vslabs : 0) * kCodeSlab : operand + p.vslabs * kSlab;
          const uint32_t bar_v = p.vq ? bar_s : bar_d, bar_k = p.kq ? bar_s : bar_d;
          const uint32_t slab_v = p.vq ? kCodeSlab : kSlab, slab_k = p.kq ? kCodeSlab : kSlab;
          const int32_t end_v = 64 * p.vslabs, end_k = 64 * p.kslabs;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (at[i] < 0) continue;
            uint32_t to = to_v + (i << p.box_shift) * (slab_v / kKeys);
#pragma unroll 2
            for (int32_t x = 0; x < end_v; x += 64, to += slab_v) tma_load_3d(to, &p.tv, bar_v, x, head, at[i]);
            to = to_k + (i << p.box_shift) * (slab_k / kKeys);
#pragma unroll 2
            for (int32_t x = 0; x < end_k; x += 64, to += slab_k) tma_load_3d(to, &p.tk, bar_k, x, head, at[i]);
          }
        }
        __syncwarp();
        if (direct) {
          armed[0] |= 1u << st;
          armed_parity[0] = (armed_parity[0] & ~(1u << st)) | (par_d << st);
        }
        if (staged) {
          armed[1] |= 1u << sg;
          armed_parity[1] = (armed_parity[1] & ~(1u << sg)) | (par_s << sg);
        }
        kv.next(p.ns);
        code.next(p.nsg);
      }
    }
    // Let every copy in flight land before the block leaves: whoever waits for the last ones may give
    // up only after this warp has come through, so it asks no flag.
    if (!p.stall_loads) {
      for (int i = 0; i < kMaxStages; ++i) {
        // (a stage that converters share may stay open for them: then nothing is in flight after the limit)
        if (armed[0] & (1u << i)) bounded_drain(smem_u32(&ms.kv_full[i]), (armed_parity[0] >> i) & 1u, kDrainNs);
        if (armed[1] & (1u << i)) bounded_drain(smem_u32(&ms.code_full[i]), (armed_parity[1] >> i) & 1u, kDrainNs);
      }
      if (armed[2]) bounded_drain(smem_u32(&ms.q_full), armed_parity[2], kDrainNs);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    const bool bf = !p.f16;
    const uint32_t id_s_v = idesc_f16(bf && p.vq == 0, false, false, 128, kKeys);   // V1: the latent part of the key
    const uint32_t id_s_k = idesc_f16(bf && p.kq == 0, false, false, 128, kKeys);
    const uint32_t id_o = idesc_f16(bf && p.vq == 0, true, false, 128, static_cast<uint32_t>(NR));
    const uint64_t q_desc = sdesc_kmajor_sw128(s0);
    const uint64_t k_desc = sdesc_kmajor_sw128(s0 + p.off_ring + p.kslab0 * kSlab);
    const uint64_t v_desc = sdesc_mnmajor_sw128(s0 + p.off_ring, kSlab);
    const uint64_t p_desc = sdesc_kmajor_sw128(s0 + p.off_p);
    const int v_chunks = (p.Dv + 127) / 128;
    const int q_step = NR * 128 >> 4;
    int32_t jt = 0, pieces = 0;
    Ring ring_s, ring_o;
    bool ok = true;
    while (ok && walk.next(p, w)) {
      const int32_t n = w.tb - w.ta;
      if (n <= 0) continue;
      if (!bounded_wait_warp(smem_u32(k_quant ? &ms.q_ready : &ms.q_full), pieces & 1, p.wait_ns, abort_flag)) break;
      // the accumulator's last readers (the epilogue of the piece before) are waited for at
      // this piece's first P, which they write
      ++pieces;
      int32_t qk = 0, pv = 0;
      uint64_t t_start = 0;
      uint32_t spins = 0;
      while (pv < n) {  // whichever product is ready next; the whole warp goes the same way
        const int32_t u = jt + qk, v = jt + pv;
        const int st_s = ring_s.stage, st_o = ring_o.stage;
        const bool go_s = qk < n && qk - pv < 2 && mbar_test_wait(smem_u32(&ms.kv_full[st_s]), ring_s.parity);
        if (__all_sync(0xffffffffu, go_s)) {
          tc_fence_after();
          if (elect_one()) {
            const uint64_t kb = k_desc + static_cast<uint64_t>(st_s * (p.stage_bytes >> 4));
            const uint32_t d = tmem + (u & 1) * kKeys;
            for (int sl = 0; sl < p.qslabs; ++sl)
              mma4_f16_ss<2, 2>(d, q_desc + sl * q_step, kb + sl * (kSlab >> 4), p.v1 && sl < p.vslabs ? id_s_v : id_s_k,
                                sl > 0, min(4, (p.Dk - sl * 64) / 16));
            tc_commit(smem_u32(&ms.s_full[u & 1]));
            if (qk + 1 == n) tc_commit(smem_u32(&ms.q_empty));
          }
          __syncwarp();
          ring_s.next(p.ns);
          ++qk;
          spins = 0;
          continue;
        }
        const bool go_o = pv < qk && mbar_test_wait(smem_u32(&ms.p_ready), v & 1);
        if (__all_sync(0xffffffffu, go_o)) {
          tc_fence_after();
          if (elect_one()) {
            const uint64_t va = v_desc + static_cast<uint64_t>(st_o * (p.stage_bytes >> 4));
            for (int c = 0; c < v_chunks; ++c)
              mma4_f16_ss<128, 2>(tmem + kSCols + c * NR, va + c * (2 * kSlab >> 4), p_desc, id_o, pv > 0, 4);
            if (PLO)
              for (int c = 0; c < v_chunks; ++c)
                mma4_f16_ss<128, 2>(tmem + kSCols + c * NR, va + c * (2 * kSlab >> 4), p_desc + (NR * 128 >> 4), id_o, true, 4);
            tc_commit(smem_u32(&ms.kv_empty[st_o]));
            tc_commit(smem_u32(&ms.pv_done));
          }
          __syncwarp();
          ring_o.next(p.ns);
          ++pv;
          spins = 0;
          continue;
        }
        if ((++spins & 31u) == 0) {
          const uint64_t now = globaltimer_ns();
          int give_up = 0;
          if (spins == 32u) t_start = now;
          else give_up = *abort_flag || now - t_start > p.wait_ns;
          if (__any_sync(0xffffffffu, give_up)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
        }
      }
      jt += n;
    }
    if (elect_one()) tc_commit(smem_u32(&ms.drain));  // every product must finish before TMEM is released
    __syncwarp();
    bounded_drain(smem_u32(&ms.drain), 0, kDrainNs);
    __syncwarp();
  }
  } else if (warp >= kSoftmaxWarps) {
    set_max_regs_dec<kRegsConvert>();
    // ------------------------------------------------------------ codes to fp16 operands
    const int tid = threadIdx.x - kSoftmax;
    const int sl0 = p.vq ? 0 : p.vslabs, sl1 = p.vslabs + (p.kq ? p.kslabs : 0);  // the slabs that hold codes
    bool ok = p.nsg != 0 && !p.stall_loads;
    int32_t u = 0;
    Ring kv, code;
    while (ok && walk.next(p, w)) {
      for (int32_t t = w.ta; ok && t < w.tb; ++t, ++u) {
        const int st = kv.stage, sg = code.stage;
        ok = bounded_wait_warp(smem_u32(&ms.code_full[sg]), code.parity, p.wait_ns, abort_flag) &&
             bounded_wait_warp(smem_u32(&ms.kv_empty[st]), kv.parity ^ 1u, p.wait_ns, abort_flag);
        if (!ok) break;
        uint8_t* stage = smem + p.off_ring + st * p.stage_bytes;
        const uint8_t* from = smem + p.off_staging + sg * p.staging_bytes;
        const uint64_t valid = ms.valid[u % kValidRing];
        // 64 keys x 4 chunks of 16 codes per slab, two rounds of 128 threads; two slabs' loads
        // are in flight together
        const int key0 = tid >> 2, c = tid & 3;
        const bool have[2] = {((valid >> key0) & 1) != 0, ((valid >> (key0 + 32)) & 1) != 0};
        auto convert = [&](auto kind, int lo, int hi) {
          constexpr int K = decltype(kind)::value;
#pragma unroll 1
          for (int sl = lo; sl < hi; sl += 2) {
            uint4 x[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              x[h] = make_uint4(0, 0, 0, 0);
              if (have[h & 1] && sl + (h >> 1) < hi)
                x[h] = *reinterpret_cast<const uint4*>(from + (sl - sl0 + (h >> 1)) * kCodeSlab + (key0 + 32 * (h & 1)) * 64 + c * 16);
            }
#pragma unroll
            for (int h = 0; h < 4; ++h)
              if (h < 2 || sl + 1 < hi) store_codes<K>(stage + (sl + (h >> 1)) * kSlab + (key0 + 32 * (h & 1)) * 128, key0, c, x[h]);
          }
        };
        for (int lo = sl0; lo < sl1;) {      // slabs of one kind: all of them, or the value's and then the key's
          const int32_t kind = lo < p.vslabs ? p.vq : p.kq;
          const int hi = lo < p.vslabs && p.kq != p.vq ? p.vslabs : sl1;
          with_kind(kind, [&](auto k) { convert(k, lo, hi); });
          lo = hi;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&ms.kv_full[st]));
          mbar_arrive(smem_u32(&ms.code_empty[sg]));
        }
        kv.next(p.ns);
        code.next(p.nsg);
      }
    }
  } else {
    set_max_regs_inc<kRegsSoftmax>();
    // ------------------------------------------------------------ softmax, rescaling, epilogue
    const int tid = threadIdx.x, quad = warp & 3, half = warp >> 2;
    const int row = quad * 32 + lane;                // the row this thread owns, with the other half's
    const int col0 = half * 32;                      // its columns of S
    const uint32_t lane_base = static_cast<uint32_t>(32 * quad) << 16;
    const int v_chunks = (p.Dv + 127) / 128;
    int32_t jt = 0, piece = 0, loaded = 0;
    Ring kv;
    bool ok = true;
    for (; ok && walk.next(p, w); ++piece) {
      const int32_t n = w.tb - w.ta;
      bar_softmax();                                 // the previous piece's row arrays are done with
      const bool live = row < w.rows;
      const int32_t my_tok = w.tok + (p.hblocks > 1 ? 0 : static_cast<int32_t>(static_cast<uint32_t>(row) / static_cast<uint32_t>(p.hb)));
      if (half == 0 && row < NR)
        out_row[row] = live ? (w.q_start + my_tok) * p.heads + w.head + row - (my_tok - w.tok) * p.hb : -1;
      if (piece == 0 && tid == 0 && w.t0 > 0) {
        // the block behind the first cut through an item joins the item's pieces
        const int64_t item0 = start - w.t0;
        const int32_t first = static_cast<int32_t>(item0 / per), last = static_cast<int32_t>((item0 + w.T - 1) / per);
        int32_t* mt = p.join.meta + 8 * blockIdx.x;
        mt[1] = first;
        mt[2] = last;
        mt[3] = w.rows;
        mt[4] = 0;
        mt[5] = w.q_start + w.tok;
        mt[6] = w.head;
        mt[7] = w.n;
        mt[0] = first + 1 == static_cast<int32_t>(blockIdx.x) ? 1 : 0;
      }
      if (k_quant && n > 0) {
        ok = scale_q<F16>(p, w.n, w.rows, smem, row_scale, row_const, warp, lane, smem_u32(&ms.q_full), loaded & 1, abort_flag);
        fence_proxy_async_smem();
        ok = bar_or(ok ? 0u : 1u) == 0;
        if (!ok) break;
        if (lane == 0) mbar_arrive(smem_u32(&ms.q_ready));
        ++loaded;
      }
      const float sl2 = live && k_quant && n > 0 ? row_scale[row] : p.sl2;
      const float lazy = lazy_slack(kLazy, sl2);
      const int32_t seen = p.causal && live ? min(w.len, max(0, w.len - w.Lq + my_tok + 1)) : w.len;
      const bool rows_here = quad * 32 < w.rows;     // uniform in the warp
      float m = neg_inf(), l = 0.f;
      for (int32_t j = 0; j < n; ++j) {
        const int32_t u = jt + j;
        if (!bounded_wait_warp(smem_u32(&ms.s_full[u & 1]), (u >> 1) & 1, p.wait_ns, abort_flag)) ok = false;
        tc_fence_after();
        uint32_t s[32];
        float top = neg_inf();
        const uint64_t valid = ms.valid[u % kValidRing];
        if (ok && rows_here) {
          tmem_ld_x32(tmem + lane_base + (u & 1) * kKeys + col0, s);
          tmem_ld_wait();
          const int32_t nv = seen - (w.ta + j) * kKeys - col0;  // keys of these 32 that the row sees
          uint32_t mask = static_cast<uint32_t>(valid >> col0);
          if (nv < 32) mask &= nv <= 0 ? 0u : (1u << nv) - 1;
          if (__any_sync(0xffffffffu, mask != ~0u)) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((mask >> c) & 1)) s[c] = __float_as_uint(neg_inf());
          }
          float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
          for (int c = 0; c < 32; c += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx[e] = fmaxf(mx[e], fmaxf(__uint_as_float(s[c + e]), __uint_as_float(s[c + 4 + e])));
          top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        }
        // a row's maximum grew, or a wait gave up
        const uint32_t any = bar_or((live && top > m + lazy) || !ok ? 1u : 0u);
        if (j > 0) {  // P's buffer is free, and the accumulator complete, once the last product is
          if (ok && !bounded_wait_warp(smem_u32(&ms.pv_done), (u - 1) & 1, p.wait_ns, abort_flag)) ok = false;
          tc_fence_after();
        }
        if (any) {
          if (row < NR) xch[half * NR + row] = top;
          if (bar_or(ok ? 0u : 1u)) {  // the group leaves together
            ok = false;
            break;
          }
          float f = 1.f;
          if (live) top = fmaxf(top, xch[(half ^ 1) * NR + row]);
          if (live && top > m + lazy) {
            f = ex2((m - top) * sl2);
            l *= f;
            m = top;
          }
          bar_softmax();
          if (half == 0 && row < NR) xch[row] = f;
          bar_softmax();
          if (j > 0) {
#pragma unroll 1
            for (int c = 0; c < v_chunks; ++c) {
              if (c * 128 + quad * 32 >= p.Dv) break;
#pragma unroll 1
              for (int col = half * 8; col < w.rows; col += 16) {
                const uint32_t at = tmem + lane_base + kSCols + c * NR + col;
                uint32_t o[8];
                tmem_ld_x8(at, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * xch[col + e]);
                tmem_st_x8(at, o);
              }
            }
            tmem_st_wait();
          }
        }
        if (ok && rows_here) {
          const float neg = m == neg_inf() ? kLift : fmaf(-m, sl2, kLift);
          float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          uint32_t x[16], lo[16];
          exp_batch<!P16, PLO>(s, make_float2(sl2, sl2), make_float2(neg, neg), acc, x, lo);
          if (live) {
            uint8_t* prow = smem + p.off_p + row * 128;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int at = ((4 * half + c) ^ (row & 7)) << 4;
              *reinterpret_cast<uint4*>(prow + at) = make_uint4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
              if (PLO) *reinterpret_cast<uint4*>(prow + NR * 128 + at) = make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
            }
          }
          const float2 sum = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
          l += sum.x + sum.y;
        }
        if (p.vq == 0 && valid != ~0ull) {  // zero the value rows that do not exist, four threads per row
          const int key = tid >> 2;
          if (!((valid >> key) & 1)) {
            uint8_t* vrow = smem + p.off_ring + kv.stage * p.stage_bytes + key * 128 + (tid & 3) * 32;
            for (int c = 0; c < p.vslabs; ++c) {
              *reinterpret_cast<uint4*>(vrow + c * kSlab) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(vrow + c * kSlab + 16) = make_uint4(0, 0, 0, 0);
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ms.p_ready));
        kv.next(p.ns);
      }
      if (ok && n > 0) ok = bounded_wait_warp(smem_u32(&ms.pv_done), (jt + n - 1) & 1, p.wait_ns, abort_flag);
      if (row < NR) xch[half * NR + row] = l;
      ok = bar_or(ok ? 0u : 1u) == 0;
      if (!ok) break;
      tc_fence_after();
      jt += n;

      // ---- epilogue: final rows, or the piece's statistics and accumulator
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (piece == 0 && w.t0 > 0 ? 0 : 1);
      const bool whole = w.whole();
      if (half == 0 && row < NR) {
        l += xch[NR + row];
        inv_sum[row] = l != 0.f ? 1.f / l : 0.f;  // a row that sees nothing is 0; a NaN stays one
        const float shift = k_quant && n > 0 && live ? row_const[row] : 0.f;
        if (live && whole && p.lse)
          p.lse[out_row[row]] = l != 0.f ? fmaf(m, sl2, -kLift) * 0.6931471805599453f + logf(l) + shift : neg_inf();
        if (live && !whole) p.join.stats[slot * NR + row] = make_float4(m == neg_inf() ? neg_inf() : fmaf(m, sl2, -kLift), l, shift, 0.f);
      }
      bar_softmax();
      // Rolled loops over eight rows at a time: this code runs once a piece, and each line of
      // it comes from L2 (unrolled over 16 rows it took 26k cycles for 64 rows of 512).
#pragma unroll 1
      for (int c = 0; c < v_chunks; ++c) {
        const int ch = c * 128 + row;                 // this lane's channel
        if (c * 128 + quad * 32 >= p.Dv) break;
        float2 so = make_float2(1.f, 0.f);
        if (whole && p.vq) so = value_quant(p, w.n, min(ch, p.Dv - 1));
        const float inv_s = 1.f / so.x;
        float* part = p.join.parts + slot * NR * p.Dv + ch;
#pragma unroll 1
        for (int col = half * 8; col < w.rows; col += 16) {
          uint32_t o[8];
          if (n > 0) {
            tmem_ld_x8(tmem + lane_base + kSCols + c * NR + col, o);
            tmem_ld_wait();
          }
          if (ch >= p.Dv || (!whole && n == 0)) continue;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int r = col + e;
            if (r >= w.rows) break;
            if (whole) {
              const float inv = inv_sum[r];
              const float y = inv != 0.f ? (__uint_as_float(o[e]) * inv - so.y) * inv_s : 0.f;
              p.out[static_cast<int64_t>(out_row[r]) * p.Dv + ch] = to_half<F16>(y);
            } else {
              part[r * p.Dv] = __uint_as_float(o[e]);
            }
          }
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && *abort_flag) *p.status = 1;
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

struct Plan {
  int32_t NR, G, hb, tb, hblocks;
  int32_t whole, room;          // room: blocks that the workspace is sized for
  int64_t items;                // at most
  int32_t ns, nsg;
  int32_t vslabs, kslabs, qslabs, kslab0, stage, staging, off_p, off_ring, off_staging, off_misc, smem;
};

bool p_in_two(const PagedLaunch& L) { return L.f16 && (L.kq != 0 || L.vq != 0); }
int p_bytes(const PagedLaunch& L, int nr) { return nr * 128 * (p_in_two(L) ? 2 : 1); }

// The rows of a tile: as many as a sequence's tokens and heads fill on average, so that a
// decode step does not pay for 128, within what shared memory leaves for two stages.
bool plan(const PagedLaunch& L, Plan* pl) {
  const bool v1 = L.variant == 1;
  const int g = L.heads / static_cast<int32_t>(L.N);
  pl->vslabs = (L.Dv + 63) / 64;
  pl->kslabs = ((v1 ? L.R : L.Dkv) + 63) / 64;
  pl->qslabs = v1 ? pl->vslabs + pl->kslabs : pl->kslabs;
  pl->kslab0 = v1 ? 0 : pl->vslabs;
  pl->stage = (pl->vslabs + pl->kslabs) * kSlab;
  const bool staged = L.kq != 0 || L.vq != 0;
  pl->staging = ((L.vq ? pl->vslabs : 0) + (L.kq ? pl->kslabs : 0)) * kCodeSlab;
  const int64_t mean = (L.total_q + L.B - 1) / L.B * g;
  int nr = mean <= 16 ? 16 : mean <= 32 ? 32 : mean <= 64 ? 64 : 128;
  const int chunks = (L.Dv + 127) / 128;
  for (;; nr >>= 1) {
    if (nr < 16) return false;
    if (kSCols + chunks * nr > 512) continue;
    const int fixed = pl->qslabs * nr * 128 + p_bytes(L, nr) + ((static_cast<int>(sizeof(Misc)) + 15) & ~15) + row_arrays_bytes(nr) + 16;
    const int left = kSmemMax - fixed;
    if (!staged) {
      pl->nsg = 0;
      pl->ns = std::min(kMaxStages, left / pl->stage);
      if (pl->ns < 2) continue;
    } else {
      if (left < pl->stage + pl->staging) continue;
      // as many operand stages as leave two staging ones (a tile on its way, one being converted)
      pl->ns = std::max(1, std::min(4, (left - 2 * pl->staging) / pl->stage));
      if (pl->ns == 1 && left >= 2 * pl->stage + pl->staging) pl->ns = 2;
      pl->nsg = std::min(4, (left - pl->ns * pl->stage) / pl->staging);
    }
    break;
  }
  pl->NR = nr;
  pl->off_p = pl->qslabs * nr * 128;
  pl->off_ring = pl->off_p + p_bytes(L, nr);
  pl->off_staging = pl->off_ring + pl->ns * pl->stage;
  pl->off_misc = pl->off_staging + pl->nsg * pl->staging;
  pl->smem = pl->off_misc + ((static_cast<int>(sizeof(Misc)) + 15) & ~15) + row_arrays_bytes(nr) + 16;
  // one block per SM, and no more than there are tiles at the largest lengths
  pl->hb = std::min(g, nr);
  pl->tb = nr / pl->hb;
  pl->hblocks = g > nr ? (g + nr - 1) / nr : 1;
  if (pl->hblocks > 1) pl->tb = 1;
  const int64_t rts = pl->hblocks > 1 ? L.total_q * pl->hblocks : std::min<int64_t>(L.total_q, L.total_q / pl->tb + L.B);
  pl->items = rts * L.N;
  const int64_t T = std::max<int64_t>(1, (L.max_seq_len + kKeys - 1) / kKeys);
  const double share = static_cast<double>(pl->items) / kMaxBlocks, rounds = std::ceil(share);  // rounds of whole items
  pl->whole = (rounds - share) * static_cast<double>(T) <= kJoinTiles + kJoinAll * std::min(share, 1.0);
  const auto blocks = [](int64_t runs) { return static_cast<int32_t>(std::min<int64_t>(kMaxBlocks, std::max<int64_t>(1, runs))); };
  pl->G = blocks(pl->whole ? pl->items : pl->items * T);
  // as if items were cut always: a workspace that is sized at the largest batch, which may take
  // whole items, serves the smaller ones, which cut theirs
  pl->room = blocks(pl->items * T);
  return true;
}

template <bool F16, bool P16, bool PLO>
cudaError_t launch(const Params& p, int blocks, int64_t items, int smem, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto kernel = paged_attention_kernel<F16, P16, PLO>;
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev);
  }
  kernel<<<blocks, kThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return p.whole ? cudaSuccess : launch_join(p.join, F16, blocks, items, stream);
}

}  // namespace

size_t paged_attention_workspace(const PagedLaunch& L) {
  if (paged_tile_serves(L)) return kAttnHeader + paged_tile_workspace(L);
  Plan pl;
  if (!plan(L, &pl)) return 0;
  return kAttnHeader + join_bytes(pl.room, pl.NR, L.Dv);
}

cudaError_t launch_paged_attention(const PagedLaunch& L, cudaStream_t stream, const char** why) {
  if (paged_tile_serves(L)) return launch_paged_tile(L, stream, why);
  Plan pl;
  if (!plan(L, &pl)) {
    *why = "no tile shape fits";
    return cudaErrorInvalidValue;
  }
  Params p{};
  p.join.NR = p.join.sub = pl.NR;
  join_place(&p.join, L.partials, pl.G);
  pl.G = std::min(pl.G, device_sm_count());
  p.out = L.out;
  p.lse = L.lse;
  p.k_scale = L.k_scale;
  p.k_offset = L.k_offset;
  p.v_scale = L.v_scale;
  p.v_offset = L.v_offset;
  p.cu_q = L.cu_q;
  p.seq_lens = L.seq_lens;
  p.table = L.table;
  p.err_count = L.err_count;
  p.status = L.status;
  p.join.out = L.out;
  p.join.lse = L.lse;
  p.join.v_scale = L.v_scale;
  p.join.v_offset = L.v_offset;
  p.join.o_hs = L.Dv;
  p.join.o_ts = static_cast<int64_t>(L.Dv) * L.heads;
  p.join.heads = L.heads;
  p.join.hb = pl.hb;
  p.join.tb = pl.tb;
  p.join.Dv = L.Dv;
  p.join.per_head = L.variant == 2;
  p.join.v_scalar = L.v_scalar;
  p.table_stride = L.table_stride;
  const int64_t room = L.mode == kModeNorm ? L.cache_seq : L.table_stride * L.block_size;
  p.cap = std::min<int64_t>(room, L.max_seq_len);
  p.block_num = L.block_num;
  p.cache_seq = L.cache_seq;
  p.B = static_cast<int32_t>(L.B);
  p.total_q = static_cast<int32_t>(L.total_q);
  p.N = static_cast<int32_t>(L.N);
  p.heads = L.heads;
  p.g = L.heads / static_cast<int32_t>(L.N);
  p.NR = pl.NR;
  p.block_size = static_cast<int32_t>(L.block_size);
  p.bs_shift = -1;
  for (int s = 0; s < 31; ++s)
    if ((int64_t(1) << s) == L.block_size) p.bs_shift = s;
  p.v1 = L.variant == 1;
  p.Dk = L.Dkv;
  p.Dv = L.Dv;
  p.Dko = p.v1 ? L.R : L.Dkv;
  p.mode = L.mode;
  p.f16 = L.f16;
  p.kq = L.kq;
  p.vq = L.vq;
  p.k_scalar = L.k_scalar;
  p.v_scalar = L.v_scalar;
  p.causal = L.causal;
  p.hb = pl.hb;
  p.tb = pl.tb;
  p.hblocks = pl.hblocks;
  p.box_rows = L.mode == kModeNorm || L.block_size % 64 == 0 ? 64 : L.block_size % 32 == 0 ? 32 : 16;
  p.box_shift = p.box_rows == 64 ? 6 : p.box_rows == 32 ? 5 : 4;
  if (!encode_maps([&] {
        return make_q_map(&p.tq, L, pl.hb, pl.tb) && make_map(&p.tv, L.v_cache, L, L.Dv, L.vq, p.box_rows) &&
               make_map(&p.tk, L.k_cache, L, p.Dko, L.kq, p.box_rows);
      })) {
    *why = "cuTensorMapEncodeTiled failed or is unavailable";
    return cudaErrorInvalidValue;
  }
  p.vslabs = pl.vslabs;
  p.kslabs = pl.kslabs;
  p.qslabs = pl.qslabs;
  p.kslab0 = pl.kslab0;
  p.ns = pl.ns;
  p.nsg = pl.nsg;
  p.stage_bytes = pl.stage;
  p.staging_bytes = pl.staging;
  p.off_p = pl.off_p;
  p.off_ring = pl.off_ring;
  p.off_staging = pl.off_staging;
  p.off_misc = pl.off_misc;
  p.scale = L.scale;
  p.sl2 = static_cast<float>(static_cast<double>(L.scale) * 1.4426950408889634);
  p.wait_ns = static_cast<uint64_t>(L.wait_ns);
  p.whole = pl.whole;
  p.stall_loads = L.stall_loads;

  if (L.f16)
    return p_in_two(L) ? launch<true, true, true>(p, pl.G, pl.items, pl.smem, stream)
                       : launch<true, true, false>(p, pl.G, pl.items, pl.smem, stream);
  return L.vq ? launch<false, true, false>(p, pl.G, pl.items, pl.smem, stream)
              : launch<false, false, false>(p, pl.G, pl.items, pl.smem, stream);
}

}  // namespace ra
