// The attention kernel for many query rows: two 128-row tiles of queries against a stream
// of key tiles, for packed prompts (packed_attention.cuh) and for chunks of new tokens over
// paged caches (paged_tile.cuh).
//
// A work item is two row tiles of one head (packed) or of one kv head's group of heads
// (paged: a row is a (token, head) pair), against the keys of one sequence.  The key tiles
// of all items form one line that is cut into equal runs, one per block (attn_join.cuh), and a
// block streams through its run: while one tile's softmax runs, the tensor core works on
// the other's products, and the next item's queries arrive while this one ends.
//
//   S = Q K^T from shared memory, O += P V with P read from TMEM, where the softmax left
//   it in place of S; tensor memory: S / P of the two row tiles (128 columns each), then
//   their O (128 each).
//
// Warps 0-3 and 4-7: softmax of the two row tiles, one row per thread, which also rescale
// and write O; warp 8: TMA; warp 9: MMA; warp 10 finds the block's pieces (a walk over the
// sequences' lengths, full of loads and divisions) ahead of the others and hands them over
// in shared memory; with quantised caches warps 12-15 convert codes.
// P is rounded to the type of its operand, as the tensor core takes it: half a step of each
// weight, beside that of the result (bf16: 2.3e-3 off in all, 1.7e-3 with fp32 weights).
// The running maximum follows only when a tile exceeds it by 2^kLazy (the factor cancels
// between the weighted sum and the sum of weights), so O is rescaled in the first few tiles
// of a piece and hardly ever after.  Quantised keys and values enter the products as codes,
// as in paged_rows.cuh.  Every wait on an mbarrier is bounded in time (status word); the
// groups of softmax warps that meet at other barriers leave a piece, and the loop, together.
#pragma once

#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "attention.h"
#include "attn_join.cuh"
#include "attn_ptx.cuh"
#include "internal.h"
#include "kv_cache.h"
#include "paged_codes.cuh"

namespace ra {
namespace {

constexpr int kTileRows = 128;              // query rows of a tile
constexpr float kTileLazy = 8.f;            // log2 of how far a tile may exceed the running maximum
constexpr uint64_t kTileDrainNs = 200000000ull;
constexpr int kTileValid = 16;              // > key tiles between the loads and the softmax
constexpr int kTileMinRun = 4;              // key tiles per block below which a cut costs more than it gives
constexpr int kTilePieces = 4;              // pieces handed over ahead
// What an item costs beside its key tiles (its queries' arrival, its rows' way out), in key
// tiles: they stand at the item's start in the line.
constexpr int kTileExtra = 2;
// Items per block from which blocks take whole items: at most about a 16th is lost to uneven
// ends, and nothing is joined.  With few sequences they take every G-th item, so that the
// blocks are at one head or two at a time and read its keys from L2 together (480p
// self-attention: 14.2 ms; 17.3 with runs cut anywhere, whose blocks stream 40 heads' keys
// from HBM, which costs the tensor core power as well as time); over many sequences, each of
// which a strided walk would have to look up, they take consecutive ones.
constexpr int kTileWholeItems = 16, kTileStrideSeqs = 64;
enum TileRuns : int32_t { kRunsCut = 0, kRunsWhole = 1, kRunsStrided = 2 };

struct TileParams {
  CUtensorMap tq, tk, tv;
  JoinParams join;                          // also out, lse, strides, the value's scales
  const int32_t *cu_q, *cu_k;               // packed: first tokens; paged: cu_k holds the sequences' lengths
  const int32_t* table;
  int32_t* err_count;
  int32_t* status;
  const float *k_scale, *k_offset;
  int64_t table_stride, cap, block_num, cache_seq;
  int32_t B, total_q, total_k;
  int32_t items;                            // heads an item can have: query heads (packed), kv heads (paged)
  int32_t heads_first;                      // the line's order within a sequence: heads within row blocks (1), or
                                            // row blocks within heads (0)
  int32_t g;                                // query heads per kv head
  int32_t Dk, ksteps;
  int32_t causal, mode, block_size, bs_shift, box_rows, box_shift;
  int32_t q_swap, k_swap, v_swap;           // packed: the map's axes are (channels, tokens, heads)
  int32_t kq, vq;
  int32_t out32;                            // every row of out starts on 32 bytes
  float scale, sl2;                         // softmax scale, and with log2(e)
  uint64_t wait_ns;
  int32_t stall_loads;
  // EXT
  Window window;
  int32_t cu_step, shifts;
  SharedPrefix prefix;
};

// KS, VS: 64-channel slabs of a key and a value; KT: keys per tile; QUANT: both caches hold
// codes; PAGED: keys through a block table
template <int KS, int VS, int KT, bool QUANT>
struct TileShape {
  static constexpr int kThreads = QUANT ? 512 : 384;
  static constexpr int kQTile = KS * kTileRows * 128;
  static constexpr int kSlab = KT * 128;
  static constexpr int kK = KS * kSlab, kV = VS * kSlab;
  static constexpr int kCode = (KS > VS ? KS : VS) * KT * 64;   // a staging slot: a tile's codes of either cache
  static constexpr int kFree = 232448 - 2 * kQTile - (3 << 10);  // TileMisc takes less than 3 KB
  static constexpr int kNsg = QUANT ? 2 : 0;
  static constexpr int kPairs = (kFree - kNsg * kCode) / (kK + kV);
  static constexpr int kNv = kPairs > 5 ? 5 : kPairs;
  static constexpr int kNkMost = (kFree - kNsg * kCode - kNv * kV) / kK;
  static constexpr int kNk = kNkMost > 5 ? 5 : kNkMost;
  static constexpr int kOffK = 2 * kQTile;
  static constexpr int kOffV = kOffK + kNk * kK;
  static constexpr int kOffCode = kOffV + kNv * kV;
  static constexpr int kOffMisc = kOffCode + kNsg * kCode;
  static_assert(kNk >= 1 && kNv >= 1, "shared memory budget");
};
__device__ __forceinline__ void tile_span(const int32_t* cu, int32_t b, int32_t B, int32_t total, int32_t& start,
                                          int32_t& len, int32_t step = 1) {
  if (cu == nullptr) {
    len = total / B;
    start = b * len;
    return;
  }
  const int32_t lo = min(max(__ldg(cu + b), 0), total), hi = min(max(__ldg(cu + b + step), lo), total);
  start = lo;
  len = hi - lo;
}

// Key tiles that block b of a sequence's rows counts for in the line: q0 + step (b + 1)
// between 1 and most (step 0: most), and kTileExtra.  Packed causal prompts have step 2: 256 rows see 256
// keys more than the 256 before them.  Paged chunks count all of the sequence's keys for every
// block, masked or not.
struct TileCount {
  int32_t blocks, q0, step, most;
  __device__ __forceinline__ int32_t of(int32_t b) const {
    return kTileExtra + (step == 0 ? most : max(1, min(most, q0 + step * (b + 1))));
  }
  // of the first n blocks
  __device__ int64_t sum(int32_t n) const {
    const int64_t extra = static_cast<int64_t>(n) * kTileExtra;
    if (step == 0) return extra + static_cast<int64_t>(n) * most;
    const int32_t lo = min(n, max(0, (1 - q0 + step - 1) / step - 1));       // blocks that count 1
    const int32_t hi = max(lo, min(n, max(0, (most - q0 + step - 1) / step - 1)));  // and those below `most`
    const int64_t mid = hi - lo;
    return extra + lo + mid * q0 + step * ((static_cast<int64_t>(lo) + 1 + hi) * mid / 2) + static_cast<int64_t>(n - hi) * most;
  }
};

// What a piece of a call with a window or a prefix has beside the rest: tiles of the sinks or the prefix, and how
// much further the others' positions are; the first row's window; positions of the prefix, whose
// tiles are those ahead.
struct TileAhead {
  int32_t ahead, skip, win, prefix;
};
struct TileNoneAhead {
  static constexpr int32_t ahead = 0, skip = 0, win = 0, prefix = 0;
};
template <bool EXT>
struct TilePiece : std::conditional_t<EXT, TileAhead, TileNoneAhead> {
  int32_t end;                              // there is no further piece
  int32_t first;                            // the first of its block
  int32_t b, head, kv_head, tok, q_start, Lq, k_start, Lk;
  int32_t rows[2];                          // of the two row tiles
  int32_t t0, take, T;                      // tiles [t0, t0 + take) of the item's T in the line
  int32_t ta, tb[2];                        // those that a row of either tile sees: [ta, tb[i])
  int32_t from, to;                         // blocks that share the item, where the block before began it
  __device__ __forceinline__ bool whole() const { return take == T; }
  __device__ __forceinline__ int32_t n(int i) const { return max(0, tb[i] - ta); }
  // the first position of tile t
  template <int KT>
  __device__ __forceinline__ int32_t pos(int32_t t) const { return t * KT + (EXT && t >= this->ahead ? this->skip : 0); }
  // where the keys that tile t counts end; `seen` stands for the sequence's own
  __device__ __forceinline__ int32_t end_of(int32_t t, int32_t seen) const {
    return EXT && this->prefix > 0 && t < this->ahead ? this->prefix : seen;
  }
};

template <bool EXT>
struct TileMisc {
  uint64_t k_full[5], k_empty[5], v_full[5], v_empty[5], c_full[2], c_empty[2];
  uint64_t q_full[2], q_ready[2], q_empty[2], s_full[2], p_ready[2], o_done[2], drain;
  uint64_t piece_full[kTilePieces], piece_empty[kTilePieces];
  uint64_t valid[kTileValid][2];
  uint32_t holes[kTileValid];               // whether keys before the sequence's end are absent: a page is (EXT: 2), or
                                            // no row sees them (1)
  TilePiece<EXT> pieces[kTilePieces];
  int64_t scan[16], scan_items[16];
  int64_t start_off;
  int32_t start_b;
  uint32_t tmem;
  int32_t abort;
  int32_t pad;
  float inv_scale[2][192];                  // 1 / the key's scales, for each softmax group
};

// a / b of numbers that are not negative: a 64-bit division is a hundred instructions
__device__ __forceinline__ int64_t tile_quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// The spans of 32 sequences, one to a lane: a walk over them waits for memory once.
template <int KT, bool PAGED, bool EXT>
struct TileSpans {
  int32_t base, q_start, Lq, k_start, Lk;
  int32_t prefix;                           // EXT, PAGED: positions ahead of every sequence's own
  __device__ void one(const TileParams& p, int32_t b) {
    tile_span(p.cu_q, b, p.B, p.total_q, q_start, Lq, EXT ? p.cu_step : 1);
    if (PAGED) {
      k_start = 0;
      Lk = static_cast<int32_t>(min(static_cast<int64_t>(max(__ldg(p.cu_k + b), 0)), p.cap));
    } else {
      tile_span(p.cu_k, b, p.B, p.total_k, k_start, Lk);
    }
  }
  __device__ void load_prefix(const TileParams& p) {
    prefix = EXT && PAGED ? prefix_length(p.prefix) : 0;
  }
  __device__ void load(const TileParams& p, int32_t from) {
    base = from;
    const int32_t b = from + static_cast<int32_t>(threadIdx.x & 31);
    q_start = Lq = k_start = Lk = 0;
    if (b < p.B) one(p, b);
  }
  __device__ TileCount count(const TileParams& p, int32_t Lq, int32_t Lk) const {
    const int32_t tokens = 2 * p.join.tb;
    TileCount c;
    c.blocks = static_cast<int32_t>((static_cast<uint32_t>(Lq) + tokens - 1) / static_cast<uint32_t>(tokens));
    c.most = max(1, (Lk + KT - 1) / KT + (EXT && PAGED ? (prefix + KT - 1) / KT : 0));
    if (EXT) c.most = min(c.most, p.window.most);
    c.step = p.causal && !PAGED ? 2 * kTileRows / KT : 0;
    c.q0 = Lk >= Lq ? (Lk - Lq + KT - 1) / KT : -((Lq - Lk) / KT);
    return c;
  }
  // of the sequence that the thread holds
  __device__ int64_t work(const TileParams& p, int64_t* items) const {
    const TileCount c = count(p, Lq, Lk);
    *items += static_cast<int64_t>(c.blocks) * p.items;
    return c.sum(c.blocks) * p.items;
  }
};

// Walks a block's pieces, a whole warp at once.
template <int KT, bool PAGED, bool EXT>
struct TileWalk {
  int32_t b, item, blk, t;                  // next: sequence, head, row block, key tile
  int64_t rem;
  TilePiece<EXT> w;                         // of the sequence that c is of: its spans
  TileCount c;
  int32_t runs;                             // TileRuns
  TileSpans<KT, PAGED, EXT> spans;

  __device__ TileCount count(const TileParams& p, int32_t b, TilePiece<EXT>& w) {
    if (b >= spans.base + 32) spans.load(p, b);
    w.q_start = __shfl_sync(0xffffffffu, spans.q_start, b - spans.base);
    w.Lq = __shfl_sync(0xffffffffu, spans.Lq, b - spans.base);
    w.k_start = __shfl_sync(0xffffffffu, spans.k_start, b - spans.base);
    w.Lk = __shfl_sync(0xffffffffu, spans.Lk, b - spans.base);
    return spans.count(p, w.Lq, w.Lk);
  }
  // to offset `off` of sequence b, for `run` tiles
  __device__ void seek(const TileParams& p, int32_t seq, int64_t off, int64_t run, int32_t kind) {
    b = seq;
    rem = run;
    runs = kind;
    if (runs == kRunsStrided) {             // the block's first item is item blockIdx.x of all
      b = 0;
      rem = 1;
      t = item = blk = 0;
      c = count(p, b, w);
      skip(p, blockIdx.x);
      return;
    }
    c = count(p, b, w);
    const int64_t per_head = c.sum(c.blocks), each = p.heads_first ? p.items : 1;
    if (!p.heads_first) {
      item = static_cast<int32_t>(tile_quotient(off, per_head));
      off -= item * per_head;
    }
    int32_t lo = 0, hi = c.blocks - 1;      // the last block that begins at or before off
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) / 2;
      if (c.sum(mid) * each <= off) lo = mid;
      else hi = mid - 1;
    }
    blk = lo;
    off -= c.sum(lo) * each;
    if (p.heads_first) {
      item = static_cast<int32_t>(tile_quotient(off, c.of(blk)));
      off -= static_cast<int64_t>(item) * c.of(blk);
    }
    t = static_cast<int32_t>(off);
    if (runs == kRunsWhole && t > 0) {      // an item that the block before began
      rem -= c.of(blk) - t;
      advance(p);
    }
  }
  // n items on
  __device__ void skip(const TileParams& p, int64_t n) {
    n += p.heads_first ? static_cast<int64_t>(blk) * p.items + item : static_cast<int64_t>(item) * c.blocks + blk;
    while (n >= static_cast<int64_t>(p.items) * c.blocks) {
      n -= static_cast<int64_t>(p.items) * c.blocks;
      if (++b >= p.B) return;
      c = count(p, b, w);
    }
    const uint32_t inner = p.heads_first ? p.items : c.blocks;  // n < items * blocks < 2^31
    const int32_t outer = static_cast<int32_t>(static_cast<uint32_t>(n) / inner);
    const int32_t rest = static_cast<int32_t>(n - static_cast<int64_t>(outer) * inner);
    blk = p.heads_first ? outer : rest;
    item = p.heads_first ? rest : outer;
  }
  __device__ void advance(const TileParams& p) {
    t = 0;
    if (runs == kRunsStrided) {
      skip(p, gridDim.x);
      return;
    }
    if (p.heads_first) {
      if (++item < p.items) return;
      item = 0;
      if (++blk < c.blocks) return;
      blk = 0;
    } else {
      if (++blk < c.blocks) return;
      blk = 0;
      if (++item < p.items) return;
      item = 0;
    }
    do {
      if (++b >= p.B) return;
      c = count(p, b, w);
    } while (c.blocks == 0);
  }
  // the next piece into w
  __device__ bool next(const TileParams& p) {
    if (rem <= 0 || b >= p.B) return false;
    const int32_t T = c.of(blk);
    w.b = b;
    w.T = T;
    w.t0 = t;
    w.take = runs != kRunsCut ? T : static_cast<int32_t>(min(static_cast<int64_t>(T - t), rem));
    w.kv_head = PAGED ? item : static_cast<int32_t>(static_cast<uint32_t>(item) / static_cast<uint32_t>(p.g));
    w.head = PAGED ? item * p.g : item;
    w.tok = blk * 2 * p.join.tb;
    int32_t skip = 0;
    if constexpr (EXT) {
      w.prefix = spans.prefix;
      w.win = window_from(p.window, w.tok + w.Lk - w.Lq);
      w.ahead = PAGED && p.prefix.len ? (w.prefix + KT - 1) / KT : p.window.tiles;
      skip = PAGED && p.prefix.len ? -w.ahead : max(0, w.win / KT - w.ahead);
      w.skip = skip * KT;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int32_t first = w.tok + i * p.join.tb, tokens = max(0, min(p.join.tb, w.Lq - first));
      const int32_t seen = p.causal ? min(w.Lk, max(0, first + tokens + w.Lk - w.Lq)) : w.Lk;
      w.rows[i] = tokens * p.join.hb;
      w.tb[i] = tokens == 0 ? 0 : min(w.t0 + w.take - kTileExtra, (seen + KT - 1) / KT - skip);
    }
    w.ta = max(0, w.t0 - kTileExtra);
    if (runs != kRunsStrided) rem -= w.take;
    t += w.take;
    return true;
  }
  __device__ void done(const TileParams& p) {  // with the piece that next gave
    if (t == w.T) advance(p);
  }
};

// whether all 128 threads of a softmax group are well
__device__ __forceinline__ bool group_ok(uint32_t id, bool ok) {
  uint32_t bad;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(bad)
      : "r"(ok ? 0u : 1u), "r"(id)
      : "memory");
  return bad == 0;
}

// The next piece that warp 10 handed over, for a whole warp; false at the end or when a wait
// gave up.  GROUP: over codes the softmax groups meet at barriers in a piece, which have no time
// limit, so the warps of a group (barrier `id`) take a piece, or leave, together.
template <bool GROUP = false, bool EXT>
__device__ __forceinline__ bool take_piece(TileMisc<EXT>& ms, Ring& ring, TilePiece<EXT>& w, uint64_t limit, volatile int* abort_flag,
                                           bool& ok, uint32_t id = 0) {
  ok = ok && bounded_wait_warp(smem_u32(&ms.piece_full[ring.stage]), ring.parity, limit, abort_flag);
  if (GROUP) ok = group_ok(id, ok);
  if (!ok) return false;
  w = ms.pieces[ring.stage];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&ms.piece_empty[ring.stage]));
  ring.next(kTilePieces);
  return !w.end;
}

template <bool F16>
__device__ __forceinline__ float tile_half(uint32_t u) {
  return F16 ? __half2float(__ushort_as_half(static_cast<uint16_t>(u))) : __uint_as_float(u << 16);
}

// Hides a row's keys from nv on and those of [lo, hi), 32 columns at a time: a choice for each element only
// where some row of the warp does not see all of them.  (A comparison and a choice for each of 128 columns,
// on a pipe of half the rate, took 1600 cycles of a masked tile's 3200: 9001 tokens of 7 prompts in a
// window of 1024 166 us, 162 with this.)
template <int KT>
__device__ __forceinline__ void hide_keys(uint32_t (&s)[KT], int32_t nv, int32_t lo, int32_t hi) {
  if (!__any_sync(0xffffffffu, nv < KT || (hi > lo && lo < KT))) return;
#pragma unroll
  for (int c = 0; c < KT; c += 32) {
    uint32_t seen = nv - c >= 32 ? ~0u : nv <= c ? 0u : (1u << (nv - c)) - 1;
    const int32_t from = max(lo - c, 0), to = min(hi - c, 32);
    if (to > from) seen &= ~((~0u >> (32 - to)) & (~0u << from));
    if (__any_sync(0xffffffffu, seen != ~0u)) {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (!((seen >> e) & 1)) s[c + e] = __float_as_uint(neg_inf());
    }
  }
}

// F16: q and out (and 16-bit caches) are fp16; P16: P and the value operand are
// EXT: windows; rows that leave in fp32 for another call, or join another's (Prior)
template <int KS, int VS, int KT, bool F16, bool QUANT, bool PAGED, bool EXT>
__global__ void __launch_bounds__(QUANT ? 512 : 384, 1) tile_attention_kernel(const __grid_constant__ TileParams p) {
  using SH = TileShape<KS, VS, KT, QUANT>;
  constexpr bool P16 = F16 || QUANT;
  // fp16 results over codes: q / s is rounded to 11 bits, like the result; so that P's rounding
  // does not add a third error of that size, P goes in as two fp16 numbers (hi + lo).  The
  // products of a tile cost half as much again, which the softmax hides for the most part.
  constexpr bool kPLo = F16 && QUANT;
  constexpr float kLift = P16 ? kHalfLift : 0.f;
  // Registers per thread: launched with 168 (QUANT: 128) each, then moved to the softmax:
  // 2 x 216 + 72 = 3 x 168; 2 x 192 + 64 + 64 = 4 x 128
  constexpr int kRegsSoftmax = QUANT ? 192 : 216, kRegsRest = QUANT ? 64 : 72;
  constexpr int kTmaWarp = 8, kMmaWarp = 9, kPieceWarp = 10, kConvert0 = 12;
  extern __shared__ __align__(1024) uint8_t smem[];
  TileMisc<EXT>& ms = *reinterpret_cast<TileMisc<EXT>*>(smem + SH::kOffMisc);
  const uint32_t s0 = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  using Walk = TileWalk<KT, PAGED, EXT>;

  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&ms.tmem), 512);
    tmem_relinquish();
  } else if (threadIdx.x == 0) {
    for (int s = 0; s < SH::kNk; ++s) {
      mbar_init(smem_u32(&ms.k_full[s]), QUANT ? 4 : 1);
      mbar_init(smem_u32(&ms.k_empty[s]), 1);
    }
    for (int s = 0; s < SH::kNv; ++s) {
      mbar_init(smem_u32(&ms.v_full[s]), QUANT ? 4 : 1);
      mbar_init(smem_u32(&ms.v_empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ms.c_full[i]), 1);
      mbar_init(smem_u32(&ms.c_empty[i]), 4);
      mbar_init(smem_u32(&ms.q_full[i]), 1);
      mbar_init(smem_u32(&ms.q_ready[i]), 4);
      mbar_init(smem_u32(&ms.q_empty[i]), 1);
      mbar_init(smem_u32(&ms.s_full[i]), 1);
      mbar_init(smem_u32(&ms.p_ready[i]), 4);
      mbar_init(smem_u32(&ms.o_done[i]), 1);
    }
    for (int i = 0; i < kTilePieces; ++i) {
      mbar_init(smem_u32(&ms.piece_full[i]), 1);
      mbar_init(smem_u32(&ms.piece_empty[i]), QUANT ? 14 : 10);  // the warps that read a piece
    }
    mbar_init(smem_u32(&ms.drain), 1);
    ms.abort = 0;
    fence_mbar_init();
    p.join.meta[8 * blockIdx.x] = 0;        // nothing to join, unless the first piece says so below
  } else if (threadIdx.x == 32 * kTmaWarp) {
    prefetch_tensormap(&p.tq);
    prefetch_tensormap(&p.tk);
    prefetch_tensormap(&p.tv);
  }
  grid_launch_dependents();

  // ---- this block's run of key tiles.  Up to 32 sequences the warp that walks them finds it
  // alone, beside the set-up above; more are counted by all threads.
  const bool few = p.B <= 32;
  Walk walk;
  int64_t per = 0, start = 0;
  if (few ? warp == kPieceWarp : true) {
    walk.spans.load_prefix(p);
    walk.spans.load(p, 0);
    int64_t mine = 0, items = 0;
    int32_t b_lo = lane, b_hi = lane;
    if (few) {
      if (lane < p.B) mine = walk.spans.work(p, &items);
    } else {
      const int32_t chunk = (p.B + SH::kThreads - 1) / SH::kThreads;
      b_lo = min(p.B, static_cast<int32_t>(threadIdx.x) * chunk);
      b_hi = min(p.B, b_lo + chunk);
      TileSpans<KT, PAGED, EXT> one;
      one.prefix = walk.spans.prefix;
      for (int32_t b = b_lo; b < b_hi; ++b) {
        one.one(p, b);
        mine += one.work(p, &items);
      }
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
      items += __shfl_xor_sync(0xffffffffu, items, o);
    }
    int64_t before = incl - mine, W = 0;
    if (few) {
      W = __shfl_sync(0xffffffffu, incl, 31);
    } else {
      if (lane == 31) {
        ms.scan[warp] = incl;
        ms.scan_items[warp] = items;
      }
      __syncthreads();
      items = 0;
#pragma unroll
      for (int w = 0; w < SH::kThreads / 32; ++w) {
        const int64_t t = ms.scan[w];
        if (w < warp) before += t;
        W += t;
        items += ms.scan_items[w];
      }
    }
    // equal runs, but of kTileMinRun tiles at least where the items have that many
    const int64_t G = gridDim.x;
    per = tile_quotient(W + G - 1, G);
    if (per < kTileMinRun && items > 0) per = max(per, min(static_cast<int64_t>(kTileMinRun), tile_quotient(W + items - 1, items)));
    const int32_t runs = items < kTileWholeItems * G ? kRunsCut : p.B <= kTileStrideSeqs ? kRunsStrided : kRunsWhole;
    start = per * blockIdx.x;
    const bool here = before <= start && start < before + mine;
    int32_t at_b = p.B;
    int64_t at_off = 0;
    if (few) {
      const uint32_t at = __ballot_sync(0xffffffffu, here);
      if (at) {
        at_b = __ffs(at) - 1;
        at_off = start - __shfl_sync(0xffffffffu, before, at_b);
      }
    } else {
      if (here) {
        TileSpans<KT, PAGED, EXT> one;
        one.prefix = walk.spans.prefix;
        int32_t b = b_lo;
        int64_t off = start - before, unused = 0;
        for (; b < b_hi; ++b) {
          one.one(p, b);
          const int64_t w = one.work(p, &unused);
          if (off < w) break;
          off -= w;
        }
        ms.start_b = b;
        ms.start_off = off;
      }
      __syncthreads();
      if (start < W) {
        at_b = ms.start_b;
        at_off = ms.start_off;
      }
    }
    if (warp == kPieceWarp) {
      walk.b = p.B;                         // a block without a run (strided: every block has its 16 items and more)
      walk.rem = 0;
      if (W > 0 && (start < W || runs == kRunsStrided)) walk.seek(p, at_b, at_off, min(per, W - start), runs);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem;
  volatile int* abort_flag = &ms.abort;
  TilePiece<EXT> w{};
  Ring pieces;
  if (warp >= 8 && warp < 12) {
    set_max_regs_dec<kRegsRest>();
    if (warp == kPieceWarp) {
      // ------------------------------------------------------------ pieces
      bool more = true, first = true;
      while (more) {
        more = walk.next(p);
        walk.w.end = more ? 0 : 1;
        walk.w.first = first ? 1 : 0;
        if (first && more && walk.w.t0 > 0) {
          const int64_t item0 = start - walk.w.t0;
          walk.w.from = static_cast<int32_t>(tile_quotient(item0, per));
          walk.w.to = static_cast<int32_t>(tile_quotient(item0 + walk.w.T - 1, per));
        }
        first = false;
        if (!bounded_wait_warp(smem_u32(&ms.piece_empty[pieces.stage]), pieces.parity ^ 1u, p.wait_ns, abort_flag)) break;
        if (__any_sync(0xffffffffu, *abort_flag)) break;  // no piece for those that are about to leave
        if (lane == 0) {
          ms.pieces[pieces.stage] = walk.w;
          mbar_arrive(smem_u32(&ms.piece_full[pieces.stage]));
        }
        __syncwarp();
        pieces.next(kTilePieces);
        if (more) walk.done(p);
      }
    } else if (warp == kTmaWarp && !p.stall_loads) {
      // ------------------------------------------------------------ loads
      const int groups = PAGED ? KT >> p.box_shift : 1;
      const int per_trip = PAGED ? 32 / groups * groups : 32;
      Ring kr, vr, cr;
      uint32_t q_par[2] = {0, 0}, u = 0;
      // copies in flight, by ring: which stages, and the parity of their last use
      uint32_t armed_k = 0, armed_v = 0, armed_c = 0, armed_q = 0, par_k = 0, par_v = 0, par_c = 0, par_q = 0;
      bool ok = true;
      auto mark = [](uint32_t& armed, uint32_t& par, int st, uint32_t parity) {
        armed |= 1u << st;
        par = (par & ~(1u << st)) | (parity << st);
      };
      while (take_piece(ms, pieces, w, p.wait_ns, abort_flag, ok)) {
        const int32_t t_end = max(w.tb[0], w.tb[1]);
        if (w.ta >= t_end) continue;
        // Cache rows: lane i holds where group `base + i` of the piece starts, per_trip groups
        // of box_rows keys per trip to the block table.
        int64_t row = -1;
        bool hidden = false;                // EXT: no row sees the group, and its page may be gone
        int32_t base = w.ta * groups - per_trip;
        // the queries, once the products of the last ones are through with them
        auto load_q = [&] {
          for (int i = 0; ok && i < 2; ++i) {
            if (w.n(i) == 0) continue;
            ok = bounded_wait_warp(smem_u32(&ms.q_empty[i]), q_par[i] ^ 1u, p.wait_ns, abort_flag);
            if (!ok) break;
            if (elect_one()) {
              const uint32_t bar = smem_u32(&ms.q_full[i]);
              const int32_t tok = w.q_start + w.tok + i * p.join.tb;
              mbar_arrive_expect_tx(bar, KS * p.join.tb * p.join.hb * 128);
#pragma unroll
              for (int c = 0; c < KS; ++c)
                tma_load_3d(s0 + i * SH::kQTile + c * kTileRows * 128, &p.tq, bar, 64 * c, p.q_swap ? tok : w.head,
                            p.q_swap ? w.head : tok);
            }
            __syncwarp();
            mark(armed_q, par_q, i, q_par[i]);
            q_par[i] ^= 1u;
          }
        };
        // A block's first queries go first: with codes their scaling stands before the first product.
        if (EXT && w.first) load_q();
        for (int32_t t = w.ta; ok && t < t_end; ++t, ++u) {
          uint32_t have = 1;                // which of the tile's groups exist
          if (PAGED) {
            if (t * groups >= base + per_trip) {
              base += per_trip;
              int32_t pos = (base + lane) << p.box_shift;
              const bool own = !EXT || base + lane >= w.ahead * groups;
              if constexpr (EXT) {
                if (own) pos += w.skip;
                hidden = pos + p.box_rows <= w.win && pos >= p.window.sinks;
              }
              row = -1;
              if (lane < per_trip && base + lane < t_end * groups && pos < (EXT && !own && w.prefix > 0 ? w.prefix : w.Lk) && !hidden) {
                if (p.mode == kModeNorm) {
                  row = (static_cast<int64_t>(w.b) * p.items + w.kv_head) * p.cache_seq + pos;
                } else {
                  const int32_t pg = p.bs_shift >= 0 ? pos >> p.bs_shift : pos / p.block_size;
                  const int32_t in = pos - pg * p.block_size;
                  const int32_t* table = EXT && !own && w.prefix > 0 ? p.prefix.table : p.table + w.b * p.table_stride;
                  const int64_t page = __ldg(table + pg);
                  if (page >= 0 && page < p.block_num)
                    row = p.mode == kModePa ? page * p.block_size + in : (page * p.items + w.kv_head) * p.block_size + in;
                  else if (p.err_count)
                    atomicAdd(p.err_count, 1);
                }
              }
            }
            have = (__ballot_sync(0xffffffffu, row >= 0) >> (t * groups - base)) & ((1u << groups) - 1);
          }
          const uint32_t live = __popc(have);
          const int32_t pos0 = w.template pos<KT>(t), end = w.end_of(t, w.Lk);
          const int32_t y = PAGED ? (p.mode == kModePa ? w.kv_head : 0) : w.kv_head;
          // 0: the key tile, 1: the value tile
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            if (side == 1 && t == w.ta && !(EXT && w.first)) {
              // behind the first key tile, whose place in the ring is free earlier
              load_q();
              if (!ok) break;
            }
            const int st = side ? vr.stage : kr.stage;
            const uint32_t par = side ? vr.parity : kr.parity;
            if (QUANT)
              ok = bounded_wait_warp(smem_u32(&ms.c_empty[cr.stage]), cr.parity ^ 1u, p.wait_ns, abort_flag);
            else
              ok = bounded_wait_warp(smem_u32(side ? &ms.v_empty[st] : &ms.k_empty[st]), par ^ 1u, p.wait_ns, abort_flag);
            if (!ok) break;
            const int slabs = side ? VS : KS;
            const uint32_t bar = smem_u32(QUANT ? &ms.c_full[cr.stage] : side ? &ms.v_full[st] : &ms.k_full[st]);
            const uint32_t dst = s0 + (QUANT ? SH::kOffCode + cr.stage * SH::kCode
                                             : side ? SH::kOffV + st * SH::kV : SH::kOffK + st * SH::kK);
            const uint32_t row_bytes = QUANT ? 64 : 128;
            const CUtensorMap* map = side ? &p.tv : &p.tk;
            if (side == 0 && PAGED) {
              uint64_t lo = 0, hi = 0;      // which of the tile's keys exist
              for (int g = 0; g < groups; ++g) {
                const int32_t at = g << p.box_shift, keys = min(p.box_rows, end - (pos0 + at));
                if (!((have >> g) & 1)) continue;
                const uint64_t bits = keys >= 64 ? ~0ull : (1ull << keys) - 1;
                if (at < 64) lo |= bits << at;
                else hi |= bits << (at - 64);
                if (keys > 64) hi |= keys >= 128 ? ~0ull : (1ull << (keys - 64)) - 1;
              }
              const uint32_t absent = min(groups, (end - pos0 + p.box_rows - 1) >> p.box_shift) - live;
              uint32_t unseen = 0;
              if constexpr (EXT)
                unseen = __popc(__ballot_sync(0xffffffffu, hidden && lane >= t * groups - base && lane < (t + 1) * groups - base));
              if (lane == 0) {
                ms.valid[u % kTileValid][0] = lo;
                ms.valid[u % kTileValid][1] = hi;
                ms.holes[u % kTileValid] = absent == 0 ? 0 : EXT && absent == unseen ? 1 : 2;
              }
              __syncwarp();
            }
            if (PAGED) {
              if (elect_one()) mbar_arrive_expect_tx(bar, live * slabs * p.box_rows * row_bytes);
              __syncwarp();
              for (int g = 0; g < groups; ++g) {
                const int32_t z = __shfl_sync(0xffffffffu, static_cast<int32_t>(row), t * groups - base + g);
                if (((have >> g) & 1) && elect_one()) {
                  const uint32_t to = dst + (g << p.box_shift) * row_bytes;
#pragma unroll
                  for (int c = 0; c < slabs; ++c)
                    tma_load_3d(to + c * KT * row_bytes, map, bar, 64 * c, y, z);
                }
                __syncwarp();
              }
            } else {
              if (elect_one()) {
                const int32_t z = w.k_start + pos0, swap = side ? p.v_swap : p.k_swap;
                mbar_arrive_expect_tx(bar, side ? SH::kV : SH::kK);
#pragma unroll
                for (int c = 0; c < slabs; ++c) tma_load_3d(dst + c * SH::kSlab, map, bar, 64 * c, swap ? z : y, swap ? y : z);
              }
              __syncwarp();
            }
            if (QUANT) {
              mark(armed_c, par_c, cr.stage, cr.parity);
              cr.next(SH::kNsg);
            } else if (side) {
              mark(armed_v, par_v, st, par);
              vr.next(SH::kNv);
            } else {
              mark(armed_k, par_k, st, par);
              kr.next(SH::kNk);
            }
          }
        }
      }
      // Let every copy in flight land before the block leaves: whoever waits for the last ones may
      // give up only after this warp has come through, so it asks no flag.
      for (int i = 0; i < 5; ++i) {
        if (armed_k >> i & 1) bounded_drain(smem_u32(&ms.k_full[i]), par_k >> i & 1, kTileDrainNs);
        if (armed_v >> i & 1) bounded_drain(smem_u32(&ms.v_full[i]), par_v >> i & 1, kTileDrainNs);
        if (armed_c >> i & 1) bounded_drain(smem_u32(&ms.c_full[i]), par_c >> i & 1, kTileDrainNs);
        if (armed_q >> i & 1) bounded_drain(smem_u32(&ms.q_full[i]), par_q >> i & 1, kTileDrainNs);
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ products
      constexpr uint32_t id_s = idesc_f16(!P16, false, false, kTileRows, KT);
      constexpr uint32_t id_o = idesc_f16(!P16, false, true, kTileRows, VS * 64);
      const uint64_t q_desc = sdesc_kmajor_sw128(s0), k_desc = sdesc_kmajor_sw128(s0 + SH::kOffK);
      const uint64_t v_desc = sdesc_mnmajor_sw128(s0 + SH::kOffV, SH::kSlab);
      Ring kr, vr;
      uint32_t q_par[2] = {0, 0}, p_par[2] = {0, 0};
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t par) {
        if (ok) ok = bounded_wait_warp(smem_u32(bar), par, p.wait_ns, abort_flag);
        return ok;
      };
      auto issue_s = [&](int i, int st, bool last) {  // one lane
        const uint64_t a = q_desc + static_cast<uint64_t>(i * (SH::kQTile >> 4));
        const uint64_t bd = k_desc + static_cast<uint64_t>(st * (SH::kK >> 4));
#pragma unroll
        for (int k = 0; k < KS * 4; ++k)
          if (k < (KS - 1) * 4 || k < p.ksteps)
            mma_f16_ss(tmem + 128 * i, a + (k >> 2) * (kTileRows * 128 >> 4) + (k & 3) * 2,
                       bd + (k >> 2) * (SH::kSlab >> 4) + (k & 3) * 2, id_s, k > 0);
        tc_commit(smem_u32(&ms.s_full[i]));
        if (last) tc_commit(smem_u32(&ms.q_empty[i]));
      };
      while (take_piece(ms, pieces, w, p.wait_ns, abort_flag, ok)) {
        const int32_t n0 = w.n(0), n1 = w.n(1), n = max(n0, n1);
        if (n == 0) continue;
        if (!wait(&ms.k_full[kr.stage], kr.parity)) break;
        for (int i = 0; i < 2; ++i) {
          const int32_t ni = i ? n1 : n0;
          if (ni == 0) continue;
          if (!wait(QUANT ? &ms.q_ready[i] : &ms.q_full[i], q_par[i])) break;
          q_par[i] ^= 1u;
          tc_fence_after();
          if (elect_one()) issue_s(i, kr.stage, ni == 1);
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) tc_commit(smem_u32(&ms.k_empty[kr.stage]));
        __syncwarp();
        kr.next(SH::kNk);
        for (int32_t j = 0; ok && j < n; ++j) {
          if (!wait(&ms.v_full[vr.stage], vr.parity)) break;
          if (j + 1 < n && !wait(&ms.k_full[kr.stage], kr.parity)) break;
          for (int i = 0; i < 2; ++i) {
            const int32_t ni = i ? n1 : n0;
            if (j >= ni) continue;
            if (!wait(&ms.p_ready[i], p_par[i])) break;
            p_par[i] ^= 1u;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t bd = v_desc + static_cast<uint64_t>(vr.stage * (SH::kV >> 4));
#pragma unroll
              for (int k = 0; k < KT / 16; ++k)
                mma_f16_ts(tmem + 256 + 128 * i, tmem + 128 * i + 8 * k, bd + 128 * k, id_o, j > 0 || k > 0);
              if (kPLo)
#pragma unroll
                for (int k = 0; k < KT / 16; ++k)
                  mma_f16_ts(tmem + 256 + 128 * i, tmem + 128 * i + KT / 2 + 8 * k, bd + 128 * k, id_o, true);
              if (j + 1 < ni) issue_s(i, kr.stage, j + 2 == ni);
              else tc_commit(smem_u32(&ms.o_done[i]));
            }
            __syncwarp();
          }
          if (!ok) break;
          if (elect_one()) {
            tc_commit(smem_u32(&ms.v_empty[vr.stage]));
            if (j + 1 < n) tc_commit(smem_u32(&ms.k_empty[kr.stage]));
          }
          __syncwarp();
          vr.next(SH::kNv);
          if (j + 1 < n) kr.next(SH::kNk);
        }
      }
      if (elect_one()) tc_commit(smem_u32(&ms.drain));  // every product must finish before TMEM is released
      __syncwarp();
      bounded_drain(smem_u32(&ms.drain), 0, kTileDrainNs);
      __syncwarp();
    }
  } else if (QUANT && warp >= kConvert0) {
    // ------------------------------------------------------------ codes to fp16 operands
    set_max_regs_dec<kRegsRest>();
    const int tid = threadIdx.x - 32 * kConvert0;
    Ring kr, vr, cr;
    uint32_t u = 0;
    bool ok = !p.stall_loads;
    while (take_piece(ms, pieces, w, p.wait_ns, abort_flag, ok)) {
      const int32_t t_end = max(w.tb[0], w.tb[1]);
      for (int32_t t = w.ta; ok && t < t_end; ++t, ++u) {
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
          Ring& r = side ? vr : kr;
          ok = bounded_wait_warp(smem_u32(&ms.c_full[cr.stage]), cr.parity, p.wait_ns, abort_flag) &&
               bounded_wait_warp(smem_u32(side ? &ms.v_empty[r.stage] : &ms.k_empty[r.stage]), r.parity ^ 1u, p.wait_ns,
                                 abort_flag);
          if (!ok) break;
          uint8_t* stage = smem + (side ? SH::kOffV + r.stage * SH::kV : SH::kOffK + r.stage * SH::kK);
          const uint8_t* from = smem + SH::kOffCode + cr.stage * SH::kCode;
          const uint64_t valid[2] = {ms.valid[u % kTileValid][0], ms.valid[u % kTileValid][1]};
          // KT keys x 4 chunks of 16 codes per slab, 32 keys a round of the 128 threads
          const int c = tid & 3, rounds = (side ? VS : KS) * (KT / 32);
          with_kind(side ? p.vq : p.kq, [&](auto kind) {
            constexpr int K = decltype(kind)::value;
#pragma unroll 1
            for (int h0 = 0; h0 < rounds; h0 += 4) {
              uint4 x[4];
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const int sl = (h0 + h) / (KT / 32), key = (tid >> 2) + 32 * ((h0 + h) % (KT / 32));
                x[h] = make_uint4(0, 0, 0, 0);
                if (h0 + h < rounds && (valid[key >> 6] >> (key & 63)) & 1)
                  x[h] = *reinterpret_cast<const uint4*>(from + sl * KT * 64 + key * 64 + c * 16);
              }
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const int sl = (h0 + h) / (KT / 32), key = (tid >> 2) + 32 * ((h0 + h) % (KT / 32));
                if (h0 + h < rounds) store_codes<K>(stage + sl * SH::kSlab + key * 128, key, c, x[h]);
              }
            }
          });
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(side ? &ms.v_full[r.stage] : &ms.k_full[r.stage]));
            mbar_arrive(smem_u32(&ms.c_empty[cr.stage]));
          }
          r.next(side ? SH::kNv : SH::kNk);
          cr.next(SH::kNsg);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax, one row per thread
    set_max_regs_inc<kRegsSoftmax>();
    const int i = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_addr = tmem + 128 * i + lane_base, o_addr = tmem + 256 + 128 * i + lane_base;
    uint32_t s_par = 0, o_par = 0, q_par = 0, u = 0;
    Ring vr;
    bool ok = true;
    while (take_piece<QUANT>(ms, pieces, w, p.wait_ns, abort_flag, ok, 1 + i)) {
      const int32_t n = w.n(i), n_both = max(w.n(0), w.n(1));
      const bool live = row < w.rows[i];
      const int32_t in_tile = static_cast<int32_t>(static_cast<uint32_t>(row) / static_cast<uint32_t>(p.join.hb));
      const int32_t tok = w.tok + i * p.join.tb + in_tile, head = w.head + row - in_tile * p.join.hb;
      const int32_t seen = !p.causal ? w.Lk : min(w.Lk, max(0, tok + 1 + w.Lk - w.Lq));
      const int32_t from = EXT ? window_from(p.window, tok + w.Lk - w.Lq) : 0;  // of the row's window
      if (w.first && threadIdx.x == 0 && w.t0 > 0) {
        // the block behind the first cut through an item joins the item's pieces
        int32_t* mt = p.join.meta + 8 * blockIdx.x;
        mt[1] = w.from;
        mt[2] = w.to;
        mt[3] = w.rows[0];
        mt[4] = w.rows[1];
        mt[5] = w.q_start + w.tok;
        mt[6] = w.head;
        mt[7] = w.kv_head;
        mt[0] = w.from + 1 == static_cast<int32_t>(blockIdx.x) ? 1 : 0;
      }
      // where the row goes
      const bool whole = w.whole();
      const int64_t token = w.q_start + tok;
      const int64_t part_row = (2 * static_cast<int64_t>(blockIdx.x) + (w.first && w.t0 > 0 ? 0 : 1)) * 2 * kTileRows + i * kTileRows + row;
      uint16_t* const dst = p.join.out + token * p.join.o_ts + head * p.join.o_hs;
      float* const part = p.join.parts + part_row * p.join.Dv;
      float sl2 = p.sl2, shift = 0.f;
      if (QUANT && n > 0) {
        // The row of q over the key's scales, behind a power of two that keeps its elements
        // below 2^15 (a bound serves: fp16 holds 11 bits down to 2^-14), in place.
        const int tid = threadIdx.x & 127;
        float* inv = ms.inv_scale[i];
        const float* ks = p.k_scale + static_cast<int64_t>(w.kv_head) * p.Dk;
        float top = 0.f;
        for (int c = tid; c < p.Dk; c += 128) inv[c] = rcp(__ldg(ks + c));
        asm volatile("bar.sync %0, 128;" ::"r"(1 + i) : "memory");
        for (int c = 0; c < p.Dk; c += 4) {
          const float4 x = *reinterpret_cast<const float4*>(inv + c);
          top = fmaxf(fmaxf(fmaxf(top, fabsf(x.x)), fmaxf(fabsf(x.y), fabsf(x.z))), fabsf(x.w));
        }
        ok = bounded_wait_warp(smem_u32(&ms.q_full[i]), q_par, p.wait_ns, abort_flag);
        q_par ^= 1u;
        uint8_t* mine_row = smem + i * SH::kQTile + row * 128;
        auto at = [&](int c) { return mine_row + (c >> 3) * kTileRows * 128 + (((c & 7) ^ (row & 7)) << 4); };
        uint32_t big = 0;  // |q| as bits orders like the value in either type
        const int nck = p.Dk / 8;
#pragma unroll 2
        for (int c = 0; c < nck; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(at(c));
          big = __vmaxu2(__vmaxu2(big, x.x & 0x7FFF7FFFu), x.y & 0x7FFF7FFFu);
          big = __vmaxu2(__vmaxu2(big, x.z & 0x7FFF7FFFu), x.w & 0x7FFF7FFFu);
        }
        big = max(big & 0xFFFFu, big >> 16);
        const int k = max(-100, min(100, -(scale_exponent(tile_half<F16>(big)) + scale_exponent(top) + 15)));
        const float up = exp2_int(k);
        sl2 = p.sl2 * exp2_int(-k);
        if ((EXT ? p.shifts != 0 : p.join.lse != nullptr) && p.k_offset) {
          const float* ko = p.k_offset + static_cast<int64_t>(w.kv_head) * p.Dk;
#pragma unroll 1
          for (int c = 0; c < nck; ++c) {
            const uint4 z = *reinterpret_cast<const uint4*>(at(c));
            const uint32_t z4[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
              shift -= tile_half<F16>((z4[e >> 1] >> (16 * (e & 1))) & 0xFFFFu) / __ldg(ks + 8 * c + e) * __ldg(ko + 8 * c + e) * p.scale;
          }
        }
#pragma unroll 2
        for (int c = 0; c < nck; ++c) {
          const uint4 z = *reinterpret_cast<const uint4*>(at(c));
          const float4 a = *reinterpret_cast<const float4*>(inv + 8 * c), b = *reinterpret_cast<const float4*>(inv + 8 * c + 4);
          uint4 y;
          y.x = pack_f16x2(tile_half<F16>(z.x & 0xFFFFu) * (a.x * up), tile_half<F16>(z.x >> 16) * (a.y * up));
          y.y = pack_f16x2(tile_half<F16>(z.y & 0xFFFFu) * (a.z * up), tile_half<F16>(z.y >> 16) * (a.w * up));
          y.z = pack_f16x2(tile_half<F16>(z.z & 0xFFFFu) * (b.x * up), tile_half<F16>(z.z >> 16) * (b.y * up));
          y.w = pack_f16x2(tile_half<F16>(z.w & 0xFFFFu) * (b.z * up), tile_half<F16>(z.w >> 16) * (b.w * up));
          *reinterpret_cast<uint4*>(at(c)) = y;
        }
        fence_proxy_async_smem();
        ok = group_ok(1 + i, ok);             // inv is read, every row is written
        if (!ok) break;
        if (lane == 0) mbar_arrive(smem_u32(&ms.q_ready[i]));
      }
      const float lazy = lazy_slack(kTileLazy, sl2);
      float m = neg_inf(), l = 0.f;
      for (int32_t j = 0; j < n; ++j) {
        if (!bounded_wait_warp(smem_u32(&ms.s_full[i]), s_par, p.wait_ns, abort_flag)) {
          ok = false;
          break;
        }
        s_par ^= 1u;
        tc_fence_after();
        const int32_t pos0 = w.template pos<KT>(w.ta + j), keys_end = w.end_of(w.ta + j, w.Lk);
        uint32_t s[KT];
#pragma unroll
        for (int c = 0; c < KT; c += 32) tmem_ld_x32(s_addr + c, s + c);
        tmem_ld_wait();
        const int32_t nv = w.end_of(w.ta + j, seen) - pos0;  // keys of this tile that the row sees
        if constexpr (EXT) {
          hide_keys<KT>(s, nv, max(p.window.sinks - pos0, 0), from - pos0);
        } else if (__any_sync(0xffffffffu, nv < KT)) {
#pragma unroll
          for (int c = 0; c < KT; ++c)
            if (c >= nv) s[c] = __float_as_uint(neg_inf());
        }
        const uint32_t hole = PAGED ? ms.holes[(u + j) % kTileValid] : 0;
        const bool holes = hole != 0;
        uint64_t gap[2] = {0, 0};           // keys before the end that do not exist (bad pages)
        if (holes) {
          const int32_t end = keys_end - pos0;
          const uint64_t* v = ms.valid[(u + j) % kTileValid];
          gap[0] = ~v[0] & (end >= 64 ? ~0ull : (1ull << end) - 1);
          if (KT > 64) {
            const int32_t keys = min(end, KT) - 64;
            gap[1] = keys <= 0 ? 0ull : ~v[1] & (keys >= 64 ? ~0ull : (1ull << keys) - 1);
          }
          if (!EXT || hole == 2) {
#pragma unroll
            for (int c = 0; c < KT; ++c)
              if ((gap[c >> 6] >> (c & 63)) & 1) s[c] = __float_as_uint(neg_inf());
          }
        }
        float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
        for (int c = 0; c < KT; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx[e] = fmaxf(mx[e], fmaxf(__uint_as_float(s[c + e]), __uint_as_float(s[c + 4 + e])));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // (each row by its own: the rows of a warp do not change one another's rounding, and
        // lanes without a row hold whatever was in shared memory)
        const bool grow = live && top > m + lazy;
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2((m - top) * sl2) : 1.f;
          if (grow) m = top;
          l *= f;
          if (j > 0) {  // S(j) was issued behind O += P V of tile j - 1, so O is complete here
#pragma unroll 1
            for (int c = 0; c < VS * 64; c += 32) {
              uint32_t o[32];
              tmem_ld_x32(o_addr + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st_x32(o_addr + c, o);
            }
          }
        }
        const float neg = m == neg_inf() ? kLift : fmaf(-m, sl2, kLift);
        const float2 sl = make_float2(sl2, sl2), ng = make_float2(neg, neg);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int h = 0; h < KT / 32; ++h) {
          uint32_t x[16], lo[16];
          exp_batch<!P16, kPLo>(s + 32 * h, sl, ng, acc, x, lo);
          tmem_st_x16(s_addr + 16 * h, x);  // P takes the place of S: KT / 2 columns of pairs
          if (kPLo) tmem_st_x16(s_addr + KT / 2 + 16 * h, lo);
        }
        const float2 sum = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
        l += sum.x + sum.y;
        if (!QUANT && (pos0 + KT > keys_end || holes)) {
          // value rows that are no key's meet P = 0, but 0 times a stray NaN or infinity is
          // NaN: zero them in shared memory
          const int32_t end = keys_end - pos0;
          if (!bounded_wait_warp(smem_u32(&ms.v_full[vr.stage]), vr.parity, p.wait_ns, abort_flag)) {
            tmem_st_wait();                 // of P: tensor memory is freed only behind its stores
            ok = false;
            break;
          }
          if (row < KT && (row >= end || ((gap[row >> 6] >> (row & 63)) & 1))) {
#pragma unroll 1
            for (int c = 0; c < VS; ++c) {
              uint4* dst = reinterpret_cast<uint4*>(smem + SH::kOffV + vr.stage * SH::kV + c * SH::kSlab + row * 128);
#pragma unroll
              for (int e = 0; e < 8; ++e) dst[e] = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ms.p_ready[i]));
        vr.next(SH::kNv);
      }
      if (ok && n > 0) {
        ok = bounded_wait_warp(smem_u32(&ms.o_done[i]), o_par, p.wait_ns, abort_flag);
        o_par ^= 1u;
      }
      if (QUANT) ok = group_ok(1 + i, ok);    // they meet at barriers, so they leave together
      if (!ok) break;
      tc_fence_after();
      for (int32_t j = n; j < n_both; ++j) vr.next(SH::kNv);  // tiles that only the other rows see
      u += n_both;

      // ---- final rows, or the piece's statistics and accumulator
      const float inv = l != 0.f ? rcp(l) : 0.f;  // a row that sees nothing is 0; a NaN stays one
      float2 share = make_float2(1.f, 0.f);
      const int64_t at = EXT ? token * p.join.heads + head : 0;
      if (live) {
        if (EXT && whole && (p.join.prior.stats_out || p.join.prior.stats)) {
          prior_end(p.join.prior, at, fmaf(m, sl2, -kLift), l, l != 0.f ? shift : 0.f, true, p.join.lse, share);
        } else if (whole) {
          if (p.join.lse)
            p.join.lse[token * p.join.heads + head] = l != 0.f ? fmaf(m, sl2, -kLift) * 0.6931471805599453f + logf(l) + shift : neg_inf();
        } else {
          p.join.stats[part_row] = make_float4(m == neg_inf() ? neg_inf() : fmaf(m, sl2, -kLift), l, shift, 0.f);
        }
      }
      const bool store = live && (whole || n > 0);
#pragma unroll 1
      for (int c = 0; c < VS * 64; c += 16) {
        if (c >= p.join.Dv) break;
        uint32_t o[16];
        if (n > 0) {
          tmem_ld_x16(o_addr + c, o);
          tmem_ld_wait();
        }
        if (!store) continue;
        if (!whole) {
          store_32(part + c, o);
          store_32(part + c + 8, o + 8);
          continue;
        }
        float y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = l != 0.f ? __uint_as_float(o[e]) * inv : 0.f;
        if (QUANT && l != 0.f) {
          const float* vs = p.join.v_scale + static_cast<int64_t>(w.kv_head) * p.join.Dv + c;
          const float* vo = p.join.v_offset ? p.join.v_offset + static_cast<int64_t>(w.kv_head) * p.join.Dv + c : nullptr;
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = (y[e] - (vo ? __ldg(vo + e) : 0.f)) * rcp(__ldg(vs + e));
        }
        if constexpr (EXT) {
          if (p.join.prior.rows_out) {
            float* const to = p.join.prior.rows_out + at * p.join.Dv + c;
            uint32_t u[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(y[e]);
            store_32(to, u);
            store_32(to + 8, u + 8);
            continue;
          }
          if (p.join.prior.rows) {
            const float4* o4 = reinterpret_cast<const float4*>(p.join.prior.rows + at * p.join.Dv + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 x = o4[e];
              y[4 * e] = fmaf(y[4 * e], share.x, x.x * share.y);
              y[4 * e + 1] = fmaf(y[4 * e + 1], share.x, x.y * share.y);
              y[4 * e + 2] = fmaf(y[4 * e + 2], share.x, x.z * share.y);
              y[4 * e + 3] = fmaf(y[4 * e + 3], share.x, x.w * share.y);
            }
          }
        }
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = pack_half2<!F16>(y[2 * e], y[2 * e + 1]);
        if (p.out32) {
          store_32(dst + c, h);
        } else {
          *reinterpret_cast<uint4*>(dst + c) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(h[4], h[5], h[6], h[7]);
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

template <int KS, int VS, int KT, bool F16, bool QUANT, bool PAGED, bool EXT = false>
cudaError_t launch_tile(const TileParams& p, int blocks, int64_t items, bool cuts, cudaStream_t stream) {
  using SH = TileShape<KS, VS, KT, QUANT>;
  constexpr int smem = SH::kOffMisc + static_cast<int>(sizeof(TileMisc<EXT>));
  static_assert(smem <= 232448, "shared memory budget");
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto kernel = tile_attention_kernel<KS, VS, KT, F16, QUANT, PAGED, EXT>;
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev);
  }
  kernel<<<blocks, SH::kThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return cuts ? launch_join<EXT>(p.join, F16, blocks, items, stream) : cudaSuccess;
}

// Whether the runs of `blocks` blocks cut items that all count for T key tiles (the kernel's own
// arithmetic).
inline bool tile_runs_cut(int64_t items, int64_t T, int64_t blocks) {
  if (items >= kTileWholeItems * blocks) return false;
  int64_t per = (items * T + blocks - 1) / blocks;
  if (per < kTileMinRun) per = std::max(per, std::min<int64_t>(kTileMinRun, T));
  return per % T != 0;
}

// Blocks for items of at most `tiles` key tiles: one per SM, and no more than there are items
// or runs of kTileMinRun tiles.
inline int tile_blocks(int64_t items, int64_t tiles) {
  return static_cast<int>(std::min<int64_t>(kMaxBlocks, std::max<int64_t>(items, items * tiles / kTileMinRun)));
}

}  // namespace
}  // namespace ra
