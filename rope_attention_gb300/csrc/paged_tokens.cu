// Attention of one token or a few over V2 caches: the kernel for up to 16 rows per sequence and kv head
// (a row is a token's head) of the calls with a window or a shared prefix.
//
//   S^T[key, row] = K q^T,  O^T[channel, row] += V^T P^T
//
// Here the work is the reading of the cache: a key of 320 codes meets 8 to 16 rows, 16 to 32 operations
// a byte where the tensor core does some 280 a byte of HBM, so the products go through warp-level MMAs
// on registers, and what counts is a short way from shared memory to the result.
//  * A tile is 64 keys.  Four warps take it, 16 keys each; the next four the next one.  A warp keeps its
//    own maximum, sum and accumulator, so nothing is exchanged before the end of a piece.
//  * M is the keys (then the channels) and N the rows, eight at a time: 8 rows cost half of what 16
//    would in the usual order.  S^T leaves the MMA as P^T's operand up to a transposition of 8 x 8
//    blocks within the warp.
//  * Codes become fp16 in registers.  The contraction's order is free as long as both operands have
//    the same: a lane takes 16 neighbouring channels of its keys for four steps (q is laid out to match), and
//    of the values 16 neighbouring channels of four keys, whose bytes it interleaves.  Rows of 192 and
//    64 bytes, and of 128 with the swizzle, then have no bank conflicts.
//  * Another warp walks the block table and issues TMA boxes of 16 to 64 keys into two to twelve stages:
//    whole rows of codes, 128 bytes of 16-bit ones.  (Two, one for each team, are what 16-bit rows of 192 + 128
//    channels and 9 to 16 rows leave room for: a team's next tile is on its way only when it has freed the
//    last.)  A third walks the pieces ahead of the others and lays out their queries.
// The runs of tiles, their parts and the join are paged_rows.cuh's.  The maximum follows only when a
// tile exceeds it by 2^kLazy.  Every wait on an mbarrier is bounded in time (status word); the warps meet
// at the end of a piece and leave it, or the loop, together.
// Measured: 8 sequences, 64 heads over 8, int8, 4096 positions in the window and 64 sinks 35 us, of which 28 tiles a
// block are 15 (5.6 TB/s while they run), a block's start 6 and the join 7 (57 us in paged_rows.cuh's kernel); 16 rows
// of 541 bf16 positions 14 us.  The same window over bf16 rows: 64 heads (four stages) 41 us, 4.1 TB/s; 128 heads, two stages,
// 51 us, 3.4 TB/s.  Bound by latency: the start, the join, and a tile's chain of loads, conversion, S, softmax and O.
#include "paged_tokens.cuh"

namespace ra {
namespace {

__device__ __forceinline__ uint4 lds_128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// D (+)= A B: 16 x 8 x 16
template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The chunk (16 bytes of a key's row) that lane t takes for its j-th load.  Eight lanes load at once, four
// chunks of two neighbouring keys: in rows of 128 bytes with the swizzle the even chunks of one
// meet the odd banks of the other, and so on.
template <bool KQ>
__device__ __forceinline__ int key_chunk(const Params& p, int j, int t) {
  if (!KQ || p.kslab0) return 8 * (j >> 1) + 2 * t + (j & 1);
  return 4 * j + t;
}

// Rows g (+ 8) of a piece's queries as the second operand of S^T, in to[nt][24][lane]: for codes over the
// key's scales and behind a power of two per row (paged_rows.cuh, scale_q), which row_scale undoes.
// Lane t of a row's four has its 16-byte chunks key_chunk(p, j, t): of 16-bit keys 8 channels each, two
// steps; of codes 16 channels, four steps.  One warp; rolled loops, as every line of code comes
// from L2 at the start of a block.
template <bool F16, bool KQ, int NT>
__device__ __forceinline__ void prepare_q(const Params& p, TokenPiece& w, uint32_t* to, int lane) {
  constexpr int kChunks = KQ ? 3 : 6, kWide = KQ ? 16 : 8;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll 1
  for (int nt = 0; nt < NT; ++nt, to += 24 * 32) {
    const int r = g + 8 * nt;
    const bool live = r < w.rows;
    const uint16_t* q = p.q + (static_cast<int64_t>(w.row[r].x) * p.heads + w.row[r].y) * p.Dk;
    uint32_t big = 0;           // |q| as bits orders like the value in either type
    uint4 x[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const int c = key_chunk<KQ>(p, i * 4 / (kWide / 2), t) * kWide + (KQ ? 8 * (i & 1) : 0);
      x[i] = live && c < p.Dk ? __ldg(reinterpret_cast<const uint4*>(q + c)) : make_uint4(0, 0, 0, 0);
    }
    float least = 3e38f, shift = 0.f;
    const float* ks = KQ ? p.k_scale + static_cast<int64_t>(w.kv_head) * p.Dk : nullptr;
    if constexpr (KQ) {
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int c = 16 * key_chunk<KQ>(p, j, t) + 4 * h;
          const float4 v = c < p.Dk ? __ldg(reinterpret_cast<const float4*>(ks + c)) : make_float4(3e38f, 3e38f, 3e38f, 3e38f);
          least = fminf(fminf(fminf(least, fabsf(v.x)), fminf(fabsf(v.y), fabsf(v.z))), fabsf(v.w));
        }
    }
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        to[(4 * i + e) * 32 + lane] = u[e];
        big = __vmaxu2(big, u[e] & 0x7FFF7FFFu);
      }
    }
    if constexpr (KQ) {
      big = max(big & 0xFFFFu, big >> 16);
      float top = rcp(least);
      if (p.shifts && p.k_offset) {
        const float* ko = p.k_offset + static_cast<int64_t>(w.kv_head) * p.Dk;
#pragma unroll 1
        for (int c = t; c < p.Dk && live; c += 4) shift += half_to_float<F16>(__ldg(q + c)) / __ldg(ks + c) * __ldg(ko + c);
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        shift += __shfl_xor_sync(0xffffffffu, shift, o);
      }
      const int k = max(-100, min(100, -(scale_exponent(half_to_float<F16>(big)) + scale_exponent(top) + 15)));
      const float up = exp2_int(k);
#pragma unroll 1
      for (int j = 0; j < kChunks; ++j) {
        const int c = 16 * key_chunk<KQ>(p, j, t);
        if (c >= p.Dk) continue;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(ks + c + 4 * h));
          uint32_t* const at = to + (8 * j + 2 * h) * 32 + lane;
          const uint32_t u0 = at[0], u1 = at[32];
          at[0] = pack_f16x2(half_to_float<F16>(u0 & 0xFFFFu) * (rcp(v.x) * up), half_to_float<F16>(u0 >> 16) * (rcp(v.y) * up));
          at[32] = pack_f16x2(half_to_float<F16>(u1 & 0xFFFFu) * (rcp(v.z) * up), half_to_float<F16>(u1 >> 16) * (rcp(v.w) * up));
        }
      }
      if (t == 0) {
        w.row_scale[r] = p.sl2 * exp2_int(-k);
        w.row_const[r] = -shift * p.scale;
      }
    } else if (t == 0) {
      w.row_scale[r] = p.sl2;
      w.row_const[r] = 0.f;
    }
  }
}

// F16: q, out and 16-bit caches are fp16, not bf16.  KQ, VQ: keys, values are codes.  NT: rows / 8.
template <bool F16, bool KQ, bool VQ, int NT>
__global__ void __launch_bounds__(kTokenThreads, 1) paged_tokens_kernel(const __grid_constant__ Params p) {
  constexpr bool K16 = F16 || KQ, P16 = F16 || VQ, PLO = F16 && (KQ || VQ);   // as in paged_rows.cuh
  constexpr float kLift = P16 ? kHalfLift : 0.f;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* meet = reinterpret_cast<float*>(smem + p.off_p);            // [warp][row][kTokenRow]
  uint32_t* queries = reinterpret_cast<uint32_t*>(meet + kTokenWarps * 8 * NT * kTokenRow);  // [2][NT][24][32]
  TokenMisc& ms = *reinterpret_cast<TokenMisc*>(smem + p.off_misc);
  const uint32_t s0 = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ns; ++s) {
      mbar_init(smem_u32(&ms.full[s]), 1);
      mbar_init(smem_u32(&ms.empty[s]), kTileWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&ms.piece_full[s]), 1);
      mbar_init(smem_u32(&ms.piece_empty[s]), kTokenWarps);
    }
    ms.abort = 0;
    fence_mbar_init();
    p.join.meta[8 * blockIdx.x] = 0;      // nothing to join, unless the first piece says so below
  } else if (threadIdx.x == 32 * kTokenLoad) {
    prefetch_tensormap(&p.tk);
    prefetch_tensormap(&p.tv);
  }
  grid_launch_dependents();
  Walker<true> walk;
  int64_t per, start;
  if (p.B > 32 || warp >= kTokenWarps) find_run<true, kTokenThreads>(p, blockIdx.x, gridDim.x, walk, ms.run, per, start);  // (B > 32: with a barrier)
  __syncthreads();
  volatile int* abort_flag = &ms.abort;
  Piece w{};
  Ring ring, pieces;
  bool ok = true;

  if (warp >= kTokenWarps) {
    set_max_regs_dec<kRegsOther>();
    start_run(p, walk, ms.run);
  }
  if (warp == kTokenPieces) {
    // ------------------------------------------------------------ pieces
    bool more = true;
    for (int32_t piece = 0; more; ++piece) {
      more = walk.next(p, w);
      if (!bounded_wait_warp(smem_u32(&ms.piece_empty[pieces.stage]), pieces.parity ^ 1u, p.wait_ns, abort_flag)) break;
      if (__any_sync(0xffffffffu, *abort_flag)) break;  // no piece for those that are about to leave
      TokenPiece& to = ms.pieces[pieces.stage];
      if (more) {
        const bool began = piece == 0 && w.t0 > 0;      // an item that the block before began
        if (began && lane == 0) {
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
        // row `lane`: its token and head (rows behind the last stand for it), and what it sees
        const int32_t r = min(lane, w.rows - 1);
        const int32_t tok = p.hblocks > 1 ? 0 : static_cast<int32_t>(static_cast<uint32_t>(r) / static_cast<uint32_t>(p.hb));
        const int32_t at = w.len - w.Lq + w.tok + tok;
        const int32_t seen = p.causal ? min(w.len, max(0, at + 1)) : w.len, from = window_from(p.window, at);
        const int32_t seen_least = __reduce_min_sync(0xffffffffu, seen), from_most = __reduce_max_sync(0xffffffffu, from);
        if (lane < 16) {
          to.row[lane] = make_int2(w.q_start + w.tok + tok, w.head + r - tok * p.hb);
          to.seen[lane] = seen;
          to.from[lane] = from;
        }
        if (lane == 0) {
          to.rows = w.rows;
          to.kv_head = w.n;
          to.ta = w.ta;
          to.n = max(0, w.tb - w.ta);
          to.ahead = w.ahead;
          to.skip = w.skip;
          to.prefix = w.prefix;
          to.whole = w.whole();
          to.slot = 2 * static_cast<int32_t>(blockIdx.x) + (began ? 0 : 1);
          to.seen_least = seen_least;
          to.from_most = from_most;
        }
        __syncwarp();
        if (w.tb > w.ta) prepare_q<F16, KQ, NT>(p, to, queries + pieces.stage * NT * 24 * 32, lane);
        else if (lane < 16) to.row_scale[lane] = p.sl2, to.row_const[lane] = 0.f;
      }
      if (lane == 0) to.end = more ? 0 : 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ms.piece_full[pieces.stage]));
      pieces.next(2);
    }
  } else if (warp == kTokenLoad) {
    // ------------------------------------------------------------ loads
    const int groups = kKeys >> p.box_shift;
    const int32_t v_row = VQ ? p.Dv : 128, k_row = KQ ? p.Dk : 128;  // bytes of a box's row
    const uint32_t group_bytes = p.box_rows * (p.kslabs * k_row + p.vslabs * v_row);
    uint32_t armed = 0, armed_parity = 0;  // copies in flight
    int32_t u = 0;
    ok = !p.stall_loads;
    while (ok && walk.next(p, w)) {
      if (w.ta >= w.tb) continue;
      // Cache rows.  Lane i holds where group `base + i` of the piece starts.
      const int32_t g_end = w.tb * groups, head = p.mode == kModePa ? w.n : 0;
      int64_t row = -1;
      int32_t base = w.ta * groups - 32;
      for (int32_t t = w.ta; t < w.tb; ++t, ++u) {
        if (t * groups >= base + 32) {
          base += 32;
          const bool own = base + lane >= w.ahead * groups;
          const int32_t pos = ((base + lane) << p.box_shift) + (own ? w.skip : 0);
          const bool hidden = pos + p.box_rows <= w.from && pos >= p.window.sinks;  // no row sees any: its page may be gone
          row = -1;
          if (base + lane < g_end && pos < (!own && w.prefix > 0 ? w.prefix : w.len) && !hidden) {
            if (p.mode == kModeNorm) {
              row = (static_cast<int64_t>(w.b) * p.N + w.n) * p.cache_seq + pos;
            } else {
              const int32_t pg = p.bs_shift >= 0 ? pos >> p.bs_shift : pos / p.block_size;
              const int32_t in = pos - pg * p.block_size;
              const int32_t* table = !own && w.prefix > 0 ? p.prefix.table : p.table + w.b * p.table_stride;
              const int64_t page = __ldg(table + pg);
              if (page >= 0 && page < p.block_num)
                row = p.mode == kModePa ? page * p.block_size + in : (page * p.N + w.n) * p.block_size + in;
              else if (p.err_count)
                atomicAdd(p.err_count, 1);
            }
          }
        }
        const int st = ring.stage;
        ok = bounded_wait_warp(smem_u32(&ms.empty[st]), ring.parity ^ 1u, p.wait_ns, abort_flag);
        if (!ok) break;
        int32_t at[4];
        uint64_t bits = 0;
        uint32_t live = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          at[i] = -1;
          if (i < groups) {
            at[i] = __shfl_sync(0xffffffffu, static_cast<int32_t>(row), t * groups - base + i);
            const int32_t have = min(p.box_rows, w.template end_of<true>(t, w.len) - (w.template pos<true>(t) + (i << p.box_shift)));
            if (at[i] >= 0) {
              bits |= (~0ull >> (64 - have)) << (i << p.box_shift);
              ++live;
            }
          }
        }
        if (elect_one()) {
          const uint32_t bar = smem_u32(&ms.full[st]), stage = s0 + st * p.stage_bytes;
          ms.valid[u % kValidRing] = bits;
          mbar_arrive_expect_tx(bar, live * group_bytes);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (at[i] < 0) continue;
            uint32_t to = stage + (i << p.box_shift) * v_row;
            for (int32_t c = 0; c < (VQ ? 1 : p.vslabs); ++c, to += kSlab) tma_load_3d(to, &p.tv, bar, 64 * c, head, at[i]);
            to = stage + p.off_staging + (i << p.box_shift) * k_row;
            for (int32_t c = 0; c < (KQ ? 1 : p.kslabs); ++c, to += kSlab) tma_load_3d(to, &p.tk, bar, 64 * c, head, at[i]);
          }
        }
        __syncwarp();
        armed |= 1u << st;
        armed_parity = (armed_parity & ~(1u << st)) | (ring.parity << st);
        ring.next(p.ns);
      }
    }
    // let every copy in flight land before the block leaves
    if (!p.stall_loads)
      for (int i = 0; i < kTokenStages; ++i)
        if (armed & (1u << i)) bounded_drain(smem_u32(&ms.full[i]), (armed_parity >> i) & 1u, kDrainNs);
    __syncwarp();
  } else if (warp < kTokenWarps) {
    set_max_regs_inc<kRegsCompute>();
    // ------------------------------------------------------------ products and softmax
    const int g = lane >> 2, t = lane & 3, quarter = warp & 3, team = warp >> 2;
    const int32_t key_a = 16 * quarter + g;          // and key_a + 8, which swizzles alike: the lane's keys of S^T
    const int32_t k_row = KQ ? p.Dk : 128, v_row = p.Dv;  // bytes of a row of codes (or of a slab's)
    // where the lane's chunks lie in a stage: of codes three of a key, and of four values; of 16-bit rows
    // the two of a slab, and its channels' (ldmatrix)
    uint32_t k_at[KQ ? 3 : 2], v_at[VQ ? 4 : 1];
    if constexpr (KQ) {
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        const int chunk = key_chunk<KQ>(p, c, t);
        k_at[c] = p.off_staging + key_a * k_row + ((p.kslab0 ? chunk ^ (key_a & 7) : chunk) << 4);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 2; ++c) k_at[c] = p.off_staging + key_a * 128 + (((2 * t + c) ^ (key_a & 7)) << 4);
    }
    if constexpr (VQ) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {      // (beyond a short row: channels that nobody has)
        const int key = 16 * quarter + 2 * t + (i & 1) + 8 * (i >> 1);
        v_at[i] = key * v_row + ((v_row == 128 ? g ^ (key & 7) : g) << 4);
      }
    } else {
      const int key = 16 * quarter + (lane & 7) + (lane & 16 ? 8 : 0);
      v_at[0] = key * 128 + (((lane & 8 ? 1 : 0) ^ (key & 7)) << 4);
    }
    int32_t u = 0;
    while (true) {
      ok = ok && bounded_wait_warp(smem_u32(&ms.piece_full[pieces.stage]), pieces.parity, p.wait_ns, abort_flag);
      // together, and only when the last piece's results are read
      if (bar_or(ok ? 0u : 1u)) {
        ok = false;
        break;
      }
      const TokenPiece& w = ms.pieces[pieces.stage];
      if (w.end) break;
      const int32_t n = w.n, ta = w.ta, ahead = w.ahead, skip = w.skip;
      // the rows of another call that this one's join: on their way from here
      float4 prior[NT];
      float4 prior_stats[NT];
      if (p.join.prior.rows && w.whole) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const int2 row = w.row[warp + kTokenWarps * i];
          const int64_t at = static_cast<int64_t>(row.x) * p.heads + row.y;
          prior[i] = *reinterpret_cast<const float4*>(p.join.prior.rows + at * p.Dv + min(4 * lane, p.Dv - 4));
          prior_stats[i] = p.join.prior.stats[at];
        }
      }
      uint32_t qf[NT][24];
      // The lane's rows: 8 nt + 2 t + e.
      float m[NT][2], l[NT][2], sl2[NT][2], lazy[NT][2], neg[NT][2];
      float acc[8][NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 24; ++i) qf[nt][i] = queries[((pieces.stage * NT + nt) * 24 + i) * 32 + lane];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[nt][e] = neg_inf();
          neg[nt][e] = kLift;
          l[nt][e] = 0.f;
          sl2[nt][e] = w.row_scale[8 * nt + 2 * t + e];
          lazy[nt][e] = lazy_slack(kLazy, sl2[nt][e]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.f;
      }

      for (int32_t j = 0; j < n; ++j, ++u, ring.next(p.ns)) {
        if ((j & (kTeams - 1)) != team) continue;
        if (!bounded_wait_warp(smem_u32(&ms.full[ring.stage]), ring.parity, p.wait_ns, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t stage = s0 + ring.stage * p.stage_bytes;
        // ---- S^T
        float s[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[h][nt][e] = 0.f;
        if constexpr (KQ) {
          with_kind(p.kq, [&](auto kind) {
            constexpr int K = decltype(kind)::value;
#pragma unroll
            for (int c = 0; c < 3; ++c) {
              if (64 * c >= p.Dk) break;
              uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
              if (16 * key_chunk<KQ>(p, c, t) < p.Dk) {    // (beyond the row lies another, which may be anything)
                xa = lds_128(stage + k_at[c]);
                xb = lds_128(stage + k_at[c] + 8 * k_row);
              }
              const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint2 a = codes_to_half<K>(wa[i]), b = codes_to_half<K>(wb[i]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_16816<K16>(s[i & 1][nt], a.x, b.x, a.y, b.y, qf[nt][8 * c + 2 * i], qf[nt][8 * c + 2 * i + 1]);
              }
            }
          });
        } else {
#pragma unroll
          for (int c = 0; c < 6; ++c) {
            if (64 * (c >> 1) >= p.Dk) break;
            const uint32_t at = stage + (c >> 1) * kSlab + k_at[c & 1];
            const uint4 a = lds_128(at), b = lds_128(at + 8 * 128);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_16816<K16>(s[0][nt], a.x, b.x, a.y, b.y, qf[nt][4 * c], qf[nt][4 * c + 1]);
              mma_16816<K16>(s[1][nt], a.z, b.z, a.w, b.w, qf[nt][4 * c + 2], qf[nt][4 * c + 3]);
            }
          }
        }
        // ---- what the rows see
        const int32_t pos0 = (ta + j) * kKeys + (ta + j >= ahead ? skip : 0);
        const int32_t shared = ta + j < ahead ? w.prefix : 0;  // of a tile of the prefix: where that ends
        const uint32_t valid = static_cast<uint32_t>(ms.valid[u % kValidRing] >> (16 * quarter)) & 0xFFFFu;
        const bool edge = valid != 0xFFFFu || pos0 + kKeys > (shared > 0 ? shared : w.seen_least) || (w.from_most > pos0 && pos0 + kKeys > p.window.sinks);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[0][nt][e] += s[1][nt][e];
        if (edge) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int32_t key = key_a + 8 * h, pos = pos0 + key;
            const bool there = (valid >> (key & 15)) & 1;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e)
              {
                const int r = 8 * nt + 2 * t + e;
                if (!there || pos >= (shared > 0 ? shared : w.seen[r]) || (pos < w.from[r] && pos >= p.window.sinks)) s[0][nt][2 * h + e] = neg_inf();
              }
          }
        }
        // ---- the running maximum
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) grow |= fmaxf(s[0][nt][e], s[0][nt][2 + e]) > m[nt][e] + lazy[nt][e];
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
              if (top > m[nt][e] + lazy[nt][e]) {
                const float f = ex2((m[nt][e] - top) * sl2[nt][e]);
                m[nt][e] = top;
                neg[nt][e] = fmaf(-top, sl2[nt][e], kLift);
                l[nt][e] *= f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  acc[i][nt][e] *= f;
                  acc[i][nt][2 + e] *= f;
                }
              }
            }
        }
        // ---- P^T
        uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float pr[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) pr[e] = ex2(fmaf(s[0][nt][e], sl2[nt][e & 1], neg[nt][e & 1]));
          l[nt][0] += pr[0] + pr[2];
          l[nt][1] += pr[1] + pr[3];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = pack_half2<!P16>(pr[2 * h], pr[2 * h + 1]);
            hi[nt][h] = transpose_8x8(x);
            if constexpr (PLO) {
              const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&x));
              lo[nt][h] = transpose_8x8(pack_half2<false>(pr[2 * h] - r.x, pr[2 * h + 1] - r.y));
            }
          }
        }
        // ---- value rows that do not exist meet P = 0, but 0 times a stray NaN is NaN
        if (valid != 0xFFFFu) {
          uint8_t* const rows = smem + ring.stage * p.stage_bytes;
          for (int key = lane & 15; key < 16; key += 16) {  // two lanes to a key
            if ((valid >> key) & 1) continue;
            for (int i = lane >> 4; i < (VQ ? v_row / 16 : 8 * p.vslabs); i += 2)
              *reinterpret_cast<uint4*>(rows + (VQ ? (16 * quarter + key) * v_row + i * 16
                                                   : (i >> 3) * kSlab + (16 * quarter + key) * 128 + (i & 7) * 16)) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();       // the next copy into this stage comes behind these
          __syncwarp();
        }
        // ---- O^T
        if constexpr (VQ) {
          const uint4 r0 = lds_128(stage + v_at[0]), r1 = lds_128(stage + v_at[1]), r2 = lds_128(stage + v_at[2]),
                      r3 = lds_128(stage + v_at[3]);
          with_kind(p.vq, [&](auto kind) {
            constexpr int K = decltype(kind)::value;
            const uint32_t x0[4] = {r0.x, r0.y, r0.z, r0.w}, x1[4] = {r1.x, r1.y, r1.z, r1.w};
            const uint32_t x2[4] = {r2.x, r2.y, r2.z, r2.w}, x3[4] = {r3.x, r3.y, r3.z, r3.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t sel = h ? 0x7362u : 0x5140u;
                const uint2 a = codes_to_half<K>(__byte_perm(x0[i], x1[i], sel)), b = codes_to_half<K>(__byte_perm(x2[i], x3[i], sel));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  mma_16816<P16>(acc[2 * i + h][nt], a.x, a.y, b.x, b.y, hi[nt][0], hi[nt][1]);
                  if constexpr (PLO) mma_16816<P16>(acc[2 * i + h][nt], a.x, a.y, b.x, b.y, lo[nt][0], lo[nt][1]);
                }
              }
          });
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (16 * i >= p.Dv) break;
            uint32_t a[4];
            ldmatrix_x4_trans(stage + (i >> 2) * kSlab + (v_at[0] ^ ((i & 3) << 5)), a);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_16816<P16>(acc[i][nt], a[0], a[1], a[2], a[3], hi[nt][0], hi[nt][1]);
              if constexpr (PLO) mma_16816<P16>(acc[i][nt], a[0], a[1], a[2], a[3], lo[nt][0], lo[nt][1]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ms.empty[ring.stage]));
      }

      // ---- the warps' results meet
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], o);
          if (g == 0) ms.stats[warp][8 * nt + 2 * t + e] = make_float2(m[nt][e], l[nt][e]);
        }
      if (bar_or(ok ? 0u : 1u)) {
        ok = false;
        break;
      }
      float* const mine = meet + warp * 8 * NT * kTokenRow;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * nt + 2 * t + e;
          float top = neg_inf();
#pragma unroll
          for (int i = 0; i < kTokenWarps; ++i) top = fmaxf(top, ms.stats[i][r].x);
          // (NaN scores leave m at -inf and the sum NaN)
          const float f = top == neg_inf() ? 1.f : ex2((m[nt][e] - top) * sl2[nt][e]);
          float* const to = mine + r * kTokenRow;
          if constexpr (VQ) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<float4*>(to + 16 * g + 4 * i) =
                  make_float4(acc[2 * i][nt][e] * f, acc[2 * i][nt][2 + e] * f, acc[2 * i + 1][nt][e] * f, acc[2 * i + 1][nt][2 + e] * f);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              to[16 * i + g] = acc[i][nt][e] * f;
              to[16 * i + 8 + g] = acc[i][nt][2 + e] * f;
            }
          }
        }
      bar_softmax();
      // ---- final rows, or the piece's statistics and accumulator: a lane has four channels of a row
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        const int r = warp + kTokenWarps * k, ch = 4 * lane;
        if (r < w.rows) {
          const float scale = w.row_scale[r], off = w.row_const[r];
          float top = neg_inf(), sum = 0.f;
#pragma unroll
          for (int i = 0; i < kTokenWarps; ++i) top = fmaxf(top, ms.stats[i][r].x);
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int i = 0; i < kTokenWarps; ++i) {
            const float2 x = ms.stats[i][r];
            sum = fmaf(x.y, top == neg_inf() ? 1.f : ex2((x.x - top) * scale), sum);
            const float4 v = *reinterpret_cast<const float4*>(meet + (i * 8 * NT + r) * kTokenRow + ch);
            o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
          }
          const float top2 = top == neg_inf() ? neg_inf() : fmaf(top, scale, -kLift);
          const JoinRow row{r, w.row[r].x, w.row[r].y};
          if (w.whole) {
            const float2 share = join_row_end<true>(p.join, row, top2, sum, off, lane == 0, &prior_stats[k]);
            if (ch < p.Dv) join_store<F16, true>(p.join, row, w.kv_head, ch, o, sum, share, &prior[k]);
          } else {
            const int64_t at = static_cast<int64_t>(w.slot) * p.NR + r;
            if (lane == 0) p.join.stats[at] = make_float4(top2, sum, off, 0.f);
            if (ch < p.Dv && n > 0) *reinterpret_cast<float4*>(p.join.parts + at * p.Dv + ch) = o;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ms.piece_empty[pieces.stage]));
      pieces.next(2);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) *p.status = 1;
}

// Codes as boxes of whole rows, swizzled where they have 128 bytes; 16-bit rows as make_map's
bool make_rows_map(CUtensorMap* m, const void* base, const PagedLaunch& L, int32_t width, int32_t quant, int32_t box_rows) {
  if (quant == 0) return make_map(m, base, L, width, 0, box_rows);
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const uint64_t row = static_cast<uint64_t>(width);
  const bool pa = L.mode == kModePa;
  const uint64_t slots = L.mode == kModeNorm ? static_cast<uint64_t>(L.B) * L.cache_seq
                                             : static_cast<uint64_t>(L.block_num) * L.block_size;
  cuuint64_t dims[3] = {row, pa ? static_cast<cuuint64_t>(L.N) : 1, pa ? slots : slots * L.N};
  cuuint64_t strides[2] = {row, pa ? row * L.N : row};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(width), 1, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool F16, bool KQ, bool VQ>
cudaError_t launch_tokens(const Params& p, const Plan& pl, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(paged_tokens_kernel<F16, KQ, VQ, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(paged_tokens_kernel<F16, KQ, VQ, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev);
  }
  const auto kernel = pl.NR == 8 ? paged_tokens_kernel<F16, KQ, VQ, 1> : paged_tokens_kernel<F16, KQ, VQ, 2>;
  kernel<<<pl.G, kTokenThreads, pl.smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return p.whole ? cudaSuccess : launch_join<true>(p.join, F16, pl.G, pl.items, stream);
}

}  // namespace

bool paged_tokens_serves(const PagedLaunch& L) {
  return L.variant == 2 && L.Dkv <= kTokenDk && L.Dv <= kTokenDv && (L.total_q + L.B - 1) / L.B * (L.heads / L.N) <= 16;
}

cudaError_t launch_paged_tokens(const PagedLaunch& L, cudaStream_t stream, const char** why) {
  Plan pl{};
  plan_tokens(L, &pl);
  Params p = row_params(L, pl);
  pl.G = std::min(pl.G, device_sm_count());
  p.q = L.q;
  if (!encode_maps([&] {
        return make_rows_map(&p.tk, L.k_cache, L, L.Dkv, L.kq, p.box_rows) &&
               make_rows_map(&p.tv, L.v_cache, L, L.Dv, L.vq, p.box_rows);
      })) {
    *why = "cuTensorMapEncodeTiled failed or is unavailable";
    return cudaErrorInvalidValue;
  }
  p.vslabs = pl.vslabs;
  p.kslabs = pl.kslabs;
  p.kslab0 = pl.kslab0;
  p.ns = pl.ns;
  p.stage_bytes = pl.stage;
  p.off_staging = pl.off_staging;
  p.off_p = pl.off_p;
  p.off_misc = pl.off_misc;
  p.whole = pl.whole;
  const int which = (L.f16 ? 4 : 0) + (L.kq ? 2 : 0) + (L.vq ? 1 : 0);
  switch (which) {
    case 0: return launch_tokens<false, false, false>(p, pl, stream);
    case 1: return launch_tokens<false, false, true>(p, pl, stream);
    case 2: return launch_tokens<false, true, false>(p, pl, stream);
    case 3: return launch_tokens<false, true, true>(p, pl, stream);
    case 4: return launch_tokens<true, false, false>(p, pl, stream);
    case 5: return launch_tokens<true, false, true>(p, pl, stream);
    case 6: return launch_tokens<true, true, false>(p, pl, stream);
    default: return launch_tokens<true, true, true>(p, pl, stream);
  }
}

}  // namespace ra
