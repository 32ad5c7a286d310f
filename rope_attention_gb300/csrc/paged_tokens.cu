// Attention of one token or a few over V2 caches: the kernel for up to 16 rows per sequence and kv head
// (a row is a token's head) of the calls with a window or a shared prefix.
//
//   S^T[key, row] = K q^T,  O^T[channel, row] += V^T P^T
//
// Here the work is the reading of the cache: a key of 320 codes meets 8 to 16 rows, 16 to 32 operations
// a byte where the tensor core does some 280 a byte of HBM, so the products go through warp-level MMAs
// on registers, and what counts is a short way from shared memory to the result.
//  * A tile is 64 keys.  Four warps take it, 16 keys each; the other four the next one.  A warp keeps its
//    own maximum, sum and accumulator, so nothing is exchanged before the end of a piece.
//  * M is the keys (then the channels) and N the rows, eight at a time: 8 rows cost half of what 16
//    would in the usual order.  S^T leaves the MMA as P^T's operand up to a transposition of 8 x 8
//    blocks within the warp.
//  * Codes become fp16 in registers.  The contraction's order is free as long as both operands have
//    the same: a lane takes 16 neighbouring channels of its keys for four steps (q is laid out to match), and
//    of the values 16 neighbouring channels of four keys, whose bytes it interleaves.  For that the
//    keys of a block stand in the order kOrder, with which neither load has bank conflicts.
//  * A ninth warp walks the block table and issues TMA boxes of 64 bytes (16-bit values: 128) x 16 to
//    64 keys, four to nine tiles ahead.
// The runs of tiles, their parts and the join are paged_rows.cuh's.  The maximum follows only when a
// tile exceeds it by 2^kLazy.  Every wait on an mbarrier is bounded in time (status word); the warps meet
// at the end of a piece and leave it, or the loop, together.
#include "paged_rows.cuh"

namespace ra {
namespace {

constexpr int kTokenWarps = 8, kTileWarps = 4;
// 16 rows: the warps that compute take registers from a third warpgroup, one warp of which loads
// (2 x 216 + 72 = 3 x 168; with 288 threads ptxas has 168 for each and spills 280 bytes)
__host__ __device__ constexpr int token_threads(int nt) { return nt == 1 ? 32 * (kTokenWarps + 1) : 384; }
constexpr int kRegsCompute = 216, kRegsLoad = 72;
constexpr int kTokenStages = 12;          // at most
constexpr int kBoxSlab = kKeys * 64;      // 64 keys x 64 bytes
constexpr int kTokenRow = 132;            // floats of a row where the warps' results meet
constexpr int kTokenDk = 192, kTokenDv = 128;
// key of place m among 8: lanes m / 4 take two of them with a load of K, lanes m % 4 four with one of V
constexpr uint32_t kOrder = 0x65742130u;

struct TokenMisc {
  uint64_t full[kTokenStages], empty[kTokenStages];
  uint64_t valid[kValidRing];
  RunScan<384> run;
  float2 stats[kTokenWarps][16];          // (max, sum) of each warp's rows
  float row_scale[16], row_const[16];
  int32_t abort;
};

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
// Rows g and g + 8 of the piece's queries as the second operand of S^T: for codes over the key's scales
// and behind a power of two per row (paged_rows.cuh, scale_q), which row_scale undoes.
//   16-bit keys: slab j (32 channels), lane t of a row's four: channels 32 j + 8 t .. + 7, two steps
//   codes:       slab j (64 channels): channels 64 j + 16 t .. + 15, four steps
template <bool F16, bool KQ, int NT>
__device__ __forceinline__ void load_q(const Params& p, const Piece& w, int64_t q_row0, uint32_t (&qf)[NT][24], float (&scale)[NT],
                                       TokenMisc& ms, int warp, int lane) {
  constexpr int kSlabs = KQ ? 3 : 6, kWide = KQ ? 16 : 8;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = g + 8 * nt;
    const bool live = r < w.rows;
    const int32_t tok = p.hblocks > 1 ? 0 : static_cast<int32_t>(static_cast<uint32_t>(r) / static_cast<uint32_t>(p.hb));
    const uint16_t* q = p.q + (q_row0 + static_cast<int64_t>(tok) * p.heads + (r - tok * p.hb)) * p.Dk;
    uint32_t x[24];
#pragma unroll
    for (int j = 0; j < kSlabs; ++j) {
      const int c = j * 4 * kWide + t * kWide;
#pragma unroll
      for (int h = 0; h < kWide / 8; ++h) {
        const uint4 v = live && c + 8 * h < p.Dk ? __ldg(reinterpret_cast<const uint4*>(q + c + 8 * h)) : make_uint4(0, 0, 0, 0);
        const int at = j * kWide / 2 + 4 * h;
        x[at] = v.x, x[at + 1] = v.y, x[at + 2] = v.z, x[at + 3] = v.w;
      }
    }
    if constexpr (!KQ) {
#pragma unroll
      for (int i = 0; i < 24; ++i) qf[nt][i] = x[i];
      scale[nt] = p.sl2;
    } else {
      const float* ks = p.k_scale + static_cast<int64_t>(w.n) * p.Dk;
      const float* ko = p.k_offset ? p.k_offset + static_cast<int64_t>(w.n) * p.Dk : nullptr;
      uint32_t big = 0;         // |q| as bits orders like the value in either type
      float top = 0.f, shift = 0.f;
#pragma unroll
      for (int i = 0; i < 24; ++i) big = __vmaxu2(big, x[i] & 0x7FFF7FFFu);
      big = max(big & 0xFFFFu, big >> 16);
      float inv[48];
#pragma unroll
      for (int j = 0; j < 3; ++j)
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int c = 64 * j + 16 * t + 4 * h;
          const float4 s = c < p.Dk ? __ldg(reinterpret_cast<const float4*>(ks + c)) : make_float4(1.f, 1.f, 1.f, 1.f);
          const float4 o = ko && p.shifts && c < p.Dk ? __ldg(reinterpret_cast<const float4*>(ko + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
          const float s4[4] = {s.x, s.y, s.z, s.w}, o4[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 16 * j + 4 * h + e;
            inv[i] = c < p.Dk ? rcp(s4[e]) : 0.f;
            top = fmaxf(top, fabsf(inv[i]));
            if (p.shifts) shift += half_to_float<F16>((x[i >> 1] >> (16 * (i & 1))) & 0xFFFFu) / s4[e] * o4[e];
          }
        }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        shift += __shfl_xor_sync(0xffffffffu, shift, o);
      }
      const int k = max(-100, min(100, -(scale_exponent(half_to_float<F16>(big)) + scale_exponent(top) + 15)));
      const float up = exp2_int(k);
#pragma unroll
      for (int i = 0; i < 24; ++i)
        qf[nt][i] = pack_f16x2(half_to_float<F16>(x[i] & 0xFFFFu) * (inv[2 * i] * up), half_to_float<F16>(x[i] >> 16) * (inv[2 * i + 1] * up));
      scale[nt] = p.sl2 * exp2_int(-k);
      if (warp == 0 && t == 0) {            // for the end of the piece
        ms.row_scale[r] = scale[nt];
        ms.row_const[r] = -shift * p.scale;
      }
    }
  }
}

// F16: q, out and 16-bit caches are fp16, not bf16.  KQ, VQ: keys, values are codes.  NT: rows / 8.
template <bool F16, bool KQ, bool VQ, int NT>
__global__ void __launch_bounds__(token_threads(NT), 1) paged_tokens_kernel(const __grid_constant__ Params p) {
  constexpr bool K16 = F16 || KQ, P16 = F16 || VQ, PLO = F16 && (KQ || VQ);   // as in paged_rows.cuh
  constexpr float kLift = P16 ? kHalfLift : 0.f;
  constexpr int kVSlab = VQ ? kBoxSlab : kSlab;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* meet = reinterpret_cast<float*>(smem + p.off_p);            // [warp][row][kTokenRow]
  TokenMisc& ms = *reinterpret_cast<TokenMisc*>(smem + p.off_misc);
  const uint32_t s0 = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.ns; ++s) {
      mbar_init(smem_u32(&ms.full[s]), 1);
      mbar_init(smem_u32(&ms.empty[s]), kTileWarps);
    }
    ms.abort = 0;
    fence_mbar_init();
    p.join.meta[8 * blockIdx.x] = 0;      // nothing to join, unless the first piece says so below
  } else if (threadIdx.x == 32 * kTokenWarps) {
    prefetch_tensormap(&p.tk);
    prefetch_tensormap(&p.tv);
  }
  grid_launch_dependents();
  Walker<true> walk;
  int64_t per, start;
  find_run<true, token_threads(NT)>(p, walk, ms.run, per, start);
  __syncthreads();
  start_run(p, walk, ms.run);
  volatile int* abort_flag = &ms.abort;
  Piece w{};
  Ring ring;
  bool ok = true;

  if (warp >= kTokenWarps) {
    if (NT == 2) set_max_regs_dec<kRegsLoad>();
  }
  if (warp == kTokenWarps) {
    // ------------------------------------------------------------ loads
    const int groups = kKeys >> p.box_shift;
    const uint32_t group_bytes = p.box_rows * (p.kslabs * 64 + p.vslabs * (VQ ? 64 : 128));
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
          int32_t pos = (base + lane) << p.box_shift;
          if (base + lane >= p.window.tiles * groups) pos += w.skip;
          const bool hidden = pos + p.box_rows <= w.from && pos >= p.window.sinks;  // no row sees any: its page may be gone
          row = -1;
          if (base + lane < g_end && pos < w.len && !hidden) {
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
            const int32_t have = min(p.box_rows, w.len - (w.template pos<true>(p, t) + (i << p.box_shift)));
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
            uint32_t to = stage + (i << p.box_shift) * (VQ ? 64 : 128);
            for (int32_t c = 0; c < p.vslabs; ++c, to += kVSlab) tma_load_3d(to, &p.tv, bar, 64 * c, head, at[i]);
            to = stage + p.vslabs * kVSlab + (i << p.box_shift) * 64;
            for (int32_t c = 0; c < p.kslabs; ++c, to += kBoxSlab) tma_load_3d(to, &p.tk, bar, (KQ ? 64 : 32) * c, head, at[i]);
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
    if (NT == 2) set_max_regs_inc<kRegsCompute>();
    // ------------------------------------------------------------ products and softmax
    const int g = lane >> 2, t = lane & 3, quarter = warp & 3, tile_half = warp >> 2;
    const int32_t key_a = 16 * quarter + ((kOrder >> (4 * g)) & 7);   // and key_a + 8: the lane's keys of S^T
    // keys of a value operand: two and two more 8 further
    const int32_t key_v0 = 16 * quarter + ((kOrder >> (8 * t)) & 7), key_v1 = 16 * quarter + ((kOrder >> (8 * t + 4)) & 7);
    const int32_t key_m = 16 * quarter + ((kOrder >> (4 * (lane & 7))) & 7) + (lane & 16 ? 8 : 0);  // ldmatrix: the lane's key
    int32_t u = 0, piece = 0;
    for (; ok && walk.next(p, w); ++piece) {
      const int32_t n = w.tb - w.ta;
      const int64_t q_row0 = static_cast<int64_t>(w.q_start + w.tok) * p.heads + w.head;
      if (piece == 0 && threadIdx.x == 0 && w.t0 > 0) {
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
      uint32_t qf[NT][24];
      float q_scale[NT];                    // of row g + 8 nt
      if (n > 0) load_q<F16, KQ, NT>(p, w, q_row0, qf, q_scale, ms, warp, lane);
      // The lane's rows: 8 nt + 2 t + e.  What they see, and the scale of their scores.
      int32_t seen[NT][2], from[NT][2], seen_least = 0x7fffffff, from_most = 0;
      float m[NT][2], l[NT][2], sl2[NT][2], lazy[NT][2];
      float acc[8][NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * nt + 2 * t + e;
          const int32_t tok = p.hblocks > 1 ? 0 : static_cast<int32_t>(static_cast<uint32_t>(min(r, w.rows - 1)) / static_cast<uint32_t>(p.hb));
          const int32_t at = w.len - w.Lq + w.tok + tok;
          seen[nt][e] = p.causal ? min(w.len, max(0, at + 1)) : w.len;
          from[nt][e] = window_from(p.window, at);
          seen_least = min(seen_least, seen[nt][e]);
          from_most = max(from_most, from[nt][e]);
          m[nt][e] = neg_inf();
          l[nt][e] = 0.f;
          sl2[nt][e] = p.sl2;
        }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][nt][e] = 0.f;
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        seen_least = min(seen_least, __shfl_xor_sync(0xffffffffu, seen_least, o));
        from_most = max(from_most, __shfl_xor_sync(0xffffffffu, from_most, o));
      }
      if (KQ && n > 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) sl2[nt][e] = __shfl_sync(0xffffffffu, q_scale[nt], 4 * (2 * t + e));
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) lazy[nt][e] = lazy_slack(kLazy, sl2[nt][e]);

      for (int32_t j = 0; j < n; ++j, ++u, ring.next(p.ns)) {
        if ((j & 1) != tile_half) continue;
        if (!bounded_wait_warp(smem_u32(&ms.full[ring.stage]), ring.parity, p.wait_ns, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t stage = s0 + ring.stage * p.stage_bytes, k_base = stage + p.vslabs * kVSlab;
        // ---- S^T
        float s[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[h][nt][e] = 0.f;
        const uint32_t ka = k_base + key_a * 64 + t * 16;
        if constexpr (KQ) {
          with_kind(p.kq, [&](auto kind) {
            constexpr int K = decltype(kind)::value;
#pragma unroll
            for (int c = 0; c < 3; ++c) {
              if (c >= p.kslabs) break;
              const uint4 xa = lds_128(ka + c * kBoxSlab), xb = lds_128(ka + c * kBoxSlab + 8 * 64);
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
            if (c >= p.kslabs) break;
            const uint4 a = lds_128(ka + c * kBoxSlab), b = lds_128(ka + c * kBoxSlab + 8 * 64);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_16816<K16>(s[0][nt], a.x, b.x, a.y, b.y, qf[nt][4 * c], qf[nt][4 * c + 1]);
              mma_16816<K16>(s[1][nt], a.z, b.z, a.w, b.w, qf[nt][4 * c + 2], qf[nt][4 * c + 3]);
            }
          }
        }
        // ---- what the rows see
        const int32_t pos0 = w.template pos<true>(p, w.ta + j);
        const uint32_t valid = static_cast<uint32_t>(ms.valid[u % kValidRing] >> (16 * quarter)) & 0xFFFFu;
        const bool edge = valid != 0xFFFFu || pos0 + kKeys > seen_least || (from_most > pos0 && pos0 + kKeys > p.window.sinks);
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
                if (!there || pos >= seen[nt][e] || (pos < from[nt][e] && pos >= p.window.sinks)) s[0][nt][2 * h + e] = neg_inf();
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
          for (int e = 0; e < 4; ++e) {
            const float neg = m[nt][e & 1] == neg_inf() ? kLift : fmaf(-m[nt][e & 1], sl2[nt][e & 1], kLift);
            pr[e] = ex2(fmaf(s[0][nt][e], sl2[nt][e & 1], neg));
          }
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
          constexpr int kParts = VQ ? 4 : 8;
          for (int i = lane; i < 16 * kParts; i += 32) {
            const int key = i / kParts;
            if ((valid >> key) & 1) continue;
            for (int c = 0; c < p.vslabs; ++c)
              *reinterpret_cast<uint4*>(smem + ring.stage * p.stage_bytes + c * kVSlab + (16 * quarter + key) * (VQ ? 64 : 128) +
                                        (i % kParts) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();       // the next copy into this stage comes behind these
          __syncwarp();
        }
        // ---- O^T
        if constexpr (VQ) {
          // 16 bytes of a row: chunk g of two slabs of four, swizzled by 64 bytes
          const uint32_t vb = stage + (g >> 2) * kBoxSlab;
          auto row = [&](int32_t key) { return lds_128(vb + key * 64 + (((g & 3) ^ ((key >> 1) & 3)) << 4)); };
          const uint4 r0 = row(key_v0), r1 = row(key_v1), r2 = row(key_v0 + 8), r3 = row(key_v1 + 8);
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
            const int chunk = 2 * (i & 3) + (lane & 8 ? 1 : 0);
            ldmatrix_x4_trans(stage + (i >> 2) * kSlab + key_m * 128 + ((chunk ^ (key_m & 7)) << 4), a);
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
      ok = bar_or(ok ? 0u : 1u) == 0;
      if (!ok) break;
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
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (piece == 0 && w.t0 > 0 ? 0 : 1);
      const bool whole = w.whole();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = 8 * nt + warp, ch = 4 * lane;
        if (r < w.rows) {
          const float scale = KQ && n > 0 ? ms.row_scale[r] : p.sl2, off = KQ && n > 0 ? ms.row_const[r] : 0.f;
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
          const int32_t tok = p.hblocks > 1 ? 0 : static_cast<int32_t>(static_cast<uint32_t>(r) / static_cast<uint32_t>(p.hb));
          JoinRow row;
          row.part = r;
          row.token = w.q_start + w.tok + tok;
          row.head = w.head + r - tok * p.hb;
          if (whole) {
            const float2 share = join_row_end<true>(p.join, row, top2, sum, off, lane == 0);
            if (ch < p.Dv) join_store<F16, true>(p.join, row, w.n, ch, o, sum, share);
          } else {
            if (lane == 0) p.join.stats[slot * p.NR + r] = make_float4(top2, sum, off, 0.f);
            if (ch < p.Dv && n > 0) *reinterpret_cast<float4*>(p.join.parts + (slot * p.NR + r) * p.Dv + ch) = o;
          }
        }
      }
      bar_softmax();                      // stats, scales and results may be written again
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) *p.status = 1;
}

// K as 64-byte boxes without a swizzle; V of codes swizzled by 64 bytes, else like an MMA operand
bool make_box_map(CUtensorMap* m, const void* base, const PagedLaunch& L, int32_t width, int32_t quant, int32_t box_rows, bool swizzle) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const uint64_t row = static_cast<uint64_t>(width) * (quant ? 1 : 2);
  const bool pa = L.mode == kModePa;
  const uint64_t slots = L.mode == kModeNorm ? static_cast<uint64_t>(L.B) * L.cache_seq
                                             : static_cast<uint64_t>(L.block_num) * L.block_size;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), pa ? static_cast<cuuint64_t>(L.N) : 1, pa ? slots : slots * L.N};
  cuuint64_t strides[2] = {row, pa ? row * L.N : row};
  cuuint32_t box[3] = {quant ? 64u : 32u, 1, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, quant ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

void plan_tokens(const PagedLaunch& L, Plan* pl) {
  const int g = L.heads / static_cast<int32_t>(L.N);
  pl->NR = (L.total_q + L.B - 1) / L.B * g <= 8 ? 8 : 16;
  pl->vslabs = (L.Dv + 63) / 64;
  pl->kslabs = (L.Dkv * (L.kq ? 1 : 2) + 63) / 64;
  pl->stage = pl->kslabs * kBoxSlab + pl->vslabs * (L.vq ? kBoxSlab : kSlab);
  const int fixed = kTokenWarps * pl->NR * kTokenRow * 4 + ((static_cast<int>(sizeof(TokenMisc)) + 15) & ~15);
  pl->ns = std::min(kTokenStages, (kSmemMax - fixed) / pl->stage);
  pl->off_p = pl->ns * pl->stage;
  pl->off_misc = pl->off_p + kTokenWarps * pl->NR * kTokenRow * 4;
  pl->smem = pl->off_misc + ((static_cast<int>(sizeof(TokenMisc)) + 15) & ~15);
  share_out(L, pl);
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
  if (pl.NR == 8) paged_tokens_kernel<F16, KQ, VQ, 1><<<pl.G, token_threads(1), pl.smem, stream>>>(p);
  else paged_tokens_kernel<F16, KQ, VQ, 2><<<pl.G, token_threads(2), pl.smem, stream>>>(p);
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
        return make_box_map(&p.tk, L.k_cache, L, L.Dkv, L.kq, p.box_rows, false) &&
               (L.vq ? make_box_map(&p.tv, L.v_cache, L, L.Dv, L.vq, p.box_rows, true) : make_map(&p.tv, L.v_cache, L, L.Dv, 0, p.box_rows));
      })) {
    *why = "cuTensorMapEncodeTiled failed or is unavailable";
    return cudaErrorInvalidValue;
  }
  p.vslabs = pl.vslabs;
  p.kslabs = pl.kslabs;
  p.ns = pl.ns;
  p.stage_bytes = pl.stage;
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
