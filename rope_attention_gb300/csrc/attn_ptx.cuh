// Inline-PTX helpers of the attention kernels (sm_103a): one-CTA tcgen05 MMAs on 16-bit
// operands, TMEM loads and stores and TMA tile loads, each written from the PTX
// ISA, and the bounded waits' bookkeeping that those kernels share.
#pragma once

#include "ptx.cuh"

namespace ra {

// one probe of an mbarrier's phase, without the suspension try_wait may take
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// ---------------------------------------------------------------- TMEM (one CTA)
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 lanes x 32 (16) columns of 32 bits: lane i of the warp holds its TMEM lane's columns
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32],"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16],"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}

// ---------------------------------------------------------------- MMA (kind::f16, fp32 accumulators)
// Instruction descriptor: D fp32 (1 in bits [4,6)), A and B type in bits [7,10) / [10,13)
// (0 fp16, 1 bf16: the same for both), transpose A / B (MN-major) in bits 15 / 16, N >> 3
// in [17,23), M >> 4 in [24,29).
__host__ __device__ constexpr uint32_t idesc_f16(bool bf16, bool a_mn, bool b_mn, uint32_t m, uint32_t n) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// true in one lane, always the same one.  The whole warp must be there; operands computed
// inside the branch it guards stay in uniform registers, where the MMA takes them from.
// (Measured: M = 128, N = 64 MMAs in a loop go out every 50 cycles, the tensor core's own
// rate; behind a comparison of the thread index every 74, and one by one every 170-200.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
// `steps` (1..4) consecutive K = 16 steps of D[tmem] (+)= A[smem] B[smem], the descriptors
// SA and SB further in 16-byte units at each step; `acc` 0 starts D anew.
template <int SA, int SB>
__device__ __forceinline__ void mma4_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc,
                                            uint32_t steps) {
  asm volatile(
      "{\n\t.reg .pred p0, p1, p2, p3, on;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.b32 p0, %4, 0;\n\tsetp.gt.u32 p1, %5, 1;\n\tsetp.gt.u32 p2, %5, 2;\n\tsetp.gt.u32 p3, %5, 3;\n\t"
      "setp.eq.b32 on, 0, 0;\n\t"
      "add.s64 a1, %1, %6;\n\tadd.s64 b1, %2, %7;\n\t"
      "add.s64 a2, %1, %8;\n\tadd.s64 b2, %2, %9;\n\t"
      "add.s64 a3, %1, %10;\n\tadd.s64 b3, %2, %11;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p0;\n\t"
      "@p1 tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, on;\n\t"
      "@p2 tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, on;\n\t"
      "@p3 tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, on;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(steps), "n"(SA), "n"(SB), "n"(2 * SA), "n"(2 * SB), "n"(3 * SA),
      "n"(3 * SB)
      : "memory");
}
// arrive on the mbarrier once every tcgen05 operation this thread issued so far has completed
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// MN-major operand in 128-byte swizzled rows: each row holds 64 elements of the M (or N)
// axis for one k; 8-row atoms (1024 bytes) follow one another along k, and the next 64
// elements of the M (N) axis start `mn_stride` bytes on.
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t saddr, uint32_t mn_stride) {
  return sdesc(saddr, mn_stride, 1024, kLayoutSwizzle128B);
}

// ---------------------------------------------------------------- loads
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, uint32_t bar, int32_t x, int32_t y,
                                            int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// 32 bytes, one whole sector: a thread that owns a row writes it without half-written sectors
__device__ __forceinline__ void store_32(void* dst, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// ---------------------------------------------------------------- kernels that follow one another
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// until the kernel before has ended and its writes are visible
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---------------------------------------------------------------- registers
// every warp of the warpgroup; the shares of a block add up to what it was launched with
template <int N>
__device__ __forceinline__ void set_max_regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_max_regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---------------------------------------------------------------- arithmetic
// 2^x, flushing subnormal results: the probabilities they stand for are below 2^-126
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// log2 of what fp16 probabilities are held with.  The largest is 2^0 to 2^8 (the maximum follows
// only when a tile exceeds it by that), fp16 ends at 2^16 and its least number is 2^-24: without
// the factor a key 2^-25 below a row's largest left the weighted sum, but not the sum of weights
// (300 keys 2^-25.2 below one sink: all of their share lost), with it one 2^-32 below.
constexpr float kHalfLift = 7.f;
template <bool BF16>
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  if constexpr (BF16) return pack_bf16x2(lo, hi);
  else return pack_f16x2(lo, hi);
}
// 32 probabilities 2^(s scale + neg): their pairs rounded to 16 bits in w, their fp32 sums in
// acc.  All the exponentials of a batch go out before the first result is used: a warp
// issues in order, and with each used at once 64 elements took 827 cycles (one warp per
// scheduler; 882 for two), against 353 (615) in batches of 32, near the rate of the
// exponential unit (8 lanes a cycle: 256, 512).
// LO (fp16): what the rounding left, rounded itself, in lo.
template <bool BF16, bool LO = false>
__device__ __forceinline__ void exp_batch(const uint32_t* s, float2 scale, float2 neg, float2 (&acc)[4], uint32_t* w,
                                          uint32_t* lo = nullptr) {
  static_assert(!(BF16 && LO), "");
  float2 t[16];
#pragma unroll
  for (int i = 0; i < 16; ++i)
    t[i] = __ffma2_rn(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), scale, neg);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    t[i].x = ex2(t[i].x);
    t[i].y = ex2(t[i].y);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    acc[i & 3] = __fadd2_rn(acc[i & 3], t[i]);
    if constexpr (BF16)
      asm volatile("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(t[i].y), "f"(t[i].x));
    else
      asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(t[i].y), "f"(t[i].x));
    if constexpr (LO) {
      const float2 rest = __ffma2_rn(__half22float2(*reinterpret_cast<const __half2*>(&w[i])), make_float2(-1.f, -1.f), t[i]);
      asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo[i]) : "f"(rest.y), "f"(rest.x));
    }
  }
}
// How far a row's scores may pass its maximum before that follows, from log2 to scores of that
// scale; finite, so that a first score passes -inf + slack whatever the scale.
__device__ __forceinline__ float lazy_slack(float log2, float scale) { return fminf(log2 / scale, 3e38f); }
__device__ __forceinline__ float neg_inf() { return __int_as_float(static_cast<int>(0xff800000u)); }

}  // namespace ra
