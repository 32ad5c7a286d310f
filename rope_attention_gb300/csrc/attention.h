// Internal interface of the attention kernels (packed_attention.cu, paged_attention.cu)
// and of the cache read (cache_read.cu) for the C-ABI layer.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace ra {

constexpr size_t kAttnHeader = 256;  // workspace: status word + padding, ahead of the partial results

struct PackedLaunch {
  const uint16_t *q, *k, *v;   // bf16 or fp16 bit patterns
  uint16_t* out;
  float* lse;                  // [total_q, nq] or null
  const int32_t *cu_q, *cu_k;  // [B + 1] or null (equal lengths)
  int64_t B, total_q, total_k;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;  // token and head strides, in elements
  int32_t nq, nkv, d;
  int32_t causal, f16;
  float scale;
  int32_t* status;
  uint8_t* partials;           // workspace behind the header
  int64_t wait_ns;
  int32_t stall_loads;
};
// Bytes of workspace (header included) of any call with these sizes.
size_t packed_attention_workspace(const PackedLaunch& L);
cudaError_t launch_packed_attention(const PackedLaunch& L, cudaStream_t stream, const char** why);

struct PagedLaunch {
  const uint16_t* q;           // [total_q, heads, Dk] bf16 or fp16 bit patterns
  uint16_t* out;               // [total_q, heads, Dv]
  float* lse;                  // [total_q, heads] or null
  const void *k_cache, *v_cache;
  const float *k_scale, *k_offset, *v_scale, *v_offset;
  const int32_t *cu_q, *seq_lens, *table;
  int32_t* err_count;
  int64_t B, total_q, N, block_num, block_size, table_stride, cache_seq;
  int32_t heads, Dkv, Dv, R, variant, mode;
  int32_t f16, kq, vq;         // 16-bit type; KvQuant of the two caches
  int32_t k_scalar, v_scalar;
  int32_t causal;
  float scale;
  int64_t max_seq_len;
  int32_t* status;
  uint8_t* partials;           // workspace behind the header
  int64_t wait_ns;
  int32_t stall_loads;
};
// Bytes of workspace (header included) of any call with these sizes.
size_t paged_attention_workspace(const PagedLaunch& L);
cudaError_t launch_paged_attention(const PagedLaunch& L, cudaStream_t stream, const char** why);
// The kernel for many rows per sequence and kv head (paged_tile.cu): whether it takes the
// call, its part of the workspace, and the launch.
bool paged_tile_serves(const PagedLaunch& L);
size_t paged_tile_workspace(const PagedLaunch& L);
cudaError_t launch_paged_tile(const PagedLaunch& L, cudaStream_t stream, const char** why);

struct ReadLaunch {
  const int64_t* index;
  const void *k_cache, *v_cache;
  const float *k_scale, *k_offset, *v_scale, *v_offset;
  uint16_t *k_out, *v_out;     // [B, N, S, k_w], [B, N, S, v_w]
  int32_t* err_count;
  int64_t B, N, S, block_num, block_size, cache_seq;
  int32_t kw, vw, mode, f16, kq, vq, k_scalar, v_scalar, variant;
};
cudaError_t launch_cache_read(const ReadLaunch& L, cudaStream_t stream);

}  // namespace ra
