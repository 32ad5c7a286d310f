// Internal interface of the attention kernels (packed_attention.cuh, paged_rows.cuh, paged_tile.cuh)
// and of the cache read (cache_read.cu) for the C-ABI layer.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace ra {

constexpr size_t kAttnHeader = 256;  // workspace: status word + padding, ahead of the partial results
constexpr int64_t kMostPositions = 0x7fffff00;  // of a sequence: tile coordinates stay within 31 bits

struct PackedLaunch {
  const uint16_t *q, *k, *v;   // bf16 or fp16 bit patterns
  uint16_t* out;
  float* lse;                  // [total_q, nq] or null
  const int32_t *cu_q, *cu_k;  // [B + 1] or null (equal lengths)
  int64_t B, total_q, total_k;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;  // token and head strides, in elements
  int32_t nq, nkv, d;
  int32_t causal, f16;
  int64_t window, sinks;       // keys that a query sees: the last `window` up to its own, and the first `sinks`; 0: all
  float scale;
  int32_t* status;
  uint8_t* partials;           // workspace behind the header
  int64_t wait_ns;
  int32_t stall_loads;
};
// Bytes of workspace (header included) of any call with these sizes.
size_t packed_attention_workspace(const PackedLaunch& L);
cudaError_t launch_packed_attention(const PackedLaunch& L, cudaStream_t stream, const char** why);
cudaError_t launch_packed_window(const PackedLaunch& L, cudaStream_t stream, const char** why);  // with a window

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
  int64_t window, sinks;       // as above
  // A shared prefix, in one of two ways.  One call has it ahead of every sequence's own positions
  // (prefix_len and so on), or two calls make one: the first, over the sequences' own positions, leaves its
  // rows in fp32 (rows_out) with their statistics; the second, over the prefix, takes the tokens of all
  // sequences for one's (cu_step: cu_q[0] .. cu_q[cu_step]) and joins its rows with those (prior).
  int32_t cu_step;             // entries of cu_q to a sequence's end: 1 but in the second call
  float* rows_out;             // [total_q, heads, Dv], or null
  float4* stats_out;           // [total_q, heads]: (log2 of the largest weight, the sum of the weights over it, the
                               // lse's share of the key offsets, 0)
  const float* prior;
  const float4* prior_stats;
  int32_t shifts;              // the second call writes the lse: that share is wanted
  const int32_t *prefix_len, *prefix_table;
  int64_t prefix_entries, max_prefix_len;
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
// with a window, rows_out or prior
cudaError_t launch_paged_extended(const PagedLaunch& L, cudaStream_t stream, const char** why);
// Sequences behind a shared prefix, in one call (`behind` it) or in two (their `own` positions, then `over` the
// prefix, whose rows join the own).
cudaError_t launch_paged_prefix(const PagedLaunch& own, const PagedLaunch& over, const PagedLaunch& behind, cudaStream_t stream,
                                const char** why);
// The kernel for many rows per sequence and kv head (paged_tile.cuh): whether it takes the
// call, its part of the workspace, and the launch.
bool paged_tile_serves(const PagedLaunch& L);
size_t paged_tile_workspace(const PagedLaunch& L);
int64_t paged_tile_tokens(const PagedLaunch& L);  // of an item, and the keys of a tile
int paged_tile_keys(const PagedLaunch& L);
cudaError_t launch_paged_tile(const PagedLaunch& L, cudaStream_t stream, const char** why);
cudaError_t launch_paged_tile_extended(const PagedLaunch& L, cudaStream_t stream, const char** why);

// The kernel for up to 16 rows per sequence and kv head of the calls with a window or a prefix
// (paged_tokens.cu).  Its workspace is paged_attention's for the same sizes.
bool paged_tokens_serves(const PagedLaunch& L);
cudaError_t launch_paged_tokens(const PagedLaunch& L, cudaStream_t stream, const char** why);

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
