// Internal interface of the paging kernels (cache_paging.cu) for the C-ABI layer.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace ra {

constexpr int64_t kPagingRequests = 16384;     // of a call: three words of shared memory each
constexpr int64_t kPagingTokens = 1LL << 30;
constexpr int64_t kPagingEntries = 0x7fffff00;   // of a block table: indexes a little behind its end stay within 31 bits

struct PagingLaunch {
  int64_t B, block_num, block_size, table_stride, max_tokens;
  const int32_t* counts;       // extend: new tokens; slots: tokens; truncate: tokens kept, or null (none)
  const int32_t* starts;       // slots: first positions, or null (0)
  const int32_t* seq_lens;     // extend, truncate
  int32_t* table;
  int32_t* free_pages;
  const int32_t* free_count;
  int64_t* index;
  int32_t* cu;
  int32_t *new_lens, *new_free_count;
  int32_t* err_count;
};
cudaError_t launch_cache_extend(const PagingLaunch& L, cudaStream_t stream);
cudaError_t launch_cache_slots(const PagingLaunch& L, cudaStream_t stream);
cudaError_t launch_cache_truncate(const PagingLaunch& L, cudaStream_t stream);

}  // namespace ra
