// packed_attention: its workspace, and packed_attention.cuh's kernel over every key.
#include "packed_attention.cuh"

namespace ra {

size_t packed_attention_workspace(const PackedLaunch& L) { return kAttnHeader + join_bytes(most_blocks(L), 2 * kTileRows, L.d); }

cudaError_t launch_packed_attention(const PackedLaunch& L, cudaStream_t stream, const char** why) {
  return launch_packed<false>(L, stream, why);
}

}  // namespace ra
