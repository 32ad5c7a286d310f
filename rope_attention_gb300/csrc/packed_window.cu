// packed_window_attention: packed_attention.cuh's kernel over the keys of a window and the sinks.
#include "packed_attention.cuh"

namespace ra {

cudaError_t launch_packed_window(const PackedLaunch& L, cudaStream_t stream, const char** why) {
  return launch_packed<true>(L, stream, why);
}

}  // namespace ra
