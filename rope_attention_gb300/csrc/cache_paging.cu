// The paging of the caches: pages from a free list to requests that grow and back, and the slot
// of every token.
//
//   extend:   request b of l_b tokens gets n_b more.  It needs need_b = ceil((l_b + n_b) / bs) -
//             ceil(l_b / bs) pages; those of requests 0 .. b - 1 come before it on the free list
//             (a stack: page i of those taken is the i-th from its top), so a prefix sum of the
//             needs gives every new page its place, and a prefix sum of the n_b every token its
//             row.  slot(b, pos) = table[b, pos / bs] * bs + pos % bs.
//   slots:    the same without pages: positions start_b .. start_b + n_b - 1.
//   truncate: the pages behind the tokens kept go back, in an order that makes extend take
//             them out again as they were.
//
// Every block sums over all requests for itself (they are in L2, a few thousand at most) and then
// takes its share of the tokens, whose request it finds by bisection in shared memory.  extend and
// truncate are one cluster: lengths and the count of free pages may be written where they were
// read, once every block of the cluster has read them, and no second launch is needed.
// Bound by latency: a launch and five dependent loads.
#include <algorithm>

#include "cache_paging.h"
#include "internal.h"

namespace ra {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMostCluster = 8;

struct Params {
  PagingLaunch L;
  int32_t cap;                  // positions that a row of the table has room for
  int32_t bs, shift;            // block size; its log2, or -1
  int32_t per_thread;           // requests
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int32_t page_of(const Params& p, int32_t pos) {
  return p.shift >= 0 ? pos >> p.shift : static_cast<int32_t>(static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.bs));
}
__device__ __forceinline__ int32_t pages_of(const Params& p, int32_t n) {
  return n == 0 ? 0 : page_of(p, n - 1) + 1;
}
// the sum of x over the threads before this one, and over all
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* sums, int64_t& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int64_t mine = sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, mine, o);
    if (lane >= o) mine += up;
  }
  total = __shfl_sync(0xffffffffu, mine, 31);
  const int64_t before = __shfl_sync(0xffffffffu, mine, max(warp - 1, 0));
  __syncthreads();              // sums may be written again
  return (warp > 0 ? before : 0) + incl - x;
}
// the last of n ascending values that is not above t (the first is 0)
__device__ __forceinline__ int32_t last_not_above(const int32_t* v, int32_t n, int32_t t) {
  int32_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (v[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Shared memory: where each request's tokens start, its first position, and its first page among
// those taken (-1: it gets none of what it asks for).
template <bool EXTEND>
__global__ void __launch_bounds__(kThreads, 1) slots_kernel(const __grid_constant__ Params p) {
  extern __shared__ int32_t shared[];
  __shared__ int64_t sums[32];
  const PagingLaunch& L = p.L;
  const int32_t B = static_cast<int32_t>(L.B), tid = threadIdx.x;
  int32_t *cu = shared, *first = shared + B, *pages = shared + 2 * B;
  const int32_t max_tokens = static_cast<int32_t>(L.max_tokens);
  const int32_t b0 = tid * p.per_thread, b1 = min(B, b0 + p.per_thread);
  const int32_t avail = EXTEND ? min(max(*L.free_count, 0), static_cast<int32_t>(L.block_num)) : 0;
  int64_t tokens = 0, total = 0;
  for (int32_t b = b0; b < b1; ++b) {
    const int32_t n = max(L.counts[b], 0);
    int32_t at = EXTEND ? L.seq_lens[b] : L.starts ? L.starts[b] : 0;
    at = EXTEND ? min(max(at, 0), p.cap) : max(at, 0);
    first[b] = at;
    pages[b] = n;
    tokens += n;
  }
  __syncthreads();
  int64_t before = block_scan(tokens, sums, total);
  int64_t need = 0, taken = 0;
  for (int32_t b = b0; b < b1; ++b) {
    const int32_t n = pages[b], at = first[b];
    cu[b] = static_cast<int32_t>(min(before, static_cast<int64_t>(max_tokens)));
    before += n;
    if (EXTEND) {
      const bool fits = n <= p.cap - at && before <= max_tokens;
      pages[b] = fits ? pages_of(p, at + n) - pages_of(p, at) : -1;
      need += max(pages[b], 0);
    }
  }
  int32_t refused = 0;
  if (EXTEND) {
    int64_t all = 0;
    int64_t upto = block_scan(need, sums, all);
    for (int32_t b = b0; b < b1; ++b) {
      const int32_t want = pages[b];
      const bool served = want == 0 || (want > 0 && upto + want <= avail);
      pages[b] = served ? (want == 0 ? 0 : static_cast<int32_t>(upto)) : -1;
      if (want > 0 && served) taken = upto + want;
      upto += max(want, 0);
      // (its tokens' rows: cu[b] is this thread's own)
      if (!served && L.counts[b] > 0) ++refused;
    }
    // requests that get pages come first, so the last one's end is what is taken
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const int64_t other = __shfl_xor_sync(0xffffffffu, taken, o);
      taken = max(taken, other);
      refused += __shfl_xor_sync(0xffffffffu, refused, o);
    }
    if ((tid & 31) == 0) {
      sums[tid >> 5] = taken;
      if (blockIdx.x == 0 && refused > 0 && L.err_count) atomicAdd(L.err_count, refused);
    }
  }
  __syncthreads();

  // ---- tokens
  const int32_t rows = static_cast<int32_t>(min(total, static_cast<int64_t>(max_tokens)));
  int32_t bad = 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + tid; t < max_tokens; t += static_cast<int64_t>(gridDim.x) * kThreads) {
    int64_t slot = -1;
    if (t < rows) {
      const int32_t b = last_not_above(cu, B, static_cast<int32_t>(t));
      const int32_t at = first[b], from = pages[b];
      const int64_t pos = static_cast<int64_t>(at) + t - cu[b];
      if (pos < p.cap && (!EXTEND || from >= 0)) {
        const int32_t pg = page_of(p, static_cast<int32_t>(pos)), in = static_cast<int32_t>(pos) - pg * p.bs;
        int32_t page;
        const int32_t have = EXTEND ? pages_of(p, at) : 0x7fffffff;
        if (pg < have) {
          page = L.table[b * L.table_stride + pg];
        } else {
          page = L.free_pages[avail - 1 - (from + pg - have)];
          if (in == 0) L.table[b * L.table_stride + pg] = page;
        }
        if (page >= 0 && page < L.block_num) slot = static_cast<int64_t>(page) * p.bs + in;
        else ++bad;
      } else if (!EXTEND) {
        ++bad;
      }
    }
    L.index[t] = slot;
  }
  if (bad > 0 && L.err_count) atomicAdd(L.err_count, bad);
  if (EXTEND) cluster_barrier();            // every block has read lengths and count
  if (blockIdx.x != 0) return;
  for (int32_t b = tid; b < B; b += kThreads) {
    L.cu[b] = cu[b];
    if (EXTEND) L.new_lens[b] = first[b] + (pages[b] >= 0 ? max(L.counts[b], 0) : 0);
  }
  if (tid == 0) {
    L.cu[B] = rows;
    if (EXTEND) {
      int64_t most = 0;
      for (int w = 0; w < kWarps; ++w) most = max(most, sums[w]);
      *L.new_free_count = avail - static_cast<int32_t>(most);
    }
  }
}

// Shared memory: where each request's pages start among those looked at, and its first such page.
__global__ void __launch_bounds__(kThreads, 1) truncate_kernel(const __grid_constant__ Params p) {
  extern __shared__ int32_t shared[];
  __shared__ int64_t sums[32];
  __shared__ int32_t counts[kMostCluster];  // valid pages of each block's share
  const PagingLaunch& L = p.L;
  const int32_t B = static_cast<int32_t>(L.B), tid = threadIdx.x;
  int32_t *cu = shared, *first = shared + B, *kept = shared + 2 * B;
  const int32_t b0 = tid * p.per_thread, b1 = min(B, b0 + p.per_thread);
  // (a block's shared memory is written to only when it has started)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const int32_t block_num = static_cast<int32_t>(L.block_num), count = min(max(*L.free_count, 0), block_num);
  int64_t looked = 0, total = 0;
  for (int32_t b = b0; b < b1; ++b) {
    const int32_t len = min(max(L.seq_lens[b], 0), p.cap), keep = L.counts ? min(max(L.counts[b], 0), len) : 0;
    kept[b] = keep;
    first[b] = pages_of(p, keep);
    cu[b] = pages_of(p, len) - first[b];
    looked += cu[b];
  }
  __syncthreads();
  int64_t before = block_scan(looked, sums, total);
  for (int32_t b = b0; b < b1; ++b) {
    const int32_t n = cu[b];
    cu[b] = static_cast<int32_t>(before);   // B * table_stride < 2^31
    before += n;
  }
  __syncthreads();
  const int64_t share = (total + gridDim.x - 1) / gridDim.x;
  const int64_t lo = min(total, share * blockIdx.x), hi = min(total, lo + share);
  auto page_at = [&](int64_t i) {
    const int32_t b = last_not_above(cu, B, static_cast<int32_t>(i));
    return L.table[b * L.table_stride + first[b] + static_cast<int32_t>(i) - cu[b]];
  };
  int32_t valid = 0;
  for (int64_t i = lo + tid; i < hi; i += kThreads) {
    const int32_t page = page_at(i);
    valid += page >= 0 && page < block_num;
  }
  int64_t mine = 0;
  block_scan(valid, sums, mine);
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (tid < gridDim.x) {        // to every block of the cluster
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(to)
                 : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(&counts[blockIdx.x]))), "r"(tid));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(static_cast<int32_t>(mine)) : "memory");
  }
  cluster_barrier();            // and every block has read lengths and count
  int32_t at = 0, all = 0;
  for (uint32_t c = 0; c < gridDim.x; ++c) {
    if (c < blockIdx.x) at += counts[c];
    all += counts[c];
  }
  const int32_t room = min(all, block_num - count);  // more than the cache has would be some twice
  for (int64_t i0 = lo; i0 < hi; i0 += kThreads) {
    const int32_t page = i0 + tid < hi ? page_at(i0 + tid) : -1;
    const bool good = page >= 0 && page < block_num;
    int64_t here = 0;
    const int32_t i = at + static_cast<int32_t>(block_scan(good ? 1 : 0, sums, here));
    if (good && i < room) L.free_pages[count + room - 1 - i] = page;
    at += static_cast<int32_t>(here);
  }
  if (blockIdx.x != 0) return;
  for (int32_t b = tid; b < B; b += kThreads) L.new_lens[b] = kept[b];
  if (tid == 0) {
    *L.new_free_count = count + room;
    if (total > room && L.err_count) atomicAdd(L.err_count, static_cast<int32_t>(total) - room);
  }
}

Params make_params(const PagingLaunch& L) {
  Params p{};
  p.L = L;
  p.cap = static_cast<int32_t>(std::min<int64_t>(0x7fffff00, L.table_stride * L.block_size));
  p.bs = static_cast<int32_t>(L.block_size);
  p.shift = -1;
  for (int s = 0; s < 31; ++s)
    if ((int64_t(1) << s) == L.block_size) p.shift = s;
  p.per_thread = static_cast<int32_t>((L.B + kThreads - 1) / kThreads);
  return p;
}

cudaError_t launch(void (*kernel)(Params), const Params& p, int64_t blocks, bool cluster, cudaStream_t stream) {
  const int smem = static_cast<int>(p.L.B) * 12;
  cudaError_t e = cudaSuccess;
  if (smem > 40 << 10) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {static_cast<unsigned>(blocks), 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = cluster ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// blocks of a cluster for so many tokens or pages: 1, 2, 4 or 8
int64_t cluster_for(int64_t n) {
  int64_t c = 1;
  while (c < kMostCluster && c * kThreads * 2 < n) c *= 2;
  return c;
}

}  // namespace

cudaError_t launch_cache_extend(const PagingLaunch& L, cudaStream_t stream) {
  return launch(slots_kernel<true>, make_params(L), cluster_for(L.max_tokens), true, stream);
}
cudaError_t launch_cache_slots(const PagingLaunch& L, cudaStream_t stream) {
  const int64_t blocks = std::min<int64_t>(device_sm_count(), (L.max_tokens + kThreads - 1) / kThreads);
  return launch(slots_kernel<false>, make_params(L), blocks, false, stream);
}
cudaError_t launch_cache_truncate(const PagingLaunch& L, cudaStream_t stream) {
  return launch(truncate_kernel, make_params(L), cluster_for(std::min(L.block_num, L.B * L.table_stride)), true, stream);
}

}  // namespace ra
