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
// read, once every block of the cluster has read them, and no second launch is needed.  An extend by
// more tokens than a cluster writes as fast as all SMs is two launches: the tokens, then the state.
// Bound by latency: a launch, three dependent loads and a scan.  Measured: 256 requests and a token each
// 5.1 to 6.2 us; 33000 tokens for 16 requests 8.5 to 9.7 (12.3 with four blocks; sixteen are no faster); 18700 pages of
// 300 requests back 8.2, 3000 requests of up to 9000 tokens in pages of 16 99.
#include <algorithm>

#include "cache_paging.h"
#include "internal.h"

namespace ra {
namespace {

constexpr int kMostThreads = 1024;
constexpr int kMostCluster = 8;

struct Params {
  PagingLaunch L;
  int32_t cap;                  // positions that a row of the table has room for
  int32_t bs, shift;            // block size; its log2, or -1
  int32_t per_thread;           // requests
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ int32_t page_of(const Params& p, int32_t pos) {
  return p.shift >= 0 ? pos >> p.shift : static_cast<int32_t>(static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.bs));
}
__device__ __forceinline__ int32_t pages_of(const Params& p, int32_t n) {
  return n == 0 ? 0 : page_of(p, n - 1) + 1;
}
// the sums of x and y over the threads before this one, and over all; `sums` is written
struct Sums {
  int64_t x[32];
  int32_t y[32];
};
__device__ __forceinline__ void block_scan(int64_t& x, int32_t& y, Sums& sums, int64_t& all_x, int32_t& all_y) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t in_x = x;
  int32_t in_y = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up_x = __shfl_up_sync(0xffffffffu, in_x, o);
    const int32_t up_y = __shfl_up_sync(0xffffffffu, in_y, o);
    if (lane >= o) in_x += up_x, in_y += up_y;
  }
  if (lane == 31) sums.x[warp] = in_x, sums.y[warp] = in_y;
  __syncthreads();
  const bool there = lane < static_cast<int>(blockDim.x >> 5);
  int64_t wx = there ? sums.x[lane] : 0;
  int32_t wy = there ? sums.y[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up_x = __shfl_up_sync(0xffffffffu, wx, o);
    const int32_t up_y = __shfl_up_sync(0xffffffffu, wy, o);
    if (lane >= o) wx += up_x, wy += up_y;
  }
  all_x = __shfl_sync(0xffffffffu, wx, 31);
  all_y = __shfl_sync(0xffffffffu, wy, 31);
  const int64_t before_x = __shfl_sync(0xffffffffu, wx, max(warp - 1, 0));
  const int32_t before_y = __shfl_sync(0xffffffffu, wy, max(warp - 1, 0));
  x = (warp > 0 ? before_x : 0) + in_x - x;
  y = (warp > 0 ? before_y : 0) + in_y - y;
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
// AT_ONCE: tokens of a thread whose loads are on their way together, 1 where no thread has more.
// PART: both in one cluster; or the tokens by any number of blocks, and the lengths and the count by one.
enum SlotsPart { kBoth, kTokens, kState };
template <bool EXTEND, int AT_ONCE, SlotsPart PART>
__global__ void __launch_bounds__(kMostThreads, 1) slots_kernel(const __grid_constant__ Params p) {
  extern __shared__ int32_t shared[];
  __shared__ Sums sums;
  __shared__ int32_t most_taken;
  const PagingLaunch& L = p.L;
  const int32_t B = static_cast<int32_t>(L.B), tid = threadIdx.x, threads = blockDim.x;
  int32_t *cu = shared, *first = shared + B, *pages = shared + 2 * B;
  const int32_t max_tokens = static_cast<int32_t>(L.max_tokens);
  const int32_t b0 = tid * p.per_thread, b1 = min(B, b0 + p.per_thread);
  const int32_t avail = EXTEND ? min(max(*L.free_count, 0), static_cast<int32_t>(L.block_num)) : 0;
  if (tid == 0) most_taken = 0;
  // A request that fits into its row needs pages.  (One whose tokens pass max_tokens gets none, but so
  // do all behind it that have tokens: their needs may be counted.)
  int64_t before = 0, total = 0;
  int32_t need = 0, all = 0;
  for (int32_t b = b0; b < b1; ++b) {
    const int32_t n = max(L.counts[b], 0);
    int32_t at = EXTEND ? L.seq_lens[b] : L.starts ? L.starts[b] : 0;
    at = EXTEND ? min(max(at, 0), p.cap) : max(at, 0);
    first[b] = at;
    pages[b] = n;
    before += n;
    if (EXTEND && n <= p.cap - at) need += pages_of(p, at + n) - pages_of(p, at);
  }
  __syncwarp();
  if (EXTEND && PART == kBoth) cluster_arrive();  // this block has read lengths and count
  block_scan(before, need, sums, total, all);
  int32_t refused = 0;
  for (int32_t b = b0; b < b1; ++b) {
    const int32_t n = pages[b], at = first[b];
    cu[b] = static_cast<int32_t>(min(before, static_cast<int64_t>(max_tokens)));
    before += n;
    if (EXTEND) {
      const bool in_row = n <= p.cap - at;
      const int32_t want = in_row ? pages_of(p, at + n) - pages_of(p, at) : 0;
      const bool served = in_row && before <= max_tokens && (want == 0 || need + want <= avail);
      pages[b] = served ? (want == 0 ? 0 : need) : -1;
      need += want;
      // requests that get pages come first, so the last one's end is what is taken
      if (served && want > 0) atomicMax(&most_taken, need);
      if (!served && n > 0) ++refused;
    }
  }
  if (EXTEND && PART != kState && blockIdx.x == 0 && refused > 0 && L.err_count) atomicAdd(L.err_count, refused);
  __syncthreads();

  // ---- tokens
  const int32_t rows = static_cast<int32_t>(min(total, static_cast<int64_t>(max_tokens)));
  int32_t bad = 0;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * threads;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * threads + tid; PART != kState && t0 < max_tokens; t0 += AT_ONCE * stride) {
    // where each token's page stands: in the table, or on the free list (and then in the table as well)
    const int32_t* from[AT_ONCE];
    int32_t* to[AT_ONCE];
    int32_t in[AT_ONCE], page[AT_ONCE];
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const int64_t t = t0 + k * stride;
      from[k] = nullptr;
      to[k] = nullptr;
      in[k] = 0;
      if (t >= rows) continue;
      const int32_t b = last_not_above(cu, B, static_cast<int32_t>(t));
      const int32_t at = first[b], taken = pages[b];
      const int64_t pos = static_cast<int64_t>(at) + t - cu[b];
      if (pos < p.cap && (!EXTEND || taken >= 0)) {
        const int32_t pg = page_of(p, static_cast<int32_t>(pos));
        const int32_t have = EXTEND ? pages_of(p, at) : 0x7fffffff;
        in[k] = static_cast<int32_t>(pos) - pg * p.bs;
        int32_t* const entry = L.table + b * L.table_stride + pg;
        from[k] = pg < have ? entry : L.free_pages + (avail - 1 - (taken + pg - have));
        if (pg >= have && in[k] == 0) to[k] = entry;
      } else if (!EXTEND) {
        ++bad;
      }
    }
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) page[k] = from[k] ? *from[k] : -1;
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const int64_t t = t0 + k * stride;
      if (t >= max_tokens) break;
      const bool good = page[k] >= 0 && page[k] < L.block_num;
      if (from[k] && !good) ++bad;
      if (EXTEND && to[k]) *to[k] = page[k];
      L.index[t] = good ? static_cast<int64_t>(page[k]) * p.bs + in[k] : -1;
    }
  }
  if (bad > 0 && L.err_count) atomicAdd(L.err_count, bad);
  __syncwarp();                             // (lanes leave the loop after different turns; the wait is the warp's)
  if (EXTEND && PART == kBoth) cluster_wait();  // every block has read lengths and count
  if (blockIdx.x != 0) return;
  for (int32_t b = tid; b < B; b += threads) {
    if (PART != kState) L.cu[b] = cu[b];
    if (EXTEND && PART != kTokens) {
      // (a request's tokens, of which pages[b] says whether it gets them: what its successor starts behind)
      const int32_t n = (b + 1 < B ? cu[b + 1] : rows) - cu[b];
      L.new_lens[b] = first[b] + (pages[b] >= 0 ? n : 0);
    }
  }
  if (tid == 0) {
    if (PART != kState) L.cu[B] = rows;
    if (EXTEND && PART != kTokens) *L.new_free_count = avail - most_taken;
  }
}

// Shared memory: where each request's pages start among those looked at, and its first such page.
__global__ void __launch_bounds__(kMostThreads, 1) truncate_kernel(const __grid_constant__ Params p) {
  extern __shared__ int32_t shared[];
  __shared__ Sums sums, sums2;
  __shared__ int32_t counts[kMostCluster];  // valid pages of each block's share
  const PagingLaunch& L = p.L;
  const int32_t B = static_cast<int32_t>(L.B), tid = threadIdx.x, threads = blockDim.x;
  int32_t *cu = shared, *first = shared + B, *kept = shared + 2 * B;
  const int32_t b0 = tid * p.per_thread, b1 = min(B, b0 + p.per_thread);
  // (a block's shared memory is written to only when it has started)
  cluster_arrive();
  const int32_t block_num = static_cast<int32_t>(L.block_num), count = min(max(*L.free_count, 0), block_num);
  int64_t unused = 0, unused_all = 0;
  int32_t before = 0, total = 0;            // B * table_stride < 2^31
  for (int32_t b = b0; b < b1; ++b) {
    const int32_t len = min(max(L.seq_lens[b], 0), p.cap), keep = L.counts ? min(max(L.counts[b], 0), len) : 0;
    kept[b] = keep;
    first[b] = pages_of(p, keep);
    cu[b] = pages_of(p, len) - first[b];
    before += cu[b];
  }
  block_scan(unused, before, sums, unused_all, total);
  for (int32_t b = b0; b < b1; ++b) {
    const int32_t n = cu[b];
    cu[b] = before;
    before += n;
  }
  __syncthreads();
  // a thread's share of the pages, in order
  const int32_t each = static_cast<int32_t>((static_cast<int64_t>(total) + gridDim.x * threads - 1) / (gridDim.x * threads));
  const int64_t lo64 = (static_cast<int64_t>(blockIdx.x) * threads + tid) * each;
  const int32_t lo = static_cast<int32_t>(min(lo64, static_cast<int64_t>(total))), hi = static_cast<int32_t>(min(lo64 + each, static_cast<int64_t>(total)));
  int32_t b = lo < hi ? last_not_above(cu, B, lo) : 0;
  const int32_t b_lo = b;
  auto page_at = [&](int32_t i) {           // i and the request ascend
    while (b + 1 < B && cu[b + 1] <= i) ++b;
    return L.table[b * L.table_stride + first[b] + i - cu[b]];
  };
  constexpr int kHeld = 8;                  // pages that a thread keeps, so that they are looked up once
  int32_t held[kHeld], valid = 0;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) held[k] = lo + k < hi ? page_at(lo + k) : -1;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) valid += held[k] >= 0 && held[k] < block_num;
  for (int32_t i = lo + kHeld; i < hi; ++i) {
    const int32_t page = page_at(i);
    valid += page >= 0 && page < block_num;
  }
  int32_t at = valid, mine = 0;
  block_scan(unused, at, sums2, unused_all, mine);
  cluster_wait();
  if (tid < gridDim.x) {                    // to every block of the cluster
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(to)
                 : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(&counts[blockIdx.x]))), "r"(tid));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(mine) : "memory");
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();                           // and every block has read lengths and count
  int32_t all = 0;
  for (uint32_t c = 0; c < gridDim.x; ++c) {
    if (c < blockIdx.x) at += counts[c];
    all += counts[c];
  }
  const int32_t room = min(all, block_num - count);  // more than the cache has would be some twice
  auto put = [&](int32_t page) {
    if (page < 0 || page >= block_num) return;
    if (at < room) L.free_pages[count + room - 1 - at] = page;
    ++at;
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k) put(held[k]);
  b = b_lo;
  for (int32_t i = lo + kHeld; i < hi; ++i) put(page_at(i));
  if (blockIdx.x != 0) return;
  for (int32_t i = tid; i < B; i += threads) L.new_lens[i] = kept[i];
  if (tid == 0) {
    *L.new_free_count = count + room;
    if (total > room && L.err_count) atomicAdd(L.err_count, total - room);
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
  return p;
}

template <auto KERNEL>
cudaError_t launch(Params p, int64_t blocks, int threads, bool cluster, cudaStream_t stream) {
  const int smem = static_cast<int>(p.L.B) * 12;
  p.per_thread = static_cast<int32_t>((p.L.B + threads - 1) / threads);
  cudaError_t e = cudaSuccess;
  if (smem > 40 << 10) e = allow_all_shared_memory<KERNEL>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {static_cast<unsigned>(blocks), 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = cluster && blocks > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, KERNEL, p);
}

// threads of a block for so many items of its own and so many requests: fewer warps meet sooner
int threads_for(int64_t n, int64_t B) {
  const int64_t most = std::max(n, B);
  return most <= 256 ? 256 : most <= 512 ? 512 : kMostThreads;
}
// blocks of a cluster for so many tokens or pages: 1, 2, 4 or 8
int64_t cluster_for(int64_t n) {
  int64_t c = 1;
  while (c < kMostCluster && c * kMostThreads < n) c *= 2;
  return c;
}

}  // namespace

cudaError_t launch_cache_extend(const PagingLaunch& L, cudaStream_t stream) {
  // (a cluster writes 1 us more for each 8000 tokens; the second launch takes 3)
  constexpr int64_t kOneCluster = 1 << 16;
  const Params p = make_params(L);
  if (L.max_tokens > kOneCluster) {
    const cudaError_t e = launch<slots_kernel<true, 4, kTokens>>(p, device_sm_count(), kMostThreads, false, stream);
    return e != cudaSuccess ? e : launch<slots_kernel<true, 1, kState>>(p, 1, threads_for(1, L.B), false, stream);
  }
  const int64_t c = cluster_for(L.max_tokens);
  const int threads = threads_for((L.max_tokens + c - 1) / c, L.B);
  return c * threads >= L.max_tokens ? launch<slots_kernel<true, 1, kBoth>>(p, c, threads, true, stream)
                                     : launch<slots_kernel<true, 4, kBoth>>(p, c, threads, true, stream);
}
cudaError_t launch_cache_slots(const PagingLaunch& L, cudaStream_t stream) {
  const int threads = threads_for(L.max_tokens, L.B);
  const int64_t blocks = std::min<int64_t>(device_sm_count(), (L.max_tokens + threads - 1) / threads);
  const Params p = make_params(L);
  return blocks * threads >= L.max_tokens ? launch<slots_kernel<false, 1, kBoth>>(p, blocks, threads, false, stream)
                                          : launch<slots_kernel<false, 4, kBoth>>(p, blocks, threads, false, stream);
}
cudaError_t launch_cache_truncate(const PagingLaunch& L, cudaStream_t stream) {
  const int64_t n = std::min(L.block_num, L.B * L.table_stride), c = cluster_for(n);
  return launch<truncate_kernel>(make_params(L), c, threads_for(n / c, L.B), true, stream);
}

}  // namespace ra
