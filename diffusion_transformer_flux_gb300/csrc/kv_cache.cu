// kv_cache.cu -- the bookkeeping of a paged cache of keys and values, and the write of new ones.
//
// block_tables: request b goes from before[b] to after[b] tokens, so from ceil(before / page) to ceil(after / page) pages.
// Pages given back go onto a stack of free pages, then pages wanted come from its top, both in the order of requests and
// of their pages within a request, so that the result is the same from call to call.  The order is a prefix sum over the
// requests, taken by one CTA (1024 requests at a time); what each request moves is read and written by its thread, or by
// its warp where it is more than a few pages.  The new tokens' positions and slots follow from the sums: each token
// finds its request by a binary search.  Up to kMapInPlace tokens the same CTA writes them (one launch, the step of
// answering requests, where latency is all); more of them go to a second kernel over the whole GPU.
//
// kv_cache_write: bound by memory, each new key and value read and written once in 16-byte pieces, four in flight a thread.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace mmdit {
namespace {

constexpr int kTableThreads = 1024;
constexpr int kMapInPlace = 4096;
constexpr int kOwnPages = 4;  // a request that moves at most that many pages is its thread's alone

struct Growth {
  int before, after, held, need;  // tokens, pages
};
__device__ __forceinline__ Growth growth_of(const BlockTableArgs& a, int b) {
  Growth g = {0, 0, 0, 0};
  if (b < a.batch) {
    const int most = a.width << a.page_shift;  // at most 2^30
    const int up = (1 << a.page_shift) - 1;
    g.before = min(max(a.before[b], 0), most), g.after = min(max(a.after[b], 0), most);
    g.held = (g.before + up) >> a.page_shift, g.need = (g.after + up) >> a.page_shift;
  }
  return g;
}

// Exclusive prefix sum over the CTA's threads and the total.
template <typename T>
__device__ __forceinline__ T scan_threads(T v, T* warp_sums, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[31];
  const T r = x - v + (warp ? warp_sums[warp - 1] : 0);
  __syncthreads();
  return r;
}

// Positions and slots of tokens first, first + step, ...
__device__ __forceinline__ void map_tokens(const BlockTableArgs& a, int64_t first, int64_t step) {
  const int end = a.cu[a.batch];
  for (int64_t i = first; i < a.capacity; i += step) {
    int64_t pos = 0, slot = -1;
    if (i < end) {
      int lo = 0, hi = a.batch;  // cu[lo] <= i < cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= i)
          lo = mid;
        else
          hi = mid;
      }
      const int most = a.width << a.page_shift;
      pos = min(max(a.before[lo], 0), most) + (i - a.cu[lo]);
      const int page = a.tables[static_cast<int64_t>(lo) * a.width + (pos >> a.page_shift)];
      if (page >= 0 && page < a.n_pages)
        slot = (static_cast<int64_t>(page) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
    }
    if (a.positions) a.positions[i] = pos;
    if (a.slots) a.slots[i] = slot;
  }
}

__global__ void __launch_bounds__(kTableThreads) block_tables_kernel(const __grid_constant__ BlockTableArgs a, int map_here) {
  __shared__ int sums[32];
  __shared__ long long sums64[32];
  const int lane = threadIdx.x & 31;
  pdl_wait();
  const int n_free = min(max(*a.n_free, 0), a.n_pages);
  // ---------------- pages given back: onto the stack
  int top = n_free;
  for (int b0 = 0; b0 < a.batch; b0 += kTableThreads) {
    const int b = b0 + threadIdx.x;
    const Growth g = growth_of(a, b);
    const int* row = a.tables + static_cast<int64_t>(b) * a.width;
    const int lost = max(g.held - g.need, 0);
    const unsigned many = __ballot_sync(0xffffffffu, lost > kOwnPages);
    int count = 0;  // entries that are pages: a request that found none free has entries without one
    if (lost <= kOwnPages)
      for (int p = g.need; p < g.held; ++p) count += static_cast<unsigned>(row[p]) < static_cast<unsigned>(a.n_pages);
    for (unsigned m = many; m; m &= m - 1) {
      const int src = __ffs(m) - 1;
      const int need = __shfl_sync(0xffffffffu, g.need, src), held = __shfl_sync(0xffffffffu, g.held, src);
      const int* r = a.tables + static_cast<int64_t>(b - lane + src) * a.width;
      int c = 0;
      for (int p = need + lane; p < held; p += 32) c += static_cast<unsigned>(r[p]) < static_cast<unsigned>(a.n_pages);
#pragma unroll
      for (int o = 16; o; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
      if (lane == src) count = c;
    }
    int total;
    int at = top + scan_threads(count, sums, total);
    if (lost <= kOwnPages)
      for (int p = g.need; p < g.held; ++p)
        if (static_cast<unsigned>(row[p]) < static_cast<unsigned>(a.n_pages)) {
          if (at < a.n_pages) a.free_pages[at] = row[p];
          ++at;
        }
    for (unsigned m = many; m; m &= m - 1) {
      const int src = __ffs(m) - 1;
      const int need = __shfl_sync(0xffffffffu, g.need, src), held = __shfl_sync(0xffffffffu, g.held, src);
      int to = __shfl_sync(0xffffffffu, at, src);
      const int* r = a.tables + static_cast<int64_t>(b - lane + src) * a.width;
      for (int p0 = need; p0 < held; p0 += 32) {
        const int page = p0 + lane < held ? r[p0 + lane] : -1;
        const bool there = static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages);
        const unsigned mask = __ballot_sync(0xffffffffu, there);
        const int place = to + __popc(mask & ((1u << lane) - 1));
        if (there && place < a.n_pages) a.free_pages[place] = page;
        to += __popc(mask);
      }
    }
    top += total;
  }
  top = min(top, a.n_pages);
  __syncthreads();
  // ---------------- pages wanted, and the new tokens' places
  int taken = 0;
  long long tokens = 0, left_out = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kTableThreads) {
    const int b = b0 + threadIdx.x;
    const Growth g = growth_of(a, b);
    const int gained = max(g.need - g.held, 0);
    int total;
    const int rank = taken + scan_threads(gained, sums, total);
    taken += total;
    if (gained <= kOwnPages) {
      int* row = a.tables + static_cast<int64_t>(b) * a.width;
      for (int p = g.held; p < g.need; ++p) {
        const int from = top - 1 - (rank + p - g.held);
        row[p] = from >= 0 ? a.free_pages[from] : -1;
      }
    }
    for (unsigned m = __ballot_sync(0xffffffffu, gained > kOwnPages); m; m &= m - 1) {
      const int src = __ffs(m) - 1;
      const int need = __shfl_sync(0xffffffffu, g.need, src), held = __shfl_sync(0xffffffffu, g.held, src);
      const int r0 = __shfl_sync(0xffffffffu, rank, src);
      int* row = a.tables + static_cast<int64_t>(b - lane + src) * a.width;
      for (int p = held + lane; p < need; p += 32) {
        const int from = top - 1 - (r0 + p - held);
        row[p] = from >= 0 ? a.free_pages[from] : -1;
      }
    }
    const int fresh = max(g.after - g.before, 0);
    long long sum;
    const long long first = tokens + scan_threads(static_cast<long long>(fresh), sums64, sum);
    tokens += sum;
    if (b < a.batch) {
      a.cu[b] = static_cast<int>(min(first, static_cast<long long>(a.capacity)));
      const long long asked = max(static_cast<long long>(a.after[b]) - max(a.before[b], 0), 0ll);
      left_out += max(asked - fresh, 0ll);
    }
  }
  {
    long long sum;
    scan_threads(left_out, sums64, sum);
    left_out = sum + max(tokens - a.capacity, 0ll);
  }
  if (threadIdx.x == 0) {
    a.cu[a.batch] = static_cast<int>(min(tokens, static_cast<long long>(a.capacity)));
    *a.n_free_out = max(top - taken, 0);
    a.missing[0] = max(taken - top, 0);
    a.missing[1] = static_cast<int>(min(left_out, static_cast<long long>(INT32_MAX)));
  }
  __syncthreads();
  if (map_here) map_tokens(a, threadIdx.x, kTableThreads);
}

__global__ void __launch_bounds__(256) token_map_kernel(const __grid_constant__ BlockTableArgs a) {
  pdl_wait();
  map_tokens(a, static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, static_cast<int64_t>(gridDim.x) * 256);
}

constexpr int kWriteThreads = 256;
constexpr int kWriteItems = 4;  // 16-byte pieces of a thread in flight

__global__ void __launch_bounds__(kWriteThreads) kv_write_kernel(const __grid_constant__ CacheWriteArgs a, int tokens_per_cta) {
  pdl_wait();
  const int per_head = a.head_dim / 8, per_token = a.heads * per_head;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_cta;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(tokens_per_cta), a.tokens - t0));
  const int items = tokens * 2 * per_token;
  const int64_t slots = static_cast<int64_t>(a.n_pages) << a.page_shift;
  for (int i0 = threadIdx.x; i0 < items; i0 += kWriteThreads * kWriteItems) {
    uint4 v[kWriteItems];
    uint4* to[kWriteItems];
#pragma unroll
    for (int u = 0; u < kWriteItems; ++u) {
      to[u] = nullptr;
      const int i = i0 + u * kWriteThreads;
      if (i >= items) continue;
      const int t = i / (2 * per_token), rest = i % (2 * per_token), is_v = rest >= per_token;
      const int piece = rest - is_v * per_token, h = piece / per_head, c = piece % per_head;
      const int64_t slot = a.slots[t0 + t];
      if (slot < 0 || slot >= slots) continue;
      const HeadsView& from = is_v ? a.v : a.k;
      const PagesView& page = is_v ? a.v_pages : a.k_pages;
      v[u] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(from.ptr) + (t0 + t) * from.stride_t +
                                             h * from.stride_h + c * 8);
      to[u] = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(page.ptr) + (slot >> a.page_shift) * page.stride_page +
                                       (slot & ((1 << a.page_shift) - 1)) * page.stride_t + h * page.stride_h + c * 8);
    }
#pragma unroll
    for (int u = 0; u < kWriteItems; ++u)
      if (to[u]) *to[u] = v[u];
  }
}

}  // namespace

cudaError_t launch_block_tables(const BlockTableArgs& a, cudaStream_t stream) {
  const int map_here = a.capacity <= kMapInPlace || !(a.positions || a.slots) ? 1 : 0;
  cudaError_t e = launch_pdl(block_tables_kernel, dim3(1), dim3(kTableThreads), 0, stream, a, map_here);
  if (e != cudaSuccess) return e;
  count_launch();
  if (!map_here) {
    const int grid = static_cast<int>(std::min<int64_t>((a.capacity + 255) / 256, 8 * num_sms()));
    e = launch_pdl(token_map_kernel, dim3(grid), dim3(256), 0, stream, a);
    if (e != cudaSuccess) return e;
    count_launch();
  }
  return cudaGetLastError();
}

cudaError_t launch_kv_write(const CacheWriteArgs& a, cudaStream_t stream) {
  // as many tokens to a CTA as give each thread its pieces once
  const int per_token = 2 * a.heads * (a.head_dim / 8);
  const int each = std::max(1, kWriteThreads * kWriteItems / per_token);
  const int64_t grid = (a.tokens + each - 1) / each;
  const cudaError_t e = launch_pdl(kv_write_kernel, dim3(static_cast<unsigned>(grid)), dim3(kWriteThreads), 0, stream, a, each);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace mmdit
