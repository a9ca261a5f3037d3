// kv_cache.cu -- the bookkeeping of a paged cache of keys and values, and the write of new ones.
//
// block_tables: request b goes from before[b] to after[b] tokens, so from ceil(before / page) to ceil(after / page) pages.
// Pages given back go onto a stack of free pages, then pages wanted come from its top, both in the order of requests and
// of their pages within a request, so that the result is the same from call to call.  The order is a prefix sum over the
// requests, taken by one CTA (1024 requests at a time); what each request moves is read and written by its thread, or where
// it is more than a few pages by a warp: its own, unless a warp has more than kOwnRequests of them (64 new prompts: 15.2 us, as
// 32 requests of a warp wait for one another; shared among the 32 warps 8.2; one finished request among 256: 8.1 us by its own
// warp, 9.7 shared).  The new tokens' positions and slots follow from the sums: each token
// finds its request by a binary search.  Up to kMapInPlace tokens the same CTA writes them (one launch, the step of
// answering requests, where latency is all); more of them go to a second kernel over the whole GPU.
//
// kv_cache_write: bound by memory, each new key and value read and written once in 16-byte pieces, two in flight a thread (9216
// tokens of 8 heads of 128: 13.6 us, 5.5 TB/s; with the compiler's integer divisions for a piece's place 15.4).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace mmdit {
namespace {

constexpr int kTableThreads = 1024;
constexpr int kMapInPlace = 4096;
constexpr int kTableWarps = kTableThreads / 32;
constexpr int kOwnPages = 4;  // a request that moves at most that many pages is its thread's alone
constexpr int kOwnRequests = 2;  // of others a warp moves as many of its own; where one has more, all warps share all of them

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

// A request's entries [first, last) that change, and their place among the pages that move.
struct Move {
  int first, last, place;
};

// Exclusive prefix sums over the CTA's threads and the totals, of two values at once (so that they share the barriers).
template <typename T, typename U>
__device__ __forceinline__ void scan_threads(T& v, U& w, T* v_sums, U* w_sums, T& v_total, U& w_total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
  U y = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x1 = __shfl_up_sync(0xffffffffu, x, o);
    const U y1 = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += x1, y += y1;
  }
  if (lane == 31) v_sums[warp] = x, w_sums[warp] = y;
  __syncthreads();
  if (warp == 0) {
    T p = v_sums[lane];
    U q = w_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T p1 = __shfl_up_sync(0xffffffffu, p, o);
      const U q1 = __shfl_up_sync(0xffffffffu, q, o);
      if (lane >= o) p += p1, q += q1;
    }
    v_sums[lane] = p, w_sums[lane] = q;
  }
  __syncthreads();
  v_total = v_sums[31], w_total = w_sums[31];
  v = x - v + (warp ? v_sums[warp - 1] : 0), w = y - w + (warp ? w_sums[warp - 1] : 0);
  __syncthreads();
}
template <typename T>
__device__ __forceinline__ T scan_threads(T v, T* sums, T& total) {
  __shared__ int none[32];
  int zero = 0, zeros;
  scan_threads(v, zero, sums, none, total, zeros);
  return v;
}

// Where each request's tokens start, in shared memory as far as they fit: a search has no step that waits for memory (256
// requests of one token: 8.4 us with the sums and lengths in global memory, 7.7 so).
constexpr int kMapRequests = 2048;
struct MapShared {
  int cu[kMapRequests + 1], before[kMapRequests];
};

// Positions and slots of tokens first, first + step, ...
__device__ __forceinline__ void map_tokens(const BlockTableArgs& a, const int* cu, const int* before, int64_t first, int64_t step) {
  const int end = cu[a.batch];
  for (int64_t i = first; i < a.capacity; i += step) {
    int64_t pos = 0, slot = -1;
    if (i < end) {
      int lo = 0, hi = a.batch;  // cu[lo] <= i < cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= i)
          lo = mid;
        else
          hi = mid;
      }
      const int most = a.width << a.page_shift;
      pos = min(max(before[lo], 0), most) + (i - cu[lo]);
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
  __shared__ MapShared map;
  __shared__ Move moves[kTableThreads];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool fits = a.batch <= kMapRequests;
  pdl_wait();
  pdl_trigger();
  const int n_free = min(max(*a.n_free, 0), a.n_pages);
  // ---------------- pages given back: onto the stack
  int top = n_free;
  for (int b0 = 0; b0 < a.batch; b0 += kTableThreads) {
    const int b = b0 + threadIdx.x;
    const int here = min(a.batch - b0, kTableThreads);
    const Growth g = growth_of(a, b);
    const int* row = a.tables + static_cast<int64_t>(b) * a.width;
    const int lost = max(g.held - g.need, 0);
    int count = 0;  // entries that are pages: a request that found none free has entries without one
    if (lost <= kOwnPages)
      for (int p = g.need; p < g.held; ++p) count += static_cast<unsigned>(row[p]) < static_cast<unsigned>(a.n_pages);
    const unsigned many = __ballot_sync(0xffffffffu, lost > kOwnPages);
    const bool spread = __syncthreads_or(__popc(many) > kOwnRequests);
    auto count_pages = [&](int r, int first, int last) {
      const int* from = a.tables + static_cast<int64_t>(b0 + r) * a.width;
      int c = 0;
      for (int p = first + lane; p < last; p += 32) c += static_cast<unsigned>(from[p]) < static_cast<unsigned>(a.n_pages);
#pragma unroll
      for (int o = 16; o; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
      return c;
    };
    auto give_back = [&](int r, int first, int last, int to) {
      const int* from = a.tables + static_cast<int64_t>(b0 + r) * a.width;
      for (int p0 = first; p0 < last; p0 += 32) {
        const int page = p0 + lane < last ? from[p0 + lane] : -1;
        const bool there = static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages);
        const unsigned mask = __ballot_sync(0xffffffffu, there);
        const int place = to + __popc(mask & ((1u << lane) - 1));
        if (there && place < a.n_pages) a.free_pages[place] = page;
        to += __popc(mask);
      }
    };
    if (spread) {
      moves[threadIdx.x] = {g.need, g.held, 0};
      __syncthreads();
      for (int r = warp; r < here; r += kTableWarps) {
        const Move m = moves[r];
        if (m.last - m.first <= kOwnPages) continue;
        const int c = count_pages(r, m.first, m.last);
        if (lane == 0) moves[r].place = c;
      }
      __syncthreads();
      if (lost > kOwnPages) count = moves[threadIdx.x].place;
    } else {
      for (unsigned m = many; m; m &= m - 1) {
        const int src = __ffs(m) - 1;
        const int c = count_pages(warp * 32 + src, __shfl_sync(0xffffffffu, g.need, src), __shfl_sync(0xffffffffu, g.held, src));
        if (lane == src) count = c;
      }
    }
    int total;
    int at = top + scan_threads(count, sums, total);
    if (lost <= kOwnPages)
      for (int p = g.need; p < g.held; ++p)
        if (static_cast<unsigned>(row[p]) < static_cast<unsigned>(a.n_pages)) {
          if (at < a.n_pages) a.free_pages[at] = row[p];
          ++at;
        }
    if (spread) {
      if (lost > kOwnPages) moves[threadIdx.x].place = at;
      __syncthreads();
      for (int r = warp; r < here; r += kTableWarps) {
        const Move m = moves[r];
        if (m.last - m.first > kOwnPages) give_back(r, m.first, m.last, m.place);
      }
      __syncthreads();
    } else {
      for (unsigned m = many; m; m &= m - 1) {
        const int src = __ffs(m) - 1;
        give_back(warp * 32 + src, __shfl_sync(0xffffffffu, g.need, src), __shfl_sync(0xffffffffu, g.held, src),
                  __shfl_sync(0xffffffffu, at, src));
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
    const int here = min(a.batch - b0, kTableThreads);
    const Growth g = growth_of(a, b);
    const int gained = max(g.need - g.held, 0), fresh = max(g.after - g.before, 0);
    int rank = gained, total;
    long long first = fresh, sum;
    scan_threads(rank, first, sums, sums64, total, sum);
    rank += taken, first += tokens;
    taken += total, tokens += sum;
    if (gained <= kOwnPages) {
      int* row = a.tables + static_cast<int64_t>(b) * a.width;
      for (int p = g.held; p < g.need; ++p) {
        const int from = top - 1 - (rank + p - g.held);
        row[p] = from >= 0 ? a.free_pages[from] : -1;
      }
    }
    const unsigned many = __ballot_sync(0xffffffffu, gained > kOwnPages);
    auto hand_out = [&](int r, int first, int last, int place) {
      int* to = a.tables + static_cast<int64_t>(b0 + r) * a.width;
      for (int p = first + lane; p < last; p += 32) {
        const int from = top - 1 - (place + p - first);
        to[p] = from >= 0 ? a.free_pages[from] : -1;
      }
    };
    if (__syncthreads_or(__popc(many) > kOwnRequests)) {
      moves[threadIdx.x] = {g.held, g.need, rank};
      __syncthreads();
      for (int r = warp; r < here; r += kTableWarps) {
        const Move m = moves[r];
        if (m.last - m.first > kOwnPages) hand_out(r, m.first, m.last, m.place);
      }
      __syncthreads();
    } else {
      for (unsigned m = many; m; m &= m - 1) {
        const int src = __ffs(m) - 1;
        hand_out(warp * 32 + src, __shfl_sync(0xffffffffu, g.held, src), __shfl_sync(0xffffffffu, g.need, src),
                 __shfl_sync(0xffffffffu, rank, src));
      }
    }
    if (b < a.batch) {
      const int start = static_cast<int>(min(first, static_cast<long long>(a.capacity)));
      a.cu[b] = start;
      if (fits) map.cu[b] = start, map.before[b] = g.before;
      const long long asked = max(static_cast<long long>(a.after[b]) - max(a.before[b], 0), 0ll);
      left_out += max(asked - fresh, 0ll);
    }
  }
  if (__syncthreads_or(left_out != 0)) {
    long long sum;
    scan_threads(left_out, sums64, sum);
    left_out = sum;
  }
  left_out += max(tokens - a.capacity, 0ll);
  if (threadIdx.x == 0) {
    const int end = static_cast<int>(min(tokens, static_cast<long long>(a.capacity)));
    a.cu[a.batch] = end;
    if (fits) map.cu[a.batch] = end;
    *a.n_free_out = max(top - taken, 0);
    a.missing[0] = max(taken - top, 0);
    a.missing[1] = static_cast<int>(min(left_out, static_cast<long long>(INT32_MAX)));
  }
  __syncthreads();
  if (map_here) map_tokens(a, fits ? map.cu : a.cu, fits ? map.before : a.before, threadIdx.x, kTableThreads);
}

__global__ void __launch_bounds__(256) token_map_kernel(const __grid_constant__ BlockTableArgs a) {
  __shared__ MapShared map;
  const bool fits = a.batch <= kMapRequests;
  pdl_wait();
  if (fits) {
    for (int i = threadIdx.x; i <= a.batch; i += 256) map.cu[i] = a.cu[i];
    for (int i = threadIdx.x; i < a.batch; i += 256) map.before[i] = a.before[i];
    __syncthreads();
  }
  map_tokens(a, fits ? map.cu : a.cu, fits ? map.before : a.before, static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x,
             static_cast<int64_t>(gridDim.x) * 256);
}

constexpr int kWriteThreads = 128;
constexpr int kWriteItems = 2;  // 16-byte pieces of a thread in flight (1, 2, 4: 1.9, 1.9, 2.7 us for 32 tokens, 16.6, 13.6, 13.5 for 9216)

__global__ void __launch_bounds__(kWriteThreads)
    kv_write_kernel(const __grid_constant__ CacheWriteArgs a, int tokens_per_cta, Divisor by_token, Divisor by_head) {
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
      const int t = by_token.quotient(i), rest = i - t * 2 * per_token, is_v = rest >= per_token;
      const int piece = rest - is_v * per_token, h = by_head.quotient(piece), c = piece - h * per_head;
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
  const bool places = a.positions || a.slots;
  const int map_here = places && a.capacity <= kMapInPlace ? 1 : 0;
  cudaError_t e = launch_pdl(block_tables_kernel, dim3(1), dim3(kTableThreads), 0, stream, a, map_here);
  if (e != cudaSuccess) return e;
  count_launch();
  if (places && !map_here) {
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
  const cudaError_t e = launch_pdl(kv_write_kernel, dim3(static_cast<unsigned>(grid)), dim3(kWriteThreads), 0, stream, a, each,
                                   Divisor(per_token), Divisor(a.head_dim / 8));
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace mmdit
