// attention_tiles.cuh -- what the kernels over packed sequences and paged caches share: their arguments,
// the place of a tile among the sequences, and the treatment of values that part of a tile must not see.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace mmdit {

constexpr int kSeqTile = 128;                  // rows of a query tile, keys of a key tile
constexpr int kSeqBlock = kSeqTile * 128;      // bytes of 128 rows of 64 bf16 (one 128-byte swizzle column block)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A row that sees no key is 0, its log-sum -inf.  One that sees keys whose scores are all -inf has no weights (0 / 0): it is NaN, and
// so is its log-sum.  Where its keys are split, a part of such keys alone has this log2-sum and zeros: beside any other it weighs
// nothing, and if it is the largest the row is NaN.
constexpr float kNoWeights = -3.402823466e38f;

// The largest b < n with start(b) <= x, for start rising with b and start(0) <= x (else 0): a search by 32 places at a
// time, by all lanes of a warp (2 rounds of loads up to 1024 sequences).
template <typename F>
__device__ __forceinline__ int find_segment(int n, int x, F start) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int b = lo + lane * step;
    const bool below = b < hi && start(b) <= x;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u);
    lo += last * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// One packed sequence: rows [q0, q0 + n) are its queries, [k0, k0 + m) its keys (m alone for a paged cache).  The lengths
// are the device's; whatever they hold, the rows stay within the tensors.
struct Segment {
  int q0, n, k0, m;
};

__device__ __forceinline__ void clip_segment(const int* cu, int b, int total, int& first, int& count) {
  const int lo = min(max(cu[b], 0), total), hi = min(max(cu[b + 1], 0), total);
  first = lo, count = max(hi - lo, 0);
}

// The number of keys that query i of the segment sees: all, or those up to its own position m - n + i.
__device__ __forceinline__ int keys_seen(const Segment& s, int i, int causal) {
  return causal ? min(max(s.m - s.n + i + 1, 0), s.m) : s.m;
}

// The tiles of a packed batch (of `span` rows of the sequences in cu; `other` is the other side's prefix sums, or null) in the
// order in which they are handed out, held by the lanes of a warp.  Dear ones go first, so that the GPU's SMs end together.
//   Up to 32 sequences: a lane holds one each, sorted by the other side's length.  Where a tile's cost falls with its number
//   (causal) the tiles of all sequences come level by level, else sequence by sequence; number x is found by counting.
//   More: sequence b's tiles are number cu[b] / span + b and the following, which leaves each at least as many numbers as
//   it needs without a prefix sum; those left over are of no tile, and the sequences come in their order.  Where sequences of
//   up to `skip` rows have no tiles (they are another kernel's, and most of a batch) nearly all numbers would be of no
//   tile: there the tiles are counted, 32 sequences at a time, on from where the last search ended.
// `from_end`: a sequence's last tile is its dearest.
struct TileOrder {
  const int *cu, *other;
  int total, other_total, batch, span, causal, from_end, skip;
  int n;                                                // numbers
  int seq, first, count, other_first, other_count;      // this lane's sequence
  int tiles;
  int level, base;                                      // where the last search ended

  __device__ __forceinline__ void init(const int* cu_, int total_, const int* other_, int other_total_, int batch_, int span_,
                                       int causal_, int from_end_, int skip_ = 0) {
    cu = cu_, total = total_, other = other_, other_total = other_total_, batch = batch_, span = span_;
    causal = causal_, from_end = from_end_, skip = skip_, level = 0, base = 0;
    if (batch > 32 && skip > 0) {
      n = 0;
      for (int b = 0; b < batch; b += 32) n += tiles_of(b + (threadIdx.x & 31));
#pragma unroll
      for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      return;
    }
    if (batch > 32) {
      n = total / span + batch;
      return;
    }
    const int lane = threadIdx.x & 31, i = min(lane, batch - 1);
    seq = lane;
    clip_segment(cu, i, total, first, count);
    other_first = 0, other_count = 0;
    if (other) clip_segment(other, i, other_total, other_first, other_count);
    const int length = other ? other_count : count;
    int rank = lane < batch ? 0 : lane, from = lane;
    for (int j = 0; j < batch; ++j) {
      const int l = __shfl_sync(0xffffffffu, length, j);
      rank += lane < batch && (l > length || (l == length && j < lane));
    }
    for (int j = 0; j < batch; ++j)
      if (__shfl_sync(0xffffffffu, rank, j) == lane) from = j;
    seq = __shfl_sync(0xffffffffu, seq, from), first = __shfl_sync(0xffffffffu, first, from);
    count = __shfl_sync(0xffffffffu, count, from), other_first = __shfl_sync(0xffffffffu, other_first, from);
    other_count = __shfl_sync(0xffffffffu, other_count, from);
    tiles = lane < batch && count > skip ? (count + span - 1) / span : 0;
    n = tiles;
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  }

  __device__ __forceinline__ int tiles_of(int b) const {
    if (b >= batch) return 0;
    int f, c;
    clip_segment(cu, b, total, f, c);
    return c > skip ? (c + span - 1) / span : 0;
  }

  struct Found {
    int b, first, count, other_first, other_count;
    int start;  // the tile's first row in its sequence
  };
  // Number x < n; false where it is of no tile.
  __device__ __forceinline__ bool find(int x, Found& f) {
    int tile;
    if (batch > 32 && skip > 0) {  // level: the first of 32 sequences, base: the tiles before it
      if (x < base) level = 0, base = 0;
      for (; level < batch; level += 32) {
        const int mine = tiles_of(level + (threadIdx.x & 31));
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, sum, o);
          if ((threadIdx.x & 31) >= o) sum += y;
        }
        const unsigned after = __ballot_sync(0xffffffffu, base + sum > x);
        if (after) {
          const int lane = __ffs(after) - 1;
          f.b = level + lane;
          tile = x - base - __shfl_sync(0xffffffffu, sum - mine, lane);
          if (from_end) tile = __shfl_sync(0xffffffffu, mine, lane) - 1 - tile;
          clip_segment(cu, f.b, total, f.first, f.count);
          f.other_first = f.other_count = 0;
          f.start = tile * span;
          return true;
        }
        base += __shfl_sync(0xffffffffu, sum, 31);
      }
      return false;
    }
    if (batch > 32) {
      const int y = from_end ? n - 1 - x : x;
      f.b = find_segment(batch, y, [&](int i) { return min(max(cu[i], 0), total) / span + i; });
      clip_segment(cu, f.b, total, f.first, f.count);
      f.other_first = f.other_count = 0;
      if (other) clip_segment(other, f.b, other_total, f.other_first, f.other_count);
      tile = y - (f.first / span + f.b);
    } else {
      int lane;
      if (causal) {
        if (x < base) level = 0, base = 0;
        unsigned have = __ballot_sync(0xffffffffu, tiles > level);
        while (x >= base + __popc(have) && have) {
          base += __popc(have), ++level;
          have = __ballot_sync(0xffffffffu, tiles > level);
        }
        const unsigned mine = 1u << (threadIdx.x & 31);
        lane = __ffs(__ballot_sync(0xffffffffu, (have & mine) && __popc(have & (mine - 1)) == x - base)) - 1;
        lane = max(lane, 0);
        tile = level;
      } else {
        int sum = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, sum, o);
          if ((threadIdx.x & 31) >= o) sum += y;
        }
        const unsigned after = __ballot_sync(0xffffffffu, sum > x);
        lane = after ? __ffs(after) - 1 : 0;
        tile = x - __shfl_sync(0xffffffffu, sum - tiles, lane);
      }
      f.b = __shfl_sync(0xffffffffu, seq, lane), f.first = __shfl_sync(0xffffffffu, first, lane);
      f.count = __shfl_sync(0xffffffffu, count, lane), f.other_first = __shfl_sync(0xffffffffu, other_first, lane);
      f.other_count = __shfl_sync(0xffffffffu, other_count, lane);
      if (from_end) tile = __shfl_sync(0xffffffffu, tiles, lane) - 1 - tile;
    }
    f.start = tile * span;
    return tile >= 0 && f.start < f.count;
  }
};

// Whether one of eight bf16 values is not finite: its exponent is all ones, and adding one to that carries into the sign's place.
__device__ __forceinline__ uint32_t not_finite(const uint4& v) {
  constexpr uint32_t kExp = 0x7F807F80u, kOne = 0x00800080u;
  return (((v.x & kExp) + kOne) | ((v.y & kExp) + kOne) | ((v.z & kExp) + kOne) | ((v.w & kExp) + kOne)) & 0x80008000u;
}

// Rows [r0, 128) of a [128][D] bf16 tile (128-byte swizzle, 64-column blocks) that not every row of the other operand's
// tile may see.  A product multiplies them by weights of zero, and zero times an infinity or a NaN is NaN; so rows from `end` on
// (of no token of this sequence) become zeros, and non-finite elements of the others become zeros that are remembered:
// worst[c] takes the smallest number first + r of such a row r in column c.  A row that does see it writes NaN there in the
// end.  Called by 64 threads; eight pieces are in flight in each.
template <int D>
__device__ __forceinline__ void scrub_rows(uint8_t* tile, int r0, int end, int first, int* worst, volatile int* any, int tid) {
  constexpr int kChunks = D / 8;
  auto at = [&](int i) {
    const int r = i / kChunks, c = i % kChunks;
    return reinterpret_cast<uint4*>(tile + (c >> 3) * kSeqBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4));
  };
  const int stop = min(max(end, r0), kSeqTile) * kChunks;
  for (int i0 = r0 * kChunks + tid; i0 < stop; i0 += 8 * 64) {
    uint4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = i0 + 64 * u < stop ? *at(i0 + 64 * u) : make_uint4(0, 0, 0, 0);
    uint32_t bad = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) bad |= (not_finite(v[u]) ? 1u : 0u) << u;
    if (bad == 0) continue;
    for (int u = 0; u < 8; ++u)
      if (bad >> u & 1u) {
        const int i = i0 + 64 * u, c = i % kChunks;
        uint16_t* e = reinterpret_cast<uint16_t*>(at(i));
        for (int k = 0; k < 8; ++k)
          if ((e[k] & 0x7F80u) == 0x7F80u) {
            e[k] = 0;
            atomicMin(worst + c * 8 + k, first + i / kChunks);
          }
        *any = 1;
      }
  }
  for (int i = stop + tid; i < kSeqTile * kChunks; i += 64) *at(i) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
}

// 32 rows of D bf16 values out of a warp's 32 x D / 8 16-byte pieces in shared memory (piece c of a row at c ^ (row & 7)), whole rows
// at a time: lane l holds the address `row` of row l (null: not written).  A thread that stored its own row would touch 32
// lines with each store (5000 cycles for a CTA's two tiles against 1000).
template <int D>
__device__ __forceinline__ void store_rows(const uint8_t* pieces, const __nv_bfloat16* row, int head_dim) {
  constexpr int kChunks = D / 8, kRows = 32 / kChunks;
  const int lane = threadIdx.x & 31, c = lane % kChunks, r0 = lane / kChunks;
#pragma unroll 4
  for (int i = 0; i < 32 / kRows; ++i) {
    const int r = i * kRows + r0;
    const uint64_t p = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(row), r);
    const uint4 v = *reinterpret_cast<const uint4*>(pieces + r * (2 * D) + ((c ^ (r & 7)) << 4));
    if (p && c * 8 < head_dim) reinterpret_cast<uint4*>(p)[c] = v;
  }
}
// The pieces of 32 columns (from 32 e) of this lane's row.
template <int D>
__device__ __forceinline__ void put_pieces(uint8_t* pieces, int e, const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 u;
    u.x = pack_bf16x2(v[8 * i + 0], v[8 * i + 1]), u.y = pack_bf16x2(v[8 * i + 2], v[8 * i + 3]);
    u.z = pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), u.w = pack_bf16x2(v[8 * i + 6], v[8 * i + 7]);
    *reinterpret_cast<uint4*>(pieces + lane * (2 * D) + (((4 * e + i) ^ (lane & 7)) << 4)) = u;
  }
}

// The same for 32 columns at a time, from 2 KB: piece c of row r at c ^ (r / 2 & 3) of its 64 bytes.
__device__ __forceinline__ void put_pieces32(uint8_t* pieces, const float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 u;
    u.x = pack_bf16x2(v[8 * i + 0], v[8 * i + 1]), u.y = pack_bf16x2(v[8 * i + 2], v[8 * i + 3]);
    u.z = pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), u.w = pack_bf16x2(v[8 * i + 6], v[8 * i + 7]);
    *reinterpret_cast<uint4*>(pieces + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)) = u;
  }
}
__device__ __forceinline__ void store_rows32(const uint8_t* pieces, const __nv_bfloat16* row, int columns) {
  const int lane = threadIdx.x & 31, c = lane & 3, r0 = lane >> 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + r0;
    const uint64_t p = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(row), r);
    const uint4 v = *reinterpret_cast<const uint4*>(pieces + r * 64 + ((c ^ (r >> 1 & 3)) << 4));
    if (p && c * 8 < columns) reinterpret_cast<uint4*>(p)[c] = v;
  }
}

// mbar_wait for what lasts as long as a work item does (its tiles are others' work): of 2^28 keys some seconds.  The limit
// counts from the last change of `*progress`, which the warp that hands out items and loads tiles changes with each.
__device__ __forceinline__ bool mbar_wait_item(uint64_t* bar, uint32_t parity, volatile uint32_t* progress, volatile int* abort,
                                               uint32_t* status, uint32_t err_bit) {
  if (mbar_test(bar, parity)) return true;
  uint64_t t0 = global_timer_ns();
  uint32_t before = *progress;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_test(bar, parity)) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      const uint32_t now = *progress;
      if (now == before) {
        *abort = 1;
        atomicOr(status, err_bit);
        return false;
      }
      before = now, t0 = global_timer_ns();
    }
  }
}

// One lane of a converged warp.  What is computed before it stays uniform, so that the operands of the instructions behind
// it need no moves out of a lane's registers.
__device__ __forceinline__ bool one_lane() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Moves registers between the warpgroups of a CTA: the sum of the shares is what the launch gave.
template <int R>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
// 384 threads are launched with 168 each: 128 x 72 + 256 x 216.
constexpr int kLaunchRegisters = 168, kServiceRegisters = 72, kSoftmaxRegisters = 216;
static_assert(128 * kServiceRegisters + 256 * kSoftmaxRegisters <= 384 * kLaunchRegisters, "shares of the launch's registers");

// A box of a 4D tensor.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y, int32_t z,
                                            int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// The same of what is read once: its lines are the first to make room in L2 (code, lengths, tables and the other operators' data
// stay).
__device__ __forceinline__ uint64_t read_once_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y, int32_t z,
                                            int32_t w, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z), "r"(w), "l"(policy)
      : "memory");
}

}  // namespace mmdit
