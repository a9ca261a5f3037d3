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

// Rows [r0, 128) of a [128][D] bf16 tile (128-byte swizzle, 64-column blocks `block` bytes apart) that not every
// row of the other operand's tile may see.  A product multiplies them by weights of zero, and zero times an infinity or a
// NaN is NaN; so rows from `end` on (of no token of this sequence) become zeros, and non-finite elements of the others
// become zeros that are remembered: worst[c] takes the smallest (SMALLEST) or largest number first + r of such a row r in
// column c.  A row that does see it writes NaN there in the end.
template <int D, bool SMALLEST>
__device__ __forceinline__ void scrub_rows(uint8_t* tile, int block, int r0, int end, int first, int* worst,
                                           volatile int* any, int tid, int threads) {
  constexpr int kChunks = D / 8;
  for (int i = r0 * kChunks + tid; i < kSeqTile * kChunks; i += threads) {
    const int r = i / kChunks, c = i % kChunks;
    uint4* p = reinterpret_cast<uint4*>(tile + (c >> 3) * block + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    if (r >= end) {
      *p = make_uint4(0, 0, 0, 0);
      continue;
    }
    uint4 v = *p;
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool found = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t mask = 0x7F80u << (16 * (e & 1));
      if ((w[e >> 1] & mask) == mask) {
        w[e >> 1] &= (e & 1) ? 0x0000FFFFu : 0xFFFF0000u;
        if (SMALLEST)
          atomicMin(worst + c * 8 + e, first + r);
        else
          atomicMax(worst + c * 8 + e, first + r);
        found = true;
      }
    }
    if (found) {
      *p = make_uint4(w[0], w[1], w[2], w[3]);
      *any = 1;
    }
  }
  fence_proxy_async_smem();
}

// `n` (a multiple of 8, up to 32) bf16 values of one row.
__device__ __forceinline__ void store_cols(__nv_bfloat16* p, const float (&v)[32], int n) {
  if (n >= 32) {
    store32(p, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (8 * i < n) {
      uint4 u;
      u.x = pack_bf16x2(v[8 * i + 0], v[8 * i + 1]), u.y = pack_bf16x2(v[8 * i + 2], v[8 * i + 3]);
      u.z = pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), u.w = pack_bf16x2(v[8 * i + 6], v[8 * i + 7]);
      reinterpret_cast<uint4*>(p)[i] = u;
    }
}

// One lane of a converged warp.  What is computed before it stays uniform, so that the operands of the instructions behind
// it need no moves out of a lane's registers.
__device__ __forceinline__ bool one_lane() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// A box of a 4D tensor.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y, int32_t z,
                                            int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

}  // namespace mmdit
