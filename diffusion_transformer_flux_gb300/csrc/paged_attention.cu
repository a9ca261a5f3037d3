// paged_attention.cu -- attention of few rows over a paged cache (the single tokens of answering requests), and the
// join of a sequence's parts.
//
// The arithmetic is attention_varlen.cu's; here a sequence has at most 16 rows (new tokens by the heads of a group), so
// the cost is reading its keys and values once.  The keys of all sequences lie behind one another as steps of 64 keys, and a
// CTA takes an equal run of them (at least kFewLeast, so that its part is worth its join) for one key head: whatever the
// lengths, the CTAs that the GPU holds at once end together.  A sequence's start counts as kFewStart steps (without that, one
// CTA worked through 8 sequences of 20 keys: 29 us).  The key heads' CTAs of a run are neighbours, as the key heads'
// keys are in memory (each head's runs behind the last head's: 111 against 96 us for one token over 120000).  A run covers the
// end of one sequence's steps, whole ones, and the start of another's; whole ones are written at once, the others leave
// normalised float32 parts and their log2-sums (at most two to a CTA), which paged_few_join_kernel adds in a fixed order.
// Where no sequence has more than kFewWhole steps a CTA takes one sequence and key head, and nothing is joined.
//
// In a step each of the four warps takes 16 keys: its own ring of TMA copies (a lane for each box: a page's rows by 64
// columns), its own running maximum and its own float32 output, so no warp waits for another before the end.  The products
// are mma.sync m16n8k16 with the keys as the 16 (a tcgen05 product of 128 rows would be seven eighths padding, and its
// hand-over through tensor memory costs more than these 16 instructions for 16 keys): S^T = K Q^T, whose accumulators, as bf16
// pairs turned by movmatrix, are the second operand of O^T += V^T P^T; more than 8 rows are two such columns.  The maximum
// is reduced over the lanes only where one of them has a score 2^8 above it.  With the queries as the 16, copies of 16 bytes by
// every lane and a maximum for each tile a warp had 640 instructions a tile to issue, and it was 111 us.
//
// What bounds it is the reading and, for short runs, what precedes it, where each access that waits for
// the one before costs 2000 cycles with nothing in the caches: the lengths, the first pages (all stages' at once) and Q (16
// bytes a thread, through shared memory: 4-byte loads of fragments took 9 us) are three such steps, and the code is kept
// short, its rare parts out of the loop.  Pages are read once and make room first in L2, so that these stay in it (4 x 8 tokens:
// 39 -> 34 us).  Two stages of a warp (128 KB on the way on an SM) read faster than three: 180 against 188 us for the batch.
// One token over 120000 (492 MB): 75 us, 6.56 TB/s; 32 tokens over up to 16384 (1.25 GB): 180 us, 6.88 TB/s; 4 tokens over up
// to 8192 of 8 sequences (160 MB): 32 us.
#include <algorithm>

#include "attention_tiles.cuh"

namespace mmdit {
namespace {

constexpr int kFewThreads = 128;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewKeys = 16;  // of a warp's tile
constexpr float kFewThreshold = 8.0f;  // in log2 units: how far a maximum grows before the output is rescaled
static_assert(kFewStep == kFewWarps * kFewKeys, "a step is a tile for each warp");

template <int D>
struct FewCfg {
  static constexpr int kBlock = kFewKeys * 128;      // 16 keys of 64 columns (one 128-byte swizzle column block)
  static constexpr int kTile = (D / 64) * kBlock;    // K or V of a tile
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kRing = kStages * 2 * kTile;
  static constexpr int kSmem = kFewWarps * kRing + 1024;  // 65 KB: two CTAs on an SM
};
static_assert(FewCfg<64>::kSmem >= kFewWarps * kFewRows * (64 + 2) * 4 &&
                  FewCfg<128>::kSmem >= kFewWarps * kFewRows * (128 + 2) * 4,
              "the parts of the warps lie in the rings at the end");

struct FewShared {
  uint64_t full[kFewWarps][4];
  int abort_flag;
  int any_bad;
  int worst[128];
  uint4 q[kFewRows][128 / 8 + 1];
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// An 8 x 8 matrix of 16-bit elements, two to a lane, turned.
__device__ __forceinline__ uint32_t turn8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The byte of 16-byte piece c of key r in a tile.
template <int D>
__device__ __forceinline__ uint32_t few_at(int r, int c) {
  return static_cast<uint32_t>((c >> 3) * FewCfg<D>::kBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// The steps of a sequence of few rows for one key head, and their number in the runs: its start counts as kFewStart more, which
// lie before them.
__device__ __forceinline__ int steps_of(const SeqAttnArgs& a, int b) {
  const int lo = min(max(a.cu_q[b], 0), a.tokens_q), hi = min(max(a.cu_q[b + 1], 0), a.tokens_q);
  const int m = min(max(a.kv_lens[b], 0), a.max_keys);  // read beside the others, not behind their test
  return hi <= lo || hi - lo > a.few_tokens ? 0 : max((m + kFewStep - 1) / kFewStep, 1);
}
__device__ __forceinline__ int counted(int steps) { return steps > 0 ? steps + kFewStart : 0; }
// Their number up to sequence `until` (all: batch), by all lanes of a warp.
__device__ __forceinline__ int steps_before(const SeqAttnArgs& a, int until) {
  int sum = 0;
  for (int b = threadIdx.x & 31; b < until; b += 32) sum += counted(steps_of(a, b));
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}
// Steps of a run: CTA c takes run c / hk of key head c % hk.
__device__ __forceinline__ int run_length(const SeqAttnArgs& a, int total) {
  const int runs = a.few_ctas / a.hk;
  return max(static_cast<int>((static_cast<uint32_t>(total) + runs - 1) / static_cast<uint32_t>(runs)), kFewLeast);
}
// Where row r of a CTA's first part or of its last lies (in rows of D).
__device__ __forceinline__ size_t few_row(int64_t cta, int last, int r) {
  return (static_cast<size_t>(cta) * 2 + last) * kFewRows + r;
}

// V rows of a warp's tile that some of its rows must not see (see scrub_rows), and those behind the last token.
template <int D>
__device__ __noinline__ void few_scrub(uint8_t* tile, int key0, int all_see, int m, int* worst, int* any_bad) {
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < kFewKeys * (D / 8); i += 32) {
    const int r = i / (D / 8), c = i % (D / 8), key = key0 + r;
    uint4* at = reinterpret_cast<uint4*>(tile + few_at<D>(r, c));
    if (key >= m) {
      *at = make_uint4(0, 0, 0, 0);
    } else if (key >= all_see && not_finite(*at)) {
      uint16_t* e = reinterpret_cast<uint16_t*>(at);
      for (int k = 0; k < 8; ++k)
        if ((e[k] & 0x7F80u) == 0x7F80u) {
          e[k] = 0;
          atomicMin(worst + c * 8 + k, key);
          *any_bad = 1;
        }
    }
  }
  fence_proxy_async_smem();  // a copy follows these writes
  __syncwarp();
}

// What a warp carries from one call of few_rows to the next: the parity of each stage's next phase.
struct FewTurns {
  uint32_t bits;
};

// Keys [k_begin, k_end) of one sequence and key head; `part`: the row of the parts that takes the result, or -1 where these are
// all its keys.  N: 1 for up to 8 rows, 2 for up to 16.  False where a wait gave up.
template <int D, int N>
__device__ __forceinline__ bool few_rows(const SeqAttnArgs& a, const CUtensorMap* tm_k, const CUtensorMap* tm_v, uint8_t* smem,
                                         FewShared* sh, FewTurns& turns, const Segment& seg, int b, int hk, int k_begin, int k_end,
                                         int64_t part) {
  using C = FewCfg<D>;
  constexpr int kStages = C::kStages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = seg.n * a.group;
  const int* table = a.tables + static_cast<int64_t>(b) * a.table_width;
  uint8_t* ring = smem + warp * C::kRing;
  const uint32_t ring_s = smem_addr(ring);
  const int g = lane >> 2, t = lane & 3;  // fragments: the lane's keys (or columns) g, g + 8, its rows 2t, 2t + 1
  const int n_tiles = (k_end - k_begin + kFewKeys - 1) / kFewKeys;
  const int all_see = keys_seen(seg, 0, a.causal);
  for (int i = threadIdx.x; i < D; i += kFewThreads) sh->worst[i] = INT32_MAX;
  if (threadIdx.x == 0) sh->any_bad = 0;
  constexpr int kChunks = D / 8, kQ = (8 * N * kChunks + kFewThreads - 1) / kFewThreads;
  uint4 q[kQ];
#pragma unroll
  for (int i = 0; i < kQ; ++i) {
    const int r = (threadIdx.x + i * kFewThreads) / kChunks, c = (threadIdx.x + i * kFewThreads) % kChunks;
    q[i] = make_uint4(0, 0, 0, 0);
    if (r < rows && c * 8 < a.head_dim)
      q[i] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q.ptr) +
                                            (static_cast<int64_t>(seg.q0) + r / a.group) * a.q.stride_t +
                                            (hk * a.group + r % a.group) * a.q.stride_h)[c];
  }

  // ---------------- copies: lane `op` copies box (piece of the tile's keys, 64 columns, K or V)
  const int box_rows = min(a.page_rows, kFewKeys), pieces = kFewKeys / box_rows;
  const int piece = lane % pieces, half = lane / pieces % (D / 64), is_v = lane / (pieces * (D / 64));
  const bool copies = is_v < 2;
  const uint64_t policy = read_once_policy();
  auto page_of = [&](int i) -> int {  // of this lane's box of tile i; -1: none
    const int key = k_begin + i * kFewKeys + piece * box_rows;
    if (!copies || i >= n_tiles || key >= k_end) return -1;
    const int p = table[key >> a.page_shift];
    return p >= 0 && p < a.n_pages ? p : -1;
  };
  uint32_t gone = 0;  // two bits a stage: halves of its tile without a page
  auto load = [&](int i, int page, int stage) {
    const uint32_t lost = ~__ballot_sync(0xffffffffu, page >= 0);
    const uint32_t bits = pieces == 2 ? lost & 3u : (lost & 1u) * 3u;
    gone = (gone & ~(3u << (2 * stage))) | bits << (2 * stage);
    if (lane == 0) mbar_arrive_expect_tx(&sh->full[warp][stage], 2 * C::kTile);
    __syncwarp();
    if (copies) {
      const int key = k_begin + i * kFewKeys + piece * box_rows;
      tma_load_4d(ring + (2 * stage + is_v) * C::kTile + half * C::kBlock + piece * box_rows * 128, is_v ? tm_v : tm_k,
                  &sh->full[warp][stage], half * 64, key & ((1 << a.page_shift) - 1), hk, page < 0 ? a.n_pages : page, policy);
    }
  };
  int next;
  {
    int first[kStages];
#pragma unroll
    for (int s = 0; s < kStages; ++s) first[s] = page_of(warp + s * kFewWarps);
    next = page_of(warp + kStages * kFewWarps);
#pragma unroll
    for (int s = 0; s < kStages; ++s)
      if (warp + s * kFewWarps < n_tiles) load(warp + s * kFewWarps, first[s], s);
  }

  // ---------------- Q rows as second operands: row g (+ 8), columns 16 k + 2t .. and + 8
#pragma unroll
  for (int i = 0; i < kQ; ++i) {
    const int r = (threadIdx.x + i * kFewThreads) / kChunks, c = (threadIdx.x + i * kFewThreads) % kChunks;
    if (r < 8 * N) sh->q[r][c] = q[i];
  }
  __syncthreads();
  uint32_t qf[N][D / 16][2];
  int lim[N][2];  // keys that rows 2t, 2t + 1 (+ 8) see
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int k = 0; k < D / 16; k += 2) {
      uint32_t f[4];
      ldmatrix4(smem_addr(&sh->q[8 * n + (lane & 7)][2 * k + (lane >> 3)]), f);
      qf[n][k][0] = f[0], qf[n][k][1] = f[1], qf[n][k + 1][0] = f[2], qf[n][k + 1][1] = f[3];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 2 * t + e + 8 * n;
      lim[n][e] = row < rows ? keys_seen(seg, row / a.group, a.causal) : 0;
    }
  }
  float o[N][D / 16][4];
  float m_run[N][2], l_run[N][2];
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o[n][d][0] = o[n][d][1] = o[n][d][2] = o[n][d][3] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) m_run[n][e] = -INFINITY, l_run[n][e] = 0.f;
  }

  bool ok = true;
  int stage = 0;
  for (int i = warp; i < n_tiles; i += kFewWarps) {
    ok = __all_sync(0xffffffffu, mbar_wait(&sh->full[warp][stage], turns.bits >> stage & 1u, &sh->abort_flag, a.status, kErrAttnWait));
    if (!ok) break;
    turns.bits ^= 1u << stage;
    const int key0 = k_begin + i * kFewKeys;
    const uint32_t ks = ring_s + 2 * stage * C::kTile, vs = ks + C::kTile;
    const uint32_t lost = gone >> (2 * stage) & 3u;
    // S^T: keys g, g + 8 by rows 2t, 2t + 1; two sums of each, so that no product waits for the one before it
    float s[N][4];
    {
      float u[N][4];
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = u[n][e] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t f[4];  // (keys 0-7, columns 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15)
        ldmatrix4(ks + few_at<D>((lane & 7) + ((lane >> 3 & 1) << 3), 2 * k + (lane >> 4)), f);
#pragma unroll
        for (int n = 0; n < N; ++n) mma_bf16(k & 1 ? u[n] : s[n], f, qf[n][k][0], qf[n][k][1]);
      }
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = (s[n][e] + u[n][e]) * a.scale_log2;
    }
    const bool part_seen = key0 + kFewKeys > all_see || lost;
    if (part_seen) {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + g + 8 * (e >> 1);
          if (key >= lim[n][e & 1] || (lost >> (e >> 1) & 1u)) s[n][e] = -INFINITY;
        }
    }
    bool up = false;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) up |= fmaxf(s[n][e], s[n][e + 2]) > m_run[n][e] + kFewThreshold;
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(s[n][e], s[n][e + 2]);
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
          if (mx > m_run[n][e] + kFewThreshold) {  // also from -inf, where the factor is 0
            const float f = fast_exp2(m_run[n][e] - mx);
            m_run[n][e] = mx;
            l_run[n][e] *= f;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) o[n][d][e] *= f, o[n][d][e + 2] *= f;
          }
        }
    }
    // P^T as bf16 pairs (each weight is off by at most 2^-8 of itself), turned: rows g by keys 2t, 2t + 1 and + 8
    uint32_t pf[N][2];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float m = m_run[n][e & 1] == -INFINITY ? 0.f : m_run[n][e & 1];  // a row that has seen no key yet: exp2(-inf - 0) = 0
        p[e] = fast_exp2(s[n][e] - m);
        l_run[n][e & 1] += p[e];
      }
      pf[n][0] = turn8x8(pack_bf16x2(p[0], p[1])), pf[n][1] = turn8x8(pack_bf16x2(p[2], p[3]));
    }
    if (part_seen) few_scrub<D>(ring + (2 * stage + 1) * C::kTile, key0, all_see, seg.m, sh->worst, &sh->any_bad);
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      uint32_t f[4];  // V^T: columns g, g + 8 by keys 2t, 2t + 1 (registers 0, 1), + 8 (2, 3)
      ldmatrix4_trans(vs + few_at<D>((lane & 7) + ((lane >> 4) << 3), 2 * d + (lane >> 3 & 1)), f);
#pragma unroll
      for (int n = 0; n < N; ++n) mma_bf16(o[n][d], f, pf[n][0], pf[n][1]);
    }
    __syncwarp();
    // the stage takes the tile kStages steps ahead
    const int ahead = i + kStages * kFewWarps;
    if (ahead < n_tiles) load(ahead, next, stage);
    next = page_of(ahead + kFewWarps);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  if (!ok) {  // give the copies already issued a bounded chance to land
    int never = 0;
    for (int s = 0; s < kStages; ++s) mbar_wait(&sh->full[warp][s], turns.bits >> s & 1u, &never, a.status, 0);
  }

  // ---------------- the warps' parts, over their rings: maximum and sum of 16 rows, then the rows
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l_run[n][e] += __shfl_xor_sync(0xffffffffu, l_run[n][e], x);
  __syncthreads();
  if (*reinterpret_cast<volatile int*>(&sh->abort_flag)) return false;
  float* parts = reinterpret_cast<float*>(smem);
  float* mine = parts + warp * kFewRows * (D + 2);
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 2 * t + e + 8 * n;
      if (g == 0) mine[r * 2] = m_run[n][e], mine[r * 2 + 1] = l_run[n][e];
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        mine[2 * kFewRows + r * D + 16 * d + g] = o[n][d][e];
        mine[2 * kFewRows + r * D + 16 * d + 8 + g] = o[n][d][e + 2];
      }
    }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 2); i += kFewThreads) {
    const int r = i / (D / 2), col = (i % (D / 2)) * 2;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) top = fmaxf(top, parts[w * kFewRows * (D + 2) + r * 2]);
    float sum = 0.f, x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      const float* p = parts + w * kFewRows * (D + 2);
      // no maximum: no keys or scores that are all -inf, and zeros, or scores that are all NaN, and NaN
      const float e = p[r * 2] == -INFINITY ? 1.f : fast_exp2(p[r * 2] - top);
      const float2 v = *reinterpret_cast<const float2*>(p + 2 * kFewRows + r * D + col);
      sum += e * p[r * 2 + 1], x += e * v.x, y += e * v.y;
    }
    bool no_weights = false;  // no sum: does the row see a key that has a page?  (A warp's lanes work on one row.)
    if (sum == 0.f) {
      const int end = min(keys_seen(seg, r / a.group, a.causal), k_end);
      for (int p0 = k_begin >> a.page_shift; end > k_begin && (p0 << a.page_shift) < end; p0 += 32) {
        const int p = p0 + lane;
        no_weights |= (p << a.page_shift) < end && static_cast<unsigned>(table[p]) < static_cast<unsigned>(a.n_pages);
      }
      no_weights = __any_sync(0xffffffffu, no_weights);
    }
    const float inv = sum == 0.f ? (no_weights && part < 0 ? __int_as_float(0x7FC00000) : 0.f) : 1.f / sum;
    x *= inv, y *= inv;
    if (sh->any_bad) {
      const int l = keys_seen(seg, r / a.group, a.causal);
      if (sh->worst[col] < l) x = __int_as_float(0x7FC00000);
      if (sh->worst[col + 1] < l) y = __int_as_float(0x7FC00000);
    }
    const int64_t tok = static_cast<int64_t>(seg.q0) + r / a.group;
    const int head = hk * a.group + r % a.group;
    const float lse2 = sum == 0.f ? (!no_weights ? -INFINITY : part < 0 ? __int_as_float(0x7FC00000) : kNoWeights) : top + log2f(sum);
    if (part >= 0) {
      const size_t at = static_cast<size_t>(part) + r;
      *reinterpret_cast<float2*>(a.few_part + at * D + col) = make_float2(x, y);
      if (col == 0) a.few_lse[at] = lse2;
    } else {
      if (col < a.head_dim)
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out.ptr) + tok * a.out.stride_t + head * a.out.stride_h + col) =
            pack_bf16x2(x, y);
      if (col == 0 && a.lse) a.lse[tok * a.hq + head] = lse2 * kLn2;
    }
  }
  fence_proxy_async_smem();  // the rings' next copies follow these reads and writes
  __syncthreads();
  return true;
}

// A CTA's share.
template <int D>
__device__ __forceinline__ void few_share(const SeqAttnArgs& a, const CUtensorMap* tm_k, const CUtensorMap* tm_v, uint8_t* smem,
                                          FewShared* sh) {
  FewTurns turns = {0};
  Segment seg;
  auto segment = [&](int b) {
    clip_segment(a.cu_q, b, a.tokens_q, seg.q0, seg.n);
    seg.k0 = 0, seg.m = min(max(a.kv_lens[b], 0), a.max_keys);
  };
  if (a.few_whole) {
    const int hk = blockIdx.x % a.hk, b = blockIdx.x / a.hk;
    segment(b);
    if (seg.n == 0 || seg.n > a.few_tokens) return;
    if (seg.n * a.group <= 8)
      few_rows<D, 1>(a, tm_k, tm_v, smem, sh, turns, seg, b, hk, 0, seg.m, -1);
    else
      few_rows<D, 2>(a, tm_k, tm_v, smem, sh, turns, seg, b, hk, 0, seg.m, -1);
    return;
  }
  const int lane = threadIdx.x & 31;
  // the sequence of the run's first step and the steps before it: 32 sequences at a time, again from the start where these
  // are not all
  int total = 0, mine = 0, sum = 0;
  for (int b = 0; b < a.batch; b += 32) {
    mine = sum = b + lane < a.batch ? counted(steps_of(a, b + lane)) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    total += __shfl_sync(0xffffffffu, sum, 31);
  }
  const int hk = blockIdx.x % a.hk, run = run_length(a, total);
  const int64_t begin64 = static_cast<int64_t>(blockIdx.x / a.hk) * run;
  if (begin64 >= total) return;
  const int begin = static_cast<int>(begin64), end = static_cast<int>(min(static_cast<int64_t>(total), begin64 + run));
  int base = 0, b0 = 0;
  for (; b0 < a.batch; b0 += 32) {
    if (a.batch > 32) {
      mine = sum = b0 + lane < a.batch ? counted(steps_of(a, b0 + lane)) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
    }
    const unsigned after = __ballot_sync(0xffffffffu, base + sum > begin);
    if (after) {
      const int l = __ffs(after) - 1;
      base += __shfl_sync(0xffffffffu, sum - mine, l);
      b0 += l;
      break;
    }
    base += __shfl_sync(0xffffffffu, sum, 31);
  }
  int at = begin;
  for (int b = b0; at < end && b < a.batch; ++b) {
    const int steps = steps_of(a, b);
    if (steps == 0) continue;
    const int first = max(at - base - kFewStart, 0), last = min(end - base - kFewStart, steps);
    const bool later = at > begin;
    base += steps + kFewStart;
    at = base;
    if (first >= last) continue;  // only its start lies in this run
    segment(b);
    const bool whole = first == 0 && last == steps;
    const int64_t part = whole ? -1 : static_cast<int64_t>(few_row(blockIdx.x, later, 0));
    const int k0 = first * kFewStep, k1 = min(seg.m, last * kFewStep);
    const bool ok = seg.n * a.group <= 8 ? few_rows<D, 1>(a, tm_k, tm_v, smem, sh, turns, seg, b, hk, k0, k1, part)
                                         : few_rows<D, 2>(a, tm_k, tm_v, smem, sh, turns, seg, b, hk, k0, k1, part);
    if (!ok) return;
  }
}

template <int D>
__global__ void __launch_bounds__(kFewThreads, 2)
    paged_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ SeqAttnArgs a) {
  extern __shared__ uint8_t few_raw[];
  __shared__ FewShared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(few_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  if (threadIdx.x == 0) {
    for (int w = 0; w < kFewWarps; ++w)
      for (int s = 0; s < FewCfg<D>::kStages; ++s) mbar_init(&sh.full[w][s], 1);
    sh.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  __syncthreads();
  // Behind the tile kernel, which waited for what this one reads before it let this one start: the two work beside one another,
  // and only the end of this one waits for the other's.
  if (!a.few_behind) pdl_wait();
  pdl_trigger();
  if (a.clear && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  few_share<D>(a, &tm_k, &tm_v, smem, &sh);
  if (a.few_behind) pdl_wait();
}

// out = sum_p 2^(L_p - L) O_p, L = log2 sum_p 2^L_p, of the parts p of a row: parts first, first + step, ... by one warp, a lane D / 32
// columns; `top` is the largest L_p of all.
template <int D, typename Row>
__device__ __forceinline__ void add_parts(const float* part, const float* part_lse, int first, int step, int parts, Row row_of,
                                          float top, float& sum, float (&v)[D / 32]) {
  constexpr int kCols = D / 32;
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int p = first; p < parts; p += step) {
    const size_t row = row_of(p);
    const float l = part_lse[row];
    const float* src = part + row * D + lane * kCols;
    float u[kCols];
    if constexpr (kCols == 4) {
      const float4 w = *reinterpret_cast<const float4*>(src);
      u[0] = w.x, u[1] = w.y, u[2] = w.z, u[3] = w.w;
    } else {
      const float2 w = *reinterpret_cast<const float2*>(src);
      u[0] = w.x, u[1] = w.y;
    }
    // a part without keys counts for nothing, NaN log-sums (NaN scores) reach the output
    const float e = l == -INFINITY ? 0.f : fast_exp2(l - top);
    sum += e;
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[i] += l == -INFINITY ? 0.f : e * u[i];
  }
}
template <int D>
__device__ __forceinline__ void write_joined(const SeqAttnArgs& a, int64_t tok, int head, float top, float sum, const float (&v)[D / 32]) {
  constexpr int kCols = D / 32;
  const int lane = threadIdx.x & 31, col = lane * kCols;
  if (top == kNoWeights) sum = __int_as_float(0x7FC00000);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out.ptr) + tok * a.out.stride_t + head * a.out.stride_h + col;
  if (col < a.head_dim)
#pragma unroll
    for (int i = 0; i < kCols; i += 2) *reinterpret_cast<uint32_t*>(dst + i) = pack_bf16x2(v[i] * inv, v[i + 1] * inv);
  if (lane == 0 && a.lse) a.lse[static_cast<size_t>(tok) * a.hq + head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}
template <typename Row>
__device__ __forceinline__ float top_of(const float* part_lse, int first, int step, int parts, Row row_of) {
  float top = -INFINITY;
  for (int p = first; p < parts; p += step) top = fmaxf(top, part_lse[row_of(p)]);
  return warp_max(top);
}

constexpr int kJoinWarps = 8;
constexpr int kJoinAlone = 16;  // so many parts of a row one warp adds by itself

// The rows of paged_few_kernel whose steps several CTAs took: blockIdx.x a sequence and key head.
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_few_join_kernel(const __grid_constant__ SeqAttnArgs a) {
  __shared__ float s_sum[kJoinWarps], s_top[kJoinWarps];
  __shared__ float s_out[kJoinWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The lengths were there before paged_few_kernel let this one start; its parts are there after pdl_wait(), which no CTA
  // returns without: the kernel behind this one waits for this one alone.
  const int b = blockIdx.x / a.hk, hk = blockIdx.x % a.hk;
  Segment seg;
  clip_segment(a.cu_q, b, a.tokens_q, seg.q0, seg.n);
  const int steps = steps_of(a, b), rows = steps > 0 ? seg.n * a.group : 0;
  const int run = run_length(a, steps_before(a, a.batch)), first = steps_before(a, b);
  const int run0 = (first + kFewStart) / run, run1 = (first + kFewStart + steps - 1) / run;
  pdl_wait();
  pdl_trigger();
  if (steps == 0 || run0 == run1) return;
  // the first run began before this sequence: its later part
  const bool behind = first > run0 * run;
  const int parts = run1 - run0 + 1;
  const bool alone = parts <= kJoinAlone;
  const int step = alone ? kJoinWarps * gridDim.y : gridDim.y;
  for (int r = alone ? blockIdx.y * kJoinWarps + warp : blockIdx.y; r < rows; r += step) {
    auto row_of = [&](int p) { return few_row(static_cast<int64_t>(run0 + p) * a.hk + hk, p == 0 && behind, r); };
    const int64_t tok = static_cast<int64_t>(seg.q0) + r / a.group;
    const int head = hk * a.group + r % a.group;
    constexpr int kCols = D / 32;
    float sum = 0.f, v[kCols] = {};
    if (alone) {
      const float top = top_of(a.few_lse, lane, 32, parts, row_of);
      add_parts<D>(a.few_part, a.few_lse, 0, 1, parts, row_of, top, sum, v);
      write_joined<D>(a, tok, head, top, sum, v);
      continue;
    }
    // all warps: each every eighth part, then the warps' sums in order
    float top = top_of(a.few_lse, threadIdx.x, kJoinWarps * 32, parts, row_of);
    if (lane == 0) s_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_top[w]);
    add_parts<D>(a.few_part, a.few_lse, warp, kJoinWarps, parts, row_of, top, sum, v);
#pragma unroll
    for (int i = 0; i < kCols; ++i) s_out[warp][lane * kCols + i] = v[i];
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      for (int w = 1; w < kJoinWarps; ++w) {
        sum += s_sum[w];
#pragma unroll
        for (int i = 0; i < kCols; ++i) v[i] += s_out[w][lane * kCols + i];
      }
      write_joined<D>(a, tok, head, top, sum, v);
    }
    __syncthreads();
  }
}

// A row's parts of the tile kernel, by eight lanes.  Read in L2: see paged_join_kernel.
template <int D>
__device__ __forceinline__ void add_tile_parts(const SeqAttnArgs& a, int64_t item, int tok, int head, int lane, int parts) {
  constexpr int kCols = D / 32;  // float4 of a lane
  const size_t stride = static_cast<size_t>(a.tokens_q) * a.hq;
  float top = -INFINITY;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) top = fmaxf(top, __ldcg(&a.part_lse[p * stride + item]));
  float sum = 0.f;
  float4 v[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int p = 0; p < parts; ++p) {
    const float l = __ldcg(&a.part_lse[p * stride + item]);
    const float4* src = reinterpret_cast<const float4*>(a.part + (p * stride + item) * D) + lane;
    float4 u[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) u[i] = __ldcg(src + 8 * i);
    if (l == -INFINITY) continue;  // no keys: counts for nothing; a NaN reaches the output
    const float e = fast_exp2(l - top);
    sum += e;
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[i].x += e * u[i].x, v[i].y += e * u[i].y, v[i].z += e * u[i].z, v[i].w += e * u[i].w;
  }
  if (top == kNoWeights) sum = __int_as_float(0x7FC00000);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out.ptr) + static_cast<int64_t>(tok) * a.out.stride_t + head * a.out.stride_h;
#pragma unroll
  for (int i = 0; i < kCols; ++i) {
    const int col = 32 * i + 4 * lane;
    if (col < a.head_dim)
      *reinterpret_cast<uint2*>(dst + col) = make_uint2(pack_bf16x2(v[i].x * inv, v[i].y * inv), pack_bf16x2(v[i].z * inv, v[i].w * inv));
  }
  if (lane == 0 && a.lse) a.lse[item] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// The rows of the tile kernel whose keys were split: a warp to four of them, so that enough reads are on their way (a warp to
// each: 17 against 12 us for two parts of 32000 rows of 128).
constexpr int kJoinRows = 4 * kJoinWarps;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const __grid_constant__ SeqAttnArgs a) {
  const int lane = threadIdx.x & 7;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kJoinRows + (threadIdx.x >> 3);
  const int tok = static_cast<int>(item / a.hq), head = static_cast<int>(item % a.hq);
  // the last sequence that starts at or before the token (empty ones before it share its start), by all lanes for each token
  int b = 0;
  for (int r = 0, found = -1; r < 32; r += 8) {
    const int t = __shfl_sync(0xffffffffu, tok, r);
    if (t == found || t >= a.tokens_q) continue;
    found = t;
    const int x = find_segment(a.batch, t, [&](int i) { return min(max(a.cu_q[i], 0), a.tokens_q); });
    if (tok == t) b = x;
  }
  int parts = 0;
  if (tok < a.tokens_q) {
    Segment seg;
    clip_segment(a.cu_q, b, a.tokens_q, seg.q0, seg.n);
    if (tok >= seg.q0 && tok < seg.q0 + seg.n && seg.n > a.few_tokens)
      parts = (min(max(a.kv_lens[b], 0), a.max_keys) + a.split_keys - 1) / a.split_keys;
  }
  // No thread returns without waiting (see paged_few_join_kernel).  Behind that one, which let this one start when the tile kernel
  // had ended, the two work beside one another and the end waits: the parts are complete, and are read in L2, as no wait of this
  // kernel's has made them visible to its SM.
  if (!a.join_beside) pdl_wait();
  if (parts > 1) add_tile_parts<D>(a, item, tok, head, lane, parts);
  if (a.join_beside) pdl_wait();
}

template <int D>
cudaError_t launch_few_dim(const SeqAttnArgs& a, const SeqAttnMaps& m, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(paged_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, FewCfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged_few_kernel<D>, dim3(a.few_ctas), dim3(kFewThreads), FewCfg<D>::kSmem, stream, m.few_k, m.few_v, a);
  if (e != cudaSuccess || a.few_whole) return e;
  count_launch();
  // a CTA to a sequence and key head, more where these are few and their parts many
  const int all = a.batch * a.hk, more = std::max(1, std::min(a.few_join_rows, 2 * num_sms() / all));
  return launch_pdl(paged_few_join_kernel<D>, dim3(all, more), dim3(kJoinWarps * 32), 0, stream, a);
}

}  // namespace

cudaError_t launch_paged_few(const SeqAttnArgs& a, const SeqAttnMaps& m, cudaStream_t stream) {
  const cudaError_t e = a.head_dim <= 64 ? launch_few_dim<64>(a, m, stream) : launch_few_dim<128>(a, m, stream);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_paged_join(const SeqAttnArgs& a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.tokens_q) * a.hq + kJoinRows - 1) / kJoinRows)), block(kJoinWarps * 32);
  const cudaError_t e = a.head_dim <= 64 ? launch_pdl(paged_join_kernel<64>, grid, block, 0, stream, a)
                                         : launch_pdl(paged_join_kernel<128>, grid, block, 0, stream, a);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace mmdit
