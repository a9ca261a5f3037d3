// attention_varlen_bwd.cu -- gradients of the attention over packed sequences, on tcgen05 tensor cores.
//
// With p_ij = exp(z_ij - lse_i) from the forward's lse, delta_i = dout_i . out_i and dz_ij = p_ij (dout_i . v_j - delta_i):
//   dv_j = sum_i p_ij dout_i,   dk_j = scale sum_i dz_ij q_i,   dq_i = scale sum_j dz_ij k_j,
// dk and dv summed over the query heads of a key head's group.  Two passes, one over key tiles and one over query tiles, each
// recompute z and dout . v: seven products where one pass would need five, but that one has to add its dq into
// memory from every key tile, in an order that changes the bits, through float32 traffic of several times the tensors' size.
// Here every sum stays in tensor memory and is written once, in bf16.
//
// Both passes are one kernel, with a resident tile pair F (of 128 rows) and moving tile pairs M:
//   keys:    F = K, V;     M = Q, dO;   S = K Q^T, dP = V dO^T;   dV += P dO,  dK += dS Q     (rows of S are keys)
//   queries: F = Q, dO;    M = K, V;    S = Q K^T, dP = dO V^T;   dQ += dS K                  (rows of S are queries)
// A tile of queries is 128 / group tokens by the group's heads, as in the forward, so the sum over the group's heads is the sum
// over a moving tile's rows.  A moving tile is worked on in halves of 64 rows, so that one half's products run while the
// other half's P and dS are formed.  Twelve warps:
//   warp 0       TMA: F once, then M tiles into two stages
//   warp 1       MMA issuer: S, dP of half h of tile i + 1 follow the accumulating products of half h of tile i
//   warps 2, 3   keys: -lse and -delta of the tile's rows; both: rows that part of the tile must not see (scrub_pair)
//   warps 4..7   half 0: one row of S and dP per thread, P = exp2(c S - L) and dS = P (dP - delta) back into tensor memory as
//                bf16 pairs (the operands of the accumulating products, each off by at most 2^-9 of itself); warps 8..11 half 1
// TMEM columns: S [0,128), dP [128,256), then dV and dK, or dQ, D each.
#include "attention_tiles.cuh"

namespace mmdit {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmP = 0, kTmD = 128, kTmAcc = 256;
constexpr int kStages = 2;

template <int D>
struct Cfg {
  static constexpr int kTileBytes = (D / 64) * kSeqBlock;
  static constexpr int kData = (2 + 2 * kStages) * kTileBytes;
  static constexpr int kSums = kData;                              // keys: per stage -L, then -delta, of 128 rows
  static constexpr int kBar = kSums + kStages * 2 * kSeqTile * 4;
  static constexpr int kSmem = kBar + 512 + 1024;
  static constexpr uint32_t kIdescS = make_idesc<kKindF16>(128, 64);
  static constexpr uint32_t kIdescAcc = make_idesc<kKindF16>(128, D) | kIdescBMnMajor;
};

struct Barriers {
  uint64_t f_full;
  uint64_t st_full[kStages];
  uint64_t st_clean[kStages];
  uint64_t st_empty[kStages];
  uint64_t sums_full[kStages];
  uint64_t st_issued[kStages];  // queries: the copies of a tile to clean are on the way (so st_full's phase is this tile's)
  uint64_t sp_full[2];
  uint64_t pd_full[2];
  uint64_t done;
  uint64_t drain;
  uint32_t tmem_slot;
  int abort_flag;
  int worst;  // the row of M that is not finite and that most rows of F see (keys: the last query row, queries: the first key)
};
static_assert(sizeof(Barriers) <= 512, "barriers");

__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Rows [lo, hi) of a tile that hold a non-finite element become zeros and are noted, rows [zero_from, 128) become zeros.
// Called by 64 threads; eight pieces are in flight in each.
template <int D, bool KEYS>
__device__ __forceinline__ void scrub_pair(uint8_t* tile, int lo, int hi, int zero_from, int first, int* worst, int tid) {
  constexpr int kChunks = D / 8;
  auto at = [&](int i) {
    const int r = i / kChunks, c = i % kChunks;
    return reinterpret_cast<uint4*>(tile + (c >> 3) * kSeqBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4));
  };
  const int stop = min(hi, kSeqTile) * kChunks;
  for (int i0 = lo * kChunks + tid; i0 < stop; i0 += 8 * 64) {
    uint4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = i0 + 64 * u < stop ? *at(i0 + 64 * u) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (not_finite(v[u])) {
        *at(i0 + 64 * u) = make_uint4(0, 0, 0, 0);
        if (KEYS)
          atomicMax(worst, first + (i0 + 64 * u) / kChunks);
        else
          atomicMin(worst, first + (i0 + 64 * u) / kChunks);
      }
  }
  for (int i = max(zero_from, 0) * kChunks + tid; i < kSeqTile * kChunks; i += 64) *at(i) = make_uint4(0, 0, 0, 0);
}

template <int D, bool KEYS>
__global__ void __launch_bounds__(kThreads, 1)
    seq_attention_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                             const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                             const __grid_constant__ SeqAttnBwdArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Barriers* sb = reinterpret_cast<Barriers*>(smem + C::kBar);
  volatile int* abort_flag = &sb->abort_flag;
  auto f_tile = [&](int x) { return smem + x * C::kTileBytes; };
  auto m_tile = [&](int st, int x) { return smem + (2 + 2 * st + x) * C::kTileBytes; };
  auto sums = [&](int st) { return reinterpret_cast<float*>(smem + C::kSums) + st * 2 * kSeqTile; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_wait();
  // ---------------- this CTA's tile
  const int hk = blockIdx.x % a.hk, G = a.group, T = a.tile_tokens;
  Segment seg;
  int first, count;  // first row of F (a key, or a token), moving tiles
  int m_first = 0;   // keys: the first token that sees a key of the tile
  if constexpr (KEYS) {
    const int idx = blockIdx.x / a.hk;  // the first keys have the most queries
    const int b = find_segment(a.batch, idx, [&](int i) { return min(max(a.cu_k[i], 0), a.tokens_k) / kSeqTile + i; });
    clip_segment(a.cu_k, b, a.tokens_k, seg.k0, seg.m);
    clip_segment(a.cu_q, b, a.tokens_q, seg.q0, seg.n);
    first = (idx - (seg.k0 / kSeqTile + b)) * kSeqTile;
    if (first < 0 || first >= seg.m) return;
    m_first = a.causal ? max(first - seg.m + seg.n, 0) : 0;
    count = seg.n > m_first ? (seg.n - m_first + T - 1) / T : 0;
  } else {
    const int idx = (gridDim.x - 1 - blockIdx.x) / a.hk;  // the last queries see the most keys
    const int b = find_segment(a.batch, idx, [&](int i) { return min(max(a.cu_q[i], 0), a.tokens_q) / T + i; });
    clip_segment(a.cu_q, b, a.tokens_q, seg.q0, seg.n);
    clip_segment(a.cu_k, b, a.tokens_k, seg.k0, seg.m);
    first = (idx - (seg.q0 / T + b)) * T;
    if (first < 0 || first >= seg.n) return;
    count = (keys_seen(seg, min(first + T, seg.n) - 1, a.causal) + kSeqTile - 1) / kSeqTile;
  }
  const int lag = seg.m - seg.n;  // query i stands at lag + i
  const int all_see = KEYS ? 0 : keys_seen(seg, first, a.causal);
  // rows of moving tile i: [0, zero_from) are of this sequence, those of [lo, hi) not seen by every row of F
  auto rows_of = [&](int i, int& lo, int& hi, int& zero_from) {
    if constexpr (KEYS) {
      const int t = m_first + i * T, last_key = min(first + kSeqTile, seg.m) - 1;
      zero_from = G * min(T, seg.n - t);
      lo = 0, hi = a.causal ? min(G * min(max(last_key - lag - t, 0), T), zero_from) : 0;
      return zero_from < G * T || hi > 0;
    } else {
      zero_from = min(seg.m - i * kSeqTile, kSeqTile);
      lo = max(all_see - i * kSeqTile, 0), hi = zero_from;
      return (i + 1) * kSeqTile > all_see;
    }
  };

  if (threadIdx.x == 0) {
    mbar_init(&sb->f_full, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sb->st_full[s], 1);
      mbar_init(&sb->st_clean[s], 64);
      mbar_init(&sb->st_empty[s], 1);
      mbar_init(&sb->sums_full[s], 64);
      mbar_init(&sb->st_issued[s], 1);
    }
    for (int h = 0; h < 2; ++h) mbar_init(&sb->sp_full[h], 1), mbar_init(&sb->pd_full[h], 128);
    mbar_init(&sb->done, 1);
    mbar_init(&sb->drain, 1);
    sb->abort_flag = 0;
    sb->worst = KEYS ? -1 : INT32_MAX;
    fence_mbar_init();
  }
  if (KEYS && G * T < kSeqTile) {
    // rows that no box fills: the products that sum over a moving tile's rows read them
    const int rows = kSeqTile - G * T;
    for (int i = threadIdx.x; i < kStages * 2 * (D / 64) * rows * 8; i += kThreads) {
      const int c = i % 8, r = G * T + (i / 8) % rows, blk = i / (8 * rows);
      *reinterpret_cast<uint4*>(smem + 2 * C::kTileBytes + blk * kSeqBlock + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(&sb->tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sb->tmem_slot;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, abort_flag, a.status, kErrAttnWait); };

  if (warp == 0) {
    if (lane == 0 && count > 0) {
      // ---------------- TMA producer
      const CUtensorMap *f0 = KEYS ? &tm_k : &tm_q, *f1 = KEYS ? &tm_v : &tm_do;
      const CUtensorMap *m0 = KEYS ? &tm_q : &tm_k, *m1 = KEYS ? &tm_do : &tm_v;
      tma_prefetch_desc(f0), tma_prefetch_desc(f1), tma_prefetch_desc(m0), tma_prefetch_desc(m1);
      const int bytes_q = (D / 64) * G * T * 128;  // a box of queries
      const int f_head = KEYS ? hk : hk * G, m_head = KEYS ? hk * G : hk;
      const int f_row = KEYS ? seg.k0 + first : seg.q0 + first;
      mbar_arrive_expect_tx(&sb->f_full, 2 * (KEYS ? C::kTileBytes : bytes_q));
      for (int h = 0; h < D / 64; ++h) {
        tma_load_3d(f_tile(0) + h * kSeqBlock, f0, &sb->f_full, h * 64, f_head, f_row);
        tma_load_3d(f_tile(1) + h * kSeqBlock, f1, &sb->f_full, h * 64, f_head, f_row);
      }
      int issued = 0;
      for (int i = 0; i < count; ++i) {
        const int st = i % kStages;
        if (!wait(&sb->st_empty[st], (static_cast<uint32_t>(i / kStages) & 1u) ^ 1u)) break;
        const int row = KEYS ? seg.q0 + m_first + i * T : seg.k0 + i * kSeqTile;
        mbar_arrive_expect_tx(&sb->st_full[st], 2 * (KEYS ? bytes_q : C::kTileBytes));
        for (int h = 0; h < D / 64; ++h) {
          tma_load_3d(m_tile(st, 0) + h * kSeqBlock, m0, &sb->st_full[st], h * 64, m_head, row);
          tma_load_3d(m_tile(st, 1) + h * kSeqBlock, m1, &sb->st_full[st], h * 64, m_head, row);
        }
        int lo, hi, zero_from;
        if (!KEYS && rows_of(i, lo, hi, zero_from)) mbar_arrive(&sb->st_issued[st]);
        issued = i + 1;
      }
      if (*abort_flag) {
        int never = 0;
        mbar_wait(&sb->f_full, 0, &never, a.status, 0);
        for (int t = max(issued - kStages, 0); t < issued; ++t)
          mbar_wait(&sb->st_full[t % kStages], static_cast<uint32_t>(t / kStages) & 1u, &never, a.status, 0);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && count > 0) {
      // ---------------- MMA issuer
      auto koff = [](int k) -> uint64_t { return static_cast<uint64_t>(((k >> 2) * kSeqBlock + (k & 3) * 32) >> 4); };
      const uint64_t df0 = sdesc_kmajor_sw128(smem_addr(f_tile(0))), df1 = sdesc_kmajor_sw128(smem_addr(f_tile(1)));
      uint32_t cleaned = 0;
      auto scores = [&](int i, int h) -> bool {  // S and dP of half h of tile i
        const int st = i % kStages;
        if (h == 0) {
          if (!wait(&sb->st_full[st], static_cast<uint32_t>(i / kStages) & 1u)) return false;
          int lo, hi, zero_from;
          if (rows_of(i, lo, hi, zero_from)) {
            if (!wait(&sb->st_clean[st], cleaned >> st & 1u)) return false;
            cleaned ^= 1u << st;
          }
          tc_fence_after();
        }
        const uint64_t dm0 = sdesc_kmajor_sw128(smem_addr(m_tile(st, 0)) + h * 64 * 128);
        const uint64_t dm1 = sdesc_kmajor_sw128(smem_addr(m_tile(st, 1)) + h * 64 * 128);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma<kKindF16>(tmem + kTmP + 64 * h, df0 + koff(k), dm0 + koff(k), C::kIdescS, k > 0 ? 1u : 0u);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma<kKindF16>(tmem + kTmD + 64 * h, df1 + koff(k), dm1 + koff(k), C::kIdescS, k > 0 ? 1u : 0u);
        tc_commit(&sb->sp_full[h]);
        return true;
      };
      bool ok = wait(&sb->f_full, 0) && scores(0, 0) && scores(0, 1);
      for (int i = 0; ok && i < count; ++i) {
        const int st = i % kStages;
        for (int h = 0; ok && h < 2; ++h) {
          ok = wait(&sb->pd_full[h], static_cast<uint32_t>(i) & 1u);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dm0 = sdesc_mnmajor_sw128(smem_addr(m_tile(st, 0)) + h * 64 * 128, kSeqBlock);
          const uint64_t dm1 = sdesc_mnmajor_sw128(smem_addr(m_tile(st, 1)) + h * 64 * 128, kSeqBlock);
          const uint32_t more = i > 0 || h > 0 ? 1u : 0u;
          if constexpr (KEYS) {
#pragma unroll
            for (int k = 0; k < 4; ++k)  // dV
              tc_mma_ts_f16(tmem + kTmAcc, tmem + kTmP + 64 * h + 8 * k, dm1 + static_cast<uint64_t>((k * 2048) >> 4), C::kIdescAcc,
                            k > 0 ? 1u : more);
#pragma unroll
            for (int k = 0; k < 4; ++k)  // dK
              tc_mma_ts_f16(tmem + kTmAcc + D, tmem + kTmD + 64 * h + 8 * k, dm0 + static_cast<uint64_t>((k * 2048) >> 4),
                            C::kIdescAcc, k > 0 ? 1u : more);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)  // dQ
              tc_mma_ts_f16(tmem + kTmAcc, tmem + kTmP + 64 * h + 8 * k, dm0 + static_cast<uint64_t>((k * 2048) >> 4), C::kIdescAcc,
                            k > 0 ? 1u : more);
          }
          if (h == 1) tc_commit(&sb->st_empty[st]);
          if (i + 1 < count) ok = scores(i + 1, h);
        }
      }
      if (ok) tc_commit(&sb->done);
      if (*abort_flag) {
        int never = 0;
        tc_commit(&sb->drain);
        mbar_wait(&sb->drain, 0, &never, a.status, 0);
      }
    }
  } else if (warp < 4) {
    // ---------------- sums of the moving rows, and rows that part of F must not see
    const int tid = static_cast<int>(threadIdx.x) - 64;
    uint32_t cleaned = 0;  // per stage: the parity of its next tile to clean
    for (int i = 0; i < count; ++i) {
      const int st = i % kStages;
      bool w = true;
      if constexpr (KEYS) {
        w = wait(&sb->st_empty[st], (static_cast<uint32_t>(i / kStages) & 1u) ^ 1u);
        if (!__all_sync(0xffffffffu, w)) break;
        const int t = m_first + i * T, rows = G * min(T, seg.n - t);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = tid + 64 * e;
          float2 s = make_float2(0.f, 0.f);
          if (r < rows) s = a.sums[(static_cast<size_t>(seg.q0) + t + r / G) * a.hq + hk * G + r % G];
          sums(st)[r] = -s.x, sums(st)[kSeqTile + r] = -s.y;
        }
        mbar_arrive(&sb->sums_full[st]);
      }
      int lo, hi, zero_from;
      if (!rows_of(i, lo, hi, zero_from)) continue;
      // (keys: st_empty has told that the stage's previous tile is done)
      if (!KEYS) w = wait(&sb->st_issued[st], cleaned >> st & 1u), cleaned ^= 1u << st;
      if (w) w = wait(&sb->st_full[st], static_cast<uint32_t>(i / kStages) & 1u);
      if (!__all_sync(0xffffffffu, w)) break;
      const int at = KEYS ? G * (m_first + i * T) : i * kSeqTile;
      scrub_pair<D, KEYS>(m_tile(st, 0), lo, hi, zero_from, at, &sb->worst, tid);
      if (KEYS) scrub_pair<D, KEYS>(m_tile(st, 1), lo, hi, zero_from, at, &sb->worst, tid);
      fence_proxy_async_smem();
      mbar_arrive(&sb->st_clean[st]);
    }
  } else {
    // ---------------- P and dS of half h; then the sums
    const int h = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_p = tmem + kTmP + 64 * h + lane_off, t_d = tmem + kTmD + 64 * h + lane_off;
    const uint64_t scale2 = f32x2(a.scale_log2, a.scale_log2);
    // queries: this row's sums and the keys it sees; keys: the first query row (tokens by group) that sees it
    const int tok = first + row / G;
    const bool valid = KEYS ? first + row < seg.m : row < G * T && tok < seg.n;
    const int lim = KEYS || !valid ? 0 : keys_seen(seg, tok, a.causal);
    const int from = !KEYS ? 0 : !valid ? INT32_MAX : a.causal ? G * max(first + row - lag, 0) : 0;
    uint64_t neg_l = 0, neg_d = 0;
    if constexpr (!KEYS) {
      float2 s = make_float2(0.f, 0.f);
      if (valid) s = a.sums[(static_cast<size_t>(seg.q0) + tok) * a.hq + hk * G + row % G];
      neg_l = f32x2(-s.x, -s.x), neg_d = f32x2(-s.y, -s.y);
    }
    bool live = true;
    for (int i = 0; i < count; ++i) {
      const int st = i % kStages;
      bool w = wait(&sb->sp_full[h], static_cast<uint32_t>(i) & 1u);
      if (KEYS && w) w = wait(&sb->sums_full[st], static_cast<uint32_t>(i / kStages) & 1u);
      if (!__all_sync(0xffffffffu, w)) { live = false; break; }
      tc_fence_after();
      // columns [lo, hi) of the tile are seen by this row
      int lo, hi;
      if constexpr (KEYS) {
        const int t = m_first + i * T;
        hi = G * min(T, seg.n - t), lo = from == INT32_MAX ? kSeqTile : max(from - G * t, 0);
      } else {
        lo = 0, hi = lim - i * kSeqTile;
      }
      const bool part = __any_sync(0xffffffffu, lo > 64 * h || hi < 64 * h + 64);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t s[32], d[32];
        tmem_ld32(t_p + 32 * c, s);
        tmem_ld32(t_d + 32 * c, d);
        tmem_ld_deps64(s, d);
        uint32_t pk[16], dk[16];
        const float4* l4 = reinterpret_cast<const float4*>(sums(st) + 64 * h + 32 * c);
        const float4* d4 = reinterpret_cast<const float4*>(sums(st) + kSeqTile + 64 * h + 32 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          uint64_t nl[2] = {neg_l, neg_l}, nd[2] = {neg_d, neg_d};
          if constexpr (KEYS) {
            const float4 x = l4[e], y = d4[e];
            nl[0] = f32x2(x.x, x.y), nl[1] = f32x2(x.z, x.w), nd[0] = f32x2(y.x, y.y), nd[1] = f32x2(y.z, y.w);
          }
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int k = 4 * e + 2 * g;
            float p0, p1, z0, z1;
            f32x2_split(ffma2(f32x2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), scale2, nl[g]), p0, p1);
            p0 = fast_exp2(p0), p1 = fast_exp2(p1);
            f32x2_split(fmul2(f32x2(p0, p1), fadd2(f32x2(__uint_as_float(d[k]), __uint_as_float(d[k + 1])), nd[g])), z0, z1);
            if (part) {
              const int col = 64 * h + 32 * c + k;
              if (col < lo || col >= hi) p0 = z0 = 0.f;
              if (col + 1 < lo || col + 1 >= hi) p1 = z1 = 0.f;
            }
            pk[k / 2] = pack_bf16x2(p0, p1), dk[k / 2] = pack_bf16x2(z0, z1);
          }
        }
        // over columns that were read: packed pairs take half as many
        if constexpr (KEYS) {
          tmem_st16(t_p + 16 * c, pk);
          tmem_st16(t_d + 16 * c, dk);
        } else {
          tmem_st16(t_p + 16 * c, dk);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&sb->pd_full[h]);
    }
    bool w = live;
    if (w && count > 0) w = wait(&sb->done, 0);
    if (__all_sync(0xffffffffu, w)) {
      tc_fence_after();
      const int worst = *reinterpret_cast<volatile int*>(&sb->worst);
      // through the resident tiles' memory, whose products are done
      uint8_t* pieces = smem + (warp - 4) * 32 * 2 * D;
      if (KEYS || D == 128 || h == 0) {
        // keys: half 0 writes dV, half 1 dK; queries: each half 64 columns of dQ
        const HeadsView& out = !KEYS ? a.dq : h ? a.dk : a.dv;
        const int64_t at = KEYS ? (static_cast<int64_t>(seg.k0) + first + row) * out.stride_t + hk * out.stride_h
                                : (static_cast<int64_t>(seg.q0) + tok) * out.stride_t + (hk * G + row % G) * out.stride_h;
        __nv_bfloat16* dst = valid ? static_cast<__nv_bfloat16*>(out.ptr) + at : nullptr;
        const bool bad = valid && (KEYS ? worst >= from : worst < lim);
        const float f = bad ? __int_as_float(0x7FC00000) : KEYS && h == 0 ? 1.f : a.scale;
        const int blocks = KEYS ? D / 64 : 1, block0 = KEYS ? 0 : h;  // of 64 columns
#pragma unroll 1
        for (int k = block0; k < block0 + blocks; ++k) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v[32];
            uint32_t r[32];
            if (count > 0) tmem_ld32_wait(tmem + kTmAcc + (KEYS ? h * D : 0) + k * 64 + e * 32 + lane_off, r);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = count > 0 ? __uint_as_float(r[i]) * f : 0.f;
            put_pieces<64>(pieces, e, v);
          }
          __syncwarp();
          store_rows<64>(pieces, dst ? dst + k * 64 : nullptr, a.head_dim - k * 64);
          __syncwarp();
        }
      }
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// (lse log2(e), dout . out) of every row, float32: 16 lanes to a row.  Rows of no sequence are read and not used.
__global__ void __launch_bounds__(256) seq_sums_kernel(const __grid_constant__ SeqAttnBwdArgs a) {
  pdl_wait();
  if (a.clear && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  const int c = (threadIdx.x & 15) * 8;
  if (row >= static_cast<int64_t>(a.tokens_q) * a.hq) return;
  const int64_t t = row / a.hq, h = row % a.hq;
  float s = 0.f;
  if (c < a.head_dim) {
    const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.dout.ptr) + t * a.dout.stride_t +
                                                    h * a.dout.stride_h + c);
    const uint4 y =
        *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.out.ptr) + t * a.out.stride_t + h * a.out.stride_h + c);
    s = bf16_lo(x.x) * bf16_lo(y.x) + bf16_hi(x.x) * bf16_hi(y.x) + bf16_lo(x.y) * bf16_lo(y.y) + bf16_hi(x.y) * bf16_hi(y.y) +
        bf16_lo(x.z) * bf16_lo(y.z) + bf16_hi(x.z) * bf16_hi(y.z) + bf16_lo(x.w) * bf16_lo(y.w) + bf16_hi(x.w) * bf16_hi(y.w);
  }
  const unsigned half = 0xffffu << (threadIdx.x & 16);
#pragma unroll
  for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(half, s, o);
  if ((threadIdx.x & 15) == 0) a.sums[row] = make_float2(a.lse[row] * kLog2e, s);
}

template <int D, bool KEYS>
cudaError_t launch_pass(const SeqAttnBwdArgs& a, const SeqAttnBwdMaps& m, cudaStream_t stream) {
  const int64_t tiles = (KEYS ? a.tokens_k / kSeqTile : a.tokens_q / a.tile_tokens) + static_cast<int64_t>(a.batch);
  if (tiles * a.hk > INT32_MAX) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(seq_attention_bwd_kernel<D, KEYS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(seq_attention_bwd_kernel<D, KEYS>, dim3(static_cast<unsigned>(tiles * a.hk)), dim3(kThreads), Cfg<D>::kSmem,
                 stream, m.q, m.dout, m.k, m.v, a);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_seq_attention_bwd(const SeqAttnBwdArgs& a, const SeqAttnBwdMaps& m, cudaStream_t stream) {
  cudaError_t e;
  if (a.tokens_q > 0) {
    const int64_t rows = static_cast<int64_t>(a.tokens_q) * a.hq;
    e = launch_pdl(seq_sums_kernel, dim3(static_cast<unsigned>((rows + 15) / 16)), dim3(256), 0, stream, a);
    if (e != cudaSuccess) return e;
    count_launch();
  }
  if (a.tokens_k > 0) {
    e = a.head_dim <= 64 ? launch_pass<64, true>(a, m, stream) : launch_pass<128, true>(a, m, stream);
    if (e != cudaSuccess) return e;
  }
  if (a.tokens_q > 0) {
    e = a.head_dim <= 64 ? launch_pass<64, false>(a, m, stream) : launch_pass<128, false>(a, m, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace mmdit
