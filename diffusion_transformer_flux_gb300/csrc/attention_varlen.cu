// attention_varlen.cu -- attention over packed sequences, or over a paged cache, on tcgen05 tensor cores.
//
// Per sequence of n queries and m keys, and per query head h with its key head h / (Hq / Hk):
//   z_ij = scale q_i . k_j over the keys j that query i sees (all, or with `causal` those up to its position m - n + i),
//   out_i = sum_j exp(z_ij - lse_i) v_j,   lse_i = log sum_j exp(z_ij);   a row that sees no key gives 0 and -inf.
//
// The query heads of a group read the same keys, so a tile's 128 rows are 128 / group tokens by the group's heads (row
// r is token r / group, head r % group): a key tile is loaded once for all of them, and a short chunk of new tokens
// fills a tile `group` times as well.  A CTA owns two such tiles (A and B, consecutive tokens) of one key head and walks
// the keys in tiles of 128 with an online softmax.  The CTAs find their sequence by a search in cu_q: sequence b's
// first tile pair is number cu_q[b] / (2 tokens) + b, which leaves each at least as many numbers as it needs without a
// prefix sum; numbers that are left over end at once.  Tiles with the most keys have the lowest block numbers.
//
// Twelve warps:
//   warp 0       TMA: both Q tiles once, then K and V tiles into a ring (in a paged cache a lane for each page of a tile)
//   warp 1       MMA issuer: S_A(0) S_B(0) | PV_A(j) S_A(j+1) PV_B(j) S_B(j+1) | ..., so that the tensor core works on one
//                query tile while the softmax of the other runs
//   warps 2, 3   tiles of V that part of the rows must not see: see scrub_rows
//   warps 4..7   softmax of tile A, warps 8..11 of tile B: one query row per thread.  P = exp2(S c - m) goes back over the
//                score columns as bf16 pairs (V is bf16 and one product's operands have one type; each weight is off by at
//                most 2^-9 of itself), from where the PV product reads it.  The row's sum is of the unrounded weights,
//                in float32: it is also the returned lse.  The running maximum only moves (and O is
//                rescaled in TMEM) when a row's maximum grows by more than 2^8.
// TMEM columns: S/P of A [0,128), S/P of B [128,256), O of A [256,256+D), O of B [384,384+D).
// V is read as it lies ([key][d], MN-major), K and Q K-major.  Heads of up to 64 run with D = 64, up to 128 with D = 128;
// columns behind head_dim are zeros that the TMA fills in.
//
// Over a paged cache the keys of a CTA's tile may be split over gridDim.y CTAs (few rows, long contexts); each then writes
// its part normalised in float32 with its log-sum, and paged_combine_kernel joins them.
#include "attention_tiles.cuh"

namespace mmdit {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;  // in log2 units

template <int D>
struct Cfg {
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kTileBytes = (D / 64) * kSeqBlock;
  static constexpr int kData = (2 + 2 * kStages) * kTileBytes;
  static constexpr int kSmem = kData + 1024 + 1024;
  static constexpr uint32_t kIdescS = make_idesc<kKindF16>(128, 128);
  static constexpr uint32_t kIdescPV = make_idesc<kKindF16>(128, D) | kIdescBMnMajor;
};

template <int D>
struct Barriers {
  uint64_t q_full;
  uint64_t k_full[Cfg<D>::kStages];
  uint64_t v_full[Cfg<D>::kStages];
  uint64_t v_clean[Cfg<D>::kStages];
  uint64_t v_issued[Cfg<D>::kStages];  // tiles to clean: their copies are on the way (so v_full's phase is this tile's)
  uint64_t k_empty[Cfg<D>::kStages];
  uint64_t v_empty[Cfg<D>::kStages];
  uint64_t s_full[2];
  uint64_t p_full[2][2];  // per tile: the weights of its first 64 keys, of its last
  uint64_t o_full[2];
  uint64_t drain;
  uint32_t tmem_slot;
  int abort_flag;
  int any_bad;
  // paged: pieces of tile j whose page does not exist; two rounds of the ring, as a K tile is free before all rows read this
  uint32_t lost_pages[2 * Cfg<D>::kStages];
  int worst[D];
};
static_assert(sizeof(Barriers<128>) <= 1024 && sizeof(Barriers<64>) <= 1024, "barriers");

template <int D, bool PAGED>
__device__ __forceinline__ void softmax_role(Barriers<D>* sb, int X, uint32_t tmem, const SeqAttnArgs& a, const Segment& seg,
                                             int hk, int t0, int cnt, int js, int split, int n_splits, bool last) {
  volatile int* abort_flag = &sb->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;
  const int row = quarter * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t s_cols = tmem + static_cast<uint32_t>(X * 128) + lane_off;
  const uint32_t o_cols = tmem + 256u + static_cast<uint32_t>(X * 128) + lane_off;
  const int tok = t0 + X * a.tile_tokens + row / a.group;  // of the sequence
  const bool valid = row < a.tile_tokens * a.group && tok < seg.n;
  // rows of no token compute on whatever their lines hold and are not stored
  const int lim = valid ? keys_seen(seg, tok, a.causal) : INT32_MAX;
  const float c = a.scale_log2;
  float m_run = -INFINITY, l_run = 0.f;
  for (int j = 0; j < cnt; ++j) {
    const int st = j % Cfg<D>::kStages;
    bool w = mbar_wait(&sb->s_full[X], static_cast<uint32_t>(j) & 1u, abort_flag, a.status, kErrAttnWait);
    // the producer's note on the tile's pages is published with the K tile's barrier
    if (PAGED && w)
      w = mbar_wait(&sb->k_full[st], static_cast<uint32_t>(j / Cfg<D>::kStages) & 1u, abort_flag, a.status, kErrAttnWait);
    if (!__all_sync(0xffffffffu, w)) return;
    tc_fence_after();
    // the products are done in their order: with the last tile's scores of K_j, V_(j-1) is read as well
    if (last && (threadIdx.x & 127) == 0) {
      mbar_arrive(&sb->k_empty[st]);
      if (j > 0) mbar_arrive(&sb->v_empty[(j - 1) % Cfg<D>::kStages]);
    }
    const int rel = lim - (js + j) * kSeqTile;  // keys of this tile that the row sees
    // the 128 scores of this row
    uint32_t r0[32], r1[32], r2[32], r3[32];
    tmem_ld64_wait(s_cols, r0, r1);
    tmem_ld32(s_cols + 64, r2);
    tmem_ld32(s_cols + 96, r3);
    float mx0 = -INFINITY, mx1 = -INFINITY;
    const bool part = __any_sync(0xffffffffu, rel < kSeqTile);
    if (!part) {  // while the second half is on its way
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        mx0 = fmax3(mx0, __uint_as_float(r0[i]), __uint_as_float(r0[i + 1]));
        mx1 = fmax3(mx1, __uint_as_float(r1[i]), __uint_as_float(r1[i + 1]));
      }
    }
    tmem_ld_deps64(r2, r3);
    bool whole = !part;
    if (part) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (i >= rel) r0[i] = __float_as_uint(-INFINITY);
        if (32 + i >= rel) r1[i] = __float_as_uint(-INFINITY);
        if (64 + i >= rel) r2[i] = __float_as_uint(-INFINITY);
        if (96 + i >= rel) r3[i] = __float_as_uint(-INFINITY);
      }
    }
    if (PAGED) {
      const uint32_t lost = *reinterpret_cast<volatile uint32_t*>(&sb->lost_pages[j % (2 * Cfg<D>::kStages)]);
      if (lost) {  // pieces of at least 8 keys
        whole = false;
        uint32_t eights = 0;
        for (int e = 0; e < 16; ++e) eights |= (lost >> (e * 8 / a.page_rows) & 1u) << e;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (eights >> (i / 8) & 1u) r0[i] = __float_as_uint(-INFINITY);
          if (eights >> (4 + i / 8) & 1u) r1[i] = __float_as_uint(-INFINITY);
          if (eights >> (8 + i / 8) & 1u) r2[i] = __float_as_uint(-INFINITY);
          if (eights >> (12 + i / 8) & 1u) r3[i] = __float_as_uint(-INFINITY);
        }
      }
    }
    if (!whole) {
      mx0 = mx1 = -INFINITY;
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        mx0 = fmax3(mx0, __uint_as_float(r0[i]), __uint_as_float(r0[i + 1]));
        mx1 = fmax3(mx1, __uint_as_float(r1[i]), __uint_as_float(r1[i + 1]));
      }
    }
    {
      float mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        mx2 = fmax3(mx2, __uint_as_float(r2[i]), __uint_as_float(r2[i + 1]));
        mx3 = fmax3(mx3, __uint_as_float(r3[i]), __uint_as_float(r3[i + 1]));
      }
      mx0 = fmaxf(mx0, mx2), mx1 = fmaxf(mx1, mx3);
    }
    const float mx = fmaxf(mx0, mx1) * c;
    float alpha = 1.f;
    bool rescale = false;
    if (j == 0) {
      m_run = mx;
    } else if (mx > m_run + kRescaleThreshold) {  // also from -inf, where alpha is 0
      alpha = fast_exp2(m_run - mx);
      m_run = mx;
      rescale = true;
    }
    // O holds sum_{t<j} P_t V_t (PV(j-1) was issued before S(j), whose completion we saw)
    if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
      for (int e = 0; e < D / 16; ++e) {
        uint32_t r[16];
        tmem_ld16_wait(o_cols + e * 16, r);
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
        tmem_st16(o_cols + e * 16, r);
      }
    }
    // a row that has seen no key yet: exp2(-inf - 0) = 0
    const float m_use = m_run == -INFINITY ? 0.f : m_run;
    const uint64_t scale2 = f32x2(c, c);
    const uint64_t negm2 = f32x2(-m_use, -m_use);
    uint64_t sum_a = f32x2(0.f, 0.f), sum_b = f32x2(0.f, 0.f);
    auto emit = [&](const uint32_t (&sc)[32], uint32_t col) {
      uint32_t pk[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x, y;
        f32x2_split(ffma2(f32x2(__uint_as_float(sc[2 * i]), __uint_as_float(sc[2 * i + 1])), scale2, negm2), x, y);
        x = fast_exp2(x), y = fast_exp2(y);
        pk[i] = pack_bf16x2(x, y);
        if (i & 1)
          sum_b = fadd2(sum_b, f32x2(x, y));
        else
          sum_a = fadd2(sum_a, f32x2(x, y));
      }
      tmem_st16(s_cols + col, pk);
    };
    emit(r0, 0);   // keys [0, 32)   -> columns [0, 16)
    emit(r1, 16);  // keys [32, 64)  -> columns [16, 32)
    // the product of these keys may run while the others' weights are formed
    tmem_st_wait();
    tc_fence_before();
    mbar_arrive(&sb->p_full[X][0]);
    emit(r2, 32);  // keys [64, 96)  -> columns [32, 48)
    emit(r3, 48);  // keys [96, 128) -> columns [48, 64)
    float sum;
    {
      float a0, a1, b0, b1;
      f32x2_split(sum_a, a0, a1);
      f32x2_split(sum_b, b0, b1);
      sum = (a0 + a1) + (b0 + b1);
    }
    tmem_st_wait();
    tc_fence_before();
    mbar_arrive(&sb->p_full[X][1]);
    l_run = l_run * alpha + sum;
  }
  if (cnt > 0) {
    const bool w = mbar_wait(&sb->o_full[X], 0, abort_flag, a.status, kErrAttnWait);
    if (!__all_sync(0xffffffffu, w)) return;
    tc_fence_after();
  }
  const float inv_l = l_run == 0.f ? 0.f : 1.f / l_run;
  const float lse2 = l_run == 0.f ? -INFINITY : m_run + log2f(l_run);
  const size_t out_row = valid ? (static_cast<size_t>(seg.q0) + tok) * a.hq + hk * a.group + row % a.group : 0;
  const bool any_bad = sb->any_bad != 0;
  float* part = nullptr;
  __nv_bfloat16* out = nullptr;
  if (valid && n_splits > 1) {
    const size_t at = static_cast<size_t>(split) * a.tokens_q * a.hq + out_row;
    part = a.part + at * D;
    a.part_lse[at] = lse2;
  } else if (valid) {
    out = static_cast<__nv_bfloat16*>(a.out.ptr) + (static_cast<int64_t>(seg.q0) + tok) * a.out.stride_t +
          (hk * a.group + row % a.group) * a.out.stride_h;
    if (a.lse) a.lse[out_row] = lse2 * kLn2;
  }
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    float v[32];
    if (cnt > 0) {
      uint32_t r[32];
      tmem_ld32_wait(o_cols + e * 32, r);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]) * inv_l;
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.f;
    }
    if (any_bad) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (*reinterpret_cast<volatile int*>(&sb->worst[e * 32 + i]) < lim) v[i] = __int_as_float(0x7FC00000);
    }
    if (part)
      store32(part + e * 32, v);
    else if (out && e * 32 < a.head_dim)
      store_cols(out + e * 32, v, a.head_dim - e * 32);
  }
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
    seq_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ SeqAttnArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Barriers<D>* sb = reinterpret_cast<Barriers<D>*>(smem + C::kData);
  volatile int* abort_flag = &sb->abort_flag;
  auto q_tile = [&](int x) { return smem + x * C::kTileBytes; };
  auto k_tile = [&](int st) { return smem + (2 + st) * C::kTileBytes; };
  auto v_tile = [&](int st) { return smem + (2 + C::kStages + st) * C::kTileBytes; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_wait();
  if (a.clear && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.status = 0;
  // ---------------- this CTA's tokens and keys
  const int hk = blockIdx.x % a.hk;
  const int pair = (gridDim.x - 1 - blockIdx.x) / a.hk;
  const int span = 2 * a.tile_tokens;
  const int b = find_segment(a.batch, pair, [&](int i) { return min(max(a.cu_q[i], 0), a.tokens_q) / span + i; });
  Segment seg;
  clip_segment(a.cu_q, b, a.tokens_q, seg.q0, seg.n);
  const int t0 = (pair - (seg.q0 / span + b)) * span;
  if (t0 < 0 || t0 >= seg.n) return;
  int split_tiles = INT32_MAX, n_splits = 1;
  if constexpr (PAGED) {
    if (seg.n * a.group <= a.few_rows) return;  // another kernel's
    seg.k0 = 0, seg.m = min(max(a.kv_lens[b], 0), a.max_keys);
    if (a.split_keys > 0) {
      split_tiles = a.split_keys / kSeqTile;
      n_splits = (seg.m + a.split_keys - 1) / a.split_keys;
      if (blockIdx.y > 0 && static_cast<int>(blockIdx.y) >= n_splits) return;
    }
  } else {
    clip_segment(a.cu_k, b, a.tokens_k, seg.k0, seg.m);
  }
  const int split = blockIdx.y;
  const int js = split * (split_tiles == INT32_MAX ? 0 : split_tiles);
  int cnt[2], bytes_q = 0;  // key tiles of each query tile
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int first = t0 + x * a.tile_tokens, rows = min(seg.n - first, a.tile_tokens);
    const int tiles = rows > 0 ? (keys_seen(seg, first + rows - 1, a.causal) + kSeqTile - 1) / kSeqTile : 0;
    cnt[x] = max(min(tiles - js, split_tiles), 0);
    if (cnt[x] > 0) bytes_q += (D / 64) * a.group * a.tile_tokens * 128;
  }
  const int n_kv = max(cnt[0], cnt[1]);
  const int all_see = keys_seen(seg, t0, a.causal);  // keys that every row of the CTA sees
  auto to_scrub = [&](int j) { return (js + j + 1) * kSeqTile > all_see; };

  if (threadIdx.x == 0) {
    mbar_init(&sb->q_full, 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sb->k_full[s], 1);
      mbar_init(&sb->v_full[s], 1);
      mbar_init(&sb->v_clean[s], 64);
      mbar_init(&sb->v_issued[s], 1);
      mbar_init(&sb->k_empty[s], 1);
      mbar_init(&sb->v_empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sb->s_full[x], 1);
      mbar_init(&sb->p_full[x][0], 128);
      mbar_init(&sb->p_full[x][1], 128);
      mbar_init(&sb->o_full[x], 1);
    }
    mbar_init(&sb->drain, 1);
    sb->abort_flag = 0;
    sb->any_bad = 0;
    fence_mbar_init();
  }
  if (threadIdx.x >= 256) {
    const int i = threadIdx.x - 256;
    if (i < D) sb->worst[i] = INT32_MAX;
  }
  if (warp == 1) {
    tmem_alloc(&sb->tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sb->tmem_slot;

  if (warp == 0) {
    // ---------------- TMA producer
    if (n_kv > 0) {
      if (lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        mbar_arrive_expect_tx(&sb->q_full, bytes_q);
        for (int x = 0; x < 2; ++x)
          if (cnt[x] > 0)
            for (int h = 0; h < D / 64; ++h)
              tma_load_3d(q_tile(x) + h * kSeqBlock, &tm_q, &sb->q_full, h * 64, hk * a.group, seg.q0 + t0 + x * a.tile_tokens);
      }
      int issued = 0;
      const int pieces = PAGED ? kSeqTile / a.page_rows : 1;
      auto page_of = [&](int j) -> int {  // the page of this lane's piece of tile j: -1 behind the last key, -2 if there is none
        const int key = (js + j) * kSeqTile + lane * a.page_rows;
        if (lane >= pieces || key >= seg.m) return -1;
        const int p = a.tables[static_cast<int64_t>(b) * a.table_width + (key >> a.page_shift)];
        return p >= 0 && p < a.n_pages ? p : -2;
      };
      // K runs ahead of V by a tile: it is free once its scores are formed, V when they have been multiplied
      auto empty = [&](uint64_t* bar, int j) {
        const bool w = mbar_wait(bar, (static_cast<uint32_t>(j / C::kStages) & 1u) ^ 1u, abort_flag, a.status, kErrAttnWait);
        return __all_sync(0xffffffffu, w) != 0;
      };
      auto load = [&](uint8_t* tile, const CUtensorMap* map, uint64_t* bar, int j, int page) {
        if constexpr (PAGED) {
          if (lane == 0) mbar_arrive_expect_tx(bar, C::kTileBytes);
          __syncwarp();
          if (lane < pieces) {
            const int z = page < 0 ? a.n_pages : page;  // behind the last page: the box reads zeros
            const int y = ((js + j) * kSeqTile + lane * a.page_rows) & ((1 << a.page_shift) - 1);
            for (int h = 0; h < D / 64; ++h)
              tma_load_4d(tile + h * kSeqBlock + lane * a.page_rows * 128, map, bar, h * 64, y, hk, z);
          }
        } else if (lane == 0) {
          mbar_arrive_expect_tx(bar, C::kTileBytes);
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(tile + h * kSeqBlock, map, bar, h * 64, hk, seg.k0 + (js + j) * kSeqTile);
        }
      };
      int page = PAGED ? page_of(0) : 0, next = PAGED && n_kv > 1 ? page_of(1) : 0;
      int k_issued = 0;
      auto load_k = [&](int j, int p) {
        const int st = j % C::kStages;
        if (!empty(&sb->k_empty[st], j)) return false;
        if constexpr (PAGED) {
          const uint32_t lost = __ballot_sync(0xffffffffu, p == -2);
          if (lane == 0) *reinterpret_cast<volatile uint32_t*>(&sb->lost_pages[j % (2 * C::kStages)]) = lost;
        }
        load(k_tile(st), &tm_k, &sb->k_full[st], j, p);
        k_issued = j + 1;
        return true;
      };
      bool ok = load_k(0, page);
      for (int j = 0; ok && j < n_kv; ++j) {
        const int st = j % C::kStages;
        if (j + 1 < n_kv) ok = load_k(j + 1, next);
        if (!ok || !empty(&sb->v_empty[st], j)) break;
        load(v_tile(st), &tm_v, &sb->v_full[st], j, page);
        if (lane == 0 && to_scrub(j)) mbar_arrive(&sb->v_issued[st]);
        issued = j + 1;
        page = next;
        if (PAGED && j + 2 < n_kv) next = page_of(j + 2);
      }
      if (*abort_flag) {
        // give the copies already issued a bounded chance to land before the CTA exits
        int never = 0;
        mbar_wait(&sb->q_full, 0, &never, a.status, 0);
        for (int t = max(k_issued - C::kStages, 0); t < k_issued; ++t)
          mbar_wait(&sb->k_full[t % C::kStages], static_cast<uint32_t>(t / C::kStages) & 1u, &never, a.status, 0);
        for (int t = max(issued - C::kStages, 0); t < issued; ++t)
          mbar_wait(&sb->v_full[t % C::kStages], static_cast<uint32_t>(t / C::kStages) & 1u, &never, a.status, 0);
      }
    }
  } else if (warp == 1) {
    if (n_kv > 0) {
      // ---------------- MMA issuer: the tensor core's queue is short, so whatever this warp waits for leaves it idle.  The
      // warp's lanes test the barriers of a step side by side, one lane issues.
      // K-step k of a K-major operand tile: 16 elements into its 128-byte swizzle atoms
      auto koff = [](int k) -> uint64_t { return static_cast<uint64_t>(((k >> 2) * kSeqBlock + (k & 3) * 32) >> 4); };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.status, kErrAttnWait)) != 0;
      };
      auto mma_s = [&](int x, int j) {  // S_x(j) = Q_x K_j^T into columns [128x, 128x + 128)
        const uint64_t q_desc = sdesc_kmajor_sw128(smem_addr(q_tile(x)));
        const uint64_t k_desc = sdesc_kmajor_sw128(smem_addr(k_tile(j % C::kStages)));
        const uint32_t d_s = tmem + static_cast<uint32_t>(x * 128);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) tc_mma<kKindF16>(d_s, q_desc + koff(k), k_desc + koff(k), C::kIdescS, k > 0 ? 1u : 0u);
        tc_commit(&sb->s_full[x]);
      };
      auto mma_pv = [&](int x, int j, int half) {  // O_x += P_x(j) V_j over half of the keys, P read from TMEM over S_x
        const uint64_t v_desc = sdesc_mnmajor_sw128(smem_addr(v_tile(j % C::kStages)), kSeqBlock);
        const uint32_t p_cols = tmem + static_cast<uint32_t>(x * 128);  // 16 keys per 8 columns
        const uint32_t d_o = tmem + 256u + static_cast<uint32_t>(x * 128);
#pragma unroll
        for (int k = 4 * half; k < 4 * half + 4; ++k)
          tc_mma_ts_f16(d_o, p_cols + static_cast<uint32_t>(k * 8), v_desc + static_cast<uint64_t>((k * 2048) >> 4), C::kIdescPV,
                        (j > 0 || k > 0) ? 1u : 0u);
      };
      uint32_t cleaned = 0;  // per stage: the parity of its next cleaned tile
      bool ok = wait(lane == 0 ? &sb->q_full : &sb->k_full[0], 0);
      if (ok && one_lane())
        for (int x = 0; x < 2; ++x)
          if (cnt[x] > 0) mma_s(x, 0);
      __syncwarp();
      for (int j = 0; ok && j < n_kv; ++j) {
        const int st = j % C::kStages;
        bool first = true;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok || j >= cnt[x]) continue;
          uint64_t* bar = &sb->p_full[x][0];
          uint32_t parity = static_cast<uint32_t>(j) & 1u;
          if (first) {  // and what both tiles' products of this step read
            if (lane == 1) bar = &sb->v_full[st], parity = static_cast<uint32_t>(j / C::kStages) & 1u;
            if (lane == 2 && j + 1 < n_kv)
              bar = &sb->k_full[(j + 1) % C::kStages], parity = static_cast<uint32_t>((j + 1) / C::kStages) & 1u;
            if (to_scrub(j)) {
              if (lane == 3) bar = &sb->v_clean[st], parity = cleaned >> st & 1u;
              cleaned ^= 1u << st;
            }
            first = false;
          }
          ok = wait(bar, parity);
          if (ok && one_lane()) {
            tc_fence_after();
            mma_pv(x, j, 0);
          }
          __syncwarp();
          ok = ok && wait(&sb->p_full[x][1], static_cast<uint32_t>(j) & 1u);
          if (ok && one_lane()) {
            tc_fence_after();
            mma_pv(x, j, 1);
            if (j + 1 == cnt[x]) tc_commit(&sb->o_full[x]);
            if (j + 1 < cnt[x]) mma_s(x, j + 1);
          }
          __syncwarp();
        }
      }
      if (!ok && one_lane()) {
        // wait (bounded) for every MMA issued so far before TMEM is released
        int never = 0;
        tc_commit(&sb->drain);
        mbar_wait(&sb->drain, 0, &never, a.status, 0);
      }
    }
  } else if (warp < 4) {
    // ---------------- V rows that part of the tile's queries must not see
    uint32_t cleaned = 0;  // per stage: the parity of its next tile to clean
    for (int j = 0; j < n_kv; ++j) {
      if (!to_scrub(j)) continue;
      const int st = j % C::kStages, key = (js + j) * kSeqTile;
      bool w = mbar_wait(&sb->v_issued[st], cleaned >> st & 1u, abort_flag, a.status, kErrAttnWait);
      cleaned ^= 1u << st;
      if (w) w = mbar_wait(&sb->v_full[st], static_cast<uint32_t>(j / C::kStages) & 1u, abort_flag, a.status, kErrAttnWait);
      if (!__all_sync(0xffffffffu, w)) break;
      scrub_rows<D, true>(v_tile(st), kSeqBlock, max(all_see - key, 0), seg.m - key, key, sb->worst, &sb->any_bad,
                          static_cast<int>(threadIdx.x) - 64, 64);
      mbar_arrive(&sb->v_clean[st]);
    }
  } else {
    softmax_role<D, PAGED>(sb, (warp - 4) >> 2, tmem, a, seg, hk, t0, cnt[(warp - 4) >> 2], js, split, n_splits,
                           (warp - 4) >> 2 == (cnt[1] > 0 ? 1 : 0));
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool PAGED>
cudaError_t launch_dim(const SeqAttnArgs& a, const SeqAttnMaps& m, int pairs, int splits, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(seq_attention_kernel<D, PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(seq_attention_kernel<D, PAGED>, dim3(static_cast<unsigned>(pairs) * a.hk, splits), dim3(kThreads),
                    Cfg<D>::kSmem, stream, m.q, m.k, m.v, a);
}

}  // namespace

int seq_tile_tokens(int group) { return kSeqTile / group; }

bool encode_heads_map(CUtensorMap* map, const HeadsView& v, int head_dim, int heads, int64_t tokens, int box_heads, int box_tokens) {
  // a stride of an extent of one is never used; the encoder wants a multiple of 16 bytes all the same
  const uint64_t dims[3] = {static_cast<uint64_t>(head_dim), static_cast<uint64_t>(heads), static_cast<uint64_t>(tokens)};
  const uint64_t strides[2] = {heads > 1 ? static_cast<uint64_t>(v.stride_h) * 2 : 16,
                               tokens > 1 ? static_cast<uint64_t>(v.stride_t) * 2 : 16};
  const uint32_t box[3] = {64, static_cast<uint32_t>(box_heads), static_cast<uint32_t>(box_tokens)};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, v.ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool encode_pages_map(CUtensorMap* map, const PagesView& v, int head_dim, int heads, int n_pages, int page_size, int rows) {
  const uint64_t dims[4] = {static_cast<uint64_t>(head_dim), static_cast<uint64_t>(page_size), static_cast<uint64_t>(heads),
                            static_cast<uint64_t>(n_pages)};
  const uint64_t strides[3] = {static_cast<uint64_t>(v.stride_t) * 2, heads > 1 ? static_cast<uint64_t>(v.stride_h) * 2 : 16,
                               n_pages > 1 ? static_cast<uint64_t>(v.stride_page) * 2 : 16};
  const uint32_t box[4] = {64, static_cast<uint32_t>(rows), 1, 1};
  return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

cudaError_t launch_seq_attention(SeqAttnArgs a, const SeqAttnMaps& m, int paged, int splits, cudaStream_t stream) {
  a.tile_tokens = seq_tile_tokens(a.group);
  const int64_t pairs = a.tokens_q / (2 * a.tile_tokens) + static_cast<int64_t>(a.batch);
  if (pairs * a.hk > INT32_MAX) return cudaErrorInvalidValue;
  const int p = static_cast<int>(pairs);
  cudaError_t e;
  if (a.head_dim <= 64)
    e = paged ? launch_dim<64, true>(a, m, p, splits, stream) : launch_dim<64, false>(a, m, p, splits, stream);
  else
    e = paged ? launch_dim<128, true>(a, m, p, splits, stream) : launch_dim<128, false>(a, m, p, splits, stream);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace mmdit
