// attention_varlen.cu -- attention over packed sequences, or over a paged cache, on tcgen05 tensor cores.
//
// Per sequence of n queries and m keys, and per query head h with its key head h / (Hq / Hk):
//   z_ij = scale q_i . k_j over the keys j that query i sees (all, or with `causal` those up to its position m - n + i),
//   out_i = sum_j exp(z_ij - lse_i) v_j,   lse_i = log sum_j exp(z_ij);   a row that sees no key gives 0 and -inf,
// one whose scores are all -inf NaN.
//
// The query heads of a group read the same keys, so a tile's 128 rows are 128 / group tokens by the group's heads (row
// r is token r / group, head r % group): a key tile is loaded once for all of them, and a short chunk of new tokens
// fills a tile `group` times as well.  A work item is two such tiles (A and B, consecutive tokens) of one key head, which walk
// the keys in tiles of 128 with an online softmax.  Items with the most keys come first (TileOrder); one CTA to an SM takes its
// first by its number and further ones from a counter, loads the next one's tiles while it ends the last, and forms the next
// one's first scores while its softmax warps write the last one's rows (a CTA for each item: 20500 cycles beside 2800 a key
// tile).
//
// Twelve warps:
//   warp 0       items and TMA: both Q tiles, then K and V tiles into rings (in a paged cache a lane for each page of a tile)
//   warp 1       MMA issuer: S_A(0) S_B(0) | PV_A(j) S_A(j+1) PV_B(j) S_B(j+1) | ..., so that the tensor core works on one
//                query tile while the softmax of the other runs
//   warps 2, 3   tiles of V that part of the rows must not see: see scrub_rows
//   warps 4..7   softmax of tile A, warps 8..11 of tile B: one query row per thread.  P = exp2(S c - m) goes back over the
//                score columns as bf16 pairs (V is bf16 and one product's operands have one type; each weight is off by at
//                most 2^-8 of itself), from where the PV product reads it, in two halves.  The row's sum is of the unrounded
//                weights, in float32: it is also the returned lse.  The running maximum only moves (and O is
//                rescaled in TMEM) when a row's maximum grows by more than 2^8.
// TMEM columns: S/P of A [0,128), S/P of B [128,256), O of A [256,256+D), O of B [384,384+D).
// V is read as it lies ([key][d], MN-major), K and Q K-major.  Heads of up to 64 run with D = 64, up to 128 with D = 128;
// columns behind head_dim are zeros that the TMA fills in.  The products of heads of up to 96 leave out the last 32 (KD: 23
// sequences of 25 heads of 96, 305 us with all 128 columns, 283 so).
//
// What bounds it is the chain of a tile, scores, softmax, weights, product, scores: 2950 cycles for two tiles of 128 rows by 128
// keys, 2048 of them the tensor core's, no pipe full; and 8000 cycles where an item ends and the next begins (its last
// product, 4500 for the rows on their way out, the first softmax).  Heads of 128, 32 + 8, causal: 2 x 4608 tokens 268 us
// (1.30 PFLOP/s), 16384 tokens 1.41 ms (1.56); heads of 64, 2 x 4608: 214 us (0.81).
//
// Over a paged cache the keys of an item may be split over several (few rows, long contexts); each then writes
// its part normalised in float32 with its log-sum, and paged_join_kernel joins them.
#include <algorithm>

#include "attention_tiles.cuh"

namespace mmdit {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;  // in log2 units

template <int D>
struct Cfg {
  static constexpr int kStages = D == 128 ? 2 : 4;  // of K and of V
  static constexpr int kTileBytes = (D / 64) * kSeqBlock;
  static constexpr int kPieces = (2 + 2 * kStages) * kTileBytes;  // rows on their way out, 64 columns of 32 rows for each warp
  static constexpr int kBar = kPieces + 8 * 32 * 128;
  static constexpr int kSmem = kBar + 2048 + 1024;
  static constexpr uint32_t kIdescS = make_idesc<kKindF16>(128, 128);
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

// A work item: two query tiles of one sequence and key head, key tiles [js, js + cnt[x]) of each.
struct Work {
  int live;  // 0: no more items
  int b, hk, t0, split, n_splits, js;
  int cnt[2];
  int all_see;  // keys that every row sees
  Segment seg;
};

template <int D>
struct Barriers {
  uint64_t work_full[2], work_empty[2];
  uint64_t q_full, q_empty;
  uint64_t k_full[Cfg<D>::kStages], k_empty[Cfg<D>::kStages];
  uint64_t v_full[Cfg<D>::kStages], v_empty[Cfg<D>::kStages];
  uint64_t v_clean[Cfg<D>::kStages];
  uint64_t v_issued[Cfg<D>::kStages];  // tiles to clean: their copies are on the way (so v_full's phase is this tile's)
  uint64_t s_full[2];
  uint64_t p_full[2][2];  // per tile: the weights of its first 64 keys, of its last
  uint64_t o_full[2];
  uint64_t drain;
  uint32_t tmem_slot;
  int abort_flag;
  uint32_t progress;  // see mbar_wait_item
  int any_bad[2];
  // paged: pieces of an item's tile j whose page does not exist; two rounds of the ring for each of the two items, as a K tile
  // is free before all rows have read this
  uint32_t lost_pages[2][2 * Cfg<D>::kStages];
  Work work[2];
  int worst[2][D];
};
static_assert(sizeof(Barriers<128>) <= 2048 && sizeof(Barriers<64>) <= 2048, "barriers");

// The next item of the counter, by all lanes of a warp: the first lane asks, all have the answer.
__device__ __forceinline__ uint32_t ask_next(const SeqAttnArgs& a) {
  return a.next && (threadIdx.x & 31) == 0 ? atomicAdd(a.next, 1u) : 0;
}
__device__ __forceinline__ int next_of(const SeqAttnArgs& a, uint32_t ticket) {
  return a.first_next + static_cast<int>(__shfl_sync(0xffffffffu, ticket, 0));
}

__device__ __forceinline__ bool to_scrub(const Work& w, int j) { return (w.js + j + 1) * kSeqTile > w.all_see; }

template <int D, int KD, bool PAGED>
__device__ __forceinline__ void softmax_role(Barriers<D>* sb, int X, uint32_t tmem, const SeqAttnArgs& a, uint8_t* pieces) {
  constexpr int kStages = Cfg<D>::kStages;
  volatile int* abort_flag = &sb->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;
  const int row = quarter * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t s_cols = tmem + static_cast<uint32_t>(X * 128) + lane_off;
  const uint32_t o_cols = tmem + 256u + static_cast<uint32_t>(X * 128) + lane_off;
  const float c = a.scale_log2;
  const int row_tok = row / a.group, row_head = row % a.group;
  uint32_t s_turn = 0, o_turn = 0;  // parities of the barriers' next phases
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.status, kErrAttnWait)) != 0;
  };
  for (uint32_t it = 0;; ++it) {
    const int slot = it & 1;
    // an item of one tile is the other tile's warps' alone
    if (!__all_sync(0xffffffffu, mbar_wait_item(&sb->work_full[slot], it >> 1 & 1u, &sb->progress, abort_flag, a.status, kErrAttnWait))) return;
    const Work w = sb->work[slot];
    if (!w.live) return;
    const int cnt = X ? w.cnt[1] : w.cnt[0];
    const bool last = X == (w.cnt[1] > 0 ? 1 : 0);  // the tile whose products come last
    const int tok = w.t0 + X * a.tile_tokens + row_tok;  // of the sequence
    const bool valid = row < a.tile_tokens * a.group && tok < w.seg.n;
    // rows of no token compute on whatever their lines hold and are not stored
    const int lim = valid ? keys_seen(w.seg, tok, a.causal) : INT32_MAX;
    float m_run = -INFINITY, l_run = 0.f;
    bool saw = !PAGED && lim > 0;  // a key: paged, one that has a page
    int st = 0;
    for (int j = 0; j < cnt; ++j) {
      if (!wait(&sb->s_full[X], s_turn)) return;
      s_turn ^= 1u;
      tc_fence_after();
      // the products are done in their order: with the last tile's scores of K_j, V_(j-1) is read as well
      if (last && (threadIdx.x & 127) == 0) {
        mbar_arrive(&sb->k_empty[st]);
        if (j > 0) mbar_arrive(&sb->v_empty[st == 0 ? kStages - 1 : st - 1]);
      }
      st = st + 1 == kStages ? 0 : st + 1;
      const int rel = lim - (w.js + j) * kSeqTile;  // keys of this tile that the row sees
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
        // noted before the tile's K was loaded, whose barrier the MMA warp had to see for these scores
        const uint32_t lost = *reinterpret_cast<volatile uint32_t*>(&sb->lost_pages[slot][j % (2 * kStages)]);
        if (lost) {  // pieces of at least 8 keys
          whole = false;
          uint32_t eights = 0;
          for (int e = 0; e < 16; ++e) {
            eights |= (lost >> (e * 8 / a.page_rows) & 1u) << e;
            saw |= e * 8 < rel && !(eights >> e & 1u);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (eights >> (i / 8) & 1u) r0[i] = __float_as_uint(-INFINITY);
            if (eights >> (4 + i / 8) & 1u) r1[i] = __float_as_uint(-INFINITY);
            if (eights >> (8 + i / 8) & 1u) r2[i] = __float_as_uint(-INFINITY);
            if (eights >> (12 + i / 8) & 1u) r3[i] = __float_as_uint(-INFINITY);
          }
        } else {
          saw |= rel > 0;
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
        for (int e = 0; e < KD / 16; ++e) {
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
      if (!wait(&sb->o_full[X], o_turn)) return;
      o_turn ^= 1u;
      tc_fence_after();
      if (last && (threadIdx.x & 127) == 0) mbar_arrive(&sb->v_empty[(cnt - 1) % kStages]);
    }
    // no sum: no keys, or scores that are all -inf (see kNoWeights)
    const float nan = __int_as_float(0x7FC00000);
    const float inv_l = l_run == 0.f ? (saw && w.n_splits == 1 ? nan : 0.f) : 1.f / l_run;
    const float lse2 = l_run == 0.f ? (!saw ? -INFINITY : w.n_splits == 1 ? nan : kNoWeights) : m_run + log2f(l_run);
    const int head = w.hk * a.group + row_head;
    const size_t out_row = valid ? (static_cast<size_t>(w.seg.q0) + tok) * a.hq + head : 0;
    const bool any_bad = *reinterpret_cast<volatile int*>(&sb->any_bad[slot]) != 0;
    float* part = nullptr;
    __nv_bfloat16* out = nullptr;
    if (valid && w.n_splits > 1) {
      const size_t at = static_cast<size_t>(w.split) * a.tokens_q * a.hq + out_row;
      part = a.part + at * D;
      a.part_lse[at] = lse2;
    } else if (valid) {
      out = static_cast<__nv_bfloat16*>(a.out.ptr) + (static_cast<int64_t>(w.seg.q0) + tok) * a.out.stride_t + head * a.out.stride_h;
      if (a.lse) a.lse[out_row] = lse2 * kLn2;
    }
#pragma unroll 1
    for (int e = 0; e < D / 32; ++e) {
      float v[32];
      uint32_t r[32];
      if (cnt > 0) tmem_ld32_wait(o_cols + e * 32, r);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = cnt > 0 ? __uint_as_float(r[i]) * inv_l : 0.f;
      if (any_bad) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (*reinterpret_cast<volatile int*>(&sb->worst[slot][e * 32 + i]) < lim) v[i] = __int_as_float(0x7FC00000);
      }
      if (w.n_splits == 1) {
        put_pieces<64>(pieces, e & 1, v);
        if (e & 1) {
          __syncwarp();
          store_rows<64>(pieces, out ? out + (e - 1) * 32 : nullptr, a.head_dim - (e - 1) * 32);
          __syncwarp();
        }
      } else if (part) {
        store32(part + e * 32, v);
      }
    }
    // O has been read: the next item's first product may write it once this warp hands over that item's weights
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sb->work_empty[slot]);
  }
}

template <int D, int KD, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
    seq_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ SeqAttnArgs a) {
  using C = Cfg<D>;
  constexpr int kStages = C::kStages;
  constexpr uint32_t kIdescPV = make_idesc<kKindF16>(128, KD) | kIdescBMnMajor;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Barriers<D>* sb = reinterpret_cast<Barriers<D>*>(smem + C::kBar);
  volatile int* abort_flag = &sb->abort_flag;
  auto q_tile = [&](int x) { return smem + x * C::kTileBytes; };
  auto k_tile = [&](int st) { return smem + (2 + st) * C::kTileBytes; };
  auto v_tile = [&](int st) { return smem + (2 + kStages + st) * C::kTileBytes; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sb->work_full[s], 1);
      mbar_init(&sb->work_empty[s], 1 + 2 + 8);  // warps 1, 2, 3 and the softmax warps
      mbar_init(&sb->s_full[s], 1);
      mbar_init(&sb->p_full[s][0], 128);
      mbar_init(&sb->p_full[s][1], 128);
      mbar_init(&sb->o_full[s], 1);
    }
    mbar_init(&sb->q_full, 1);
    mbar_init(&sb->q_empty, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sb->k_full[s], 1);
      mbar_init(&sb->k_empty[s], 1);
      mbar_init(&sb->v_full[s], 1);
      mbar_init(&sb->v_empty[s], 1);
      mbar_init(&sb->v_clean[s], 64);
      mbar_init(&sb->v_issued[s], 1);
    }
    mbar_init(&sb->drain, 1);
    sb->abort_flag = 0;
    sb->progress = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sb->tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sb->tmem_slot;
  pdl_wait();
  if (PAGED && a.few_rows) pdl_trigger();  // paged_few_kernel takes the SMs that run out of items
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.status, kErrAttnWait)) != 0;
  };
  auto wait_item = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_item(bar, parity, &sb->progress, abort_flag, a.status, kErrAttnWait)) != 0;
  };

  if (warp >= 4) {
    more_registers<kSoftmaxRegisters>();
    softmax_role<D, KD, PAGED>(sb, (warp - 4) >> 2, tmem, a, smem + C::kPieces + (warp - 4) * 32 * 128);
  } else if (fewer_registers<kServiceRegisters>(), warp == 0) {
    // ---------------- items and TMA
    if (lane == 0) tma_prefetch_desc(&tm_q), tma_prefetch_desc(&tm_k), tma_prefetch_desc(&tm_v);
    if (a.clear && blockIdx.x == 0 && lane == 0) *a.status = 0;
    const int pieces = PAGED ? kSeqTile / a.page_rows : 1;
    TileOrder order;
    order.init(a.cu_q, a.tokens_q, PAGED ? nullptr : a.cu_k, a.tokens_k, a.batch, 2 * a.tile_tokens, a.causal, 1,
               PAGED ? a.few_tokens : 0);
    const int per_split = order.n * a.hk, items = per_split * a.splits;
    uint32_t q_turn = 0, k_turn = 0, v_turn = 0;  // the next phases' parities; k, v: a bit for each stage
    uint32_t k_used = 0, v_used = 0;
    bool ok = true, q_used = false;
    int item = blockIdx.x;
    uint32_t steps = 0;
    auto progress = [&]() {
      if (lane == 0) *const_cast<volatile uint32_t*>(&sb->progress) = ++steps;
    };
    for (uint32_t it = 0; ok; ++it) {
      Work w;
      w.live = 0;
      for (; item < items; item = a.next ? next_of(a, ask_next(a)) : items) {
        progress();
        const int rest = item % per_split;
        TileOrder::Found at;
        if (!order.find(rest / a.hk, at)) continue;
        w.b = at.b, w.hk = rest % a.hk, w.split = item / per_split, w.t0 = at.start;
        w.seg = {at.first, at.count, at.other_first, at.other_count};
        int split_tiles = INT32_MAX;
        w.n_splits = 1, w.js = 0;
        if constexpr (PAGED) {
          w.seg.k0 = 0, w.seg.m = min(max(a.kv_lens[w.b], 0), a.max_keys);
          if (a.split_keys > 0) {
            split_tiles = a.split_keys / kSeqTile;
            w.n_splits = max((w.seg.m + a.split_keys - 1) / a.split_keys, 1);
            if (w.split >= w.n_splits) continue;
            w.js = w.split * split_tiles;
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int first = w.t0 + x * a.tile_tokens, rows = min(w.seg.n - first, a.tile_tokens);
          const int tiles = rows > 0 ? (keys_seen(w.seg, first + rows - 1, a.causal) + kSeqTile - 1) / kSeqTile : 0;
          w.cnt[x] = max(min(tiles - w.js, split_tiles), 0);
        }
        w.all_see = keys_seen(w.seg, w.t0, a.causal);
        w.live = 1;
        break;
      }
      const int slot = it & 1;
      ok = wait(&sb->work_empty[slot], (it >> 1 & 1u) ^ 1u);
      if (!ok) break;
      for (int i = lane; i < D; i += 32) *reinterpret_cast<volatile int*>(&sb->worst[slot][i]) = INT32_MAX;
      __syncwarp();
      if (lane == 0) {
        sb->work[slot] = w;
        *reinterpret_cast<volatile int*>(&sb->any_bad[slot]) = 0;
        mbar_arrive(&sb->work_full[slot]);
      }
      __syncwarp();
      if (!w.live) break;
      const int n_kv = max(w.cnt[0], w.cnt[1]);
      if (n_kv > 0) {
        ok = wait(&sb->q_empty, q_turn ^ 1u);
        if (!ok) break;
        if (lane == 0) {
          const int bytes = (D / 64) * a.group * a.tile_tokens * 128;
          mbar_arrive_expect_tx(&sb->q_full, (w.cnt[0] > 0 ? bytes : 0) + (w.cnt[1] > 0 ? bytes : 0));
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (w.cnt[x] > 0)
#pragma unroll
              for (int h = 0; h < D / 64; ++h)
                tma_load_3d(q_tile(x) + h * kSeqBlock, &tm_q, &sb->q_full, h * 64, w.hk * a.group,
                            w.seg.q0 + w.t0 + x * a.tile_tokens);
        }
        q_turn ^= 1u, q_used = true;
      }
      auto page_of = [&](int j) -> int {  // the page of this lane's piece of tile j: -1 behind the last key, -2 if there is none
        const int key = (w.js + j) * kSeqTile + lane * a.page_rows;
        if (lane >= pieces || key >= w.seg.m) return -1;
        const int p = a.tables[static_cast<int64_t>(w.b) * a.table_width + (key >> a.page_shift)];
        return p >= 0 && p < a.n_pages ? p : -2;
      };
      auto load = [&](uint8_t* tile, const CUtensorMap* map, uint64_t* bar, int j, int page) {
        if constexpr (PAGED) {
          if (lane == 0) mbar_arrive_expect_tx(bar, C::kTileBytes);
          __syncwarp();
          if (lane < pieces) {
            const int z = page < 0 ? a.n_pages : page;  // behind the last page: the box reads zeros
            const int y = ((w.js + j) * kSeqTile + lane * a.page_rows) & ((1 << a.page_shift) - 1);
            for (int h = 0; h < D / 64; ++h)
              tma_load_4d(tile + h * kSeqBlock + lane * a.page_rows * 128, map, bar, h * 64, y, w.hk, z);
          }
        } else if (lane == 0) {
          mbar_arrive_expect_tx(bar, C::kTileBytes);
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(tile + h * kSeqBlock, map, bar, h * 64, w.hk, w.seg.k0 + (w.js + j) * kSeqTile);
        }
      };
      auto load_k = [&](int j, int st, int p) {
        if (!wait(&sb->k_empty[st], (k_turn >> st & 1u) ^ 1u)) return false;
        k_turn ^= 1u << st, k_used |= 1u << st;
        if constexpr (PAGED) {
          const uint32_t lost = __ballot_sync(0xffffffffu, p == -2);
          if (lane == 0) {
            *reinterpret_cast<volatile uint32_t*>(&sb->lost_pages[slot][j % (2 * kStages)]) = lost;
            __threadfence_block();
          }
        }
        load(k_tile(st), &tm_k, &sb->k_full[st], j, p);
        return true;
      };
      // K runs ahead of V by a tile: it is free once its scores are formed, V when they have been multiplied
      int page = PAGED && n_kv > 0 ? page_of(0) : 0, next = PAGED && n_kv > 1 ? page_of(1) : 0, st = 0;
      if (n_kv > 0) ok = load_k(0, 0, page);
      // The next item's number is on its way while the last two tiles are: a CTA that took it with its first ones would keep a
      // short item waiting behind a long one.
      uint32_t ticket = 0;
      if (n_kv == 0) ticket = ask_next(a);
      for (int j = 0; ok && j < n_kv; ++j) {
        progress();
        if (j == max(n_kv - 2, 0)) ticket = ask_next(a);
        const int after = st + 1 == kStages ? 0 : st + 1;
        if (j + 1 < n_kv) ok = load_k(j + 1, after, next);
        ok = ok && wait(&sb->v_empty[st], (v_turn >> st & 1u) ^ 1u);
        if (!ok) break;
        v_turn ^= 1u << st, v_used |= 1u << st;
        load(v_tile(st), &tm_v, &sb->v_full[st], j, page);
        if (lane == 0 && to_scrub(w, j)) mbar_arrive(&sb->v_issued[st]);
        page = next, st = after;
        if (PAGED && j + 2 < n_kv) next = page_of(j + 2);
      }
      item = a.next ? next_of(a, ticket) : items;
    }
    if (!ok) {
      // give the copies already issued a bounded chance to land before the CTA exits
      int never = 0;
      if (q_used) mbar_wait(&sb->q_full, q_turn ^ 1u, &never, a.status, 0);
      for (int s = 0; s < kStages; ++s) {
        if (k_used >> s & 1u) mbar_wait(&sb->k_full[s], (k_turn >> s & 1u) ^ 1u, &never, a.status, 0);
        if (v_used >> s & 1u) mbar_wait(&sb->v_full[s], (v_turn >> s & 1u) ^ 1u, &never, a.status, 0);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer: the tensor core's queue is short, so whatever this warp waits for leaves it idle.  The
    // warp's lanes test the barriers of a step side by side, one lane issues.
    // Steps are unrolled over the ring, so that stages and descriptors are constants and few instructions lie
    // between a barrier and the products behind it.
    // Of a descriptor only the address in its lower half changes; K-step k of a K-major tile is 16 elements into its
    // 128-byte swizzle atoms.
    auto koff = [](int k) -> uint32_t { return static_cast<uint32_t>(((k >> 2) * kSeqBlock + (k & 3) * 32) >> 4); };
    auto desc = [](uint64_t base, uint32_t lo) { return (base & 0xFFFFFFFF00000000ull) | lo; };
    const uint64_t k_base = sdesc_kmajor_sw128(smem_addr(k_tile(0))), v_base = sdesc_mnmajor_sw128(smem_addr(v_tile(0)), kSeqBlock);
    uint32_t q_lo = static_cast<uint32_t>(sdesc_kmajor_sw128(smem_addr(q_tile(0)))), k_lo = static_cast<uint32_t>(k_base),
             v_lo = static_cast<uint32_t>(v_base);
    constexpr uint32_t kStep = static_cast<uint32_t>(C::kTileBytes) >> 4;
    auto mma_s = [&](int x, int st) {  // S_x = Q_x K^T into columns [128x, 128x + 128)
#pragma unroll
      for (int k = 0; k < KD / 16; ++k)
        tc_mma<kKindF16>(tmem + x * 128, desc(k_base, q_lo + x * kStep + koff(k)), desc(k_base, k_lo + st * kStep + koff(k)),
                         C::kIdescS, k > 0 ? 1u : 0u);
      tc_commit(&sb->s_full[x]);
    };
    auto mma_pv = [&](int x, int st, int half, uint32_t more) {  // O_x += P_x V over half of the keys, P from TMEM over S_x
#pragma unroll
      for (int k = 4 * half; k < 4 * half + 4; ++k)  // 16 keys in 8 columns of P
        tc_mma_ts_f16(tmem + 256u + x * 128, tmem + x * 128 + k * 8, desc(v_base, v_lo + st * kStep + ((k * 2048) >> 4)),
                      kIdescPV, k > 0 ? 1u : more);
    };
    uint32_t q_turn = 0, k_turn = 0, v_turn = 0, clean_turn = 0, p_turn = 0;  // parities; p: a bit for each tile
    bool ok = true;
    for (uint32_t it = 0; ok; ++it) {
      const int slot = it & 1;
      ok = wait_item(&sb->work_full[slot], it >> 1 & 1u);
      if (!ok) break;
      const int cnt0 = sb->work[slot].cnt[0], cnt1 = sb->work[slot].cnt[1], live = sb->work[slot].live;
      // tiles from here on are to be cleaned
      const int clean_from = sb->work[slot].all_see / kSeqTile - sb->work[slot].js;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sb->work_empty[slot]);
      if (!live) break;
      const int n_kv = max(cnt0, cnt1);
      if (n_kv == 0) continue;
      ok = wait(lane == 0 ? &sb->q_full : &sb->k_full[0], lane == 0 ? q_turn : k_turn & 1u);
      q_turn ^= 1u, k_turn ^= 1u;
      if (ok && one_lane()) {
        tc_fence_after();
        if (cnt0 > 0) mma_s(0, 0);
        if (cnt1 > 0) mma_s(1, 0);
        if (n_kv == 1) tc_commit(&sb->q_empty);
      }
      __syncwarp();
      for (int j0 = 0; ok && j0 < n_kv; j0 += kStages) {
#pragma unroll
        for (int st = 0; st < kStages; ++st) {
          const int j = j0 + st;
          if (!ok || j >= n_kv) break;
          constexpr int kLast = kStages - 1;
          const int after = st == kLast ? 0 : st + 1;
          const uint32_t more = j > 0 ? 1u : 0u;
          if (j >= clean_from) {
            ok = wait(&sb->v_clean[st], clean_turn >> st & 1u);
            clean_turn ^= 1u << st;
          }
          // the first tile's step also awaits V_j and K_(j+1)
          const bool both = j < cnt0 && j < cnt1;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int cnt = x ? cnt1 : cnt0;
            if (!ok || j >= cnt) continue;
            const bool first = x == 0 || !both;
            asm volatile("" : "+r"(q_lo), "+r"(k_lo), "+r"(v_lo));  // the sums below are formed here, not kept in registers
            {
              const bool v_too = first && lane == 1, k_too = first && lane == 2 && j + 1 < n_kv;
              ok = wait(v_too ? &sb->v_full[st] : k_too ? &sb->k_full[after] : &sb->p_full[x][0],
                        (v_too ? v_turn >> st : k_too ? k_turn >> after : p_turn >> x) & 1u);
            }
            if (ok && one_lane()) {
              tc_fence_after();
              mma_pv(x, st, 0, more);
            }
            __syncwarp();
            ok = ok && wait(&sb->p_full[x][1], p_turn >> x & 1u);
            p_turn ^= 1u << x;
            if (ok && one_lane()) {
              tc_fence_after();
              mma_pv(x, st, 1, 1u);
              if (j + 1 < cnt)
                mma_s(x, after);
              else
                tc_commit(&sb->o_full[x]);
              // the item's last scores: its queries are read
              if (j + 2 == n_kv && x == (cnt1 > 0 ? 1 : 0)) tc_commit(&sb->q_empty);
            }
            __syncwarp();
          }
          v_turn ^= 1u << st;
          if (j + 1 < n_kv) k_turn ^= 1u << after;
        }
      }
    }
    if (!ok && one_lane()) {
      // wait (bounded) for every MMA issued so far before TMEM is released
      int never = 0;
      tc_commit(&sb->drain);
      mbar_wait(&sb->drain, 0, &never, a.status, 0);
    }
  } else {
    // ---------------- V rows that part of an item's queries must not see
    const int tid = static_cast<int>(threadIdx.x) - 64;
    uint32_t v_turn = 0, clean_turn = 0;
    bool ok = true;
    for (uint32_t it = 0; ok; ++it) {
      const int slot = it & 1;
      ok = wait_item(&sb->work_full[slot], it >> 1 & 1u);
      if (!ok) break;
      const Work w = sb->work[slot];
      if (w.live) {
        const int n_kv = max(w.cnt[0], w.cnt[1]);
        int st = 0;
        for (int j = 0; ok && j < n_kv; ++j, st = st + 1 == kStages ? 0 : st + 1) {
          const uint32_t parity = v_turn >> st & 1u;
          v_turn ^= 1u << st;
          if (!to_scrub(w, j)) continue;
          ok = wait_item(&sb->v_issued[st], clean_turn >> st & 1u) && wait(&sb->v_full[st], parity);
          clean_turn ^= 1u << st;
          if (!ok) break;
          const int key = (w.js + j) * kSeqTile;
          scrub_rows<D>(v_tile(st), max(w.all_see - key, 0), w.seg.m - key, key, sb->worst[slot], &sb->any_bad[slot], tid);
          mbar_arrive(&sb->v_clean[st]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sb->work_empty[slot]);
      if (!w.live) break;
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int KD, bool PAGED>
cudaError_t launch_dim(const SeqAttnArgs& a, const SeqAttnMaps& m, int grid, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(seq_attention_kernel<D, KD, PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(seq_attention_kernel<D, KD, PAGED>, dim3(grid), dim3(kThreads), Cfg<D>::kSmem, stream, m.q, m.k, m.v, a);
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

cudaError_t launch_seq_attention(SeqAttnArgs a, const SeqAttnMaps& m, int paged, int splits, uint32_t* counter, cudaStream_t stream) {
  a.tile_tokens = seq_tile_tokens(a.group);
  const int64_t pairs = a.tokens_q / (2 * a.tile_tokens) + static_cast<int64_t>(a.batch);
  const int64_t items = pairs * a.hk * splits;
  a.splits = splits;
  const int grid = static_cast<int>(std::min<int64_t>(items, num_sms()));
  cudaError_t e;
  if (items > grid) {  // further items are handed out by a counter (status word and counter share the workspace's first line)
    if ((e = cudaMemsetAsync(counter, 0, sizeof(uint32_t), stream)) != cudaSuccess) return e;
    pdl_begin_call();  // the kernel follows a memset: an ordinary launch
    a.next = counter, a.first_next = grid;
  }
  if (a.head_dim <= 64)
    e = paged ? launch_dim<64, 64, true>(a, m, grid, stream) : launch_dim<64, 64, false>(a, m, grid, stream);
  else if (a.head_dim <= 96)
    e = paged ? launch_dim<128, 96, true>(a, m, grid, stream) : launch_dim<128, 96, false>(a, m, grid, stream);
  else
    e = paged ? launch_dim<128, 128, true>(a, m, grid, stream) : launch_dim<128, 128, false>(a, m, grid, stream);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace mmdit
