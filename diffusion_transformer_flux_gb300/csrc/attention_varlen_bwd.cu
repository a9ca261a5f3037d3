// attention_varlen_bwd.cu -- gradients of the attention over packed sequences, on tcgen05 tensor cores.
//
// With p_ij = exp(z_ij - lse_i) from the forward's lse, delta_i = dout_i . out_i and dz_ij = p_ij (dout_i . v_j - delta_i):
//   dv_j = sum_i p_ij dout_i,   dk_j = scale sum_i dz_ij q_i,   dq_i = scale sum_j dz_ij k_j,
// dk and dv summed over the query heads of a key head's group.  Two passes, one over key tiles and one over query tiles, each
// recompute z and dout . v: seven products where one pass would need five, but that one has to add its dq into
// memory from every key tile, in an order that changes the bits, through float32 traffic of several times the tensors' size.
// Here every sum stays in tensor memory and is written once, in bf16.  The pass over queries starts on the SMs that the one over
// keys leaves.  2 x 4608 tokens of 32 + 8 heads of 128: 943 us (923 TFLOP/s of the five products), of 24 heads of 64: 510 us
// (640); 9 documents of up to 2041 tokens of 32 + 8 heads of 128: 255 us (677).
//
// Both passes are one kernel, whose work items have a resident tile pair F (of 128 rows) and moving tile pairs M:
//   keys:    F = K, V;     M = Q, dO;   S = K Q^T, dP = V dO^T;   dV += P dO,  dK += dS Q     (rows of S are keys)
//   queries: F = Q, dO;    M = K, V;    S = Q K^T, dP = dO V^T;   dQ += dS K                  (rows of S are queries)
// A tile of queries is 128 / group tokens by the group's heads, as in the forward, so the sum over the group's heads is the sum
// over a moving tile's rows.  Moving tiles have up to 64 rows and take turns in two buffers of S and dP, so that the products
// of one run while P and dS of the other are formed; their ring in shared memory holds four to eight (the load of one takes
// as long as the work on two).  With N = 64 a product of two tiles in shared memory reads 6 KB for 32 cycles of
// multiplication (48 cycles); where tensor memory has room for F (queries, and keys with D = 64), F is copied there.  Items are
// found and handed out as in the forward.
// In the pass over keys L and delta belong to the columns of S and dP.  The products subtract them: a last step of 16 columns
// has ones in three columns of its F side and -L / c (or -delta), cut into three bf16 numbers, in those columns of its M
// side, so that the accumulators hold S - L / c and dP - delta.  (Read from shared memory by each row they took longer than
// the arithmetic, beside products that read shared memory at its full rate: 1330 against 770 cycles a tile with D = 64.)
// Twelve warps:
//   warp 0       items and TMA: F, then M tiles
//   warp 1       MMA issuer: S, dP of tile u + 2 follow the accumulating products of tile u
//   warps 2, 3   keys: the last step's M side; both: rows that part of F must not see (scrub_pair)
//   warps 4..7   tiles of even number: one row of S and dP per thread, P = exp2(c S - L) and dS = P (dP - delta) back into tensor
//                memory as bf16 pairs (the operands of the accumulating products, each off by at most 2^-8 of itself);
//                warps 8..11 those of odd number
// TMEM columns: S [0,128), dP [128,256), then dV and dK, or dQ, D each, and F from 384 where it fits.
#include <algorithm>
#include <type_traits>

#include "attention_tiles.cuh"

namespace mmdit {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmP = 0, kTmD = 128, kTmAcc = 256, kTmF = 384, kTmExt = 448;
constexpr int kUnit = 64;  // rows of a moving tile
constexpr int kBwdService = 152, kBwdRows = 176;  // registers of the warps that issue, of the warps of rows
static_assert(128 * kBwdService + 256 * kBwdRows <= 384 * kLaunchRegisters, "shares of the launch's registers");

template <int D, bool KEYS>
struct Cfg {
  static constexpr bool kFInTmem = !KEYS || D == 64;
  static constexpr bool kFInRing = !KEYS;  // F passes through two slots of the ring (a pair of 128 rows has their size)
  static constexpr int kTileBytes = (D / 64) * kSeqBlock;  // of F
  static constexpr int kUnitBlock = kUnit * 128;           // 64 rows of 64 columns
  static constexpr int kHalfSlot = (D / 64) * kUnitBlock;
  static constexpr int kSlotBytes = 2 * kHalfSlot;         // the moving pair
  static constexpr int kSlots = D == 64 ? 8 : KEYS ? 4 : 6;
  static constexpr int kRing = kFInRing ? 0 : 2 * kTileBytes;
  static constexpr int kPieces = kRing + kSlots * kSlotBytes;  // rows on their way out, 32 columns of 32 rows for each warp
  static constexpr int kExt = kPieces + 8 * 32 * 64;           // keys: the last step, 32 bytes a row: M's per slot, then F's two
  static constexpr int kExtM = kUnit * 32, kExtF = kSeqTile * 32;
  static constexpr int kBar = kExt + (KEYS ? kSlots * kExtM + 2 * kExtF : 0);
  static constexpr int kSmem = kBar + 1024 + 1024;
  static constexpr uint32_t kIdescS = make_idesc<kKindF16>(128, kUnit);
  static constexpr uint32_t kIdescAcc = make_idesc<kKindF16>(128, D) | kIdescBMnMajor;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct Work {
  int live;   // 0: no more items
  int hk;
  int first, count;  // first row of F in its sequence (a key, or a token), moving tiles
  int m_first;       // keys: the first token that sees a key of the tile
  int all_see;       // queries: keys that every row sees
  int clean_to, clean_from;  // tiles [0, clean_to) and [clean_from, count) have rows to clean
  int part, parts;           // keys: which part of the moving tiles this is, of how many
  Segment seg;
};

struct Barriers {
  uint64_t work_full[2], work_empty[2];
  uint64_t f_full, f_copied, f_empty;
  uint64_t st_full[8], st_clean[8], st_empty[8];  // st_full: the copies, and in the pass over keys the last step's rows
  uint64_t st_issued[8];  // the copies of a tile to clean are on the way (so st_full's phase is this tile's)
  uint64_t sp_full[2];
  uint64_t pd_full[2];
  uint64_t done, acc_free;
  uint64_t drain;
  uint32_t tmem_slot;
  int abort_flag;
  uint32_t progress;  // see mbar_wait_item
  int worst[2];  // per item: the row of M that is not finite and that most rows of F see (keys: the last token, queries: the first key)
  Work work[2];
};
static_assert(sizeof(Barriers) <= 1024, "barriers");

// The wait for earlier loads of tensor memory, their registers threaded through it.
__device__ __forceinline__ void tmem_ld32_deps(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Rows [lo, hi) of a moving tile that hold a non-finite element have it zeroed and are noted (queries: by their token first + r / group,
// keys: first + r), rows [zero_from, 64) become zeros.
// Called by THREADS threads; eight pieces are in flight in each.
template <int D, bool KEYS, int THREADS>
__device__ __forceinline__ void scrub_pair(uint8_t* tile, int lo, int hi, int zero_from, int first, int group, int* worst, int tid) {
  constexpr int kChunks = D / 8;
  auto at = [&](int i) {
    const int r = i / kChunks, c = i % kChunks;
    return reinterpret_cast<uint4*>(tile + (c >> 3) * kUnit * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
  };
  const int stop = min(hi, kUnit) * kChunks;
  for (int i0 = lo * kChunks + tid; i0 < stop; i0 += 8 * THREADS) {
    uint4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = i0 + THREADS * u < stop ? *at(i0 + THREADS * u) : make_uint4(0, 0, 0, 0);
    uint32_t bad = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) bad |= (not_finite(v[u]) ? 1u : 0u) << u;
    for (; bad; bad &= bad - 1) {
      const int i = i0 + THREADS * (__ffs(bad) - 1);
      *at(i) = make_uint4(0, 0, 0, 0);
      if (KEYS)
        atomicMax(worst, first + i / kChunks / group);
      else
        atomicMin(worst, first + i / kChunks);
    }
  }
  for (int i = max(zero_from, 0) * kChunks + tid; i < kUnit * kChunks; i += THREADS) *at(i) = make_uint4(0, 0, 0, 0);
}

// The moving tiles of `first`'s key tile: the first token that sees one of its keys, and their number; and how many parts of how
// many tiles they are worked on in (at least kPartUnits to a part, so that its sums are worth their way through memory).
constexpr int kPartUnits = 8;
struct KeyTile {
  int m_first, count, per_part, parts;
};
__device__ __forceinline__ KeyTile key_tile(const SeqAttnBwdArgs& a, const Segment& seg, int first) {
  KeyTile t;
  t.m_first = a.causal ? max(first - seg.m + seg.n, 0) : 0;
  t.count = seg.n > t.m_first ? (seg.n - t.m_first + a.unit_tokens - 1) / a.unit_tokens : 0;
  t.per_part = max((t.count + a.parts - 1) / a.parts, kPartUnits);
  t.parts = max((t.count + t.per_part - 1) / t.per_part, 1);
  return t;
}
// Where the float32 sums of part p of key row `row` lie: dv, then dk.
template <int D>
__device__ __forceinline__ size_t part_at(const SeqAttnBwdArgs& a, int p, int64_t row, int hk) {
  return ((static_cast<size_t>(p) * a.tokens_k + row) * a.hk + hk) * 2 * D;
}

// Rows of moving tile u: [0, zero_from) are of this sequence, those of [lo, hi) not seen by every row of F.
template <bool KEYS>
__device__ __forceinline__ void rows_of(const SeqAttnBwdArgs& a, const Work& w, int u, int& lo, int& hi, int& zero_from) {
  if constexpr (KEYS) {
    const int T = a.unit_tokens, t = w.m_first + u * T, last_key = min(w.first + kSeqTile, w.seg.m) - 1;
    zero_from = a.group * min(T, w.seg.n - t);
    lo = 0;
    hi = a.causal ? min(a.group * min(max(last_key - (w.seg.m - w.seg.n) - t, 0), T), zero_from) : 0;
  } else {
    zero_from = min(w.seg.m - u * kUnit, kUnit);
    lo = max(w.all_see - u * kUnit, 0), hi = zero_from;
  }
}
// Whether tile u has such rows: once for each item, as the MMA warp has no time for it at each tile.
template <bool KEYS>
__device__ __forceinline__ void set_cleaning(const SeqAttnBwdArgs& a, Work& w) {
  if constexpr (KEYS) {
    const int T = a.unit_tokens, before = min(w.first + kSeqTile, w.seg.m) - 1 - (w.seg.m - w.seg.n) - w.m_first;
    w.clean_to = a.causal ? (max(before, 0) + T - 1) / T : 0;
    w.clean_from = (w.seg.n - w.m_first) / T;  // a last tile of fewer tokens
  } else {
    w.clean_to = 0, w.clean_from = w.all_see / kUnit;
  }
}
__device__ __forceinline__ bool to_clean(const Work& w, int u) { return u < w.clean_to || u >= w.clean_from; }

// x as the sum of three bf16 numbers (24 bits; what is not finite is the first alone).
__device__ __forceinline__ void cut(float x, uint32_t (&v)[3]) {
  float left = x;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const __nv_bfloat16 b = __float2bfloat16(left);
    v[i] = __bfloat16_as_ushort(b);
    left = isfinite(x) ? left - __bfloat162float(b) : 0.f;
  }
}

// The next item of the counter, by all lanes of a warp: the first lane asks, all have the answer.
__device__ __forceinline__ uint32_t ask_next(uint32_t* counter) { return (threadIdx.x & 31) == 0 ? atomicAdd(counter, 1u) : 0; }
__device__ __forceinline__ int next_of(int first_next, uint32_t ticket) {
  return first_next + static_cast<int>(__shfl_sync(0xffffffffu, ticket, 0));
}

template <int D, bool KEYS>
__device__ __forceinline__ void rows_role(Barriers* sb, uint8_t* smem, uint32_t tmem, const SeqAttnBwdArgs& a) {
  using C = Cfg<D, KEYS>;
  volatile int* abort_flag = &sb->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
  const int G = a.group, T = a.tile_tokens;
  const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t t_p = tmem + kTmP + 64 * h + lane_off, t_d = tmem + kTmD + 64 * h + lane_off;
  const uint64_t scale2 = f32x2(a.scale_log2, a.scale_log2);
  const int row_tok = row / G, row_head = row % G;
  uint8_t* pieces = smem + C::kPieces + (warp - 4) * 32 * 64;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.status, kErrAttnWait)) != 0;
  };
  uint32_t f_turn = 0, sp_turn = 0, done_turn = 0, st_turn = 0;  // parities of the next phases (st: a bit for each slot)
  int slot_u = 0;                                                // the next slot of the ring
  auto next_slot = [&]() {
    st_turn ^= 1u << slot_u;
    slot_u = slot_u + 1 == C::kSlots ? 0 : slot_u + 1;
  };
  for (uint32_t it = 0;; ++it) {
    const int slot = it & 1;
    if (!__all_sync(0xffffffffu, mbar_wait_item(&sb->work_full[slot], it >> 1 & 1u, &sb->progress, abort_flag, a.status, kErrAttnWait))) return;
    const Work w = sb->work[slot];
    if (!w.live) return;
    const int lag = w.seg.m - w.seg.n;  // query i stands at lag + i
    // queries: this row's sums and the keys it sees; keys: the first token that sees it
    const int tok = w.first + row_tok;
    const bool valid = KEYS ? w.first + row < w.seg.m : row < G * T && tok < w.seg.n;
    const int lim = KEYS || !valid ? 0 : keys_seen(w.seg, tok, a.causal);
    const int from = !KEYS ? 0 : !valid ? INT32_MAX : a.causal ? max(w.first + row - lag, 0) : 0;
    uint64_t neg_l = 0, neg_d = 0;
    if constexpr (!KEYS) {
      float2 s = make_float2(0.f, 0.f);
      if (valid) s = __ldcg(&a.sums[(static_cast<size_t>(w.seg.q0) + tok) * a.hq + w.hk * G + row_head]);  // see `behind` below
      neg_l = f32x2(-s.x, -s.x), neg_d = f32x2(-s.y, -s.y);
    }
    if (C::kFInTmem && w.count > 0) {
      // F into tensor memory, these warps its first tile, the others its second; the last item's scores are formed
      const uint8_t* tile;
      if constexpr (C::kFInRing) {
        if (h) next_slot();
        if (!wait(&sb->st_full[slot_u], st_turn >> slot_u & 1u)) return;
        tile = smem + slot_u * C::kSlotBytes + row * 128;
        next_slot();
        if (!h) next_slot();
      } else {
        if (!wait(&sb->f_full, f_turn)) return;
        f_turn ^= 1u;
        tile = smem + h * C::kTileBytes + row * 128;
      }
#pragma unroll
      for (int b = 0; b < D / 64; ++b) {
        uint32_t r[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 v = *reinterpret_cast<const uint4*>(tile + b * kSeqBlock + ((c ^ (row & 7)) << 4));
          r[4 * c] = v.x, r[4 * c + 1] = v.y, r[4 * c + 2] = v.z, r[4 * c + 3] = v.w;
        }
        tmem_st32(tmem + kTmF + h * (D / 2) + b * 32 + lane_off, r);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&sb->f_copied);
    }
    int held = -1;  // the slot of these warps' last tile
    for (int u = 0; u < w.count; ++u, next_slot()) {
      if ((u & 1) != h) continue;
      if (!wait(&sb->sp_full[h], sp_turn)) return;
      sp_turn ^= 1u;
      tc_fence_after();
      // the products are done in their order: with these scores the tile before the last has been used up, with the last ones F
      if ((threadIdx.x & 127) == 0) {
        if (held >= 0) mbar_arrive(&sb->st_empty[held]);
        if (!C::kFInTmem && u + 1 == w.count) mbar_arrive(&sb->f_empty);
      }
      held = slot_u;
      // columns [lo, hi) of the tile are seen by this row
      int lo, hi;
      if constexpr (KEYS) {
        // in tokens first: a sequence's rows (tokens by the group) may be more than 32 bits count
        const int t = w.m_first + u * a.unit_tokens;
        hi = G * min(a.unit_tokens, w.seg.n - t), lo = G * min(max(from - t, 0), a.unit_tokens);
      } else {
        lo = 0, hi = lim - u * kUnit;
      }
      const bool part = __any_sync(0xffffffffu, lo > 0 || hi < kUnit);
      uint32_t s[2][32], d[32];
      tmem_ld64_wait(t_p, s[0], s[1]);
      tmem_ld32(t_d, d);
      // P over the scores' registers
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        uint32_t* x = s[e >> 3] + (e & 7) * 4;
        float p0, p1, p2, p3;
        const uint64_t a0 = f32x2(__uint_as_float(x[0]), __uint_as_float(x[1])), a1 = f32x2(__uint_as_float(x[2]), __uint_as_float(x[3]));
        f32x2_split(KEYS ? fmul2(a0, scale2) : ffma2(a0, scale2, neg_l), p0, p1);
        f32x2_split(KEYS ? fmul2(a1, scale2) : ffma2(a1, scale2, neg_l), p2, p3);
        x[0] = __float_as_uint(fast_exp2(p0)), x[1] = __float_as_uint(fast_exp2(p1));
        x[2] = __float_as_uint(fast_exp2(p2)), x[3] = __float_as_uint(fast_exp2(p3));
      }
      // dS of 32 columns; a tile that is seen in part has a loop of its own, a branch for each pair would hold every chain up
      auto columns = [&](auto in_part, int c) {
        uint32_t pk[16], dk[16];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          float p0 = __uint_as_float(s[c][k]), p1 = __uint_as_float(s[c][k + 1]), z0, z1;
          const uint64_t g = f32x2(__uint_as_float(d[k]), __uint_as_float(d[k + 1]));
          f32x2_split(fmul2(f32x2(p0, p1), KEYS ? g : fadd2(g, neg_d)), z0, z1);
          if constexpr (decltype(in_part)::value) {
            const int col = 32 * c + k;
            if (col < lo || col >= hi) p0 = z0 = 0.f;
            if (col + 1 < lo || col + 1 >= hi) p1 = z1 = 0.f;
          }
          pk[k / 2] = pack_bf16x2(p0, p1), dk[k / 2] = pack_bf16x2(z0, z1);
        }
        // over columns that were read: packed pairs take half as many
        if constexpr (KEYS) {
          tmem_st16(t_p + 16 * c, pk);
          tmem_st16(t_d + 16 * c, dk);
        } else {
          tmem_st16(t_p + 16 * c, dk);
        }
      };
      tmem_ld32_deps(d);
      if (part)
        columns(std::true_type{}, 0);
      else
        columns(std::false_type{}, 0);
      tmem_ld32_wait(t_d + 32, d);
      if (part)
        columns(std::true_type{}, 1);
      else
        columns(std::false_type{}, 1);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&sb->pd_full[h]);
    }
    if (w.count > 0) {
      if (!wait(&sb->done, done_turn)) return;
      done_turn ^= 1u;
      tc_fence_after();
      if (held >= 0 && (threadIdx.x & 127) == 0) mbar_arrive(&sb->st_empty[held]);
    }
    const int worst = *reinterpret_cast<volatile int*>(&sb->worst[slot]);
    if (KEYS || D == 128 || h == 0) {
      // keys: half 0 writes dV, half 1 dK; queries: each half 64 columns of dQ
      const HeadsView& out = !KEYS ? a.dq : h ? a.dk : a.dv;
      const int64_t at = KEYS ? (static_cast<int64_t>(w.seg.k0) + w.first + row) * out.stride_t + w.hk * out.stride_h
                              : (static_cast<int64_t>(w.seg.q0) + tok) * out.stride_t + (w.hk * G + row_head) * out.stride_h;
      __nv_bfloat16* dst = valid ? static_cast<__nv_bfloat16*>(out.ptr) + at : nullptr;
      const bool bad = valid && (KEYS ? worst >= from : worst < lim);
      const float f = bad ? __int_as_float(0x7FC00000) : KEYS && h == 0 ? 1.f : a.scale;
      const int blocks = KEYS ? D / 32 : 2, block0 = KEYS ? 0 : 2 * h;  // of 32 columns
#pragma unroll 1
      for (int k = block0; k < block0 + blocks; ++k) {
        float v[32];
        uint32_t r[32];
        if (w.count > 0) tmem_ld32_wait(tmem + kTmAcc + (KEYS ? h * D : 0) + k * 32 + lane_off, r);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = w.count > 0 ? __uint_as_float(r[i]) * f : 0.f;
        if (KEYS && w.parts > 1) {  // finished by seq_parts_kernel
          if (valid)
            store32(a.part + part_at<D>(a, w.part, static_cast<int64_t>(w.seg.k0) + w.first + row, w.hk) + h * D + k * 32, v);
          continue;
        }
        put_pieces32(pieces, v);
        __syncwarp();
        store_rows32(pieces, dst ? dst + k * 32 : nullptr, a.head_dim - k * 32);
        __syncwarp();
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      if (w.count > 0) mbar_arrive(&sb->acc_free);  // the sums have been read
      mbar_arrive(&sb->work_empty[slot]);
    }
  }
}

template <int D, bool KEYS>
__global__ void __launch_bounds__(kThreads, 1)
    seq_attention_bwd_kernel(const __grid_constant__ CUtensorMap tm_f0, const __grid_constant__ CUtensorMap tm_f1,
                             const __grid_constant__ CUtensorMap tm_m0, const __grid_constant__ CUtensorMap tm_m1,
                             const __grid_constant__ SeqAttnBwdArgs a, int first_next) {
  using C = Cfg<D, KEYS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Barriers* sb = reinterpret_cast<Barriers*>(smem + C::kBar);
  volatile int* abort_flag = &sb->abort_flag;
  auto f_tile = [&](int x) { return smem + x * C::kTileBytes; };
  auto m_tile = [&](int sl, int x) { return smem + C::kRing + sl * C::kSlotBytes + x * C::kHalfSlot; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.group, T = a.tile_tokens, U = a.unit_tokens;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sb->work_full[s], 1);
      mbar_init(&sb->work_empty[s], 1 + 2 + 8);  // warps 1, 2, 3 and the warps of rows
      mbar_init(&sb->sp_full[s], 1);
      mbar_init(&sb->pd_full[s], 128);
    }
    mbar_init(&sb->f_full, 1);
    mbar_init(&sb->f_copied, 256);
    mbar_init(&sb->f_empty, 1);
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&sb->st_full[s], KEYS ? 1 + 32 : 1);
      mbar_init(&sb->st_clean[s], KEYS ? 32 : 64);
      mbar_init(&sb->st_empty[s], 1);
      mbar_init(&sb->st_issued[s], 1);
    }
    mbar_init(&sb->done, 1);
    mbar_init(&sb->acc_free, 8);
    mbar_init(&sb->drain, 1);
    sb->abort_flag = 0;
    sb->progress = 0;
    fence_mbar_init();
  }
  if (KEYS && G * U < kUnit) {
    // rows that no box fills: the products that sum over a moving tile's rows read them
    const int rows = kUnit - G * U;
    for (int i = threadIdx.x; i < C::kSlots * 2 * (D / 64) * rows * 8; i += kThreads) {
      const int c = i % 8, r = G * U + (i / 8) % rows, blk = i / (8 * rows);
      *reinterpret_cast<uint4*>(smem + C::kRing + blk * C::kUnitBlock + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  if (KEYS && !C::kFInTmem) {
    // the last step's F side: ones in columns 0 to 2 for S, 3 to 5 for dP (32-byte swizzle: rows 4 to 7 of 8 have their halves
    // exchanged)
    for (int i = threadIdx.x; i < 2 * kSeqTile * 2; i += kThreads) {
      const int x = i / (2 * kSeqTile), r = i / 2 % kSeqTile, c = i & 1;
      const uint4 v = c ? make_uint4(0, 0, 0, 0) : x ? make_uint4(0, 0x3F800000u, 0x3F803F80u, 0) : make_uint4(0x3F803F80u, 0x3F80u, 0, 0);
      *reinterpret_cast<uint4*>(smem + C::kExt + C::kSlots * C::kExtM + x * C::kExtF + r * 32 + ((c ^ (r >> 2 & 1)) << 4)) = v;
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
  // The pass over queries reads nothing that the one over keys writes: it takes the SMs that run out of the other's items, and
  // only its end waits for that one's.  What it reads of this call's, the row sums and the counter, was complete when that one's CTAs
  // let this one start; it reads them in L2 (__ldcg, an atomic), where they are, as no wait of its own makes them visible to an SM.
  const bool behind = !KEYS && a.tokens_k > 0;
  if (!behind) pdl_wait();
  pdl_trigger();
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.status, kErrAttnWait)) != 0;
  };
  auto wait_item = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_item(bar, parity, &sb->progress, abort_flag, a.status, kErrAttnWait)) != 0;
  };

  if (warp >= 4) {
    more_registers<kBwdRows>();
    if (KEYS && C::kFInTmem && warp < 8) {  // published with the first item's F
      uint32_t r[16] = {0x3F803F80u, 0x3F80u, 0, 0, 0, 0, 0, 0, 0, 0x3F800000u, 0x3F803F80u, 0, 0, 0, 0, 0};
      tmem_st16(tmem + kTmExt + (static_cast<uint32_t>((warp & 3) * 32) << 16), r);
      tmem_st_wait();
    }
    rows_role<D, KEYS>(sb, smem, tmem, a);
  } else if (fewer_registers<kBwdService>(), warp == 0) {
    // ---------------- items and TMA
    if (lane == 0) tma_prefetch_desc(&tm_f0), tma_prefetch_desc(&tm_f1), tma_prefetch_desc(&tm_m0), tma_prefetch_desc(&tm_m1);
    uint32_t* counter = a.counters + (KEYS ? 0 : 1);
    const int bytes_f = KEYS ? C::kTileBytes : (D / 64) * G * T * 128, bytes_m = KEYS ? (D / 64) * G * U * 128 : C::kHalfSlot;
    TileOrder order;
    if constexpr (KEYS)
      order.init(a.cu_k, a.tokens_k, a.cu_q, a.tokens_q, a.batch, kSeqTile, a.causal, 0);  // the first keys have the most queries
    else
      order.init(a.cu_q, a.tokens_q, a.cu_k, a.tokens_k, a.batch, T, a.causal, 1);  // the last queries see the most keys
    const int items = order.n * a.hk * (KEYS ? a.parts : 1);
    uint32_t f_turn = 0, st_turn = 0, st_used = 0;
    int sl = 0;
    bool ok = true, f_used = false;
    auto take_slot = [&]() {  // the next slot of the ring, once it is empty
      ok = wait(&sb->st_empty[sl], (st_turn >> sl & 1u) ^ 1u);
      st_turn ^= 1u << sl;
      if (ok) st_used |= 1u << sl;
      return ok;
    };
    auto next_slot = [&]() { sl = sl + 1 == C::kSlots ? 0 : sl + 1; };
    int item = blockIdx.x;
    uint32_t steps = 0;
    auto progress = [&]() {
      if (lane == 0) *const_cast<volatile uint32_t*>(&sb->progress) = ++steps;
    };
    for (uint32_t it = 0; ok; ++it) {
      Work w;
      w.live = 0;
      for (; item < items; item = items > first_next ? next_of(first_next, ask_next(counter)) : items) {
        progress();
        TileOrder::Found at;
        if (!order.find(item / a.hk / (KEYS ? a.parts : 1), at)) continue;
        w.hk = item % a.hk, w.first = at.start, w.part = 0, w.parts = 1;
        if constexpr (KEYS) {
          w.seg = {at.other_first, at.other_count, at.first, at.count};
          const KeyTile t = key_tile(a, w.seg, w.first);
          w.part = item / a.hk % a.parts, w.parts = t.parts;
          if (w.part >= w.parts) continue;
          w.m_first = t.m_first + w.part * t.per_part * U;
          w.count = min(t.count - w.part * t.per_part, t.per_part);
          w.all_see = 0;
        } else {
          w.seg = {at.first, at.count, at.other_first, at.other_count};
          w.count = (keys_seen(w.seg, min(w.first + T, w.seg.n) - 1, a.causal) + kUnit - 1) / kUnit;
          w.m_first = 0;
          w.all_see = keys_seen(w.seg, w.first, a.causal);
        }
        set_cleaning<KEYS>(a, w);
        w.live = 1;
        break;
      }
      const int slot = it & 1;
      ok = wait(&sb->work_empty[slot], (it >> 1 & 1u) ^ 1u);
      if (!ok) break;
      if (lane == 0) {
        sb->work[slot] = w;
        *reinterpret_cast<volatile int*>(&sb->worst[slot]) = KEYS ? -1 : INT32_MAX;
        mbar_arrive(&sb->work_full[slot]);
      }
      __syncwarp();
      if (!w.live) break;
      if (w.count > 0) {
        const int f_head = KEYS ? w.hk : w.hk * G, f_row = KEYS ? w.seg.k0 + w.first : w.seg.q0 + w.first;
        if constexpr (C::kFInRing) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!take_slot()) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(&sb->st_full[sl], bytes_f);
#pragma unroll
              for (int b = 0; b < D / 64; ++b)
                tma_load_3d(m_tile(sl, 0) + b * kSeqBlock, x ? &tm_f1 : &tm_f0, &sb->st_full[sl], b * 64, f_head, f_row);
            }
            __syncwarp();
            next_slot();
          }
        } else {
          ok = wait(&sb->f_empty, f_turn ^ 1u);
          f_turn ^= 1u;
          if (ok) f_used = true;
          if (ok && lane == 0) {
            mbar_arrive_expect_tx(&sb->f_full, 2 * bytes_f);
#pragma unroll
            for (int b = 0; b < D / 64; ++b) {
              tma_load_3d(f_tile(0) + b * kSeqBlock, &tm_f0, &sb->f_full, b * 64, f_head, f_row);
              tma_load_3d(f_tile(1) + b * kSeqBlock, &tm_f1, &sb->f_full, b * 64, f_head, f_row);
            }
          }
          __syncwarp();
        }
      }
      // the next item's number is on its way while the last two units are, no sooner: a short item waits behind no long one
      const bool more = items > first_next;
      uint32_t ticket = 0;
      if (more && w.count == 0) ticket = ask_next(counter);
      for (int u = 0; ok && u < w.count; ++u) {
        progress();
        if (more && u == max(w.count - 2, 0)) ticket = ask_next(counter);
        if (!take_slot()) break;
        if (lane == 0) {
          const int m_head = KEYS ? w.hk * G : w.hk, row = KEYS ? w.seg.q0 + w.m_first + u * U : w.seg.k0 + u * kUnit;
          mbar_arrive_expect_tx(&sb->st_full[sl], 2 * bytes_m);
#pragma unroll
          for (int b = 0; b < D / 64; ++b) {
            tma_load_3d(m_tile(sl, 0) + b * C::kUnitBlock, &tm_m0, &sb->st_full[sl], b * 64, m_head, row);
            tma_load_3d(m_tile(sl, 1) + b * C::kUnitBlock, &tm_m1, &sb->st_full[sl], b * 64, m_head, row);
          }
          if (to_clean(w, u)) mbar_arrive(&sb->st_issued[sl]);
        }
        __syncwarp();
        next_slot();
      }
      item = more ? next_of(first_next, ticket) : items;
    }
    if (!ok) {
      // give the copies already issued a bounded chance to land before the CTA exits
      int never = 0;
      if (f_used) mbar_wait(&sb->f_full, f_turn ^ 1u, &never, a.status, 0);
      for (int s = 0; s < C::kSlots; ++s)
        if (st_used >> s & 1u) mbar_wait(&sb->st_full[s], (st_turn >> s & 1u) ^ 1u, &never, a.status, 0);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer: one lane issues, the warp stays converged; of a descriptor only the address in its lower half
    // changes (see attention_varlen.cu)
    auto koff = [](int k, int block) -> uint32_t { return static_cast<uint32_t>(((k >> 2) * block + (k & 3) * 32) >> 4); };
    auto desc = [](uint64_t base, uint32_t lo) { return (base & 0xFFFFFFFF00000000ull) | lo; };
    const uint64_t k_base = sdesc_kmajor_sw128(smem_addr(m_tile(0, 0))), n_base = sdesc_mnmajor_sw128(smem_addr(m_tile(0, 0)), C::kUnitBlock);
    uint32_t f_lo = static_cast<uint32_t>(sdesc_kmajor_sw128(smem_addr(f_tile(0)))), k_lo = static_cast<uint32_t>(k_base),
             n_lo = static_cast<uint32_t>(n_base);
    // the last step's rows of 32 bytes: 32-byte swizzle, 8 rows a group
    constexpr uint64_t kExtDesc = static_cast<uint64_t>(1) << 16 | static_cast<uint64_t>(256 >> 4) << 32 | static_cast<uint64_t>(1) << 46 |
                                  static_cast<uint64_t>(6) << 61;
    uint32_t e_lo = static_cast<uint32_t>(kExtDesc) | (smem_addr(smem + C::kExt) & 0x3FFFFu) >> 4;
    constexpr uint32_t kExtM = C::kExtM >> 4, kExtF = C::kExtF >> 4;
    constexpr uint32_t kSlot = static_cast<uint32_t>(C::kSlotBytes) >> 4, kHalf = static_cast<uint32_t>(C::kHalfSlot) >> 4,
                       kF = static_cast<uint32_t>(C::kTileBytes) >> 4;
    auto scores = [&](int sl, int h) {  // S and dP of the tile in slot sl into buffer h
      const uint32_t m_lo = k_lo + sl * kSlot;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t to = tmem + (x ? kTmD : kTmP) + 64 * h;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t m = desc(k_base, m_lo + x * kHalf + koff(k, C::kUnitBlock));
          if constexpr (C::kFInTmem)
            tc_mma_ts_f16(to, tmem + kTmF + x * (D / 2) + k * 8, m, C::kIdescS, k > 0 ? 1u : 0u);
          else
            tc_mma<kKindF16>(to, desc(k_base, f_lo + x * kF + koff(k, kSeqBlock)), m, C::kIdescS, k > 0 ? 1u : 0u);
        }
        if constexpr (KEYS) {
          const uint64_t m = desc(kExtDesc, e_lo + sl * kExtM);
          if constexpr (C::kFInTmem)
            tc_mma_ts_f16(to, tmem + kTmExt + x * 8, m, C::kIdescS, 1u);
          else
            tc_mma<kKindF16>(to, desc(kExtDesc, e_lo + C::kSlots * kExtM + x * kExtF), m, C::kIdescS, 1u);
        }
      }
      tc_commit(&sb->sp_full[h]);
    };
    auto products = [&](int sl, int h, uint32_t more) {
      const uint32_t m_lo = n_lo + sl * kSlot;
#pragma unroll
      for (int x = KEYS ? 0 : 1; x < 2; ++x)  // dV += P dO and dK += dS Q, or dQ += dS K
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_ts_f16(tmem + kTmAcc + (KEYS ? x * D : 0), tmem + (KEYS && x ? kTmD : kTmP) + 64 * h + 8 * k,
                        desc(n_base, m_lo + (x ? 0 : kHalf) + ((k * 2048) >> 4)), C::kIdescAcc, k > 0 ? 1u : more);
    };
    uint32_t f_turn = 0, st_turn = 0, clean_turn = 0, pd_turn = 0, acc_turn = 1;  // parities (st, clean: a bit for each slot, pd: for each buffer)
    int done_slot = 0, sl = 0;  // the ring's slots: of the products, of the scores (two tiles ahead)
    auto next = [&](int s) { return s + 1 == C::kSlots ? 0 : s + 1; };
    bool ok = true;
    for (uint32_t it = 0; ok; ++it) {
      const int slot = it & 1;
      ok = wait_item(&sb->work_full[slot], it >> 1 & 1u);
      if (!ok) break;
      const Work w = sb->work[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sb->work_empty[slot]);
      if (!w.live) break;
      if (w.count == 0) continue;
      ok = wait(C::kFInTmem ? &sb->f_copied : &sb->f_full, f_turn);
      f_turn ^= 1u;
      if (ok && C::kFInTmem) {
        if (C::kFInRing) {  // the two slots F came through
          if (lane < 2) mbar_arrive(&sb->st_empty[lane ? next(sl) : sl]);
          st_turn ^= (1u << sl) | (1u << next(sl));
          sl = next(next(sl)), done_slot = sl;
        } else if (lane == 0) {
          mbar_arrive(&sb->f_empty);
        }
        __syncwarp();
      }
      // whether the copies of tile u have been cleaned
      auto cleaned = [&](int u) {
        if (ok && to_clean(w, u)) {
          ok = wait(&sb->st_clean[sl], clean_turn >> sl & 1u);
          clean_turn ^= 1u << sl;
        }
        return ok;
      };
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (ok && h < w.count) {
          ok = wait(&sb->st_full[sl], st_turn >> sl & 1u);
          st_turn ^= 1u << sl;
          if (cleaned(h) && one_lane()) {
            tc_fence_after();
            scores(sl, h);
          }
          __syncwarp();
          sl = next(sl);
        }
      // a step: the products of tile u, the scores of tile u + 2 into the same buffer, and one commit, which stands for both
      for (int u0 = 0; ok && u0 < w.count; u0 += 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int u = u0 + h;
          if (!ok || u >= w.count) break;
          asm volatile("" : "+r"(f_lo), "+r"(k_lo), "+r"(n_lo), "+r"(e_lo));  // the sums below are formed here, not kept in registers
          const bool ahead = u + 2 < w.count;
          if (ahead && !cleaned(u + 2)) break;
          const bool acc_too = u == 0 && lane == 1, st_too = ahead && lane == 2;
          ok = wait(acc_too ? &sb->acc_free : st_too ? &sb->st_full[sl] : &sb->pd_full[h],
                    (acc_too ? acc_turn : st_too ? st_turn >> sl : pd_turn >> h) & 1u);
          pd_turn ^= 1u << h;
          if (ok && one_lane()) {
            tc_fence_after();
            products(done_slot, h, u > 0 ? 1u : 0u);
            if (ahead) scores(sl, h);
            if (u + 1 == w.count) tc_commit(&sb->done);
          }
          __syncwarp();
          done_slot = next(done_slot);
          if (ahead) st_turn ^= 1u << sl, sl = next(sl);
        }
      }
      acc_turn ^= 1u;
    }
    if (!ok && one_lane()) {
      int never = 0;
      tc_commit(&sb->drain);
      mbar_wait(&sb->drain, 0, &never, a.status, 0);
    }
  } else {
    // ---------------- keys: warp 2 the sums of the moving rows, warp 3 rows that part of F must not see; queries: both warps those
    const int tid = KEYS ? lane : static_cast<int>(threadIdx.x) - 64;
    uint32_t st_turn = 0, clean_turn = 0;  // a bit for each slot: the tile's turn, that of the next tile to clean
    int sl = 0;
    auto next_slot = [&]() {
      st_turn ^= 1u << sl;
      sl = sl + 1 == C::kSlots ? 0 : sl + 1;
    };
    bool ok = true;
    for (uint32_t it = 0; ok; ++it) {
      const int slot = it & 1;
      ok = wait_item(&sb->work_full[slot], it >> 1 & 1u);
      if (!ok) break;
      const Work w = sb->work[slot];
      if (C::kFInRing && w.live && w.count > 0) next_slot(), next_slot();
      const int count = w.live ? w.count : 0;
      if (KEYS && warp == 2) {
        // the sums of three tiles are on their way (one at a time they held the pass up: 1400 cycles a tile)
        constexpr int kAhead = 3;
        float2 fetched[kAhead][2];
        auto fetch = [&](int u, float2 (&to)[2]) {
          const int t = w.m_first + u * U, rows = u < count ? G * min(U, w.seg.n - t) : 0;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = lane + 32 * e;
            to[e] = make_float2(0.f, 0.f);
            if (r < rows) to[e] = a.sums[(static_cast<size_t>(w.seg.q0) + t + r / G) * a.hq + w.hk * G + r % G];
          }
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(i, fetched[i]);
        for (int u = 0; ok && u < count; ++u, next_slot()) {
          float2 s[2] = {fetched[0][0], fetched[0][1]};
#pragma unroll
          for (int i = 0; i + 1 < kAhead; ++i) fetched[i][0] = fetched[i + 1][0], fetched[i][1] = fetched[i + 1][1];
          fetch(u + kAhead, fetched[kAhead - 1]);
          ok = wait(&sb->st_empty[sl], (st_turn >> sl & 1u) ^ 1u);
          if (!ok) break;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = lane + 32 * e;
            uint32_t x[3], y[3];
            cut(s[e].x * a.minus_inv_scale, x), cut(-s[e].y, y);
            uint8_t* row = smem + C::kExt + sl * C::kExtM + r * 32;
            *reinterpret_cast<uint4*>(row + ((r >> 2 & 1) << 4)) = make_uint4(x[0] | x[1] << 16, x[2] | y[0] << 16, y[1] | y[2] << 16, 0);
            *reinterpret_cast<uint4*>(row + (((r >> 2 & 1) ^ 1) << 4)) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          mbar_arrive(&sb->st_full[sl]);
        }
      } else {
        for (int u = 0; ok && u < count; ++u, next_slot()) {
          if (!to_clean(w, u)) continue;
          int lo, hi, zero_from;
          rows_of<KEYS>(a, w, u, lo, hi, zero_from);
          if constexpr (KEYS) {  // rows to clean are noted in their sums
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = lane + 32 * e;
              if (r < hi) bad |= isnan(a.sums[(static_cast<size_t>(w.seg.q0) + w.m_first + u * U + r / G) * a.hq + w.hk * G + r % G].x);
            }
            if (!__any_sync(0xffffffffu, bad)) hi = 0;
          }
          ok = wait_item(&sb->st_issued[sl], clean_turn >> sl & 1u) && wait(&sb->st_full[sl], st_turn >> sl & 1u);
          clean_turn ^= 1u << sl;
          if (!ok) break;
          const int at = KEYS ? w.m_first + u * U : u * kUnit;
          scrub_pair<D, KEYS, KEYS ? 32 : 64>(m_tile(sl, 0), lo, hi, zero_from, at, KEYS ? G : 1, &sb->worst[slot], tid);
          if (KEYS) scrub_pair<D, KEYS, 32>(m_tile(sl, 1), lo, hi, zero_from, at, G, &sb->worst[slot], tid);
          fence_proxy_async_smem();
          mbar_arrive(&sb->st_clean[sl]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sb->work_empty[slot]);
      if (!w.live) break;
    }
  }

  if (behind) pdl_wait();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// (lse log2(e), dout . out) of every row, float32: LANES lanes to a row (16 bytes of it each), four rows in flight.  A row whose q
// or dout is not finite has NaN for the first, which tells the pass over keys to look at its tile.  Rows of no sequence are
// read and not used.
constexpr int kSumsRows = 4;
template <int LANES>
__global__ void __launch_bounds__(256) seq_sums_kernel(const __grid_constant__ SeqAttnBwdArgs a, Divisor by_heads) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0, a.counters[0] = 0, a.counters[1] = 0;
  constexpr int kAtOnce = 256 / LANES;
  const int lane = threadIdx.x & (LANES - 1), c = lane * 8;
  const int64_t rows = static_cast<int64_t>(a.tokens_q) * a.hq;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kAtOnce * kSumsRows + threadIdx.x / LANES;
  const bool there = c < a.head_dim;
  uint4 x[kSumsRows], y[kSumsRows], z[kSumsRows];
  float lse[kSumsRows];
#pragma unroll
  for (int e = 0; e < kSumsRows; ++e) {
    const int64_t row = row0 + kAtOnce * e;
    x[e] = y[e] = z[e] = make_uint4(0, 0, 0, 0), lse[e] = 0.f;
    if (row < rows && there) {
      const int t = by_heads.quotient(row), h = static_cast<int>(row - static_cast<int64_t>(t) * a.hq);
      auto at = [&](const HeadsView& v) {
        return *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(v.ptr) + t * v.stride_t + h * v.stride_h + c);
      };
      x[e] = at(a.dout), y[e] = at(a.out), z[e] = at(a.q);
      if (lane == 0) lse[e] = a.lse[row];
    }
  }
  const unsigned mine = (0xffffffffu >> (32 - LANES)) << (threadIdx.x & 31 & ~(LANES - 1));
#pragma unroll
  for (int e = 0; e < kSumsRows; ++e) {
    const int64_t row = row0 + kAtOnce * e;
    float s = bf16_lo(x[e].x) * bf16_lo(y[e].x) + bf16_hi(x[e].x) * bf16_hi(y[e].x) + bf16_lo(x[e].y) * bf16_lo(y[e].y) +
              bf16_hi(x[e].y) * bf16_hi(y[e].y) + bf16_lo(x[e].z) * bf16_lo(y[e].z) + bf16_hi(x[e].z) * bf16_hi(y[e].z) +
              bf16_lo(x[e].w) * bf16_lo(y[e].w) + bf16_hi(x[e].w) * bf16_hi(y[e].w);
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const bool bad = (__ballot_sync(0xffffffffu, not_finite(x[e]) || not_finite(z[e])) & mine) != 0;
    if (lane == 0 && row < rows) a.sums[row] = make_float2(bad ? __int_as_float(0x7FC00000) : lse[e] * kLog2e, s);
  }
}

// dk and dv of key rows whose queries were worked on in parts: the parts' float32 sums, added in their order.  A warp to a row,
// two key heads of it at a time.
template <int D>
__global__ void __launch_bounds__(256) seq_parts_kernel(const __grid_constant__ SeqAttnBwdArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  int parts = 0;
  if (row < a.tokens_k) {
    const int b = find_segment(a.batch, static_cast<int>(row), [&](int i) { return min(max(a.cu_k[i], 0), a.tokens_k); });
    Segment seg;
    clip_segment(a.cu_k, b, a.tokens_k, seg.k0, seg.m);
    clip_segment(a.cu_q, b, a.tokens_q, seg.q0, seg.n);
    if (row >= seg.k0 && row < seg.k0 + seg.m) parts = key_tile(a, seg, (static_cast<int>(row) - seg.k0) / kSeqTile * kSeqTile).parts;
  }
  pdl_wait();
  if (parts <= 1) return;
  constexpr int kCols = D / 16;  // of dv by the lower half of the lanes, of dk by the upper
  const HeadsView& out = lane < 16 ? a.dv : a.dk;
  const int col = (lane & 15) * kCols;
  for (int hk = 0; hk < a.hk; hk += 2) {
    float4 sum[2][kCols / 4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i) sum[h][i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int p = 0; p < parts; ++p)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4* v = reinterpret_cast<const float4*>(a.part + part_at<D>(a, p, row, min(hk + h, a.hk - 1)) + lane * kCols);
#pragma unroll
        for (int i = 0; i < kCols / 4; ++i) {
          const float4 x = v[i];
          sum[h][i].x += x.x, sum[h][i].y += x.y, sum[h][i].z += x.z, sum[h][i].w += x.w;
        }
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (hk + h >= a.hk) break;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out.ptr) + row * out.stride_t + (hk + h) * out.stride_h + col;
#pragma unroll
      for (int i = 0; i < kCols / 4; ++i)
        if (col + 4 * i < a.head_dim)
          reinterpret_cast<uint2*>(dst)[i] =
              make_uint2(pack_bf16x2(sum[h][i].x, sum[h][i].y), pack_bf16x2(sum[h][i].z, sum[h][i].w));
    }
  }
}

template <int D, bool KEYS>
cudaError_t launch_pass(const SeqAttnBwdArgs& a, const SeqAttnBwdMaps& m, cudaStream_t stream) {
  const int64_t items =
      ((KEYS ? a.tokens_k / kSeqTile : a.tokens_q / a.tile_tokens) + static_cast<int64_t>(a.batch)) * a.hk * (KEYS ? a.parts : 1);
  using C = Cfg<D, KEYS>;
  cudaError_t e = cudaFuncSetAttribute(seq_attention_bwd_kernel<D, KEYS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = static_cast<int>(std::min<int64_t>(items, num_sms()));
  e = launch_pdl(seq_attention_bwd_kernel<D, KEYS>, dim3(grid), dim3(kThreads), C::kSmem, stream, KEYS ? m.f_k : m.f_q,
                 KEYS ? m.f_v : m.f_dout, KEYS ? m.m_q : m.m_k, KEYS ? m.m_dout : m.m_v, a, grid);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_seq_attention_bwd(const SeqAttnBwdArgs& a, const SeqAttnBwdMaps& m, cudaStream_t stream) {
  // the first kernel also clears the status word and the counters
  const int64_t rows = static_cast<int64_t>(a.tokens_q) * a.hq;
  const int lanes = a.head_dim <= 64 ? 8 : 16, per_cta = 256 / lanes * kSumsRows;
  const dim3 sums_grid(static_cast<unsigned>(std::max<int64_t>((rows + per_cta - 1) / per_cta, 1)));
  cudaError_t e = lanes == 8 ? launch_pdl(seq_sums_kernel<8>, sums_grid, dim3(256), 0, stream, a, Divisor(a.hq))
                             : launch_pdl(seq_sums_kernel<16>, sums_grid, dim3(256), 0, stream, a, Divisor(a.hq));
  if (e != cudaSuccess) return e;
  count_launch();
  if (a.tokens_k > 0) {
    e = a.head_dim <= 64 ? launch_pass<64, true>(a, m, stream) : launch_pass<128, true>(a, m, stream);
    if (e != cudaSuccess) return e;
  }
  if (a.tokens_q > 0) {
    e = a.head_dim <= 64 ? launch_pass<64, false>(a, m, stream) : launch_pass<128, false>(a, m, stream);
    if (e != cudaSuccess) return e;
  }
  if (a.tokens_k > 0 && a.parts > 1) {
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.tokens_k) + 7) / 8));
    e = a.head_dim <= 64 ? launch_pdl(seq_parts_kernel<64>, grid, dim3(256), 0, stream, a)
                         : launch_pdl(seq_parts_kernel<128>, grid, dim3(256), 0, stream, a);
    if (e != cudaSuccess) return e;
    count_launch();
  }
  return cudaGetLastError();
}

}  // namespace mmdit
