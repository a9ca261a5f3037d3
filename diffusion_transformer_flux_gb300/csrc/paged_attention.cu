// paged_attention.cu -- attention of few rows over a paged cache (the single tokens of answering requests), and the
// join of a sequence's parts.
//
// The arithmetic is attention_varlen.cu's; here a sequence has at most 16 rows (new tokens by the heads of a group), so
// the cost is reading its keys and values once.  A CTA takes `few_keys` consecutive keys of one key head; its four warps
// take 16 keys in turn, each with its own ring of asynchronous copies, its own running maximum and its own float32
// output, so no warp waits for another before the end.  The products are mma.sync m16n8k16 (a tcgen05 product of 128
// rows would be seven eighths padding, and its hand-over through tensor memory costs more than these 32 instructions for
// 16 keys).  Rows of the ring that stand for no token are zeros (copies of size zero), so no stale value of a page enters.
//
// Sequences whose keys one CTA covers are written at once; the others leave normalised float32 parts and their log2-sums,
// which paged_combine_kernel adds in a fixed order.
#include "attention_tiles.cuh"

namespace mmdit {
namespace {

constexpr int kFewThreads = 128;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewKeys = 16;  // of a warp's tile
constexpr int kFewStages = 3;
constexpr float kFewThreshold = 8.0f;  // in log2 units: how far a maximum grows before the output is rescaled

template <int D>
struct FewCfg {
  static constexpr int kRow = D * 2;                 // bytes of a key
  static constexpr int kTile = kFewKeys * kRow;      // K or V of a tile
  static constexpr int kRing = kFewStages * 2 * kTile;
  static constexpr int kSmem = kFewWarps * kRing;
  static constexpr int kChunks = D / 8;              // 16-byte chunks of a key
};
static_assert(FewCfg<64>::kSmem >= kFewWarps * kFewRows * (64 + 2) * 4 &&
                  FewCfg<128>::kSmem >= kFewWarps * kFewRows * (128 + 2) * 4,
              "the parts of the warps lie in the rings at the end");

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Where row r of (sequence b, key head hk) lies in part `split` (in rows of D).
__device__ __forceinline__ size_t few_row(const SeqAttnArgs& a, int split, int b, int hk, int r) {
  return ((static_cast<size_t>(split) * a.batch + b) * a.hk + hk) * kFewRows + r;
}

// The byte of chunk c of key r in a tile: chunks of eight keys that lie behind one another fall on different banks.
template <int D>
__device__ __forceinline__ uint32_t few_at(int r, int c) {
  return static_cast<uint32_t>(r * FewCfg<D>::kRow + ((c ^ (r & 7)) << 4));
}

template <int D>
__global__ void __launch_bounds__(kFewThreads) paged_few_kernel(const __grid_constant__ SeqAttnArgs a) {
  using C = FewCfg<D>;
  extern __shared__ __align__(128) uint8_t few_smem[];
  __shared__ int worst[D];
  __shared__ int any_bad;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  if (a.clear && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.status = 0;
  const int hk = blockIdx.x % a.hk, b = blockIdx.x / a.hk, split = blockIdx.y;
  Segment seg;
  clip_segment(a.cu_q, b, a.tokens_q, seg.q0, seg.n);
  seg.k0 = 0, seg.m = min(max(a.kv_lens[b], 0), a.max_keys);
  const int rows = seg.n * a.group;
  if (rows == 0 || rows > kFewRows) return;
  const int n_splits = max((seg.m + a.few_keys - 1) / a.few_keys, 1);
  if (split >= n_splits) return;
  const int k_begin = split * a.few_keys, k_end = min(seg.m, k_begin + a.few_keys);
  const int* table = a.tables + static_cast<int64_t>(b) * a.table_width;
  uint8_t* ring = few_smem + warp * C::kRing;
  const uint32_t ring_s = smem_addr(ring);
  const int g = lane >> 2, t = lane & 3;  // the lane's rows g, g + 8 and columns 2t, 2t + 1 of a product's fragments
  const int chunk = lane % C::kChunks, key_of_lane = lane / C::kChunks;
  constexpr int kKeysPerStep = 32 / C::kChunks;
  const bool chunk_there = chunk * 8 < a.head_dim;
  const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(a.k_pages.ptr) + hk * a.k_pages.stride_h + chunk * 8;
  const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(a.v_pages.ptr) + hk * a.v_pages.stride_h + chunk * 8;
  const int n_tiles = (k_end - k_begin + kFewKeys - 1) / kFewKeys;
  const int page_mask = (1 << a.page_shift) - 1;

  if (threadIdx.x < D) worst[threadIdx.x] = INT32_MAX;
  if (threadIdx.x == 0) any_bad = 0;
  __syncthreads();
  int lim[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = g + 8 * h;
    lim[h] = r < rows ? keys_seen(seg, r / a.group, a.causal) : 0;
  }
  const int all_see = keys_seen(seg, 0, a.causal);
  // Q rows as the products' A fragments: 16-bit pairs (row g or g + 8, columns 16 k + 2t .. or + 8)
  uint32_t qf[D / 16][4];
#pragma unroll
  for (int k = 0; k < D / 16; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = g + 8 * (i & 1), col = 16 * k + 2 * t + 8 * (i >> 1);
      qf[k][i] = 0;
      if (r < rows && col < a.head_dim)
        qf[k][i] = *reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q.ptr) +
                                                      (static_cast<int64_t>(seg.q0) + r / a.group) * a.q.stride_t +
                                                      (hk * a.group + r % a.group) * a.q.stride_h + col);
    }
  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};

  // the pages that the two halves of a tile lie on (pages have at least 8 keys); -1: none
  auto pages_of = [&](int i, int (&p)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = k_begin + i * kFewKeys + 8 * h;
      const int v = i < n_tiles && key < k_end ? table[key >> a.page_shift] : -1;
      p[h] = v >= 0 && v < a.n_pages ? v : -1;
    }
  };
  uint32_t gone = 0;  // two bits a stage: halves of its tile without a page
  auto load = [&](int i, const int (&p)[2], int stage) {
    const int key0 = k_begin + i * kFewKeys;
    const uint32_t ks = ring_s + stage * 2 * C::kTile, vs = ks + C::kTile;
    gone = (gone & ~(3u << (2 * stage))) | (((p[0] < 0 ? 1u : 0u) | (p[1] < 0 ? 2u : 0u)) << (2 * stage));
#pragma unroll
    for (int s = 0; s < kFewKeys / kKeysPerStep; ++s) {
      const int r = s * kKeysPerStep + key_of_lane, key = key0 + r;
      const int64_t page = r < 8 ? p[0] : p[1], slot = key & page_mask;
      const bool there = key < k_end && page >= 0 && chunk_there;
      const __nv_bfloat16* ka = there ? kp + page * a.k_pages.stride_page + slot * a.k_pages.stride_t : kp - chunk * 8;
      const __nv_bfloat16* va = there ? vp + page * a.v_pages.stride_page + slot * a.v_pages.stride_t : vp - chunk * 8;
      copy16(ks + few_at<D>(r, chunk), ka, there);
      copy16(vs + few_at<D>(r, chunk), va, there);
    }
  };
  int next[2];
  pages_of(warp, next);
#pragma unroll
  for (int s = 0; s < kFewStages - 1; ++s) {
    const int i = warp + s * kFewWarps;
    if (i < n_tiles) load(i, next, s);
    copies_commit();
    pages_of(i + kFewWarps, next);
  }
  int stage = 0;
  for (int i = warp; i < n_tiles; i += kFewWarps) {
    copies_wait<kFewStages - 2>();
    __syncwarp();
    {
      // the stage that the step before read takes the tile kFewStages - 1 steps ahead
      const int ahead = i + (kFewStages - 1) * kFewWarps;
      if (ahead < n_tiles) load(ahead, next, stage == 0 ? kFewStages - 1 : stage - 1);
      copies_commit();
      pages_of(ahead + kFewWarps, next);
    }
    const int key0 = k_begin + i * kFewKeys;
    const uint32_t ks = ring_s + stage * 2 * C::kTile, vs = ks + C::kTile;
    const uint32_t lost = gone >> (2 * stage) & 3u;
    stage = stage + 1 == kFewStages ? 0 : stage + 1;
    // S = Q K^T: keys [0, 8) and [8, 16)
    float s0[4] = {0, 0, 0, 0}, s1[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t f[4];  // (keys 0-7, columns 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15)
      ldmatrix4(ks + few_at<D>((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), f);
      mma_bf16(s0, qf[k], f[0], f[1]);
      mma_bf16(s1, qf[k], f[2], f[3]);
    }
    uint32_t vf[D / 16][4];
#pragma unroll
    for (int n = 0; n < D / 16; ++n)  // (keys 0-7, columns 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15)
      ldmatrix4_trans(vs + few_at<D>(lane & 15, 2 * n + (lane >> 4)), vf[n]);
    if (key0 + kFewKeys > all_see || lost) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = key0 + 2 * t + (e & 1), l = lim[e >> 1];
        if (key >= l || (lost & 1u)) s0[e] = -INFINITY;
        if (key + 8 >= l || (lost & 2u)) s1[e] = -INFINITY;
      }
      // V rows that some of the rows must not see: see scrub_rows.  Register halves hold keys 2t and 2t + 1 (+ 8).
#pragma unroll
      for (int n = 0; n < D / 16; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = key0 + 2 * t + h + 8 * (e & 1), col = 16 * n + 8 * (e >> 1) + g;
            const uint32_t mask = 0x7F80u << (16 * h);
            if (key >= all_see && (vf[n][e] & mask) == mask) {
              vf[n][e] &= h ? 0x0000FFFFu : 0xFFFF0000u;
              atomicMin(&worst[col], key);
              any_bad = 1;
            }
          }
    }
    float mx[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(fmaxf(s0[2 * h], s0[2 * h + 1]), fmaxf(s1[2 * h], s1[2 * h + 1]));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2)) * a.scale_log2;
    }
    const bool up0 = mx[0] > m_run[0] + kFewThreshold, up1 = mx[1] > m_run[1] + kFewThreshold;
    if (__any_sync(0xffffffffu, up0 || up1)) {
      const float f0 = up0 ? fast_exp2(m_run[0] - mx[0]) : 1.f, f1 = up1 ? fast_exp2(m_run[1] - mx[1]) : 1.f;
      if (up0) m_run[0] = mx[0];
      if (up1) m_run[1] = mx[1];
      l_run[0] *= f0, l_run[1] *= f1;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) o[n][0] *= f0, o[n][1] *= f0, o[n][2] *= f1, o[n][3] *= f1;
    }
    uint32_t pf[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float m = m_run[h] == -INFINITY ? 0.f : m_run[h];
      const float p0 = fast_exp2(fmaf(s0[2 * h], a.scale_log2, -m)), p1 = fast_exp2(fmaf(s0[2 * h + 1], a.scale_log2, -m));
      const float p2 = fast_exp2(fmaf(s1[2 * h], a.scale_log2, -m)), p3 = fast_exp2(fmaf(s1[2 * h + 1], a.scale_log2, -m));
      l_run[h] += (p0 + p1) + (p2 + p3);
      pf[h] = pack_bf16x2(p0, p1), pf[2 + h] = pack_bf16x2(p2, p3);
    }
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      mma_bf16(o[2 * n], pf, vf[n][0], vf[n][1]);
      mma_bf16(o[2 * n + 1], pf, vf[n][2], vf[n][3]);
    }
    __syncwarp();
  }
  copies_wait<0>();
  // the warps' parts, over their rings: maximum and sum of 16 rows, then the rows
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 1);
    l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 2);
  }
  __syncthreads();
  float* parts = reinterpret_cast<float*>(few_smem);
  float* mine = parts + warp * kFewRows * (D + 2);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = g + 8 * h;
    if (t == 0) mine[r * 2] = m_run[h], mine[r * 2 + 1] = l_run[h];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<float2*>(mine + 2 * kFewRows + r * D + 8 * n + 2 * t) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
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
      const float e = p[r * 2] == -INFINITY ? 0.f : fast_exp2(p[r * 2] - top);
      const float2 v = *reinterpret_cast<const float2*>(p + 2 * kFewRows + r * D + col);
      sum += e * p[r * 2 + 1], x += e * v.x, y += e * v.y;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    x *= inv, y *= inv;
    if (any_bad) {
      const int l = keys_seen(seg, r / a.group, a.causal);
      if (worst[col] < l) x = __int_as_float(0x7FC00000);
      if (worst[col + 1] < l) y = __int_as_float(0x7FC00000);
    }
    const int64_t tok = static_cast<int64_t>(seg.q0) + r / a.group;
    const int head = hk * a.group + r % a.group;
    const float lse2 = sum == 0.f ? -INFINITY : top + log2f(sum);
    if (n_splits > 1) {
      const size_t at = few_row(a, split, b, hk, r);
      *reinterpret_cast<float2*>(a.few_part + at * D + col) = make_float2(x, y);
      if (col == 0) a.few_lse[at] = lse2;
    } else {
      if (col < a.head_dim)
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out.ptr) + tok * a.out.stride_t + head * a.out.stride_h + col) =
            pack_bf16x2(x, y);
      if (col == 0 && a.lse) a.lse[tok * a.hq + head] = lse2 * kLn2;
    }
  }
}

// One CTA for each (token, head) whose keys were split: out = sum_s 2^(L_s - L) O_s, L = log2 sum_s 2^L_s.  Warp w adds parts
// w, w + 4, ..., each lane D / 32 columns; the warps' sums are added in order.
template <int D>
__global__ void __launch_bounds__(128) paged_combine_kernel(const __grid_constant__ SeqAttnArgs a) {
  __shared__ float s_sum[4], s_top[4];
  __shared__ float s_out[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  const int tok = blockIdx.x, head = blockIdx.y;
  // the last sequence that starts at or before the token: empty ones before it share its start
  const int b = find_segment(a.batch, tok, [&](int i) { return min(max(a.cu_q[i], 0), a.tokens_q); });
  Segment seg;
  clip_segment(a.cu_q, b, a.tokens_q, seg.q0, seg.n);
  if (tok < seg.q0 || tok >= seg.q0 + seg.n) return;
  const int m = min(max(a.kv_lens[b], 0), a.max_keys);
  const bool few = seg.n * a.group <= a.few_rows;
  const int each = few ? a.few_keys : a.split_keys;
  const int n_splits = each > 0 ? (m + each - 1) / each : 1;
  if (n_splits <= 1) return;
  const float *part = few ? a.few_part : a.part, *part_lse = few ? a.few_lse : a.part_lse;
  const int hk = head / a.group, row = (tok - seg.q0) * a.group + head % a.group;
  const size_t at = few ? few_row(a, 0, b, hk, row) : static_cast<size_t>(tok) * a.hq + head;
  const size_t stride = few ? few_row(a, 1, 0, 0, 0) : static_cast<size_t>(a.tokens_q) * a.hq;
  float top = -INFINITY;
  for (int s = threadIdx.x; s < n_splits; s += 128) top = fmaxf(top, part_lse[s * stride + at]);
  top = warp_max(top);
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
  top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
  constexpr int kCols = D / 32;
  float sum = 0.f, v[kCols] = {};
#pragma unroll 4
  for (int s = warp; s < n_splits; s += 4) {
    const float l = part_lse[s * stride + at];
    const float* p = part + (s * stride + at) * D + lane * kCols;
    float u[kCols];
    if constexpr (kCols == 4) {
      const float4 w = *reinterpret_cast<const float4*>(p);
      u[0] = w.x, u[1] = w.y, u[2] = w.z, u[3] = w.w;
    } else {
      const float2 w = *reinterpret_cast<const float2*>(p);
      u[0] = w.x, u[1] = w.y;
    }
    // a part without keys counts for nothing, NaN log-sums (NaN scores) reach the output
    const float e = l == -INFINITY ? 0.f : fast_exp2(l - top);
    sum += e;
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[i] += e == 0.f && l == -INFINITY ? 0.f : e * u[i];
  }
#pragma unroll
  for (int i = 0; i < kCols; ++i) s_out[warp][lane * kCols + i] = v[i];
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  const float total = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
  const float inv = total == 0.f ? 0.f : 1.f / total;
  const int col = threadIdx.x * 2;
  if (col < a.head_dim) {
    const float x = ((s_out[0][col] + s_out[1][col]) + (s_out[2][col] + s_out[3][col])) * inv;
    const float y = ((s_out[0][col + 1] + s_out[1][col + 1]) + (s_out[2][col + 1] + s_out[3][col + 1])) * inv;
    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out.ptr) + tok * a.out.stride_t + head * a.out.stride_h + col) =
        pack_bf16x2(x, y);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[static_cast<size_t>(tok) * a.hq + head] = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
}

template <int D>
cudaError_t launch_few_dim(const SeqAttnArgs& a, int splits, cudaStream_t stream) {
  const cudaError_t e =
      cudaFuncSetAttribute(paged_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, FewCfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_few_kernel<D>, dim3(static_cast<unsigned>(a.batch) * a.hk, splits), dim3(kFewThreads), FewCfg<D>::kSmem,
                    stream, a);
}

}  // namespace

cudaError_t launch_paged_few(const SeqAttnArgs& a, int splits, cudaStream_t stream) {
  const cudaError_t e = a.head_dim <= 64 ? launch_few_dim<64>(a, splits, stream) : launch_few_dim<128>(a, splits, stream);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_paged_combine(const SeqAttnArgs& a, cudaStream_t stream) {
  const dim3 grid(a.tokens_q, a.hq);
  const cudaError_t e = a.head_dim <= 64 ? launch_pdl(paged_combine_kernel<64>, grid, dim3(128), 0, stream, a)
                                         : launch_pdl(paged_combine_kernel<128>, grid, dim3(128), 0, stream, a);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace mmdit
