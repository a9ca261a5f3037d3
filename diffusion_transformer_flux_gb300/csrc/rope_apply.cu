// rope_apply.cu -- rotary positions applied to q and k, and the gradient of that.
//
// Pair j of a head's first rot_dim elements is (2j, 2j + 1) (interleaved) or (j, j + rot_dim / 2) (half):
//   (a, b) -> m (a cos - b sin, a sin + b cos),   angle p f_j, p the token's position,
// the rest of the head passes unchanged; the gradient is the transposed rotation (sin negated).  The
// angle comes either from the position and the frequencies of an mmdit_rope_cfg or from cos / sin tables.
//
// A position far into a context makes p f_j large, and a float32 angle would keep few bits of its
// fraction of a turn.  The configuration therefore holds f_j / 2 pi as a 64-bit fixed-point fraction of
// a turn, and the product with the integer position, taken modulo 2^64, is the exact fraction of the
// angle (negative positions included); its upper 32 bits feed sincospi.  The frequencies' own rounding
// (2^-53 relative, from the host's double) is then all that is left: 2^-36 of a turn at position 2^20.
//
// Bound by memory: each element read and written once.  A CTA takes TT tokens, its threads first form
// the tokens' cos and sin in shared memory (once for all heads), then rotate all heads of q and k in
// pieces of V elements per half (16-byte accesses for V = 8): interleaved pieces hold whole pairs;
// half pieces are a run of V first elements and the V second ones.  V is the largest of 8, 4, 2, 1 that
// divides rot_dim / 2.  A piece is read before it is written by the same thread, so the rotation may be
// done in place.
#include "../../include/mmdit.h"
#include "internal.h"
#include "rowwise.cuh"

namespace mmdit {
namespace {

constexpr int kRopeThreads = 256;

template <int P>
struct RopeTurns {
  uint64_t f[P];
};

struct RopeArgs {
  mmdit_rope_view in[2], out[2];  // q, k
  int heads[2];
  const int64_t* pos;
  int64_t pos_bstride;
  const float *cos, *sin;  // [batch, seq, pairs] tables, or null
  int64_t tokens;          // batch * seq
  int seq, head_dim, rot_dim;
  float mscale, sign;      // sign -1 for the gradient
};

// V elements <-> floats
template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float (&v)[V]) {
  if constexpr (V == 8) {
    load8(p, v);
  } else if constexpr (sizeof(T) == 2 && V == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
  } else if constexpr (sizeof(T) == 4 && V == 4) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = to_f32(p[i]);
  }
}
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&v)[V]) {
  if constexpr (V == 8) {
    store8(p, v);
  } else if constexpr (sizeof(T) == 2 && V == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else if constexpr (sizeof(T) == 4 && V == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) put(p + i, v[i]);
  }
}

template <typename T, int V, bool INTER, int P>
__global__ void __launch_bounds__(kRopeThreads) rope_apply_kernel(const RopeArgs a, const __grid_constant__ RopeTurns<P> turns,
                                                                  int tt) {
  extern __shared__ float table[];  // [tt][2][pairs]
  pdl_wait();
  const int pairs = a.rot_dim >> 1;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tt;
  const int n_tok = a.tokens - t0 < tt ? static_cast<int>(a.tokens - t0) : tt;
  for (int i = threadIdx.x; i < n_tok * pairs; i += kRopeThreads) {
    const int t = i / pairs, j = i - t * pairs;
    const int64_t tok = t0 + t;
    float c, s;
    if (a.cos) {
      c = __ldg(a.cos + tok * pairs + j), s = __ldg(a.sin + tok * pairs + j);
    } else {
      const int64_t b = tok / a.seq;
      const int64_t p = __ldg(a.pos + b * a.pos_bstride + (tok - b * a.seq));
      const uint64_t phase = static_cast<uint64_t>(p) * turns.f[j];
      // the signed fraction of a turn in half turns: [-1, 1)
      sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);
    }
    table[(2 * t) * pairs + j] = c * a.mscale;
    table[(2 * t + 1) * pairs + j] = s * a.mscale * a.sign;
  }
  __syncthreads();
  // pieces of a head: rotated ones, then the ones that pass
  const int turned = INTER ? (a.rot_dim + V - 1) / V : pairs / V;
  const int per_head = turned + (INTER ? a.head_dim / V - turned : (a.head_dim - a.rot_dim) / V);
  const int heads = a.heads[0] + a.heads[1];
  const int items = n_tok * heads * per_head;
  for (int i = threadIdx.x; i < items; i += kRopeThreads) {
    const int hh = i / per_head, piece = i - hh * per_head;
    const int t = hh / heads, h0 = hh - t * heads;
    const int which = h0 >= a.heads[0];
    const int h = which ? h0 - a.heads[0] : h0;
    const int64_t tok = t0 + t, b = tok / a.seq, s = tok - b * a.seq;
    const mmdit_rope_view &vi = a.in[which], &vo = a.out[which];
    const T* src = static_cast<const T*>(vi.ptr) + b * vi.stride_b + s * vi.stride_s + h * vi.stride_h;
    T* dst = static_cast<T*>(vo.ptr) + b * vo.stride_b + s * vo.stride_s + h * vo.stride_h;
    const float* cs = table + (2 * t) * pairs;
    const float* sn = cs + pairs;
    float x[V];
    if constexpr (INTER) {
      load_v<T, V>(src + piece * V, x);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        const int j = piece * (V / 2) + e;
        if (j < pairs) {
          const float u = x[2 * e], w = x[2 * e + 1];
          x[2 * e] = u * cs[j] - w * sn[j];
          x[2 * e + 1] = u * sn[j] + w * cs[j];
        }
      }
      store_v<T, V>(dst + piece * V, x);
    } else if (piece < turned) {
      float y[V];
      load_v<T, V>(src + piece * V, x);
      load_v<T, V>(src + pairs + piece * V, y);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float c = cs[piece * V + e], w = sn[piece * V + e];
        const float u = x[e];
        x[e] = u * c - y[e] * w;
        y[e] = u * w + y[e] * c;
      }
      store_v<T, V>(dst + piece * V, x);
      store_v<T, V>(dst + pairs + piece * V, y);
    } else {
      const int at = a.rot_dim + (piece - turned) * V;
      load_v<T, V>(src + at, x);
      store_v<T, V>(dst + at, x);
    }
  }
}

template <typename T, int P>
cudaError_t run_rope(const mmdit_rope_cfg& cfg, const RopeArgs& a, cudaStream_t stream) {
  RopeTurns<P> turns;
  const int pairs = cfg.rot_dim / 2;
  for (int j = 0; j < P; ++j) turns.f[j] = j < pairs ? cfg.turns[j] : 0;
  // A CTA per token while they are few; four tokens to a CTA once every SM has its fill
  const int tt = a.tokens >= 32 * static_cast<int64_t>(num_sms()) ? 4 : 1;
  const int64_t grid = (a.tokens + tt - 1) / tt;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const int v = pairs % 8 == 0 ? 8 : pairs % 4 == 0 ? 4 : pairs % 2 == 0 ? 2 : 1;
  auto kern = cfg.interleaved ? rope_apply_kernel<T, 8, true, P>
              : v == 8        ? rope_apply_kernel<T, 8, false, P>
              : v == 4        ? rope_apply_kernel<T, 4, false, P>
              : v == 2        ? rope_apply_kernel<T, 2, false, P>
                              : rope_apply_kernel<T, 1, false, P>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(kRopeThreads),
                    static_cast<size_t>(tt) * 2 * pairs * sizeof(float), stream, a, turns, tt);
}

}  // namespace

cudaError_t launch_rope_apply(int act, const mmdit_rope_cfg& cfg, int batch, int seq, int head_dim,
                              const mmdit_rope_view in[2], const mmdit_rope_view out[2], const int heads[2],
                              const int64_t* pos, int64_t pos_bstride, const float* cos, const float* sin,
                              int transposed, cudaStream_t stream) {
  RopeArgs a;
  for (int i = 0; i < 2; ++i) a.in[i] = in[i], a.out[i] = out[i], a.heads[i] = heads[i];
  a.pos = pos, a.pos_bstride = pos_bstride, a.cos = cos, a.sin = sin;
  a.tokens = static_cast<int64_t>(batch) * seq, a.seq = seq, a.head_dim = head_dim, a.rot_dim = cfg.rot_dim;
  a.mscale = cfg.mscale, a.sign = transposed ? -1.f : 1.f;
  if (a.tokens == 0 || heads[0] + heads[1] == 0) return cudaSuccess;
  // the frequencies travel as a kernel argument: 512 bytes for the usual heads, 2 KB for wide ones
  const bool few = cfg.rot_dim <= 128;
  const cudaError_t e = act == 1 ? (few ? run_rope<__nv_bfloat16, 64>(cfg, a, stream) : run_rope<__nv_bfloat16, 256>(cfg, a, stream))
                                 : (few ? run_rope<float, 64>(cfg, a, stream) : run_rope<float, 256>(cfg, a, stream));
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace mmdit
