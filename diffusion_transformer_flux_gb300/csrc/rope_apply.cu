// rope_apply.cu -- rotary positions applied to q and k, and the gradient of that.
//
// Pair j of a head's first rot_dim elements is (2j, 2j + 1) (interleaved) or (j, j + rot_dim / 2) (half):
//   (a, b) -> m (a cos - b sin, a sin + b cos),   angle p f_j, p the token's position,
// the rest of the head passes unchanged; the gradient is the transposed rotation (sin negated).  The
// angle comes either from the position and the frequencies of an mmdit_rope_cfg or from cos / sin tables.
//
// A position far into a context makes p f_j large, and a float32 angle would keep few bits of its
// fraction of a turn.  The configuration therefore holds f_j / 2 pi as a 64-bit fixed-point fraction of
// a turn, and the product with the integer position, taken modulo 2^64, is the exact fraction of its
// angle (negative positions included).  The fraction's upper 32 bits, as a float32 number of half turns, feed
// sincospi: off by at most 2^-26 of a turn at every position.  The held frequency is itself rounded, by
// 5 2^-53 of itself (four operations in double on the host) and the 64th bit, so position p adds
// |p| (f 5 2^-53 / 2 pi + 2^-64) of a turn: 2^-33 at 2^20, as much as the rest from 2^27 on.
//
// Bound by memory: each element read and written once.  Thread (x, y, z) of a CTA takes piece x of heads y,
// y + blockDim.y, ... of token z: interleaved pieces are 8 elements, half pieces a run of V first elements and the
// V second ones, V the largest of 8, 4, 2, 1 that divides rot_dim / 2; the pieces behind rot_dim pass.  The first
// heads' loads are on their way while the CTA forms its tokens' cos and sin in shared memory, once for all
// heads.  A CTA holds as many heads as it has threads for, and more tokens where a token has few: 2 x 4608
// tokens of 32 + 8 heads of 128, interleaved, in 32.5 us, 5.8 TB/s (a CTA that walks four tokens in turn: 75 us,
// one list of items with divided indices: 51, 64-bit divisions of the token alone: 41).  V of 2 and 1 load and store
// single elements, behind rot_dim too: 2 x 4608 tokens of 40 heads of 80 with 20 rotated take 82.9 us in the half
// layout, interleaved 24.7.  A piece is read before it is written by the same thread, so the rotation may be done
// in place.
#include <algorithm>

#include "../../include/mmdit.h"
#include "internal.h"
#include "rowwise.cuh"

namespace mmdit {
namespace {

constexpr int kRopeThreads = 256;     // of a CTA where a head has at most as many pieces
constexpr int kRopeMaxThreads = 512;  // head_dim 512 with V = 1 has up to 511

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

// A piece as loaded: packed for the 16-byte ones, so that several fit a thread's registers.  The loads are plain: the
// heads may be rotated in place.
template <typename T, int V>
struct Piece {
  float v[V];
  __device__ __forceinline__ void load(const T* p) { load_v<T, V>(p, v); }
  __device__ __forceinline__ void to_f32(float (&x)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = v[i];
  }
};
template <>
struct Piece<__nv_bfloat16, 8> : Raw8<__nv_bfloat16> {
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { load_rw(p); }
};

template <typename T, int V, bool INTER, int P>
__global__ void __launch_bounds__(kRopeMaxThreads, 2) rope_apply_kernel(const RopeArgs a, const __grid_constant__ RopeTurns<P> turns) {
  extern __shared__ float table[];  // [tokens of the CTA][2][stride]
  constexpr int kU = INTER ? 4 : 2;          // heads in flight
  constexpr int kPairs = INTER ? V / 2 : V;  // pairs of a piece
  pdl_wait();
  pdl_trigger();
  const int pairs = a.rot_dim >> 1, stride = (pairs + 3) & ~3;
  const int b = blockIdx.y, s0 = blockIdx.x * blockDim.z, s = s0 + threadIdx.z;  // the grid is (token groups, batch)
  const int piece = threadIdx.x, turned = INTER ? (a.rot_dim + V - 1) / V : pairs / V;
  const bool turn = piece < turned;
  const int at = INTER || turn ? piece * V : a.rot_dim + (piece - turned) * V;
  // where head 0 of q (and of k, as far before it as q has heads) has this piece
  const int hq = a.heads[0];
  auto base = [&](const mmdit_rope_view& v, int before) {
    return static_cast<T*>(v.ptr) + b * v.stride_b + s * v.stride_s - before * v.stride_h + at;
  };
  const T *src_q = base(a.in[0], 0), *src_k = base(a.in[1], hq);
  T *dst_q = base(a.out[0], 0), *dst_k = base(a.out[1], hq);
  const int heads = s < a.seq ? hq + a.heads[1] : 0;
  const float* cs = table + 2 * threadIdx.z * stride + piece * kPairs;
  const float* sn = cs + stride;
  for (int h0 = threadIdx.y, first = 1; first || h0 < heads; h0 += kU * blockDim.y, first = 0) {
    Piece<T, V> x[kU], y[INTER ? 1 : kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int h = h0 + u * blockDim.y;
      if (h < heads) {
        const T* p = h < hq ? src_q + h * a.in[0].stride_h : src_k + h * a.in[1].stride_h;
        x[u].load(p);
        if constexpr (!INTER)
          if (turn) y[u].load(p + pairs);
      }
    }
    if (first) {
      const int threads = blockDim.x * blockDim.y * blockDim.z;
      const int tid = (threadIdx.z * blockDim.y + threadIdx.y) * blockDim.x + threadIdx.x;
      for (int i = tid; i < static_cast<int>(blockDim.z) * pairs; i += threads) {
        const int t = i / pairs, j = i - t * pairs;
        if (s0 + t >= a.seq) break;
        float c, w;
        if (a.cos) {
          const int64_t row = (static_cast<int64_t>(b) * a.seq + s0 + t) * pairs + j;
          c = __ldg(a.cos + row), w = __ldg(a.sin + row);
        } else {
          const int64_t pos = __ldg(a.pos + b * a.pos_bstride + s0 + t);
          const uint64_t phase = static_cast<uint64_t>(pos) * turns.f[j];
          // the signed fraction of a turn in half turns: [-1, 1)
          sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &w, &c);
        }
        table[2 * t * stride + j] = c * a.mscale;
        table[(2 * t + 1) * stride + j] = w * a.mscale * a.sign;
      }
      __syncthreads();
    }
    // the piece's cos and sin: in registers for all heads where they are few, else read at each use (16 more
    // registers would cost a quarter of the resident CTAs)
    float c[kPairs], n[kPairs];
    if (INTER && turn) {
      load_v<float, kPairs>(cs, c);
      load_v<float, kPairs>(sn, n);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int h = h0 + u * blockDim.y;
      if (h >= heads) continue;
      T* out = h < hq ? dst_q + h * a.out[0].stride_h : dst_k + h * a.out[1].stride_h;
      float v[V], w[V];
      x[u].to_f32(v);
      if (turn) {
        if constexpr (INTER) {
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            if (piece * kPairs + e < pairs) {  // the last piece may end behind rot_dim
              const float p = v[2 * e], q = v[2 * e + 1];
              v[2 * e] = p * c[e] - q * n[e], v[2 * e + 1] = p * n[e] + q * c[e];
            }
          }
        } else {
          y[u].to_f32(w);
          load_v<float, kPairs>(cs, c);
          load_v<float, kPairs>(sn, n);
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            const float p = v[e], q = w[e];
            v[e] = p * c[e] - q * n[e], w[e] = p * n[e] + q * c[e];
          }
          store_v<T, V>(out + pairs, w);
        }
      }
      store_v<T, V>(out, v);
    }
  }
}

template <typename T, int P>
cudaError_t run_rope(const mmdit_rope_cfg& cfg, const RopeArgs& a, int batch, cudaStream_t stream) {
  RopeTurns<P> turns;
  const int pairs = cfg.rot_dim / 2;
  for (int j = 0; j < P; ++j) turns.f[j] = j < pairs ? cfg.turns[j] : 0;
  const int v = pairs % 8 == 0 ? 8 : pairs % 4 == 0 ? 4 : pairs % 2 == 0 ? 2 : 1;
  auto kern = cfg.interleaved ? rope_apply_kernel<T, 8, true, P>
              : v == 8        ? rope_apply_kernel<T, 8, false, P>
              : v == 4        ? rope_apply_kernel<T, 4, false, P>
              : v == 2        ? rope_apply_kernel<T, 2, false, P>
                              : rope_apply_kernel<T, 1, false, P>;
  // pieces of a head, heads of a CTA (each thread takes as many as it keeps in flight) and tokens of a CTA,
  // one while there are too few of them to fill the SMs
  const int turned = cfg.interleaved ? (cfg.rot_dim + 7) / 8 : pairs / v;
  const int pieces = cfg.interleaved ? a.head_dim / 8 : turned + (a.head_dim - cfg.rot_dim) / v;
  const int heads = a.heads[0] + a.heads[1], most = kRopeThreads / pieces > 0 ? kRopeThreads / pieces : 1;
  const int flight = cfg.interleaved ? 4 : 2, per = (heads + flight - 1) / flight, y = per < most ? per : most;
  const int64_t tokens = static_cast<int64_t>(batch) * a.seq;
  int64_t z = kRopeThreads / (pieces * y);
  z = std::max<int64_t>(1, std::min<int64_t>({z, 8, a.seq, tokens / (4 * num_sms())}));
  const dim3 grid(static_cast<unsigned>((a.seq + z - 1) / z), static_cast<unsigned>(batch));
  return launch_pdl(kern, grid, dim3(pieces, y, static_cast<unsigned>(z)),
                    static_cast<size_t>(z) * 2 * ((pairs + 3) / 4 * 4) * sizeof(float), stream, a, turns);
}

}  // namespace

cudaError_t launch_rope_apply(int act, const mmdit_rope_cfg& cfg, int batch, int seq, int head_dim,
                              const mmdit_rope_view in[2], const mmdit_rope_view out[2], const int heads[2],
                              const int64_t* pos, int64_t pos_bstride, const float* cos, const float* sin,
                              int transposed, cudaStream_t stream) {
  RopeArgs a;
  for (int i = 0; i < 2; ++i) a.in[i] = in[i], a.out[i] = out[i], a.heads[i] = heads[i];
  a.pos = pos, a.pos_bstride = pos_bstride, a.cos = cos, a.sin = sin;
  a.seq = seq, a.head_dim = head_dim, a.rot_dim = cfg.rot_dim;
  a.mscale = cfg.mscale, a.sign = transposed ? -1.f : 1.f;
  if (batch == 0 || seq == 0 || heads[0] + heads[1] == 0) return cudaSuccess;
  // the frequencies travel as a kernel argument: 512 bytes for the usual heads, 2 KB for wide ones
  const bool few = cfg.rot_dim <= 128;
  const cudaError_t e = act == 1 ? (few ? run_rope<__nv_bfloat16, 64>(cfg, a, batch, stream) : run_rope<__nv_bfloat16, 256>(cfg, a, batch, stream))
                                 : (few ? run_rope<float, 64>(cfg, a, batch, stream) : run_rope<float, 256>(cfg, a, batch, stream));
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace mmdit
