// rmsnorm.cu -- the residual stream's addition, its RMSNorm and the E4M3 cast of the normalised row
// in one pass, and the norm's gradients.
//
// Forward, per row:   h = x + res  (rounded once to the residual's type: the value that is stored is
// the value that is normalised, so a backward pass that reads the stored h sees the same row),
//   r = 1 / sqrt(mean(h^2) + eps),   y = h r g,
// and y is written in the activation type, as E4M3 codes in 1 x 128 tiles with the scales of
// block_scale (block_scale.cuh), or both; the codes are cast from the float32 y, not from its
// bf16 rounding.
// Backward, with n = h r and a = dy g:   dh = r (a - n mean(a n)) + dh_in,   dg = sum over rows of dy n.
//
// Both are bound by memory: a row to a CTA (of short rows several), read once into registers in 16-byte pieces,
// every statistic in float32.  A row of `dim` elements is dim / 8 chunks; thread t holds chunks t, t + T, ...
// (T threads, at most 4 chunks each), so a 128-wide tile's 16 chunks lie in 16 neighbouring lanes and
// its amax is four shuffles.
#include "block_scale.cuh"
#include "internal.h"
#include "rowwise.cuh"

namespace mmdit {
namespace {

constexpr int kNormMaxThreads = 512;

// Sum over the blockDim.x threads of a row, the same in each of them.  `red` holds one float per warp of the
// CTA; a caller with several sums alternates between two of them, so that one barrier per sum is enough.
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;  // blockDim.x a multiple of 32: the row is this warp
  float* mine = red + threadIdx.y * warps;
  if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < warps; ++i) t += mine[i];
  return t;
}

template <typename T>
__device__ __forceinline__ float round_to(float v);
template <>
__device__ __forceinline__ float round_to<float>(float v) { return v; }
template <>
__device__ __forceinline__ float round_to<__nv_bfloat16>(float v) { return __bfloat162float(__float2bfloat16(v)); }

struct NormFwdArgs {
  const void *x, *res, *gain;
  void *h, *y;
  uint8_t* yq;
  float *sy, *rstd;
  int64_t ldx;
  int rows, dim;
  float eps;
};

template <typename T, typename TR, int NC>
__global__ void __launch_bounds__(kNormMaxThreads) add_rmsnorm_fwd_kernel(const NormFwdArgs a) {
  __shared__ float red[kNormMaxThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int chunks = a.dim >> 3;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool row_ok = row < a.rows;  // the rows behind the last take part in the barrier alone
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const TR* res = a.res ? static_cast<const TR*>(a.res) + row * a.dim : nullptr;
  float v[NC][8];
  Raw8<T> rx[NC];
  Raw8<TR> rr[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (row_ok && c < chunks) {
      rx[i].load(x + 8 * c);
      if (res) rr[i].load_rw(res + 8 * c);  // h may be the residual itself
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (row_ok && c < chunks) {
      rx[i].to_f32(v[i]);
      if (res) {
        float w[8];
        rr[i].to_f32(w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = round_to<TR>(v[i][e] + w[e]);
        if (a.h) store8(static_cast<TR*>(a.h) + row * a.dim + 8 * c, v[i]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    }
  }
  const float r = 1.f / sqrtf(row_sum(ss, red) / static_cast<float>(a.dim) + a.eps);
  if (a.rstd && row_ok && threadIdx.x == 0) a.rstd[row] = r;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    const bool in = row_ok && c < chunks;
    if (in) {
      float g[8];
      load8(static_cast<const T*>(a.gain) + 8 * c, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * r * g[e];
      if (a.y) store8(static_cast<T*>(a.y) + row * a.dim + 8 * c, v[i]);
    }
    if (a.yq) {  // every lane takes part in the shuffles; chunks behind the row hold zeros
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[i][e]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float s = block_scale(m);
      if (in) {
        *reinterpret_cast<uint2*>(a.yq + row * a.dim + 8 * c) = e4m3x8(v[i], s);
        if ((c & 15) == 0) a.sy[static_cast<int64_t>(c >> 4) * a.rows + row] = s;
      }
    }
  }
}

struct NormBwdArgs {
  const void *dy, *h, *gain;
  const float* rstd;
  const void* dh_in;
  void *dh, *dx;
  float* part;  // [gridDim.x, dim], or null
  uint32_t* status;  // cleared
  int rows, dim;
};

// A CTA holds blockDim.y groups of blockDim.x threads; group k of all groups takes rows k, k + groups, ... and
// keeps its share of dg in registers.  A row's operands stay packed as they were loaded while the row's sum is
// formed (12 registers per 8 bf16 elements instead of 24 float32 ones) and the next row's are already on
// their way, so two CTAs to an SM keep the memory busy: 4095 x 5120 bf16 in 33.1 us, 5.1 TB/s, the sums of dg and
// their second kernel included (floats kept across the sum, no prefetch: 60 us).
template <typename T, typename TR, int NC, int MAX>
__global__ void __launch_bounds__(MAX, MAX <= 320 ? 2 : 1) add_rmsnorm_bwd_kernel(const NormBwdArgs a) {
  __shared__ float red[2][MAX / 32];
  __shared__ float sums[NC == 1 ? 2048 : 1];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0 && threadIdx.y == 0) *a.status = 0;
  const int chunks = a.dim >> 3;
  const float inv_dim = 1.f / static_cast<float>(a.dim);
  const int64_t groups = static_cast<int64_t>(gridDim.x) * blockDim.y, group = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  float dg[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[i][e] = 0.f;
  struct Row {
    Raw8<T> dy[NC];
    Raw8<TR> h[NC], in[NC];
    float r;
  };
  auto load = [&](int64_t row, Row& x) {
    if (row >= a.rows) return;
    const int64_t off = row * a.dim;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < chunks) {
        x.dy[i].load(static_cast<const T*>(a.dy) + off + 8 * c);
        x.h[i].load(static_cast<const TR*>(a.h) + off + 8 * c);
        if (a.dh_in) x.in[i].load_rw(static_cast<const TR*>(a.dh_in) + off + 8 * c);  // dh may be dh_in itself
      }
    }
    x.r = __ldg(a.rstd + row);
  };
  Row cur, next;
  load(group, cur);
  int turn = 0;
  // every group of a CTA makes the same number of turns: the row's sum is a barrier of the whole CTA
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * blockDim.y; base < a.rows; base += groups, turn ^= 1) {
    const int64_t row = base + threadIdx.y;
    if constexpr (NC <= 2) load(row + groups, next);
    float dot = 0.f;
    if (row < a.rows) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < chunks) {
          float g[8], dy[8], n[8];
          load8(static_cast<const T*>(a.gain) + 8 * c, g);
          cur.dy[i].to_f32(dy);
          cur.h[i].to_f32(n);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float t = dy[e] * (n[e] * cur.r);
            dg[i][e] += t;
            dot = fmaf(t, g[e], dot);
          }
        }
      }
    }
    const float mean = row_sum(dot, red[turn]) * inv_dim;
    if (row < a.rows) {
      const int64_t off = row * a.dim;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < chunks) {
          float g[8], dy[8], n[8], d[8];
          load8(static_cast<const T*>(a.gain) + 8 * c, g);
          cur.dy[i].to_f32(dy);
          cur.h[i].to_f32(n);
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = cur.r * (dy[e] * g[e] - n[e] * cur.r * mean);
          if (a.dh_in) {
            float in[8];
            cur.in[i].to_f32(in);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] += in[e];
          }
          store8(static_cast<TR*>(a.dh) + off + 8 * c, d);
          if (a.dx) store8(static_cast<T*>(a.dx) + off + 8 * c, d);
        }
      }
    }
    if constexpr (NC <= 2)
      cur = next;
    else
      load(row + groups, cur);
  }
  if (!a.part) return;
  if constexpr (NC == 1) {
    if (blockDim.y > 1) {  // the CTA's groups first, in order
      float* mine = sums + (threadIdx.y * blockDim.x + threadIdx.x) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) mine[e] = dg[0][e];
      __syncthreads();
      if (threadIdx.y > 0) return;
      for (int k = 1; k < static_cast<int>(blockDim.y); ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) dg[0][e] += mine[k * blockDim.x * 8 + e];
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < chunks) store8(a.part + static_cast<int64_t>(blockIdx.x) * a.dim + 8 * c, dg[i]);
  }
}

// Threads and chunks per thread of a row of `chunks` 8-element chunks: the fewest chunks per thread
// (1, 2 or 4) with at most `most` threads.
inline int norm_threads(int chunks, int nc) { return ((chunks + nc - 1) / nc + 31) / 32 * 32; }
inline int norm_nc(int chunks, int most) {
  for (int nc = 1; nc < 4; nc *= 2)
    if (norm_threads(chunks, nc) <= most) return nc;
  return 4;
}

// Rows to a CTA: short rows share one of 256 threads (16384 x 256 in CTAs of one warp: 10.6 us, of eight rows 6.2).
inline int norm_rows(int threads) { return threads < 256 ? 256 / threads : 1; }

template <typename T, typename TR>
cudaError_t run_fwd(const NormFwdArgs& a, cudaStream_t stream) {
  const int chunks = a.dim / 8, nc = norm_nc(chunks, 256), threads = norm_threads(chunks, nc), rows = norm_rows(threads);
  auto kern = nc == 1 ? add_rmsnorm_fwd_kernel<T, TR, 1> : nc == 2 ? add_rmsnorm_fwd_kernel<T, TR, 2> : add_rmsnorm_fwd_kernel<T, TR, 4>;
  return launch_pdl(kern, dim3(static_cast<unsigned>((a.rows + static_cast<int64_t>(rows) - 1) / rows)), dim3(threads, rows), 0,
                    stream, a);
}

// The backward's launch: chunks per thread, threads of a row, rows of a CTA and CTAs, each with its sums of dg: four
// CTAs to an SM with one chunk per thread, two otherwise.  By registers fewer stay resident: three with one chunk (72;
// with a float32 stream two, 93 to 96), two of up to 320 threads with more, one of the 512-thread forms (111 to 128).
// Where the launch has more than that, its last turn is partly empty: 20479 x 1024 bf16 42.6 us, 3.9 TB/s, 3411 x
// 6144 38.6 us, 4.4 TB/s (5119 x 4096 and 4095 x 5120, whose CTAs all stay: 33 us, 5.1 TB/s).  320 threads is what
// two CTAs of 96 registers have room for; for them the float32-stream forms spill 76 and 204 bytes (4095 x 5120 with
// a float32 stream: 61.0 us, 4.8 TB/s; 5119 x 4096 50.3 us, 5.8 TB/s).
struct BwdShape {
  int nc, threads, rows, grid;
};
BwdShape bwd_shape(int rows, int dim) {
  BwdShape s;
  const int chunks = dim / 8;
  s.nc = chunks <= 256 ? 1 : chunks <= 2 * kNormMaxThreads ? 2 : 4;
  s.threads = norm_threads(chunks, s.nc);
  s.rows = norm_rows(s.threads);
  const int ctas = rows / s.rows + (rows % s.rows != 0), most = (s.nc == 1 ? 4 : 2) * num_sms();
  s.grid = ctas < most ? ctas : most;
  return s;
}

template <typename T, typename TR>
cudaError_t run_bwd(const NormBwdArgs& a, const BwdShape& s, cudaStream_t stream) {
  auto kern = s.nc == 1                       ? add_rmsnorm_bwd_kernel<T, TR, 1, 256>
              : s.nc == 2 && s.threads <= 256 ? add_rmsnorm_bwd_kernel<T, TR, 2, 256>
              : s.nc == 2 && s.threads <= 320 ? add_rmsnorm_bwd_kernel<T, TR, 2, 320>
              : s.nc == 2                     ? add_rmsnorm_bwd_kernel<T, TR, 2, kNormMaxThreads>
                                              : add_rmsnorm_bwd_kernel<T, TR, 4, kNormMaxThreads>;
  return launch_pdl(kern, dim3(s.grid), dim3(s.threads, s.rows), 0, stream, a);
}

}  // namespace

int add_rmsnorm_bwd_parts(int rows, int dim) {
  return bwd_shape(rows, dim).grid;
}

cudaError_t launch_add_rmsnorm_fwd(int act, int res_f32, int rows, int dim, float eps, const void* x, int64_t ldx,
                                   const void* res, const void* gain, void* h, void* y, uint8_t* yq, float* sy,
                                   float* rstd, cudaStream_t stream) {
  if (rows <= 0) return cudaSuccess;
  const NormFwdArgs a{x, res, gain, h, y, yq, sy, rstd, ldx, rows, dim, eps};
  cudaError_t e = act == 0 ? run_fwd<float, float>(a, stream)
                  : res_f32 ? run_fwd<__nv_bfloat16, float>(a, stream)
                            : run_fwd<__nv_bfloat16, __nv_bfloat16>(a, stream);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_add_rmsnorm_bwd(int act, int res_f32, int rows, int dim, const void* dy, const void* h,
                                   const void* gain, const float* rstd, const void* dh_in, void* dh, void* dx,
                                   float* dgain, float* part, uint32_t* status, cudaStream_t stream) {
  if (rows <= 0) return cudaSuccess;
  const BwdShape s = bwd_shape(rows, dim);
  const NormBwdArgs a{dy, h, gain, rstd, dh_in, dh, dx, dgain ? part : nullptr, status, rows, dim};
  cudaError_t e = act == 0 ? run_bwd<float, float>(a, s, stream)
                  : res_f32 ? run_bwd<__nv_bfloat16, float>(a, s, stream)
                            : run_bwd<__nv_bfloat16, __nv_bfloat16>(a, s, stream);
  if (e != cudaSuccess) return e;
  count_launch();
  if (dgain) return launch_colsum_finish(part, s.grid, dim, dgain, stream);
  return cudaGetLastError();
}

}  // namespace mmdit
