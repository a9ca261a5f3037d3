// rmsnorm.cu -- the residual stream's addition, its RMSNorm and the E4M3 cast of the normalised row
// in one pass, and the norm's gradients.
//
// Forward, per row:   h = x + res  (rounded once to the residual's type: the value that is stored is
// the value that is normalised, so a backward pass that reads the stored h sees the same row),
//   r = 1 / sqrt(mean(h^2) + eps),   y = h r g,
// and y is written in the activation type, as E4M3 codes in 1 x 128 tiles with the scales of
// fp8_block_scale (block_scale.cuh), or both; the codes are cast from the float32 y, not from its
// bf16 rounding.
// Backward, with n = h r and a = dy g:   dh = r (a - n mean(a n)) + dh_in,   dg = sum over rows of dy n.
//
// Both are bound by memory: one row per CTA, read once into registers in 16-byte pieces, every
// statistic in float32.  A row of `dim` elements is dim / 8 chunks; thread t holds chunks t, t + T, ...
// (T threads, at most 4 chunks each), so a 128-wide tile's 16 chunks lie in 16 neighbouring lanes and
// its amax is four shuffles.
#include "block_scale.cuh"
#include "internal.h"
#include "rowwise.cuh"

namespace mmdit {
namespace {

constexpr int kNormMaxThreads = 512;

// Sum over the CTA's threads, the same in every thread; `red` holds one float per warp, and the
// caller alternates between two of them so that one barrier per call is enough.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < warps; ++i) t += red[i];
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
  __shared__ float red[2][kNormMaxThreads / 32];
  pdl_wait();
  const int chunks = a.dim >> 3;
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const TR* res = a.res ? static_cast<const TR*>(a.res) + row * a.dim : nullptr;
  float v[NC][8];
  Raw8<T> rx[NC];
  Raw8<TR> rr[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < chunks) {
      rx[i].load(x + 8 * c);
      if (res) rr[i].load(res + 8 * c);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < chunks) {
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
  const float r = 1.f / sqrtf(block_sum(ss, red[0]) / static_cast<float>(a.dim) + a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = r;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    const bool in = c < chunks;
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
  int rows, dim;
};

// CTA b takes rows b, b + gridDim.x, ... and keeps its share of dg in registers.
template <typename T, typename TR, int NC>
__global__ void __launch_bounds__(kNormMaxThreads) add_rmsnorm_bwd_kernel(const NormBwdArgs a) {
  __shared__ float red[2][kNormMaxThreads / 32];
  pdl_wait();
  const int chunks = a.dim >> 3;
  const float inv_dim = 1.f / static_cast<float>(a.dim);
  float dg[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[i][e] = 0.f;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const int64_t off = row * a.dim;
    Raw8<T> rdy[NC];
    Raw8<TR> rh[NC], rin[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < chunks) {
        rdy[i].load(static_cast<const T*>(a.dy) + off + 8 * c);
        rh[i].load(static_cast<const TR*>(a.h) + off + 8 * c);
        if (a.dh_in) rin[i].load(static_cast<const TR*>(a.dh_in) + off + 8 * c);
      }
    }
    const float r = __ldg(a.rstd + row);
    float av[NC][8], nv[NC][8];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < chunks) {
        float g[8], dy[8];
        load8(static_cast<const T*>(a.gain) + 8 * c, g);
        rdy[i].to_f32(dy);
        rh[i].to_f32(nv[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          nv[i][e] *= r;
          dg[i][e] = fmaf(dy[e], nv[i][e], dg[i][e]);
          av[i][e] = dy[e] * g[e];
          dot = fmaf(av[i][e], nv[i][e], dot);
        }
      }
    }
    const float mean = block_sum(dot, red[turn]) * inv_dim;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < chunks) {
        float d[8], in[8];
        if (a.dh_in) rin[i].to_f32(in);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          d[e] = r * (av[i][e] - nv[i][e] * mean);
          if (a.dh_in) d[e] += in[e];
        }
        store8(static_cast<TR*>(a.dh) + off + 8 * c, d);
        if (a.dx) store8(static_cast<T*>(a.dx) + off + 8 * c, d);
      }
    }
  }
  if (a.part) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < chunks) store8(a.part + static_cast<int64_t>(blockIdx.x) * a.dim + 8 * c, dg[i]);
    }
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

template <typename T, typename TR>
cudaError_t run_fwd(const NormFwdArgs& a, cudaStream_t stream) {
  const int chunks = a.dim / 8, nc = norm_nc(chunks, 256), threads = norm_threads(chunks, nc);
  auto kern = nc == 1 ? add_rmsnorm_fwd_kernel<T, TR, 1> : nc == 2 ? add_rmsnorm_fwd_kernel<T, TR, 2> : add_rmsnorm_fwd_kernel<T, TR, 4>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(a.rows)), dim3(threads), 0, stream, a);
}

template <typename T, typename TR>
cudaError_t run_bwd(const NormBwdArgs& a, int grid, cudaStream_t stream) {
  const int chunks = a.dim / 8, nc = norm_nc(chunks, 256), threads = norm_threads(chunks, nc);
  auto kern = nc == 1 ? add_rmsnorm_bwd_kernel<T, TR, 1> : nc == 2 ? add_rmsnorm_bwd_kernel<T, TR, 2> : add_rmsnorm_bwd_kernel<T, TR, 4>;
  return launch_pdl(kern, dim3(grid), dim3(threads), 0, stream, a);
}

}  // namespace

int add_rmsnorm_bwd_blocks(int rows) {
  const int most = 4 * num_sms();
  return rows < most ? rows : most;
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
                                   float* dgain, float* part, cudaStream_t stream) {
  if (rows <= 0) return cudaSuccess;
  const int grid = add_rmsnorm_bwd_blocks(rows);
  const NormBwdArgs a{dy, h, gain, rstd, dh_in, dh, dx, dgain ? part : nullptr, rows, dim};
  cudaError_t e = act == 0 ? run_bwd<float, float>(a, grid, stream)
                  : res_f32 ? run_bwd<__nv_bfloat16, float>(a, grid, stream)
                            : run_bwd<__nv_bfloat16, __nv_bfloat16>(a, grid, stream);
  if (e != cudaSuccess) return e;
  count_launch();
  if (dgain) return launch_colsum_finish(part, grid, dim, dgain, stream);
  return cudaGetLastError();
}

}  // namespace mmdit
