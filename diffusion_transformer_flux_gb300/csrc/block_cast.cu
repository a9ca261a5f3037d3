// block_cast.cu -- E4M3 casts with a scale for each block of 128: the operands of the block-scaled
// linear and of its gradients, from one read of the source.
//
// Activations and gradients x [R, C] are cast in 1 x 128 tiles along their rows (q [R, C], s
// [ceil(C/128), R]) and, for a product that contracts over the rows, in 128 x 1 tiles of their columns
// stored transposed (q_t [C, ld], s_t [ceil(R/128), C]); weights in 128 x 128 tiles, whose codes serve
// both directions under one scale (s [ceil(R/128), ceil(C/128)]).  ld is R rounded up to 16, the codes
// behind column R are zero.  A scale is block_scale(amax) (block_scale.cuh), a code E4M3(v s), v s in
// float32, rounded to nearest even.  With `part` the call also leaves each 128-row block's column sums
// of x there (fixed order), of which a bias gradient is made.
//
// Bound by memory: 2 (or 4) bytes read and 2 written per element.  One CTA per 128 x 128 tile; thread
// (g, c) of 16 x 16 holds rows 8 g .. 8 g + 7 of the 8 columns 8 c .. 8 c + 7, so that a row tile's amax
// is a shuffle over 16 lanes, a column's is 8 register maxima and one pass through shared memory, and
// the transposed codes of a column are 8 neighbouring bytes.  They are turned through shared memory in
// 8-byte pieces, piece g of column k at place g ^ (k / 8), which spreads a half warp's stores over all
// banks.
#include "block_scale.cuh"
#include "internal.h"
#include "rowwise.cuh"

namespace mmdit {
namespace {

constexpr int kTile = 128;

struct BlockCastArgs {
  const void* x;
  uint8_t* q;    // [R, ldq], or null
  float* s;
  uint8_t* qt;   // [C, ldt], or null
  float* st;
  float* part;   // [ceil(R/128), C], or null
  uint32_t* status;  // cleared when not null (the first kernel of a call that has a status word)
  int rows, cols;
  int64_t ldq, ldt;
};

template <typename T, bool SQUARE>
__global__ void __launch_bounds__(256) block_cast_kernel(const BlockCastArgs a) {
  __shared__ float col_max[16][kTile];
  __shared__ uint2 turned[kTile * 16];
  __shared__ float red[8];
  pdl_wait();
  pdl_trigger();
  if (a.status && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  const int tiles_c = (a.cols + kTile - 1) / kTile;
  const int tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int g = threadIdx.x >> 4, c8 = threadIdx.x & 15;
  const int r0 = tr * kTile + 8 * g, col = tc * kTile + 8 * c8;
  const bool col_ok = col < a.cols;  // columns come in whole groups of 8
  float v[8][8];
  Raw8<T> raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col_ok && r0 + i < a.rows) raw[i].load(static_cast<const T*>(a.x) + static_cast<int64_t>(r0 + i) * a.cols + col);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (col_ok && r0 + i < a.rows) {
      raw[i].to_f32(v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    }
  }
  float rm[8], cm[8], cs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    rm[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) rm[i] = fmaxf(rm[i], fabsf(v[i][e]));
  }
  float square_scale = 1.f;
  if constexpr (SQUARE) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, rm[i]);
    m = warp_max(m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, red[i]);
    square_scale = block_scale(m);
    if (threadIdx.x == 0) a.s[static_cast<int64_t>(tr) * tiles_c + tc] = square_scale;
  }
  if (a.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s = square_scale;
      if constexpr (!SQUARE) {
        float m = rm[i];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        s = block_scale(m);
      }
      if (r0 + i < a.rows) {
        if (col_ok) *reinterpret_cast<uint2*>(a.q + static_cast<int64_t>(r0 + i) * a.ldq + col) = e4m3x8(v[i], s);
        if (!SQUARE && c8 == 0) a.s[static_cast<int64_t>(tc) * a.rows + r0 + i] = s;
      }
    }
  }
  if (!a.qt && !a.part) return;
  if (a.part) {  // column sums: 8 rows in registers, then the 16 row groups in order
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cs[e] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[e] += v[i][e];
      col_max[g][8 * c8 + e] = cs[e];
    }
    __syncthreads();
    if (threadIdx.x < kTile && tc * kTile + static_cast<int>(threadIdx.x) < a.cols) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) t += col_max[k][threadIdx.x];
      a.part[static_cast<int64_t>(tr) * a.cols + tc * kTile + threadIdx.x] = t;
    }
    __syncthreads();
  }
  if (!a.qt) return;
  float scale[8];
  if constexpr (SQUARE) {
#pragma unroll
    for (int e = 0; e < 8; ++e) scale[e] = square_scale;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cm[e] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) cm[e] = fmaxf(cm[e], fabsf(v[i][e]));
      col_max[g][8 * c8 + e] = cm[e];
    }
    __syncthreads();
    if (threadIdx.x < kTile) {
      float m = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) m = fmaxf(m, col_max[k][threadIdx.x]);
      const float s = block_scale(m);
      if (tc * kTile + static_cast<int>(threadIdx.x) < a.cols)
        a.st[static_cast<int64_t>(tr) * a.cols + tc * kTile + threadIdx.x] = s;
      col_max[0][threadIdx.x] = s;  // row 0 of this column: read above by this thread alone
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) scale[e] = col_max[0][8 * c8 + e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[i][e];
    turned[(8 * c8 + e) * 16 + (g ^ c8)] = e4m3x8(w, scale[e]);
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int piece = threadIdx.x + p * 256, k = piece >> 3, u = piece & 7;
    const int row = tr * kTile + 16 * u;
    if (tc * kTile + k < a.cols && row < a.ldt) {
      const uint2 lo = turned[k * 16 + ((2 * u) ^ (k >> 3))], hi = turned[k * 16 + ((2 * u + 1) ^ (k >> 3))];
      *reinterpret_cast<uint4*>(a.qt + static_cast<int64_t>(tc * kTile + k) * a.ldt + row) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
}

}  // namespace

cudaError_t launch_block_cast(int act, int square, int rows, int cols, const void* x, uint8_t* q, int64_t ldq, float* s,
                              uint8_t* qt, int64_t ldt, float* st, float* part, uint32_t* status, cudaStream_t stream) {
  if (rows <= 0 || cols <= 0) return cudaSuccess;
  const int64_t tiles = static_cast<int64_t>((rows + kTile - 1) / kTile) * ((cols + kTile - 1) / kTile);
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  const BlockCastArgs a{x, q, s, qt, st, part, status, rows, cols, ldq, ldt};
  auto kern = act == 1 ? (square ? block_cast_kernel<__nv_bfloat16, true> : block_cast_kernel<__nv_bfloat16, false>)
                       : (square ? block_cast_kernel<float, true> : block_cast_kernel<float, false>);
  const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>(tiles)), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace mmdit
