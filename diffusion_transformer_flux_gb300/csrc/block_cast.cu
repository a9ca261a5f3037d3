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
// (g, c) of 32 x 16 holds rows 4 g .. 4 g + 3 of the 8 columns 8 c .. 8 c + 7, so that a row tile's amax
// is a shuffle over 16 lanes, a column's is 4 register maxima and one pass through shared memory, and
// the transposed codes of a column are 4 neighbouring bytes.  They are turned through shared memory in
// 4-byte pieces, piece g of column k at place g ^ 2 (k / 8), which spreads a warp's stores over all banks.
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

// A thread keeps its 32 elements as they were loaded (16 registers for bf16) and turns them into floats where it
// needs them, so that three CTAs share an SM: 4095 x 4096 bf16 both ways in 16.9 us, 4.0 TB/s, one way in 10.8 or 11.7, in
// 128 x 128 tiles both ways 14.7 (256 threads with 64 elements each: 17.5 us, as floats 23.3).  40 registers are what
// three CTAs leave; 20 to 24 bytes are spilled for them.
constexpr int kCastThreads = 512, kRows = 4, kGroups = kTile / kRows;
template <typename T, bool SQUARE>
__global__ void __launch_bounds__(kCastThreads, sizeof(T) == 2 ? 3 : 2) block_cast_kernel(const BlockCastArgs a) {
  __shared__ float col_red[kGroups][kTile];
  __shared__ uint32_t turned[kTile * kGroups];
  __shared__ float red[kCastThreads / 32];
  pdl_wait();
  pdl_trigger();
  if (a.status && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  const int tiles_c = (a.cols + kTile - 1) / kTile;
  const int tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
  const int g = threadIdx.x >> 4, c8 = threadIdx.x & 15;
  const int r0 = tr * kTile + kRows * g, col = tc * kTile + 8 * c8;
  const bool col_ok = col < a.cols;  // columns come in whole groups of 8
  Raw8<T> raw[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    raw[i] = Raw8<T>{};
    if (col_ok && r0 + i < a.rows) raw[i].load(static_cast<const T*>(a.x) + static_cast<int64_t>(r0 + i) * a.cols + col);
  }
  float square_scale = 1.f;
  if constexpr (SQUARE) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float v[8];
      raw[i].to_f32(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
    }
    m = warp_max(m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int i = 1; i < kCastThreads / 32; ++i) m = fmaxf(m, red[i]);
    square_scale = block_scale(m);
    if (threadIdx.x == 0) a.s[static_cast<int64_t>(tr) * tiles_c + tc] = square_scale;
  }
  if (a.q) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float v[8], s = square_scale;
      raw[i].to_f32(v);
      if constexpr (!SQUARE) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        s = block_scale(m);
      }
      if (r0 + i < a.rows) {
        if (col_ok) *reinterpret_cast<uint2*>(a.q + static_cast<int64_t>(r0 + i) * a.ldq + col) = e4m3x8(v, s);
        if (!SQUARE && c8 == 0) a.s[static_cast<int64_t>(tc) * a.rows + r0 + i] = s;
      }
    }
  }
  if (a.part) {  // column sums: the thread's rows, then the row groups in order
    float cs[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float v[8];
      raw[i].to_f32(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) cs[e] += v[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) col_red[g][8 * c8 + e] = cs[e];
    __syncthreads();
    if (threadIdx.x < kTile && tc * kTile + static_cast<int>(threadIdx.x) < a.cols) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < kGroups; ++k) t += col_red[k][threadIdx.x];
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
    for (int e = 0; e < 8; ++e) scale[e] = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float v[8];
      raw[i].to_f32(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) scale[e] = fmaxf(scale[e], fabsf(v[e]));
    }
    // 16-byte stores, so that a warp's two row groups fill the banks
    float4* mine = reinterpret_cast<float4*>(&col_red[g][8 * c8]);
    mine[0] = make_float4(scale[0], scale[1], scale[2], scale[3]);
    mine[1] = make_float4(scale[4], scale[5], scale[6], scale[7]);
    __syncthreads();
    if (threadIdx.x < kTile) {
      float m = 0.f;
#pragma unroll
      for (int k = 0; k < kGroups; ++k) m = fmaxf(m, col_red[k][threadIdx.x]);
      const float s = block_scale(m);
      if (tc * kTile + static_cast<int>(threadIdx.x) < a.cols)
        a.st[static_cast<int64_t>(tr) * a.cols + tc * kTile + threadIdx.x] = s;
      col_red[0][threadIdx.x] = s;  // row 0 of this column: read above by this thread alone
    }
    __syncthreads();
    const float4* s4 = reinterpret_cast<const float4*>(&col_red[0][8 * c8]);
    const float4 lo = s4[0], hi = s4[1];
    scale[0] = lo.x, scale[1] = lo.y, scale[2] = lo.z, scale[3] = lo.w;
    scale[4] = hi.x, scale[5] = hi.y, scale[6] = hi.z, scale[7] = hi.w;
  }
  // the transposed codes of each column's rows
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float s = scale[e];
    turned[(8 * c8 + e) * kGroups + (g ^ (2 * c8))] =
        e4m3x2(raw[0].at(e) * s, raw[1].at(e) * s) | (e4m3x2(raw[2].at(e) * s, raw[3].at(e) * s) << 16);
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < kTile * 8 / kCastThreads; ++p) {
    const int piece = threadIdx.x + p * kCastThreads, k = piece >> 3, u = piece & 7, c = k >> 3;
    const int row = tr * kTile + 16 * u;
    if (tc * kTile + k < a.cols && row < a.ldt) {
      // places 4 u ^ 2 c .. of the column: the four pieces of rows 16 u .. 16 u + 15, halves swapped for odd c
      const uint4 w = *reinterpret_cast<const uint4*>(&turned[k * kGroups + ((4 * u) ^ ((2 * c) & ~3))]);
      *reinterpret_cast<uint4*>(a.qt + static_cast<int64_t>(tc * kTile + k) * a.ldt + row) =
          c & 1 ? make_uint4(w.z, w.w, w.x, w.y) : w;
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
  const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>(tiles)), dim3(kCastThreads), 0, stream, a);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

}  // namespace mmdit
