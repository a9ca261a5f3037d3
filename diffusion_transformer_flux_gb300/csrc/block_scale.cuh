// block_scale.cuh -- the scale of an E4M3 tile, shared by the kernels that cast.
#pragma once

#include "common.cuh"

namespace mmdit {

// The scale of a tile whose largest magnitude is `amax`: 448 times the float32 reciprocal of amax (two
// IEEE roundings, so any float32 program reproduces the codes), which puts the largest element on E4M3's
// largest value; 1 for a tile of zeros; at most 2^100, so that a tile below 448 2^-100 keeps fewer bits
// instead of overflowing its scale (an infinite scale would turn the tile's zeros into NaN).
__device__ __forceinline__ float block_scale(float amax) {
  return amax > 0.f ? fminf(__fmul_rn(__frcp_rn(amax), 448.f), 1.2676506002282294e30f) : 1.f;
}

}  // namespace mmdit
