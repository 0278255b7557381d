// matmul.h -- what the forms of the block-scaled product share: the output's
// matrices and their elements.
#pragma once

#include "layer.cuh"

namespace psopt {

// The kernels compute tiles of x y^T; x is the call's a, or its b (`swap`), when
// out[y][x] takes the tile's (x, y).
struct OutputArgs {
  void* out;
  const void* addend;
  int64_t out_pitch, addend_pitch;
  int swap;
};

__device__ __forceinline__ void put(Bf16* p, float v) { p->bits = (uint16_t)bf16_pair(v, 0.0f); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// Element (x, y) of the tiles' product in a matrix of `pitch`.
__device__ __forceinline__ int64_t place(const OutputArgs& a, int64_t pitch, int x, int y) {
  return a.swap ? y * pitch + x : x * pitch + y;
}

// One operand of at most kFewRows rows (matmul_few.cu).
constexpr int64_t kFewRows = 8;
cudaError_t launch_matmul_few(const opt_matmul_args& a, const OutputArgs& out, cudaStream_t s);

}  // namespace psopt
