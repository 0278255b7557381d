// dequantize.cu -- what a kept matrix becomes in the backward pass: its values, and
// its transposed operand (opt_layer.h).
//
// Mathematics: a value is its code times 2^e, exact in fp32; the transposed operand's
// scales and codes are the quantizer's for those values, in blocks along the rows.
#include "tile.cuh"

namespace psopt {
namespace {

constexpr int kThreads = 256;

// Plain values alone: a chunk to a thread.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const __grid_constant__ opt_dequantize_args a) {
  __shared__ __align__(16) Ragged<T, VEC, kThreads / 32> ragged;
  T* buffer = ragged.chunk[VEC ? 0 : (int)(threadIdx.y * blockDim.x + threadIdx.x) >> 5];
  const int64_t c = 8 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x);
  const int valid = (int)max(min(a.cols - c, (int64_t)8), (int64_t)0);
  for (int64_t r = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; r < a.rows; r += (int64_t)gridDim.y * blockDim.y) {
    const Source<E4m3, VEC> kept(a.d_codes, a.d_scales, a.codes_pitch, a.rows, a.cols, r);
    float x[8];
    kept.values(kept.ahead(c, valid), c, valid, x);
    if (!VEC || valid > 0) store_at<VEC>(a.d_x, a.x_pitch, a.cols, r, c, valid, x, buffer);
  }
}

// A 128 x 128 tile to a CTA, each thread with an 8 x 8 square.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kTileThreads, 2) dequantize_tile_kernel(const __grid_constant__ opt_dequantize_args a,
                                                                         int64_t col_tiles) {
  __shared__ TileTurn sh;
  const int64_t r0 = 128 * (blockIdx.x / col_tiles), c0 = 128 * (blockIdx.x % col_tiles);
  const int rows = (int)min(a.rows - r0, (int64_t)128), cols = (int)min(a.cols - c0, (int64_t)128);
  const int square = threadIdx.x & 15, band = threadIdx.x >> 4, l = 8 * band;
  const int64_t c = c0 + 8 * square;
  Raw<float> raw[8];
  {
    KeptAsk ask[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int valid = l + i < rows ? max(min(cols - 8 * square, 8), 0) : 0;
      ask[i] = Source<E4m3, VEC>(a.d_codes, a.d_scales, a.codes_pitch, a.rows, a.cols, r0 + l + i).ahead(c, valid);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int valid = l + i < rows ? max(min(cols - 8 * square, 8), 0) : 0;
      float x[8];
      values8(ask[i].codes, scale_of(ask[i].byte), x);
#pragma unroll
      for (int j = 0; j < 8; ++j) raw[i].w[j] = j < valid ? f2u(x[j]) : 0u;
      if (a.d_x != nullptr && valid > 0)
        store8<VEC>(static_cast<T*>(a.d_x) + (r0 + l + i) * a.x_pitch + c, valid, x);
    }
  }
  turn_square(raw, sh, r0, c0, cols, static_cast<uint8_t*>(a.d_scales_t), (a.rows + 511) / 512);
  __syncthreads();
  store_turned(sh, static_cast<uint8_t*>(a.d_codes_t), a.codes_t_pitch, r0, c0, rows, cols);
}

template <typename T, bool VEC>
cudaError_t launch(const opt_dequantize_args& a, cudaStream_t s) {
  if (a.d_codes_t == nullptr) {
    const ChunkGrid g(a.rows, a.cols, kThreads);
    dequantize_kernel<T, VEC><<<g.grid, g.block, 0, s>>>(a);
  } else {
    const int64_t col_tiles = (a.cols + 127) / 128;
    dequantize_tile_kernel<T, VEC><<<(unsigned)((a.rows + 127) / 128 * col_tiles), kTileThreads, 0, s>>>(a, col_tiles);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dequantize(const opt_dequantize_args& a, cudaStream_t s) {
  const int64_t es = a.dtype == OPT_F32 ? 4 : 2;
  const bool vec = a.cols % 8 == 0 && (a.d_x == nullptr || (((uintptr_t)a.d_x & 15u) == 0 &&
                                                            (a.rows == 1 || a.x_pitch * es % 16 == 0)));
  if (a.dtype == OPT_F32) return vec ? launch<float, true>(a, s) : launch<float, false>(a, s);
  return vec ? launch<Bf16, true>(a, s) : launch<Bf16, false>(a, s);
}

}  // namespace psopt
