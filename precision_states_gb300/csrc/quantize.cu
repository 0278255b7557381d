// quantize.cu -- a matrix to E4M3 codes with a scale for each block of 128, as
// it is and/or transposed (opt_layer.h).
//
// One CTA per 128 x 128 tile, which holds whole blocks of either orientation:
// x is read once.  The tile lies in shared memory in fp32, its rows one element
// apart in banks so that rows and columns are both read without conflicts.
#include "layer.cuh"

namespace psopt {
namespace {

constexpr int kThreads = 256;
constexpr int kPitch = 129;
constexpr int kSmem = 128 * kPitch * 4;

// Eight values along a row (step 1) or a column (step kPitch) of the tile.
__device__ __forceinline__ void tile8(const float* p, int step, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = p[j * step];
}

// Codes and scales of one orientation: line l of the tile (a row, or a column
// of x) runs along `step`; 16 threads take a line's 128 elements.  `lines` and
// `len` are what exists; `whole` non-zero: the tile's one scale's magnitude.
template <bool WHOLE>
__device__ __forceinline__ void write_lines(const float* tile, int line_step, int step, int lines, int len,
                                            uint32_t whole_top, bool whole_odd, uint8_t* codes, int64_t pitch,
                                            uint8_t* scales, int64_t line0, int64_t block, int64_t panel) {
  const int c = 8 * (threadIdx.x & 15);
  for (int l = threadIdx.x >> 4; l < 128; l += kThreads / 16) {
    float x[8];
    tile8(tile + l * line_step + c * step, step, x);
    uint32_t top = whole_top;
    bool odd = whole_odd;
    if (!WHOLE) {
      top = max16(top8(x));
      odd = top >= kInfBits;
      if (__any_sync(0xFFFFFFFFu, odd)) {
        const uint32_t finite = max16(finite_top8(x));
        if (odd) top = finite;
      }
    }
    if (l < lines) {
      const uint32_t byte = scale_byte(top);
      const int valid = min(len - c, 8);
      if (valid > 0)
        store_codes8(codes + (line0 + l) * pitch + 128 * block + c, valid, codes8(x, inverse_scale(byte), odd));
      if (c == 0) scales[scale_place(line0 + l, block, panel)] = (uint8_t)byte;
    }
  }
}

template <typename T, bool VEC, bool WHOLE>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const __grid_constant__ opt_quantize_args a,
                                                            int64_t col_tiles) {
  extern __shared__ float tile[];
  __shared__ uint32_t tops[2][kThreads / 32];
  const int64_t r0 = 128 * (blockIdx.x / col_tiles), c0 = 128 * (blockIdx.x % col_tiles);
  const int rows = (int)min(a.rows - r0, (int64_t)128), cols = (int)min(a.cols - c0, (int64_t)128);
  const int c = 8 * (threadIdx.x & 15);
  uint32_t top = 0, finite = 0;
  for (int l = threadIdx.x >> 4; l < 128; l += kThreads / 16) {
    float x[8] = {};
    const int valid = min(cols - c, 8);
    if (l < rows && valid > 0) load8<VEC>(static_cast<const T*>(a.d_x) + (r0 + l) * a.x_pitch + c0 + c, valid, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) tile[l * kPitch + c + j] = x[j];
    if (WHOLE) {
      top = max(top, top8(x));
      finite = max(finite, finite_top8(x));
    }
  }
  bool odd = false;
  if (WHOLE) {
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    finite = __reduce_max_sync(0xFFFFFFFFu, finite);
    if ((threadIdx.x & 31) == 0) {
      tops[0][threadIdx.x >> 5] = top;
      tops[1][threadIdx.x >> 5] = finite;
    }
  }
  __syncthreads();
  if (WHOLE) {
    for (int w = 0; w < kThreads / 32; ++w) {
      odd = odd || tops[0][w] >= kInfBits;
      finite = max(finite, tops[1][w]);
    }
  }
  if (a.d_codes != nullptr)
    write_lines<WHOLE>(tile, kPitch, 1, rows, cols, finite, odd, static_cast<uint8_t*>(a.d_codes), a.codes_pitch,
                       static_cast<uint8_t*>(a.d_scales), r0, c0 >> 7, (a.cols + 511) / 512);
  if (a.d_codes_t != nullptr)
    write_lines<WHOLE>(tile, 1, kPitch, cols, rows, finite, odd, static_cast<uint8_t*>(a.d_codes_t), a.codes_t_pitch,
                       static_cast<uint8_t*>(a.d_scales_t), c0, r0 >> 7, (a.rows + 511) / 512);
}

template <typename T, bool VEC, bool WHOLE>
cudaError_t launch(const opt_quantize_args& a, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(quantize_kernel<T, VEC, WHOLE>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int64_t col_tiles = (a.cols + 127) / 128;
  quantize_kernel<T, VEC, WHOLE>
      <<<(unsigned)((a.rows + 127) / 128 * col_tiles), kThreads, kSmem, s>>>(a, col_tiles);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const opt_quantize_args& a, cudaStream_t s) {
  const bool vec = a.cols % 8 == 0 && ((uintptr_t)a.d_x & 15u) == 0 &&
                   (a.rows == 1 || a.x_pitch * (int64_t)sizeof(T) % 16 == 0);
  if (a.block_rows == 128) return vec ? launch<T, true, true>(a, s) : launch<T, false, true>(a, s);
  return vec ? launch<T, true, false>(a, s) : launch<T, false, false>(a, s);
}

}  // namespace

cudaError_t launch_quantize(const opt_quantize_args& a, cudaStream_t s) {
  return a.dtype == OPT_F32 ? launch_t<float>(a, s) : launch_t<Bf16>(a, s);
}

}  // namespace psopt
