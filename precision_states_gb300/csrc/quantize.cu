// quantize.cu -- a matrix to E4M3 codes with a scale for each block of 128, as
// it is and/or transposed (opt_layer.h).
//
// One CTA per 128 x 128 tile, which holds whole blocks of either orientation, so
// x is read once: 256 threads, each with an 8 x 8 square in registers (all of its
// loads in flight together).  A row's block is 16 lanes; a column's block is the
// 16 squares below one another, whose maxima meet in shared memory.  The
// transposed codes are turned within a square by byte permutes and go through
// shared memory once more, as codes, so that they leave in whole 128-byte lines.
// Maxima are taken on the words as they lie (two BF16 at a time).
//
// 14336 x 4096 fp32 in blocks of 128 x 128, both orientations: 58.4 us, 6.0 TB/s
// (0.91 of the measured copy; 111.9 with the tile in shared memory as fp32), BF16
// 37.3 us (0.95).  In blocks of 1 x 128 both orientations' scaling bounds it: 8192
// x 4096 BF16 28.5 us (0.71), one orientation 19.3 (0.78).  8191 x 1024 BF16 takes
// 10.9 us: less than one tile per CTA slot, so a tile's latency is the time.
#include "tile.cuh"

namespace psopt {
namespace {

constexpr int kThreads = kTileThreads;

template <typename T, bool VEC, bool WHOLE>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? VEC ? 4 : 3 : 2)
quantize_kernel(const __grid_constant__ opt_quantize_args a, int64_t col_tiles) {
  __shared__ TileTurn sh;
  __shared__ uint32_t tops[2][kThreads / 32];
  const int64_t r0 = 128 * (blockIdx.x / col_tiles), c0 = 128 * (blockIdx.x % col_tiles);
  const int rows = (int)min(a.rows - r0, (int64_t)128), cols = (int)min(a.cols - c0, (int64_t)128);
  const int square = threadIdx.x & 15, band = threadIdx.x >> 4, c = 8 * square, l = 8 * band;

  Raw<T> raw[8];
  {
    const T* x = static_cast<const T*>(a.d_x);
    const T* p = x + (r0 + l) * a.x_pitch + c0;
    const auto row = [&](int i) {
      return Row<T, VEC>(p + i * a.x_pitch, x, x + (a.rows - 1) * a.x_pitch + a.cols);
    };
    const auto valid = [&](int i) { return l + i < rows ? max(min(cols - c, 8), 0) : 0; };
    Ahead<T, VEC> ahead[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ahead[i] = {};
      if (!VEC || valid(i) > 0) ahead[i] = row(i).ahead(c, valid(i));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = row(i).chunk(ahead[i], c, valid(i));
  }

  // the tile's one block
  uint32_t top = 0;
  bool odd = false;
  if (WHOLE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, top_of(magnitudes(raw[i], false)));
    uint32_t finite = top;
    if (top >= kInfBits) {
      finite = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) finite = max(finite, top_of(magnitudes(raw[i], true)));
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    finite = __reduce_max_sync(0xFFFFFFFFu, finite);
    if ((threadIdx.x & 31) == 0) {
      tops[0][threadIdx.x >> 5] = top;
      tops[1][threadIdx.x >> 5] = finite;
    }
    __syncthreads();
    top = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      odd = odd || tops[0][w] >= kInfBits;
      top = max(top, tops[1][w]);
    }
  }

  // rows
  if (a.d_codes != nullptr || WHOLE) {
    uint2 turned[8];
    uint32_t byte[8];
    if (!WHOLE) {
      // the eight rows' maxima together, so that their exchanges overlap
#pragma unroll
      for (int i = 0; i < 8; ++i) byte[i] = top_of(magnitudes(raw[i], false));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) byte[i] = max(byte[i], __shfl_xor_sync(0xFFFFFFFFu, byte[i], o));
#pragma unroll
      for (int i = 0; i < 8; ++i) odd = odd || byte[i] >= kInfBits;
      odd = __any_sync(0xFFFFFFFFu, odd);
      if (odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i) byte[i] = top16(top_of(magnitudes(raw[i], true)));
      }
    }
    uint8_t* p = static_cast<uint8_t*>(a.d_codes) + (r0 + l) * a.codes_pitch + c0 + c;
#pragma unroll
    for (int i = 0; i < 8; ++i, p += a.codes_pitch) {
      float x[8];
      unpack(raw[i], x);
      byte[i] = scale_byte(WHOLE ? top : byte[i]);
      turned[i] = codes8(x, inverse_scale(byte[i]), odd);
      if (a.d_codes != nullptr && l + i < rows && c < cols) store_codes8(p, cols - c, turned[i]);
    }
    if (a.d_codes != nullptr)
      store_bytes(static_cast<uint8_t*>(a.d_scales), byte, square, r0 + l, rows - l, c0 >> 7, (a.cols + 511) / 512);
    if (a.d_codes_t == nullptr) return;
    if (WHOLE) put_turned(turned, sh.codes, c, band);
  }

  // columns
  const int64_t panel = (a.rows + 511) / 512;
  uint8_t* scales = static_cast<uint8_t*>(a.d_scales_t);
  if (!WHOLE) {
    turn_square(raw, sh, r0, c0, cols, scales, panel);
  } else if (threadIdx.x < cols) {
    scales[scale_place(c0 + threadIdx.x, r0 >> 7, panel)] = (uint8_t)scale_byte(top);
  }
  __syncthreads();
  store_turned(sh, static_cast<uint8_t*>(a.d_codes_t), a.codes_t_pitch, r0, c0, rows, cols);
}

template <typename T, bool VEC, bool WHOLE>
cudaError_t launch(const opt_quantize_args& a, cudaStream_t s) {
  const int64_t col_tiles = (a.cols + 127) / 128;
  quantize_kernel<T, VEC, WHOLE><<<(unsigned)((a.rows + 127) / 128 * col_tiles), kThreads, 0, s>>>(a, col_tiles);
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
