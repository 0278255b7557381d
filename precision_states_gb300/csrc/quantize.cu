// quantize.cu -- a matrix to E4M3 codes with a scale for each block of 128, as
// it is and/or transposed (opt_layer.h).
//
// One CTA per 128 x 128 tile, which holds whole blocks of either orientation, so
// x is read once: 256 threads, each with an 8 x 8 square in registers (all of its
// loads in flight together).  A row's block is 16 lanes; a column's block is the
// 16 squares below one another, whose maxima meet in shared memory.  The
// transposed codes are turned within a square by byte permutes and go through
// shared memory once more, as codes, so that they leave in whole 128-byte lines.
#include "layer.cuh"

namespace psopt {
namespace {

constexpr int kThreads = 256;

// 4 x 4 bytes, rows to columns.
__device__ __forceinline__ void turn4(uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  const uint32_t ab0 = __byte_perm(a, b, 0x5140), ab1 = __byte_perm(a, b, 0x7362);
  const uint32_t cd0 = __byte_perm(c, d, 0x5140), cd1 = __byte_perm(c, d, 0x7362);
  a = __byte_perm(ab0, cd0, 0x5410);
  b = __byte_perm(ab0, cd0, 0x7632);
  c = __byte_perm(ab1, cd1, 0x5410);
  d = __byte_perm(ab1, cd1, 0x7632);
}

// A square's codes (rows l .. l + 7 of columns c .. c + 7) into the columns' lines.
__device__ __forceinline__ void put_turned(uint2 (&w)[8], uint2 (*lines)[16], int c, int band) {
  turn4(w[0].x, w[1].x, w[2].x, w[3].x);
  turn4(w[4].x, w[5].x, w[6].x, w[7].x);
  turn4(w[0].y, w[1].y, w[2].y, w[3].y);
  turn4(w[4].y, w[5].y, w[6].y, w[7].y);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    lines[c + j][band ^ (c >> 3)] = make_uint2(w[j].x, w[4 + j].x);
    lines[c + 4 + j][band ^ (c >> 3)] = make_uint2(w[j].y, w[4 + j].y);
  }
}

// m: this square's maxima of its eight columns -> those of the whole columns.
__device__ __forceinline__ void column_tops(uint32_t (&m)[8], uint32_t (*part)[128], uint32_t* whole, int band, int c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) m[j] = max(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], 16));   // the warp's two bands
  if ((band & 1) == 0) {
    *reinterpret_cast<uint4*>(&part[band >> 1][c]) = make_uint4(m[0], m[1], m[2], m[3]);
    *reinterpret_cast<uint4*>(&part[band >> 1][c + 4]) = make_uint4(m[4], m[5], m[6], m[7]);
  }
  __syncthreads();
  if (threadIdx.x < 128) {
    uint32_t t = 0;
#pragma unroll
    for (int b = 0; b < 8; ++b) t = max(t, part[b][threadIdx.x]);
    whole[threadIdx.x] = t;
  }
  __syncthreads();
  const uint4 lo = *reinterpret_cast<const uint4*>(whole + c), hi = *reinterpret_cast<const uint4*>(whole + c + 4);
  m[0] = lo.x; m[1] = lo.y; m[2] = lo.z; m[3] = lo.w;
  m[4] = hi.x; m[5] = hi.y; m[6] = hi.z; m[7] = hi.w;
}

template <typename T, bool VEC, bool WHOLE>
__global__ void __launch_bounds__(kThreads, 2) quantize_kernel(const __grid_constant__ opt_quantize_args a,
                                                               int64_t col_tiles) {
  // warps' maxima of columns; then the transposed codes, 16 pieces of 8 bytes per column, pieces turned by column
  __shared__ __align__(16) union {
    uint32_t top[8][128];
    uint2 codes[128][16];
  } sh;
  __shared__ __align__(16) uint32_t tops_t[128];
  __shared__ uint32_t tops[2][kThreads / 32];
  const int64_t r0 = 128 * (blockIdx.x / col_tiles), c0 = 128 * (blockIdx.x % col_tiles);
  const int rows = (int)min(a.rows - r0, (int64_t)128), cols = (int)min(a.cols - c0, (int64_t)128);
  const int square = threadIdx.x & 15, band = threadIdx.x >> 4, c = 8 * square, l = 8 * band;

  Raw<T> raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    raw[i] = Raw<T>{};
    if (l + i < rows && c < cols)
      raw[i] = load_raw<VEC>(static_cast<const T*>(a.d_x) + (r0 + l + i) * a.x_pitch + c0 + c, min(cols - c, 8));
  }

  // the tile's one block
  uint32_t top = 0;
  bool odd = false;
  if (WHOLE) {
    uint32_t finite = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x[8];
      unpack(raw[i], x);
      top = max(top, top8(x));
    }
    if (top >= kInfBits) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x[8];
        unpack(raw[i], x);
        finite = max(finite, finite_top8(x));
      }
    } else {
      finite = top;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      finite = max(finite, __shfl_xor_sync(0xFFFFFFFFu, finite, o));
    }
    if ((threadIdx.x & 31) == 0) {
      tops[0][threadIdx.x >> 5] = top;
      tops[1][threadIdx.x >> 5] = finite;
    }
    __syncthreads();
    top = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      odd = odd || tops[0][w] >= kInfBits;
      top = max(top, tops[1][w]);
    }
  }

  // rows
  if (a.d_codes != nullptr || WHOLE) {
    const int64_t panel = (a.cols + 511) / 512;
    uint2 turned[8];
    uint32_t tops8[8];
    if (!WHOLE) {
      // the eight rows' maxima together, so that their exchanges overlap
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x[8];
        unpack(raw[i], x);
        tops8[i] = top8(x);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) tops8[i] = max(tops8[i], __shfl_xor_sync(0xFFFFFFFFu, tops8[i], o));
#pragma unroll
      for (int i = 0; i < 8; ++i) odd = odd || tops8[i] >= kInfBits;
      odd = __any_sync(0xFFFFFFFFu, odd);
      if (odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float x[8];
          unpack(raw[i], x);
          tops8[i] = top16(finite_top8(x));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x[8];
      unpack(raw[i], x);
      const uint32_t byte = scale_byte(WHOLE ? top : tops8[i]);
      const uint2 w = codes8(x, inverse_scale(byte), odd);
      if (a.d_codes != nullptr && l + i < rows) {
        if (c < cols)
          store_codes8(static_cast<uint8_t*>(a.d_codes) + (r0 + l + i) * a.codes_pitch + c0 + c, cols - c, w);
        if (square == 0)
          static_cast<uint8_t*>(a.d_scales)[scale_place(r0 + l + i, c0 >> 7, panel)] = (uint8_t)byte;
      }
      turned[i] = w;
    }
    if (a.d_codes_t == nullptr) return;
    if (WHOLE) {
      put_turned(turned, sh.codes, c, band);
    }
  }

  // columns
  const int64_t panel = (a.rows + 511) / 512;
  uint8_t* scales = static_cast<uint8_t*>(a.d_scales_t);
  if (!WHOLE) {
    uint32_t m[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x[8];
      unpack(raw[i], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j] = max(m[j], magnitude(x[j]));
    }
    column_tops(m, sh.top, tops_t, band, c);
    odd = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) odd = odd || m[j] >= kInfBits;
    if (__syncthreads_or(odd)) {       // rare: the columns' finite maxima
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x[8];
        unpack(raw[i], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = finite_bits(x[j]) ? max(m[j], magnitude(x[j])) : m[j];
      }
      column_tops(m, sh.top, tops_t, band, c);
      odd = true;
    }
    uint32_t byte[8];
    float inv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      byte[j] = scale_byte(m[j]);
      inv[j] = inverse_scale(byte[j]);
    }
    if (band == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < cols) scales[scale_place(c0 + c + j, r0 >> 7, panel)] = (uint8_t)byte[j];
    }
    uint2 turned[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x[8];
      unpack(raw[i], x);
      if (odd) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = finite_bits(x[j]) ? x[j] : u2f(0x7FC00000u);
      }
      times8(x, inv);
      turned[i] = codes8(x);
    }
    put_turned(turned, sh.codes, c, band);
  } else if (threadIdx.x < cols) {
    scales[scale_place(c0 + threadIdx.x, r0 >> 7, panel)] = (uint8_t)scale_byte(top);
  }
  __syncthreads();
  // 16 lanes write a column's 128 codes
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int col = 16 * i + band;
    if (col < cols && 8 * square < rows)
      store_codes8(static_cast<uint8_t*>(a.d_codes_t) + (c0 + col) * a.codes_t_pitch + r0 + 8 * square, rows - 8 * square,
                   sh.codes[col][square ^ (col >> 3)]);
  }
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
