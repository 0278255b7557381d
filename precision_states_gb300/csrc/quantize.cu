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

// Magnitudes of a chunk as they lie in its words (two BF16, or one fp32, each),
// compared as integers; infinity and NaN are above every finite value.
template <typename T>
struct Magnitudes {
  static constexpr int kWords = Raw<T>::kWords;
  uint32_t w[kWords];
};
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b, Bf16) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b, float) { return max(a, b); }
__device__ __forceinline__ uint32_t word_magnitude(uint32_t w, Bf16) { return w & 0x7FFF7FFFu; }
__device__ __forceinline__ uint32_t word_magnitude(uint32_t w, float) { return w & 0x7FFFFFFFu; }
// The same with the elements that are not finite as 0.
__device__ __forceinline__ uint32_t finite_magnitude(uint32_t w, Bf16) {
  const uint32_t lo = w & 0x7FFFu, hi = w & 0x7FFF0000u;
  return (lo < 0x7F80u ? lo : 0u) | (hi < kInfBits ? hi : 0u);
}
__device__ __forceinline__ uint32_t finite_magnitude(uint32_t w, float) {
  return (w & 0x7FFFFFFFu) < kInfBits ? w & 0x7FFFFFFFu : 0u;
}
// Of a chunk; as fp32 bits.
template <typename T>
__device__ __forceinline__ Magnitudes<T> magnitudes(const Raw<T>& r, bool finite) {
  Magnitudes<T> m;
#pragma unroll
  for (int k = 0; k < Raw<T>::kWords; ++k) m.w[k] = finite ? finite_magnitude(r.w[k], T()) : word_magnitude(r.w[k], T());
  return m;
}
__device__ __forceinline__ uint32_t top_of(const Magnitudes<Bf16>& m) {
  const uint32_t t = larger(larger(m.w[0], m.w[1], Bf16()), larger(m.w[2], m.w[3], Bf16()), Bf16());
  return max(t << 16, t & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t top_of(const Magnitudes<float>& m) {
  return max(max(max(m.w[0], m.w[1]), max(m.w[2], m.w[3])), max(max(m.w[4], m.w[5]), max(m.w[6], m.w[7])));
}
__device__ __forceinline__ void expand(const Magnitudes<Bf16>& m, uint32_t (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = m.w[k] << 16;
    x[2 * k + 1] = m.w[k] & 0xFFFF0000u;
  }
}
__device__ __forceinline__ void expand(const Magnitudes<float>& m, uint32_t (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = m.w[k];
}

// A square's magnitudes by column (its eight rows' largest) -> those of the
// tile's whole columns, by way of shared memory.
template <typename T>
__device__ __forceinline__ void column_tops(const Raw<T> (&raw)[8], bool finite, uint32_t (*part)[128], uint32_t* whole,
                                            uint32_t (&top)[8]) {
  constexpr int W = Magnitudes<T>::kWords;
  const int square = threadIdx.x & 15, band = threadIdx.x >> 4;
  Magnitudes<T> m = magnitudes(raw[0], finite);
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    const Magnitudes<T> n = magnitudes(raw[i], finite);
#pragma unroll
    for (int k = 0; k < W; ++k) m.w[k] = larger(m.w[k], n.w[k], T());
  }
#pragma unroll
  for (int k = 0; k < W; ++k) m.w[k] = larger(m.w[k], __shfl_xor_sync(0xFFFFFFFFu, m.w[k], 16), T());   // the warp's two bands
  if ((band & 1) == 0) {
#pragma unroll
    for (int k = 0; k < W; k += 4)
      *reinterpret_cast<uint4*>(&part[band >> 1][W * square + k]) = make_uint4(m.w[k], m.w[k + 1], m.w[k + 2], m.w[k + 3]);
  }
  __syncthreads();
  if (threadIdx.x < 16 * W) {
    uint32_t t = part[0][threadIdx.x];
#pragma unroll
    for (int b = 1; b < 8; ++b) t = larger(t, part[b][threadIdx.x], T());
    whole[threadIdx.x] = t;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < W; k += 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(whole + W * square + k);
    m.w[k] = v.x; m.w[k + 1] = v.y; m.w[k + 2] = v.z; m.w[k + 3] = v.w;
  }
  expand(m, top);
}

// Scale bytes of eight lines (rows or columns) that every lane of a square group
// holds: lane i of the first eight stores that of line i.
__device__ __forceinline__ void store_bytes(uint8_t* scales, const uint32_t (&byte)[8], int i, int64_t line0, int lines,
                                            int64_t block, int64_t panel) {
  if (i >= 8 || i >= lines) return;
  uint32_t v = byte[0];
#pragma unroll
  for (int k = 1; k < 8; ++k) v = i == k ? byte[k] : v;
  scales[scale_place(line0 + i, block, panel)] = (uint8_t)v;
}

template <typename T, bool VEC, bool WHOLE>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? VEC ? 4 : 3 : 2)
quantize_kernel(const __grid_constant__ opt_quantize_args a, int64_t col_tiles) {
  // warps' maxima of columns; then the transposed codes, 16 pieces of 8 bytes per
  // column, pieces turned by column
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
    uint32_t byte[8];
    column_tops(raw, false, sh.top, tops_t, byte);
    odd = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) odd = odd || byte[j] >= kInfBits;
    odd = __syncthreads_or(odd);
    if (odd) column_tops(raw, true, sh.top, tops_t, byte);       // rare
    float inv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      byte[j] = scale_byte(byte[j]);
      inv[j] = inverse_scale(byte[j]);
    }
    // each band stores one of a square's eight columns
    store_bytes(scales, byte, band, c0 + c, cols - c, r0 >> 7, panel);
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
    if (odd) __syncthreads();          // the second maxima are read before their place is written
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
