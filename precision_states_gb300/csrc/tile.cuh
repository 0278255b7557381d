// tile.cuh -- device-side building blocks of the operators that work on a 128 x 128
// tile, which holds whole blocks of either orientation: 256 threads, each with an
// 8 x 8 square (thread t: columns 8 (t mod 16), rows 8 (t / 16)).
#pragma once

#include "layer.cuh"

namespace psopt {

constexpr int kTileThreads = 256;

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

// Shared memory of a tile on its way to the other orientation: warps' maxima of
// columns; then the transposed codes, 16 pieces of 8 bytes per column, pieces turned
// by column.
struct __align__(16) TileTurn {
  union {
    uint32_t top[8][128];
    uint2 codes[128][16];
  };
  uint32_t tops_t[128];
};

// The tile at (r0, c0), of which every thread holds its square, in blocks of 128 x 1:
// scale bytes to `scales` (those of the transposed operand, ceil(rows / 512) tiles
// wide), codes to sh.codes.  A barrier later they can be stored.
template <typename T>
__device__ __forceinline__ void turn_square(const Raw<T> (&raw)[8], TileTurn& sh, int64_t r0, int64_t c0, int cols,
                                            uint8_t* scales, int64_t panel) {
  const int square = threadIdx.x & 15, band = threadIdx.x >> 4, c = 8 * square;
  uint32_t byte[8];
  column_tops(raw, false, sh.top, sh.tops_t, byte);
  bool odd = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) odd = odd || byte[j] >= kInfBits;
  odd = __syncthreads_or(odd);
  if (odd) column_tops(raw, true, sh.top, sh.tops_t, byte);       // rare
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
}
// 16 lanes write a column's 128 codes.
__device__ __forceinline__ void store_turned(const TileTurn& sh, uint8_t* codes_t, int64_t pitch, int64_t r0, int64_t c0,
                                             int rows, int cols) {
  const int square = threadIdx.x & 15, band = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int col = 16 * i + band;
    if (col < cols && 8 * square < rows)
      store_codes8(codes_t + (c0 + col) * pitch + r0 + 8 * square, rows - 8 * square, sh.codes[col][square ^ (col >> 3)]);
  }
}

// The largest magnitudes of two 1 x 128 blocks that 16 lanes hold chunks of, by whole warps:
// BF16's go through the exchanges together.
__device__ __forceinline__ void tops16(uint32_t& a, uint32_t& b, Bf16) {
  uint32_t both = a | b >> 16;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) both = larger(both, __shfl_xor_sync(0xFFFFFFFFu, both, o), Bf16());
  a = both & 0xFFFF0000u;
  b = both << 16;
}
__device__ __forceinline__ void tops16(uint32_t& a, uint32_t& b, float) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
    b = max(b, __shfl_xor_sync(0xFFFFFFFFu, b, o));
  }
}

// 16 codes, the first `left` of which exist.
__device__ __forceinline__ void store_codes16(uint8_t* p, const uint32_t (&word)[4], int left) {
  if (left >= 16) {
    st_cs_u4(p, make_uint4(word[0], word[1], word[2], word[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 15; ++i)
      if (i < left) p[i] = (uint8_t)(word[i >> 2] >> (8 * (i & 3)));
  }
}

}  // namespace psopt
