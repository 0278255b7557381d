// layer.cuh -- device-side building blocks shared by the training-layer
// operators: eight-element loads and stores of BF16 and fp32 rows, the dropout
// draws of eight consecutive elements, block scales and their place in the
// scale tiles.
//
// Every row-wise operator cuts a row into chunks of eight elements, one per
// thread: 16 bytes of BF16, 32 of fp32, 8 of codes, one Philox call, and a
// sixteenth of a 128-element block.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "layer.h"

namespace psopt {

struct Bf16 { uint16_t bits; };   // storage type of an OPT_BF16 element

// Eight elements as they lie in memory (16 or 32 bytes): what a thread holds of
// a row that it has loaded ahead.
template <typename T>
struct Raw {
  static constexpr int kWords = 2 * sizeof(T);
  uint32_t w[kWords];
};

// Eight elements at p.  VEC: all eight exist and p is 16-byte aligned;
// otherwise the first `valid` exist, and the others read as 0.
template <bool VEC, typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p, int valid) {
  Raw<T> r;
  if constexpr (VEC) {
#pragma unroll
    for (int k = 0; k < Raw<T>::kWords; k += 4)
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(r.w[k]), "=r"(r.w[k + 1]), "=r"(r.w[k + 2]), "=r"(r.w[k + 3])
                   : "l"(reinterpret_cast<const uint32_t*>(p) + k));
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.w[j] = j < valid ? f2u(p[j]) : 0u;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      r.w[k] = (2 * k < valid ? (uint32_t)p[2 * k].bits : 0u) |
               (2 * k + 1 < valid ? (uint32_t)p[2 * k + 1].bits << 16 : 0u);
  }
  return r;
}
__device__ __forceinline__ void unpack(const Raw<float>& r, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = u2f(r.w[j]);
}
__device__ __forceinline__ void unpack(const Raw<Bf16>& r, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = u2f(r.w[k] << 16);
    x[2 * k + 1] = u2f(r.w[k] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ float element(const Bf16* p) { return u2f((uint32_t)p->bits << 16); }
__device__ __forceinline__ float element(const float* p) { return *p; }
// An element's fp32 bits if it exists, else 0: a load under a predicate, so that the
// compiler neither branches around it nor waits for it before the next one (as it
// did for 16-bit elements: 82 x 431 x 212 with a BF16 addend took 14.1 us, 6.7 so).
__device__ __forceinline__ uint32_t bits_if(const Bf16* p, bool exists) {
  uint16_t b;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.s32 q, %2, 0;\n\tmov.b16 %0, 0;\n\t@q ld.global.u16 %0, [%1];\n\t}"
               : "=h"(b) : "l"(p), "r"((int)exists));
  return (uint32_t)b << 16;
}
__device__ __forceinline__ uint32_t bits_if(const float* p, bool exists) {
  uint32_t b;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.s32 q, %2, 0;\n\tmov.b32 %0, 0;\n\t@q ld.global.u32 %0, [%1];\n\t}"
               : "=r"(b) : "l"(p), "r"((int)exists));
  return b;
}

template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* p, int valid, float (&x)[8]) {
  unpack(load_raw<VEC>(p, valid), x);
}

// A chunk under way: the words that it lies in, which load_ahead only asks for and
// chunk_of makes the chunk of.  Apart, because a shift or a branch beside the load
// waits for it, and so for every chunk in turn: the norm of 4853 x 7001 BF16 rows took
// 107.7 us so (97.3 since) and 165.9 with both in one.
template <typename T, bool VEC>
struct Ahead {
  static constexpr int kWords = Raw<T>::kWords + (!VEC && sizeof(T) == 2 ? 1 : 0);
  uint32_t w[kWords];
};
// A row of a rows x cols matrix.  Not VEC, BF16: `words` are the ones it lies in,
// and a chunk's five exist where first <= c <= last (the words of a few chunks at the
// matrix's ends reach beyond it).  valid: of the chunk at column c, 0 to 8 (VEC:
// 8; what has no chunk does not call).
template <typename T, bool VEC>
struct Row {
  const T* start;
  const uint32_t* words;
  int64_t last;
  int first, half;
  // at s, of a matrix from m to `end`
  __device__ __forceinline__ Row(const T* s, const T* m, const T* end) : start(s) {
    if constexpr (!VEC && sizeof(T) == 2) {
      words = reinterpret_cast<const uint32_t*>((uintptr_t)start & ~(uintptr_t)3);
      half = (int)((uintptr_t)start >> 1) & 1;
      first = start == m ? half : 0;
      last = end - reinterpret_cast<const T*>(words) - 10;
    }
  }
  __device__ __forceinline__ Row(const void* base, int64_t pitch, int64_t rows, int64_t cols, int64_t r)
      : start(static_cast<const T*>(base) + r * pitch) {
    if constexpr (!VEC && sizeof(T) == 2) {
      words = reinterpret_cast<const uint32_t*>((uintptr_t)start & ~(uintptr_t)3);
      half = (int)((uintptr_t)start >> 1) & 1;
      first = r == 0 ? half : 0;
      // a row with another behind it lies whole, with nine elements more (a shorter way to
      // `last` than from the matrix's end: those gradients 125 us so, 119 this way)
      last = r + 1 < rows && pitch >= 16 ? (int64_t)1 << 40 : (rows - 1 - r) * pitch + cols + half - 10;
    }
  }
  __device__ __forceinline__ bool whole(int64_t c) const { return c <= last && c >= first; }
  __device__ __forceinline__ Ahead<T, VEC> ahead(int64_t c, int valid) const {
    Ahead<T, VEC> r;
    if constexpr (VEC) {
      const Raw<T> v = load_raw<true>(start + c, 8);
#pragma unroll
      for (int k = 0; k < Raw<T>::kWords; ++k) r.w[k] = v.w[k];
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < 8; ++j) r.w[j] = bits_if(start + c + j, j < valid);
    } else {
      asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.s32 q, %6, 0;\n\t"
                   "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\tmov.b32 %4, 0;\n\t"
                   "@q ld.global.u32 %0, [%5];\n\t@q ld.global.u32 %1, [%5+4];\n\t@q ld.global.u32 %2, [%5+8];\n\t"
                   "@q ld.global.u32 %3, [%5+12];\n\t@q ld.global.u32 %4, [%5+16];\n\t}"
                   : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4])
                   : "l"(words + (c >> 1)), "r"((int)(valid > 0 && whole(c))));
    }
    return r;
  }
  // The chunk; elements from `valid` on read as 0.  One whose words reach beyond the
  // matrix is loaded here, element by element but together: the gradients of 129 x 1031
  // BF16 rows 4.7 us, 5.8 in a loop.  ONE_BY_ONE: in a loop, which costs the main path
  // fewer registers (strided dropout: see there).
  template <bool ONE_BY_ONE = false>
  __device__ __forceinline__ Raw<T> chunk(const Ahead<T, VEC>& a, int64_t c, int valid) const {
    Raw<T> r;
    if constexpr (VEC || sizeof(T) == 4) {
#pragma unroll
      for (int k = 0; k < Raw<T>::kWords; ++k) r.w[k] = a.w[k];
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) r.w[k] = __funnelshift_r(a.w[k], a.w[k + 1], 16 * half);
      if (valid < 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) r.w[k] = 2 * k + 1 < valid ? r.w[k] : 2 * k < valid ? r.w[k] & 0xFFFFu : 0u;
      }
      if (ONE_BY_ONE && valid > 0 && !whole(c)) {
        uint64_t part[2] = {0, 0};
#pragma unroll 1
        for (int j = 0; j < valid; ++j) {
          const uint64_t v = (uint64_t)start[c + j].bits << (16 * (j & 3));
          if (j < 4) part[0] |= v;
          else part[1] |= v;
        }
        r.w[0] = (uint32_t)part[0]; r.w[1] = (uint32_t)(part[0] >> 32);
        r.w[2] = (uint32_t)part[1]; r.w[3] = (uint32_t)(part[1] >> 32);
      } else if (valid > 0 && !whole(c)) {
        uint32_t b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = bits_if(start + c + j, j < valid);
#pragma unroll
        for (int k = 0; k < 4; ++k) r.w[k] = b[2 * k] >> 16 | b[2 * k + 1];
      }
    }
    return r;
  }
};

// Nearest BF16 of two values (a NaN as the converter's canonical one).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
template <bool VEC>
__device__ __forceinline__ void store8(Bf16* p, int valid, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = bf16_pair(x[2 * k], x[2 * k + 1]);
  if (VEC) {
    st_cs_u4(p, make_uint4(w[0], w[1], w[2], w[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) p[j].bits = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(float* p, int valid, const float (&x)[8]) {
  if (VEC) {
    st_cs_u4(p, make_uint4(f2u(x[0]), f2u(x[1]), f2u(x[2]), f2u(x[3])));
    st_cs_u4(p + 4, make_uint4(f2u(x[4]), f2u(x[5]), f2u(x[6]), f2u(x[7])));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) p[j] = x[j];
  }
}

// Storage of a warp's 32 consecutive chunks on their way to a row that starts at
// any place: lanes' chunks in, consecutive words out, so that a store covers 128
// bytes and not two in every sixteen.
template <typename T, bool VEC, int WARPS>
struct Ragged {
  T chunk[VEC ? 1 : WARPS][VEC ? 1 : 256];
  __device__ __forceinline__ T* of_warp() { return chunk[VEC ? 0 : threadIdx.x >> 5]; }
};
__device__ __forceinline__ void store_words(float* p, int n, const uint32_t* v, int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (32 * i + lane < n) reinterpret_cast<uint32_t*>(p)[32 * i + lane] = v[32 * i + lane];
}
// BF16 from p's first whole word on, `head` (0 or 1) elements behind p.
__device__ __forceinline__ void store_words(Bf16* p, int head, int n, const uint32_t* v, int lane) {
  uint32_t* out = reinterpret_cast<uint32_t*>(p + head);
  if (n == 256) {
#pragma unroll
    for (int i = 0; i < 3; ++i) out[32 * i + lane] = v[32 * i + lane];
    if (head == 0 || lane < 31) out[96 + lane] = v[96 + lane];
    else p[255].bits = (uint16_t)v[127];
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = head + 2 * (32 * i + lane);
    if (e + 1 < n) out[32 * i + lane] = v[32 * i + lane];
    else if (e < n) p[e].bits = (uint16_t)v[32 * i + lane];
  }
}
// Store of the chunk at column c (this lane's; its warp's lie side by side) of row
// r.  Not VEC: by whole warps, in which chunks beyond the row come with valid 0.
template <bool VEC, typename T>
__device__ __forceinline__ void store_at(void* base, int64_t pitch, int64_t cols, int64_t r, int64_t c, int valid,
                                         const float (&x)[8], T* buffer) {
  T* row = static_cast<T*>(base) + r * pitch;
  if constexpr (VEC) {
    store8<true>(row + c, 8, x);
  } else {
    const int lane = threadIdx.x & 31;
    const int64_t tile = c - 8 * lane;
    const int n = (int)max(min(cols - tile, (int64_t)256), (int64_t)0);
    uint32_t* words = reinterpret_cast<uint32_t*>(buffer);
    if constexpr (sizeof(T) == 4) {
      float4* b = reinterpret_cast<float4*>(buffer + 8 * lane);
      b[0] = make_float4(x[0], x[1], x[2], x[3]);
      b[1] = make_float4(x[4], x[5], x[6], x[7]);
      __syncwarp();
      store_words(row + tile, n, words, lane);
    } else {
      uint32_t w[5];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = bf16_pair(x[2 * k], x[2 * k + 1]);
      const int head = (int)((uintptr_t)(row + tile) >> 1) & 1;       // elements before the first whole word
      if (lane == 0 && head && n > 0) row[tile].bits = (uint16_t)w[0];
      w[4] = __shfl_down_sync(0xFFFFFFFFu, w[0], 1);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16 * head);      // pairs that lie in one word
      *reinterpret_cast<uint4*>(words + 4 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
      __syncwarp();
      store_words(row + tile, head, n, words, lane);
    }
    __syncwarp();
  }
}

// ----------------------------------------------------------------- dropout
// The draws of elements i .. i + 7 of the matrix's row-major order as 128
// bits, element i + j in bits 16 j: the generator's four words as they are when
// i is a multiple of 8 (VEC), else two calls' eight words moved down by i mod 8
// half-words.
// The generator's ten rounds with each product formed once, 64 bits wide.
__device__ __forceinline__ uint4 drop_group(uint64_t g, const DropArgs& d) {
  uint32_t x = (uint32_t)g, y = (uint32_t)(g >> 32) | 0x80000000u, z = d.tensor, w = d.step32;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)0xD2511F53u * x, p1 = (uint64_t)0xCD9E8D57u * z;
    x = (uint32_t)(p1 >> 32) ^ y ^ d.rk[2 * r];
    y = (uint32_t)p1;
    z = (uint32_t)(p0 >> 32) ^ w ^ d.rk[2 * r + 1];
    w = (uint32_t)p0;
  }
  return make_uint4(x, y, z, w);
}
__device__ __forceinline__ bool draws(const DropArgs& d) { return d.threshold != 0u && d.threshold < 65536u; }
// Not VEC: a chunk's second call is its neighbour's first, so a lane takes it from the
// next one, and lane 31 from `edge`, where one warp has put the calls that follow each
// warp's 32 chunks (see Edges): it took 16 of 141 us from the gradients of 8000 x 4001
// BF16 rows.  Without an edge each lane makes both.  By whole warps.
template <bool VEC>
__device__ __forceinline__ uint4 drop_draws(uint64_t i, const DropArgs& d, const uint4* edge) {
  const uint4 lo = drop_group(i >> 3, d);
  const int off = (int)(i & 7);
  if (VEC) return lo;
  uint4 hi;
  if (edge == nullptr) {
    if (off == 0) return lo;
    hi = drop_group((i >> 3) + 1, d);
  } else {
    hi.x = __shfl_down_sync(0xFFFFFFFFu, lo.x, 1);
    hi.y = __shfl_down_sync(0xFFFFFFFFu, lo.y, 1);
    hi.z = __shfl_down_sync(0xFFFFFFFFu, lo.z, 1);
    hi.w = __shfl_down_sync(0xFFFFFFFFu, lo.w, 1);
    if ((threadIdx.x & 31) == 31) hi = *edge;
  }
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (off & 4) {
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
  }
  if (off & 2) {
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
  }
  if (off & 1) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// sum <- sum + dropout(x) for the eight elements from i on.  Draws are compared
// in the upper half of a word (a draw is at least T iff it is there at least T
// shifted up): no half is taken apart, and a kept element costs one fused
// multiply-add.  T = 65536 keeps nothing.
template <bool VEC>
__device__ __forceinline__ void add_dropped8(float (&sum)[8], const float (&x)[8], uint64_t i, const DropArgs& d,
                                             const uint4* edge) {
  if (d.threshold == 0u) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += x[j];
  } else if (draws(d)) {
    const uint4 r = drop_draws<VEC>(i, d, edge);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w}, least = d.threshold << 16;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if ((w[k] << 16) >= least) sum[2 * k] = fmaf(x[2 * k], d.factor, sum[2 * k]);
      if (w[k] >= least) sum[2 * k + 1] = fmaf(x[2 * k + 1], d.factor, sum[2 * k + 1]);
    }
  }
}

// The generator calls behind each warp's 32 chunks, of a CTA that holds NG times its
// threads' chunks of a row, `i` being the number of its first element.  `put` fills the
// half that `turn` names, by the first threads; a barrier later the warps take theirs.
template <bool VEC, int N>
struct Edges {
  uint4 call[VEC ? 1 : 2][VEC ? 1 : N];
  __device__ __forceinline__ void put(int turn, uint64_t i, int ng, const DropArgs& d) {
    if constexpr (!VEC) {
      const int warps = (int)blockDim.x >> 5, t = (int)threadIdx.x;
      if (t < warps * ng && draws(d)) call[turn][t] = drop_group((i >> 3) + 32 * (t + 1), d);
    }
  }
  __device__ __forceinline__ const uint4* of_warp(int turn, int k) const {
    return VEC ? nullptr : &call[turn][k * ((int)blockDim.x >> 5) + ((int)threadIdx.x >> 5)];
  }
};

// ------------------------------------------------------------ block scales
// Scale byte of a block from the bits of its largest finite magnitude: with
// magnitude 1.f 2^E, E - 8 if 1.f <= 1.75 (448 = 1.75 2^8) else E - 7, never
// below -127 (which also serves blocks of zeros and of subnormals).  What is added
// carries into the exponent where the fraction is above 0.75.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top_bits) {
  return (uint32_t)max((int)((top_bits + 0x1FFFFFu) >> 23) - 8, 0);
}
// The same as a biased exponent in place, e + 135 (so byte + 8), from which the inverse scale
// and the byte are an instruction each.  An infinity gives 255, a NaN 255 or 256, and
// finite values above 1.75 2^127 255 too.
__device__ __forceinline__ uint32_t scale_field(uint32_t top_bits) {
  return max((top_bits + 0x1FFFFFu) & 0xFF800000u, 8u << 23);
}
constexpr uint32_t kOddField = 255u << 23;
__device__ __forceinline__ float inverse_of_field(uint32_t field) { return u2f((262u << 23) - field); }
__device__ __forceinline__ uint32_t byte_of_field(uint32_t field) { return (field >> 23) - 8u; }
// 2^-e for a scale byte; scale_byte never exceeds 247, so this is normal.
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return u2f((254u - byte) << 23); }

__device__ __forceinline__ bool finite_bits(float x) { return (f2u(x) & 0x7F800000u) != 0x7F800000u; }
// Magnitudes are compared as integers: their order, with infinity and NaN above
// every finite value.
constexpr uint32_t kInfBits = 0x7F800000u;
__device__ __forceinline__ uint32_t magnitude(float x) { return f2u(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t top8(const float (&x)[8]) {
  return max(max(max(magnitude(x[0]), magnitude(x[1])), max(magnitude(x[2]), magnitude(x[3]))),
             max(max(magnitude(x[4]), magnitude(x[5])), max(magnitude(x[6]), magnitude(x[7]))));
}
// The largest of three magnitudes in one instruction; a NaN stays one.
__device__ __forceinline__ float largest3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// top8 by those (bits of an infinity or NaN are at least kInfBits).
__device__ __forceinline__ uint32_t top8_of(const float (&x)[8]) {
  return f2u(largest3(largest3(x[0], x[1], x[2]), largest3(x[3], x[4], x[5]), largest3(x[6], x[7], x[7])));
}
// The same of the finite elements.
__device__ __forceinline__ uint32_t finite_top8(const float (&x)[8]) {
  uint32_t t = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) t = max(t, finite_bits(x[j]) ? magnitude(x[j]) : 0u);
  return t;
}
// Over the 16 lanes of a 128-element block.
__device__ __forceinline__ uint32_t top16(uint32_t t) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) t = max(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
  return t;
}
// The scale byte of the 1 x 128 block that 16 lanes hold eight elements each of,
// by the whole warp; `odd`: it holds an infinity or NaN.
__device__ __forceinline__ uint32_t block_byte(const float (&x)[8], bool& odd) {
  uint32_t top = top16(top8(x));
  odd = top >= kInfBits;
  if (__any_sync(0xFFFFFFFFu, odd)) {
    const uint32_t finite = top16(finite_top8(x));
    if (odd) top = finite;
  }
  return scale_byte(top);
}

// Two fp32 products per instruction.
__device__ __forceinline__ void scaled8(const float (&x)[8], float f, float (&y)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) unpk(mul2(pk(x[j], x[j + 1]), pk(f, f)), y[j], y[j + 1]);
}
__device__ __forceinline__ void times8(float (&x)[8], const float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) unpk(mul2(pk(x[j], x[j + 1]), pk(f[j], f[j + 1])), x[j], x[j + 1]);
}

__device__ __forceinline__ uint2 codes8(const float (&v)[8]) {
  return make_uint2(e4m3x2_rn(v[0], v[1]) | (e4m3x2_rn(v[2], v[3]) << 16),
                    e4m3x2_rn(v[4], v[5]) | (e4m3x2_rn(v[6], v[7]) << 16));
}
// Codes of eight elements over 2^e (inv = 2^-e); `odd` says that the block
// holds an infinity or NaN, which the converter would clamp or keep: both are
// stored as NaN.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv, bool odd) {
  float v[8];
  scaled8(x, inv, v);
  if (odd) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!finite_bits(x[j])) v[j] = u2f(0x7FC00000u);
  }
  return codes8(v);
}
// Store of up to eight codes at an 8-byte aligned place.
__device__ __forceinline__ void store_codes8(uint8_t* p, int valid, uint2 w) {
  if (valid >= 8) {
    st_cs_u2(p, w);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) p[j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
  }
}

// Accesses under a predicate, without a branch: eight elements of a 16-byte aligned place
// (0 if it is not on), eight of them or eight codes to such a place, and a byte.
template <typename T>
__device__ __forceinline__ Raw<T> load_if(const T* p, bool on) {
  Raw<T> r;
#pragma unroll
  for (int k = 0; k < Raw<T>::kWords; k += 4)
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.s32 q, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
                 "@q ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
                 : "=&r"(r.w[k]), "=&r"(r.w[k + 1]), "=&r"(r.w[k + 2]), "=&r"(r.w[k + 3])
                 : "l"(reinterpret_cast<const uint32_t*>(p) + k), "r"((int)on));
  return r;
}
__device__ __forceinline__ uint2 load_codes_if(const uint8_t* p, bool on) {
  uint2 r;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.s32 q, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
               "@q ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];\n\t}" : "=&r"(r.x), "=&r"(r.y) : "l"(p), "r"((int)on));
  return r;
}
__device__ __forceinline__ uint32_t load_byte_if(const uint8_t* p, bool on) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.s32 q, %2, 0;\n\tmov.b32 %0, 0;\n\t@q ld.global.u8 %0, [%1];\n\t}"
               : "=&r"(r) : "l"(p), "r"((int)on));
  return r;
}
__device__ __forceinline__ void store_if(void* p, uint4 v, bool on) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.s32 q, %5, 0;\n\t@q st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};\n\t}"
               :: "l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"((int)on) : "memory");
}
__device__ __forceinline__ void store_if(void* p, uint2 v, bool on) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.s32 q, %3, 0;\n\t@q st.global.cs.v2.u32 [%0], {%1,%2};\n\t}"
               :: "l"(p), "r"(v.x), "r"(v.y), "r"((int)on) : "memory");
}
__device__ __forceinline__ void store_byte_if(uint8_t* p, uint32_t v, bool on) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.s32 q, %2, 0;\n\t@q st.global.u8 [%0], %1;\n\t}" :: "l"(p), "r"(v), "r"((int)on) : "memory");
}
__device__ __forceinline__ void store8_if(Bf16* p, const float (&x)[8], bool on) {
  store_if(p, make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7])), on);
}
__device__ __forceinline__ void store8_if(float* p, const float (&x)[8], bool on) {
  store_if(p, make_uint4(f2u(x[0]), f2u(x[1]), f2u(x[2]), f2u(x[3])), on);
  store_if(p + 4, make_uint4(f2u(x[4]), f2u(x[5]), f2u(x[6]), f2u(x[7])), on);
}
// Codes of a chunk whose block's largest magnitude `top` is finite, and the block's scale
// byte where `first` says so.
__device__ __forceinline__ void put_finite_if(uint8_t* codes, uint8_t* scale, const float (&x)[8], uint32_t top, bool on, bool first) {
  const uint32_t byte = scale_byte(top);
  float v[8];
  scaled8(x, inverse_scale(byte), v);
  store_if(codes, codes8(v), on);
  store_byte_if(scale, byte, first);
}

// The same from the block's field.
__device__ __forceinline__ void put_field_if(uint8_t* codes, uint8_t* scale, const float (&x)[8], uint32_t field, bool on, bool first) {
  float v[8];
  scaled8(x, inverse_of_field(field), v);
  store_if(codes, codes8(v), on);
  store_byte_if(scale, byte_of_field(field), first);
}

// Place of the scale byte of row r, block b (opt_layer.h); panel = ceil(B / 4).
__host__ __device__ __forceinline__ int64_t scale_place(int64_t r, int64_t b, int64_t panel) {
  return 512 * ((r >> 7) * panel + (b >> 2)) + 16 * (r & 31) + 4 * ((r >> 5) & 3) + (b & 3);
}

// ------------------------------------------------------------ kept matrices
struct E4m3 {};                   // element type of a kept matrix, codes with scales

// The scale that a byte stands for: 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  // byte 0 is a subnormal, and 255 the only one whose successor has bit 8
  return u2f(max(byte << 23, 0x00400000u) | (((byte + 1u) << 14) & 0x00400000u));
}
// Eight codes of an 8-byte aligned place, the first `valid` of which exist; the others
// read as 0.
__device__ __forceinline__ uint2 load_codes8(const uint8_t* p, int valid) {
  uint2 w = make_uint2(0u, 0u);
  if (valid >= 8) {
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(p));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = j < valid ? (uint32_t)p[j] << (8 * (j & 3)) : 0u;
      if (j < 4) w.x |= b;
      else w.y |= b;
    }
  }
  return w;
}
// The values that eight codes stand for.
__device__ __forceinline__ void values8(uint2 w, float scale, float (&x)[8]) {
  e4m3x2_dec(w.x & 0xFFFFu, x[0], x[1]);
  e4m3x2_dec(w.x >> 16, x[2], x[3]);
  e4m3x2_dec(w.y & 0xFFFFu, x[4], x[5]);
  e4m3x2_dec(w.y >> 16, x[6], x[7]);
  scaled8(x, scale, x);
}
// Codes of eight values with their block's scale byte, and the byte by the block's first
// lane: to a row's chunk at `codes` and the place `at` of its scale.
__device__ __forceinline__ void put_chunk(uint8_t* codes, uint8_t* scales, int64_t at, int valid, uint2 w, uint32_t byte) {
  if (valid <= 0) return;
  store_codes8(codes, valid, w);
  if ((threadIdx.x & 15) == 0) scales[at] = (uint8_t)byte;
}
// Eight values as codes with the scale of the 1 x 128 block that 16 lanes hold, by
// whole warps; elements from `valid` on are 0.
__device__ __forceinline__ void put_codes8(uint8_t* codes, uint8_t* scales, int64_t at, int valid, const float (&x)[8]) {
  bool odd;
  const uint32_t byte = block_byte(x, odd);
  put_chunk(codes, scales, at, valid, codes8(x, inverse_scale(byte), odd), byte);
}
// The same where the block's largest magnitude `top` is known, and finite.
__device__ __forceinline__ void put_finite8(uint8_t* codes, uint8_t* scales, int64_t at, int valid, const float (&x)[8],
                                            uint32_t top) {
  const uint32_t byte = scale_byte(top);
  float v[8];
  scaled8(x, inverse_scale(byte), v);
  put_chunk(codes, scales, at, valid, codes8(v), byte);
}

// A row of a plain matrix (S its element type) or of a kept one (S E4m3), by chunks:
// `ahead` asks for one, `values` makes it eight fp32 values.
template <typename S, bool VEC>
struct Source {
  Row<S, VEC> row;
  using Ask = Ahead<S, VEC>;
  __device__ __forceinline__ Source(const void* base, const void*, int64_t pitch, int64_t rows, int64_t cols, int64_t r)
      : row(base, pitch, rows, cols, r) {}
  __device__ __forceinline__ Ask ahead(int64_t c, int valid) const { return row.ahead(c, valid); }
  __device__ __forceinline__ void values(const Ask& a, int64_t c, int valid, float (&x)[8]) const {
    unpack(row.chunk(a, c, valid), x);
  }
};
struct KeptAsk {
  uint2 codes;
  uint32_t byte;
};
template <bool VEC>
struct Source<E4m3, VEC> {
  const uint8_t *codes, *scales;
  using Ask = KeptAsk;
  int64_t r, panel;
  __device__ __forceinline__ Source(const void* base, const void* tiles, int64_t pitch, int64_t, int64_t cols, int64_t row)
      : codes(static_cast<const uint8_t*>(base) + row * pitch), scales(static_cast<const uint8_t*>(tiles)), r(row),
        panel((cols + 511) / 512) {}
  __device__ __forceinline__ Ask ahead(int64_t c, int valid) const {
    KeptAsk a = {};
    if (valid > 0) {
      a.codes = load_codes8(codes + c, valid);
      a.byte = scales[scale_place(r, c >> 7, panel)];
    }
    return a;
  }
  __device__ __forceinline__ void values(const Ask& a, int64_t, int, float (&x)[8]) const {
    values8(a.codes, scale_of(a.byte), x);
  }
};

// Blocks of chunks by rows: a row's chunks (to whole 128-element blocks and whole warps)
// in equal parts of at most a CTA's threads, and as many rows as fill it.
struct ChunkGrid {
  dim3 grid, block;
  ChunkGrid(int64_t rows, int64_t cols, int threads) {
    const int64_t slots = (cols + 255) / 256 * 32, parts = (slots + threads - 1) / threads;
    const int64_t width = ((slots + parts - 1) / parts + 31) / 32 * 32, high = threads / width;
    const int64_t groups = (rows + high - 1) / high;
    block = dim3((unsigned)width, (unsigned)(high < rows ? high : rows));
    grid = dim3((unsigned)((slots + width - 1) / width), (unsigned)(groups < 65535 ? groups : 65535));
  }
  // At most about `ctas` of them, in equal shares of rows.
  void limit(int64_t ctas) {
    const int64_t most = ctas / grid.x;
    if (grid.y > most) grid.y = (unsigned)(most < 1 ? 1 : most);
  }
};

// ---------------------------------------------------------------- reductions
// Sum over a CTA of at most 32 warps, the same bits in every thread: lanes by a
// butterfly, then the warps' sums in order.  `part` holds 33 floats; two
// consecutive sums need different ones.
__device__ __forceinline__ float cta_sum(float v, float* part, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// 1 / sqrt(v): rsqrtf, whose error of up to two units in the last place would move
// a block's scale where its largest value lies that near to a power of two times
// 448, and one Newton step (r += r (1 - v r^2) / 2), for positive finite v.
__device__ __forceinline__ float reciprocal_root(float v) {
  const float r = rsqrtf(v);
  const float half_error = fmaf(-0.5f * v * r, r, 0.5f);
  return r > 0.0f && r < 1e30f ? fmaf(r, half_error, r) : r;
}

}  // namespace psopt
