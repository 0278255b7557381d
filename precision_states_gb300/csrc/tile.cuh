// tile.cuh -- what the operators that make 8-bit operands share beside layer.cuh:
// magnitudes of chunks as they lie in memory, and stores of 16 codes.
#pragma once

#include "layer.cuh"

namespace psopt {

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
