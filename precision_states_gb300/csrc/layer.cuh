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

// Eight elements at p.  VEC: all eight exist and p is 16-byte aligned;
// otherwise the first `valid` exist, and the others read as 0.
template <bool VEC>
__device__ __forceinline__ void load8(const Bf16* p, int valid, float (&x)[8]) {
  if (VEC) {
    uint4 w;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(p));
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = u2f(ws[k] << 16);
      x[2 * k + 1] = u2f(ws[k] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = j < valid ? u2f((uint32_t)p[j].bits << 16) : 0.0f;
  }
}
template <bool VEC>
__device__ __forceinline__ void load8(const float* p, int valid, float (&x)[8]) {
  if (VEC) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float4 v;
      asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];"
                   : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p + 4 * k));
      x[4 * k] = v.x; x[4 * k + 1] = v.y; x[4 * k + 2] = v.z; x[4 * k + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = j < valid ? p[j] : 0.0f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(Bf16* p, int valid, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = bf16x2_rn(x[2 * k], x[2 * k + 1]);
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

// ----------------------------------------------------------------- dropout
// The draws of elements i .. i + 7 of the matrix's row-major order as 128
// bits, element i + j in bits 16 j: the generator's four words as they are when
// i is a multiple of 8 (VEC), else two calls' eight words moved down by i mod 8
// half-words.
__device__ __forceinline__ uint4 drop_group(uint64_t g, const DropArgs& d) {
  return philox10_rk(make_uint4((uint32_t)g, (uint32_t)(g >> 32) | 0x80000000u, d.tensor, d.step32), d.rk);
}
template <bool VEC>
__device__ __forceinline__ uint4 drop_draws(uint64_t i, const DropArgs& d) {
  const uint4 lo = drop_group(i >> 3, d);
  const int off = (int)(i & 7);
  if (VEC || off == 0) return lo;
  const uint4 hi = drop_group((i >> 3) + 1, d);
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
// x <- dropout(x) for the eight elements from i on.
template <bool VEC>
__device__ __forceinline__ void drop8(float (&x)[8], uint64_t i, const DropArgs& d) {
  if (d.threshold == 0u) return;
  const uint4 r = drop_draws<VEC>(i, d);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t draw = (w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
    x[j] = draw >= d.threshold ? x[j] * d.factor : 0.0f;
  }
}

// ------------------------------------------------------------ block scales
// Scale byte of a block from the bits of its largest finite magnitude: with
// magnitude 1.f 2^E, E - 8 if 1.f <= 1.75 (448 = 1.75 2^8) else E - 7, never
// below -127 (which also serves blocks of zeros and of subnormals).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top_bits) {
  const int e = (int)(top_bits >> 23) - 8 + ((top_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 0);
}
// 2^-e for a scale byte; scale_byte never exceeds 247, so this is normal.
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return u2f((254u - byte) << 23); }

__device__ __forceinline__ uint32_t magnitude(float x) { return f2u(x) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u;

// Largest magnitude's bits of eight elements (as integers: the order of the
// magnitudes, with infinity and NaN above all); finite_top8 leaves those out.
__device__ __forceinline__ uint32_t top8(const float (&x)[8]) {
  uint32_t t = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) t = max(t, magnitude(x[j]));
  return t;
}
__device__ __forceinline__ uint32_t finite_top8(const float (&x)[8]) {
  uint32_t t = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) t = max(t, magnitude(x[j]) < kInfBits ? magnitude(x[j]) : 0u);
  return t;
}
// Largest of a value over the 16 lanes of a 128-element block.
__device__ __forceinline__ uint32_t max16(uint32_t t) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) t = max(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
  return t;
}

// Codes of eight elements over 2^e (inv = 2^-e); `odd` says that the block
// holds an infinity or NaN, which the converter would clamp or keep: both are
// stored as NaN.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv, bool odd) {
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = x[j] * inv;
  if (odd) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (magnitude(x[j]) >= kInfBits) v[j] = u2f(0x7FC00000u);
  }
  return make_uint2(e4m3x2_rn(v[0], v[1]) | (e4m3x2_rn(v[2], v[3]) << 16),
                    e4m3x2_rn(v[4], v[5]) | (e4m3x2_rn(v[6], v[7]) << 16));
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

// Place of the scale byte of row r, block b (opt_layer.h); panel = ceil(B / 4).
__host__ __device__ __forceinline__ int64_t scale_place(int64_t r, int64_t b, int64_t panel) {
  return 512 * ((r >> 7) * panel + (b >> 2)) + 16 * (r & 31) + 4 * ((r >> 5) & 3) + (b & 3);
}

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

}  // namespace psopt
