// matmul_few.cu -- the product of opt_matmul when one operand has at most eight
// rows (new tokens against a weight): the other operand's bytes are the time, so
// they go from memory to registers once, in long pieces, with no staging.
//
// A warp takes 16 rows of the long operand and 256 of the depth at a time: lane
// (g, t) loads the 16 bytes at depth 64 c + 16 t of rows g and g + 8, for the
// four c at once (256 contiguous bytes of each row in flight), and those of row
// g of the short operand.  Both sides use the same permutation of the depth, so
// the loaded words are the fragments of mma.sync m16n8k32 as they are; at eight
// columns the product is far from any tensor peak, and tcgen05's way through
// shared memory and tensor memory only adds latency (1 x 4096 x 4096: 4.7 us
// here, 6.9 there; 1 x 14336 x 4096: 12.1 and 13.3).  A block of 128 is summed
// with no scale, then added to the fp32 sum with both scales.  A CTA's warps
// share the depth of its 16 rows; their sums are added in order.
//
// Bound by the weight's bytes once they are many (1 x 57344 x 4096: 38.7 us, 6.1
// TB/s, 0.92 of the measured copy), by launch and one wave's latency before.
// 512 of the depth per step at two CTAs per SM took 17.7 us instead of 12.1, and
// the next step's loads ahead of this step's products 15.2.
#include "layer.cuh"
#include "matmul.h"

namespace psopt {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kRows = 16, kCols = 8, kDepth = 256;      // of a warp's step

struct FewArgs {
  const uint8_t* x;            // the long operand: codes, scales, rows
  const uint8_t* sx;
  const uint8_t* y;            // the short one
  const uint8_t* sy;
  int64_t x_pitch, y_pitch;
  int nx, ny, panel;
  uint32_t k;                  // unsigned: a step beyond 2^31 - 1 must not wrap
  OutputArgs out;
};

// 16 codes at depth c of a row; those at or beyond k read as 0 (CHECK: there may
// be such).
template <bool CHECK>
__device__ __forceinline__ uint4 load16(const uint8_t* row, uint32_t c, uint32_t k) {
  uint4 w = make_uint4(0u, 0u, 0u, 0u);
  if (!CHECK || c + 16 <= k) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(row + c));
  } else if (c < k) {
    uint32_t v[4] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (c + i < k) v[i >> 2] |= (uint32_t)row[c + i] << (8 * (i & 3));
    w = make_uint4(v[0], v[1], v[2], v[3]);
  }
  return w;
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// v times the scales of bytes bx and by: by one power of two where it is a
// normal number, else in halves, so that nothing on the way leaves fp32's range
// before the result does.
__device__ __forceinline__ float power_of_two(int e) { return e < -126 ? u2f(0x00400000u) : u2f((uint32_t)(e + 127) << 23); }
__device__ __noinline__ float scaled_rare(float v, int bx, int by) {
  const int e = bx + by - 254, half = e >> 1;
  return bx == 255 || by == 255 ? u2f(0x7FC00000u) : v * power_of_two(half) * power_of_two(e - half);
}

struct Step {          // a warp's words of one step of the depth
  uint4 u[4], v[4], w[4];
};
template <bool CHECK>
__device__ __forceinline__ void load_step(Step& d, const uint8_t* x0, const uint8_t* x1, const uint8_t* y, uint32_t c0,
                                          uint32_t k) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    d.u[c] = load16<CHECK>(x0, c0 + 64 * c, k);
    d.v[c] = load16<CHECK>(x1, c0 + 64 * c, k);
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) d.w[c] = load16<CHECK>(y, c0 + 64 * c, k);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) matmul_few_kernel(const __grid_constant__ FewArgs a) {
  __shared__ float part[kWarps][kRows][kCols];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int row0 = blockIdx.x * kRows;
  // rows that do not exist repeat the last one; their sums are not written
  const int r0 = min(row0 + g, a.nx - 1), r1 = min(row0 + g + 8, a.nx - 1);
  const int y0 = min(2 * t, a.ny - 1), y1 = min(2 * t + 1, a.ny - 1);
  const uint8_t* x0 = a.x + r0 * a.x_pitch;
  const uint8_t* x1 = a.x + r1 * a.x_pitch;
  const uint8_t* y = a.y + min(g, a.ny - 1) * a.y_pitch;
  const uint8_t* sx0 = a.sx + scale_place(r0, 0, a.panel);
  const uint8_t* sx1 = a.sx + scale_place(r1, 0, a.panel);
  const uint8_t* sy0 = a.sy + scale_place(y0, 0, a.panel);
  const uint8_t* sy1 = a.sy + scale_place(y1, 0, a.panel);
  float acc[4] = {};
  for (uint32_t at = warp * kDepth; at < a.k; at += kWarps * kDepth) {
    Step d;
    if (at + kDepth <= a.k) load_step<false>(d, x0, x1, y, at + 16 * t, a.k);
    else load_step<true>(d, x0, x1, y, at + 16 * t, a.k);
    const uint32_t tile = (at >> 9) * 512, shift = (at >> 4) & 16;      // the scale bytes of this half of a tile
    const auto word = [&](const uint8_t* s) { return *reinterpret_cast<const uint32_t*>(s + tile) >> shift; };
    const uint32_t s0 = word(sx0), s1 = word(sx1), q0 = word(sy0), q1 = word(sy1);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (at + 128 * b >= a.k) break;
      float sum[4] = {};
#pragma unroll
      for (int c = 2 * b; c < 2 * b + 2; ++c) {
        mma(sum, d.u[c].x, d.v[c].x, d.u[c].y, d.v[c].y, d.w[c].x, d.w[c].y);
        mma(sum, d.u[c].z, d.v[c].z, d.u[c].w, d.v[c].w, d.w[c].z, d.w[c].w);
      }
      const int bx[2] = {(int)((s0 >> (8 * b)) & 255u), (int)((s1 >> (8 * b)) & 255u)};
      const int by[2] = {(int)((q0 >> (8 * b)) & 255u), (int)((q1 >> (8 * b)) & 255u)};
      const int low = min(bx[0], bx[1]) + min(by[0], by[1]) - 127, top = max(bx[0], bx[1]), top_y = max(by[0], by[1]);
      if (low >= 1 && top + top_y - 127 <= 254 && max(top, top_y) < 255) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(sum[i], u2f((uint32_t)(bx[i >> 1] + by[i & 1] - 127) << 23), acc[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += scaled_rare(sum[i], bx[i >> 1], by[i & 1]);
      }
    }
  }
  part[warp][g][2 * t] = acc[0];
  part[warp][g][2 * t + 1] = acc[1];
  part[warp][g + 8][2 * t] = acc[2];
  part[warp][g + 8][2 * t + 1] = acc[3];
  __syncthreads();
  const int r = threadIdx.x % kRows, c = threadIdx.x / kRows;
  if (c < a.ny && row0 + r < a.nx) {
    float s = part[0][r][c];
#pragma unroll
    for (int p = 1; p < kWarps; ++p) s += part[p][r][c];
    if (a.out.addend != nullptr)
      s += element(static_cast<const T*>(a.out.addend) + place(a.out, a.out.addend_pitch, row0 + r, c));
    put(static_cast<T*>(a.out.out) + place(a.out, a.out.out_pitch, row0 + r, c), s);
  }
}

}  // namespace

cudaError_t launch_matmul_few(const opt_matmul_args& c, const OutputArgs& out, cudaStream_t s) {
  const auto u8 = [](const void* p) { return static_cast<const uint8_t*>(p); };
  FewArgs f = {};
  f.out = out;
  f.k = (uint32_t)c.k;
  f.panel = (int)((c.k + 511) / 512);
  f.x = u8(out.swap ? c.d_b : c.d_a);
  f.sx = u8(out.swap ? c.d_b_scales : c.d_a_scales);
  f.y = u8(out.swap ? c.d_a : c.d_b);
  f.sy = u8(out.swap ? c.d_a_scales : c.d_b_scales);
  f.x_pitch = out.swap ? c.b_pitch : c.a_pitch;
  f.y_pitch = out.swap ? c.a_pitch : c.b_pitch;
  f.nx = (int)(out.swap ? c.n : c.m);
  f.ny = (int)(out.swap ? c.m : c.n);
  const unsigned grid = (unsigned)((f.nx + (int64_t)kRows - 1) / kRows);
  if (c.out_dtype == OPT_F32) matmul_few_kernel<float><<<grid, kThreads, 0, s>>>(f);
  else matmul_few_kernel<Bf16><<<grid, kThreads, 0, s>>>(f);
  return cudaGetLastError();
}

}  // namespace psopt
