// matmul.cu -- out = a b^T (+ addend) of two E4M3 operands with a scale for each
// block of 128 along the depth (opt_layer.h).
#include "layer.cuh"

namespace psopt {
namespace {

constexpr int kTile = 64, kDepth = 32, kThreads = 256;

// A 64 x 64 tile of the output per CTA, 4 x 4 outputs per thread; both
// operands' values (code times scale) lie in shared memory in fp32.
__device__ __forceinline__ void stage(float (*t)[kTile + 4], const uint8_t* codes, int64_t pitch, const uint8_t* scales,
                                      int64_t row0, int64_t rows, int64_t k0, int64_t k, int64_t panel) {
  for (int i = threadIdx.x; i < kTile * kDepth; i += kThreads) {
    const int64_t r = row0 + i / kDepth, c = k0 + i % kDepth;
    float v = 0.0f;
    if (r < rows && c < k) {
      const uint32_t b = scales[scale_place(r, c >> 7, panel)];
      v = e4m3_dec(codes[r * pitch + c]) * (b > 0u ? u2f(b << 23) : u2f(1u << 22));
    }
    t[i % kDepth][i / kDepth] = v;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) matmul_kernel(const __grid_constant__ opt_matmul_args a, int64_t col_tiles) {
  __shared__ float sa[kDepth][kTile + 4], sb[kDepth][kTile + 4];
  const int64_t m0 = kTile * (blockIdx.x / col_tiles), n0 = kTile * (blockIdx.x % col_tiles);
  const int64_t panel = (a.k + 511) / 512;
  const int tm = 4 * (threadIdx.x / 16), tn = 4 * (threadIdx.x % 16);
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < a.k; k0 += kDepth) {
    __syncthreads();
    stage(sa, static_cast<const uint8_t*>(a.d_a), a.a_pitch, static_cast<const uint8_t*>(a.d_a_scales), m0, a.m, k0, a.k, panel);
    stage(sb, static_cast<const uint8_t*>(a.d_b), a.b_pitch, static_cast<const uint8_t*>(a.d_b_scales), n0, a.n, k0, a.k, panel);
    __syncthreads();
    for (int k = 0; k < kDepth; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][tm + i], sb[k][tn + j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = m0 + tm + i, c = n0 + tn + j;
      if (r < a.m && c < a.n) {
        float v[8] = {}, x[8] = {acc[i][j]};
        if (a.d_addend != nullptr) load8<false>(static_cast<const T*>(a.d_addend) + r * a.addend_pitch + c, 1, v);
        x[0] += v[0];
        store8<false>(static_cast<T*>(a.d_out) + r * a.out_pitch + c, 1, x);
      }
    }
}

}  // namespace

cudaError_t launch_matmul(const opt_matmul_args& a, int sm_count, cudaStream_t s) {
  (void)sm_count;
  const int64_t ct = (a.n + kTile - 1) / kTile, tiles = (a.m + kTile - 1) / kTile * ct;
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  if (a.out_dtype == OPT_F32) matmul_kernel<float><<<(unsigned)tiles, kThreads, 0, s>>>(a, ct);
  else matmul_kernel<Bf16><<<(unsigned)tiles, kThreads, 0, s>>>(a, ct);
  return cudaGetLastError();
}

}  // namespace psopt
