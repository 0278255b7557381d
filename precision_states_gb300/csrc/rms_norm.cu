// rms_norm.cu -- branch dropout, residual sum, root-mean-square norm and 8-bit
// output, and their gradients (opt_layer.h).
#include "layer.cuh"

namespace psopt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Chunk c (eight elements) of row r of h = residual + dropout(x).
template <typename T, bool VEC>
__device__ __forceinline__ void h_chunk(const opt_rms_norm_args& a, const DropArgs& d, int64_t r, int64_t c, int valid,
                                        float (&h)[8]) {
  load8<VEC>(static_cast<const T*>(a.d_x) + r * a.x_pitch + c, valid, h);
  drop8<VEC>(h, (uint64_t)(r * a.cols + c), d);
  if (a.d_residual != nullptr) {
    float res[8];
    load8<VEC>(static_cast<const T*>(a.d_residual) + r * a.residual_pitch + c, valid, res);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] += res[j];
  }
}

// One CTA per row, any width: a pass for the sum of squares, a second one that
// forms h again and writes.
template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(kThreads) rms_norm_kernel(const __grid_constant__ opt_rms_norm_args a,
                                                            const __grid_constant__ DropArgs d) {
  __shared__ float part[2][33];
  const int64_t panel = (a.cols + 511) / 512;
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, turn ^= 1) {
    float sum = 0.0f, h[8];
    for (int64_t c = 8 * threadIdx.x; c < a.cols; c += 8 * kThreads) {
      h_chunk<T, VEC>(a, d, r, c, (int)min(a.cols - c, (int64_t)8), h);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(h[j], h[j], sum);
    }
    sum = cta_sum(sum, part[turn], kWarps);
    const float rstd = 1.0f / sqrtf(sum / (float)a.cols + a.eps);
    if (threadIdx.x == 0 && a.d_rstd != nullptr) a.d_rstd[r] = rstd;
    for (int64_t c0 = 0; c0 < a.cols; c0 += 8 * kThreads) {
      const int64_t c = c0 + 8 * threadIdx.x;
      const int valid = (int)max(min(a.cols - c, (int64_t)8), (int64_t)0);
      float y[8];
      if (valid > 0) {
        h_chunk<T, VEC>(a, d, r, c, valid, h);
        if (a.d_h != nullptr) store8<VEC>(static_cast<T*>(a.d_h) + r * a.h_pitch + c, valid, h);
        load8<VEC>(static_cast<const W*>(a.d_weight) + c, valid, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= h[j] * rstd;
        if (a.d_y != nullptr) store8<VEC>(static_cast<T*>(a.d_y) + r * a.y_pitch + c, valid, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = j < valid ? y[j] : 0.0f;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = 0.0f;
      }
      if (a.d_codes != nullptr) {
        uint32_t top = max16(top8(y));
        const bool odd = top >= kInfBits;
        if (__any_sync(0xFFFFFFFFu, odd)) {
          const uint32_t finite = max16(finite_top8(y));
          if (odd) top = finite;
        }
        const uint32_t byte = scale_byte(top);
        if (valid > 0) {
          store_codes8(static_cast<uint8_t*>(a.d_codes) + r * a.codes_pitch + c, valid,
                       codes8(y, inverse_scale(byte), odd));
          if ((threadIdx.x & 15) == 0)
            static_cast<uint8_t*>(a.d_scales)[scale_place(r, c >> 7, panel)] = (uint8_t)byte;
        }
      }
    }
  }
}

// One CTA per row at a time; the weight's gradient is summed over the CTA's
// rows in its row of the workspace, each column by the same thread throughout.
template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(kThreads) rms_norm_backward_kernel(
    const __grid_constant__ opt_rms_norm_backward_args a, const __grid_constant__ DropArgs d) {
  __shared__ float part[2][33];
  float* dw = a.d_dweight == nullptr ? nullptr
                                     : static_cast<float*>(a.d_workspace) + (int64_t)blockIdx.x * ((a.cols + 3) / 4 * 4);
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, turn ^= 1) {
    const T* dy_row = static_cast<const T*>(a.d_dy) + r * a.dy_pitch;
    const T* h_row = static_cast<const T*>(a.d_h) + r * a.h_pitch;
    float sum = 0.0f, dy[8], h[8], w[8];
    for (int64_t c = 8 * threadIdx.x; c < a.cols; c += 8 * kThreads) {
      const int valid = (int)min(a.cols - c, (int64_t)8);
      load8<VEC>(dy_row + c, valid, dy);
      load8<VEC>(h_row + c, valid, h);
      load8<VEC>(static_cast<const W*>(a.d_weight) + c, valid, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(dy[j] * w[j], h[j], sum);
    }
    sum = cta_sum(sum, part[turn], kWarps);
    const float rstd = a.d_rstd[r];
    const float k = rstd * rstd * (sum / (float)a.cols);
    for (int64_t c = 8 * threadIdx.x; c < a.cols; c += 8 * kThreads) {
      const int valid = (int)min(a.cols - c, (int64_t)8);
      load8<VEC>(dy_row + c, valid, dy);
      load8<VEC>(h_row + c, valid, h);
      load8<VEC>(static_cast<const W*>(a.d_weight) + c, valid, w);
      if (dw != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < valid) dw[c + j] = (r == blockIdx.x ? 0.0f : dw[c + j]) + dy[j] * (h[j] * rstd);
      }
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = rstd * (dy[j] * w[j] - h[j] * k);
      if (a.d_dh_in != nullptr) {
        load8<VEC>(static_cast<const T*>(a.d_dh_in) + r * a.dh_in_pitch + c, valid, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] += w[j];
      }
      store8<VEC>(static_cast<T*>(a.d_dh) + r * a.dh_pitch + c, valid, g);
      if (a.d_dx != nullptr) {
        drop8<VEC>(g, (uint64_t)(r * a.cols + c), d);
        store8<VEC>(static_cast<T*>(a.d_dx) + r * a.dx_pitch + c, valid, g);
      }
    }
  }
}

// dweight = the sum over the workspace's rows, in order.
__global__ void __launch_bounds__(kThreads) dweight_kernel(const float* __restrict__ parts, int n, int64_t cols,
                                                           float* __restrict__ out) {
  const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (c >= cols) return;
  const int64_t pitch = (cols + 3) / 4 * 4;
  float s = 0.0f;
  for (int p = 0; p < n; ++p) s += parts[p * pitch + c];
  out[c] = s;
}

// Rows start on 16 bytes and on a multiple of 8 elements, and hold whole chunks.
struct VecRule {
  int64_t rows, cols;
  bool ok;
  void see(const void* p, int64_t pitch, int64_t es) {
    ok = ok && (p == nullptr || (((uintptr_t)p & 15u) == 0 && (rows == 1 || pitch * es % 16 == 0)));
  }
};

template <typename T, typename W>
cudaError_t forward(const opt_rms_norm_args& a, const DropArgs& d, int sm_count, cudaStream_t s) {
  VecRule v{a.rows, a.cols, a.cols % 8 == 0};
  v.see(a.d_x, a.x_pitch, sizeof(T));
  v.see(a.d_residual, a.residual_pitch, sizeof(T));
  v.see(a.d_weight, 0, sizeof(W));
  v.see(a.d_h, a.h_pitch, sizeof(T));
  v.see(a.d_y, a.y_pitch, sizeof(T));
  const int64_t most = (int64_t)sm_count * 8;
  const int grid = (int)(a.rows < most ? a.rows : most);
  if (v.ok) rms_norm_kernel<T, W, true><<<grid, kThreads, 0, s>>>(a, d);
  else rms_norm_kernel<T, W, false><<<grid, kThreads, 0, s>>>(a, d);
  return cudaGetLastError();
}

template <typename T, typename W>
cudaError_t backward(const opt_rms_norm_backward_args& a, const DropArgs& d, int sm_count, cudaStream_t s) {
  VecRule v{a.rows, a.cols, a.cols % 8 == 0};
  v.see(a.d_dy, a.dy_pitch, sizeof(T));
  v.see(a.d_h, a.h_pitch, sizeof(T));
  v.see(a.d_weight, 0, sizeof(W));
  v.see(a.d_dh_in, a.dh_in_pitch, sizeof(T));
  v.see(a.d_dh, a.dh_pitch, sizeof(T));
  v.see(a.d_dx, a.dx_pitch, sizeof(T));
  int64_t most = (int64_t)sm_count * 4;
  if (most > kNormBackwardMaxCtas) most = kNormBackwardMaxCtas;
  const int grid = (int)(a.rows < most ? a.rows : most);
  if (v.ok) rms_norm_backward_kernel<T, W, true><<<grid, kThreads, 0, s>>>(a, d);
  else rms_norm_backward_kernel<T, W, false><<<grid, kThreads, 0, s>>>(a, d);
  if (a.d_dweight != nullptr)
    dweight_kernel<<<(unsigned)((a.cols + kThreads - 1) / kThreads), kThreads, 0, s>>>(
        static_cast<const float*>(a.d_workspace), grid, a.cols, a.d_dweight);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rms_norm(const opt_rms_norm_args& a, const DropArgs& d, int sm_count, cudaStream_t s) {
  if (a.dtype == OPT_F32)
    return a.weight_dtype == OPT_F32 ? forward<float, float>(a, d, sm_count, s) : forward<float, Bf16>(a, d, sm_count, s);
  return a.weight_dtype == OPT_F32 ? forward<Bf16, float>(a, d, sm_count, s) : forward<Bf16, Bf16>(a, d, sm_count, s);
}

cudaError_t launch_rms_norm_backward(const opt_rms_norm_backward_args& a, const DropArgs& d, int sm_count,
                                     cudaStream_t s) {
  if (a.dtype == OPT_F32)
    return a.weight_dtype == OPT_F32 ? backward<float, float>(a, d, sm_count, s)
                                     : backward<float, Bf16>(a, d, sm_count, s);
  return a.weight_dtype == OPT_F32 ? backward<Bf16, float>(a, d, sm_count, s) : backward<Bf16, Bf16>(a, d, sm_count, s);
}

}  // namespace psopt
