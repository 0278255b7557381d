// layer.h -- host-side declarations shared by the training-layer operators'
// API (layer.cu) and their launch files.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "opt_layer.h"

namespace psopt {

// Dropout as the kernels take it: threshold T of the 16-bit draws (0: no
// dropout, 65536: everything dropped), the kept elements' factor, the seed's
// round keys and the counter's upper words.
struct DropArgs {
  uint32_t threshold;
  float factor;
  uint32_t tensor, step32;
  uint32_t rk[20];
};

cudaError_t launch_dropout(const opt_dropout_args& a, const DropArgs& d, cudaStream_t s);
cudaError_t launch_rms_norm(const opt_rms_norm_args& a, const DropArgs& d, int sm_count, cudaStream_t s);
cudaError_t launch_rms_norm_backward(const opt_rms_norm_backward_args& a, const DropArgs& d, int sm_count,
                                     cudaStream_t s);
cudaError_t launch_quantize(const opt_quantize_args& a, cudaStream_t s);
cudaError_t launch_dequantize(const opt_dequantize_args& a, int sm_count, cudaStream_t s);
cudaError_t launch_gated(const opt_gated_args& a, int sm_count, cudaStream_t s);
cudaError_t launch_gated_backward(const opt_gated_backward_args& a, int sm_count, cudaStream_t s);
cudaError_t launch_head_norm(const opt_head_norm_args& a, int sm_count, cudaStream_t s);
cudaError_t launch_head_norm_backward(const opt_head_norm_backward_args& a, int sm_count, cudaStream_t s);
cudaError_t launch_matmul(const opt_matmul_args& a, int sm_count, cudaStream_t s);
bool matmul_waits(const opt_matmul_args& a);              // whether the product's kernel waits on anything
cudaError_t matmul_form(const opt_matmul_args& a, int sm_count, int32_t* form);      // opt_matmul_form, of one that waits
cudaError_t layer_flags(int* flags, cudaStream_t s);      // read and clear

// CTAs of the backward norm, and so rows of its weight-gradient partial sums:
// never more than this, whatever the device.
constexpr int64_t kNormBackwardMaxCtas = 1024;
// Rows of partial sums that the workspace holds; 0 where the weight's gradient is
// formed without them, by CTAs of the same launch that read dy and h again: up to
// 512 rows and 2^21 elements.
__host__ __device__ constexpr inline int64_t norm_backward_parts(int64_t rows, int64_t cols) {
  return rows <= 512 && rows * cols <= ((int64_t)1 << 21) ? 0 : rows < kNormBackwardMaxCtas ? rows : kNormBackwardMaxCtas;
}

// CTAs of the heads' backward pass, and so rows of its weight-gradient partial sums
// (2 x dim each).
constexpr int64_t kHeadBackwardMaxCtas = 1024;
constexpr int64_t kHeadMaxDim = 1024;
__host__ __device__ constexpr inline int64_t head_backward_parts(int64_t rows, int64_t heads) {
  return rows * heads < kHeadBackwardMaxCtas ? rows * heads : kHeadBackwardMaxCtas;
}

}  // namespace psopt
