// layer.cu -- the C ABI of the training-layer operators (opt_layer.h):
// validation on the host, then one call of the operator's launcher.
#include <cmath>

#include "common.cuh"
#include "layer.h"

namespace psopt {
namespace {

constexpr int64_t kMaxDim = 0x7FFFFFFF;

bool plain_type(int32_t t) { return t == OPT_F32 || t == OPT_BF16; }
int64_t plain_size(int32_t t) { return t == OPT_F32 ? 4 : 2; }

// A matrix of `rows` x `cols` that must be there: NULL, pitch, alignment.
int check_matrix(const void* p, int64_t pitch, int64_t rows, int64_t cols, int64_t align) {
  if (p == nullptr) return OPT_EINVAL;
  if (rows > 1 && pitch < cols) return OPT_EINVAL;
  return ((uintptr_t)p % (uintptr_t)align) ? OPT_EALIGN : OPT_OK;
}
int check_codes(const void* codes, int64_t pitch, const void* scales, int64_t rows, int64_t cols) {
  if (scales == nullptr) return OPT_EINVAL;
  if (int st = check_matrix(codes, pitch, rows, cols, 16)) return st;
  if ((rows > 1 && pitch % 16 != 0) || ((uintptr_t)scales & 15u)) return OPT_EALIGN;
  return OPT_OK;
}
int check_sizes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return OPT_EINVAL;
  return rows > kMaxDim || cols > kMaxDim ? OPT_ELIMIT : OPT_OK;
}

#define PS_TRY(expr)                 \
  do {                               \
    const int ps_st = (expr);        \
    if (ps_st != OPT_OK) return ps_st; \
  } while (0)

int drop_args(double p, uint64_t seed, uint32_t tensor, int64_t step, DropArgs* d) {
  if (!(p >= 0.0 && p <= 1.0) || step < 0) return OPT_EINVAL;
  d->threshold = (uint32_t)std::nearbyint(65536.0 * p);
  d->factor = d->threshold < 65536u ? (float)(65536.0 / (double)(65536u - d->threshold)) : 0.0f;
  d->tensor = tensor;
  d->step32 = (uint32_t)step;
  philox_round_keys(seed, d->rk);
  return OPT_OK;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? OPT_OK : OPT_ECUDA; }

int sm_count_of(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return OPT_ECUDA;
  return OPT_OK;
}

}  // namespace
}  // namespace psopt

using namespace psopt;

extern "C" {

int64_t opt_scales_bytes(int64_t rows, int64_t cols) {
  const int st = check_sizes(rows, cols);
  if (st != OPT_OK) return st;
  return ((rows + 127) / 128) * ((cols + 511) / 512) * 512;
}

int opt_dropout(const opt_dropout_args* a, void* stream) {
  if (a == nullptr) return OPT_EINVAL;
  PS_TRY(check_sizes(a->rows, a->cols));
  if (!plain_type(a->dtype)) return OPT_EUNSUPPORTED;
  DropArgs d;
  PS_TRY(drop_args(a->p, a->seed, a->tensor_index, a->step, &d));
  if (a->rows == 0 || a->cols == 0) return OPT_OK;
  const int64_t es = plain_size(a->dtype);
  PS_TRY(check_matrix(a->d_x, a->x_pitch, a->rows, a->cols, es));
  PS_TRY(check_matrix(a->d_y, a->y_pitch, a->rows, a->cols, es));
  if (a->d_residual != nullptr) PS_TRY(check_matrix(a->d_residual, a->residual_pitch, a->rows, a->cols, es));
  return status_of(launch_dropout(*a, d, static_cast<cudaStream_t>(stream)));
}

int opt_rms_norm(const opt_rms_norm_args* a, void* stream) {
  if (a == nullptr) return OPT_EINVAL;
  PS_TRY(check_sizes(a->rows, a->cols));
  if (!plain_type(a->dtype) || !plain_type(a->weight_dtype)) return OPT_EUNSUPPORTED;
  if (!(a->eps >= 0.0f) || std::isinf(a->eps)) return OPT_EINVAL;
  DropArgs d;
  PS_TRY(drop_args(a->p, a->seed, a->tensor_index, a->step, &d));
  if (a->rows == 0 || a->cols == 0) return OPT_OK;
  const int64_t es = plain_size(a->dtype);
  PS_TRY(check_matrix(a->d_x, a->x_pitch, a->rows, a->cols, es));
  PS_TRY(check_matrix(a->d_weight, a->cols, 1, a->cols, plain_size(a->weight_dtype)));
  if (a->d_residual != nullptr) PS_TRY(check_matrix(a->d_residual, a->residual_pitch, a->rows, a->cols, es));
  if (a->d_h != nullptr) PS_TRY(check_matrix(a->d_h, a->h_pitch, a->rows, a->cols, es));
  if (a->d_y != nullptr) PS_TRY(check_matrix(a->d_y, a->y_pitch, a->rows, a->cols, es));
  if (a->d_rstd != nullptr) PS_TRY(check_matrix(a->d_rstd, 1, a->rows, 1, 4));
  if (a->d_codes != nullptr || a->d_scales != nullptr)
    PS_TRY(check_codes(a->d_codes, a->codes_pitch, a->d_scales, a->rows, a->cols));
  if (a->d_h == nullptr && a->d_y == nullptr && a->d_rstd == nullptr && a->d_codes == nullptr) return OPT_EINVAL;
  int sms = 0;
  PS_TRY(sm_count_of(&sms));
  return status_of(launch_rms_norm(*a, d, sms, static_cast<cudaStream_t>(stream)));
}

int64_t opt_rms_norm_backward_workspace(int64_t rows, int64_t cols) {
  const int st = check_sizes(rows, cols);
  if (st != OPT_OK) return st;
  return norm_backward_parts(rows, cols) * ((cols + 3) / 4 * 4) * (int64_t)sizeof(float);
}

int opt_rms_norm_backward(const opt_rms_norm_backward_args* a, void* stream) {
  if (a == nullptr || a->reserved != 0) return OPT_EINVAL;
  PS_TRY(check_sizes(a->rows, a->cols));
  if (!plain_type(a->dtype) || !plain_type(a->weight_dtype)) return OPT_EUNSUPPORTED;
  DropArgs d;
  PS_TRY(drop_args(a->p, a->seed, a->tensor_index, a->step, &d));
  if (a->cols == 0) return OPT_OK;
  if (a->d_dweight != nullptr) PS_TRY(check_matrix(a->d_dweight, a->cols, 1, a->cols, 4));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->rows == 0)      // the sum over no rows
    return a->d_dweight == nullptr
               ? OPT_OK
               : status_of(cudaMemsetAsync(a->d_dweight, 0, (size_t)a->cols * sizeof(float), s));
  const int64_t es = plain_size(a->dtype);
  PS_TRY(check_matrix(a->d_dy, a->dy_pitch, a->rows, a->cols, es));
  PS_TRY(check_matrix(a->d_h, a->h_pitch, a->rows, a->cols, es));
  PS_TRY(check_matrix(a->d_weight, a->cols, 1, a->cols, plain_size(a->weight_dtype)));
  PS_TRY(check_matrix(a->d_rstd, 1, a->rows, 1, 4));
  PS_TRY(check_matrix(a->d_dh, a->dh_pitch, a->rows, a->cols, es));
  if (a->d_dh_in != nullptr) PS_TRY(check_matrix(a->d_dh_in, a->dh_in_pitch, a->rows, a->cols, es));
  if (a->d_dx != nullptr) PS_TRY(check_matrix(a->d_dx, a->dx_pitch, a->rows, a->cols, es));
  const int64_t need = opt_rms_norm_backward_workspace(a->rows, a->cols);
  if (a->d_dweight != nullptr && need > 0) {
    if (a->d_workspace == nullptr || a->workspace_bytes < need) return OPT_EINVAL;
    if ((uintptr_t)a->d_workspace & 15u) return OPT_EALIGN;
  }
  int sms = 0;
  PS_TRY(sm_count_of(&sms));
  return status_of(launch_rms_norm_backward(*a, d, sms, s));
}

int opt_quantize(const opt_quantize_args* a, void* stream) {
  if (a == nullptr) return OPT_EINVAL;
  PS_TRY(check_sizes(a->rows, a->cols));
  if (!plain_type(a->dtype)) return OPT_EUNSUPPORTED;
  if (a->block_rows != 1 && a->block_rows != 128) return OPT_EINVAL;
  if (a->rows == 0 || a->cols == 0) return OPT_OK;
  PS_TRY(check_matrix(a->d_x, a->x_pitch, a->rows, a->cols, plain_size(a->dtype)));
  if (a->d_codes == nullptr && a->d_codes_t == nullptr) return OPT_EINVAL;
  if (a->d_codes != nullptr || a->d_scales != nullptr)
    PS_TRY(check_codes(a->d_codes, a->codes_pitch, a->d_scales, a->rows, a->cols));
  if (a->d_codes_t != nullptr || a->d_scales_t != nullptr)
    PS_TRY(check_codes(a->d_codes_t, a->codes_t_pitch, a->d_scales_t, a->cols, a->rows));
  if (((a->rows + 127) / 128) * ((a->cols + 127) / 128) > kMaxDim) return OPT_ELIMIT;
  return status_of(launch_quantize(*a, static_cast<cudaStream_t>(stream)));
}

int opt_matmul(const opt_matmul_args* a, void* stream) {
  if (a == nullptr || (a->flags & ~OPT_MATMUL_WAIT_DRILL) != 0) return OPT_EINVAL;
  PS_TRY(check_sizes(a->m, a->n));
  PS_TRY(check_sizes(a->k, 0));
  if (!plain_type(a->out_dtype)) return OPT_EUNSUPPORTED;
  if (a->m == 0 || a->n == 0) return OPT_OK;
  const int64_t es = plain_size(a->out_dtype);
  PS_TRY(check_matrix(a->d_out, a->out_pitch, a->m, a->n, es));
  if (a->d_addend != nullptr) PS_TRY(check_matrix(a->d_addend, a->addend_pitch, a->m, a->n, es));
  if (a->k > 0) {
    PS_TRY(check_codes(a->d_a, a->a_pitch, a->d_a_scales, a->m, a->k));
    PS_TRY(check_codes(a->d_b, a->b_pitch, a->d_b_scales, a->n, a->k));
  }
  if (a->flags != 0 && !matmul_waits(*a)) return OPT_EUNSUPPORTED;
  int sms = 0;
  PS_TRY(sm_count_of(&sms));
  return status_of(launch_matmul(*a, sms, static_cast<cudaStream_t>(stream)));
}

int opt_matmul_form(const opt_matmul_args* a, int32_t h_form[5]) {
  if (a == nullptr || h_form == nullptr) return OPT_EINVAL;
  PS_TRY(check_sizes(a->m, a->n));
  PS_TRY(check_sizes(a->k, 0));
  for (int i = 0; i < 5; ++i) h_form[i] = 0;
  if (a->m == 0 || a->n == 0 || !matmul_waits(*a)) return OPT_OK;
  int sms = 0;
  PS_TRY(sm_count_of(&sms));
  return status_of(matmul_form(*a, sms, h_form));
}

int opt_layer_status(int32_t* h_flags, void* stream) {
  if (h_flags == nullptr) return OPT_EINVAL;
  int flags = 0;
  PS_TRY(status_of(layer_flags(&flags, static_cast<cudaStream_t>(stream))));
  *h_flags = flags;
  return OPT_OK;
}

}  // extern "C"
