// layer.cu -- the C ABI of the training-layer operators (opt_layer.h):
// validation on the host, then one call of the operator's launcher.
#include <cmath>

#include "common.cuh"
#include "layer.h"

namespace psopt {
namespace {

constexpr int64_t kMaxDim = 0x7FFFFFFF;

#define PS_TRY(expr)                 \
  do {                               \
    const int ps_st = (expr);        \
    if (ps_st != OPT_OK) return ps_st; \
  } while (0)

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

int drop_args(double p, uint64_t seed, uint32_t tensor, int64_t step, DropArgs* d) {
  if (!(p >= 0.0 && p <= 1.0) || step < 0) return OPT_EINVAL;
  d->threshold = (uint32_t)std::nearbyint(65536.0 * p);
  d->factor = d->threshold < 65536u ? (float)(65536.0 / (double)(65536u - d->threshold)) : 0.0f;
  d->tensor = tensor;
  d->step32 = (uint32_t)step;
  philox_round_keys(seed, d->rk);
  return OPT_OK;
}

// A pair of codes and scales that may be left out, but not in part.
int check_kept(const void* codes, int64_t pitch, const void* scales, int64_t rows, int64_t cols) {
  if (codes == nullptr && scales == nullptr) return OPT_OK;
  return check_codes(codes, pitch, scales, rows, cols);
}
// The same of a plain matrix.
int check_optional(const void* p, int64_t pitch, int64_t rows, int64_t cols, int64_t align) {
  return p == nullptr ? OPT_OK : check_matrix(p, pitch, rows, cols, align);
}
int check_tiles(int64_t rows, int64_t cols) {
  return ((rows + 127) / 128) * ((cols + 127) / 128) > kMaxDim ? OPT_ELIMIT : OPT_OK;
}

// What both directions of the heads' norm share; OPT_OK with rows 0 too.
template <typename A>
int check_heads(const A& a) {
  PS_TRY(check_sizes(a.rows, a.positions));
  PS_TRY(check_sizes(a.q_heads, a.k_heads));
  PS_TRY(check_sizes(a.dim, a.rot));
  if (a.dim < 1 || a.rot > a.dim || a.rot % 2 != 0 || (a.flags & ~OPT_HEADS_INTERLEAVED) != 0) return OPT_EINVAL;
  if (a.dim > kHeadMaxDim || a.q_heads * a.dim > kMaxDim || a.k_heads * a.dim > kMaxDim) return OPT_ELIMIT;
  if (!plain_type(a.dtype) || !plain_type(a.weight_dtype)) return OPT_EUNSUPPORTED;
  if (!(a.eps >= 0.0f) || std::isinf(a.eps)) return OPT_EINVAL;
  return OPT_OK;
}
// Its tables, for rows that there are.
template <typename A>
int check_turn(const A& a) {
  if (a.rot == 0) return OPT_OK;
  PS_TRY(check_matrix(a.d_cos, a.rot / 2, a.positions, a.rot / 2, 4));
  PS_TRY(check_matrix(a.d_sin, a.rot / 2, a.positions, a.rot / 2, 4));
  if (a.d_positions == nullptr) return a.rows > a.positions ? OPT_EINVAL : OPT_OK;
  return ((uintptr_t)a.d_positions & 7u) ? OPT_EALIGN : OPT_OK;
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
  PS_TRY(check_tiles(a->rows, a->cols));
  return status_of(launch_quantize(*a, static_cast<cudaStream_t>(stream)));
}

int opt_dequantize(const opt_dequantize_args* a, void* stream) {
  if (a == nullptr || a->reserved != 0) return OPT_EINVAL;
  PS_TRY(check_sizes(a->rows, a->cols));
  if (!plain_type(a->dtype)) return OPT_EUNSUPPORTED;
  if (a->rows == 0 || a->cols == 0) return OPT_OK;
  PS_TRY(check_codes(a->d_codes, a->codes_pitch, a->d_scales, a->rows, a->cols));
  PS_TRY(check_optional(a->d_x, a->x_pitch, a->rows, a->cols, plain_size(a->dtype)));
  PS_TRY(check_kept(a->d_codes_t, a->codes_t_pitch, a->d_scales_t, a->cols, a->rows));
  if (a->d_x == nullptr && a->d_codes_t == nullptr) return OPT_EINVAL;
  PS_TRY(check_tiles(a->rows, a->cols));
  int sms = 0;
  PS_TRY(sm_count_of(&sms));
  return status_of(launch_dequantize(*a, sms, static_cast<cudaStream_t>(stream)));
}

int opt_gated(const opt_gated_args* a, void* stream) {
  if (a == nullptr || a->activation < OPT_ACT_SILU || a->activation > OPT_ACT_RELU) return OPT_EINVAL;
  PS_TRY(check_sizes(a->rows, a->cols));
  if (!plain_type(a->dtype)) return OPT_EUNSUPPORTED;
  if (a->rows == 0 || a->cols == 0) return OPT_OK;
  const int64_t es = plain_size(a->dtype);
  PS_TRY(check_matrix(a->d_gate, a->gate_pitch, a->rows, a->cols, es));
  PS_TRY(check_optional(a->d_up, a->up_pitch, a->rows, a->cols, es));
  PS_TRY(check_optional(a->d_y, a->y_pitch, a->rows, a->cols, es));
  PS_TRY(check_kept(a->d_codes, a->codes_pitch, a->d_scales, a->rows, a->cols));
  PS_TRY(check_kept(a->d_gate_codes, a->gate_codes_pitch, a->d_gate_scales, a->rows, a->cols));
  PS_TRY(check_kept(a->d_up_codes, a->up_codes_pitch, a->d_up_scales, a->rows, a->cols));
  if (a->d_up == nullptr && a->d_up_codes != nullptr) return OPT_EINVAL;
  if (a->d_y == nullptr && a->d_codes == nullptr && a->d_gate_codes == nullptr && a->d_up_codes == nullptr) return OPT_EINVAL;
  int sms = 0;
  PS_TRY(sm_count_of(&sms));
  return status_of(launch_gated(*a, sms, static_cast<cudaStream_t>(stream)));
}

int opt_gated_backward(const opt_gated_backward_args* a, void* stream) {
  if (a == nullptr || a->activation < OPT_ACT_SILU || a->activation > OPT_ACT_RELU) return OPT_EINVAL;
  PS_TRY(check_sizes(a->rows, a->cols));
  if (!plain_type(a->dtype)) return OPT_EUNSUPPORTED;
  if (a->rows == 0 || a->cols == 0) return OPT_OK;
  const int64_t es = plain_size(a->dtype), rows = a->rows, cols = a->cols;
  PS_TRY(check_matrix(a->d_dy, a->dy_pitch, rows, cols, es));
  if (a->d_gate_scales != nullptr) {
    PS_TRY(check_codes(a->d_gate, a->gate_pitch, a->d_gate_scales, rows, cols));
    PS_TRY(check_kept(a->d_up, a->up_pitch, a->d_up_scales, rows, cols));
  } else {
    if (a->d_up_scales != nullptr) return OPT_EINVAL;
    PS_TRY(check_matrix(a->d_gate, a->gate_pitch, rows, cols, es));
    PS_TRY(check_optional(a->d_up, a->up_pitch, rows, cols, es));
  }
  PS_TRY(check_optional(a->d_dgate, a->dgate_pitch, rows, cols, es));
  PS_TRY(check_optional(a->d_dup, a->dup_pitch, rows, cols, es));
  PS_TRY(check_kept(a->d_dgate_codes, a->dgate_codes_pitch, a->d_dgate_scales, rows, cols));
  PS_TRY(check_kept(a->d_dup_codes, a->dup_codes_pitch, a->d_dup_scales, rows, cols));
  PS_TRY(check_kept(a->d_dgate_codes_t, a->dgate_codes_t_pitch, a->d_dgate_scales_t, cols, rows));
  PS_TRY(check_kept(a->d_dup_codes_t, a->dup_codes_t_pitch, a->d_dup_scales_t, cols, rows));
  PS_TRY(check_kept(a->d_y_codes_t, a->y_codes_t_pitch, a->d_y_scales_t, cols, rows));
  const bool dup = a->d_dup != nullptr || a->d_dup_codes != nullptr || a->d_dup_codes_t != nullptr;
  if (a->d_up == nullptr && dup) return OPT_EINVAL;
  if (!dup && a->d_dgate == nullptr && a->d_dgate_codes == nullptr && a->d_dgate_codes_t == nullptr && a->d_y_codes_t == nullptr)
    return OPT_EINVAL;
  PS_TRY(check_tiles(rows, cols));
  int sms = 0;
  PS_TRY(sm_count_of(&sms));
  return status_of(launch_gated_backward(*a, sms, static_cast<cudaStream_t>(stream)));
}

int opt_head_norm(const opt_head_norm_args* a, void* stream) {
  if (a == nullptr) return OPT_EINVAL;
  PS_TRY(check_heads(*a));
  if (a->rows == 0 || a->q_heads + a->k_heads == 0) return OPT_OK;
  const int64_t es = plain_size(a->dtype), ws = plain_size(a->weight_dtype);
  if (a->q_heads > 0) {
    const int64_t cols = a->q_heads * a->dim;
    PS_TRY(check_matrix(a->d_q, a->q_pitch, a->rows, cols, es));
    PS_TRY(check_matrix(a->d_q_weight, a->dim, 1, a->dim, ws));
    PS_TRY(check_matrix(a->d_q_out, a->q_out_pitch, a->rows, cols, es));
    PS_TRY(check_kept(a->d_q_codes, a->q_codes_pitch, a->d_q_scales, a->rows, cols));
    PS_TRY(check_tiles(a->rows, cols));
  }
  if (a->k_heads > 0) {
    const int64_t cols = a->k_heads * a->dim;
    PS_TRY(check_matrix(a->d_k, a->k_pitch, a->rows, cols, es));
    PS_TRY(check_matrix(a->d_k_weight, a->dim, 1, a->dim, ws));
    PS_TRY(check_matrix(a->d_k_out, a->k_out_pitch, a->rows, cols, es));
    PS_TRY(check_kept(a->d_k_codes, a->k_codes_pitch, a->d_k_scales, a->rows, cols));
    PS_TRY(check_tiles(a->rows, cols));
  }
  PS_TRY(check_turn(*a));
  int sms = 0;
  PS_TRY(sm_count_of(&sms));
  return status_of(launch_head_norm(*a, sms, static_cast<cudaStream_t>(stream)));
}

int64_t opt_head_norm_backward_workspace(int64_t rows, int64_t q_heads, int64_t k_heads, int64_t dim) {
  PS_TRY(check_sizes(rows, dim));
  PS_TRY(check_sizes(q_heads, k_heads));
  if (dim < 1) return OPT_EINVAL;
  if (dim > kHeadMaxDim || q_heads * dim > kMaxDim || k_heads * dim > kMaxDim) return OPT_ELIMIT;
  return head_backward_parts(rows, q_heads + k_heads) * 2 * dim * (int64_t)sizeof(float);
}

int opt_head_norm_backward(const opt_head_norm_backward_args* a, void* stream) {
  if (a == nullptr) return OPT_EINVAL;
  PS_TRY(check_heads(*a));
  const int64_t es = plain_size(a->dtype), ws = plain_size(a->weight_dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float *dq = a->d_dq_weight, *dk = a->d_dk_weight;
  if (dq != nullptr) PS_TRY(check_matrix(dq, a->dim, 1, a->dim, 4));
  if (dk != nullptr) PS_TRY(check_matrix(dk, a->dim, 1, a->dim, 4));
  const bool q_side = a->rows > 0 && a->q_heads > 0, k_side = a->rows > 0 && a->k_heads > 0;
  if (q_side && k_side && (a->d_q_scales != nullptr) != (a->d_k_scales != nullptr)) return OPT_EINVAL;
  if (q_side) {
    const int64_t cols = a->q_heads * a->dim;
    PS_TRY(check_matrix(a->d_dq_out, a->dq_out_pitch, a->rows, cols, es));
    if (a->d_q_scales != nullptr) PS_TRY(check_codes(a->d_q, a->q_pitch, a->d_q_scales, a->rows, cols));
    else PS_TRY(check_matrix(a->d_q, a->q_pitch, a->rows, cols, es));
    PS_TRY(check_matrix(a->d_q_weight, a->dim, 1, a->dim, ws));
    PS_TRY(check_matrix(a->d_dq, a->dq_pitch, a->rows, cols, es));
  }
  if (k_side) {
    const int64_t cols = a->k_heads * a->dim;
    PS_TRY(check_matrix(a->d_dk_out, a->dk_out_pitch, a->rows, cols, es));
    if (a->d_k_scales != nullptr) PS_TRY(check_codes(a->d_k, a->k_pitch, a->d_k_scales, a->rows, cols));
    else PS_TRY(check_matrix(a->d_k, a->k_pitch, a->rows, cols, es));
    PS_TRY(check_matrix(a->d_k_weight, a->dim, 1, a->dim, ws));
    PS_TRY(check_matrix(a->d_dk, a->dk_pitch, a->rows, cols, es));
  }
  if (q_side || k_side) PS_TRY(check_turn(*a));
  const bool sums = (q_side && dq != nullptr) || (k_side && dk != nullptr);
  if (sums) {
    if (a->d_workspace == nullptr ||
        a->workspace_bytes < opt_head_norm_backward_workspace(a->rows, a->q_heads, a->k_heads, a->dim)) return OPT_EINVAL;
    if ((uintptr_t)a->d_workspace & 15u) return OPT_EALIGN;
  }
  opt_head_norm_backward_args b = *a;
  if (!q_side) {      // no rows or no heads: a sum of nothing
    if (dq != nullptr) PS_TRY(status_of(cudaMemsetAsync(dq, 0, (size_t)a->dim * sizeof(float), s)));
    b.d_dq_weight = nullptr;
    b.d_q_scales = nullptr;
  }
  if (!k_side) {
    if (dk != nullptr) PS_TRY(status_of(cudaMemsetAsync(dk, 0, (size_t)a->dim * sizeof(float), s)));
    b.d_dk_weight = nullptr;
    b.d_k_scales = nullptr;
  }
  if (!q_side && !k_side) return OPT_OK;
  int sms = 0;
  PS_TRY(sm_count_of(&sms));
  return status_of(launch_head_norm_backward(b, sms, s));
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
