// dropout.cu -- y = residual + dropout(x) (opt_layer.h).
//
// Mathematics: Philox4x32-10 gives eight 16-bit draws per call, and the mask is
// recomputed wherever it is needed, so a pass moves x, the residual and y and
// nothing else.
//
// Bound by memory once a matrix is large: 16384 x 4096 BF16 with a residual takes
// 63.7 us, 6.3 TB/s (0.95 of the measured copy), at 186 instructions per eight
// elements (issue 64 % busy).  One thread per chunk and fresh CTAs, not a resident
// grid; six CTAs per SM (32 registers): with the ragged end's code in the same
// path it took 70 registers and 112 us.  One token of 4,096 takes a launch's time
// (1.8 us back to back).  Strided rows that begin anywhere take two generator calls
// per chunk and go through shared memory: 8000 x 4001 BF16 60.4 us (0.48), with the
// matrix's ragged end loaded element by element in a loop (together: 63.0, 4000 x 3001
// 27.0 for 25.7; but 33 x 769 2.4 for 2.65).
#include "layer.cuh"

namespace psopt {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxGridX = (int64_t)1 << 30;

template <typename T, bool VEC>
__device__ __forceinline__ void drop_chunk(const opt_dropout_args& a, const DropArgs& d, int64_t r, int64_t c,
                                           int valid, T* buffer) {
  const auto row = [&](const void* base, int64_t pitch) {
    const T* m = static_cast<const T*>(base);
    return Row<T, VEC>(m + r * pitch, m, m + (a.rows - 1) * pitch + a.cols);
  };
  const Row<T, VEC> x_row = row(a.d_x, a.x_pitch), res_row = row(a.d_residual, a.residual_pitch);
  const int res_valid = a.d_residual != nullptr ? valid : 0;
  const Ahead<T, VEC> x_ahead = x_row.ahead(c, valid);
  Ahead<T, VEC> res_ahead = {};
  if (!VEC || res_valid > 0) res_ahead = res_row.ahead(c, res_valid);
  float x[8], y[8];
  unpack(x_row.template chunk<true>(x_ahead, c, valid), x);
  unpack(res_row.template chunk<true>(res_ahead, c, res_valid), y);
  add_dropped8<VEC>(y, x, (uint64_t)(r * a.cols + c), d, nullptr);      // (a barrier for a CTA's one row costs more)
  store_at<VEC>(a.d_y, a.y_pitch, a.cols, r, c, valid, y, buffer);
}
// A matrix's ragged end, element by element, so that it adds nothing to the main
// path's registers; chunks of a VEC matrix start on a generator call.
template <typename T>
__device__ __forceinline__ void drop_end(const opt_dropout_args& a, const DropArgs& d, int64_t r, int64_t c, int valid) {
  const uint4 w = drop_group((uint64_t)(r * a.cols + c) >> 3, d);
#pragma unroll 1
  for (int j = 0; j < valid; ++j) {
    const uint32_t word = j < 2 ? w.x : j < 4 ? w.y : j < 6 ? w.z : w.w;
    const uint32_t draw = (word >> (16 * (j & 1))) & 0xFFFFu;
    const T* res = static_cast<const T*>(a.d_residual);
    float x[8], y[8] = {};
    load8<false>(static_cast<const T*>(a.d_x) + r * a.x_pitch + c + j, 1, x);
    if (res != nullptr) load8<false>(res + r * a.residual_pitch + c + j, 1, y);
    if (draw >= d.threshold) y[0] = fmaf(x[0], d.factor, y[0]);
    store8<false>(static_cast<T*>(a.d_y) + r * a.y_pitch + c + j, 1, y);
  }
}

// One chunk of eight elements per thread; chunk `c` of row `r` starts at 8 c.
// A contiguous matrix comes as one row.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, VEC ? 6 : 5)
dropout_kernel(const __grid_constant__ opt_dropout_args a, const __grid_constant__ DropArgs d, int64_t first) {
  __shared__ __align__(16) Ragged<T, VEC, kThreads / 32> ragged;
  const int64_t c = 8 * (first + (int64_t)blockIdx.x * kThreads + threadIdx.x);
  if ((VEC ? c : c - 8 * (int)(threadIdx.x & 31)) >= a.cols) return;      // not VEC: whole warps only
  const int valid = (int)max(min(a.cols - c, (int64_t)8), (int64_t)0);
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    if constexpr (VEC) {
      if (valid == 8) drop_chunk<T, true>(a, d, r, c, 8, ragged.of_warp());
      else drop_end<T>(a, d, r, c, valid);
    } else {
      drop_chunk<T, false>(a, d, r, c, valid, ragged.of_warp());
    }
  }
}

template <typename T>
cudaError_t launch(opt_dropout_args a, const DropArgs& d, cudaStream_t s) {
  const bool res = a.d_residual != nullptr;
  if (a.rows > 1 && a.x_pitch == a.cols && a.y_pitch == a.cols && (!res || a.residual_pitch == a.cols)) {
    a.cols *= a.rows;              // one long row: the same element numbers
    a.rows = 1;
  }
  // VEC: every full chunk starts on 16 bytes and, in element numbers, on a
  // multiple of 8 (so that it is one generator call)
  constexpr int64_t es = sizeof(T);
  const auto fits = [&](const void* p, int64_t pitch) {
    return ((uintptr_t)p & 15u) == 0 && (a.rows == 1 || pitch * es % 16 == 0);
  };
  const bool vec = fits(a.d_x, a.x_pitch) && fits(a.d_y, a.y_pitch) && (!res || fits(a.d_residual, a.residual_pitch)) &&
                   (a.rows == 1 || a.cols % 8 == 0);
  const int64_t blocks = ((a.cols + 7) / 8 + kThreads - 1) / kThreads;
  const unsigned gy = (unsigned)(a.rows < 65535 ? a.rows : 65535);
  for (int64_t b = 0; b < blocks; b += kMaxGridX) {
    const dim3 grid((unsigned)(blocks - b < kMaxGridX ? blocks - b : kMaxGridX), gy);
    if (vec) dropout_kernel<T, true><<<grid, kThreads, 0, s>>>(a, d, b * kThreads);
    else dropout_kernel<T, false><<<grid, kThreads, 0, s>>>(a, d, b * kThreads);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dropout(const opt_dropout_args& a, const DropArgs& d, cudaStream_t s) {
  return a.dtype == OPT_F32 ? launch<float>(a, d, s) : launch<Bf16>(a, d, s);
}

}  // namespace psopt
