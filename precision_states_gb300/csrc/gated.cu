// gated.cu -- y = f(gate) up between two products, its inputs kept in 8 bits, and
// its gradients in the forms that the next products take (opt_layer.h).
//
// Mathematics: f(g) = g s(g).  With e = exp(-|z|) the logistic function of z is
// 1 / (1 + e) or e / (1 + e), and its complement the other of the two, so neither
// overflows or cancels; f' = s + g s (1 - s) z'.
#include "tile.cuh"

namespace psopt {
namespace {

constexpr int kThreads = 256;
constexpr float kTwoRootTwoOverPi = 1.5957691216057308f, kCubic = 0.044715f, kLog2e = 1.4426950408889634f;

// exp(-a) for a >= 0.  EXACT: to fp32 (for fp32 elements); else by the exponential
// of two, whose argument's rounding costs a 2^-24 of the result, far below BF16's
// and E4M3's steps.
template <bool EXACT>
__device__ __forceinline__ float exp_minus(float a) {
  if constexpr (EXACT) return expf(-a);
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(a * -kLog2e));
  return r;
}

// f(g) and, if it is wanted, f'(g).
template <bool EXACT, bool SLOPE>
__device__ __forceinline__ void activation(int kind, float g, float& f, float& df) {
  if (kind == OPT_ACT_RELU) {
    const float on = g == g ? 0.0f : g;
    f = g > 0.0f ? g : on;
    df = g > 0.0f ? 1.0f : on;
    return;
  }
  if (kind == OPT_ACT_GELU) {
    const float s = normcdff(g);
    f = g * s;
    if (SLOPE) df = fmaf(g, 0.3989422804014327f * exp_minus<EXACT>(0.5f * g * g), s);
    return;
  }
  float z = g, dz = 1.0f;
  if (kind == OPT_ACT_GELU_TANH) {
    const float b = fminf(fmaxf(g, -16.0f), 16.0f);      // s is 0 or 1 beyond, and its slope 0
    z = kTwoRootTwoOverPi * fmaf(kCubic * b * b, b, b);
    dz = kTwoRootTwoOverPi * fmaf(3.0f * kCubic * b, b, 1.0f);
  }
  const float e = exp_minus<EXACT>(fabsf(z));
  const float r = EXACT ? __frcp_rn(1.0f + e) : rcp_approx(1.0f + e);
  const float er = e * r, s = z < 0.0f ? er : r;
  f = g * s;
  if (SLOPE) df = fmaf(f * (z < 0.0f ? r : er), dz, s);
}

template <bool EXACT, bool SLOPE>
__device__ __forceinline__ void activation8(int kind, const float (&g)[8], float (&f)[8], float (&df)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) activation<EXACT, SLOPE>(kind, g[j], f[j], df[j]);
}

// Where a thread stands that takes a chunk of a row: blocks of blockDim.x chunks (whole
// warps) by blockDim.y rows.
__device__ __forceinline__ int64_t first_row() { return (int64_t)blockIdx.y * blockDim.y + threadIdx.y; }
__device__ __forceinline__ int warp_of_block() { return (int)(threadIdx.y * blockDim.x + threadIdx.x) >> 5; }

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) gated_kernel(const __grid_constant__ opt_gated_args a) {
  __shared__ __align__(16) Ragged<T, VEC, kThreads / 32> ragged;
  T* buffer = ragged.chunk[VEC ? 0 : warp_of_block()];
  const int64_t c = 8 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x), panel = (a.cols + 511) / 512;
  const int valid = (int)max(min(a.cols - c, (int64_t)8), (int64_t)0);
  for (int64_t r = first_row(); r < a.rows; r += (int64_t)gridDim.y * blockDim.y) {
    const Source<T, VEC> gate(a.d_gate, nullptr, a.gate_pitch, a.rows, a.cols, r);
    const Source<T, VEC> up(a.d_up, nullptr, a.up_pitch, a.rows, a.cols, r);
    const bool has_up = a.d_up != nullptr;
    Ahead<T, VEC> ga = {}, ua = {};
    if (!VEC || valid > 0) {
      ga = gate.ahead(c, valid);
      if (has_up) ua = up.ahead(c, valid);
    }
    float g[8], u[8], y[8], unused[8];
    gate.values(ga, c, valid, g);
    activation8<sizeof(T) == 4, false>(a.activation, g, y, unused);
    if (has_up) {
      up.values(ua, c, valid, u);
      times8(y, u);
    }
    if (a.d_y != nullptr && (!VEC || valid > 0)) store_at<VEC>(a.d_y, a.y_pitch, a.cols, r, c, valid, y, buffer);
    if (a.d_codes != nullptr) put_codes8(a.d_codes, a.d_scales, a.codes_pitch, panel, r, c, valid, y);
    if (a.d_gate_codes != nullptr) put_codes8(a.d_gate_codes, a.d_gate_scales, a.gate_codes_pitch, panel, r, c, valid, g);
    if (a.d_up_codes != nullptr) put_codes8(a.d_up_codes, a.d_up_scales, a.up_codes_pitch, panel, r, c, valid, u);
  }
}

// ------------------------------------------------------------------ gradients
// Without transposed outputs: a chunk to a thread, as above.
template <typename T, typename S, bool VEC>
__global__ void __launch_bounds__(kThreads) gated_backward_kernel(const __grid_constant__ opt_gated_backward_args a) {
  __shared__ __align__(16) Ragged<T, VEC, kThreads / 32> ragged;
  T* buffer = ragged.chunk[VEC ? 0 : warp_of_block()];
  const int64_t c = 8 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x), panel = (a.cols + 511) / 512;
  const int valid = (int)max(min(a.cols - c, (int64_t)8), (int64_t)0);
  for (int64_t r = first_row(); r < a.rows; r += (int64_t)gridDim.y * blockDim.y) {
    const Source<T, VEC> dy(a.d_dy, nullptr, a.dy_pitch, a.rows, a.cols, r);
    const Source<S, VEC> gate(a.d_gate, a.d_gate_scales, a.gate_pitch, a.rows, a.cols, r);
    const Source<S, VEC> up(a.d_up, a.d_up_scales, a.up_pitch, a.rows, a.cols, r);
    const bool has_up = a.d_up != nullptr;
    Ahead<T, VEC> da = {};
    typename Source<S, VEC>::Ask ga = {}, ua = {};
    if (!VEC || valid > 0) {
      da = dy.ahead(c, valid);
      ga = gate.ahead(c, valid);
      if (has_up) ua = up.ahead(c, valid);
    }
    float d[8], g[8], u[8], f[8], df[8];
    gate.values(ga, c, valid, g);
    activation8<sizeof(T) == 4, true>(a.activation, g, f, df);
    dy.values(da, c, valid, d);
    times8(f, d);
    times8(df, d);
    if (has_up) {
      up.values(ua, c, valid, u);
      times8(df, u);
    }
    if (!VEC || valid > 0) {
      if (a.d_dgate != nullptr) store_at<VEC>(a.d_dgate, a.dgate_pitch, a.cols, r, c, valid, df, buffer);
      if (a.d_dup != nullptr) store_at<VEC>(a.d_dup, a.dup_pitch, a.cols, r, c, valid, f, buffer);
    }
    if (a.d_dgate_codes != nullptr)
      put_codes8(a.d_dgate_codes, a.d_dgate_scales, a.dgate_codes_pitch, panel, r, c, valid, df);
    if (a.d_dup_codes != nullptr) put_codes8(a.d_dup_codes, a.d_dup_scales, a.dup_codes_pitch, panel, r, c, valid, f);
  }
}

// With transposed outputs: a 128 x 128 tile to a CTA.  Matrix by matrix (dgate, dup, y)
// the square is formed from the inputs, its rows' codes are written, and it is turned;
// plain outputs come last, so that they may take an input's place.
template <typename T, typename S, bool VEC>
__global__ void __launch_bounds__(kTileThreads) gated_backward_tile_kernel(
    const __grid_constant__ opt_gated_backward_args a, int64_t col_tiles) {
  __shared__ TileTurn sh;
  const int64_t r0 = 128 * (blockIdx.x / col_tiles), c0 = 128 * (blockIdx.x % col_tiles);
  const int rows = (int)min(a.rows - r0, (int64_t)128), cols = (int)min(a.cols - c0, (int64_t)128);
  const int square = threadIdx.x & 15, band = threadIdx.x >> 4, l = 8 * band;
  const int64_t c = c0 + 8 * square, panel = (a.cols + 511) / 512, panel_t = (a.rows + 511) / 512;
  const bool has_up = a.d_up != nullptr;
  // row l + i of matrix m
  const auto form = [&](int m, int i, float (&x)[8]) {
    const int valid = l + i < rows ? max(min(cols - 8 * square, 8), 0) : 0;
    const int64_t r = r0 + (valid > 0 ? l + i : 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    if (valid == 0) return;
    float d[8], g[8], u[8], f[8], df[8];
    const Source<T, VEC> dy(a.d_dy, nullptr, a.dy_pitch, a.rows, a.cols, r);
    const Source<S, VEC> gate(a.d_gate, a.d_gate_scales, a.gate_pitch, a.rows, a.cols, r);
    const Source<S, VEC> up(a.d_up, a.d_up_scales, a.up_pitch, a.rows, a.cols, r);
    gate.values(gate.ahead(c, valid), c, valid, g);
    activation8<sizeof(T) == 4, true>(a.activation, g, f, df);
    if (m != 2) {
      dy.values(dy.ahead(c, valid), c, valid, d);
      times8(f, d);
      times8(df, d);
    }
    if (m != 1 && has_up) {
      up.values(up.ahead(c, valid), c, valid, u);
      times8(f, u);
      times8(df, u);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = j < valid ? (m == 0 ? df[j] : f[j]) : 0.0f;
  };
#pragma unroll 1
  for (int m = 0; m < 3; ++m) {
    void* codes = m == 0 ? a.d_dgate_codes : m == 1 ? a.d_dup_codes : nullptr;
    void* scales = m == 0 ? a.d_dgate_scales : a.d_dup_scales;
    const int64_t pitch = m == 0 ? a.dgate_codes_pitch : a.dup_codes_pitch;
    void* codes_t = m == 0 ? a.d_dgate_codes_t : m == 1 ? a.d_dup_codes_t : a.d_y_codes_t;
    void* scales_t = m == 0 ? a.d_dgate_scales_t : m == 1 ? a.d_dup_scales_t : a.d_y_scales_t;
    const int64_t pitch_t = m == 0 ? a.dgate_codes_t_pitch : m == 1 ? a.dup_codes_t_pitch : a.y_codes_t_pitch;
    if (codes == nullptr && codes_t == nullptr) continue;
    Raw<float> x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[8];
      form(m, i, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i].w[j] = f2u(v[j]);
      if (codes != nullptr)
        put_codes8(codes, scales, pitch, panel, r0 + l + i, c, l + i < rows ? min(cols - 8 * square, 8) : 0, v);
    }
    if (codes_t == nullptr) continue;
    turn_square(x, sh, r0, c0, cols, static_cast<uint8_t*>(scales_t), panel_t);
    __syncthreads();
    store_turned(sh, static_cast<uint8_t*>(codes_t), pitch_t, r0, c0, rows, cols);
    __syncthreads();
  }
  if (a.d_dgate == nullptr && a.d_dup == nullptr) return;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const int valid = l + i < rows ? max(min(cols - 8 * square, 8), 0) : 0;
    float x[8], v[8];
    if (a.d_dgate != nullptr) form(0, i, x);
    if (a.d_dup != nullptr) form(1, i, v);
    __syncwarp();                 // an output may lie in an input's place, of which lanes read their neighbours' words
    if (valid == 0) continue;
    if (a.d_dgate != nullptr) store8<VEC>(static_cast<T*>(a.d_dgate) + (r0 + l + i) * a.dgate_pitch + c, valid, x);
    if (a.d_dup != nullptr) store8<VEC>(static_cast<T*>(a.d_dup) + (r0 + l + i) * a.dup_pitch + c, valid, v);
  }
}

// Whole chunks that start on 16 bytes in every plain matrix.
struct VecRule {
  int64_t rows, es;
  bool ok;
  void see(const void* p, int64_t pitch) {
    ok = ok && (p == nullptr || (((uintptr_t)p & 15u) == 0 && (rows == 1 || pitch * es % 16 == 0)));
  }
};

template <typename T>
cudaError_t forward(const opt_gated_args& a, cudaStream_t s) {
  VecRule v{a.rows, sizeof(T), a.cols % 8 == 0};
  v.see(a.d_gate, a.gate_pitch);
  v.see(a.d_up, a.up_pitch);
  v.see(a.d_y, a.y_pitch);
  const ChunkGrid g(a.rows, a.cols, kThreads);
  if (v.ok) gated_kernel<T, true><<<g.grid, g.block, 0, s>>>(a);
  else gated_kernel<T, false><<<g.grid, g.block, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, typename S, bool VEC>
cudaError_t backward_vec(const opt_gated_backward_args& a, cudaStream_t s) {
  if (a.d_dgate_codes_t == nullptr && a.d_dup_codes_t == nullptr && a.d_y_codes_t == nullptr) {
    const ChunkGrid g(a.rows, a.cols, kThreads);
    gated_backward_kernel<T, S, VEC><<<g.grid, g.block, 0, s>>>(a);
  } else {
    const int64_t col_tiles = (a.cols + 127) / 128;
    gated_backward_tile_kernel<T, S, VEC><<<(unsigned)((a.rows + 127) / 128 * col_tiles), kTileThreads, 0, s>>>(a, col_tiles);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t backward(const opt_gated_backward_args& a, cudaStream_t s) {
  const bool kept = a.d_gate_scales != nullptr;
  VecRule v{a.rows, sizeof(T), a.cols % 8 == 0};
  v.see(a.d_dy, a.dy_pitch);
  v.see(kept ? nullptr : a.d_gate, a.gate_pitch);
  v.see(kept ? nullptr : a.d_up, a.up_pitch);
  v.see(a.d_dgate, a.dgate_pitch);
  v.see(a.d_dup, a.dup_pitch);
  if (kept) return v.ok ? backward_vec<T, E4m3, true>(a, s) : backward_vec<T, E4m3, false>(a, s);
  return v.ok ? backward_vec<T, T, true>(a, s) : backward_vec<T, T, false>(a, s);
}

}  // namespace

cudaError_t launch_gated(const opt_gated_args& a, cudaStream_t s) {
  return a.dtype == OPT_F32 ? forward<float>(a, s) : forward<Bf16>(a, s);
}

cudaError_t launch_gated_backward(const opt_gated_backward_args& a, cudaStream_t s) {
  return a.dtype == OPT_F32 ? backward<float>(a, s) : backward<Bf16>(a, s);
}

}  // namespace psopt
