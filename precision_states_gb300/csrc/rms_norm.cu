// rms_norm.cu -- branch dropout, residual sum, root-mean-square norm and 8-bit
// output, and their gradients (opt_layer.h).
//
// Mathematics: each row needs one sum (of h^2, or of g h) before any output, so
// a row's data stay in registers from the one load to the stores.  A row is
// taken by a CTA (by one warp, eight rows per CTA, up to 256 columns), each
// thread holding NG chunks of eight elements; a CTA goes through many rows, so
// that the weight (and the weight's gradient) stay in registers too, and the
// next row's loads are issued before the current row's sum is complete.  Rows
// too wide for that (over 16,384 columns) take a second form that reads them twice.
//
// Sums over a row, rstd and the weight's gradient are fp32 throughout; outputs are
// rounded once.
//
// Forward, 16384 x 4096 BF16 with a residual to h and codes: 72.3 us without
// dropout, 6.5 TB/s (0.97 of the measured copy), bound by memory; 89.2 us with it
// (0.79), bound by the generator's integer work (267 instructions per eight
// elements, issue 65 % busy).  Two chunks per thread at 256 threads and three CTAs
// per SM: one chunk at 512 threads took 98.3 us, four at 128 threads 108.7, four
// CTAs per SM 87.1 (but 79.7 without dropout).  Backward, 8192 x 4096 BF16 with
// dh_in, dropout and the weight's gradient: 57.7 us (0.87), of which the sum over
// the CTAs' rows takes 4; one chunk per thread at 512 threads and two CTAs per SM
// (fp32 too, in spite of some spilled registers: 8000 x 4096 120.5 us, 162.6 with one).  Few rows are launches'
// latency: one token of 4,096 2.6 us.  Rows that begin anywhere (odd widths and pitches) are
// loaded by words and stored through shared memory: 8000 x 4001 BF16 to y 49.1 us
// (94.8 element by element), the backward pass 109 (271), bound by its instructions
// (issue 70 % busy).  4853 x 7001 takes 97.3 us with one CTA of 14 warps per SM: issue
// 50 % and DRAM 28 % busy, so latency at low occupancy.  Backward with narrow rows is a
// CTA of one warp each (131072 x 128 BF16 114 us, 0.13).
#include "layer.cuh"

namespace psopt {
namespace {

constexpr int kWideThreads = 512;       // of the form that reads rows twice
constexpr int kDweightCols = 32, kDweightParts = 32, kSlabCols = 16, kSlabFewRows = 8;

// Chunk c (eight elements) of row r of h = residual + dropout(x).
template <typename T, bool VEC>
__device__ __forceinline__ void h_chunk(const opt_rms_norm_args& a, const DropArgs& d, int64_t r, int64_t c,
                                        int valid, const Ahead<T, VEC>& x_ahead, const Ahead<T, VEC>& res_ahead,
                                        const uint4* edge, float (&h)[8]) {
  float x[8];
  unpack(Row<T, VEC>(a.d_x, a.x_pitch, a.rows, a.cols, r).chunk(x_ahead, c, valid), x);
  unpack(Row<T, VEC>(a.d_residual, a.residual_pitch, a.rows, a.cols, r)
             .chunk(res_ahead, c, a.d_residual != nullptr ? valid : 0), h);
  add_dropped8<VEC>(h, x, (uint64_t)(r * a.cols + c), d, edge);
}
template <typename T, bool VEC>
__device__ __forceinline__ void load_chunk(const opt_rms_norm_args& a, int64_t r, int64_t c, int valid,
                                           Ahead<T, VEC>& x, Ahead<T, VEC>& res) {
  x = Row<T, VEC>(a.d_x, a.x_pitch, a.rows, a.cols, r).ahead(c, valid);
  if (a.d_residual != nullptr) res = Row<T, VEC>(a.d_residual, a.residual_pitch, a.rows, a.cols, r).ahead(c, valid);
}

// Everything that is written of a chunk, by whole warps; chunks beyond the row
// come with valid <= 0.
template <typename T, bool VEC>
__device__ __forceinline__ void write_chunk(const opt_rms_norm_args& a, int64_t r, int64_t c, int valid, float rstd,
                                            int64_t panel, const float (&h)[8], const float (&w)[8], T* buffer) {
  float y[8];
  scaled8(h, rstd, y);
  times8(y, w);
  if (!VEC || valid > 0) {
    if (a.d_h != nullptr) store_at<VEC>(a.d_h, a.h_pitch, a.cols, r, c, valid, h, buffer);
    if (a.d_y != nullptr) store_at<VEC>(a.d_y, a.y_pitch, a.cols, r, c, valid, y, buffer);
  }
  if (a.d_codes == nullptr) return;
  if (valid < 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = j < valid ? y[j] : 0.0f;
  }
  bool odd;
  const uint32_t byte = block_byte(y, odd);
  if (valid > 0) {
    store_codes8(static_cast<uint8_t*>(a.d_codes) + r * a.codes_pitch + c, valid, codes8(y, inverse_scale(byte), odd));
    if ((threadIdx.x & 15) == 0) static_cast<uint8_t*>(a.d_scales)[scale_place(r, c >> 7, panel)] = (uint8_t)byte;
  }
}

// Rows in registers: a row per warp (BY_WARP), or per CTA; thread t of a row holds
// chunks t + k (threads of the row) for k < NG.
template <typename T, typename W, bool VEC, bool BY_WARP, int NG, int MAX, int CTAS>
__global__ void __launch_bounds__(MAX, CTAS) rms_norm_kernel(const __grid_constant__ opt_rms_norm_args a,
                                                             const __grid_constant__ DropArgs d) {
  __shared__ float part[2][33];
  __shared__ __align__(16) Ragged<T, VEC, MAX / 32> ragged;
  __shared__ __align__(16) Edges<VEC || BY_WARP, NG * (MAX / 32)> edges;
  const int in_row = BY_WARP ? (int)(threadIdx.x & 31) : (int)threadIdx.x, of_row = BY_WARP ? 32 : (int)blockDim.x;
  const int64_t row0 = BY_WARP ? (int64_t)blockIdx.x * (MAX / 32) + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t row_step = BY_WARP ? (int64_t)gridDim.x * (MAX / 32) : gridDim.x;
  const int64_t panel = (a.cols + 511) / 512;
  const int cols = (int)a.cols;
  const float inv_cols = 1.0f / (float)cols;
  const auto column = [&](int k) { return 8 * (in_row + k * of_row); };
  const auto valid = [&](int k) { return VEC ? (column(k) < cols ? 8 : 0) : max(min(cols - column(k), 8), 0); };
  const Row<W, VEC> weight(a.d_weight, 0, 1, a.cols, 0);
  float w[NG][8];
  Ahead<T, VEC> x[NG] = {}, res[NG] = {};
  Ahead<W, VEC> w_ahead[NG] = {};
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    if (VEC && valid(k) <= 0) continue;
    if (row0 < a.rows) load_chunk<T, VEC>(a, row0, column(k), valid(k), x[k], res[k]);
    w_ahead[k] = weight.ahead(column(k), valid(k));
  }
#pragma unroll
  for (int k = 0; k < NG; ++k) unpack(weight.chunk(w_ahead[k], column(k), valid(k)), w[k]);
  if (!VEC && !BY_WARP) {
    edges.put(0, (uint64_t)(row0 * a.cols), NG, d);
    __syncthreads();
  }
  int turn = 0;
  for (int64_t r = row0; r < a.rows; r += row_step, turn ^= 1) {
    float h[NG][8];
    f2_t sums = 0;                    // +0 in both lanes
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      h_chunk<T, VEC>(a, d, r, column(k), valid(k), x[k], res[k], BY_WARP ? nullptr : edges.of_warp(turn, k), h[k]);
      // the next row, while this one's sum is formed
      if ((!VEC || valid(k) > 0) && r + row_step < a.rows)
        load_chunk<T, VEC>(a, r + row_step, column(k), valid(k), x[k], res[k]);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const f2_t v = pk(h[k][j], h[k][j + 1]);
        sums = fma2(v, v, sums);
      }
    }
    float sum, second;
    unpk(sums, sum, second);
    if (!VEC && !BY_WARP && r + row_step < a.rows) edges.put(turn ^ 1, (uint64_t)((r + row_step) * a.cols), NG, d);
    sum = cta_sum(sum + second, part[turn], BY_WARP ? 1 : of_row >> 5);
    const float rstd = reciprocal_root(fmaf(sum, inv_cols, a.eps));
    if (in_row == 0 && a.d_rstd != nullptr) a.d_rstd[r] = rstd;
#pragma unroll
    for (int k = 0; k < NG; ++k) write_chunk<T, VEC>(a, r, column(k), valid(k), rstd, panel, h[k], w[k], ragged.of_warp());
  }
}

// Wide rows: a pass for the sum of squares, a second one that forms h again
// (the row is still in L2) and writes.
template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(kWideThreads) rms_norm_wide_kernel(const __grid_constant__ opt_rms_norm_args a,
                                                                     const __grid_constant__ DropArgs d) {
  __shared__ float part[2][33];
  __shared__ __align__(16) Ragged<T, VEC, kWideThreads / 32> ragged;
  const int64_t panel = (a.cols + 511) / 512;
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, turn ^= 1) {
    float sum = 0.0f, h[8], w[8];
    Ahead<T, VEC> x, res = {};
    const Row<W, VEC> weight(a.d_weight, 0, 1, a.cols, 0);
    for (int64_t c = 8 * threadIdx.x; c < a.cols; c += 8 * kWideThreads) {
      const int valid = (int)min(a.cols - c, (int64_t)8);
      load_chunk<T, VEC>(a, r, c, valid, x, res);
      h_chunk<T, VEC>(a, d, r, c, valid, x, res, nullptr, h);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(h[j], h[j], sum);
    }
    sum = cta_sum(sum, part[turn], kWideThreads / 32);
    const float rstd = reciprocal_root(fmaf(sum, 1.0f / (float)a.cols, a.eps));
    if (threadIdx.x == 0 && a.d_rstd != nullptr) a.d_rstd[r] = rstd;
    for (int64_t c0 = 0; c0 < a.cols; c0 += 8 * kWideThreads) {
      const int64_t c = c0 + 8 * threadIdx.x;
      const int valid = (int)max(min(a.cols - c, (int64_t)8), (int64_t)0);
      if (valid > 0) {
        load_chunk<T, VEC>(a, r, c, valid, x, res);
        h_chunk<T, VEC>(a, d, r, c, valid, x, res, nullptr, h);
        unpack(weight.chunk(weight.ahead(c, valid), c, valid), w);
      }
      write_chunk<T, VEC>(a, r, c, valid, rstd, panel, h, w, ragged.of_warp());
    }
  }
}

// ------------------------------------------------------------------ gradients
// What is written of a chunk of the gradients, by whole warps: dh and dx from g =
// dy weight.
template <typename T, bool VEC>
__device__ __forceinline__ void write_gradients(const opt_rms_norm_backward_args& a, const DropArgs& d, int64_t r,
                                                int64_t c, int valid, float rstd, float k, const float (&g)[8],
                                                const float (&h)[8], const float (&in)[8], T* buffer,
                                                const uint4* edge) {
  float out[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) out[j] = fmaf(rstd, fmaf(-h[j], k, g[j]), in[j]);
  store_at<VEC>(a.d_dh, a.dh_pitch, a.cols, r, c, valid, out, buffer);
  if (a.d_dx != nullptr) {
    float dx[8] = {};
    add_dropped8<VEC>(dx, out, (uint64_t)(r * a.cols + c), d, edge);
    store_at<VEC>(a.d_dx, a.dx_pitch, a.cols, r, c, valid, dx, buffer);
  }
}

// This CTA's (or, with a row per warp, this warp's) row of partial sums.
__device__ __forceinline__ float* dweight_row(const opt_rms_norm_backward_args& a, int64_t part) {
  return static_cast<float*>(a.d_workspace) + part * ((a.cols + 3) / 4 * 4);
}

__host__ __device__ __forceinline__ bool dweight_here(const opt_rms_norm_backward_args& a) {
  return norm_backward_parts(a.rows, a.cols) == 0;
}

// dweight needs no row's sum, so few rows' is formed from dy, h and rstd again (they
// are in L2) by CTAs of the same launch: no second launch, no workspace.  (Where dh
// takes dy's place they run in a launch of their own, before.)  CTA `slab` takes
// 16 columns; its half-warps share the rows in turn, and their sums are added in
// order.  Up to eight rows: a column to each thread (1 x 16384 BF16 5.1 us; 8.3 with
// 16 to a CTA, seven waves of them).
template <typename T>
__device__ __forceinline__ void dweight_slab(const opt_rms_norm_backward_args& a, int slab) {
  __shared__ float sums[32][kSlabCols];
  if (a.rows <= kSlabFewRows) {
    const int64_t c = (int64_t)slab * blockDim.x + threadIdx.x;
    if (c >= a.cols) return;
    const T* dy = static_cast<const T*>(a.d_dy) + c;
    const T* h = static_cast<const T*>(a.d_h) + c;
    uint32_t g[kSlabFewRows], v[kSlabFewRows], scale[kSlabFewRows];
#pragma unroll
    for (int r = 0; r < kSlabFewRows; ++r) {
      g[r] = bits_if(dy + r * a.dy_pitch, r < a.rows);
      v[r] = bits_if(h + r * a.h_pitch, r < a.rows);
      scale[r] = bits_if(a.d_rstd + r, r < a.rows);
    }
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < kSlabFewRows; ++r) s = fmaf(u2f(g[r]), u2f(v[r]) * u2f(scale[r]), s);
    a.d_dweight[c] = s;
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t c = (int64_t)slab * kSlabCols + (lane & (kSlabCols - 1));
  float s = 0.0f;
  if (c < a.cols) {
    const T* dy = static_cast<const T*>(a.d_dy) + c;
    const T* h = static_cast<const T*>(a.d_h) + c;
    const int rows = (int)a.rows;
    const int of = 2 * warps;
    for (int r0 = 2 * warp + (lane >> 4); r0 < rows; r0 += 8 * of) {      // eight rows' loads together
      uint32_t g[8], v[8], scale[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = r0 + k * of;
        g[k] = bits_if(dy + r * a.dy_pitch, r < rows);
        v[k] = bits_if(h + r * a.h_pitch, r < rows);
        scale[k] = bits_if(a.d_rstd + r, r < rows);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s = fmaf(u2f(g[k]), u2f(v[k]) * u2f(scale[k]), s);
    }
  }
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
  if (lane < kSlabCols) sums[warp][lane] = s;
  __syncthreads();
  if (threadIdx.x >= kSlabCols || c >= a.cols) return;
  for (int w = 1; w < warps; ++w) s += sums[w][lane];
  a.d_dweight[c] = s;
}

// CTAs from `row_ctas` on are dweight's slabs.  At 1,024 threads the
// registers hold neither the weight nor the next row (AHEAD false).
template <typename T, typename W, bool VEC, int NG, int MAX, int CTAS>
__global__ void __launch_bounds__(MAX, CTAS) rms_norm_backward_kernel(
    const __grid_constant__ opt_rms_norm_backward_args a, const __grid_constant__ DropArgs d, int row_ctas) {
  __shared__ float part[2][33];
  __shared__ __align__(16) Ragged<T, VEC, MAX / 32> ragged;
  __shared__ __align__(16) Edges<VEC, NG * (MAX / 32)> edges;
  if ((int)blockIdx.x >= row_ctas) {
    dweight_slab<T>(a, (int)blockIdx.x - row_ctas);
    return;
  }
  const int warps = blockDim.x >> 5;
  const float inv_cols = 1.0f / (float)a.cols;
  const int cols = (int)a.cols;
  const auto column = [&](int k) { return 8 * (int)(threadIdx.x + k * blockDim.x); };
  const auto valid = [&](int k) { return VEC ? (column(k) < cols ? 8 : 0) : max(min(cols - column(k), 8), 0); };
  float dw[NG][8] = {};
  const Row<W, VEC> weight(a.d_weight, 0, 1, a.cols, 0);
  const auto dy_row = [&](int64_t r) { return Row<T, VEC>(a.d_dy, a.dy_pitch, a.rows, a.cols, r); };
  const auto h_row = [&](int64_t r) { return Row<T, VEC>(a.d_h, a.h_pitch, a.rows, a.cols, r); };
  const auto in_row = [&](int64_t r) { return Row<T, VEC>(a.d_dh_in, a.dh_in_pitch, a.rows, a.cols, r); };
  Ahead<W, VEC> w[NG] = {};
  Ahead<T, VEC> dy[NG] = {}, h[NG] = {}, in[NG] = {};
  constexpr bool AHEAD = MAX < 1024;
  const auto load = [&](int k, int64_t r) {
    dy[k] = dy_row(r).ahead(column(k), valid(k));
    h[k] = h_row(r).ahead(column(k), valid(k));
  };
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    if (AHEAD && (!VEC || valid(k) > 0)) {
      load(k, blockIdx.x);
      w[k] = weight.ahead(column(k), valid(k));
    }
  }
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += row_ctas, turn ^= 1) {
    const float rstd = a.d_rstd[r];
    float g[NG][8], hv[NG][8], sum = 0.0f;
    if (!AHEAD) {
#pragma unroll
      for (int k = 0; k < NG; ++k) {
        dy[k] = h[k] = {};          // nothing of the row before to be kept
        w[k] = {};
        if (VEC && valid(k) <= 0) continue;
        load(k, r);
        w[k] = weight.ahead(column(k), valid(k));
      }
    }
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      float wv[8];
      unpack(dy_row(r).chunk(dy[k], column(k), valid(k)), g[k]);
      unpack(h_row(r).chunk(h[k], column(k), valid(k)), hv[k]);
      unpack(weight.chunk(w[k], column(k), valid(k)), wv);
      if (AHEAD && a.d_dh_in != nullptr && (!VEC || valid(k) > 0)) in[k] = in_row(r).ahead(column(k), valid(k));
      if (AHEAD && (!VEC || valid(k) > 0) && r + row_ctas < a.rows) load(k, r + row_ctas);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[k][j] = fmaf(g[k][j], hv[k][j] * rstd, dw[k][j]);
        g[k][j] *= wv[j];
        sum = fmaf(g[k][j], hv[k][j], sum);
      }
    }
    if (!VEC && a.d_dx != nullptr) {
      edges.put(turn, (uint64_t)(r * a.cols), NG, d);
      if (warps == 1) __syncwarp();
    }
    sum = cta_sum(sum, part[turn], warps);
    const float scale = rstd * rstd * (sum * inv_cols);
#pragma unroll
    for (int k = 0; k < NG; ++k)
      if (!VEC || valid(k) > 0) {
        float add[8];
        if (!AHEAD) in[k] = {};
        if (!AHEAD && a.d_dh_in != nullptr) in[k] = in_row(r).ahead(column(k), valid(k));
        unpack(in_row(r).chunk(in[k], column(k), a.d_dh_in != nullptr ? valid(k) : 0), add);
        write_gradients<T, VEC>(a, d, r, column(k), valid(k), rstd, scale, g[k], hv[k], add, ragged.of_warp(),
                                edges.of_warp(turn, k));
      }
  }
  if (a.d_dweight != nullptr && !dweight_here(a)) {
    float* out = dweight_row(a, blockIdx.x);
#pragma unroll
    for (int k = 0; k < NG; ++k)
      if (valid(k) > 0) {
        if (valid(k) == 8) {
          *reinterpret_cast<float4*>(out + column(k)) = make_float4(dw[k][0], dw[k][1], dw[k][2], dw[k][3]);
          *reinterpret_cast<float4*>(out + column(k) + 4) = make_float4(dw[k][4], dw[k][5], dw[k][6], dw[k][7]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < valid(k)) out[column(k) + j] = dw[k][j];
        }
      }
  }
}

// Wide rows, read twice; each column of the partial sums belongs to one thread.
template <typename T, typename W, bool VEC>
__global__ void __launch_bounds__(kWideThreads) rms_norm_backward_wide_kernel(
    const __grid_constant__ opt_rms_norm_backward_args a, const __grid_constant__ DropArgs d, int row_ctas) {
  __shared__ float part[2][33];
  __shared__ __align__(16) Ragged<T, VEC, kWideThreads / 32> ragged;
  if ((int)blockIdx.x >= row_ctas) {
    dweight_slab<T>(a, (int)blockIdx.x - row_ctas);
    return;
  }
  float* dw = a.d_dweight == nullptr || dweight_here(a) ? nullptr : dweight_row(a, blockIdx.x);
  const Row<W, VEC> weight(a.d_weight, 0, 1, a.cols, 0);
  const auto dy_row = [&](int64_t r) { return Row<T, VEC>(a.d_dy, a.dy_pitch, a.rows, a.cols, r); };
  const auto h_row = [&](int64_t r) { return Row<T, VEC>(a.d_h, a.h_pitch, a.rows, a.cols, r); };
  const auto in_row = [&](int64_t r) { return Row<T, VEC>(a.d_dh_in, a.dh_in_pitch, a.rows, a.cols, r); };
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.rows; r += row_ctas, turn ^= 1) {
    const auto load = [&](int64_t c, int valid, float (&g)[8], float (&h)[8], float (&w)[8]) {
      const Ahead<T, VEC> g_ahead = dy_row(r).ahead(c, valid), h_ahead = h_row(r).ahead(c, valid);
      const Ahead<W, VEC> w_ahead = weight.ahead(c, valid);
      unpack(dy_row(r).chunk(g_ahead, c, valid), g);
      unpack(h_row(r).chunk(h_ahead, c, valid), h);
      unpack(weight.chunk(w_ahead, c, valid), w);
    };
    float sum = 0.0f;
    for (int64_t c = 8 * threadIdx.x; c < a.cols; c += 8 * kWideThreads) {
      float g[8], h[8], w[8];
      load(c, (int)min(a.cols - c, (int64_t)8), g, h, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(g[j] * w[j], h[j], sum);
    }
    sum = cta_sum(sum, part[turn], kWideThreads / 32);
    const float rstd = a.d_rstd[r];
    const float k = rstd * rstd * (sum / (float)a.cols);
    for (int64_t c0 = 0; c0 < a.cols; c0 += 8 * kWideThreads) {
      const int64_t c = c0 + 8 * threadIdx.x;
      const int valid = (int)max(min(a.cols - c, (int64_t)8), (int64_t)0);
      float g[8] = {}, h[8] = {}, w[8] = {}, in[8] = {};
      if (valid > 0) {
        load(c, valid, g, h, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (dw != nullptr && j < valid)
            dw[c + j] = fmaf(g[j], h[j] * rstd, r == (int64_t)blockIdx.x ? 0.0f : dw[c + j]);
          g[j] *= w[j];
        }
        if (a.d_dh_in != nullptr)
          unpack(in_row(r).chunk(in_row(r).ahead(c, valid), c, valid), in);
      }
      if (!VEC || valid > 0) write_gradients<T, VEC>(a, d, r, c, valid, rstd, k, g, h, in, ragged.of_warp(), nullptr);
    }
  }
}

// dweight = the sum over the workspace's `n` rows in a fixed order: a CTA takes
// 32 columns, thread row p the partial sums p, p + 32, ..., and the 32 thread
// rows are added in order.
__global__ void __launch_bounds__(kDweightCols * kDweightParts) dweight_kernel(const float* __restrict__ parts, int n,
                                                                               int64_t cols, float* __restrict__ out) {
  __shared__ float sums[kDweightParts][kDweightCols + 1];
  const int x = threadIdx.x % kDweightCols, p0 = threadIdx.x / kDweightCols;
  const int64_t c = (int64_t)blockIdx.x * kDweightCols + x, pitch = (cols + 3) / 4 * 4;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 4
    for (int p = p0; p < n; p += kDweightParts) s += parts[p * pitch + c];
  }
  sums[p0][x] = s;
  __syncthreads();
  if (p0 != 0 || c >= cols) return;
#pragma unroll
  for (int p = 1; p < kDweightParts; ++p) s += sums[p][x];
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

template <typename T, typename W, bool VEC, bool BY_WARP, int NG, int MAX, int CTAS>
cudaError_t forward_rows(const opt_rms_norm_args& a, const DropArgs& d, int sm_count, int threads, cudaStream_t s) {
  static OccupancyCache cache[33];
  const auto kernel = rms_norm_kernel<T, W, VEC, BY_WARP, NG, MAX, CTAS>;
  const int64_t rows_per_cta = BY_WARP ? MAX / 32 : 1, need = (a.rows + rows_per_cta - 1) / rows_per_cta;
  const int64_t most = (int64_t)sm_count * cached_occupancy(kernel, cache[threads / 32], threads, 0);
  kernel<<<(unsigned)(need < most ? need : most), threads, 0, s>>>(a, d);
  return cudaGetLastError();
}

template <typename T, typename W, bool VEC>
cudaError_t forward_vec(const opt_rms_norm_args& a, const DropArgs& d, int sm_count, cudaStream_t s) {
  const int64_t chunks = (a.cols + 7) / 8;
  const int threads = (int)((chunks + 31) / 32) * 32;
  if (chunks <= 32) return forward_rows<T, W, VEC, true, 1, 256, 3>(a, d, sm_count, 256, s);
  if (chunks <= 256) return forward_rows<T, W, VEC, false, 1, 256, 4>(a, d, sm_count, threads, s);
  if (chunks <= 512) return forward_rows<T, W, VEC, false, 2, 256, 3>(a, d, sm_count, (int)((chunks + 63) / 64) * 32, s);
  if (chunks <= 1024) return forward_rows<T, W, VEC, false, 2, 512, 1>(a, d, sm_count, (int)((chunks + 63) / 64) * 32, s);
  // BF16: two chunks of 1,024 threads (4853 x 12440 80.9 us, four of 512 90.7; without
  // whole chunks, 12435, 203.7 and 267.6); fp32's registers want the latter (161.5, 167.1)
  if (chunks <= 2048) {
    if constexpr (sizeof(T) == 2)
      return forward_rows<T, W, VEC, false, 2, 1024, 1>(a, d, sm_count, (int)((chunks + 63) / 64) * 32, s);
    else
      return forward_rows<T, W, VEC, false, 4, 512, 1>(a, d, sm_count, (int)((chunks + 127) / 128) * 32, s);
  }
  const int64_t most = (int64_t)sm_count * 4;
  rms_norm_wide_kernel<T, W, VEC><<<(unsigned)(a.rows < most ? a.rows : most), kWideThreads, 0, s>>>(a, d);
  return cudaGetLastError();
}

template <typename T, typename W>
cudaError_t forward(const opt_rms_norm_args& a, const DropArgs& d, int sm_count, cudaStream_t s) {
  VecRule v{a.rows, a.cols, a.cols % 8 == 0};
  v.see(a.d_x, a.x_pitch, sizeof(T));
  v.see(a.d_residual, a.residual_pitch, sizeof(T));
  v.see(a.d_weight, 0, sizeof(W));
  v.see(a.d_h, a.h_pitch, sizeof(T));
  v.see(a.d_y, a.y_pitch, sizeof(T));
  return v.ok ? forward_vec<T, W, true>(a, d, sm_count, s) : forward_vec<T, W, false>(a, d, sm_count, s);
}

// CTAs of dweight's slabs, in the launch of the rows.
unsigned slabs(const opt_rms_norm_backward_args& a, int threads) {
  const int64_t cols = a.rows <= kSlabFewRows ? threads : kSlabCols;
  return a.d_dweight != nullptr && dweight_here(a) ? (unsigned)((a.cols + cols - 1) / cols) : 0u;
}

template <typename K>
void launch_backward(K kernel, const opt_rms_norm_backward_args& a, const DropArgs& d, int grid, int threads,
                     cudaStream_t s) {
  const unsigned n = slabs(a, threads);
  const bool apart = n > 0 && a.d_dh == a.d_dy;
  if (apart) kernel<<<n, threads, 0, s>>>(a, d, 0);
  kernel<<<grid + (apart ? 0u : n), threads, 0, s>>>(a, d, grid);
}

// CTAs that go through the rows, of `resident` that the device holds at once: each has
// a row of partial sums, and the workspace has room for kNormBackwardMaxCtas.
constexpr int64_t row_ctas(int64_t rows, int64_t resident) {
  const int64_t most = resident < kNormBackwardMaxCtas ? resident : kNormBackwardMaxCtas;
  return rows < most ? rows : most;
}
static_assert(row_ctas(1 << 20, 4 * 400) <= norm_backward_parts(1 << 20, 20000), "the workspace holds every CTA's row");
static_assert(row_ctas(600, 4 * 400) <= norm_backward_parts(600, 20000), "the workspace holds every CTA's row");

template <typename T, typename W, bool VEC, int NG, int MAX, int CTAS>
int backward_rows(const opt_rms_norm_backward_args& a, const DropArgs& d, int sm_count, int threads, cudaStream_t s) {
  static OccupancyCache cache[33];
  const auto kernel = rms_norm_backward_kernel<T, W, VEC, NG, MAX, CTAS>;
  if (slabs(a, MAX) > 0 && a.rows > kSlabFewRows) threads = MAX;      // dweight's rows are shared by all warps
  const int grid = (int)row_ctas(a.rows, (int64_t)sm_count * cached_occupancy(kernel, cache[threads / 32], threads, 0));
  launch_backward(kernel, a, d, grid, threads, s);
  return grid;
}

template <typename T, typename W, bool VEC>
cudaError_t backward_vec(const opt_rms_norm_backward_args& a, const DropArgs& d, int sm_count, cudaStream_t s) {
  const int64_t chunks = (a.cols + 7) / 8;
  int grid;
  if (chunks <= 512) {
    grid = backward_rows<T, W, VEC, 1, 512, 2>(a, d, sm_count, (int)((chunks + 31) / 32) * 32, s);
  } else if (chunks <= 1024) {
    grid = backward_rows<T, W, VEC, 2, 512, 1>(a, d, sm_count, (int)((chunks + 63) / 64) * 32, s);
  } else if (chunks <= 2048) {
    grid = backward_rows<T, W, VEC, 2, 1024, 1>(a, d, sm_count, (int)((chunks + 63) / 64) * 32, s);
  } else {
    grid = (int)row_ctas(a.rows, (int64_t)sm_count * 4);
    launch_backward(rms_norm_backward_wide_kernel<T, W, VEC>, a, d, grid, kWideThreads, s);
  }
  if (a.d_dweight != nullptr && !dweight_here(a))
    dweight_kernel<<<(unsigned)((a.cols + kDweightCols - 1) / kDweightCols), kDweightCols * kDweightParts, 0, s>>>(
        static_cast<const float*>(a.d_workspace), grid, a.cols, a.d_dweight);
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
  return v.ok ? backward_vec<T, W, true>(a, d, sm_count, s) : backward_vec<T, W, false>(a, d, sm_count, s);
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
