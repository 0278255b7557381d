// gated.cu -- y = f(gate) up between two products, its inputs kept in 8 bits, and
// its gradients in the forms that the next products take (opt_layer.h).
//
// Mathematics: f(g) = g s(g), f' = s + g s (1 - s) z' where s is the logistic function of
// z(g).
#include "tile.cuh"

namespace psopt {
namespace {

constexpr int kThreads = 256;
constexpr float kTwoRootTwoOverPi = 1.5957691216057308f, kCubic = 0.044715f, kLog2e = 1.4426950408889634f;

// exp(-a) for a >= 0 to fp32 (for fp32 elements).
__device__ __forceinline__ float exp_minus(float a) { return expf(-a); }
// 2^a: two units in the last place, besides the rounding of what is given as a.
__device__ __forceinline__ float exp2_near(float a) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(a));
  return r;
}

// f(g) and, if it is wanted (SLOPE), f'(g).  EXACT: for fp32 elements, to their last
// places; else s = 1 / (1 + 2^(-z log2 e)), whose errors of a few 2^-24 are far below BF16's
// and E4M3's steps (and which is 0 where it would be below 2^-128), two at a time.
template <int KIND, bool EXACT, bool SLOPE>
__device__ __forceinline__ void activation(float g, float& f, float& df) {
  if constexpr (KIND == OPT_ACT_RELU) {
    const float on = g == g ? 0.0f : g;
    f = g > 0.0f ? g : on;
    df = g > 0.0f ? 1.0f : on;
  } else if constexpr (KIND == OPT_ACT_GELU) {
    const float s = normcdff(g);
    f = g * s;
    if (SLOPE) df = fmaf(g, 0.3989422804014327f * (EXACT ? exp_minus(0.5f * g * g) : exp2_near(-0.5f * kLog2e * g * g)), s);
  } else {
    float z = g, dz = 1.0f;
    if (KIND == OPT_ACT_GELU_TANH) {
      const float b = fminf(fmaxf(g, -16.0f), 16.0f);      // s is 0 or 1 beyond, and its slope 0
      z = kTwoRootTwoOverPi * fmaf(kCubic * b * b, b, b);
      dz = kTwoRootTwoOverPi * fmaf(3.0f * kCubic * b, b, 1.0f);
    }
    // of s and 1 - s one is r and the other e r: neither overflows nor cancels
    const float e = exp_minus(fabsf(z)), r = __frcp_rn(1.0f + e), er = e * r, s = z < 0.0f ? er : r;
    f = g * s;
    if (SLOPE) df = fmaf(f * (z < 0.0f ? r : er), dz, s);
  }
}
template <int KIND, bool EXACT, bool SLOPE>
__device__ __forceinline__ void activation8(const float (&g)[8], float (&f)[8], float (&df)[8]) {
  if constexpr (EXACT || KIND == OPT_ACT_RELU || KIND == OPT_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < 8; ++j) activation<KIND, EXACT, SLOPE>(g[j], f[j], df[j]);
  } else {
    const f2_t one = pk(1.0f, 1.0f);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const f2_t gv = pk(g[j], g[j + 1]);
      f2_t z, dz = one;                                     // z: times -log2 e
      if constexpr (KIND == OPT_ACT_SILU) {
        z = mul2(gv, pk(-kLog2e, -kLog2e));
      } else {
        const f2_t b = pk(fminf(fmaxf(g[j], -16.0f), 16.0f), fminf(fmaxf(g[j + 1], -16.0f), 16.0f)), bb = mul2(b, b);
        constexpr float c = -kLog2e * kTwoRootTwoOverPi;
        z = mul2(mul2(b, pk(c, c)), fma2(bb, pk(kCubic, kCubic), one));
        dz = fma2(bb, pk(3.0f * kCubic * kTwoRootTwoOverPi, 3.0f * kCubic * kTwoRootTwoOverPi), pk(kTwoRootTwoOverPi, kTwoRootTwoOverPi));
      }
      float lo, hi;
      unpk(z, lo, hi);
      unpk(add2(pk(exp2_near(lo), exp2_near(hi)), one), lo, hi);
      const f2_t s = pk(rcp_approx(lo), rcp_approx(hi)), fv = mul2(gv, s);
      unpk(fv, f[j], f[j + 1]);
      if constexpr (SLOPE) {
        f2_t n = fma2(s, pk(-1.0f, -1.0f), one);
        if constexpr (KIND == OPT_ACT_GELU_TANH) n = mul2(n, dz);
        unpk(fma2(fv, n, s), df[j], df[j + 1]);
      }
    }
  }
}

// Where a thread stands that takes a chunk of a row: blocks of blockDim.x chunks (whole
// warps) by blockDim.y rows.
__device__ __forceinline__ int64_t first_row() { return (int64_t)blockIdx.y * blockDim.y + threadIdx.y; }
__device__ __forceinline__ int warp_of_block() { return (int)(threadIdx.y * blockDim.x + threadIdx.x) >> 5; }

// The largest magnitudes of two 1 x 128 blocks that 16 lanes hold chunks of, by whole warps:
// BF16's go through the exchanges together.
__device__ __forceinline__ void tops16(uint32_t& a, uint32_t& b, Bf16) {
  uint32_t both = a | b >> 16;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) both = larger(both, __shfl_xor_sync(0xFFFFFFFFu, both, o), Bf16());
  a = both & 0xFFFF0000u;
  b = both << 16;
}
__device__ __forceinline__ void tops16(uint32_t& a, uint32_t& b, float) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
    b = max(b, __shfl_xor_sync(0xFFFFFFFFu, b, o));
  }
}

template <typename T, int KIND, bool VEC>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && VEC ? 5 : 4) gated_kernel(const __grid_constant__ opt_gated_args a) {
  __shared__ __align__(16) Ragged<T, VEC, kThreads / 32> ragged;
  T* buffer = ragged.chunk[VEC ? 0 : warp_of_block()];
  const int64_t c = 8 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x), panel = (a.cols + 511) / 512;
  const int valid = (int)max(min(a.cols - c, (int64_t)8), (int64_t)0);
  const bool has_up = a.d_up != nullptr;
  for (int64_t r = first_row(); r < a.rows; r += (int64_t)gridDim.y * blockDim.y) {
    const Row<T, VEC> gate(a.d_gate, a.gate_pitch, a.rows, a.cols, r), up(a.d_up, a.up_pitch, a.rows, a.cols, r);
    Ahead<T, VEC> ga = {}, ua = {};
    if (!VEC || valid > 0) {
      ga = gate.ahead(c, valid);
      if (has_up) ua = up.ahead(c, valid);
    }
    const Raw<T> graw = gate.chunk(ga, c, valid), uraw = up.chunk(ua, c, has_up ? valid : 0);
    float g[8], u[8], y[8], unused[8];
    unpack(graw, g);
    activation8<KIND, sizeof(T) == 4, false>(g, y, unused);
    unpack(uraw, u);
    if (has_up) times8(y, u);
    if (a.d_y != nullptr && (!VEC || valid > 0)) store_at<VEC>(a.d_y, a.y_pitch, a.cols, r, c, valid, y, buffer);
    if (a.d_codes == nullptr && a.d_gate_codes == nullptr && a.d_up_codes == nullptr) continue;
    uint32_t top = 0, gtop = 0, utop = 0;
    if (a.d_codes != nullptr) top = top16(top8_of(y));
    if (a.d_gate_codes != nullptr || a.d_up_codes != nullptr) {
      gtop = top_of(magnitudes(graw, false));
      utop = top_of(magnitudes(uraw, false));
      tops16(gtop, utop, T());
    }
    const int64_t at = scale_place(r, c >> 7, panel);
    uint8_t *codes = static_cast<uint8_t*>(a.d_codes) + r * a.codes_pitch + c, *scales = static_cast<uint8_t*>(a.d_scales);
    uint8_t *gcodes = static_cast<uint8_t*>(a.d_gate_codes) + r * a.gate_codes_pitch + c, *gscales = static_cast<uint8_t*>(a.d_gate_scales);
    uint8_t *ucodes = static_cast<uint8_t*>(a.d_up_codes) + r * a.up_codes_pitch + c, *uscales = static_cast<uint8_t*>(a.d_up_scales);
    if (__any_sync(0xFFFFFFFFu, max(max(top, gtop), utop) >= kInfBits)) {      // rare
      if (a.d_codes != nullptr) put_codes8(codes, scales, at, valid, y);
      if (a.d_gate_codes != nullptr) put_codes8(gcodes, gscales, at, valid, g);
      if (a.d_up_codes != nullptr) put_codes8(ucodes, uscales, at, valid, u);
    } else {
      if (a.d_codes != nullptr) put_finite8(codes, scales, at, valid, y, top);
      if (a.d_gate_codes != nullptr) put_finite8(gcodes, gscales, at, valid, g, gtop);
      if (a.d_up_codes != nullptr) put_finite8(ucodes, uscales, at, valid, u, utop);
    }
  }
}

// ------------------------------------------------------------------ gradients
// Without transposed outputs: a chunk to a thread, as above.
template <typename T, typename S, int KIND, bool VEC>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && VEC ? 4 : 3)
gated_backward_kernel(const __grid_constant__ opt_gated_backward_args a) {
  __shared__ __align__(16) Ragged<T, VEC, kThreads / 32> ragged;
  T* buffer = ragged.chunk[VEC ? 0 : warp_of_block()];
  const int64_t c = 8 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x), panel = (a.cols + 511) / 512;
  const int valid = (int)max(min(a.cols - c, (int64_t)8), (int64_t)0);
  const bool has_up = a.d_up != nullptr;
  for (int64_t r = first_row(); r < a.rows; r += (int64_t)gridDim.y * blockDim.y) {
    const Source<T, VEC> dy(a.d_dy, nullptr, a.dy_pitch, a.rows, a.cols, r);
    const Source<S, VEC> gate(a.d_gate, a.d_gate_scales, a.gate_pitch, a.rows, a.cols, r);
    const Source<S, VEC> up(a.d_up, a.d_up_scales, a.up_pitch, a.rows, a.cols, r);
    Ahead<T, VEC> da = {};
    typename Source<S, VEC>::Ask ga = {}, ua = {};
    if (!VEC || valid > 0) {
      da = dy.ahead(c, valid);
      ga = gate.ahead(c, valid);
      if (has_up) ua = up.ahead(c, valid);
    }
    float d[8], g[8], u[8], f[8], df[8];
    gate.values(ga, c, valid, g);
    activation8<KIND, sizeof(T) == 4, true>(g, f, df);
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
    const int64_t at = scale_place(r, c >> 7, panel);
    if (a.d_dgate_codes != nullptr)
      put_codes8(static_cast<uint8_t*>(a.d_dgate_codes) + r * a.dgate_codes_pitch + c, static_cast<uint8_t*>(a.d_dgate_scales), at,
                 valid, df);
    if (a.d_dup_codes != nullptr)
      put_codes8(static_cast<uint8_t*>(a.d_dup_codes) + r * a.dup_codes_pitch + c, static_cast<uint8_t*>(a.d_dup_scales), at, valid, f);
  }
}

// With transposed outputs: CTAs of 1,024 threads go through tiles of 128 x 128.  First each
// thread forms two rows' chunks of dgate, dup and y, writes what goes by rows, and leaves
// the values in shared memory; then a warp takes four columns of each matrix (a lane four
// rows of them), finds the columns' maxima among its own lanes, and writes the columns'
// codes in whole lines.  The next tile's loads are under way meanwhile.
constexpr int kTurnThreads = 1024, kTile = 128 * 128;
constexpr int kTurnBytes = 3 * kTile * (int)sizeof(float);

// Place of the four columns from 4 quad on of a tile's row, in units of four values: turned so
// that neither a row's chunks nor a column's rows meet in one bank.
__device__ __forceinline__ int turned_place(int row, int quad) { return 32 * row + (quad ^ (row >> 2)); }

// A tile's values at `v` by columns: four columns of 128 rows to a warp.
__device__ __forceinline__ void put_columns(const float4* v, uint8_t* codes, uint8_t* scales, int64_t pitch, int64_t panel,
                                            int64_t r0, int64_t c0, int rows, int cols) {
  const int lane = threadIdx.x & 31, quad = threadIdx.x >> 5;
  float x[4][4];                    // [row][column]
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 t = v[turned_place(4 * lane + i, quad)];
    x[i][0] = t.x; x[i][1] = t.y; x[i][2] = t.z; x[i][3] = t.w;
  }
  uint32_t top[4], all = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    top[j] = __reduce_max_sync(0xFFFFFFFFu, f2u(largest3(largest3(x[0][j], x[1][j], x[2][j]), x[3][j], x[3][j])));
    all = max(all, top[j]);
  }
  if (all >= kInfBits) {            // rare: the finite ones' maxima, and NaN for the others
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t t = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (finite_bits(x[i][j])) t = max(t, magnitude(x[i][j]));
        else x[i][j] = u2f(0x7FC00000u);
      }
      top[j] = __reduce_max_sync(0xFFFFFFFFu, t);
    }
  }
  uint32_t byte[4], word[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) byte[j] = scale_byte(top[j]);
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const f2_t inv = pk(inverse_scale(byte[j]), inverse_scale(byte[j + 1]));
#pragma unroll
    for (int i = 0; i < 4; ++i) unpk(mul2(pk(x[i][j], x[i][j + 1]), inv), x[i][j], x[i][j + 1]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) word[j] = e4m3x2_rn(x[0][j], x[1][j]) | e4m3x2_rn(x[2][j], x[3][j]) << 16;
  uint8_t* p = codes + (c0 + 4 * quad) * pitch + r0 + 4 * lane;
  const int left = rows - 4 * lane;
#pragma unroll
  for (int j = 0; j < 4; ++j, p += pitch) {
    if (4 * quad + j >= cols) break;
    if (left >= 4) {
      st_cs_u1(p, word[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < left) p[i] = (uint8_t)(word[j] >> (8 * i));
    }
  }
  if (lane < 4 && 4 * quad + lane < cols)
    scales[scale_place(c0 + 4 * quad + lane, r0 >> 7, panel)] = (uint8_t)(lane == 0 ? byte[0] : lane == 1 ? byte[1] : lane == 2 ? byte[2] : byte[3]);
}

template <typename T, typename S, bool VEC>
struct Inputs {
  Ahead<T, VEC> dy;
  typename Source<S, VEC>::Ask gate, up;
};

template <typename T, typename S, int KIND, bool VEC>
__global__ void __launch_bounds__(kTurnThreads, 1) gated_backward_tile_kernel(
    const __grid_constant__ opt_gated_backward_args a, int64_t col_tiles, int64_t tiles) {
  extern __shared__ __align__(16) float4 held[];       // dgate, dup, y
  // plain fp32 inputs of two rows leave no registers for the next tile's
  constexpr bool AHEAD = sizeof(T) == 2 || sizeof(typename Source<S, VEC>::Ask) < 32;
  const int q = threadIdx.x & 15, row = 2 * (threadIdx.x >> 4);
  const int64_t panel = (a.cols + 511) / 512, panel_t = (a.rows + 511) / 512;
  const bool has_up = a.d_up != nullptr;
  const auto valid_of = [&](int64_t r, int64_t c) { return r < a.rows ? (int)max(min(a.cols - c, (int64_t)8), (int64_t)0) : 0; };
  const auto load = [&](int64_t tile, int i) {
    Inputs<T, S, VEC> in = {};
    const int64_t r = 128 * (tile / col_tiles) + row + i, c = 128 * (tile % col_tiles) + 8 * q;
    const int valid = valid_of(r, c);
    if (valid > 0) {
      in.dy = Source<T, VEC>(a.d_dy, nullptr, a.dy_pitch, a.rows, a.cols, r).ahead(c, valid);
      in.gate = Source<S, VEC>(a.d_gate, a.d_gate_scales, a.gate_pitch, a.rows, a.cols, r).ahead(c, valid);
      if (has_up) in.up = Source<S, VEC>(a.d_up, a.d_up_scales, a.up_pitch, a.rows, a.cols, r).ahead(c, valid);
    }
    return in;
  };
  Inputs<T, S, VEC> in[2];
  if (AHEAD) {
#pragma unroll
    for (int i = 0; i < 2; ++i) in[i] = load(blockIdx.x, i);
  }
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t r0 = 128 * (tile / col_tiles), c0 = 128 * (tile % col_tiles), c = c0 + 8 * q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!AHEAD) in[i] = load(tile, i);
      const int64_t r = r0 + row + i;
      const int valid = valid_of(r, c);
      float d[8], g[8], u[8], f[8], df[8];
      Source<S, VEC>(a.d_gate, a.d_gate_scales, a.gate_pitch, a.rows, a.cols, r).values(in[i].gate, c, valid, g);
      activation8<KIND, sizeof(T) == 4, true>(g, f, df);
      Source<T, VEC>(a.d_dy, nullptr, a.dy_pitch, a.rows, a.cols, r).values(in[i].dy, c, valid, d);
      if (has_up) {
        Source<S, VEC>(a.d_up, a.d_up_scales, a.up_pitch, a.rows, a.cols, r).values(in[i].up, c, valid, u);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = 1.0f;
      }
      times8(df, d);
      times8(d, f);                 // dup
      times8(f, u);                 // y
      if (has_up) times8(df, u);    // dgate
      // to shared memory; half of a row's lanes store their second four first
      const auto leave = [&](int m, const float (&x)[8]) {
        float4* v = held + m * (kTile / 4);
        const float4 lo = make_float4(x[0], x[1], x[2], x[3]), hi = make_float4(x[4], x[5], x[6], x[7]);
        const bool other = (q & 4) != 0;
        v[turned_place(row + i, 2 * q + (other ? 1 : 0))] = other ? hi : lo;
        v[turned_place(row + i, 2 * q + (other ? 0 : 1))] = other ? lo : hi;
      };
      if (a.d_dgate_codes_t != nullptr) leave(0, df);
      if (a.d_dup_codes_t != nullptr) leave(1, d);
      if (a.d_y_codes_t != nullptr) leave(2, f);
      if (a.d_dgate_codes != nullptr || a.d_dup_codes != nullptr) {
        uint32_t gtop = top8_of(df), utop = top8_of(d);
        tops16(gtop, utop, 0.0f);
        const int64_t at = scale_place(r, c >> 7, panel);
        uint8_t *gcodes = static_cast<uint8_t*>(a.d_dgate_codes) + r * a.dgate_codes_pitch + c, *gscales = static_cast<uint8_t*>(a.d_dgate_scales);
        uint8_t *ucodes = static_cast<uint8_t*>(a.d_dup_codes) + r * a.dup_codes_pitch + c, *uscales = static_cast<uint8_t*>(a.d_dup_scales);
        if (__any_sync(0xFFFFFFFFu, max(gtop, utop) >= kInfBits)) {      // rare
          if (a.d_dgate_codes != nullptr) put_codes8(gcodes, gscales, at, valid, df);
          if (a.d_dup_codes != nullptr) put_codes8(ucodes, uscales, at, valid, d);
        } else {
          if (a.d_dgate_codes != nullptr) put_finite8(gcodes, gscales, at, valid, df, gtop);
          if (a.d_dup_codes != nullptr) put_finite8(ucodes, uscales, at, valid, d, utop);
        }
      }
      __syncwarp();                 // an output may lie in an input's place, of which lanes read their neighbours' words
      if (valid > 0) {
        if (a.d_dgate != nullptr) store8<VEC>(static_cast<T*>(a.d_dgate) + r * a.dgate_pitch + c, valid, df);
        if (a.d_dup != nullptr) store8<VEC>(static_cast<T*>(a.d_dup) + r * a.dup_pitch + c, valid, d);
      }
    }
    __syncthreads();
    if (AHEAD && tile + gridDim.x < tiles) {
#pragma unroll
      for (int i = 0; i < 2; ++i) in[i] = load(tile + gridDim.x, i);
    }
    const int rows = (int)min(a.rows - r0, (int64_t)128), cols = (int)min(a.cols - c0, (int64_t)128);
    if (a.d_dgate_codes_t != nullptr)
      put_columns(held, static_cast<uint8_t*>(a.d_dgate_codes_t), static_cast<uint8_t*>(a.d_dgate_scales_t), a.dgate_codes_t_pitch,
                  panel_t, r0, c0, rows, cols);
    if (a.d_dup_codes_t != nullptr)
      put_columns(held + kTile / 4, static_cast<uint8_t*>(a.d_dup_codes_t), static_cast<uint8_t*>(a.d_dup_scales_t), a.dup_codes_t_pitch,
                  panel_t, r0, c0, rows, cols);
    if (a.d_y_codes_t != nullptr)
      put_columns(held + kTile / 2, static_cast<uint8_t*>(a.d_y_codes_t), static_cast<uint8_t*>(a.d_y_scales_t), a.y_codes_t_pitch,
                  panel_t, r0, c0, rows, cols);
    __syncthreads();
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

template <typename T, int KIND>
cudaError_t forward_kind(const opt_gated_args& a, cudaStream_t s) {
  VecRule v{a.rows, sizeof(T), a.cols % 8 == 0};
  v.see(a.d_gate, a.gate_pitch);
  v.see(a.d_up, a.up_pitch);
  v.see(a.d_y, a.y_pitch);
  const ChunkGrid g(a.rows, a.cols, kThreads);
  if (v.ok) gated_kernel<T, KIND, true><<<g.grid, g.block, 0, s>>>(a);
  else gated_kernel<T, KIND, false><<<g.grid, g.block, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t forward(const opt_gated_args& a, cudaStream_t s) {
  switch (a.activation) {
    case OPT_ACT_SILU: return forward_kind<T, OPT_ACT_SILU>(a, s);
    case OPT_ACT_GELU_TANH: return forward_kind<T, OPT_ACT_GELU_TANH>(a, s);
    case OPT_ACT_GELU: return forward_kind<T, OPT_ACT_GELU>(a, s);
    default: return forward_kind<T, OPT_ACT_RELU>(a, s);
  }
}

template <typename T, typename S, int KIND, bool VEC>
cudaError_t backward_vec(const opt_gated_backward_args& a, int sm_count, cudaStream_t s) {
  if (a.d_dgate_codes_t == nullptr && a.d_dup_codes_t == nullptr && a.d_y_codes_t == nullptr) {
    const ChunkGrid g(a.rows, a.cols, kThreads);
    gated_backward_kernel<T, S, KIND, VEC><<<g.grid, g.block, 0, s>>>(a);
  } else {
    static OccupancyCache cache;
    const auto kernel = gated_backward_tile_kernel<T, S, KIND, VEC>;
    const int64_t col_tiles = (a.cols + 127) / 128, tiles = (a.rows + 127) / 128 * col_tiles;
    const int64_t most = (int64_t)sm_count * cached_occupancy(kernel, cache, kTurnThreads, kTurnBytes);
    kernel<<<(unsigned)(tiles < most ? tiles : most), kTurnThreads, kTurnBytes, s>>>(a, col_tiles, tiles);
  }
  return cudaGetLastError();
}

template <typename T, int KIND>
cudaError_t backward_kind(const opt_gated_backward_args& a, int sm_count, cudaStream_t s) {
  const bool kept = a.d_gate_scales != nullptr;
  VecRule v{a.rows, sizeof(T), a.cols % 8 == 0};
  v.see(a.d_dy, a.dy_pitch);
  v.see(kept ? nullptr : a.d_gate, a.gate_pitch);
  v.see(kept ? nullptr : a.d_up, a.up_pitch);
  v.see(a.d_dgate, a.dgate_pitch);
  v.see(a.d_dup, a.dup_pitch);
  if (kept) return v.ok ? backward_vec<T, E4m3, KIND, true>(a, sm_count, s) : backward_vec<T, E4m3, KIND, false>(a, sm_count, s);
  return v.ok ? backward_vec<T, T, KIND, true>(a, sm_count, s) : backward_vec<T, T, KIND, false>(a, sm_count, s);
}
template <typename T>
cudaError_t backward(const opt_gated_backward_args& a, int sm_count, cudaStream_t s) {
  switch (a.activation) {
    case OPT_ACT_SILU: return backward_kind<T, OPT_ACT_SILU>(a, sm_count, s);
    case OPT_ACT_GELU_TANH: return backward_kind<T, OPT_ACT_GELU_TANH>(a, sm_count, s);
    case OPT_ACT_GELU: return backward_kind<T, OPT_ACT_GELU>(a, sm_count, s);
    default: return backward_kind<T, OPT_ACT_RELU>(a, sm_count, s);
  }
}

}  // namespace

cudaError_t launch_gated(const opt_gated_args& a, cudaStream_t s) {
  return a.dtype == OPT_F32 ? forward<float>(a, s) : forward<Bf16>(a, s);
}

cudaError_t launch_gated_backward(const opt_gated_backward_args& a, int sm_count, cudaStream_t s) {
  return a.dtype == OPT_F32 ? backward<float>(a, sm_count, s) : backward<Bf16>(a, sm_count, s);
}

}  // namespace psopt
