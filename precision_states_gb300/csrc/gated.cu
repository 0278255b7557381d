// gated.cu -- y = f(gate) up between two products, its inputs kept in 8 bits, and
// its gradients in the forms that the next products take (opt_layer.h).
//
// Mathematics: f(g) = g s(g); f' = s + g s (1 - s) z' where s is the logistic function of
// z(g), and f' = s + g s' where it is the normal distribution function.
#include <type_traits>

#include "tile.cuh"

namespace psopt {
namespace {

constexpr int kThreads = 256;
constexpr float kTwoRootTwoOverPi = 1.5957691216057308f, kCubic = 0.044715f, kLog2e = 1.4426950408889634f;

// exp(-a) for a >= 0 to fp32 (for fp32 elements).
__device__ __forceinline__ float exp_minus(float a) { return expf(-a); }
// 2^a and 1 / a to two units in the last place; results below 2^-126 are 0 (keeping them
// takes nine more instructions per element).
__device__ __forceinline__ float exp2_near(float a) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
  return r;
}
__device__ __forceinline__ float reciprocal_near(float a) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
  return r;
}

// f(g) and, if it is wanted (SLOPE), f'(g).  EXACT: for fp32 elements, by fp32's exponential and a
// rounded reciprocal (8 units of 2^-24, and with the tanh form's z 6 |z| more: its roundings); else
// s = 1 / (1 + 2^(-z log2 e)), whose errors of a few 2^-24 (150 where s is near 2^-126) are far below
// BF16's and E4M3's steps (and which is 0 where it would be below 2^-126), two at a time.
template <int KIND, bool EXACT, bool SLOPE>
__device__ __forceinline__ void activation(float g, float& f, float& df) {
  if constexpr (KIND == OPT_ACT_RELU) {
    const float on = g == g ? 0.0f : g;
    f = g > 0.0f ? g : on;
    df = g > 0.0f ? 1.0f : on;
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
// The normal distribution function of two values, and exp(-g^2 / 2) (EXACT: scaled).  For a = |g|, s(-a) =
// exp(-a^2 / 2) R(a); R, a scaled complementary error function, by Hastings' way (Abramowitz and
// Stegun 7.1.26): a polynomial in t = 1 / (1 + 0.4 a), here of degree nine for R / t, fitted to
// equal relative errors over 0 <= a <= 16 (in fp32 5 units of 2^-24, 8 with a reciprocal that is
// one off) and exact at 0.  (8192 x 14336 BF16 to y 120 us, with the library's function 262.)
// EXACT: the exponential times 2^64 (kBellScale), which the polynomial's coefficients take back, so
// that s is kept down to fp32's last subnormal number; and with what its argument's rounding loses.
// (4096 x 14336 fp32 to codes, both kept, 107 us; with the exponential's own subnormal results
// 109, with 0 below 2^-126 106.)
template <bool EXACT>
constexpr float kBellScale = EXACT ? 18446744073709551616.0f : 1.0f;
template <bool EXACT>
__device__ __forceinline__ void normal2(f2_t g, f2_t& s, f2_t& bell) {
  constexpr float c[10] = {1.595754921e-01f, 1.596362293e-01f,  1.330585480e-01f, 9.175205231e-02f,  -2.814983390e-02f,
                           1.220970377e-01f, -3.773407638e-01f, 3.848911524e-01f, -1.779478639e-01f, 3.242795169e-02f};
  const f2_t one = pk(1.0f, 1.0f);
  float lo, hi;
  unpk(g, lo, hi);
  const f2_t a = pk(fminf(fabsf(lo), 16.0f), fminf(fabsf(hi), 16.0f));      // s(-a) is 0 in fp32 beyond
  float tl, th;
  unpk(fma2(a, pk(0.4f, 0.4f), one), tl, th);
  const f2_t t = pk(reciprocal_near(tl), reciprocal_near(th));
  constexpr float back = 1.0f / kBellScale<EXACT>;
  f2_t q = pk(c[9] * back, c[9] * back);
#pragma unroll
  for (int k = 8; k >= 0; --k) q = fma2(q, t, pk(c[k] * back, c[k] * back));
  constexpr float h = -0.5f * kLog2e, h_rest = (float)(-0.5 * 1.4426950408889634074 - (double)h), ln2 = 0.69314718f;
  const f2_t square = mul2(a, a), hv = pk(h, h);
  // EXACT: the argument (-185 to 0) as a whole number of 2^-15, by way of 256 to 512, so that adding
  // 64 and taking the rest are exact
  constexpr float whole = 511.0f;
  f2_t u = mul2(square, hv), steps = 0;
  if constexpr (EXACT) {
    steps = fma2(square, hv, pk(whole, whole));
    u = add2(steps, pk(64.0f - whole, 64.0f - whole));
  }
  float ul, uh;
  unpk(u, ul, uh);
  bell = pk(exp2_near(ul), exp2_near(uh));
  if constexpr (EXACT) {
    const f2_t minus = pk(-1.0f, -1.0f);
    const f2_t square_rest = fma2(a, a, mul2(square, minus)), rest = fma2(square, hv, fma2(steps, minus, pk(whole, whole)));
    const f2_t all = fma2(square_rest, hv, fma2(square, pk(h_rest, h_rest), rest));
    bell = fma2(mul2(bell, pk(ln2, ln2)), all, bell);
  }
  const f2_t below = mul2(mul2(q, t), bell);
  float bl, bh, al, ah;
  unpk(below, bl, bh);
  unpk(fma2(below, pk(-1.0f, -1.0f), one), al, ah);
  s = pk(lo > 0.0f ? al : bl, hi > 0.0f ? ah : bh);
}
template <int KIND, bool EXACT, bool SLOPE>
__device__ __forceinline__ void activation8(const float (&g)[8], float (&f)[8], float (&df)[8]) {
  if constexpr (KIND == OPT_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const f2_t gv = pk(g[j], g[j + 1]);
      f2_t s, bell;
      normal2<EXACT>(gv, s, bell);
      unpk(mul2(gv, s), f[j], f[j + 1]);
      constexpr float root = 0.3989422804014327f / kBellScale<EXACT>;
      // (EXACT: the bell's part first, which is 0 where |g| is large)
      if constexpr (SLOPE) unpk(EXACT ? fma2(gv, mul2(bell, pk(root, root)), s) : fma2(mul2(gv, pk(root, root)), bell, s), df[j], df[j + 1]);
    }
  } else if constexpr (EXACT || KIND == OPT_ACT_RELU) {
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
      float lo, hi, one_lo, one_hi;
      unpk(z, lo, hi);
      lo = exp2_near(lo);
      hi = exp2_near(hi);
      unpk(add2(pk(lo, hi), one), one_lo, one_hi);
      const f2_t s = pk(reciprocal_near(one_lo), reciprocal_near(one_hi)), fv = mul2(gv, s);
      unpk(fv, f[j], f[j + 1]);
      if constexpr (SLOPE) {
        // 1 - s as e s (a difference has no digits where s is near 1, and moves the scale of a
        // block whose largest value lies on a power of two times 448); where e is infinite f is 0
        f2_t n = mul2(pk(fminf(lo, 3.0e38f), fminf(hi, 3.0e38f)), s);
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

// What is written in 8 bits of a chunk of row r at column c: y, and the inputs that are kept.
// By whole warps; elements from `valid` on are 0.
template <typename T>
__device__ __forceinline__ void put_forward(const opt_gated_args& a, int64_t at, int valid, uint8_t* codes, uint8_t* gcodes,
                                            uint8_t* ucodes, const Raw<T>& graw, const Raw<T>& uraw, const float (&y)[8]) {
  uint32_t top = 0, gtop = 0, utop = 0;
  if (codes != nullptr) top = top16(top8_of(y));
  if (gcodes != nullptr || ucodes != nullptr) {
    gtop = top_of(magnitudes(graw, false));
    utop = top_of(magnitudes(uraw, false));
    tops16(gtop, utop, T());
  }
  uint8_t *scales = static_cast<uint8_t*>(a.d_scales), *gscales = static_cast<uint8_t*>(a.d_gate_scales),
          *uscales = static_cast<uint8_t*>(a.d_up_scales);
  const bool odd = __any_sync(0xFFFFFFFFu, max(max(top, gtop), utop) >= kInfBits);      // rare
  const auto put = [&](uint8_t* p, uint8_t* tiles, const float (&x)[8], uint32_t t) {
    if (odd) put_codes8(p, tiles, at, valid, x);
    else put_finite8(p, tiles, at, valid, x, t);
  };
  if (codes != nullptr) put(codes, scales, y, top);
  float x[8];
  if (gcodes != nullptr) {
    unpack(graw, x);
    put(gcodes, gscales, x, gtop);
  }
  if (ucodes != nullptr) {
    unpack(uraw, x);
    put(ucodes, uscales, x, utop);
  }
}

__device__ __forceinline__ uint8_t* row_of(void* codes, int64_t pitch, int64_t r, int64_t c) {
  return codes == nullptr ? nullptr : static_cast<uint8_t*>(codes) + r * pitch + c;
}

// Whole chunks: a thread keeps to its column and goes down the rows by pointers, the next
// row's loads under way (a row to a thread 229 us at the size below).  KEEP: every input is
// kept; else none is (choices inside the loop: 177 us).  Bound by HBM, with the instructions
// close behind: 8192 x 14336 BF16, silu, to codes with both inputs kept 139 us, 0.87 of a copy's
// rate, issue 67 % busy; to y alone 114 us, 0.91.
template <typename T, int KIND, bool UP, bool KEEP>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3) gated_vec_kernel(const __grid_constant__ opt_gated_args a) {
  const uint32_t c = 8 * (blockIdx.x * blockDim.x + threadIdx.x), rows = (uint32_t)a.rows;
  const uint32_t step = gridDim.y * blockDim.y, panel = 512 * (uint32_t)((a.cols + 511) / 512);
  const uint32_t place = 512 * (c >> 9) + ((c >> 7) & 3);
  const bool on = c < (uint32_t)a.cols, first = on && (threadIdx.x & 15) == 0, want_y = a.d_y != nullptr, want_codes = a.d_codes != nullptr;
  uint32_t r = (uint32_t)first_row();
  const auto start = [&](auto* base, int64_t pitch) { return base + (r * pitch + c); };
  const T *gate = start(static_cast<const T*>(a.d_gate), a.gate_pitch), *up = start(static_cast<const T*>(a.d_up), a.up_pitch);
  T* y_out = start(static_cast<T*>(a.d_y), a.y_pitch);
  uint8_t *codes = start(static_cast<uint8_t*>(a.d_codes), a.codes_pitch), *gcodes = start(static_cast<uint8_t*>(a.d_gate_codes), a.gate_codes_pitch),
          *ucodes = start(static_cast<uint8_t*>(a.d_up_codes), a.up_codes_pitch);
  const int64_t gate_step = step * a.gate_pitch, up_step = step * a.up_pitch, y_step = step * a.y_pitch, codes_step = step * a.codes_pitch,
                gcodes_step = step * a.gate_codes_pitch, ucodes_step = step * a.up_codes_pitch;
  Raw<T> gnext = load_if(gate, on && r < rows), unext = {};
  if (UP) unext = load_if(up, on && r < rows);
  for (; r < rows; r += step) {
    const Raw<T> graw = gnext, uraw = unext;
    gate += gate_step;
    gnext = load_if(gate, on && r + step < rows);
    if (UP) {
      up += up_step;
      unext = load_if(up, on && r + step < rows);
    }
    float g[8], u[8], y[8], unused[8];
    unpack(graw, g);
    activation8<KIND, sizeof(T) == 4, false>(g, y, unused);
    if (UP) {
      unpack(uraw, u);
      times8(y, u);
    }
    if (want_y) {
      store8_if(y_out, y, on);
      y_out += y_step;
    }
    if (!KEEP && !want_codes) continue;
    uint32_t top = want_codes ? top16(top8_of(y)) : 0, gtop = 0, utop = 0;
    if (KEEP) {
      gtop = top_of(magnitudes(graw, false));
      if (UP) {
        utop = top_of(magnitudes(uraw, false));
        tops16(gtop, utop, T());
      } else {
        gtop = top16(gtop);
      }
    }
    const uint64_t at = (uint64_t)(r >> 7) * panel + (place + 16 * (r & 31) + ((r >> 3) & 12));
    uint8_t *scales = static_cast<uint8_t*>(a.d_scales) + at, *gscales = static_cast<uint8_t*>(a.d_gate_scales) + at,
            *uscales = static_cast<uint8_t*>(a.d_up_scales) + at;
    if (__any_sync(0xFFFFFFFFu, max(max(top, gtop), utop) >= kInfBits)) {      // rare
      if (want_codes) put_codes8(codes, scales, 0, on ? 8 : 0, y);
      if (KEEP) put_codes8(gcodes, gscales, 0, on ? 8 : 0, g);
      if (KEEP && UP) put_codes8(ucodes, uscales, 0, on ? 8 : 0, u);
    } else {
      if (want_codes) put_finite_if(codes, scales, y, top, on, first);
      if (KEEP) put_finite_if(gcodes, gscales, g, gtop, on, first);
      if (KEEP && UP) put_finite_if(ucodes, uscales, u, utop, on, first);
    }
    codes += codes_step;
    gcodes += gcodes_step;
    ucodes += ucodes_step;
  }
}
// Rows that begin anywhere, or one input of two kept: bound by the instructions that move words
// into place (issue 74 % busy).  The same 8192 x 14336 take 229 us, with one input kept 214.
template <typename T, int KIND>
__global__ void __launch_bounds__(kThreads, 4) gated_any_kernel(const __grid_constant__ opt_gated_args a) {
  __shared__ __align__(16) Ragged<T, false, kThreads / 32> ragged;
  T* buffer = ragged.chunk[warp_of_block()];
  const int64_t c = 8 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x), panel = (a.cols + 511) / 512;
  const int valid = (int)max(min(a.cols - c, (int64_t)8), (int64_t)0), up_valid = a.d_up != nullptr ? valid : 0;
  for (int64_t r = first_row(); r < a.rows; r += (int64_t)gridDim.y * blockDim.y) {
    const Row<T, false> gate(a.d_gate, a.gate_pitch, a.rows, a.cols, r), up(a.d_up, a.up_pitch, a.rows, a.cols, r);
    const Ahead<T, false> ga = gate.ahead(c, valid), ua = up.ahead(c, up_valid);
    const Raw<T> graw = gate.chunk(ga, c, valid), uraw = up.chunk(ua, c, up_valid);
    float x[8], y[8], unused[8];
    unpack(graw, x);
    activation8<KIND, sizeof(T) == 4, false>(x, y, unused);
    if (a.d_up != nullptr) {
      unpack(uraw, x);
      times8(y, x);
    }
    if (a.d_y != nullptr) store_at<false>(a.d_y, a.y_pitch, a.cols, r, c, valid, y, buffer);
    put_forward<T>(a, scale_place(r, c >> 7, panel), valid, row_of(a.d_codes, a.codes_pitch, r, c),
                   row_of(a.d_gate_codes, a.gate_codes_pitch, r, c), row_of(a.d_up_codes, a.up_codes_pitch, r, c), graw, uraw, y);
  }
}

// ------------------------------------------------------------------ gradients
// Without transposed outputs, whole chunks: down the rows by pointers, as above.  8192 x 14336
// BF16 from kept inputs to codes 141 us, 0.74 of a copy's rate, bound by instructions (issue 71 %
// busy at 40 % of the warps); between plain matrices 181 us, 0.96.  CTAs to an SM by registers:
// with three, plain fp32 spills (4096 x 14336 206 us, with two 175, 0.99).
template <typename T, typename S, int KIND, bool UP>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : sizeof(S) == 1 ? 3 : 2) gated_backward_vec_kernel(
    const __grid_constant__ opt_gated_backward_args a) {
  constexpr bool KEPT = sizeof(S) == 1;
  using In = std::conditional_t<KEPT, uint8_t, T>;
  const uint32_t c = 8 * (blockIdx.x * blockDim.x + threadIdx.x), rows = (uint32_t)a.rows;
  const uint32_t step = gridDim.y * blockDim.y, panel = 512 * (uint32_t)((a.cols + 511) / 512);
  const uint32_t place = 512 * (c >> 9) + ((c >> 7) & 3);
  const bool on = c < (uint32_t)a.cols, first = on && (threadIdx.x & 15) == 0;
  const bool plain_g = a.d_dgate != nullptr, plain_u = UP && a.d_dup != nullptr, codes_g = a.d_dgate_codes != nullptr,
             codes_u = UP && a.d_dup_codes != nullptr;
  uint32_t r = (uint32_t)first_row();
  const auto start = [&](auto* base, int64_t pitch) { return base + (r * pitch + c); };
  const T* dy = start(static_cast<const T*>(a.d_dy), a.dy_pitch);
  const In *gate = start(static_cast<const In*>(a.d_gate), a.gate_pitch), *up = start(static_cast<const In*>(a.d_up), a.up_pitch);
  T *dgate = start(static_cast<T*>(a.d_dgate), a.dgate_pitch), *dup = start(static_cast<T*>(a.d_dup), a.dup_pitch);
  uint8_t *gcodes = start(static_cast<uint8_t*>(a.d_dgate_codes), a.dgate_codes_pitch),
          *ucodes = start(static_cast<uint8_t*>(a.d_dup_codes), a.dup_codes_pitch);
  const int64_t dy_step = step * a.dy_pitch, gate_step = step * a.gate_pitch, up_step = step * a.up_pitch, dgate_step = step * a.dgate_pitch,
                dup_step = step * a.dup_pitch, gcodes_step = step * a.dgate_codes_pitch, ucodes_step = step * a.dup_codes_pitch;
  const auto scale_at = [&](uint32_t row) { return (uint64_t)(row >> 7) * panel + (place + 16 * (row & 31) + ((row >> 3) & 12)); };
  std::conditional_t<KEPT, KeptAsk, Raw<T>> gnext, unext;
  Raw<T> dnext;
  const auto ask = [&](uint32_t row) {
    const bool there = on && row < rows;
    dnext = load_if(dy, there);
    if constexpr (KEPT) {
      gnext.codes = load_codes_if(gate, there);
      gnext.byte = load_byte_if(static_cast<const uint8_t*>(a.d_gate_scales) + scale_at(row), there);
      if (UP) {
        unext.codes = load_codes_if(up, there);
        unext.byte = load_byte_if(static_cast<const uint8_t*>(a.d_up_scales) + scale_at(row), there);
      }
    } else {
      gnext = load_if(gate, there);
      if (UP) unext = load_if(up, there);
    }
  };
  const auto values = [](const auto& in, float (&x)[8]) {
    if constexpr (KEPT) values8(in.codes, scale_of(in.byte), x);
    else unpack(in, x);
  };
  ask(r);
  for (; r < rows; r += step) {
    float d[8], g[8], u[8], f[8], df[8];
    values(gnext, g);
    if (UP) values(unext, u);
    unpack(dnext, d);
    dy += dy_step;
    gate += gate_step;
    if (UP) up += up_step;
    ask(r + step);
    activation8<KIND, sizeof(T) == 4, true>(g, f, df);
    times8(df, d);
    times8(f, d);
    if (UP) times8(df, u);
    if (plain_g) {
      store8_if(dgate, df, on);
      dgate += dgate_step;
    }
    if (plain_u) {
      store8_if(dup, f, on);
      dup += dup_step;
    }
    if (!codes_g && !codes_u) continue;
    // both matrices' fields through the exchanges in one word
    uint32_t both = scale_field(top8_of(df)) >> 23 | (scale_field(UP ? top8_of(f) : 0u) >> 23) << 16;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) both = larger(both, __shfl_xor_sync(0xFFFFFFFFu, both, o), Bf16());
    uint8_t *gscales = static_cast<uint8_t*>(a.d_dgate_scales) + scale_at(r), *uscales = static_cast<uint8_t*>(a.d_dup_scales) + scale_at(r);
    if (__any_sync(0xFFFFFFFFu, max(both & 0xFFFFu, both >> 16) >= 255u)) {      // rare
      if (codes_g) put_codes8(gcodes, gscales, 0, on ? 8 : 0, df);
      if (codes_u) put_codes8(ucodes, uscales, 0, on ? 8 : 0, f);
    } else {
      if (codes_g) put_field_if(gcodes, gscales, df, both << 23, on, first);
      if (codes_u) put_field_if(ucodes, uscales, f, (both >> 16) << 23, on, first);
    }
    gcodes += gcodes_step;
    ucodes += ucodes_step;
  }
}
// The same of rows that begin anywhere (8192 x 14336 from kept inputs to codes 279 us).
template <typename T, typename S, int KIND>
__global__ void __launch_bounds__(kThreads, 3) gated_backward_any_kernel(const __grid_constant__ opt_gated_backward_args a) {
  constexpr bool VEC = false;
  __shared__ __align__(16) Ragged<T, VEC, kThreads / 32> ragged;
  T* buffer = ragged.chunk[warp_of_block()];
  const int64_t c = 8 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x), panel = (a.cols + 511) / 512;
  const int valid = (int)max(min(a.cols - c, (int64_t)8), (int64_t)0);
  const bool has_up = a.d_up != nullptr;
  for (int64_t r = first_row(); r < a.rows; r += (int64_t)gridDim.y * blockDim.y) {
    const Source<T, VEC> dy(a.d_dy, nullptr, a.dy_pitch, a.rows, a.cols, r);
    const Source<S, VEC> gate(a.d_gate, a.d_gate_scales, a.gate_pitch, a.rows, a.cols, r);
    const Source<S, VEC> up(a.d_up, a.d_up_scales, a.up_pitch, a.rows, a.cols, r);
    Ahead<T, VEC> da = {};
    typename Source<S, VEC>::Ask ga = {}, ua = {};
    da = dy.ahead(c, valid);
    ga = gate.ahead(c, valid);
    if (has_up) ua = up.ahead(c, valid);
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
    if (a.d_dgate != nullptr) store_at<VEC>(a.d_dgate, a.dgate_pitch, a.cols, r, c, valid, df, buffer);
    if (a.d_dup != nullptr) store_at<VEC>(a.d_dup, a.dup_pitch, a.cols, r, c, valid, f, buffer);
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
// codes in whole lines.  The next tile's loads are under way meanwhile.  fp32 values in shared
// memory, since both orientations round from them; 192 KB of them leave one CTA to an SM.
constexpr int kTurnThreads = 1024, kTile = 128 * 128;
constexpr int kTurnBytes = 3 * kTile * (int)sizeof(float);

// Offsets inside a tile: 32 bits for whole chunks (the host has seen that they hold them).
template <bool VEC>
using Offset = std::conditional_t<VEC, uint32_t, int64_t>;

// Place of columns 4 quad ... 4 quad + 3 of a tile's row, in units of four values: the N quads
// that a thread has of a row lie 32 / N apart, and every 16 rows are turned by one more, so that
// neither eight threads' quads of a row nor the rows 16 apart of a column meet in a bank.
template <int N>
__device__ __forceinline__ int turned_place(int row, int quad) {
  return 32 * row + (((quad / N) | (quad % N) * (32 / N)) ^ (row >> 4));
}

// A tile's values by columns: four columns to a warp, 16 rows of one of them to a lane
// (`column` is the first of them).  Their codes, 16 bytes in the rows' order, and the column's
// scale byte.
__device__ __forceinline__ uint32_t code_column(const float* column, uint32_t (&word)[4]) {
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = column[128 * i];
  const auto exchanged = [&](float t) {                 // over the column's eight lanes
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      const float other = __shfl_xor_sync(0xFFFFFFFFu, t, o);
      t = largest3(t, other, other);
    }
    return f2u(t);
  };
  float top = largest3(x[0], x[1], x[2]);
#pragma unroll
  for (int i = 3; i < 15; i += 2) top = largest3(top, x[i], x[i + 1]);
  uint32_t field = scale_field(exchanged(largest3(top, x[15], x[15])));
  if (__any_sync(0xFFFFFFFFu, field >= kOddField)) {    // rare: the finite ones' maxima, and NaN for the others
    float finite = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (finite_bits(x[i])) finite = fmaxf(finite, fabsf(x[i]));
      else x[i] = u2f(0x7FC00000u);
    }
    field = scale_field(exchanged(finite));
  }
  const float inv = inverse_of_field(field);
#pragma unroll
  for (int i = 0; i < 16; i += 2) unpk(mul2(pk(x[i], x[i + 1]), pk(inv, inv)), x[i], x[i + 1]);
#pragma unroll
  for (int k = 0; k < 4; ++k) word[k] = e4m3x2_rn(x[4 * k], x[4 * k + 1]) | e4m3x2_rn(x[4 * k + 2], x[4 * k + 3]) << 16;
  return byte_of_field(field);
}
// What a lane has of the columns: its column, and the first of its 16 rows.
__device__ __forceinline__ int lane_column() { return 4 * (threadIdx.x >> 5) + ((threadIdx.x & 31) >> 3); }
__device__ __forceinline__ int lane_row() { return 16 * (threadIdx.x & 7); }
template <int N>
__device__ __forceinline__ const float* lane_values(const float4* held) {
  const int column = lane_column();
  return reinterpret_cast<const float*>(held + turned_place<N>(lane_row(), column >> 2)) + (column & 3);
}
// Those of the tile at `v`: codes to `codes` (the tile's first column's), scale bytes to
// `scales` (the tile's).
template <bool VEC>
__device__ __forceinline__ void put_columns(const float4* v, uint8_t* codes, uint8_t* scales, int64_t pitch, int rows, int cols) {
  uint32_t word[4];
  const uint32_t byte = code_column(lane_values<2>(v), word);
  const int column = lane_column(), row = lane_row();
  if (column >= cols) return;
  store_codes16(codes + ((Offset<VEC>)column * (Offset<VEC>)pitch + row), word, rows - row);
  if (row == 0) scales[16 * (column & 31) + 4 * (column >> 5)] = (uint8_t)byte;
}

template <typename T, typename S, bool VEC>
struct Inputs {
  Ahead<T, VEC> dy;
  typename Source<S, VEC>::Ask gate, up;
};

// The whole backward pass of a training step in BF16 from kept inputs: all five 8-bit operands
// and nothing plain.  The same work as gated_backward_tile_kernel's without its choices (which
// take half of its instructions).  CTAs take runs of tiles along a row of tiles; places in a
// matrix are counted in chunks of eight or 16 elements, so that
// 32 bits hold them (turn_places_fit, below).  8192 x 14336 238 us, 0.66 of a copy's rate (356 by
// gated_backward_tile_kernel): bound by instructions and the shared memory's pipe between two
// barriers (issue 59 % busy; when it took 268 us, 186 without loads and stores of global memory,
// 169 without the columns, 120 without either).
template <int KIND>
__global__ void __launch_bounds__(kTurnThreads, 1) gated_backward_turn_kernel(const __grid_constant__ opt_gated_backward_args a,
                                                                             uint32_t row_tiles, uint32_t col_tiles, uint32_t per_cta) {
  extern __shared__ __align__(16) float4 held[];       // dgate, dup, y
  // 16 columns of a row to a thread, in two halves; then 16 rows of a column
  const uint32_t q = threadIdx.x & 7, row = threadIdx.x >> 3, t_col = lane_column(), t_row = lane_row();
  const uint32_t all_rows = (uint32_t)a.rows, all_cols = (uint32_t)a.cols;
  const uint32_t panel = 512 * ((all_cols + 511) / 512), panel_t = 512 * ((all_rows + 511) / 512);
  const uint32_t dy_pitch = (uint32_t)(a.dy_pitch >> 3), g_pitch = (uint32_t)(a.gate_pitch >> 4), u_pitch = (uint32_t)(a.up_pitch >> 4),
                 dg_pitch = (uint32_t)(a.dgate_codes_pitch >> 4), du_pitch = (uint32_t)(a.dup_codes_pitch >> 4),
                 dgt_pitch = (uint32_t)(a.dgate_codes_t_pitch >> 4), dut_pitch = (uint32_t)(a.dup_codes_t_pitch >> 4),
                 yt_pitch = (uint32_t)(a.y_codes_t_pitch >> 4);
  float4* const mine = held + turned_place<4>(row, 4 * q);      // the next quads: 8 places further each, before the row's turn
  const float* const column = lane_values<4>(held);
  struct In {
    Raw<Bf16> dy[2];
    uint4 gate, up;
    uint32_t gate_byte, up_byte;
  } in;
  const uint32_t tiles = row_tiles * col_tiles, begin = blockIdx.x * per_cta, end = min(begin + per_cta, tiles);
  uint32_t tr = begin / col_tiles, tc = begin % col_tiles;
  const auto load = [&](uint32_t tr, uint32_t tc) {
    const uint32_t r = 128 * tr + row, c = 8 * tc + q;
    const uint32_t at = panel * tr + 512 * (tc >> 2) + (tc & 3) + 16 * (row & 31) + 4 * (row >> 5);
    const Bf16* dy = static_cast<const Bf16*>(a.d_dy) + (uint64_t)(r * dy_pitch + 2 * c) * 8;
    const uint8_t *g = static_cast<const uint8_t*>(a.d_gate) + (uint64_t)(r * g_pitch + c) * 16,
                  *u = static_cast<const uint8_t*>(a.d_up) + (uint64_t)(r * u_pitch + c) * 16;
    const uint8_t *gs = static_cast<const uint8_t*>(a.d_gate_scales) + at, *us = static_cast<const uint8_t*>(a.d_up_scales) + at;
    if (128 * tr + 128 <= all_rows && 128 * tc + 128 <= all_cols) {
      in.dy[0] = load_raw<true>(dy, 8);
      in.dy[1] = load_raw<true>(dy + 8, 8);
      in.gate = ld_cs_u4(g);
      in.up = ld_cs_u4(u);
      in.gate_byte = *gs;
      in.up_byte = *us;
      return;
    }
    const bool lo = r < all_rows && 16 * c < all_cols, hi = lo && 16 * c + 8 < all_cols;      // whole chunks of eight
    in.dy[0] = load_if(dy, lo);
    in.dy[1] = load_if(dy + 8, hi);
    const uint2 g0 = load_codes_if(g, lo), g1 = load_codes_if(g + 8, hi), u0 = load_codes_if(u, lo), u1 = load_codes_if(u + 8, hi);
    in.gate = make_uint4(g0.x, g0.y, g1.x, g1.y);
    in.up = make_uint4(u0.x, u0.y, u1.x, u1.y);
    in.gate_byte = load_byte_if(gs, lo);
    in.up_byte = load_byte_if(us, lo);
  };
  // The lines of the tile two further, to L2 (loads of the next tile are asked for while this one
  // is turned, which is shorter than the way from memory): of each row two of dy's, one of
  // gate's and one of up's to a thread.
  const auto ask_l2 = [&](uint32_t tr, uint32_t tc) {
    for (; tc >= col_tiles; tc -= col_tiles) ++tr;
    if (threadIdx.x >= 512) {              // eight lines of the tiles' scales, where they begin
      const uint32_t t = threadIdx.x - 512;
      const uint8_t* scales = static_cast<const uint8_t*>((t & 4) ? a.d_up_scales : a.d_gate_scales) + (panel * tr + 512 * (tc >> 2)) + 128 * (t & 3);
      if (t < 8 && (tc & 3) == 0) asm volatile("prefetch.global.L2 [%0];" :: "l"(scales));
      return;
    }
    const uint32_t t = threadIdx.x, r = 128 * tr + (t >> 2), c = 8 * tc;
    if (r >= all_rows || 16 * c + ((t & 3) == 1 ? 64 : 0) >= all_cols) return;
    const uint8_t* p = (t & 2) == 0 ? static_cast<const uint8_t*>(a.d_dy) + (uint64_t)(r * dy_pitch + 2 * c) * 16 + 128 * (t & 1)
                       : (t & 1) == 0 ? static_cast<const uint8_t*>(a.d_gate) + (uint64_t)(r * g_pitch + c) * 16
                                      : static_cast<const uint8_t*>(a.d_up) + (uint64_t)(r * u_pitch + c) * 16;
    asm volatile("prefetch.global.L2 [%0];" :: "l"(p));
  };
  if (begin < end) load(tr, tc);
  if (begin + 1 < end) ask_l2(tr, tc + 1);
  for (uint32_t tile = begin; tile < end; ++tile) {
    const uint32_t r = 128 * tr + row, c = 8 * tc + q;
    if (tile + 2 < end) ask_l2(tr, tc + 2);
    {
      float dgate[16], dup[16];
      const float gate_scale = scale_of(in.gate_byte), up_scale = scale_of(in.up_byte);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float d[8], g[8], u[8], f[8], df[8];
        values8(h == 0 ? make_uint2(in.gate.x, in.gate.y) : make_uint2(in.gate.z, in.gate.w), gate_scale, g);
        activation8<KIND, false, true>(g, f, df);
        unpack(in.dy[h], d);
        times8(df, d);
        times8(d, f);                 // dup
        values8(h == 0 ? make_uint2(in.up.x, in.up.y) : make_uint2(in.up.z, in.up.w), up_scale, u);
        times8(f, u);                 // y
        times8(df, u);                // dgate
        const auto leave = [&](int m, const float (&x)[8]) {
          float4* v = mine + m * (kTile / 4) + 16 * h;
          v[0] = make_float4(x[0], x[1], x[2], x[3]);
          v[8] = make_float4(x[4], x[5], x[6], x[7]);
        };
        leave(0, df);
        leave(1, d);
        leave(2, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dgate[8 * h + j] = df[j];
          dup[8 * h + j] = d[j];
        }
      }
      const auto largest = [&](const float (&x)[16]) {
        float t = largest3(x[0], x[1], x[2]);
#pragma unroll
        for (int j = 3; j < 15; j += 2) t = largest3(t, x[j], x[j + 1]);
        return largest3(t, x[15], x[15]);
      };
      // both matrices' fields through the exchanges of a row's eight lanes in one word
      const auto fields = [&](float gt, float ut) {
        uint32_t both = scale_field(f2u(gt)) >> 23 | (scale_field(f2u(ut)) >> 23) << 16;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) both = larger(both, __shfl_xor_sync(0xFFFFFFFFu, both, o), Bf16());
        return both;
      };
      uint32_t both = fields(largest(dgate), largest(dup));
      if (__any_sync(0xFFFFFFFFu, max(both & 0xFFFFu, both >> 16) >= 255u)) {      // rare: the finite ones' maxima, and NaN for the others
        float gt = 0.0f, ut = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          gt = finite_bits(dgate[j]) ? fmaxf(gt, fabsf(dgate[j])) : gt;
          ut = finite_bits(dup[j]) ? fmaxf(ut, fabsf(dup[j])) : ut;
          dgate[j] = finite_bits(dgate[j]) ? dgate[j] : u2f(0x7FC00000u);
          dup[j] = finite_bits(dup[j]) ? dup[j] : u2f(0x7FC00000u);
        }
        both = fields(gt, ut);
      }
      const int left = r < all_rows ? (int)(all_cols - min(16 * c, all_cols)) : 0;
      const uint32_t at = panel * tr + 512 * (tc >> 2) + (tc & 3) + 16 * (row & 31) + 4 * (row >> 5);
      const auto put = [&](void* codes, void* scales, uint32_t pitch, const float (&x)[16], uint32_t field) {
        const float inv = inverse_of_field(field);
        uint32_t word[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float v[4];
          unpk(mul2(pk(x[4 * k], x[4 * k + 1]), pk(inv, inv)), v[0], v[1]);
          unpk(mul2(pk(x[4 * k + 2], x[4 * k + 3]), pk(inv, inv)), v[2], v[3]);
          word[k] = e4m3x2_rn(v[0], v[1]) | e4m3x2_rn(v[2], v[3]) << 16;
        }
        uint8_t* p = static_cast<uint8_t*>(codes) + (uint64_t)(r * pitch + c) * 16;
        if (left >= 16) st_cs_u4(p, make_uint4(word[0], word[1], word[2], word[3]));
        else if (left > 0) st_cs_u2(p, make_uint2(word[0], word[1]));      // a whole chunk of eight
        if (q == 0 && left > 0) static_cast<uint8_t*>(scales)[at] = (uint8_t)byte_of_field(field);
      };
      put(a.d_dgate_codes, a.d_dgate_scales, dg_pitch, dgate, both << 23);
      put(a.d_dup_codes, a.d_dup_scales, du_pitch, dup, (both >> 16) << 23);
    }
    const uint32_t col = 128 * tc + t_col, row16 = 128 * tr + t_row;
    const uint32_t at_t = panel_t * tc + 512 * (tr >> 2) + (tr & 3) + 16 * (t_col & 31) + 4 * (t_col >> 5);
    if (++tc == col_tiles) {
      tc = 0;
      ++tr;
    }
    if (tile + 1 < end) load(tr, tc);
    __syncthreads();
    const auto turn = [&](int m, void* codes, void* scales, uint32_t pitch) {
      uint32_t word[4];
      const uint32_t byte = code_column(column + m * kTile, word);
      if (col < all_cols) {
        store_codes16(static_cast<uint8_t*>(codes) + (uint64_t)(col * pitch + (row16 >> 4)) * 16, word, (int)(all_rows - row16));
        if (t_row == 0) (static_cast<uint8_t*>(scales) + at_t)[0] = (uint8_t)byte;
      }
    };
    turn(0, a.d_dgate_codes_t, a.d_dgate_scales_t, dgt_pitch);
    turn(1, a.d_dup_codes_t, a.d_dup_scales_t, dut_pitch);
    turn(2, a.d_y_codes_t, a.d_y_scales_t, yt_pitch);
    __syncthreads();
  }
}

// Any set of outputs, from any inputs: CTAs take tiles gridDim.x apart, `step_rows` and
// `step_cols` in rows and columns of tiles.  8192 x 14336 BF16 from plain inputs to all five
// operands 347 us, 0.55 of a copy's rate (514 where rows begin anywhere), bound as the kernel above.
template <typename T, typename S, int KIND, bool VEC>
__global__ void __launch_bounds__(kTurnThreads, 1) gated_backward_tile_kernel(
    const __grid_constant__ opt_gated_backward_args a, int row_tiles, int col_tiles, int step_rows, int step_cols) {
  extern __shared__ __align__(16) float4 held[];       // dgate, dup, y
  using Off = Offset<VEC>;
  constexpr bool KEPT = sizeof(S) == 1;
  // plain fp32 inputs of two rows leave no registers for the next tile's
  constexpr bool AHEAD = sizeof(T) == 2 || KEPT;
  const int q = threadIdx.x & 15, row = 2 * (threadIdx.x >> 4);
  const int64_t panel = (a.cols + 511) / 512, panel_t = (a.rows + 511) / 512;
  const int scale_row = 16 * (row & 31) + 4 * (row >> 5);      // row + 1: 16 more
  const bool has_up = a.d_up != nullptr;
  const auto rows_of = [&](int tr) { return (int)min(a.rows - 128 * (int64_t)tr, (int64_t)128); };
  const auto cols_of = [&](int tc) { return (int)min(a.cols - 128 * (int64_t)tc, (int64_t)128); };
  const auto tile_of = [&](int64_t pitch, int tr, int tc) { return 128 * ((int64_t)tr * pitch + tc); };
  const auto place_of = [&](int64_t p, int tr, int tc) { return 512 * (tr * p + (tc >> 2)) + (tc & 3); };
  const auto source = [&](const void* base, const void* tiles, int64_t pitch, int tr, int tc, int i, int valid) {
    const Off at = (Off)(row + i) * (Off)pitch + 8 * q;
    typename Source<S, VEC>::Ask ask = {};
    if constexpr (KEPT) {
      ask.codes = load_codes8(static_cast<const uint8_t*>(base) + tile_of(pitch, tr, tc) + at, valid);
      ask.byte = (static_cast<const uint8_t*>(tiles) + place_of(panel, tr, tc))[scale_row + 16 * i];
    } else if constexpr (VEC) {
      const Raw<T> r = load_raw<true>(static_cast<const T*>(base) + tile_of(pitch, tr, tc) + at, 8);
#pragma unroll
      for (int k = 0; k < Raw<T>::kWords; ++k) ask.w[k] = r.w[k];
    } else {
      ask = Source<S, VEC>(base, tiles, pitch, a.rows, a.cols, 128 * (int64_t)tr + row + i).ahead(128 * (int64_t)tc + 8 * q, valid);
    }
    return ask;
  };
  const auto load = [&](int tr, int tc, int i) {
    Inputs<T, S, VEC> in = {};
    const int valid = row + i < rows_of(tr) ? max(min(cols_of(tc) - 8 * q, 8), 0) : 0;
    if (valid > 0) {
      if constexpr (VEC) {
        const Raw<T> r = load_raw<true>(static_cast<const T*>(a.d_dy) + tile_of(a.dy_pitch, tr, tc) +
                                            ((Off)(row + i) * (Off)a.dy_pitch + 8 * q), 8);
#pragma unroll
        for (int k = 0; k < Raw<T>::kWords; ++k) in.dy.w[k] = r.w[k];
      } else {
        in.dy = Row<T, VEC>(a.d_dy, a.dy_pitch, a.rows, a.cols, 128 * (int64_t)tr + row + i).ahead(128 * (int64_t)tc + 8 * q, valid);
      }
      in.gate = source(a.d_gate, a.d_gate_scales, a.gate_pitch, tr, tc, i, valid);
      if (has_up) in.up = source(a.d_up, a.d_up_scales, a.up_pitch, tr, tc, i, valid);
    }
    return in;
  };
  int tr = (int)blockIdx.x / col_tiles, tc = (int)blockIdx.x % col_tiles;
  Inputs<T, S, VEC> in[2];
  if (AHEAD) {
#pragma unroll
    for (int i = 0; i < 2; ++i) in[i] = load(tr, tc, i);
  }
  while (tr < row_tiles) {
    const int rows = rows_of(tr), cols = cols_of(tc);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!AHEAD) in[i] = load(tr, tc, i);
      const int valid = row + i < rows ? max(min(cols - 8 * q, 8), 0) : 0;
      const int64_t r = 128 * (int64_t)tr + row + i, c = 128 * (int64_t)tc + 8 * q;      // only of rows that begin anywhere
      float d[8], g[8], u[8], f[8], df[8];
      Source<S, VEC>(a.d_gate, a.d_gate_scales, a.gate_pitch, a.rows, a.cols, r).values(in[i].gate, c, valid, g);
      activation8<KIND, sizeof(T) == 4, true>(g, f, df);
      Source<T, VEC>(a.d_dy, nullptr, a.dy_pitch, a.rows, a.cols, r).values(in[i].dy, c, valid, d);
      times8(df, d);
      times8(d, f);                 // dup
      if (has_up) {
        Source<S, VEC>(a.d_up, a.d_up_scales, a.up_pitch, a.rows, a.cols, r).values(in[i].up, c, valid, u);
        times8(f, u);               // y
        times8(df, u);              // dgate
      }
      const auto leave = [&](int m, const float (&x)[8]) {
        float4* v = held + m * (kTile / 4);
        v[turned_place<2>(row + i, 2 * q)] = make_float4(x[0], x[1], x[2], x[3]);
        v[turned_place<2>(row + i, 2 * q + 1)] = make_float4(x[4], x[5], x[6], x[7]);
      };
      if (a.d_dgate_codes_t != nullptr) leave(0, df);
      if (a.d_dup_codes_t != nullptr) leave(1, d);
      if (a.d_y_codes_t != nullptr) leave(2, f);
      if (a.d_dgate_codes != nullptr || a.d_dup_codes != nullptr) {
        uint32_t gtop = top8_of(df), utop = top8_of(d);
        tops16(gtop, utop, 0.0f);
        const bool odd = __any_sync(0xFFFFFFFFu, max(gtop, utop) >= kInfBits);      // rare
        const auto put = [&](void* codes, void* scales, int64_t pitch, const float (&x)[8], uint32_t top) {
          uint8_t* p = static_cast<uint8_t*>(codes) + tile_of(pitch, tr, tc) + ((Off)(row + i) * (Off)pitch + 8 * q);
          uint8_t* tiles = static_cast<uint8_t*>(scales) + place_of(panel, tr, tc);
          if (odd) put_codes8(p, tiles, scale_row + 16 * i, valid, x);
          else put_finite8(p, tiles, scale_row + 16 * i, valid, x, top);
        };
        if (a.d_dgate_codes != nullptr) put(a.d_dgate_codes, a.d_dgate_scales, a.dgate_codes_pitch, df, gtop);
        if (a.d_dup_codes != nullptr) put(a.d_dup_codes, a.d_dup_scales, a.dup_codes_pitch, d, utop);
      }
      __syncwarp();                 // an output may lie in an input's place, of which lanes read their neighbours' words
      if (valid > 0) {
        const auto store = [&](void* out, int64_t pitch, const float (&x)[8]) {
          store8<VEC>(static_cast<T*>(out) + tile_of(pitch, tr, tc) + ((Off)(row + i) * (Off)pitch + 8 * q), valid, x);
        };
        if (a.d_dgate != nullptr) store(a.d_dgate, a.dgate_pitch, df);
        if (a.d_dup != nullptr) store(a.d_dup, a.dup_pitch, d);
      }
    }
    __syncthreads();
    const int at_row = tr, at_col = tc;
    tr += step_rows;
    tc += step_cols;
    if (tc >= col_tiles) {
      tc -= col_tiles;
      ++tr;
    }
    if (AHEAD && tr < row_tiles) {
#pragma unroll
      for (int i = 0; i < 2; ++i) in[i] = load(tr, tc, i);
    }
    const auto turn = [&](int m, void* codes, void* scales, int64_t pitch) {
      if (codes != nullptr)
        put_columns<VEC>(held + m * (kTile / 4), static_cast<uint8_t*>(codes) + tile_of(pitch, at_col, at_row),
                         static_cast<uint8_t*>(scales) + place_of(panel_t, at_col, at_row), pitch, rows, cols);
    };
    turn(0, a.d_dgate_codes_t, a.d_dgate_scales_t, a.dgate_codes_t_pitch);
    turn(1, a.d_dup_codes_t, a.d_dup_scales_t, a.dup_codes_t_pitch);
    turn(2, a.d_y_codes_t, a.d_y_scales_t, a.y_codes_t_pitch);
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
  // and, of any matrix, 128 rows in 32-bit offsets
  void in_tile(const void* p, int64_t pitch, int64_t size) {
    ok = ok && (p == nullptr || pitch <= INT64_C(0x7FFFFFFF) / (128 * size));
  }
};

template <typename T, int KIND, bool UP, bool KEEP>
cudaError_t forward_vec(const opt_gated_args& a, ChunkGrid g, int sm_count, cudaStream_t s) {
  static OccupancyCache cache;
  const auto kernel = gated_vec_kernel<T, KIND, UP, KEEP>;
  g.limit((int64_t)sm_count * cached_occupancy(kernel, cache, kThreads, 0));
  kernel<<<g.grid, g.block, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int KIND>
cudaError_t forward_kind(const opt_gated_args& a, int sm_count, cudaStream_t s) {
  VecRule v{a.rows, sizeof(T), a.cols % 8 == 0};
  v.see(a.d_gate, a.gate_pitch);
  v.see(a.d_up, a.up_pitch);
  v.see(a.d_y, a.y_pitch);
  const bool up = a.d_up != nullptr, keep = a.d_gate_codes != nullptr;
  const ChunkGrid g(a.rows, a.cols, kThreads);
  if (v.ok && (!up || keep == (a.d_up_codes != nullptr))) {
    if (up) return keep ? forward_vec<T, KIND, true, true>(a, g, sm_count, s) : forward_vec<T, KIND, true, false>(a, g, sm_count, s);
    return keep ? forward_vec<T, KIND, false, true>(a, g, sm_count, s) : forward_vec<T, KIND, false, false>(a, g, sm_count, s);
  }
  gated_any_kernel<T, KIND><<<g.grid, g.block, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t forward(const opt_gated_args& a, int sm_count, cudaStream_t s) {
  switch (a.activation) {
    case OPT_ACT_SILU: return forward_kind<T, OPT_ACT_SILU>(a, sm_count, s);
    case OPT_ACT_GELU_TANH: return forward_kind<T, OPT_ACT_GELU_TANH>(a, sm_count, s);
    case OPT_ACT_GELU: return forward_kind<T, OPT_ACT_GELU>(a, sm_count, s);
    default: return forward_kind<T, OPT_ACT_RELU>(a, sm_count, s);
  }
}

template <typename T, typename S, int KIND, bool UP>
cudaError_t backward_rows(const opt_gated_backward_args& a, ChunkGrid g, int sm_count, cudaStream_t s) {
  static OccupancyCache cache;
  const auto kernel = gated_backward_vec_kernel<T, S, KIND, UP>;
  g.limit((int64_t)sm_count * cached_occupancy(kernel, cache, kThreads, 0));
  kernel<<<g.grid, g.block, 0, s>>>(a);
  return cudaGetLastError();
}

template <int KIND>
cudaError_t backward_turn(const opt_gated_backward_args& a, int sm_count, cudaStream_t s) {
  static OccupancyCache cache;
  const auto kernel = gated_backward_turn_kernel<KIND>;
  const int row_tiles = (int)((a.rows + 127) / 128), col_tiles = (int)((a.cols + 127) / 128);
  const int64_t tiles = (int64_t)row_tiles * col_tiles, held = (int64_t)sm_count * cached_occupancy(kernel, cache, kTurnThreads, kTurnBytes);
  const int64_t most = held > 0 ? held : 1;      // (none where the device refuses that much shared memory: the launch says so)
  const int per_cta = (int)((tiles + most - 1) / most);
  kernel<<<(unsigned)((tiles + per_cta - 1) / per_cta), kTurnThreads, kTurnBytes, s>>>(a, row_tiles, col_tiles, per_cta);
  return cudaGetLastError();
}
// Whether 32 bits hold the places that gated_backward_turn_kernel counts (to the ends of
// whole tiles).
bool turn_places_fit(const opt_gated_backward_args& a) {
  const int64_t most = INT64_C(0xFFFFFFFF), r = a.rows + 127, c = a.cols + 127;
  const auto rows_fit = [&](int64_t pitch) { return pitch >= 0 && pitch <= most && (r * (pitch >> 3) + (c >> 3)) <= most; };
  const auto cols_fit = [&](int64_t pitch) { return pitch >= 0 && pitch <= most && (c * (pitch >> 4) + (r >> 4)) <= most; };
  return rows_fit(a.dy_pitch) && rows_fit(a.gate_pitch) && rows_fit(a.up_pitch) && rows_fit(a.dgate_codes_pitch) &&
         rows_fit(a.dup_codes_pitch) && cols_fit(a.dgate_codes_t_pitch) && cols_fit(a.dup_codes_t_pitch) && cols_fit(a.y_codes_t_pitch) &&
         r / 128 * (c / 512 + 1) * 512 + 512 <= most && c / 128 * (r / 512 + 1) * 512 + 512 <= most;
}

template <typename T, typename S, int KIND, bool VEC>
cudaError_t backward_vec(const opt_gated_backward_args& a, int sm_count, cudaStream_t s) {
  if constexpr (sizeof(T) == 2 && sizeof(S) == 1 && VEC) {
    if (a.d_up != nullptr && a.d_dgate == nullptr && a.d_dup == nullptr && a.d_dgate_codes != nullptr && a.d_dup_codes != nullptr &&
        a.d_dgate_codes_t != nullptr && a.d_dup_codes_t != nullptr && a.d_y_codes_t != nullptr && turn_places_fit(a))
      return backward_turn<KIND>(a, sm_count, s);
  }
  if (a.d_dgate_codes_t == nullptr && a.d_dup_codes_t == nullptr && a.d_y_codes_t == nullptr) {
    const ChunkGrid g(a.rows, a.cols, kThreads);
    if constexpr (VEC) {
      if (a.d_up != nullptr) return backward_rows<T, S, KIND, true>(a, g, sm_count, s);
      return backward_rows<T, S, KIND, false>(a, g, sm_count, s);
    } else {
      gated_backward_any_kernel<T, S, KIND><<<g.grid, g.block, 0, s>>>(a);
    }
  } else {
    static OccupancyCache cache;
    const auto kernel = gated_backward_tile_kernel<T, S, KIND, VEC>;
    const int row_tiles = (int)((a.rows + 127) / 128), col_tiles = (int)((a.cols + 127) / 128);
    const int64_t tiles = (int64_t)row_tiles * col_tiles;
    const int64_t most = (int64_t)sm_count * cached_occupancy(kernel, cache, kTurnThreads, kTurnBytes);
    const int grid = (int)(tiles < most ? tiles : most);
    kernel<<<grid, kTurnThreads, kTurnBytes, s>>>(a, row_tiles, col_tiles, grid / col_tiles, grid % col_tiles);
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
  v.in_tile(a.d_dy, a.dy_pitch, sizeof(T));
  v.in_tile(a.d_gate, a.gate_pitch, sizeof(T));
  v.in_tile(a.d_up, a.up_pitch, sizeof(T));
  v.in_tile(a.d_dgate, a.dgate_pitch, sizeof(T));
  v.in_tile(a.d_dup, a.dup_pitch, sizeof(T));
  v.in_tile(a.d_dgate_codes, a.dgate_codes_pitch, 1);
  v.in_tile(a.d_dgate_codes_t, a.dgate_codes_t_pitch, 1);
  v.in_tile(a.d_dup_codes, a.dup_codes_pitch, 1);
  v.in_tile(a.d_dup_codes_t, a.dup_codes_t_pitch, 1);
  v.in_tile(a.d_y_codes_t, a.y_codes_t_pitch, 1);
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

cudaError_t launch_gated(const opt_gated_args& a, int sm_count, cudaStream_t s) {
  return a.dtype == OPT_F32 ? forward<float>(a, sm_count, s) : forward<Bf16>(a, sm_count, s);
}

cudaError_t launch_gated_backward(const opt_gated_backward_args& a, int sm_count, cudaStream_t s) {
  return a.dtype == OPT_F32 ? backward<float>(a, sm_count, s) : backward<Bf16>(a, sm_count, s);
}

}  // namespace psopt
