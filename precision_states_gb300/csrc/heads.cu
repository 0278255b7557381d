// heads.cu -- the norm of each query and key head with the position rotation in the
// same pass, and its gradients (opt_layer.h).
//
// Mathematics: with x a head, rstd = (mean x^2 + eps)^(-1/2) and a pair's turn by
// (c, s), an output element is rstd (x w c + x' w' s') where x' and w' are its partner's
// and s' is -s for a pair's first element and s for its second.  Backward the turn is by
// (c, -s) on dout's elements: g = dout c - dout' s'.
//
// Forms, by the heads' size and place:
// - heads of 8, 16, ... 256 elements whose rows start on 16 bytes, by strips (below): eight
//   elements to a lane and 16-byte accesses;
// - other heads of at most 256 elements: an element to a lane (16384 x 40 heads of 128, kept,
//   270 us where strips take 80, their gradients at 8192 rows 351 where they take 49);
// - longer heads, to 1,024 elements: a head to a warp at a time, in shared memory.
#include <type_traits>

#include "tile.cuh"

namespace psopt {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kAnyWarps = 4;                     // of the form for any heads: 12 KB of shared memory to a warp

// Chunks of a lane after one another, and CTAs to an SM: what the registers hold.
template <typename T>
constexpr int kForwardChunks = sizeof(T) == 2 ? 4 : 2;
template <typename T>
constexpr int kBackwardChunks = sizeof(T) == 2 ? 4 : 2;
constexpr int kForwardCtas = 2, kBackwardCtas = 2;

// One side's matrices, queries' or keys'.
struct Side {
  const void *x, *scales, *dout, *weight;
  void *out, *codes, *code_scales;
  int64_t x_pitch, dout_pitch, out_pitch, codes_pitch, cols, heads;
};
// Either call as the kernels take it: sides by number (0: queries), which a CTA or a warp picks
// out of its arguments by an index.
struct HeadCall {
  Side side[2];
  const float *cos, *sin;
  const int64_t* positions;
  int64_t rows, table;
  int dim, rot;
  int32_t weight_dtype;
  bool interleaved;
  bool wide_lines;               // the tables' lines are whole 16-byte pieces
  float eps;
};
template <typename A>
HeadCall shared_call(const A& a) {
  HeadCall c = {};
  c.cos = a.d_cos;
  c.sin = a.d_sin;
  c.positions = a.d_positions;
  c.rows = a.rows;
  c.table = a.positions;
  c.dim = (int)a.dim;
  c.rot = (int)a.rot;
  c.weight_dtype = a.weight_dtype;
  c.interleaved = (a.flags & OPT_HEADS_INTERLEAVED) != 0;
  c.wide_lines = a.rot % 8 == 0 && (((uintptr_t)a.d_cos | (uintptr_t)a.d_sin) & 15u) == 0;
  c.eps = a.eps;
  return c;
}
HeadCall call_of(const opt_head_norm_args& a) {
  HeadCall c = shared_call(a);
  c.side[0] = {a.d_q, nullptr, nullptr, a.d_q_weight, a.d_q_out, a.d_q_codes, a.d_q_scales, a.q_pitch, 0, a.q_out_pitch,
               a.q_codes_pitch, a.q_heads * a.dim, a.q_heads};
  c.side[1] = {a.d_k, nullptr, nullptr, a.d_k_weight, a.d_k_out, a.d_k_codes, a.d_k_scales, a.k_pitch, 0, a.k_out_pitch,
               a.k_codes_pitch, a.k_heads * a.dim, a.k_heads};
  return c;
}
HeadCall call_of(const opt_head_norm_backward_args& a) {
  HeadCall c = shared_call(a);
  c.side[0] = {a.d_q, a.d_q_scales, a.d_dq_out, a.d_q_weight, a.d_dq, nullptr, nullptr, a.q_pitch, a.dq_out_pitch, a.dq_pitch, 0,
               a.q_heads * a.dim, a.q_heads};
  c.side[1] = {a.d_k, a.d_k_scales, a.d_dk_out, a.d_k_weight, a.d_dk, nullptr, nullptr, a.k_pitch, a.dk_out_pitch, a.dk_pitch, 0,
               a.k_heads * a.dim, a.k_heads};
  return c;
}

// head_weight_kernel may be launched once every CTA has come here; it waits for this grid's end.
__device__ __forceinline__ void let_sums_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Sum over a warp.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// How a head's elements are paired: whole chunks with whole chunks half the rotated part
// further (rot a multiple of 16; a lane's partners are another lane's words), neighbours (its
// own), or elements half the rotated part further (by way of shared memory: 16384 x 40 heads of
// 128, kept, 136 us where whole chunks take 79).
enum Pairs { kChunks = 0, kNeighbours = 1, kElements = 2 };

// The partner's words: those of lane `partner`, or with neighbouring pairs the lane's own
// with the elements of each pair exchanged.
template <bool INTERLEAVED>
__device__ __forceinline__ Raw<Bf16> partner_of(const Raw<Bf16>& x, int partner) {
  Raw<Bf16> r;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    r.w[k] = INTERLEAVED ? __byte_perm(x.w[k], 0u, 0x1032) : __shfl_sync(0xFFFFFFFFu, x.w[k], partner);
  return r;
}
template <bool INTERLEAVED>
__device__ __forceinline__ Raw<float> partner_of(const Raw<float>& x, int partner) {
  Raw<float> r;
#pragma unroll
  for (int k = 0; k < 8; ++k) r.w[k] = INTERLEAVED ? x.w[k ^ 1] : __shfl_sync(0xFFFFFFFFu, x.w[k], partner);
  return r;
}

// ------------------------------------------------- heads of whole chunks of eight elements
// A head's chunks lie side by side in a group of lanes (a power of two of them, some idle where
// dim / 8 is none), and groups side by side fill the warp: 256 columns at a time where dim is a
// power of two (DENSE), fewer else.  A strip is U times that of one side's columns, and a lane's
// chunks are that far apart.  The next row's chunk is asked for as soon as this row's is taken.
// Bound by latency at the 16 warps that the registers leave to an SM, and by instructions (issue
// 58 % busy in either direction): 16384 x 40 heads of 128 BF16, kept, 79 us, 0.79 of a copy's
// rate, without keeping 78 (0.64); gradients of 8192 from kept inputs 49 us, 0.64.  Strips half
// as wide with three CTAs to an SM take 104 and 77 us.
// Heads of 96 leave a quarter of the lanes idle: 16384 x 52 of them 114 us, 0.43.  Lanes to a head
// by number (LANES) spare 3 to 7 % against the same at run time.

// N sums over groups of lanes (LANES of them, or where that is 0 `lanes`), their exchanges side by side.
template <int LANES, int N>
__device__ __forceinline__ void lanes_sums(float (&v)[N], int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (LANES > 0 ? o < LANES : o < lanes) {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
    }
  }
}
__device__ __forceinline__ void shared8(const float* p, float (&x)[8]) {
  const float4 lo = *reinterpret_cast<const float4*>(p), hi = *reinterpret_cast<const float4*>(p + 4);
  x[0] = lo.x; x[1] = lo.y; x[2] = lo.z; x[3] = lo.w;
  x[4] = hi.x; x[5] = hi.y; x[6] = hi.z; x[7] = hi.w;
}
// A warp's cosines and sines: this row's and the next one's lines of the tables, copied to
// shared memory in the background (in registers, asked for a row ahead, they cost the
// gradients spills; asked for when needed, the wait for them).
struct TurnLines {
  float line[2][2][128];         // [turn][cosines, sines][pair]
  // By the whole warp: the lines at position `at`, NaN outside the tables.
  __device__ __forceinline__ void ask(int turn, const HeadCall& a, int64_t at) {
    const int lane = threadIdx.x & 31, half = a.rot >> 1;
    if ((uint64_t)at >= (uint64_t)a.table) {
      const float nan = u2f(0x7FC00000u);
      for (int i = lane; i < half; i += 32) line[turn][0][i] = line[turn][1][i] = nan;
    } else if (a.wide_lines) {
      const int64_t p = at * half + 4 * lane;
      if (4 * lane < half) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;"
                     :: "r"((uint32_t)__cvta_generic_to_shared(&line[turn][0][4 * lane])), "l"(a.cos + p) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;"
                     :: "r"((uint32_t)__cvta_generic_to_shared(&line[turn][1][4 * lane])), "l"(a.sin + p) : "memory");
      }
    } else {
      for (int i = lane; i < half; i += 32) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;"
                     :: "r"((uint32_t)__cvta_generic_to_shared(&line[turn][0][i])), "l"(a.cos + (at * half + i)) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;"
                     :: "r"((uint32_t)__cvta_generic_to_shared(&line[turn][1][i])), "l"(a.sin + (at * half + i)) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // All but the lines asked for last are there.
  __device__ __forceinline__ void wait() const {
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
  }
  // The factors of a lane's eight elements, from e of the head and its pair on.  For elements
  // that are not rotated (whole: all are) they are 1 and 0, or with whole chunks, where such an
  // element is its own partner, 1/2 and 1/2: the halves' sum rounds as the product with 1.
  template <int PAIRS>
  __device__ __forceinline__ void factors(int turn, int e, int pair, int rot, bool whole, float (&c)[8], float (&s)[8]) const {
    if constexpr (PAIRS == kNeighbours) {
      const float4 cv = *reinterpret_cast<const float4*>(&line[turn][0][pair]), sv = *reinterpret_cast<const float4*>(&line[turn][1][pair]);
      c[0] = c[1] = cv.x; c[2] = c[3] = cv.y; c[4] = c[5] = cv.z; c[6] = c[7] = cv.w;
      s[0] = s[1] = sv.x; s[2] = s[3] = sv.y; s[4] = s[5] = sv.z; s[6] = s[7] = sv.w;
    } else if constexpr (PAIRS == kChunks) {
      shared8(&line[turn][0][pair], c);
      shared8(&line[turn][1][pair], s);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = e + j < (rot >> 1) ? e + j : e + j < rot ? e + j - (rot >> 1) : 0;
        c[j] = line[turn][0][at];
        s[j] = line[turn][1][at];
      }
    }
    if (!whole) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        c[j] = e + j < rot ? c[j] : PAIRS == kChunks ? 0.5f : 1.0f;
        s[j] = e + j < rot ? s[j] : PAIRS == kChunks ? 0.5f : 0.0f;
      }
    }
  }
};
// The partners of a lane's eight elements v (raw its words): another lane's words, its own, or
// by way of the warp's 256 floats at `held`, in which a head's elements lie side by side.  For
// elements that are not rotated: themselves with whole chunks, else 0, so that the product with
// s = 0 is 0 for infinities too.
template <int PAIRS, typename T>
__device__ __forceinline__ void partners_of(const Raw<T>& raw, const float (&v)[8], int partner, int e, int rot, bool whole,
                                            float* held, float (&p)[8]) {
  if constexpr (PAIRS != kElements) {
    Raw<T> r = partner_of<PAIRS == kNeighbours>(raw, partner);
    if (PAIRS == kNeighbours && !whole) {
      constexpr int kWords = sizeof(r.w) / sizeof(r.w[0]);      // (a word's elements are rotated or not together)
#pragma unroll
      for (int k = 0; k < kWords; ++k) r.w[k] = e + 8 / kWords * k < rot ? r.w[k] : 0u;
    }
    unpack(r, p);
  } else {
    const int lane = threadIdx.x & 31, half = rot >> 1;
    const float* head = held + (8 * lane - e);
    __syncwarp();                  // what was there is read
    *reinterpret_cast<float4*>(held + 8 * lane) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(held + 8 * lane + 4) = make_float4(v[4], v[5], v[6], v[7]);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = e + j >= rot ? 0.0f : head[e + j < half ? e + j + half : e + j - half];
  }
}
// How CTAs share strips: CTA b takes strip b mod (strips), and of its rows a warp each
// (b / strips) * kWarps + warp, and `stride` on.  Strips of queries come first.
struct Strips {
  int q_strips, strips;
  uint32_t stride;
  int lanes;                     // lanes to a head
};
// Columns from a lane's chunk to its next one.
template <bool DENSE>
__device__ __forceinline__ uint32_t chunk_step(const Strips& strips, int dim) { return DENSE ? 256u : (uint32_t)(32 / strips.lanes * dim); }
// What a lane is in its strip.
struct StripLane {
  uint32_t column, left;         // its first, in the side; what is there from it on (0 for an idle lane)
  uint32_t row;                  // its warp's first
  int e, pair, partner;          // of its first element: in the head, its angle; the lane with the partners
  bool rotated;
};
template <bool DENSE, int U>
__device__ __forceinline__ StripLane strip_lane(const Strips& strips, int strip, int64_t cols, int dim, int rot, bool interleaved) {
  StripLane l;
  const int lane = threadIdx.x & 31, half = rot >> 1;
  const uint32_t first = (uint32_t)strip * (chunk_step<DENSE>(strips, dim) * U);
  l.row = (blockIdx.x / (uint32_t)strips.strips) * kWarps + (threadIdx.x >> 5);
  l.e = DENSE ? (8 * lane) & (dim - 1) : 8 * (lane & (strips.lanes - 1));
  l.column = first + (DENSE ? 8 * lane : lane / strips.lanes * dim + l.e);
  l.left = !DENSE && l.e >= dim ? 0u : (uint32_t)cols - min(l.column, (uint32_t)cols);
  l.rotated = l.e < rot;
  l.pair = !l.rotated ? 0 : interleaved ? l.e >> 1 : l.e < half ? l.e : l.e - half;
  l.partner = !l.rotated ? lane : lane + (l.e < half ? half >> 3 : -(half >> 3));
  return l;
}
__device__ __forceinline__ float weight_at(const void* weight, int32_t type, int e) {
  return type == OPT_F32 ? static_cast<const float*>(weight)[e] : element(static_cast<const Bf16*>(weight) + e);
}
// Scale byte of a row, from its strip's first block on.
__device__ __forceinline__ uint64_t scale_row(uint32_t r, uint32_t panel512) {
  return (uint64_t)(r >> 7) * panel512 + (16 * (r & 31) + ((r >> 3) & 12));
}

template <typename T, int PAIRS, bool KEEP, bool DENSE, int LANES, int U>
__global__ void __launch_bounds__(kThreads, kForwardCtas) head_norm_strip_kernel(const __grid_constant__ HeadCall a,
                                                                                const Strips strips) {
  // the weight, and its partner's with the sign of the partner's term (minus for a pair's
  // first element)
  __shared__ __align__(16) float weight[256], other[256];
  __shared__ __align__(16) TurnLines lines_of[kWarps];
  TurnLines& lines = lines_of[threadIdx.x >> 5];
  __shared__ __align__(16) float rows_of[PAIRS == kElements ? kWarps : 1][256];
  float* const held = rows_of[PAIRS == kElements ? threadIdx.x >> 5 : 0];
  const int dim = a.dim, rot = a.rot, half = rot >> 1, strip = (int)(blockIdx.x % (uint32_t)strips.strips);
  const bool keys = strip >= strips.q_strips;
  const Side& side = a.side[keys];
  const StripLane l = strip_lane<DENSE, U>(strips, keys ? strip - strips.q_strips : strip, side.cols, dim, rot, PAIRS == kNeighbours);
  if ((int)threadIdx.x < dim) {
    const int e = threadIdx.x, p = e >= rot ? e : PAIRS == kNeighbours ? e ^ 1 : e < half ? e + half : e - half;
    const float v = weight_at(side.weight, a.weight_dtype, p);
    weight[e] = weight_at(side.weight, a.weight_dtype, e);
    other[e] = (PAIRS == kNeighbours ? (e & 1) == 0 : e < half) ? -v : v;
  }
  __syncthreads();
  const uint32_t rows = (uint32_t)a.rows, panel = 512 * (uint32_t)((side.cols + 511) / 512);
  const uint32_t left = l.left, step = chunk_step<DENSE>(strips, dim);      // chunk k exists where k step is below left
  const uint32_t place = 512 * (l.column >> 9) + ((l.column >> 7) & 3);
  const float inv_dim = 1.0f / (float)dim;
  const bool keep = KEEP && side.codes != nullptr;
  if (l.row >= rows) return;
  Raw<T> x[U];
#pragma unroll
  for (int k = 0; k < U; ++k) x[k] = load_if(static_cast<const T*>(side.x) + (l.row * side.x_pitch + l.column) + step * k, step * k < left);
  const auto position = [&](uint32_t r) { return a.positions == nullptr ? (int64_t)r : r < rows ? a.positions[r] : (int64_t)0; };
  int64_t at = 0;
  if (rot > 0) {
    lines.ask(0, a, position(l.row));
    at = position(l.row + strips.stride);
  }
  int turn = 0;
  for (uint32_t r = l.row; r < rows; r += strips.stride, turn ^= 1) {
    const uint32_t next = r + strips.stride;
    if (rot > 0) {
      __syncwarp();              // the lines of the row before are read
      lines.ask(turn ^ 1, a, next < rows ? at : -1);
      at = position(next + strips.stride);
    }
    float c[8], s[8], w[8];
    shared8(weight + l.e, w);
    if (rot > 0) {
      lines.wait();
      lines.template factors<PAIRS>(turn, l.e, l.pair, rot, rot == dim, c, s);
      times8(c, w);
      shared8(other + l.e, w);
      times8(s, w);
    }
    T* const out = static_cast<T*>(side.out) + (r * side.out_pitch + l.column);
    uint8_t* const codes = static_cast<uint8_t*>(side.codes) + (r * side.codes_pitch + l.column);
    uint8_t* const scales = static_cast<uint8_t*>(side.code_scales) + (scale_row(r, panel) + place);
    const T* const ahead = static_cast<const T*>(side.x) + (next * side.x_pitch + l.column);
#pragma unroll
    for (int k = 0; k < U; k += 2) {      // two chunks' exchanges side by side
      const Raw<T> raw[2] = {x[k], x[k + 1]};
      x[k] = load_if(ahead + step * k, step * k < left && next < rows);
      x[k + 1] = load_if(ahead + step * (k + 1), step * (k + 1) < left && next < rows);
      float rstd[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v[8];
        unpack(raw[i], v);
        f2_t sums = 0;                    // +0 in both lanes
#pragma unroll
        for (int j = 0; j < 8; j += 2) sums = fma2(pk(v[j], v[j + 1]), pk(v[j], v[j + 1]), sums);
        float second;
        unpk(sums, rstd[i], second);
        rstd[i] += second;
      }
      uint32_t top[2] = {0u, 0u};
      if (keep) {
        top[0] = top_of(magnitudes(raw[0], false));
        top[1] = top_of(magnitudes(raw[1], false));
        tops16(top[0], top[1], T());
      }
      lanes_sums<LANES, 2>(rstd, strips.lanes);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool on = step * (k + i) < left;
        const float root = reciprocal_root(fmaf(rstd[i], inv_dim, a.eps));
        const f2_t scale = pk(root, root);
        float v[8], y[8];
        unpack(raw[i], v);
        if (rot > 0) {
          float p[8];
          partners_of<PAIRS>(raw[i], v, l.partner, l.e, rot, rot == dim, held, p);
#pragma unroll
          for (int j = 0; j < 8; j += 2)
            unpk(mul2(fma2(pk(v[j], v[j + 1]), pk(c[j], c[j + 1]), mul2(pk(p[j], p[j + 1]), pk(s[j], s[j + 1]))), scale), y[j], y[j + 1]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; j += 2) unpk(mul2(mul2(pk(v[j], v[j + 1]), pk(w[j], w[j + 1])), scale), y[j], y[j + 1]);
        }
        store8_if(out + step * (k + i), y, on);
        if (keep) {
          uint8_t* to = scales + (512 * (k >> 1) + 2 * i);      // blocks 2 (k + i) and the next of the strip
          if (__any_sync(0xFFFFFFFFu, top[i] >= kInfBits)) put_codes8(codes + step * (k + i), to, 0, on ? 8 : 0, v);
          else put_finite_if(codes + step * (k + i), to, v, top[i], on, on && (threadIdx.x & 15) == 0);
        }
      }
    }
  }
}

// The gradients of strips.
template <typename T, typename S, int PAIRS, bool DENSE, int LANES, int U>
__global__ void __launch_bounds__(kThreads, kBackwardCtas) head_norm_backward_strip_kernel(
    const __grid_constant__ HeadCall a, const Strips strips, float* parts) {
  __shared__ float sums[kWarps][32][8];
  __shared__ __align__(16) TurnLines lines_of[kWarps];
  TurnLines& lines = lines_of[threadIdx.x >> 5];
  __shared__ __align__(16) float rows_of[PAIRS == kElements ? kWarps : 1][256];
  float* const held = rows_of[PAIRS == kElements ? threadIdx.x >> 5 : 0];
  if (parts != nullptr) let_sums_start();
  constexpr bool KEPT = sizeof(S) == 1;
  const int dim = a.dim, rot = a.rot, strip = (int)(blockIdx.x % (uint32_t)strips.strips);
  const bool keys = strip >= strips.q_strips;
  const Side& side = a.side[keys];
  const StripLane l = strip_lane<DENSE, U>(strips, keys ? strip - strips.q_strips : strip, side.cols, dim, rot, PAIRS == kNeighbours);
  const uint32_t rows = (uint32_t)a.rows, panel = 512 * (uint32_t)((side.cols + 511) / 512);
  const uint32_t left = l.left, step = chunk_step<DENSE>(strips, dim);
  const uint32_t place = 512 * (l.column >> 9) + ((l.column >> 7) & 3);
  const float inv_dim = 1.0f / (float)dim;
  float w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = DENSE || l.e < dim ? weight_at(side.weight, a.weight_dtype, l.e + j) : 0.0f;
  f2_t dw[4] = {};                 // +0 in both lanes
  // the turn back: plus for a pair's first element
  const float sign = PAIRS == kChunks && l.rotated && l.e >= (rot >> 1) ? -1.0f : 1.0f;
  const f2_t signs = pk(sign, PAIRS == kNeighbours ? -1.0f : sign);
  Raw<T> d[U];
  std::conditional_t<KEPT, KeptAsk, Raw<T>> x[U];
  const auto load = [&](int k, uint32_t r) {
    const bool on = step * k < left && r < rows;
    d[k] = load_if(static_cast<const T*>(side.dout) + (r * side.dout_pitch + l.column) + step * k, on);
    if constexpr (KEPT) {
      x[k].codes = load_codes_if(static_cast<const uint8_t*>(side.x) + (r * side.x_pitch + l.column) + step * k, on);
      // a dense strip's chunks are two blocks apart
      const uint32_t c = l.column + step * k, block = DENSE ? place + (512 * (k >> 1) + 2 * (k & 1)) : 512 * (c >> 9) + ((c >> 7) & 3);
      x[k].byte = load_byte_if(static_cast<const uint8_t*>(side.scales) + scale_row(r, panel) + block, on);
    } else {
      x[k] = load_if(static_cast<const T*>(side.x) + (r * side.x_pitch + l.column) + step * k, on);
    }
  };
#pragma unroll
  for (int k = 0; k < U; ++k) load(k, l.row);
  const auto position = [&](uint32_t r) { return a.positions == nullptr ? (int64_t)r : r < rows ? a.positions[r] : (int64_t)0; };
  int64_t at = 0;
  if (rot > 0 && l.row < rows) {
    lines.ask(0, a, position(l.row));
    at = position(l.row + strips.stride);
  }
  int turn = 0;
  for (uint32_t r = l.row; r < rows; r += strips.stride, turn ^= 1) {
    const uint32_t next = r + strips.stride;
    if (rot > 0) {
      __syncwarp();              // the lines of the row before are read
      lines.ask(turn ^ 1, a, next < rows ? at : -1);
      at = position(next + strips.stride);
      lines.wait();
    }
    const auto input = [&](int k, float (&v)[8]) {
      if constexpr (KEPT) values8(x[k].codes, scale_of(x[k].byte), v);
      else unpack(x[k], v);
    };
    T* const out = static_cast<T*>(side.out) + (r * side.out_pitch + l.column);
    float c[8], s[8];
    if (rot > 0) {
      lines.template factors<PAIRS>(turn, l.e, l.pair, rot, rot == dim, c, s);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        if constexpr (PAIRS == kElements) {
          s[j] = l.e + j < (rot >> 1) ? s[j] : -s[j];
          s[j + 1] = l.e + j + 1 < (rot >> 1) ? s[j + 1] : -s[j + 1];
        } else {
          unpk(mul2(pk(s[j], s[j + 1]), signs), s[j], s[j + 1]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const bool on = step * k < left;
      const Raw<T> raw = d[k];
      float v[8], g[8];
      input(k, v);
      load(k, next);
      unpack(raw, g);
      if (rot > 0) {
        float p[8];
        partners_of<PAIRS>(raw, g, l.partner, l.e, rot, rot == dim, held, p);
#pragma unroll
        for (int j = 0; j < 8; j += 2)
          unpk(fma2(pk(g[j], g[j + 1]), pk(c[j], c[j + 1]), mul2(pk(p[j], p[j + 1]), pk(s[j], s[j + 1]))), g[j], g[j + 1]);
      }
      f2_t squares = 0, dots = 0, t[4];      // t = g weight
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2_t xv = pk(v[2 * j], v[2 * j + 1]);
        squares = fma2(xv, xv, squares);
        t[j] = mul2(pk(g[2 * j], g[2 * j + 1]), pk(w[2 * j], w[2 * j + 1]));
        dots = fma2(t[j], xv, dots);
      }
      float sum[2], second, other;
      unpk(squares, sum[0], second);
      unpk(dots, sum[1], other);
      sum[0] += second;
      sum[1] += other;
      lanes_sums<LANES, 2>(sum, strips.lanes);
      const float root = reciprocal_root(fmaf(sum[0], inv_dim, a.eps)), pull = -root * root * (sum[1] * inv_dim);
      float dx[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2_t xv = pk(v[2 * j], v[2 * j + 1]);
        if (on) dw[j] = fma2(pk(g[2 * j], g[2 * j + 1]), mul2(xv, pk(root, root)), dw[j]);
        unpk(mul2(fma2(xv, pk(pull, pull), t[j]), pk(root, root)), dx[2 * j], dx[2 * j + 1]);
      }
      store8_if(out + step * k, dx, on);
    }
  }
  if (parts == nullptr) return;
  float sum[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) unpk(dw[j], sum[2 * j], sum[2 * j + 1]);
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[threadIdx.x >> 5][threadIdx.x & 31][j] = sum[j];
  __syncthreads();
  float* row = parts + (int64_t)blockIdx.x * 2 * dim;
  for (int t = threadIdx.x; t < 2 * dim; t += kThreads) {
    float v = 0.0f;
    if ((t >= dim) == keys) {
      const int e = keys ? t - dim : t;
      for (int k = 0; k < kWarps; ++k)
        for (int i = 0; i < 32; i += strips.lanes) v += sums[k][i + (e >> 3)][e & 7];
    }
    row[t] = v;
  }
}

// ------------------------------------------------------- heads of any size and place
// By single elements.  An element of a row, of a plain matrix or a kept one:
template <typename T>
__device__ __forceinline__ float element_at(const Side& side, int64_t r, int64_t col, int64_t panel, T) {
  return element(static_cast<const T*>(side.x) + r * side.x_pitch + col);
}
__device__ __forceinline__ float element_at(const Side& side, int64_t r, int64_t col, int64_t panel, E4m3) {
  const uint32_t byte = static_cast<const uint8_t*>(side.scales)[scale_place(r, col >> 7, panel)];
  float lo, hi;
  e4m3x2_dec(static_cast<const uint8_t*>(side.x)[r * side.x_pitch + col], lo, hi);
  return lo * scale_of(byte);
}
__device__ __forceinline__ void put_element(Bf16* p, float v) { p->bits = (uint16_t)bf16_pair(v, 0.0f); }
__device__ __forceinline__ void put_element(float* p, float v) { *p = v; }

// The turn of element j: its partner, c and s'; false outside the rotated ones.
__device__ __forceinline__ bool turn_at(const float* cos, const float* sin, int64_t at, int64_t table, int rot, bool interleaved,
                                        int j, int& partner, float& c, float& s) {
  if (j >= rot) return false;
  const int half = rot >> 1;
  const bool second = interleaved ? (j & 1) : j >= half;
  const int pair = interleaved ? j >> 1 : second ? j - half : j;
  partner = interleaved ? j ^ 1 : second ? j - half : j + half;
  if (at < 0 || at >= table) {
    c = s = u2f(0x7FC00000u);
  } else {
    c = cos[at * half + pair];
    s = sin[at * half + pair];
  }
  if (!second) s = -s;
  return true;
}

// Heads of at most 32 N elements: element j of a head is lane j mod 32's, and a warp takes
// `group` heads of a row after one another, so that the angles and the weight stay in
// registers; the next head is asked for while this one is taken.  Partners meet in shared
// memory, whose last place holds the 0 that elements without a partner meet.  Bound by
// instructions on single elements: 16384 x 50 heads of 100 168 us, 0.29 of a copy's rate,
// gradients of 4096 137, 0.13 (by the kernels for longer heads 575 and 339).
template <int N>
struct LaneTurn {
  int partner[N];
  float c[N], s[N];
  __device__ __forceinline__ void set(const HeadCall& a, int64_t r) {
    const int64_t at = a.rot > 0 && a.positions != nullptr ? a.positions[r] : r;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      partner[i] = 32 * N;
      c[i] = 1.0f;
      s[i] = 0.0f;
      turn_at(a.cos, a.sin, at, a.table, a.rot, a.interleaved, (int)(threadIdx.x & 31) + 32 * i, partner[i], c[i], s[i]);
    }
  }
};
template <int N, typename F>
__device__ __forceinline__ void lane_elements(int dim, float (&v)[N], F f) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int j = (int)(threadIdx.x & 31) + 32 * i;
    v[i] = j < dim ? f(j) : 0.0f;
  }
}

template <typename T, typename W, int N>
__global__ void __launch_bounds__(kThreads, N <= 4 ? 4 : 2) head_norm_lanes_kernel(const __grid_constant__ HeadCall a, int group) {
  __shared__ float held_by[kWarps][32 * N + 1];
  float* held = held_by[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31, dim = a.dim;
  if (lane == 0) held[32 * N] = 0.0f;
  const int64_t q_groups = (a.side[0].heads + group - 1) / group, groups = q_groups + (a.side[1].heads + group - 1) / group;
  const int64_t n = a.rows * groups;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); t < n; t += (int64_t)gridDim.x * kWarps) {
    const int64_t r = t / groups, both = t % groups;
    const bool keys = both >= q_groups;
    const Side& side = a.side[keys];
    const int64_t first = (keys ? both - q_groups : both) * group;
    const int heads = (int)(side.heads - first < group ? side.heads - first : group);
    const T* from = static_cast<const T*>(side.x) + r * side.x_pitch + first * dim;
    T* out = static_cast<T*>(side.out) + r * side.out_pitch + first * dim;
    LaneTurn<N> turn;
    turn.set(a, r);
    float w[N], ahead[N];
    lane_elements<N>(dim, w, [&](int j) { return element(static_cast<const W*>(side.weight) + j); });
    lane_elements<N>(dim, ahead, [&](int j) { return element(from + j); });
    for (int h = 0; h < heads; ++h, out += dim) {
      float x[N], sum = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = ahead[i];
      from += dim;
      if (h + 1 < heads) lane_elements<N>(dim, ahead, [&](int j) { return element(from + j); });
#pragma unroll
      for (int i = 0; i < N; ++i) {
        sum = fmaf(x[i], x[i], sum);
        x[i] *= w[i];
        held[lane + 32 * i] = x[i];
      }
      sum = warp_sum(sum);
      const float rstd = reciprocal_root(fmaf(sum, 1.0f / (float)dim, a.eps));
      __syncwarp();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float y = fmaf(x[i], turn.c[i], held[turn.partner[i]] * turn.s[i]);
        if (lane + 32 * i < dim) put_element(out + lane + 32 * i, rstd * y);
      }
      __syncwarp();              // the partners are read
    }
  }
}

// Their gradients: the first q_ctas CTAs take queries, the others keys.
template <typename T, typename S, typename W, int N>
__global__ void __launch_bounds__(kThreads, N <= 4 ? 3 : 2) head_norm_backward_lanes_kernel(
    const __grid_constant__ HeadCall a, int group, int q_ctas, float* parts) {
  __shared__ float held_by[kWarps][32 * N + 1];
  if (parts != nullptr) let_sums_start();
  float* held = held_by[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31, dim = a.dim;
  if (lane == 0) held[32 * N] = 0.0f;
  const bool keys = (int)blockIdx.x >= q_ctas;
  const Side& side = a.side[keys];
  const int64_t cta = keys ? blockIdx.x - q_ctas : blockIdx.x, ctas = keys ? gridDim.x - q_ctas : q_ctas;
  const int64_t groups = (side.heads + group - 1) / group, n = a.rows * groups, panel = (side.cols + 511) / 512;
  float w[N], dw[N];
  lane_elements<N>(dim, w, [&](int j) { return element(static_cast<const W*>(side.weight) + j); });
#pragma unroll
  for (int i = 0; i < N; ++i) dw[i] = 0.0f;
  for (int64_t t = cta * kWarps + (threadIdx.x >> 5); t < n; t += ctas * kWarps) {
    const int64_t r = t / groups, first = t % groups * group;
    const int heads = (int)(side.heads - first < group ? side.heads - first : group);
    int64_t col = first * dim;
    const T* dout = static_cast<const T*>(side.dout) + r * side.dout_pitch;
    T* out = static_cast<T*>(side.out) + r * side.out_pitch;
    LaneTurn<N> turn;
    turn.set(a, r);
    float x_ahead[N], d_ahead[N];
    const auto ask = [&](int64_t c) {
      lane_elements<N>(dim, x_ahead, [&](int j) { return element_at(side, r, c + j, panel, S()); });
      lane_elements<N>(dim, d_ahead, [&](int j) { return element(dout + c + j); });
    };
    ask(col);
    for (int h = 0; h < heads; ++h, col += dim) {
      float x[N], g[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[i] = x_ahead[i];
        g[i] = d_ahead[i];
      }
      if (h + 1 < heads) ask(col + dim);
#pragma unroll
      for (int i = 0; i < N; ++i) held[lane + 32 * i] = g[i];
      __syncwarp();
      float square = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        g[i] = fmaf(g[i], turn.c[i], -held[turn.partner[i]] * turn.s[i]);
        square = fmaf(x[i], x[i], square);
        dot = fmaf(g[i] * w[i], x[i], dot);
      }
      square = warp_sum(square);          // (and the partners are read)
      dot = warp_sum(dot);
      const float rstd = reciprocal_root(fmaf(square, 1.0f / (float)dim, a.eps));
      const float pull = rstd * rstd * (dot * (1.0f / (float)dim));
#pragma unroll
      for (int i = 0; i < N; ++i) {
        dw[i] = fmaf(g[i], x[i] * rstd, dw[i]);
        if (lane + 32 * i < dim) put_element(out + col + lane + 32 * i, rstd * fmaf(-x[i], pull, g[i] * w[i]));
      }
      __syncwarp();
    }
  }
  if (parts == nullptr) return;
#pragma unroll
  for (int i = 0; i < N; ++i) held[lane + 32 * i] = dw[i];
  __syncthreads();
  for (int t = threadIdx.x; t < 2 * dim; t += kThreads) {
    float v = 0.0f;
    if ((t >= dim) == keys)
      for (int k = 0; k < kWarps; ++k) v += held_by[k][t >= dim ? t - dim : t];
    parts[(int64_t)blockIdx.x * 2 * dim + t] = v;
  }
}

// Heads of more elements (8192 x 20 heads of 300 225 us, 0.14 of a copy's rate; not made faster,
// since attention heads are shorter).
template <typename T, typename W>
__global__ void __launch_bounds__(32 * kAnyWarps) head_norm_any_kernel(const __grid_constant__ HeadCall a) {
  __shared__ float held[kAnyWarps][kHeadMaxDim];
  float* x = held[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31, dim = a.dim, rot = a.rot;
  const int64_t heads = a.side[0].heads + a.side[1].heads, n = a.rows * heads;
  for (int64_t i = (int64_t)blockIdx.x * kAnyWarps + (threadIdx.x >> 5); i < n; i += (int64_t)gridDim.x * kAnyWarps) {
    const int64_t r = i / heads, both = i % heads;
    const Side& side = a.side[both >= a.side[0].heads];
    const int64_t col = (both >= a.side[0].heads ? both - a.side[0].heads : both) * dim;
    const W* weight = static_cast<const W*>(side.weight);
    const int64_t at = rot > 0 && a.positions != nullptr ? a.positions[r] : r;
    float sum = 0.0f;
#pragma unroll 4
    for (int j = lane; j < dim; j += 32) {
      const float v = element_at(side, r, col + j, 0, T());
      x[j] = v;
      sum = fmaf(v, v, sum);
    }
    sum = warp_sum(sum);
    const float rstd = reciprocal_root(fmaf(sum, 1.0f / (float)dim, a.eps));
    __syncwarp();
#pragma unroll 4
    for (int j = lane; j < dim; j += 32) {
      int p = j;
      float c, s, y = x[j] * element(weight + j);
      if (turn_at(a.cos, a.sin, at, a.table, rot, a.interleaved, j, p, c, s))
        y = fmaf(y, c, x[p] * element(weight + p) * s);
      put_element(static_cast<T*>(side.out) + r * side.out_pitch + col + j, rstd * y);
    }
    __syncwarp();
  }
}

// The weights' gradients of a warp's heads are summed in shared memory, queries' first and
// then, in a launch's second half of CTAs, keys' (`q_ctas` CTAs take queries).
template <typename T, typename S, typename W>
__global__ void __launch_bounds__(32 * kAnyWarps) head_norm_backward_any_kernel(
    const __grid_constant__ HeadCall a, int q_ctas, float* parts) {
  __shared__ float held[kAnyWarps][2][kHeadMaxDim];
  __shared__ float sums[kAnyWarps][kHeadMaxDim];
  if (parts != nullptr) let_sums_start();
  const int wi = threadIdx.x >> 5, lane = threadIdx.x & 31, dim = a.dim, rot = a.rot;
  float *x = held[wi][0], *d = held[wi][1], *dw = sums[wi];
  const bool keys = (int)blockIdx.x >= q_ctas;
  const Side& side = a.side[keys];
  const int64_t cta = keys ? blockIdx.x - q_ctas : blockIdx.x, ctas = keys ? gridDim.x - q_ctas : q_ctas;
  const int64_t n = a.rows * side.heads, panel = (side.cols + 511) / 512;
  const W* weight = static_cast<const W*>(side.weight);
  for (int j = lane; j < dim; j += 32) dw[j] = 0.0f;
  for (int64_t i = cta * kAnyWarps + wi; i < n; i += ctas * kAnyWarps) {
    const int64_t r = i / side.heads, col = i % side.heads * dim;
    const int64_t at = rot > 0 && a.positions != nullptr ? a.positions[r] : r;
#pragma unroll 4
    for (int j = lane; j < dim; j += 32) {
      x[j] = element_at(side, r, col + j, panel, S());
      d[j] = element(static_cast<const T*>(side.dout) + r * side.dout_pitch + col + j);
    }
    __syncwarp();
    const auto turned = [&](int j) {
      int p = j;
      float c, s;
      return turn_at(a.cos, a.sin, at, a.table, rot, a.interleaved, j, p, c, s)
                 ? fmaf(d[j], c, -d[p] * s) : d[j];
    };
    float square = 0.0f, dot = 0.0f;
#pragma unroll 4
    for (int j = lane; j < dim; j += 32) {
      square = fmaf(x[j], x[j], square);
      dot = fmaf(turned(j) * element(weight + j), x[j], dot);
    }
    square = warp_sum(square);
    dot = warp_sum(dot);
    const float rstd = reciprocal_root(fmaf(square, 1.0f / (float)dim, a.eps));
    const float pull = rstd * rstd * (dot * (1.0f / (float)dim));
#pragma unroll 4
    for (int j = lane; j < dim; j += 32) {
      const float g = turned(j);
      dw[j] = fmaf(g, x[j] * rstd, dw[j]);
      put_element(static_cast<T*>(side.out) + r * side.out_pitch + col + j, rstd * fmaf(-x[j], pull, g * element(weight + j)));
    }
    __syncwarp();
  }
  if (parts == nullptr) return;
  __syncthreads();
  for (int t = threadIdx.x; t < 2 * dim; t += 32 * kAnyWarps) {
    float v = 0.0f;
    if ((t >= dim) == keys)
      for (int k = 0; k < kAnyWarps; ++k) v += sums[k][t >= dim ? t - dim : t];
    parts[(int64_t)blockIdx.x * 2 * dim + t] = v;
  }
}

// The weights' gradients: the partial sums' rows in a fixed order, 32 columns to a CTA.  Thread
// row p takes rows p, p + 32, ..., ten loads at a time; then a warp each column's 32 sums.
// Launched while the rows' kernel still runs, it waits for that one's end.
constexpr int kSumCols = 32, kSumParts = 32;
__global__ void __launch_bounds__(kSumCols * kSumParts) head_weight_kernel(const float* parts, int n, int dim, float* dq, float* dk) {
  __shared__ float sums[kSumParts][kSumCols + 1];
  const int x = threadIdx.x % kSumCols, p0 = threadIdx.x / kSumCols, t = blockIdx.x * kSumCols + x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s = 0.0f;
  if (t < 2 * dim) {
    for (int p = p0; p < n; p += 10 * kSumParts) {
      float v[10];
#pragma unroll
      for (int i = 0; i < 10; ++i) v[i] = p + i * kSumParts < n ? parts[(int64_t)(p + i * kSumParts) * 2 * dim + t] : 0.0f;
#pragma unroll
      for (int i = 0; i < 10; ++i) s += v[i];
    }
  }
  sums[p0][x] = s;
  __syncthreads();
  s = warp_sum(sums[x][p0]);          // column p0's
  const int c = blockIdx.x * kSumCols + p0;
  if (x != 0 || c >= 2 * dim) return;
  if (c < dim) {
    if (dq != nullptr) dq[c] = s;
  } else if (dk != nullptr) {
    dk[c - dim] = s;
  }
}

// Whether heads are at most 256 elements, whole chunks of eight that start on 16 bytes.
struct Whole {
  int64_t rows;
  bool ok;
  void see(const void* p, int64_t pitch, int64_t es) {
    ok = ok && ((uintptr_t)p & 15u) == 0 && (rows == 1 || pitch * es % 16 == 0);
  }
};
template <typename A>
Pairs pairs_of(const A& a) {
  return a.flags & OPT_HEADS_INTERLEAVED ? kNeighbours : a.rot % 16 == 0 ? kChunks : kElements;
}

// Strips of U chunks, and their CTAs: as many for each as its rows fill, within `most` in all.
template <typename A>
Strips strips_of(const A& a, int u, int64_t most, int64_t* ctas) {
  Strips s;
  s.lanes = 1;
  while (8 * s.lanes < a.dim) s.lanes *= 2;
  const int64_t width = 32 / s.lanes * a.dim * u;
  s.q_strips = (int)((a.q_heads * a.dim + width - 1) / width);
  s.strips = s.q_strips + (int)((a.k_heads * a.dim + width - 1) / width);
  const int64_t need = (a.rows + kWarps - 1) / kWarps, have = most / s.strips;
  const int64_t each = need <= have ? need : have > 0 ? have : 1;
  s.stride = (uint32_t)(each * kWarps);
  *ctas = each * s.strips;
  return s;
}

template <typename T, int PAIRS, bool KEEP, bool DENSE, int LANES>
cudaError_t forward_strip(const opt_head_norm_args& a, int sm_count, cudaStream_t s) {
  static OccupancyCache cache;
  const auto kernel = head_norm_strip_kernel<T, PAIRS, KEEP, DENSE, LANES, kForwardChunks<T>>;
  int64_t ctas;
  const Strips strips = strips_of(a, kForwardChunks<T>, (int64_t)sm_count * cached_occupancy(kernel, cache, kThreads, 0), &ctas);
  kernel<<<(unsigned)ctas, kThreads, 0, s>>>(call_of(a), strips);
  return cudaGetLastError();
}
// The commonest groups of lanes by their number; others find theirs at run time.
template <typename T, int PAIRS, bool KEEP>
cudaError_t forward_strips(const opt_head_norm_args& a, int sm_count, cudaStream_t s) {
  if constexpr (PAIRS != kElements) {
    if (a.dim == 64) return forward_strip<T, PAIRS, KEEP, true, 8>(a, sm_count, s);
    if (a.dim == 128) return forward_strip<T, PAIRS, KEEP, true, 16>(a, sm_count, s);
  }
  return forward_strip<T, PAIRS, KEEP, true, 0>(a, sm_count, s);
}
template <typename T, int PAIRS>
cudaError_t forward_sparse_strips(const opt_head_norm_args& a, int sm_count, cudaStream_t s) {
  if constexpr (PAIRS != kElements) {
    if (a.dim > 64 && a.dim < 128) return forward_strip<T, PAIRS, false, false, 16>(a, sm_count, s);
  }
  return forward_strip<T, PAIRS, false, false, 0>(a, sm_count, s);
}

cudaError_t keep(const void* x, int64_t x_pitch, void* codes, void* scales, int64_t pitch, int64_t rows, int64_t cols,
                 int32_t dtype, cudaStream_t s) {
  if (codes == nullptr || cols == 0) return cudaSuccess;
  opt_quantize_args q = {};
  q.d_x = x;
  q.d_codes = codes;
  q.d_scales = scales;
  q.x_pitch = x_pitch;
  q.codes_pitch = pitch;
  q.rows = rows;
  q.cols = cols;
  q.dtype = dtype;
  q.block_rows = 1;
  return launch_quantize(q, s);
}

// Heads that a warp takes after one another: one while there are fewer heads than warps, at
// most eight.
int lane_group(int64_t heads, int sm_count) {
  const int64_t each = heads / ((int64_t)sm_count * 2 * kWarps);
  return each < 1 ? 1 : each > 8 ? 8 : (int)each;
}

template <typename T, typename W, int N>
cudaError_t forward_lanes(const opt_head_norm_args& a, int sm_count, cudaStream_t s) {
  static OccupancyCache cache;
  const auto kernel = head_norm_lanes_kernel<T, W, N>;
  const int group = lane_group(a.rows * (a.q_heads + a.k_heads), sm_count);
  const int64_t tasks = a.rows * ((a.q_heads + group - 1) / group + (a.k_heads + group - 1) / group);
  const int64_t need = (tasks + kWarps - 1) / kWarps, most = (int64_t)sm_count * cached_occupancy(kernel, cache, kThreads, 0);
  kernel<<<(unsigned)(need < most ? need : most), kThreads, 0, s>>>(call_of(a), group);
  return cudaGetLastError();
}

template <typename T, typename W>
cudaError_t forward(const opt_head_norm_args& a, int sm_count, cudaStream_t s) {
  Whole v{a.rows, a.dim % 8 == 0 && a.dim <= 256};
  if (a.q_heads > 0) {
    v.see(a.d_q, a.q_pitch, sizeof(T));
    v.see(a.d_q_out, a.q_out_pitch, sizeof(T));
  }
  if (a.k_heads > 0) {
    v.see(a.d_k, a.k_pitch, sizeof(T));
    v.see(a.d_k_out, a.k_out_pitch, sizeof(T));
  }
  opt_head_norm_args b = a;
  // blocks of 128 go with groups of lanes only where heads are of 8, 16, ... 256 elements;
  // else the quantizer keeps the inputs (before an output may take their place)
  if (!v.ok || (a.dim & (a.dim - 1)) != 0) {
    cudaError_t e = keep(a.d_q, a.q_pitch, a.d_q_codes, a.d_q_scales, a.q_codes_pitch, a.rows, a.q_heads * a.dim, a.dtype, s);
    if (e == cudaSuccess)
      e = keep(a.d_k, a.k_pitch, a.d_k_codes, a.d_k_scales, a.k_codes_pitch, a.rows, a.k_heads * a.dim, a.dtype, s);
    if (e != cudaSuccess) return e;
    b.d_q_codes = b.d_k_codes = nullptr;
  }
  if (v.ok && (a.dim & (a.dim - 1)) == 0) {
    const bool kept = b.d_q_codes != nullptr || b.d_k_codes != nullptr;
    switch (pairs_of(a)) {
      case kChunks: return kept ? forward_strips<T, kChunks, true>(b, sm_count, s) : forward_strips<T, kChunks, false>(b, sm_count, s);
      case kNeighbours: return kept ? forward_strips<T, kNeighbours, true>(b, sm_count, s) : forward_strips<T, kNeighbours, false>(b, sm_count, s);
      default: return kept ? forward_strips<T, kElements, true>(b, sm_count, s) : forward_strips<T, kElements, false>(b, sm_count, s);
    }
  }
  if (v.ok) {
    switch (pairs_of(a)) {
      case kChunks: return forward_sparse_strips<T, kChunks>(b, sm_count, s);
      case kNeighbours: return forward_sparse_strips<T, kNeighbours>(b, sm_count, s);
      default: return forward_sparse_strips<T, kElements>(b, sm_count, s);
    }
  }
  const int64_t heads = a.q_heads + a.k_heads;
  if (a.dim <= 64) return forward_lanes<T, W, 2>(b, sm_count, s);
  if (a.dim <= 128) return forward_lanes<T, W, 4>(b, sm_count, s);
  if (a.dim <= 256) return forward_lanes<T, W, 8>(b, sm_count, s);
  const int64_t need = (a.rows * heads + kAnyWarps - 1) / kAnyWarps, most = (int64_t)sm_count * 12;
  head_norm_any_kernel<T, W><<<(unsigned)(need < most ? need : most), 32 * kAnyWarps, 0, s>>>(call_of(b));
  return cudaGetLastError();
}

cudaError_t weight_sums(const opt_head_norm_backward_args& a, int ctas, cudaStream_t s) {
  if (a.d_dq_weight == nullptr && a.d_dk_weight == nullptr) return cudaGetLastError();
  cudaLaunchAttribute early = {};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3((unsigned)((2 * a.dim + kSumCols - 1) / kSumCols));
  config.blockDim = dim3(kSumCols * kSumParts);
  config.stream = s;
  config.attrs = &early;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, head_weight_kernel, static_cast<const float*>(a.d_workspace), ctas, (int)a.dim, a.d_dq_weight,
                            a.d_dk_weight);
}

// CTAs of `warps` warps for either side, which take `group` heads at a time: as many as the
// side's share of the heads in `most`, and within the workspace's rows.
struct SideCtas {
  int q, all;
};
SideCtas side_ctas(const opt_head_norm_backward_args& a, int group, int warps, int64_t most) {
  if (most > kHeadBackwardMaxCtas - 1) most = kHeadBackwardMaxCtas - 1;      // (shares are rounded up)
  const int64_t heads = a.q_heads + a.k_heads;
  const auto ctas_of = [&](int64_t h) {
    const int64_t need = (a.rows * ((h + group - 1) / group) + warps - 1) / warps, share = (most * h + heads - 1) / heads;
    return (int)(need < share ? need : share);
  };
  const int q = ctas_of(a.q_heads);
  return {q, q + ctas_of(a.k_heads)};
}
template <typename T, typename S, typename W, int N>
cudaError_t backward_lanes(const opt_head_norm_backward_args& a, int sm_count, float* parts, cudaStream_t s) {
  static OccupancyCache cache;
  const auto kernel = head_norm_backward_lanes_kernel<T, S, W, N>;
  const int group = lane_group(a.rows * (a.q_heads + a.k_heads), sm_count);
  const SideCtas ctas = side_ctas(a, group, kWarps, (int64_t)sm_count * cached_occupancy(kernel, cache, kThreads, 0));
  kernel<<<(unsigned)ctas.all, kThreads, 0, s>>>(call_of(a), group, ctas.q, parts);
  if (const cudaError_t e = cudaGetLastError()) return e;
  return weight_sums(a, ctas.all, s);
}
template <typename T, typename S, typename W>
cudaError_t backward_any(const opt_head_norm_backward_args& a, int sm_count, float* parts, cudaStream_t s) {
  if (a.dim <= 64) return backward_lanes<T, S, W, 2>(a, sm_count, parts, s);
  if (a.dim <= 128) return backward_lanes<T, S, W, 4>(a, sm_count, parts, s);
  if (a.dim <= 256) return backward_lanes<T, S, W, 8>(a, sm_count, parts, s);
  // three to an SM: a fourth's shared memory leaves L1 too little for the tables (4096 x 20 heads of
  // 300 400 us for 293; of 1024 147 either way)
  const SideCtas ctas = side_ctas(a, 1, kAnyWarps, (int64_t)sm_count * 3);
  head_norm_backward_any_kernel<T, S, W><<<(unsigned)ctas.all, 32 * kAnyWarps, 0, s>>>(call_of(a), ctas.q, parts);
  if (const cudaError_t e = cudaGetLastError()) return e;
  return weight_sums(a, ctas.all, s);
}

template <typename T, typename S, int PAIRS, bool DENSE, int LANES>
cudaError_t backward_strip(const opt_head_norm_backward_args& a, int sm_count, float* parts, cudaStream_t s) {
  static OccupancyCache cache;
  const auto kernel = head_norm_backward_strip_kernel<T, S, PAIRS, DENSE, LANES, kBackwardChunks<T>>;
  int64_t most = (int64_t)sm_count * cached_occupancy(kernel, cache, kThreads, 0), ctas;
  if (most > kHeadBackwardMaxCtas) most = kHeadBackwardMaxCtas;
  const Strips strips = strips_of(a, kBackwardChunks<T>, most, &ctas);
  kernel<<<(unsigned)ctas, kThreads, 0, s>>>(call_of(a), strips, parts);
  if (const cudaError_t e = cudaGetLastError()) return e;
  return weight_sums(a, (int)ctas, s);
}
template <typename T, typename S, int PAIRS>
cudaError_t backward_strips(const opt_head_norm_backward_args& a, int sm_count, float* parts, cudaStream_t s) {
  const bool dense = (a.dim & (a.dim - 1)) == 0;
  if constexpr (PAIRS != kElements) {
    if (a.dim == 64) return backward_strip<T, S, PAIRS, true, 8>(a, sm_count, parts, s);
    if (a.dim == 128) return backward_strip<T, S, PAIRS, true, 16>(a, sm_count, parts, s);
    if (a.dim > 64 && a.dim < 128) return backward_strip<T, S, PAIRS, false, 16>(a, sm_count, parts, s);
  }
  return dense ? backward_strip<T, S, PAIRS, true, 0>(a, sm_count, parts, s) : backward_strip<T, S, PAIRS, false, 0>(a, sm_count, parts, s);
}

template <typename T, typename S, typename W>
cudaError_t backward_from(const opt_head_norm_backward_args& a, int sm_count, cudaStream_t s) {
  Whole v{a.rows, a.dim % 8 == 0 && a.dim <= 256};
  constexpr bool kept = sizeof(S) == 1;
  if (a.q_heads > 0) {
    if (!kept) v.see(a.d_q, a.q_pitch, sizeof(T));
    v.see(a.d_dq_out, a.dq_out_pitch, sizeof(T));
    v.see(a.d_dq, a.dq_pitch, sizeof(T));
  }
  if (a.k_heads > 0) {
    if (!kept) v.see(a.d_k, a.k_pitch, sizeof(T));
    v.see(a.d_dk_out, a.dk_out_pitch, sizeof(T));
    v.see(a.d_dk, a.dk_pitch, sizeof(T));
  }
  float* parts = a.d_dq_weight != nullptr || a.d_dk_weight != nullptr ? static_cast<float*>(a.d_workspace) : nullptr;
  // (a strip of either side needs a row of the workspace; more than it has go by single heads)
  if (v.ok && (a.q_heads + a.k_heads) * a.dim <= (kHeadBackwardMaxCtas - 2) * 128) {
    switch (pairs_of(a)) {
      case kChunks: return backward_strips<T, S, kChunks>(a, sm_count, parts, s);
      case kNeighbours: return backward_strips<T, S, kNeighbours>(a, sm_count, parts, s);
      default: return backward_strips<T, S, kElements>(a, sm_count, parts, s);
    }
  }
  return backward_any<T, S, W>(a, sm_count, parts, s);
}

template <typename T, typename W>
cudaError_t backward(const opt_head_norm_backward_args& a, int sm_count, cudaStream_t s) {
  return a.d_q_scales != nullptr || a.d_k_scales != nullptr ? backward_from<T, E4m3, W>(a, sm_count, s)
                                                            : backward_from<T, T, W>(a, sm_count, s);
}

}  // namespace

cudaError_t launch_head_norm(const opt_head_norm_args& a, int sm_count, cudaStream_t s) {
  if (a.dtype == OPT_F32)
    return a.weight_dtype == OPT_F32 ? forward<float, float>(a, sm_count, s) : forward<float, Bf16>(a, sm_count, s);
  return a.weight_dtype == OPT_F32 ? forward<Bf16, float>(a, sm_count, s) : forward<Bf16, Bf16>(a, sm_count, s);
}

cudaError_t launch_head_norm_backward(const opt_head_norm_backward_args& a, int sm_count, cudaStream_t s) {
  if (a.dtype == OPT_F32)
    return a.weight_dtype == OPT_F32 ? backward<float, float>(a, sm_count, s) : backward<float, Bf16>(a, sm_count, s);
  return a.weight_dtype == OPT_F32 ? backward<Bf16, float>(a, sm_count, s) : backward<Bf16, Bf16>(a, sm_count, s);
}

}  // namespace psopt
