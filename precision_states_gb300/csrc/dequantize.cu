// dequantize.cu -- what a kept matrix becomes in the backward pass: its values, and
// its transposed operand (opt_layer.h).
//
// Mathematics: a value is its code times 2^e, exact in fp32; the transposed operand's
// scales and codes are the quantizer's for those values, in blocks along the rows.
#include "tile.cuh"

namespace psopt {
namespace {

constexpr int kThreads = 256;

// Plain values alone: a chunk to a thread.  Bound by instructions (issue 79 % busy): 16384 x 4096
// to BF16 38.5 us, 0.77 of a copy's rate, to fp32 57 us, 0.87; rows that begin anywhere 56 us.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const __grid_constant__ opt_dequantize_args a) {
  __shared__ __align__(16) Ragged<T, VEC, kThreads / 32> ragged;
  T* buffer = ragged.chunk[VEC ? 0 : (int)(threadIdx.y * blockDim.x + threadIdx.x) >> 5];
  const int64_t c = 8 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x);
  const int valid = (int)max(min(a.cols - c, (int64_t)8), (int64_t)0);
  for (int64_t r = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; r < a.rows; r += (int64_t)gridDim.y * blockDim.y) {
    const Source<E4m3, VEC> kept(a.d_codes, a.d_scales, a.codes_pitch, a.rows, a.cols, r);
    float x[8];
    kept.values(kept.ahead(c, valid), c, valid, x);
    if (!VEC || valid > 0) store_at<VEC>(a.d_x, a.x_pitch, a.cols, r, c, valid, x, buffer);
  }
}

// The transposed operand, and plain values with it: a 128 x 128 tile of codes in shared
// memory to a CTA.  A warp takes 16 columns, a lane 16 rows of four of them, two at a time:
// the column's maximum is three exchanges away, and its codes leave in whole lines.
// Word w of a tile's row (four codes) is at w with its upper three bits turned by row / 16, so
// that a warp's words (four of a row, rows 16 apart) meet in no bank.
__device__ __forceinline__ int tile_word(int row, int w) { return 32 * row + (w ^ (row >> 4 << 2)); }

// Row `row` of the tile as plain elements to a row that begins anywhere, by a warp: four elements
// to a lane, out in words (BF16 pairs that lie in one word are put together first).
__device__ __forceinline__ void tile_values(const uint32_t* codes, const float* scale, int row, float (&x)[4]) {
  const uint32_t w = codes[tile_word(row, threadIdx.x & 31)];
  e4m3x2_dec(w & 0xFFFFu, x[0], x[1]);
  e4m3x2_dec(w >> 16, x[2], x[3]);
  const f2_t factor = pk(scale[row], scale[row]);
  unpk(mul2(pk(x[0], x[1]), factor), x[0], x[1]);
  unpk(mul2(pk(x[2], x[3]), factor), x[2], x[3]);
}
__device__ __forceinline__ void put_row(float* out, const uint32_t* codes, const float* scale, int row, int cols) {
  const int e = 4 * (threadIdx.x & 31);
  float x[4];
  tile_values(codes, scale, row, x);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (e + j < cols) out[e + j] = x[j];
}
__device__ __forceinline__ void put_row(Bf16* out, const uint32_t* codes, const float* scale, int row, int cols) {
  const int lane = threadIdx.x & 31, head = (int)((uintptr_t)out >> 1) & 1;      // an element before the first whole word
  float x[4];
  tile_values(codes, scale, row, x);
  uint32_t w[3] = {bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), 0u};
  if (head && lane == 0) out[0].bits = (uint16_t)w[0];
  w[2] = __shfl_down_sync(0xFFFFFFFFu, w[0], 1);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int e = head + 4 * lane + 2 * j;
    const uint32_t pair = __funnelshift_r(w[j], w[j + 1], 16 * head);
    if (e + 1 < cols) *reinterpret_cast<uint32_t*>(out + e) = pair;
    else if (e < cols) out[e].bits = (uint16_t)pair;
  }
}

// 16 bytes to shared memory in the background, the first `left` of them from `p`, zeros then.
__device__ __forceinline__ void copy16(void* to, const uint8_t* p, int left) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               :: "r"((uint32_t)__cvta_generic_to_shared(to)), "l"(p), "r"(min(max(left, 0), 16)) : "memory");
}

// CTAs take tiles gridDim.x apart (`step_rows` and `step_cols` in tiles), the next tile's codes
// on their way while one is turned.  Three to an SM (four spill: 35 us).  Bound by instructions
// (issue 70 % busy): 16384 x 4096 turned 26.8 us, 0.74 of a copy's rate, with BF16 values 47.9,
// 0.83 (74 where their rows begin anywhere).
template <typename T, bool PLAIN, bool VEC>
__global__ void __launch_bounds__(kThreads, 3) dequantize_tile_kernel(const __grid_constant__ opt_dequantize_args a, int row_tiles,
                                                                         int col_tiles, int step_rows, int step_cols) {
  __shared__ __align__(16) uint32_t held[2][128 * 32];
  __shared__ __align__(16) float held_scale[2][128];
  const int t = threadIdx.x, lane = t & 31, row = 16 * (lane >> 2), word = 4 * (t >> 5) + (lane & 3);      // the lane's rows and columns' word
  const int64_t panel = (a.cols + 511) / 512, panel_t = (a.rows + 511) / 512;
  const uint8_t* source = static_cast<const uint8_t*>(a.d_codes) + (t >> 3) * a.codes_pitch + 16 * (t & 7);
  const uint8_t* source_scale = static_cast<const uint8_t*>(a.d_scales) + 16 * (t & 31) + 4 * ((t >> 5) & 3);
  uint8_t* target = static_cast<uint8_t*>(a.d_codes_t) + 4 * word * a.codes_t_pitch + row;
  uint8_t* target_scale = static_cast<uint8_t*>(a.d_scales_t) + 16 * ((4 * word) & 31) + 4 * (word >> 3);      // the next columns: 16 further
  uint32_t byte = 0;               // row t's scale in the tile under way
  const auto ask = [&](int tr, int tc, int turn) {
    const int rows = (int)min(a.rows - 128 * (int64_t)tr, (int64_t)128), cols = (int)min(a.cols - 128 * (int64_t)tc, (int64_t)128);
    const uint8_t* p = source + 128 * (tr * a.codes_pitch + tc);
    // rows t / 8 + 32 i, 16 codes at 16 (t mod 8)
    if (rows == 128 && cols == 128) {
#pragma unroll
      for (int i = 0; i < 4; ++i, p += 32 * a.codes_pitch) copy16(held[turn] + tile_word((t >> 3) + 32 * i, 4 * (t & 7)), p, 16);
    } else {
      // What does not exist is asked for at the matrix's own place: an address has to be aligned even
      // where nothing is copied, and the pitch of a single row may be anything.  (Rows that exist begin
      // on 16 bytes: the first does, and with a second one the pitch is a multiple of 16.)
#pragma unroll
      for (int i = 0; i < 4; ++i, p += 32 * a.codes_pitch) {
        const int left = (t >> 3) + 32 * i < rows ? cols - 16 * (t & 7) : 0;
        copy16(held[turn] + tile_word((t >> 3) + 32 * i, 4 * (t & 7)), left > 0 ? p : static_cast<const uint8_t*>(a.d_codes), left);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    byte = load_byte_if(source_scale + 512 * (tr * panel + (tc >> 2)) + (tc & 3), t < rows);
  };
  int tr = (int)blockIdx.x / col_tiles, tc = (int)blockIdx.x % col_tiles;
  ask(tr, tc, 0);
  for (int turn = 0; tr < row_tiles; turn ^= 1) {
    const int64_t r0 = 128 * (int64_t)tr, c0 = 128 * (int64_t)tc;
    const int rows = (int)min(a.rows - r0, (int64_t)128), cols = (int)min(a.cols - c0, (int64_t)128);
    uint8_t *out = target + 128 * (tc * a.codes_t_pitch + tr), *place = target_scale + 512 * (tc * panel_t + (tr >> 2)) + (tr & 3);
    const uint32_t* const codes = held[turn];
    const float* const scale = held_scale[turn];
    if (t < 128) held_scale[turn][t] = scale_of(byte);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();                 // this tile is there, and the other's place is read by nobody
    tr += step_rows;
    tc += step_cols;
    if (tc >= col_tiles) {
      tc -= col_tiles;
      ++tr;
    }
    if (tr < row_tiles) ask(tr, tc, turn ^ 1);
    if constexpr (PLAIN && VEC) {
      // a row's chunk of eight to a thread
#pragma unroll 2
      for (int i = 0; i < 8; ++i) {
        const int row = (t >> 4) + 16 * i, e = 8 * (t & 15);
        float x[8];
        values8(*reinterpret_cast<const uint2*>(codes + tile_word(row, e >> 2)), scale[row], x);
        store8_if(static_cast<T*>(a.d_x) + (r0 + row) * a.x_pitch + c0 + e, x, row < rows && e < cols);
      }
    } else if constexpr (PLAIN) {
#pragma unroll 2
      for (int row = t >> 5; row < rows; row += kThreads / 32)
        put_row(static_cast<T*>(a.d_x) + (r0 + row) * a.x_pitch + c0, codes, scale, row, cols);
    }
    const uint32_t* mine = codes + tile_word(row, word);
    float factor[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) factor[i] = scale[row + i];
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      f2_t x[16];                      // columns 2 h and 2 h + 1
      float top0 = 0.0f, top1 = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float lo, hi;
        e4m3x2_dec((mine[32 * i] >> (16 * h)) & 0xFFFFu, lo, hi);
        x[i] = mul2(pk(lo, hi), pk(factor[i], factor[i]));
      }
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        float a0, a1, b0, b1;
        unpk(x[i], a0, a1);
        unpk(x[i + 1], b0, b1);
        top0 = largest3(top0, a0, b0);
        top1 = largest3(top1, a1, b1);
      }
      const auto exchanged = [&](float v) {                 // over the column's eight lanes
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          const float other = __shfl_xor_sync(0xFFFFFFFFu, v, o);
          v = largest3(v, other, other);
        }
        return f2u(v);
      };
      uint32_t f0 = scale_field(exchanged(top0)), f1 = scale_field(exchanged(top1));
      if (__any_sync(0xFFFFFFFFu, max(f0, f1) >= kOddField)) {    // rare: the finite ones' maxima, and NaN for the others
        top0 = top1 = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float lo, hi;
          unpk(x[i], lo, hi);
          top0 = finite_bits(lo) ? fmaxf(top0, fabsf(lo)) : top0;
          top1 = finite_bits(hi) ? fmaxf(top1, fabsf(hi)) : top1;
          x[i] = pk(finite_bits(lo) ? lo : u2f(0x7FC00000u), finite_bits(hi) ? hi : u2f(0x7FC00000u));
        }
        f0 = scale_field(exchanged(top0));
        f1 = scale_field(exchanged(top1));
      }
      const f2_t inv = pk(inverse_of_field(f0), inverse_of_field(f1));
      uint32_t first[4], second[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) unpk(mul2(x[4 * k + i], inv), v[i][0], v[i][1]);
        first[k] = e4m3x2_rn(v[0][0], v[1][0]) | e4m3x2_rn(v[2][0], v[3][0]) << 16;
        second[k] = e4m3x2_rn(v[0][1], v[1][1]) | e4m3x2_rn(v[2][1], v[3][1]) << 16;
      }
      if (rows == 128 && cols == 128) {
        st_cs_u4(out, make_uint4(first[0], first[1], first[2], first[3]));
        st_cs_u4(out + a.codes_t_pitch, make_uint4(second[0], second[1], second[2], second[3]));
        store_byte_if(place, byte_of_field(f0), row == 0);
        store_byte_if(place + 16, byte_of_field(f1), row == 0);
      } else {
        const int left = cols - 4 * word - 2 * h;
        if (left > 0) store_codes16(out, first, rows - row);
        if (left > 1) store_codes16(out + a.codes_t_pitch, second, rows - row);
        store_byte_if(place, byte_of_field(f0), row == 0 && left > 0);
        store_byte_if(place + 16, byte_of_field(f1), row == 0 && left > 1);
      }
      out += 2 * a.codes_t_pitch;
      place += 32;
    }
  }
}

template <typename T, bool PLAIN, bool VEC>
cudaError_t launch_tiles(const opt_dequantize_args& a, int sm_count, cudaStream_t s) {
  static OccupancyCache cache;
  const auto kernel = dequantize_tile_kernel<T, PLAIN, VEC>;
  const int row_tiles = (int)((a.rows + 127) / 128), col_tiles = (int)((a.cols + 127) / 128);
  const int64_t tiles = (int64_t)row_tiles * col_tiles, most = (int64_t)sm_count * cached_occupancy(kernel, cache, kThreads, 0);
  const int grid = (int)(tiles < most ? tiles : most);
  kernel<<<grid, kThreads, 0, s>>>(a, row_tiles, col_tiles, grid / col_tiles, grid % col_tiles);
  return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t launch(const opt_dequantize_args& a, int sm_count, cudaStream_t s) {
  if (a.d_codes_t != nullptr) return launch_tiles<T, true, VEC>(a, sm_count, s);
  const ChunkGrid g(a.rows, a.cols, kThreads);
  dequantize_kernel<T, VEC><<<g.grid, g.block, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dequantize(const opt_dequantize_args& a, int sm_count, cudaStream_t s) {
  const int64_t es = a.dtype == OPT_F32 ? 4 : 2;
  if (a.d_x == nullptr) return launch_tiles<Bf16, false, true>(a, sm_count, s);      // the same for either type
  const bool vec = a.cols % 8 == 0 && ((uintptr_t)a.d_x & 15u) == 0 && (a.rows == 1 || a.x_pitch * es % 16 == 0);
  if (a.dtype == OPT_F32) return vec ? launch<float, true>(a, sm_count, s) : launch<float, false>(a, sm_count, s);
  return vec ? launch<Bf16, true>(a, sm_count, s) : launch<Bf16, false>(a, sm_count, s);
}

}  // namespace psopt
