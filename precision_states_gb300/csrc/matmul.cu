// matmul.cu -- out = a b^T (+ addend) of two E4M3 operands with a scale for each
// block of 128 along the depth (opt_layer.h).
//
// Mathematics: out = sum over blocks of 2^(ea + eb) times the block's sum of code
// products.  The scales are powers of two in the tensor core's own scale format,
// so tcgen05.mma (kind mxf8f6f4, block scaled) applies them as it multiplies:
// each 32-deep instruction takes one scale byte per row of either operand, and
// the four instructions of a 128-deep block take the same one.  Sums stay in the
// accumulator's fp32 over the whole depth.
//
// Roles.  The kernel computes x y^T tiles of 128 rows of x per CTA (the tensor
// memory's lanes) by NT rows of y (its columns); either operand of the call can
// be x (`swap`), so that few rows on either side become a narrow NT and not a
// mostly empty 128.  Warp 0 fills a ring of stages (128 bytes of depth of both
// tiles, 128-byte swizzle; every fourth stage the 512-byte scale tiles too) by
// TMA; warp 1 copies scale tiles to tensor memory and issues the products; warps
// 4-11 read finished accumulators and write out.  Two
// accumulators alternate, so that a tile's output overlaps the next one's
// products.  At NT 256 they share 24 columns (two of 256 and two sets of scales
// do not fit into 512): the output reads those first, and the next tile's
// products wait for that alone.
//
// CG 2: a pair of CTAs works on one tile of 256 x NT (cta_group::2): each holds
// its 128 rows of x and half of y's rows, which halves y's traffic and shared
// memory per product.
//
// Splits.  With few tiles, the depth is split over a cluster of CTAs; their
// accumulators are summed through distributed shared memory in rank order.
//
// Bound: 8192 x 14336 x 4096 takes 268 to 288 us alone, by the GPU (3.3 to 3.6
// PFLOP/s; tensor pipe 86 % busy), and 322 us in a loop, where the 1,360 W cap holds
// the clock at 1,490 MHz.
// The same loop with no loads takes 227 us: a pair's 256 x 256 tile brings 33 KB
// to each SM per block, about what its path from L2 carries in the products' time,
// and a tile's end costs the next one about 1 us.  Few tiles are latency: about 3
// us of launch and first loads, then a block's time each (0.16 us of a 16-wide
// tile to 0.32 of a pair's 256).
//
// Every wait is bounded (by the global timer): one that runs out raises
// OPT_FLAG_WAIT_TIMEOUT (opt_layer_status), and the CTA leaves after its copies
// and products in flight have ended.
#include <cuda.h>

#include "matmul.h"

namespace psopt {
namespace {

constexpr int kThreads = 384;
constexpr int kOutWarps = 8;           // two for each 32 lanes of tensor memory, half of the columns each
constexpr unsigned long long kWaitNs = 2000000000ull, kDrillNs = 1000000ull;
constexpr int kScaleTile = 512;        // bytes: 128 rows x 4 blocks
constexpr int kStageDepth = 128;
constexpr int kRingBytes = 204 * 1024;

__device__ int g_flags;

struct MatmulArgs : OutputArgs {
  int nx, ny;                // rows of x and of y
  int x_tiles, y_tiles;
  int blocks;                // ceil(k / 128)
  int panel;                 // scale tiles per 128 rows: ceil(blocks / 4)
  int split;                 // CTAs per cluster along the depth (CG 1)
  int wide;                  // rows of out allow 32-byte stores (NT 256: 16-byte copies), of the addend 32-byte loads
  int drill;                 // load nothing, so that the waits run out
  unsigned long long wait_ns;   // limit of each wait
};

template <int CG, int NT>
struct Layout {
  static constexpr int kY = NT / CG;                                   // rows of y per CTA
  static constexpr int kYScaleTiles = (NT + 127) / 128;
  static constexpr int kXBytes = 128 * kStageDepth, kYBytes = kY * kStageDepth;
  static constexpr int kScaleBytes = (1 + kYScaleTiles) * kScaleTile;
  static constexpr int kStage = kXBytes + (kYBytes + 1023) / 1024 * 1024;
  static constexpr int kFit = kRingBytes / (kStage + kScaleBytes);
  static constexpr int kStages = kFit < 12 ? kFit : 12;
  // tensor memory columns: two accumulators, two sets of scales (x: 4, y: 4 per 128 rows)
  static constexpr bool kOverlap = NT == 256;
  static constexpr int kScaleCols = 4 + 4 * kYScaleTiles;
  static constexpr int kAcc1 = kOverlap ? 256 - 2 * kScaleCols : NT;
  static constexpr int kScaleCol = kAcc1 + NT;
  static constexpr int kNeed = kScaleCol + 2 * kScaleCols;
  static constexpr int kCols = kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
  static constexpr int kBars = 2 * kStages + 5;      // full, empty, done[2], free[2], drain
  // columns that an output warp takes at a time (64 bytes of the widest tile's), and
  // the output warps' shared memory, 32 rows of 64 bytes each
  template <typename T>
  static constexpr int kOutCols = NT == 256 ? 64 / (int)sizeof(T) : NT >= 64 ? 32 : 16;
  static constexpr int kOutBytes = kOutWarps * 32 * 64;
  // dynamic shared memory: ring | scales | output | barriers, tensor memory address, failure
  static constexpr int kScaleAt = kStages * kStage;
  static constexpr int kOutAt = kScaleAt + kStages * kScaleBytes;
  static constexpr int kBarAt = kOutAt + kOutBytes;
  static constexpr int kBytes = kBarAt + kBars * 8 + 16 + 1024;        // 1024: alignment of the ring
  static_assert(kNeed <= 512, "tensor memory");
  static_assert(kBytes <= 227 * 1024, "shared memory");
  static_assert((NT + 4) * 128 * 4 <= kScaleAt || CG == 2, "split sums fit into the ring");
};

// ------------------------------------------------------------------ barriers
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, unsigned long long limit_ns) {
  if (bar_try(bar, parity)) return true;
  const unsigned long long t0 = now_ns();
  while (!bar_try(bar, parity))
    if (now_ns() - t0 > limit_ns) return false;
  return true;
}
// The same by a whole warp, with one verdict, so that what follows is uniform.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, unsigned long long limit_ns) {
  return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, limit_ns));
}
// One lane of a converged warp, always the same one.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ------------------------------------------------------- copies and products
template <int CG>
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}

// Shared-memory matrix descriptors: rows of 128 bytes, 128-byte swizzle, groups
// of 8 rows 1024 bytes apart; and scale tiles, not swizzled, 8 rows of 16 bytes
// in 128 bytes.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}
// Instruction descriptor: E4M3 by E4M3, both with the depth along their rows,
// E8M0 scales, M = 128 CG, N = NT; the scale byte of both operands.
template <int CG, int NT>
__device__ __forceinline__ uint32_t instr_desc(uint32_t byte) {
  return (byte << 4) | ((uint32_t)(NT >> 3) << 17) | (1u << 23) | ((uint32_t)CG << 27) | (byte << 29);
}
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  if (CG == 1) asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
  else asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
template <int CG>
__device__ __forceinline__ void product(uint32_t acc, uint64_t x, uint64_t y, uint32_t instr, uint32_t sx, uint32_t sy,
                                        uint32_t add) {
  if (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(acc), "l"(x), "l"(y), "r"(instr), "r"(sx), "r"(sy), "r"(add) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(acc), "l"(x), "l"(y), "r"(instr), "r"(sx), "r"(sy), "r"(add) : "memory");
}
// An arrival on `bar` (of both CTAs of a pair) when everything issued has ended.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if (CG == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(bar), "h"((uint16_t)3) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// N consecutive accumulator columns of this warp's 32 lanes (N 16 or 32).
template <int N>
__device__ __forceinline__ void acc_load(uint32_t tmem, float (&v)[N]) {
  uint32_t r[N];
  if constexpr (N == 32) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
        "%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(tmem));
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(tmem));
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = u2f(r[i]);
}

// -------------------------------------------------------------------- output
// Whether N columns from y0 on leave and arrive in wide pieces: they exist, and rows
// of out (and of the addend) allow it.
__device__ __forceinline__ bool whole(const MatmulArgs& a, int n, int y0) { return a.wide && y0 + n <= a.ny; }

// The addend of a thread's N outputs (row x of the tile, columns y0 .. y0 + N - 1),
// where its rows allow 32-byte loads or, `swap`, lie along the lanes.  It is loaded
// before the accumulator is read, so that its latency is paid once.
template <typename T, int N>
struct Addend {
  static constexpr int kWords = N * (int)sizeof(T) / 4;
  uint32_t add[kWords];

  __device__ __forceinline__ void load(const MatmulArgs& a, int x, int y0) {
    if (a.addend == nullptr || x >= a.nx || (!a.swap && !whole(a, N, y0))) return;
    const T* p = static_cast<const T*>(a.addend);
    if (!a.swap) {
      p += place(a, a.addend_pitch, x, y0);
#pragma unroll
      for (int i = 0; i < kWords; i += 8)
        asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(add[i]), "=r"(add[i + 1]), "=r"(add[i + 2]), "=r"(add[i + 3]), "=r"(add[i + 4]),
                       "=r"(add[i + 5]), "=r"(add[i + 6]), "=r"(add[i + 7])
                     : "l"(reinterpret_cast<const uint32_t*>(p) + i));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t v = bits_if(p + place(a, a.addend_pitch, x, y0 + i), y0 + i < a.ny);
        if (sizeof(T) == 4) add[i] = v;
        else if (i & 1) add[i >> 1] |= v;
        else add[i >> 1] = v >> 16;
      }
    }
  }
  __device__ __forceinline__ void sum(const MatmulArgs& a, int x, float (&v)[N]) const {
    if (a.addend == nullptr || x >= a.nx) return;
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] += sizeof(T) == 4 ? u2f(add[i]) : u2f(i & 1 ? add[i >> 1] & 0xFFFF0000u : add[i >> 1] << 16);
  }
};

// Each lane's outputs by itself: `swap`, where a store's lanes lie along a row of
// out; else N whole columns in 32-byte stores (a sector each).
template <typename T, int N>
__device__ __forceinline__ void store_lanes(const MatmulArgs& a, int x, int y0, const float (&v)[N]) {
  if (x >= a.nx) return;
  T* p = static_cast<T*>(a.out);
  if (!a.swap) {
    constexpr int kWords = N * (int)sizeof(T) / 4;
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = f2u(v[i]);
      else w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    }
    uint32_t* q = reinterpret_cast<uint32_t*>(p + place(a, a.out_pitch, x, y0));
#pragma unroll
    for (int i = 0; i < kWords; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                   ::"l"(q + i), "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]),
                     "r"(w[i + 6]), "r"(w[i + 7]) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (y0 + i < a.ny) put(p + place(a, a.out_pitch, x, y0 + i), v[i]);
  }
}

// A warp's 32 rows of N outputs and their addend in rows of any place: 16 columns
// at a time through the warp's shared memory (16-byte pieces turned as below), then
// lanes along the rows, two at a time, so that a store or load covers pieces of
// rows and not one element in each of 32.
template <typename T, int N>
__device__ __forceinline__ void store_spread(const MatmulArgs& a, uint32_t buffer, int lane, int row0, int col0,
                                             const float (&v)[N]) {
  const int c = lane & 15, r0 = lane >> 4;
  uint32_t add[N];                    // the addend, all of it on its way at once
  if (a.addend != nullptr) {
#pragma unroll
    for (int part = 0; part < N; part += 16) {
      const int col = col0 + part + c, rows = col < a.ny ? a.nx - row0 - r0 : 0;       // rows from r0 on
      const T* p = static_cast<const T*>(a.addend) + place(a, a.addend_pitch, row0 + r0, col);
#pragma unroll
      for (int k = 0; k < 16; ++k, p += 2 * a.addend_pitch) add[part + k] = bits_if(p, 2 * k < rows);
    }
  }
#pragma unroll
  for (int part = 0; part < N; part += 16) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");      // a copy before has read it
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};"
                   ::"r"(buffer + 64 * lane + 16 * (i ^ ((lane >> 1) & 3))), "f"(v[part + 4 * i]),
                     "f"(v[part + 4 * i + 1]), "f"(v[part + 4 * i + 2]), "f"(v[part + 4 * i + 3]) : "memory");
    __syncwarp();
    const int col = col0 + part + c, rows = col < a.ny ? a.nx - row0 - r0 : 0;
    T* out = static_cast<T*>(a.out) + place(a, a.out_pitch, row0 + r0, col);
    float s[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int r = 2 * k + r0;
      asm volatile("ld.shared.f32 %0, [%1];"
                   : "=f"(s[k]) : "r"(buffer + 64 * r + 16 * ((c >> 2) ^ ((r >> 1) & 3)) + 4 * (c & 3)));
    }
#pragma unroll
    for (int k = 0; k < 16; ++k, out += 2 * a.out_pitch)
      if (2 * k < rows) put(out, a.addend != nullptr ? s[k] + u2f(add[part + k]) : s[k]);
    __syncwarp();
  }
}

// A warp's 32 rows of 64 bytes, by TMA from its 2 KB of shared memory (64-byte
// swizzle: 16-byte pieces turned by half the row, so that neither side meets
// bank conflicts).  Rows beyond the matrix are left out by the copy; columns would
// be only in pieces of 16 bytes, so a row's ragged end goes another way.
// For the widest tile, whose lines a warp leaves in four or eight pieces: 8192 x
// 2304 x 768 took 18.0 us with each lane storing its own row, 16.6 this way (17.0 to 17.6 on other GPUs);
// 1024 x 4096 x 8191 to fp32 32.7 and 31.3.  Narrower tiles gain nothing: 256 x
// 4096 x 4096 in tiles of 128 took 9.7 us by lanes, 9.8 this way.
template <typename T, int N>
__device__ __forceinline__ void store_staged(const CUtensorMap* map, uint32_t buffer, int lane, int row0, int col0,
                                             bool exists, const float (&v)[N]) {
  static_assert(N * sizeof(T) == 64, "a row of the buffer");
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if constexpr (sizeof(T) == 4) w[i] = f2u(v[i]);
    else w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
  }
  // the copy before has read the buffer
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
  const uint32_t row = buffer + 64 * lane, turn = (lane >> 1) & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};"
                 ::"r"(row + 16 * (i ^ turn)), "r"(w[4 * i]), "r"(w[4 * i + 1]), "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                 : "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0 && exists) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"(map), "r"(col0), "r"(row0), "r"(buffer) : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

// A place in the ring: its stage, the phase of its barriers, and whether the ring
// is still in its first turn.
template <int S>
struct Ring {
  uint32_t stage = 0, phase = 0;
  bool first = true;
  __device__ __forceinline__ void next() {
    if (++stage == S) {
      stage = 0;
      phase ^= 1u;
      first = false;
    }
  }
};

// Tile t of the grid: panels of kGroup x tiles go through all y tiles, so that
// the tiles in flight share operands in L2.  8192 x 14336 x 4096 in a loop under
// the power cap: panels of 2, 4, 8, 16, 32 took 335, 340, 328, 322, 318 us.
constexpr int kGroup = 32;
__device__ __forceinline__ void tile_at(const MatmulArgs& a, int t, int& tx, int& ty) {
  const int per = kGroup * a.y_tiles, g = t / per, in = t - g * per;
  const int high = min(kGroup, a.x_tiles - g * kGroup);
  ty = in / high;
  tx = g * kGroup + in - ty * high;
}

template <typename T, int CG, int NT>
__global__ void __launch_bounds__(kThreads, 1)
matmul_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_y,
              const __grid_constant__ CUtensorMap map_sx, const __grid_constant__ CUtensorMap map_sy,
              const __grid_constant__ CUtensorMap map_out, const __grid_constant__ MatmulArgs a) {
  using L = Layout<CG, NT>;
  constexpr int S = L::kStages;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  const uint32_t ring = smem_addr(smem), scales = ring + L::kScaleAt, bars = ring + L::kBarAt;
  const uint32_t full = bars, empty = full + 8 * S, done = empty + 8 * S, free_ = done + 16, drain = free_ + 16;
  volatile uint32_t* tmem_at = reinterpret_cast<volatile uint32_t*>(smem + L::kBarAt + 8 * L::kBars);
  volatile uint32_t* failed = tmem_at + 1;
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const bool clustered = CG == 2 || a.split > 1;
  const uint32_t rank = clustered ? cta_rank() : 0;

  // this CTA's tiles and its part of the depth (in blocks, from a multiple of 4)
  const int per = CG == 2 ? 2 : a.split;
  const int tiles = a.x_tiles * a.y_tiles;
  const int first = blockIdx.x / per, step = gridDim.x / per;
  int kb0 = 0, kb1 = a.blocks;
  if (CG == 1 && a.split > 1) {
    kb0 = 4 * (int)((int64_t)a.panel * rank / a.split);
    kb1 = min(a.blocks, 4 * (int)((int64_t)a.panel * (rank + 1) / a.split));
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      bar_init(full + 8 * i, 1);
      bar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(done + 8 * i, 1);
      bar_init(free_ + 8 * i, kOutWarps * CG);
    }
    bar_init(drain, 1);
    *failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 3 && lane < (NT == 256 ? 5 : 4)) {
    const CUtensorMap* maps[5] = {&map_x, &map_y, &map_sx, &map_sy, &map_out};
    asm volatile("prefetch.tensormap [%0];" ::"l"(maps[lane]) : "memory");
  }
  if (warp == 2) {
    if (CG == 1) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                   ::"r"(smem_addr((const void*)tmem_at)), "r"(L::kCols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                   ::"r"(smem_addr((const void*)tmem_at)), "r"(L::kCols) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
  }
  fence_before();
  __syncthreads();
  if (clustered) cluster_sync();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_at, 0);

  const bool counts = CG == 1 || rank == 0;      // copies end on this CTA's barriers
  Ring<S> at;
  if (warp == 0) {
    // ------------------------------------------------------------- producer
    // A pair's copies all count on the leader's barrier.  This warp and the next
    // pace the ring, so their loops carry their state (stage, phase, addresses)
    // from block to block, and the whole warp runs them, one lane issuing: what
    // is the same in all lanes stays in uniform registers, which the copies and
    // products take their operands from.  (16 x 4096 x 14336: 39.0 us with one
    // thread that divided per block, 28.7 with its state carried, 20.4 by a warp.)
    const uint32_t full_at = CG == 2 ? map_to(full, 0) : full;
    constexpr uint32_t kBytes = CG * (L::kXBytes + L::kYBytes), kScales = CG * L::kScaleBytes;
    const bool issues = elected();
    bool ok = true;
    for (int t = a.drill ? tiles : first; t < tiles && ok; t += step) {
      int tx, ty;
      tile_at(a, t, tx, ty);
      const int x0 = (tx * CG + (CG == 2 ? (int)rank : 0)) * 128, y0 = ty * NT;
      const int y_row = y0 + (CG == 2 ? (int)rank * L::kY : 0);
      int sx = (x0 >> 7) * a.panel + (kb0 >> 2), sy = (y0 >> 7) * a.panel + (kb0 >> 2);
      for (int kb = kb0; kb < kb1; kb += 4, ++sx, ++sy) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (kb + j >= kb1) break;
          if (!at.first && !warp_wait(empty + 8 * at.stage, at.phase ^ 1u, a.wait_ns)) {
            ok = false;
            break;
          }
          const uint32_t bar = full_at + 8 * at.stage, dst = ring + at.stage * L::kStage;
          if (issues) {
            if (counts) bar_expect(full + 8 * at.stage, j == 0 ? kBytes + kScales : kBytes);
            if (j == 0) {
              const uint32_t sd = scales + at.stage * L::kScaleBytes;
              tma_2d<CG>(sd, &map_sx, 0, sx, bar);
#pragma unroll
              for (int i = 0; i < L::kYScaleTiles; ++i)
                tma_2d<CG>(sd + (1 + i) * kScaleTile, &map_sy, 0, sy + i * a.panel, bar);
            }
            tma_2d<CG>(dst, &map_x, (kb + j) * kStageDepth, x0, bar);
            tma_2d<CG>(dst + L::kXBytes, &map_y, (kb + j) * kStageDepth, y_row, bar);
          }
          __syncwarp();
          at.next();
        }
        if (!ok) break;
      }
    }
    if (!ok) *failed = 1;
  } else if (warp == 1 && counts) {
    // ------------------------------------------------------------- products
    const uint64_t x_desc = tile_desc(ring), y_desc = tile_desc(ring + L::kXBytes), s_desc = scale_desc(scales);
    const bool issues = elected();
    int i = 0;
    uint32_t set = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step, ++i) {
      const uint32_t acc = tmem + (i & 1) * L::kAcc1;
      // (overlapping accumulators: the release of the tile before, else of the one before that)
      if (L::kOverlap ? (i >= 1 && !warp_wait(free_ + 8 * ((i - 1) & 1), (uint32_t)((i - 1) >> 1) & 1u, a.wait_ns))
                      : (i >= 2 && !warp_wait(free_ + 8 * (i & 1), (uint32_t)((i >> 1) - 1) & 1u, a.wait_ns))) {
        ok = false;
        break;
      }
      fence_after();
      uint32_t add = 0;
      for (int kb = kb0; kb < kb1; kb += 4) {
        set = L::kScaleCols - set;                       // the two sets in turn
        const uint32_t col = tmem + L::kScaleCol + set;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (kb + j >= kb1) break;
          if (!warp_wait(full + 8 * at.stage, at.phase, a.wait_ns)) {
            ok = false;
            break;
          }
          fence_after();
          if (issues) {
            if (j == 0) {
              const uint64_t sd = s_desc + at.stage * (L::kScaleBytes >> 4);
#pragma unroll
              for (int k = 0; k <= L::kYScaleTiles; ++k) copy_scales<CG>(col + 4 * k, sd + k * (kScaleTile >> 4));
            }
            const uint64_t dx = x_desc + at.stage * (L::kStage >> 4), dy = y_desc + at.stage * (L::kStage >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              product<CG>(acc, dx + 2 * k, dy + 2 * k, instr_desc<CG, NT>(j), col, col + 4, k > 0 ? 1u : add);
            commit<CG>(empty + 8 * at.stage);
          }
          __syncwarp();
          add = 1;
          at.next();
        }
        if (!ok) break;
      }
      if (ok && issues) commit<CG>(done + 8 * (i & 1));
    }
    if (!ok) {
      *failed = 1;
      if (issues) commit<CG>(drain);       // let what was issued end
      warp_wait(drain, 0, a.wait_ns);
    }
  } else if (warp >= 4) {
    // --------------------------------------------------------------- output
    // C columns at a time; `half` 0 takes the first NT / 2 columns (all 16 of the
    // narrowest tile), 1 the others
    constexpr int C = L::template kOutCols<T>, kCols = NT == 16 ? 16 : NT / 2;
    const bool joined = CG == 1 && a.split > 1;
    const int q = warp & 3, half = (warp - 4) >> 2;      // this warp's 32 lanes of tensor memory
    const int chunks = NT == 16 && half == 1 ? 0 : kCols / C;
    const uint32_t free_at = CG == 2 ? map_to(free_, 0) : free_, buffer = ring + L::kOutAt + (warp - 4) * 2048;
    int i = 0;
    for (int t = first; t < tiles; t += step, ++i) {
      int tx, ty;
      tile_at(a, t, tx, ty);
      const int x0 = (tx * CG + (CG == 2 ? (int)rank : 0)) * 128 + q * 32, x = x0 + lane, y0 = ty * NT;
      // The shared columns first: the first accumulator's last ones, the second
      // one's first.  The half that has none frees them at once: what it
      // stands for is that it has read the tile before.  Tiles release in turn on
      // two barriers: a warp may be a tile ahead of the others, so on one its
      // arrival for this tile would count for the tile before, and the products
      // would overwrite an accumulator that a slower warp still reads.  It is never
      // two ahead: the next tile's products wait for this one's release.
      const bool down = L::kOverlap && (i & 1) == 0;
      const bool shares = L::kOverlap && half == (down ? 1 : 0);
      const auto column = [&](int j) { return half * kCols + (down ? kCols - C - j * C : j * C); };
      if (L::kOverlap && !shares) {
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive_cluster(free_at + 8 * (i & 1));
      }
      Addend<T, C> o[2];
      if (!joined && chunks > 0) o[0].load(a, x, y0 + column(0));
      if (!warp_wait(done + 8 * (i & 1), (uint32_t)(i >> 1) & 1u, a.wait_ns)) {
        *failed = 1;
        break;
      }
      fence_after();
      const uint32_t acc = tmem + (i & 1) * L::kAcc1 + ((uint32_t)(q * 32) << 16);
#pragma unroll
      for (int j = 0; j < kCols / C; ++j) {
        if (j >= chunks) break;
        const int c = column(j);
        if (!joined && j + 1 < chunks) o[(j + 1) & 1].load(a, x, y0 + column(j + 1));
        float v[C];
        acc_load<C>(acc + c, v);
        // read: the shared 24 columns, or the whole tile
        if (L::kOverlap ? shares && j == 32 / C - 1 : j == chunks - 1) {
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive_cluster(free_at + 8 * (i & 1));
        }
        if (!joined) {
          if (a.swap || whole(a, C, y0 + c)) {
            o[j & 1].sum(a, x, v);
            if constexpr (C * sizeof(T) == 64 && NT == 256)
              store_staged<T>(&map_out, buffer, lane, x0, y0 + c, x0 < a.nx, v);
            else
              store_lanes<T>(a, x, y0 + c, v);
          } else if (y0 + c < a.ny) {
            store_spread<T>(a, buffer, lane, x0, y0 + c, v);
          }
        } else {
          float* part = reinterpret_cast<float*>(smem);
          if (a.swap) {
#pragma unroll
            for (int k = 0; k < C; ++k) part[(c + k) * 128 + q * 32 + lane] = v[k];
          } else {
#pragma unroll
            for (int k = 0; k < C; k += 4)
              *reinterpret_cast<float4*>(part + (q * 32 + lane) * (NT + 4) + c + k) =
                  make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
          }
        }
      }
      if (chunks == 0 && lane == 0) bar_arrive_cluster(free_at + 8 * (i & 1));
    }
    // the last copy has read the buffer; what it writes is complete when the grid is
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  }

  __syncwarp();
  fence_before();
  __syncthreads();
  // After a wait that ran out, in whichever warp: the copies that were issued land
  // before the CTA leaves (each stage's last use; else its products waited for it).
  if (warp == 0 && counts && *failed)
    for (int i = 0; i < S; ++i) {
      if (at.first && i >= (int)at.stage) break;
      warp_wait(full + 8 * i, i < (int)at.stage ? at.phase : at.phase ^ 1u, a.wait_ns);
    }
  __syncwarp();
  if (CG == 1 && a.split > 1) {
    // sums of the cluster's parts, in rank order: each CTA takes 128 / split rows
    // of x, four outputs at a time that lie together in `out`
    cluster_sync();
    if (NT <= 128 && !*failed) {
      int tx, ty;
      tile_at(a, first, tx, ty);
      const int rows = 128 / a.split, cols = min(NT, a.ny - ty * NT);
      const int n = a.swap ? rows / 4 * cols : rows * ((cols + 3) / 4);
#pragma unroll 2
      for (int e = threadIdx.x; e < n; e += kThreads) {
        int r, c;
        if (a.swap) {
          r = (int)rank * rows + 4 * (e % (rows / 4));
          c = e / (rows / 4);
        } else {
          r = (int)rank * rows + e / ((cols + 3) / 4);
          c = 4 * (e % ((cols + 3) / 4));
        }
        const uint32_t at = ring + 4 * (a.swap ? c * 128 + r : r * (NT + 4) + c);
        float v[4] = {};
#pragma unroll
        for (int p = 0; p < 8; ++p)
          if (p < a.split) {
            float w[4];
            asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3]) : "r"(map_to(at, p)));
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = p == 0 ? w[j] : v[j] + w[j];
          }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int x = tx * 128 + r + (a.swap ? j : 0), y = ty * NT + c + (a.swap ? 0 : j);
          if (x < a.nx && y < a.ny) {
            if (a.addend != nullptr)
              v[j] += element(static_cast<const T*>(a.addend) + place(a, a.addend_pitch, x, y));
            put(static_cast<T*>(a.out) + place(a, a.out_pitch, x, y), v[j]);
          }
        }
      }
    }
  }
  if (clustered) cluster_sync();      // a pair's peer, or a reader of this CTA's part, has ended
  if (threadIdx.x == 0 && *failed) atomicOr(&g_flags, OPT_FLAG_WAIT_TIMEOUT);
  if (warp == 2) {
    fence_after();
    if (CG == 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kCols));
    else
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kCols));
  }
}

// A product over a depth of 0: the addend, or zero.
template <typename T>
__global__ void __launch_bounds__(kThreads) no_depth_kernel(const __grid_constant__ MatmulArgs a) {
  const int64_t n = (int64_t)a.nx * a.ny;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < n; e += (int64_t)gridDim.x * kThreads)
  {
    const int x = (int)(e / a.ny), y = (int)(e % a.ny);
    put(static_cast<T*>(a.out) + place(a, a.out_pitch, x, y),
        a.addend == nullptr ? 0.0f : element(static_cast<const T*>(a.addend) + place(a, a.addend_pitch, x, y)));
  }
}

__global__ void clear_flags_kernel(int seen) { atomicAnd(&g_flags, ~seen); }

// ---------------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult got;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &got) != cudaSuccess ||
        got != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// rows x bytes matrix of bytes, boxes of 128 bytes by `box` rows, 128-byte swizzle
bool codes_map(CUtensorMap* m, const void* p, int64_t k, int64_t rows, int64_t pitch, int box) {
  const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(rows > 1 ? pitch : (k + 15) / 16 * 16)};
  const cuuint32_t boxes[2] = {kStageDepth, (cuuint32_t)box}, ones[2] = {1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, boxes, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// scale tiles as rows of 128 words, one at a time
bool scales_map(CUtensorMap* m, const void* p, int64_t tiles) {
  const cuuint64_t dims[2] = {kScaleTile / 4, (cuuint64_t)tiles}, strides[1] = {kScaleTile};
  const cuuint32_t boxes[2] = {kScaleTile / 4, 1}, ones[2] = {1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(p), dims, strides, boxes, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// out, in boxes of 64 bytes by 32 rows, 64-byte swizzle
template <typename T>
bool out_map(CUtensorMap* m, const MatmulArgs& a) {
  const int64_t es = sizeof(T);
  const cuuint64_t dims[2] = {(cuuint64_t)a.ny, (cuuint64_t)a.nx};
  const cuuint64_t strides[1] = {(cuuint64_t)(a.nx > 1 ? a.out_pitch * es : (a.ny * es + 15) / 16 * 16)};
  const cuuint32_t boxes[2] = {(cuuint32_t)(64 / es), 32}, ones[2] = {1, 1};
  return encode_fn()(m, es == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.out, dims,
                     strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Operand {
  const void* codes;
  const void* scales;
  int64_t pitch, rows;
};

// Groups of CTAs (pairs, a split's cluster) that go through the tiles.  A split
// tile's cluster takes one tile; others loop.
int64_t groups(int64_t tiles, int cg, int split, int sm_count) {
  const int64_t slots = sm_count / cg;
  return split > 1 || tiles < slots ? tiles : slots;
}

template <typename T, int CG, int NT>
cudaError_t launch(const Operand& x, const Operand& y, int64_t k, MatmulArgs a, int split, int sm_count,
                   cudaStream_t s) {
  using L = Layout<CG, NT>;
  static OccupancyCache cache;
  cached_occupancy(matmul_kernel<T, CG, NT>, cache, kThreads, L::kBytes);     // enables the shared memory
  a.nx = (int)x.rows;
  a.ny = (int)y.rows;
  const int64_t xt = (x.rows + 128 * CG - 1) / (128 * CG), yt = (y.rows + NT - 1) / NT;
  if (xt * yt > 0x7FFFFFF) return cudaErrorInvalidConfiguration;
  a.x_tiles = (int)xt;
  a.y_tiles = (int)yt;
  a.split = split;
  const auto fits = [&](const void* p, int64_t pitch, int64_t to) {
    return ((uintptr_t)p & (uintptr_t)(to - 1)) == 0 && (x.rows == 1 || pitch * (int64_t)sizeof(T) % to == 0);
  };
  a.wide = !a.swap && fits(a.out, a.out_pitch, NT == 256 ? 16 : 32) &&
           (a.addend == nullptr || fits(a.addend, a.addend_pitch, 32));
  CUtensorMap mx, my, msx, msy, mo;
  if (encode_fn() == nullptr || !codes_map(&mx, x.codes, k, x.rows, x.pitch, 128) ||
      !codes_map(&my, y.codes, k, y.rows, y.pitch, L::kY) ||
      !scales_map(&msx, x.scales, (x.rows + 127) / 128 * a.panel) ||
      !scales_map(&msy, y.scales, (y.rows + 127) / 128 * a.panel) || (NT == 256 && a.wide && !out_map<T>(&mo, a)))
    return cudaErrorInvalidValue;
  if (NT != 256 || !a.wide) mo = mx;      // not used
  const int per = CG == 2 ? 2 : split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups(xt * yt, CG, split, sm_count) * per));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)per;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = per > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, matmul_kernel<T, CG, NT>, mx, my, msx, msy, mo, a);
}

// Which operand is x, the tile (128 or, by a pair of CTAs, 256 rows of x, nt of
// y) and the split, by the estimated time: the tiles that one CTA goes through,
// each its blocks' time (but no less than its output takes) and its own, plus a
// pair's start or a split's sum.  A split's CTAs take one tile each, so a second
// wave of them starts anew.  The times are fits, in ns, to one shape in several
// forms: 256 x 4096 x 4096 takes 9.8 us in 128-wide tiles, 10.1 in pairs of 128,
// 14.2 in pairs of 256 and 12.2 split in two; 2048 x 4096 x 4096 31.8, 27.4 and
// 25.5; 8192 x 2304 x 768 22.8, 22.2 and 16.6; 64 x 4096 x 4096 9.0 whole, 8.3
// split in four.  Rows of codes that do not start on lines (`on_lines` false) cost
// twice L2's accesses: 773 x 10368 x 8847 takes 111, 110 and 92 us.
struct Plan {
  int swap, cg, nt, split;
};
Plan plan(int64_t m, int64_t n, int blocks, bool on_lines, const int (&clusters)[4]) {
  static const struct { int cg, nt, block, off_line, least, tile, split; } kForms[] = {
      {1, 16, 155, 220, 1000, 400, 2300}, {1, 32, 165, 245, 1000, 400, 2500},   {1, 64, 185, 295, 1500, 400, 3300},
      {1, 128, 208, 385, 2000, 400, 5000}, {2, 128, 175, 300, 2000, 400, 0}, {2, 256, 320, 400, 1900, 900, 0}};
  constexpr double kStart = 3500, kPair = 800;
  Plan best = {0, 2, 256, 1};
  double least = 1e300;
  const int panel = (blocks + 3) / 4;
  for (const auto& f : kForms)
    for (int swap = 0; swap < (f.nt < 128 ? 2 : 1); ++swap) {
      const int64_t xr = swap ? n : m, yr = swap ? m : n;
      // scales are addressed by whole tiles of 128 rows: a narrower tile of y only where it is the only one
      if (f.nt < 128 && yr > f.nt) continue;
      const int64_t tiles = ((xr + 128 * f.cg - 1) / (128 * f.cg)) * ((yr + f.nt - 1) / f.nt);
      for (int split = 1; split <= (f.cg == 2 ? 1 : 8) && split <= panel; split *= 2) {
        const int64_t slots = clusters[f.cg == 2 ? 1 : split == 1 ? 0 : split == 2 ? 1 : split == 4 ? 2 : 3];
        const int64_t waves = (tiles + slots - 1) / slots;
        const double each = (double)((blocks + split - 1) / split) * (on_lines ? f.block : f.off_line), out = waves > 1 ? f.least : 0;
        double time = (double)waves * ((each > out ? each : out) + f.tile) + (f.cg == 2 ? kPair : 0);
        if (split > 1) time += (double)waves * f.split + (double)(waves - 1) * kStart;
        if (time < least) {
          least = time;
          best = {swap, f.cg, f.nt, split};
        }
      }
    }
  return best;
}

// Clusters of 1, 2, 4 and 8 CTAs that the device holds at once (a GB300's 152 SMs:
// 152, 76, 36, 15: clusters do not straddle its groups of SMs), asked once per
// device.
cudaError_t active_clusters(int sm_count, int (&out)[4]) {
  static std::atomic<int> cache[kMaxDevices][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) dev = 0;
  out[0] = sm_count;
  for (int i = 1; i < 4; ++i) {
    out[i] = cache[dev][i].load(std::memory_order_relaxed);
    if (out[i] > 0) continue;
    using L = Layout<1, 128>;
    const auto kernel = matmul_kernel<float, 1, 128>;
    static OccupancyCache occupancy;
    cached_occupancy(kernel, occupancy, kThreads, L::kBytes);     // enables the shared memory
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << i;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sm_count >> i << i));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::kBytes;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&out[i], kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (out[i] < 1) out[i] = 1;
    cache[dev][i].store(out[i], std::memory_order_relaxed);
  }
  return cudaSuccess;
}

cudaError_t plan_of(const opt_matmul_args& c, int sm_count, Plan* p) {
  int clusters[4];
  if (const cudaError_t e = active_clusters(sm_count, clusters); e != cudaSuccess) return e;
  const auto on_lines = [](const void* codes, int64_t rows, int64_t pitch) {
    return (rows == 1 || pitch % 128 == 0) && ((uintptr_t)codes & 127u) == 0;
  };
  *p = plan(c.m, c.n, (int)((c.k + 127) / 128), on_lines(c.d_a, c.m, c.a_pitch) && on_lines(c.d_b, c.n, c.b_pitch),
            clusters);
  return cudaSuccess;
}

template <typename T>
cudaError_t dispatch(const opt_matmul_args& c, int sm_count, cudaStream_t s) {
  MatmulArgs a = {};
  a.out = c.d_out;
  a.addend = c.d_addend;
  a.out_pitch = c.out_pitch;
  a.addend_pitch = c.addend_pitch;
  if (c.k == 0) {
    a.nx = (int)c.m;
    a.ny = (int)c.n;
    no_depth_kernel<T><<<(unsigned)sm_count * 4, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  a.drill = (c.flags & OPT_MATMUL_WAIT_DRILL) != 0;
  a.wait_ns = a.drill ? kDrillNs : kWaitNs;
  a.blocks = (int)((c.k + 127) / 128);
  a.panel = (a.blocks + 3) / 4;
  if (!matmul_waits(c)) {
    a.swap = c.m < c.n;
    return launch_matmul_few(c, a, s);
  }
  const Operand ops[2] = {{c.d_a, c.d_a_scales, c.a_pitch, c.m}, {c.d_b, c.d_b_scales, c.b_pitch, c.n}};
  Plan p;
  if (const cudaError_t e = plan_of(c, sm_count, &p); e != cudaSuccess) return e;
  a.swap = p.swap;
  const Operand &x = ops[p.swap], &y = ops[1 - p.swap];
  switch (p.nt) {
    case 16: return launch<T, 1, 16>(x, y, c.k, a, p.split, sm_count, s);
    case 32: return launch<T, 1, 32>(x, y, c.k, a, p.split, sm_count, s);
    case 64: return launch<T, 1, 64>(x, y, c.k, a, p.split, sm_count, s);
    case 128:
      return p.cg == 1 ? launch<T, 1, 128>(x, y, c.k, a, p.split, sm_count, s)
                       : launch<T, 2, 128>(x, y, c.k, a, 1, sm_count, s);
    default: return launch<T, 2, 256>(x, y, c.k, a, 1, sm_count, s);
  }
}

}  // namespace

bool matmul_waits(const opt_matmul_args& a) { return a.k > 0 && a.m > kFewRows && a.n > kFewRows; }

cudaError_t matmul_form(const opt_matmul_args& a, int sm_count, int32_t* form) {
  Plan p;
  if (const cudaError_t e = plan_of(a, sm_count, &p); e != cudaSuccess) return e;
  const int64_t xr = p.swap ? a.n : a.m, yr = p.swap ? a.m : a.n;
  const int64_t tiles = (xr + 128 * p.cg - 1) / (128 * p.cg) * ((yr + p.nt - 1) / p.nt);
  const int64_t at_once = groups(tiles, p.cg, p.split, sm_count);
  form[0] = p.cg;
  form[1] = p.nt;
  form[2] = p.split;
  form[3] = p.swap;
  form[4] = (int32_t)((tiles + at_once - 1) / at_once);
  return cudaSuccess;
}

cudaError_t launch_matmul(const opt_matmul_args& a, int sm_count, cudaStream_t s) {
  return a.out_dtype == OPT_F32 ? dispatch<float>(a, sm_count, s) : dispatch<Bf16>(a, sm_count, s);
}

// Only what was read is cleared, so that a flag raised in between by a kernel on
// another stream stays for the next call.
cudaError_t layer_flags(int* flags, cudaStream_t s) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(flags, g_flags, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess || *flags == 0) return e;
  clear_flags_kernel<<<1, 1, 0, s>>>(*flags);
  e = cudaGetLastError();
  return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace psopt
