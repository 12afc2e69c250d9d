// moe_gemm_wgrad.cu -- the weights' gradient of the grouped products:
//
//   grad_w[g] = add_to[g] + sum over g's rows r of dz[r, :]^T a[r, :]        f32 [N, K]
//
// A tile is 128 rows (of N) x 256 columns (of K) of one group's gradient on one SM; the
// contraction runs over the group's rows, 64 a stage.  Both operands are read as they lie,
// rows contiguous along N and K: MN-major operands of tcgen05.mma, in TMA boxes of 64 columns x 64
// rows.  Where a group ends inside a stage, the rows behind it belong to the next group (or to
// nobody: they may hold NaN), so the issuing warp overwrites them with zeros in both operands
// up to the next 16, and the MMAs of the stage stop there.
//
// Two reasons keep the sums out of the tensor core's accumulators for long: its additions cut off
// bits that f32 gradients of many rows would miss, and the next tile's products should not
// wait for this tile's stores.  So every 512 rows the products move to the other accumulator
// of 256 columns and the epilogue warps (a thread: one row, 128 columns) add the finished one to
// their registers.  Tiles of at most 512 rows skip the registers.  32 rows x 32 columns at a time leave
// through 4 KB of shared memory and a TMA store, which also cuts off what lies outside the
// group's matrix.  (With loads from there and stores of 16 bytes a lane a tile took its warps 1400
// instructions and 14600 cycles, six times its products.)
//
// 32768 rows of 768 x 2048 in 128 uneven groups take 178 to 185 us, 5.5 TB/s: 805 MB of gradients leave, 185 MB of rows come
// in.  With add_to 305 to 320 us, 5.7 TB/s: its boxes of 32 x 32 come by TMA, four under way to each warp, into the room of two of
// the four stages (or one, where groups have many rows), and leave from there.  (Loads of a lane's own row, each a
// latency of HBM and 32 lines: 410 us.  Tiles of 128 columns even the SMs' shares of few tiles out, to no gain.)
// 777 rows of 400 x 1040 in 13 groups with add_to take 15.5 to 16.8 us (6.7 at HBM's rate), two tiles an SM at most.
//
// With a few groups of many rows there are fewer tiles than SMs: the rows are cut into ranges whose
// sums go to the workspace, and a second kernel adds them in range order.
//
// The sums of 128 columns and their addresses do not quite fit 168 registers, the most that three of the ten warps on
// one scheduler can have: 64 to 104 bytes a thread are spilled.
#include <atomic>

#include "fp8_common.cuh"

namespace moe {
namespace gemm {
namespace {

constexpr int kThreads = 320;        // producer, MMA, eight epilogue warps
constexpr int kTileN = 128, kTileK = 256;
constexpr int kRowsStage = 64;
constexpr int kBox = 64 * kRowsStage * 2;          // 64 columns x 64 rows
constexpr int kABytes = kTileN / 64 * kBox, kBBytes = kTileK / 64 * kBox;
constexpr int kChunk = 8;            // stages of one accumulator: 512 rows
constexpr int kMaxRanges = 16;
constexpr int kRangeRows = 512;      // rows of a range, at least

struct Params {
  const int32_t* group_offsets;
  int P, N, K, G;
  const float* add_to;
  float* out;                        // grad_w, or the ranges' sums
  int ranges;
  unsigned long long wait_ns;
  unsigned int* status;
  unsigned long long* launches;
};

// kAddBoxes: boxes of add_to, 32 x 32, that are under way to a warp; 0 without add_to.  Four take half of the stages' room:
// the tile's boxes arrive while its products are added up.  One has the room of the stores' box.
template <int kAddBoxes>
struct Smem {
  static constexpr int kStages = kAddBoxes == 4 ? 2 : 4, kBoxes = kAddBoxes == 4 ? 4 : 1;
  static constexpr int A = 0;
  static constexpr int B = A + kStages * kABytes;
  static constexpr int OUT = B + kStages * kBBytes;          // 8 warps x kBoxes x 4 KB, TMA stores' sources
  static constexpr int BARS = OUT + 8 * kBoxes * 4096;       // full, empty, tfull[2], tempty[2], drain, add[8][boxes]
  static constexpr int MISC = BARS + (2 * kStages + 5 + 8 * kAddBoxes) * 8;
  static constexpr int ALLOC = MISC + 16 + 1024;
};
static_assert(Smem<0>::ALLOC <= 227 * 1024 && Smem<1>::ALLOC <= 227 * 1024 && Smem<4>::ALLOC <= 227 * 1024, "shared memory");

struct Tile {
  int g, n0, k0, range;
  int r0, r1;                        // the rows of its sum
};

__device__ __forceinline__ Tile tile_of(const Params& p, long long i, int tn, int tk) {
  Tile t;
  const long long per = static_cast<long long>(tn) * tk * p.ranges;
  t.g = static_cast<int>(i / per);
  int local = static_cast<int>(i - t.g * per);
  t.range = local / (tn * tk);
  local -= t.range * tn * tk;
  t.k0 = local / tn * kTileK;
  t.n0 = local % tn * kTileN;
  auto off = [&](int g) {
    return p.group_offsets ? min(max(__ldg(p.group_offsets + g), 0), p.P) : (g == 0 ? 0 : p.P);
  };
  const int lo = off(t.g), hi = max(off(t.g + 1), lo);
  if (p.ranges == 1) {
    t.r0 = lo;
    t.r1 = hi;
  } else {                           // whole stages
    const long long steps = (hi - lo) / kRowsStage + ((hi - lo) % kRowsStage != 0);
    t.r0 = lo + static_cast<int>(steps * t.range / p.ranges) * kRowsStage;
    const long long e = lo + steps * (t.range + 1) / p.ranges * kRowsStage;
    t.r1 = e < hi ? static_cast<int>(e) : hi;
  }
  return t;
}

__device__ __forceinline__ int steps_of(const Tile& t) { return (t.r1 - t.r0 + kRowsStage - 1) / kRowsStage; }

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// this thread's stores but for the last kLater groups have read their shared memory; all have been written
template <int kLater>
__device__ __forceinline__ void tma_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLater) : "memory");
}
__device__ __forceinline__ void tma_store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <int kAddBoxes>
__global__ void __launch_bounds__(kThreads, 1)
wgrad_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
             const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmAdd, const Params p) {
  using Smem = Smem<kAddBoxes>;
  constexpr bool kAdd = kAddBoxes > 0;
  constexpr int kStages = Smem::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = ptx::smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Smem::BARS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Smem::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Smem::MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar_full = [&](int s) { return ptx::smem_u32(bars + s); };
  auto bar_empty = [&](int s) { return ptx::smem_u32(bars + kStages + s); };
  auto bar_tfull = [&](int a) { return ptx::smem_u32(bars + 2 * kStages + a); };
  auto bar_tempty = [&](int a) { return ptx::smem_u32(bars + 2 * kStages + 2 + a); };
  const uint32_t bar_drain = ptx::smem_u32(bars + 2 * kStages + 4);
  auto bar_add = [&](int w, int c) { return ptx::smem_u32(bars + 2 * kStages + 5 + kAddBoxes * w + c); };

  count_launch(p.launches, MOE_KID_GEMM_WGRAD);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(bar_full(s), 1);
      ptx::mbar_init(bar_empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(bar_tfull(a), 1);
      ptx::mbar_init(bar_tempty(a), 8);
    }
    ptx::mbar_init(bar_drain, 1);
    if (kAdd)
      for (int i = 0; i < 8 * kAddBoxes; ++i) ptx::mbar_init(bar_add(0, i), 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::tma_prefetch_desc(&tmA);
    ptx::tma_prefetch_desc(&tmB);
    ptx::tma_prefetch_desc(&tmO);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  grid_dep_wait();
  grid_dep_launch();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int tn = (p.N + kTileN - 1) / kTileN, tk = (p.K + kTileK - 1) / kTileK;
  const long long tiles = static_cast<long long>(p.G) * tn * tk * p.ranges;
  uint32_t issued = 0;
  bool mma_any = false;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (ptx::elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (long long i = blockIdx.x; ok && i < tiles; i += gridDim.x) {
        const Tile t = tile_of(p, i, tn, tk);
        for (int r = t.r0; r < t.r1; r += kRowsStage) {
          ok = wait_bar_spin(bar_empty(stage), phase ^ 1u, abort_flag, p.status, p.wait_ns);
          if (!ok) break;
          ptx::mbar_arrive_expect_tx(bar_full(stage), kABytes + kBBytes);
#pragma unroll
          for (int b = 0; b < kTileN / 64; ++b)
            ptx::tma_load_2d(sb + Smem::A + stage * kABytes + b * kBox, &tmA, t.n0 + 64 * b, r, bar_full(stage));
#pragma unroll
          for (int b = 0; b < kTileK / 64; ++b)
            ptx::tma_load_2d(sb + Smem::B + stage * kBBytes + b * kBox, &tmB, t.k0 + 64 * b, r, bar_full(stage));
          ++issued;
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (a whole warp: it
    // clears the rows behind a group's end)
    constexpr uint32_t idesc = ptx::idesc_bf16_f32_mn(kTileN, kTileK, true, true);
    int stage = 0, acc = 0;
    uint32_t phase = 0, uses[2] = {0, 0};
    bool ok = true;
    for (long long i = blockIdx.x; ok && i < tiles; i += gridDim.x) {
      const Tile t = tile_of(p, i, tn, tk);
      const int steps = steps_of(t);
      for (int st = 0; st < steps; ++st) {
        const int in_chunk = st % kChunk;
        if (in_chunk == 0) {
          ok = wait_bar(bar_tempty(acc), ((acc ? uses[1] : uses[0]) & 1u) ^ 1u, abort_flag, p.status, p.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        ok = wait_bar(bar_full(stage), phase, abort_flag, p.status, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t a = sb + Smem::A + stage * kABytes, b = sb + Smem::B + stage * kBBytes;
        const int rows = min(kRowsStage, t.r1 - t.r0 - st * kRowsStage), ends = (rows + 15) & ~15;
        if (rows < ends) {
          for (int r = rows + (lane >> 3); r < ends; r += 4) {
#pragma unroll
            for (int x = 0; x < kTileN / 64; ++x)
              ptx::st_shared_v4(a + x * kBox + r * 128 + (lane & 7) * 16, 0u, 0u, 0u, 0u);
#pragma unroll
            for (int x = 0; x < kTileK / 64; ++x)
              ptx::st_shared_v4(b + x * kBox + r * 128 + (lane & 7) * 16, 0u, 0u, 0u, 0u);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
        }
        ptx::tc_fence_after();
        const bool last = in_chunk == kChunk - 1 || st == steps - 1;
        if (ptx::elect_one()) {
          const uint64_t da = ptx::desc_mnmajor_sw128(a, kBox), db = ptx::desc_mnmajor_sw128(b, kBox);
#pragma unroll
          for (int k = 0; k < kRowsStage / 16; ++k)
            if (16 * k < rows)
              ptx::mma_bf16(tmem + static_cast<uint32_t>(acc) * kTileK, da + 128ull * k, db + 128ull * k, idesc,
                            in_chunk != 0 || k != 0 ? 1u : 0u);
          ptx::mma_commit(bar_empty(stage));
          if (last) ptx::mma_commit(bar_tfull(acc));
        }
        __syncwarp();
        mma_any = true;
        if (last) {
          if (acc) ++uses[1]; else ++uses[0];
          acc ^= 1;
        }
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp - 2) >> 2;      // TMEM lane quarter; 128 of the columns
    const uint32_t stage = sb + Smem::OUT + (warp - 2) * Smem::kBoxes * 4096;
    // add_to's boxes in their order, [tile][c]; box i lies in place i % kBoxes
    constexpr uint32_t kPlaces = Smem::kBoxes;
    uint32_t arrived = 0, asked = 0;
    auto ask = [&](long long i, int c) {
      if (i >= tiles) return;
      if (lane == 0) {
        const Tile t = tile_of(p, i, tn, tk);
        const uint32_t at = asked % kPlaces, bar = bar_add(warp - 2, at);
        ptx::mbar_arrive_expect_tx(bar, 4096);
        tma_load_3d(stage + at * 4096, &tmAdd, t.k0 + half * 128 + 32 * c, t.n0 + q * 32, t.g, bar);
      }
      ++asked;
    };
    for (int c = 0; c < kAddBoxes; ++c) ask(blockIdx.x, c);
    int acc = 0;
    uint32_t uses[2] = {0, 0};
    bool ok = true;
    // waits for the accumulator's next sums; frees it
    auto take = [&]() {
      ok = ok && wait_bar(bar_tfull(acc), (acc ? uses[1] : uses[0]) & 1u, abort_flag, p.status, p.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      ptx::tc_fence_after();
      return tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc) * kTileK + half * 128;
    };
    auto free = [&]() {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar_tempty(acc));
      if (acc) ++uses[1]; else ++uses[0];
      acc ^= 1;
    };
    for (long long i = blockIdx.x; i < tiles; i += gridDim.x) {
      const Tile t = tile_of(p, i, tn, tk);
      const int steps = steps_of(t);
      const int z = t.range * p.G + t.g;
      // columns [32 c, + 32) of this thread's row: 128 bytes a row through a box, a store
      auto leave = [&](int c, float (&v)[32]) {
        const int col = t.k0 + half * 128 + 32 * c, row0 = t.n0 + q * 32;
        const uint32_t box = stage + (kAdd ? arrived % kPlaces * 4096 : 0), mine = box + lane * 128;
        if (kAdd) {
          ok = wait_bar(bar_add(warp - 2, arrived % kPlaces), (arrived / kPlaces) & 1u, abort_flag, p.status, p.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) return;
          ++arrived;
        } else {
          if (lane == 0) tma_store_wait_read<0>();   // the box's last store
          __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t at = mine + ((k ^ (lane & 7)) << 4);
          if (kAdd) {
            const uint4 a = ptx::ld_shared_v4(at);
            v[4 * k] += __uint_as_float(a.x);
            v[4 * k + 1] += __uint_as_float(a.y);
            v[4 * k + 2] += __uint_as_float(a.z);
            v[4 * k + 3] += __uint_as_float(a.w);
          }
          ptx::st_shared_v4(at, __float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]),
                            __float_as_uint(v[4 * k + 3]));
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        // a group for every box, also without a store: they count them
        if (lane == 0) {
          if (col < p.K && row0 < p.N) tma_store_3d(&tmO, box, col, row0, z);
          tma_store_commit();
        }
        if (kAddBoxes == 1) {        // the next box, in the same place
          if (lane == 0) tma_store_wait_read<0>();
          ask(i + (c == 3 ? gridDim.x : 0), (c + 1) & 3);
        } else if (kAdd && arrived > 1) {        // three boxes on, in the place of the box before this one
          if (lane == 0) tma_store_wait_read<1>();
          ask(i + (c > 0 ? gridDim.x : 0), (c + 3) & 3);
        }
      };
      if (steps <= kChunk) {
        uint32_t ta = 0;
        if (steps > 0) {
          ta = take();
          if (!ok) break;
        }
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float v[32];
          if (steps > 0) {
            uint32_t u[32];
            ptx::tmem_ld_32x32b_x32(ta + 32 * c, u);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(u[k]);
            if (c == 3) free();
          } else {                                 // an empty group
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = 0.0f;
          }
          leave(c, v);
          if (!ok) break;
        }
        if (!ok) break;
        continue;
      }
      float sum[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int k = 0; k < 32; ++k) sum[c][k] = 0.0f;
#pragma unroll 1
      for (int st = 0; st < steps; st += kChunk) {
        const uint32_t ta = take();
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t u[32];
          ptx::tmem_ld_32x32b_x32(ta + 32 * c, u);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) sum[c][k] += __uint_as_float(u[k]);
        }
        free();
      }
      if (!ok) break;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (ok) leave(c, sum[c]);
      if (!ok) break;
    }
    if (lane == 0) tma_store_wait();
    // a warp that gave up lets its copies land
    for (; arrived < asked; ++arrived) spin_bounded(bar_add(warp - 2, arrived % kPlaces), (arrived / kPlaces) & 1u);
  }
  // ---- exit: a CTA that gave up drains its copies and MMAs first
  __syncthreads();
  if (*abort_flag != 0) {
    if (warp == 1 && mma_any && ptx::elect_one()) {
      ptx::mma_commit(bar_drain);
      spin_bounded(bar_drain, 0);
    }
    for (uint32_t i = issued < kStages ? 0 : issued - kStages; i < issued; ++i)
      spin_bounded(bar_full(i % kStages), (i / kStages) & 1);
  }
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// the ranges' sums in range order, on add_to
__global__ void __launch_bounds__(256)
wgrad_reduce_kernel(const float* __restrict__ part, int ranges, long long n4, const float* add_to, float* out,
                    unsigned long long* launches) {
  count_launch(launches, MOE_KID_WGRAD_REDUCE);
  grid_dep_wait();
  grid_dep_launch();
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n4) return;
  const float4* q = reinterpret_cast<const float4*>(part) + i;
  float4 v[kMaxRanges];
#pragma unroll
  for (int r = 0; r < kMaxRanges; ++r)
    if (r < ranges) v[r] = __ldcg(q + r * n4);
  float4 s = ranges > 0 ? v[0] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int r = 1; r < kMaxRanges; ++r)
    if (r < ranges) {
      s.x += v[r].x; s.y += v[r].y; s.z += v[r].z; s.w += v[r].w;
    }
  if (add_to) {
    const float4 a = reinterpret_cast<const float4*>(add_to)[i];
    s.x += a.x; s.y += a.y; s.z += a.z; s.w += a.w;
  }
  reinterpret_cast<float4*>(out)[i] = s;
}

// Ranges of rows: as many as give every SM a tile, each of at least kRangeRows of the average
// group's rows
int ranges_of(int P, int N, int K, int G) {
  const long long tiles = static_cast<long long>(G) * ((N - 1ll) / kTileN + 1) * ((K - 1ll) / kTileK + 1);
  long long s = sm_count() / tiles;
  const long long most = P / G / kRangeRows;
  s = s < most ? s : most;
  s = s < kMaxRanges ? s : kMaxRanges;
  return s < 1 ? 1 : static_cast<int>(s);
}

template <int kAddBoxes>
int launch(const char* op, const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& to, const CUtensorMap& tadd,
           const Params& p, cudaStream_t stream) {
  constexpr int kBytes = Smem<kAddBoxes>::ALLOC;
  static std::atomic<int> configured[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    dev = -1;
  }
  const bool cache = dev >= 0 && dev < 64;
  if (!cache || !configured[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(wgrad_kernel<kAddBoxes>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes) != cudaSuccess)
      return set_error(MOE_ERR_CUDA, "%s: cannot reserve %d bytes of shared memory: %s", op, kBytes,
                       cudaGetErrorString(cudaGetLastError()));
    if (cache) configured[dev].store(1, std::memory_order_release);
  }
  const long long tiles =
      static_cast<long long>(p.G) * ((p.N - 1) / kTileN + 1) * ((p.K - 1) / kTileK + 1) * p.ranges;
  const int sms = sm_count();
  return launch_status(launch_kernel(wgrad_kernel<kAddBoxes>, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)),
                                     dim3(kThreads), kBytes, stream, nullptr, 0, ta, tb, to, tadd, p),
                       op);
}

}  // namespace
}  // namespace gemm
}  // namespace moe

using namespace moe;
using namespace moe::gemm;

extern "C" size_t moe_grouped_gemm_wgrad_workspace_size(int P, int N, int K, int G) {
  if (P <= 0 || N <= 0 || K <= 0 || G <= 0) return 0;
  const int s = ranges_of(P, N, K, G);   // grows with P
  return s < 2 ? 0 : static_cast<size_t>(s) * G * N * K * 4;
}

extern "C" int moe_grouped_gemm_wgrad_bf16(const void* dz_bf16, const void* a_bf16, const int32_t* group_offsets,
                                           int P, int N, int K, int G, const float* add_to, float* grad_w,
                                           void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  const char* op = "moe_grouped_gemm_wgrad_bf16";
  if (P < 0 || N < 1 || K < 1) return set_error(MOE_ERR_ARG, "%s: P=%d, N=%d, K=%d", op, P, N, K);
  if (P > kMaxDim || N > kMaxDim || K > kMaxDim)
    return set_error(MOE_ERR_ARG, "%s: P=%d, N=%d or K=%d is too large", op, P, N, K);
  if (G < 1 || G > kMaxGroups) return set_error(MOE_ERR_ARG, "%s: G=%d outside [1, %d]", op, G, kMaxGroups);
  if (N % 8 || K % 8) return set_error(MOE_ERR_ALIGN, "%s: N=%d and K=%d must be multiples of 8", op, N, K);
  if (((N - 1ll) / kTileN + 1) * ((K - 1ll) / kTileK + 1) * kMaxRanges > kMaxDim ||
      static_cast<double>(G) * N * K > 0x1p38)
    return set_error(MOE_ERR_ARG, "%s: G=%d, N=%d and K=%d are too large together", op, G, N, K);
  if (!grad_w) return set_error(MOE_ERR_ARG, "%s: grad_w is NULL", op);
  if (!group_offsets && G != 1) return set_error(MOE_ERR_ARG, "%s: group_offsets is NULL with G=%d", op, G);
  if (P > 0 && (!dz_bf16 || !a_bf16)) return set_error(MOE_ERR_ARG, "%s: dz or a is NULL", op);
  for (const void* q : {dz_bf16, a_bf16, static_cast<const void*>(add_to), static_cast<const void*>(grad_w),
                        const_cast<const void*>(workspace)})
    if (q && !aligned16(q))
      return set_error(MOE_ERR_ALIGN, "%s: dz, a, add_to, grad_w and workspace must be 16-byte aligned", op);
  if (reinterpret_cast<uintptr_t>(group_offsets) & 3u)
    return set_error(MOE_ERR_ALIGN, "%s: group_offsets must be 4-byte aligned", op);
  const size_t need = moe_grouped_gemm_wgrad_workspace_size(P, N, K, G);
  if (need > 0 && (!workspace || ws_bytes < need))
    return set_error(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes is smaller than the %zu needed", op,
                     workspace ? ws_bytes : 0, need);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t n = static_cast<size_t>(G) * N * K;
  DeviceDiag diag = device_diag();
  if (P == 0) {                      // sums of nothing
    return launch_status(launch_kernel(wgrad_reduce_kernel, dim3(static_cast<unsigned>((n / 4 + 255) / 256)), dim3(256),
                                       0, s, nullptr, 0, static_cast<const float*>(nullptr), 0,
                                       static_cast<long long>(n / 4), add_to, grad_w, diag.launches),
                         op);
  }
  Params p{};
  p.group_offsets = group_offsets;
  p.P = P; p.N = N; p.K = K; p.G = G;
  p.ranges = ranges_of(P, N, K, G);
  p.add_to = p.ranges > 1 ? nullptr : add_to;
  p.out = p.ranges > 1 ? static_cast<float*>(workspace) : grad_w;
  p.status = diag.status;
  p.launches = diag.launches;
  p.wait_ns = pipeline_wait_ns();
  CUtensorMap ta, tb;
  int rc;
  if ((rc = make_tmap(&ta, dz_bf16, P, N, kRowsStage, op, "dz")) != MOE_OK) return rc;
  if ((rc = make_tmap(&tb, a_bf16, P, K, kRowsStage, op, "a")) != MOE_OK) return rc;
  CUtensorMap to, tadd;              // 32 x 32 boxes of the groups' matrices, a range behind the other
  if ((rc = make_tmap_f32_out(&to, p.out, G * p.ranges, N, K, op)) != MOE_OK) return rc;
  tadd = to;
  if (p.add_to && (rc = make_tmap_f32_out(&tadd, const_cast<float*>(p.add_to), G, N, K, op)) != MOE_OK) return rc;
  // With many rows a group the products take longer than add_to's way and want all four stages: 512 rows a group, four boxes
  // 187 us, one 196; 585 rows 48.0 and 44.5; 8192 rows of 4096 x 4096 343 and 224 (216 without add_to).
  rc = !p.add_to      ? launch<0>(op, ta, tb, to, tadd, p, s)
       : P / G <= 512 ? launch<4>(op, ta, tb, to, tadd, p, s)
                      : launch<1>(op, ta, tb, to, tadd, p, s);
  if (rc != MOE_OK || p.ranges == 1) return rc;
  return launch_status(launch_kernel(wgrad_reduce_kernel, dim3(static_cast<unsigned>((n / 4 + 255) / 256)), dim3(256), 0, s,
                                     nullptr, 0, static_cast<const float*>(workspace), p.ranges,
                                     static_cast<long long>(n / 4), add_to, grad_w, diag.launches),
                       op);
}
