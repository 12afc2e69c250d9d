// moe_gemm_bias_act.cu -- grouped BF16 product with bias, activation, row weight and residual
// in its epilogue, on CTA pairs.
//
//   z = a w_g^T + bias,  out[dst] = bf16(act(z) pair_weight[dst] + residual[dst])
//
// A tile is 256 output columns x up to 256 consecutive rows of one group.  Weights sit on the
// MMA's M side (each SM of the pair holds 128 output columns' weights), rows on its N side, N
// their count rounded up to 16: a group pads to 16 rows, a single row costs no more than its
// weights, and per 64-wide K step an SM stages 16 KB of weights and at most 16 KB of rows, which
// one tcgen05.mma.cta_group::2 of 256 x N x 16 shares between the SMs.  Two accumulators of 256
// columns let a tile's epilogue run under the next tile's products.
//
//   warp 0      TMA producer in both CTAs: its own half of every stage, counted on the even CTA's
//               barrier
//   warp 1      tensor memory; in the even CTA the thread that issues the pair's MMAs
//   warps 2-9   epilogue in both CTAs: two groups of four warps take the tile's 32-row chunks in
//               turn.  A thread holds pairs of consecutive rows of four output columns (16 x 256-bit reads of
//               tensor memory), so that bias, activation and weight run on pairs of f32, and matrix stores
//               transpose the rounded pairs on their way to shared memory, from where rows leave as
//               16-byte pieces; the residual's rows come the same way back.  It runs under the next
//               tile's products.
//
// 65536 rows of 2048 x 768 in 128 groups, GELU and z take 182 us in a row of the same calls, 197 to 201 among others (1.03
// PFLOP/s and 4.4 TB/s), where HBM alone takes 129 and the products 109.  32768 rows against [K, N] weights take 107 to
// 110 (HBM 87).  Dense, 16384 x 4096 x 4096 reaches 1837 TFLOP/s.  What is left: the way of many groups' weights and rows
// from HBM through L2 at once (16 groups instead of 128: 149 us in a row), and the epilogue (165 without GELU and z).  (All column blocks of a row block in turn on one pair: 220 us, as the weights come from HBM
// again.  Tiles dealt by their costs: 190, though the busiest pair has 8 % more than the mean, as those that share rows and
// weights then run apart.  Stages brought to L2 ahead: 260; prefetches take the copies' own throughput.)
//
// Weights [G, N, K] are K-major operands.  Weights [G, K, N] (the rows' gradient of a layer's
// own weights) are MN-major ones, boxes of 64 columns x 64 K rows in the same stage: no
// transposed copy is kept.  Both are seen through three-dimensional maps, so a group's ragged
// end reads zeros and never its neighbour.
//
// Calls of few rows and weights [G, N, K] have a kernel of their own, below.
// Calls whose tiles cannot fill the pairs (few rows) take tiles of fewer rows, or cut K into ranges: each leaves f32 sums in
// the workspace and a second kernel adds them in range order and applies the epilogue.
#include <atomic>

#include "activation.cuh"
#include "fp8_common.cuh"
#include "pair_drain.cuh"

namespace moe {
namespace gemm {
namespace {

constexpr int kThreads = 320;
constexpr int kRowBlock = 256;       // rows of a tile at most (MMA N)
constexpr int kColBlock = 256;       // output columns of a tile, 128 per CTA
constexpr int kStages = 6;
constexpr int kWBytes = 128 * BK * 2;
constexpr int kTBytes = 128 * BK * 2;
constexpr int kMaxRanges = 16;       // of K
constexpr int kRangeSteps = 4;       // K steps of a range, at least

struct Params {
  const int32_t* group_offsets;
  int P, K, N, G;
  int row_block;                     // rows of a tile: kRowBlock, or 128 or 64
  const float* bias;
  int activation;
  uint16_t* z;
  const float* pair_weight;
  const int32_t* row_to_pair;
  const uint16_t* residual;
  uint16_t* out;
  float* part;                       // [ranges][N][part_rows] sums, or null: one range
  int ranges, part_rows;
  unsigned long long wait_ns;
  unsigned int* status;
  unsigned long long* launches;
};

struct Smem {
  static constexpr int STAGE_W = 0;
  static constexpr int STAGE_T = STAGE_W + kStages * kWBytes;
  static constexpr int EPI = STAGE_T + kStages * kTBytes;      // 2 groups x 8 KB
  static constexpr int DST = EPI + 2 * 8192;                   // int [2][256]
  static constexpr int WEIGHT = DST + 2 * kRowBlock * 4;       // float [2][256]
  static constexpr int BARS = WEIGHT + 2 * kRowBlock * 4;      // full, empty, tfull[2], tempty[2], drain
  static constexpr int MISC = BARS + (2 * kStages + 5) * 8;    // tmem slot, abort flag, scan, uses issued
  static constexpr int TILES = MISC + 64;
  static constexpr int GOFF = TILES + (kMaxGroups + 1) * 4;
  static constexpr int BYTES = GOFF + (kMaxGroups + 1) * 4;
  static constexpr int ALLOC = BYTES + 1024;
};
static_assert(Smem::ALLOC <= 227 * 1024, "shared memory");
static_assert(kThreads / 32 * 4 + 8 <= 48, "scan slots");

struct Tile {
  int g, r0, rows, n0;
};

__device__ __forceinline__ Tile tile_of(int tile, const int* start, const int* goff, int G, int n_fb, int block) {
  int lo = 0, hi = G;                // start[lo] <= tile < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= tile) lo = mid; else hi = mid;
  }
  const int local = tile - start[lo], m = local / n_fb;
  Tile t;
  t.g = lo;
  t.r0 = goff[lo] + m * block;
  t.rows = min(goff[lo + 1] - t.r0, block);
  t.n0 = (local - m * n_fb) * kColBlock;
  return t;
}

// rows of a tile that each CTA of the pair holds, the box they come in, and a CTA's bytes of a stage
__device__ __forceinline__ int half_of(const Tile& t) { return ((t.rows + 15) & ~15) >> 1; }
__device__ __forceinline__ int box_of(int half) { return half <= 16 ? 16 : half <= 32 ? 32 : half <= 64 ? 64 : 128; }
__device__ __forceinline__ uint32_t bytes_of(int box) { return kWBytes + box * BK * 2; }

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* m, int x, int y, int z,
                                                 uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// kColumns: weights [G, K, N]
template <bool kColumns>
__global__ void __launch_bounds__(kThreads, 1)
bias_act_kernel(const __grid_constant__ CUtensorMap tm16, const __grid_constant__ CUtensorMap tm32,
                const __grid_constant__ CUtensorMap tm64, const __grid_constant__ CUtensorMap tm128,
                const __grid_constant__ CUtensorMap tmW, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = ptx::smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Smem::BARS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Smem::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Smem::MISC + 4);
  int* scan = reinterpret_cast<int*>(smem + Smem::MISC + 8);
  uint32_t* s_issued = reinterpret_cast<uint32_t*>(smem + Smem::MISC + 48);
  int* start = reinterpret_cast<int*>(smem + Smem::TILES);
  int* goff = reinterpret_cast<int*>(smem + Smem::GOFF);
  int* s_dst = reinterpret_cast<int*>(smem + Smem::DST);
  float* s_w = reinterpret_cast<float*>(smem + Smem::WEIGHT);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0;
  const int unit = static_cast<int>(blockIdx.x >> 1), n_units = static_cast<int>(gridDim.x >> 1);
  auto bar_full = [&](int s) { return ptx::smem_u32(bars + s); };
  auto bar_empty = [&](int s) { return ptx::smem_u32(bars + kStages + s); };
  auto bar_tfull = [&](int a) { return ptx::smem_u32(bars + 2 * kStages + a); };
  auto bar_tempty = [&](int a) { return ptx::smem_u32(bars + 2 * kStages + 2 + a); };
  const uint32_t bar_drain = ptx::smem_u32(bars + 2 * kStages + 4);

  count_launch(p.launches, MOE_KID_GEMM_BIAS_ACT);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(bar_full(s), 1);
      ptx::mbar_init(bar_empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(bar_tfull(a), 1);
      ptx::mbar_init(bar_tempty(a), 16);   // the epilogue warps of both CTAs
    }
    ptx::mbar_init(bar_drain, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::tma_prefetch_desc(&tm16);
    ptx::tma_prefetch_desc(&tm32);
    ptx::tma_prefetch_desc(&tm64);
    ptx::tma_prefetch_desc(&tm128);
    ptx::tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    ptx::tmem_alloc2(ptx::smem_u32(tmem_slot), 2 * kRowBlock);
    ptx::tmem_relinquish2();
  }
  grid_dep_wait();
  grid_dep_launch();

  // ---- tile schedule, the same in every CTA: groups in order, their row blocks, column blocks
  const int G = p.G;
  for (int g = threadIdx.x; g <= G; g += kThreads)
    goff[g] = p.group_offsets ? min(max(__ldg(p.group_offsets + g), 0), p.P) : (g == 0 ? 0 : p.P);
  __syncthreads();
  const int n_fb = (p.N + kColBlock - 1) / kColBlock;
  auto tiles_in = [&](int g) { return (max(goff[g + 1] - goff[g], 0) + p.row_block - 1) / p.row_block * n_fb; };
  const int per = (G + kThreads - 1) / kThreads;
  const int g_lo = min(G, static_cast<int>(threadIdx.x) * per), g_hi = min(G, g_lo + per);
  int local = 0;
  for (int g = g_lo; g < g_hi; ++g) local += tiles_in(g);
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int run = incl - local, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) run += scan[w];
    total += scan[w];
  }
  for (int g = g_lo; g < g_hi; ++g) {
    start[g] = run;
    run += tiles_in(g);
  }
  if (threadIdx.x == 0) start[G] = total;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // the peer's barriers exist before any remote arrive or copy
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int nk = (p.K + BK - 1) / BK, S = p.ranges;
  const int work = total * S;
  bool mma_any = false;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int u = unit; ok && u < work; u += n_units) {
      const Tile t = tile_of(S == 1 ? u : u / S, start, goff, G, n_fb, p.row_block);
      const int sp = S == 1 ? 0 : u % S;
      const int k0 = nk * sp / S, k1 = nk * (sp + 1) / S;
      const int half = half_of(t), box = box_of(half);
      const CUtensorMap* mt = box == 16 ? &tm16 : box == 32 ? &tm32 : box == 64 ? &tm64 : &tm128;
      const int row = t.r0 + static_cast<int>(rank) * half;
      const int col = t.n0 + static_cast<int>(rank) * 128;
      const uint32_t bytes = bytes_of(box);
      for (int kb = k0; kb < k1; ++kb) {
        bool got = true;
        if (lane == 0) {
          got = wait_bar_spin(bar_empty(stage), phase ^ 1u, abort_flag, p.status, p.wait_ns);
          if (got && leader) ptx::mbar_arrive_expect_tx(bar_full(stage), 2 * bytes);
        }
        if (!__shfl_sync(0xffffffffu, got ? 1 : 0, 0)) {
          ok = false;
          break;
        }
        const uint32_t bar = ptx::mapa_shared(bar_full(stage), 0);
        const uint32_t dw = sb + Smem::STAGE_W + stage * kWBytes;
        if (lane == 0)
          ptx::tma_load_2d_pair(sb + Smem::STAGE_T + stage * kTBytes, mt, kb * BK, row, bar);
        if (kColumns) {
          if (lane == 1 || lane == 2)
            tma_load_3d_pair(dw + (lane - 1) * (kWBytes / 2), &tmW, col + 64 * (lane - 1), kb * BK, t.g, bar);
        } else if (lane == 1) {
          tma_load_3d_pair(dw, &tmW, kb * BK, col, t.g, bar);
        }
        ++issued;
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
    if (lane == 0) *s_issued = issued;
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (leader && ptx::elect_one()) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, uses[2] = {0, 0};
      bool ok = true;
      for (int u = unit; ok && u < work; u += n_units) {
        const Tile t = tile_of(S == 1 ? u : u / S, start, goff, G, n_fb, p.row_block);
        const int sp = S == 1 ? 0 : u % S;
        const int k0 = nk * sp / S, k1 = nk * (sp + 1) / S;
        const uint32_t idesc = ptx::idesc_bf16_f32_mn(256, (t.rows + 15) & ~15, kColumns, false);
        if (!wait_bar<true>(bar_tempty(acc), ((acc ? uses[1] : uses[0]) & 1u) ^ 1u, abort_flag, p.status,
                            p.wait_ns))
          break;
        ptx::tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(acc * kRowBlock);
        for (int kb = k0; kb < k1; ++kb) {
          if (!wait_bar(bar_full(stage), phase, abort_flag, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t aw = sb + Smem::STAGE_W + stage * kWBytes;
          const uint64_t dw = kColumns ? ptx::desc_mnmajor_sw128(aw, kWBytes / 2) : ptx::desc_kmajor_sw128(aw);
          const uint64_t dt = ptx::desc_kmajor_sw128(sb + Smem::STAGE_T + stage * kTBytes);
#pragma unroll
          for (int k = 0; k < BK / UMMA_K; ++k)   // 16 K rows of an MN-major block are 2048 bytes
            ptx::mma_bf16_pair(d, dw + (kColumns ? 128ull : 2ull) * k, dt + 2ull * k, idesc,
                               kb != k0 || k != 0 ? 1u : 0u);
          mma_any = true;
          ptx::mma_commit_pair(bar_empty(stage), 3);
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        ptx::mma_commit_pair(bar_tfull(acc), 3);
        if (acc) ++uses[1]; else ++uses[0];
        acc ^= 1;
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int eg = (warp - 2) >> 2;
    const int et = static_cast<int>(threadIdx.x) - 64 - 128 * eg;   // 0..127 in the group
    const int ea = static_cast<int>(threadIdx.x) - 64;              // 0..255 over both
    const int q = warp & 3;                                         // TMEM lane quarter
    // this thread's columns of the CTA's 128: f + 8 i, and its rows of eight: 2 (lane % 4) + 0, 1
    const int f = q * 32 + (lane >> 2), r2 = 2 * (lane & 3);
    const int bar_g = 1 + eg;
    const uint32_t tempty = ptx::mapa_shared(bar_tempty(0), 0);     // + 8 * acc
    // [32 rows][128 columns] bf16, 16-byte pieces XOR-swizzled by the row; for the matrix stores this
    // lane addresses row lane % 8 of each eight, the eight columns q * 32 + 8 (lane / 8)
    const uint32_t ost = sb + Smem::EPI + eg * 8192;
    const int mrow = lane & 7, mpiece = q * 4 + (lane >> 3);
    uint32_t uses[2] = {0, 0};
    int acc = 0;
    for (int u = unit; u < work; u += n_units) {
      const Tile t = tile_of(S == 1 ? u : u / S, start, goff, G, n_fb, p.row_block);
      const int sp = S == 1 ? 0 : u % S;
      const int col0 = t.n0 + static_cast<int>(rank) * 128;
      int* dst_t = s_dst + acc * kRowBlock;
      float* w_t = s_w + acc * kRowBlock;
      float b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        b[i] = p.bias && !p.part && col0 + f + 8 * i < p.N
                   ? __ldg(p.bias + static_cast<size_t>(t.g) * p.N + col0 + f + 8 * i)
                   : 0.0f;
      int d = -1;
      float w = 1.0f;
      if (ea < t.rows) {
        d = p.row_to_pair ? __ldg(p.row_to_pair + t.r0 + ea) : t.r0 + ea;
        if (d < 0 || d >= p.P) d = -1;
        else if (p.pair_weight) w = __ldg(p.pair_weight + d);
      }
      const bool landed = wait_bar(bar_tfull(acc), (acc ? uses[1] : uses[0]) & 1u, abort_flag, p.status, p.wait_ns);
      // the buffer's last readers (two tiles ago) have passed the previous tile's barrier
      dst_t[ea] = d;
      w_t[ea] = w;
      // one decision for the eight warps; publishes dst_t and w_t
      if (!ptx::bar_and(3, 256, landed)) {
        *abort_flag = 1;
        break;
      }
      ptx::tc_fence_after();
      const uint32_t taddr =
          tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * kRowBlock);
      if (32 * eg >= t.rows) {       // no chunk for this group
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote_relaxed(tempty + 8u * acc);
      }
#pragma unroll 1
      for (int j0 = 32 * eg; j0 < t.rows; j0 += 64) {
        uint4 res[4];
        if (p.residual && !p.part) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = (et + 128 * i) >> 4, c = col0 + 8 * (et & 15);
            const int to = j0 + j < t.rows ? dst_t[j0 + j] : -1;
            res[i] = to >= 0 && c < p.N
                         ? *reinterpret_cast<const uint4*>(p.residual + static_cast<size_t>(to) * p.N + c)
                         : make_uint4(0, 0, 0, 0);
          }
        }
        // [column half][row eight j, column + 8 e, row k]: v[h][4 j + 2 e + k]
        uint32_t v[2][16];
        ptx::tmem_ld_16x256b_x4(taddr + static_cast<uint32_t>(j0), v[0]);
        ptx::tmem_ld_16x256b_x4(taddr + (16u << 16) + static_cast<uint32_t>(j0), v[1]);
        ptx::tmem_ld_wait();
        if (j0 + 64 >= t.rows) {     // this warp's last read of the accumulator
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_remote_relaxed(tempty + 8u * acc);
        }
        if (p.part) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int col = col0 + f + 8 * i;
            if (col >= p.N) continue;
            float* to = p.part + (static_cast<size_t>(sp) * p.N + col) * p.part_rows + t.r0 + j0 + r2;
            const bool vec = (reinterpret_cast<uintptr_t>(to) & 7) == 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t lo = v[i >> 1][4 * j + 2 * (i & 1)], hi = v[i >> 1][4 * j + 2 * (i & 1) + 1];
              const int r = j0 + 8 * j + r2;
              if (vec && r + 1 < t.rows) {
                *reinterpret_cast<uint2*>(to + 8 * j) = make_uint2(lo, hi);
              } else {
                if (r < t.rows) to[8 * j] = __uint_as_float(lo);
                if (r + 1 < t.rows) to[8 * j + 1] = __uint_as_float(hi);
              }
            }
          }
          continue;
        }
        uint64_t y[4][4];            // [column f + 8 i][rows 8 j + r2, + 1]
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            y[i][j] = act::add2(ptx::pair(v[i >> 1][4 * j + 2 * (i & 1)], v[i >> 1][4 * j + 2 * (i & 1) + 1]),
                                ptx::pair(b[i]));
        // this group's 32 x 128 values to rows of a [P, N] matrix
        auto store = [&](uint16_t* to, bool scattered) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t pk[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 u = ptx::unpair(y[i][j]);
              pk[i] = pack_bf16x2(u.x, u.y);
            }
            const int row = 8 * j + mrow;
            ptx::stmatrix_x4_trans(ost + row * 256 + ((mpiece ^ (row & 15)) << 4), pk[0], pk[1], pk[2], pk[3]);
          }
          ptx::bar_sync(bar_g, 128);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = (et + 128 * i) >> 4, k = et & 15, c = col0 + 8 * k;
            if (j0 + j < t.rows && c < p.N) {
              const int row = scattered ? dst_t[j0 + j] : t.r0 + j0 + j;
              if (row >= 0)
                *reinterpret_cast<uint4*>(to + static_cast<size_t>(row) * p.N + c) =
                    ptx::ld_shared_v4(ost + j * 256 + ((k ^ (j & 15)) << 4));
            }
          }
          ptx::bar_sync(bar_g, 128);
        };
        if (p.z) store(p.z, false);
        act::dispatch(p.activation, [&](auto a) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[i][j] = act::apply2<decltype(a)::value>(y[i][j]);
        });
        if (p.pair_weight) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t w2 = *reinterpret_cast<const uint64_t*>(w_t + j0 + 8 * j + r2);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i][j] = ptx::mul2(y[i][j], w2);
          }
        }
        if (p.residual) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = (et + 128 * i) >> 4, k = et & 15;
            ptx::st_shared_v4(ost + j * 256 + ((k ^ (j & 15)) << 4), res[i].x, res[i].y, res[i].z, res[i].w);
          }
          ptx::bar_sync(bar_g, 128);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = 8 * j + mrow;
            uint32_t u[4];
            ptx::ldmatrix_x4_trans(ost + row * 256 + ((mpiece ^ (row & 15)) << 4), u);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i][j] = act::add2(y[i][j], ptx::pair(u[i] << 16, u[i] & 0xFFFF0000u));
          }
          __syncwarp();              // this warp's columns are read by it alone before it writes them
        }
        store(p.out, true);
      }
      if (acc) ++uses[1]; else ++uses[0];
      acc ^= 1;
    }
  }

  // ---- exit: if either CTA of the pair gave up, the MMAs and both CTAs' copies are waited for before
  // memory is freed
  __syncthreads();
  ptx::cluster_sync();
  const bool gave_up =
      *abort_flag != 0 ||
      ld_shared_cluster_u32(
          ptx::mapa_shared(ptx::smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u)) != 0;
  if (gave_up) {
    if (mma_any) {
      ptx::mma_commit_pair(bar_drain, 1);
      spin_bounded(bar_drain, 0);
    }
    if (leader && warp == 0 && lane == 0) {
      // uses come in order: u, the work item of the last use asked for, ends before use `end`
      int u = unit - n_units;
      uint32_t end = 0;
      drain_pair_copies<kStages>(
          *s_issued, ld_shared_cluster_u32(ptx::mapa_shared(ptx::smem_u32(s_issued), 1)), bar_full,
          [&](uint32_t i) {
            while (i >= end) {
              u += n_units;
              const int sp = S == 1 ? 0 : u % S;
              end += nk * (sp + 1) / S - nk * sp / S;
            }
            return bytes_of(box_of(half_of(tile_of(S == 1 ? u : u / S, start, goff, G, n_fb, p.row_block))));
          },
          [](uint32_t) { return 0u; });
    }
  }
  __syncthreads();
  ptx::cluster_sync();   // the peer may use this CTA's shared memory or TMEM until here
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc2(tmem, 2 * kRowBlock);
  }
}

// The ranges' sums in range order, then the epilogue: 32 columns x 32 rows a block, the sums
// read along rows (a thread four of them), the outputs written along columns.
__global__ void __launch_bounds__(256) join_kernel(const Params p) {
  __shared__ float s_z[32][33];
  count_launch(p.launches, MOE_KID_BIAS_ACT_JOIN);
  grid_dep_wait();
  grid_dep_launch();
  const int n0 = blockIdx.x * 32, r0 = blockIdx.y * 32;
  {
    const int n = n0 + (threadIdx.x >> 3), r = r0 + (threadIdx.x & 7) * 4;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (n < p.N && r < p.part_rows) {
      const float* q = p.part + static_cast<size_t>(n) * p.part_rows + r;
      const size_t step = static_cast<size_t>(p.N) * p.part_rows;
      float4 v[kMaxRanges];
#pragma unroll
      for (int i = 0; i < kMaxRanges; ++i)
        if (i < p.ranges) v[i] = __ldcg(reinterpret_cast<const float4*>(q + i * step));
      s = v[0];
#pragma unroll
      for (int i = 1; i < kMaxRanges; ++i)
        if (i < p.ranges) {
          s.x += v[i].x; s.y += v[i].y; s.z += v[i].z; s.w += v[i].w;
        }
    }
    float* to = &s_z[(threadIdx.x & 7) * 4][threadIdx.x >> 3];
    to[0] = s.x; to[33] = s.y; to[66] = s.z; to[99] = s.w;
  }
  __syncthreads();
  const int j = threadIdx.x >> 3, r = r0 + j, c = (threadIdx.x & 7) * 4, n = n0 + c;
  if (r >= p.P || n >= p.N) return;  // N % 8 == 0: four columns are in or out together
  int g = 0;
  if (p.group_offsets) {             // the last group that starts at or before r
    auto off = [&](int i) { return min(max(__ldg(p.group_offsets + i), 0), p.P); };
    int lo = 0, hi = p.G;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (off(mid) <= r) lo = mid; else hi = mid;
    }
    g = lo;
    if (r < off(g) || r >= off(g + 1)) return;
  }
  const int d = p.row_to_pair ? __ldg(p.row_to_pair + r) : r;
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    y[i] = s_z[j][c + i] + (p.bias ? __ldg(p.bias + static_cast<size_t>(g) * p.N + n + i) : 0.0f);
  if (p.z)
    *reinterpret_cast<uint2*>(p.z + static_cast<size_t>(r) * p.N + n) =
        make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
  if (d < 0 || d >= p.P) return;
  act::dispatch(p.activation, [&](auto a) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const float2 u = ptx::unpair(act::apply2<decltype(a)::value>(
          ptx::pair(__float_as_uint(y[i]), __float_as_uint(y[i + 1]))));
      y[i] = u.x;
      y[i + 1] = u.y;
    }
  });
  const size_t at = static_cast<size_t>(d) * p.N + n;
  if (p.pair_weight) {
    const float w = __ldg(p.pair_weight + d);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __fmul_rn(y[i], w);
  }
  if (p.residual) {
    const uint2 u = *reinterpret_cast<const uint2*>(p.residual + at);
    y[0] = __fadd_rn(y[0], __uint_as_float(u.x << 16));
    y[1] = __fadd_rn(y[1], __uint_as_float(u.x & 0xFFFF0000u));
    y[2] = __fadd_rn(y[2], __uint_as_float(u.y << 16));
    y[3] = __fadd_rn(y[3], __uint_as_float(u.y & 0xFFFF0000u));
  }
  *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
}

// ------------------------------------------------------------------ calls of few rows
constexpr int kFewRows = 16;         // rows of a CTA
constexpr int kFewWarps = 8;
constexpr int kFewCols = 8;          // output columns of a warp
constexpr int kFewFlight = 4;        // blocks of 64 K that a warp loads together

// 16 bytes, or zeros
__device__ __forceinline__ uint4 load_or_zero(const uint4* from, bool there) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(from), "r"(there ? 1 : 0));
  return v;
}

// Weights [G, N, K].  A warp holds 8 output columns for at most 16 rows of one group and takes K in turn with the other `slices` - 1
// of them, 64 at a time: a lane has 2 x 16 bytes of one of the columns, and the products of 16 rows x 8 columns
// are mma.sync's; a CTA joins the slices' sums in order.  What bounds it is the weights' way from memory: no tensor
// memory to allocate, no second launch, and a warp's loads of four blocks leave at once.  (A lane's 16
// bytes lie elsewhere in the contraction than the MMA has them, alike on both sides.)
// One row of 4096 x 1024 takes 4.3 us from HBM in a row of calls, the CTA pairs' two launches 9.2; 8192 x 8192 24 against 29;
// 1024 x 4096 3.7 against 9.1.  Eight blocks in flight are slower (4096 x 4096: 11.1 against 7.9), as one CTA fits an SM then.
// kTwo: more than eight rows (its 128 registers, two CTAs an SM, spill six: 16 bytes stored, 24 loaded a thread).
template <bool kTwo>
__global__ void __launch_bounds__(32 * kFewWarps, 2)
few_rows_kernel(const uint16_t* __restrict__ a, const uint16_t* __restrict__ w, const Params p, const int slices) {
  __shared__ float s_sum[kFewWarps][kFewRows][kFewCols];
  count_launch(p.launches, MOE_KID_GEMM_BIAS_ACT);
  count_launch(p.launches, MOE_KID_BIAS_ACT_FEW);
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  // the blockIdx.y-th block of at most 16 rows of a group
  int group = 0, r0 = static_cast<int>(blockIdx.y) * kFewRows, rows = min(p.P - r0, kFewRows);
  if (p.group_offsets) {
    int left = static_cast<int>(blockIdx.y);
    rows = 0;
    for (int i0 = 0; i0 < p.G; i0 += 32) {
      const int i = i0 + lane;
      const int lo = min(max(i < p.G ? __ldg(p.group_offsets + i) : 0, 0), p.P);
      const int hi = min(max(i < p.G ? __ldg(p.group_offsets + i + 1) : 0, 0), p.P);
      const int own = hi > lo ? (hi - lo + kFewRows - 1) / kFewRows : 0;
      int upto = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const uint32_t behind = __ballot_sync(0xffffffffu, upto > left);
      if (behind == 0) {
        left -= __shfl_sync(0xffffffffu, upto, 31);
        continue;
      }
      const int at = __ffs(behind) - 1;
      left -= __shfl_sync(0xffffffffu, upto - own, at);
      group = i0 + at;
      r0 = __shfl_sync(0xffffffffu, lo, at) + left * kFewRows;
      rows = min(__shfl_sync(0xffffffffu, hi, at) - r0, kFewRows);
      break;
    }
    if (rows == 0) return;
  }
  const int per = kFewWarps / slices;            // blocks of columns of a CTA
  const int slice = warp / per, n0 = (blockIdx.x * per + warp % per) * kFewCols, K = p.K, vecs = n0 < p.N ? K >> 3 : 0;
  const uint4* wv = reinterpret_cast<const uint4*>(w + (static_cast<size_t>(group) * p.N + n0 + g) * K);
  const uint4* a0 = reinterpret_cast<const uint4*>(a + static_cast<size_t>(r0 + min(g, rows - 1)) * K);
  const uint4* a1 = reinterpret_cast<const uint4*>(a + static_cast<size_t>(r0 + min(g + 8, rows - 1)) * K);
  const bool has0 = g < rows, has1 = kTwo && g + 8 < rows;
  float c[2][4] = {};                // two sums, two chains: rows g (0, 1) and g + 8 (2, 3), columns 2 q, 2 q + 1
#pragma unroll 1
  for (int b0 = slice; b0 * 8 < vecs; b0 += slices * kFewFlight) {
    uint4 b[kFewFlight][2], u[kFewFlight][2], v[kTwo ? kFewFlight : 1][2];
#pragma unroll
    for (int i = 0; i < kFewFlight; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = (b0 + i * slices) * 8 + 2 * q + h;
        b[i][h] = load_or_zero(wv + at, at < vecs);
        u[i][h] = load_or_zero(a0 + at, has0 && at < vecs);
        if (kTwo) v[i][h] = load_or_zero(a1 + at, has1 && at < vecs);
      }
    // keeps the products behind all of the loads: ptxas else sinks each load to its use, in turn
    asm volatile("fence.acq_rel.cta;" ::: "memory");
#pragma unroll
    for (int i = 0; i < kFewFlight; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 x = u[i][h], y = kTwo ? v[kTwo ? i : 0][h] : make_uint4(0, 0, 0, 0), w4 = b[i][h];
        ptx::mma_m16n8k16(c[0], x.x, y.x, x.y, y.y, w4.x, w4.y);
        ptx::mma_m16n8k16(c[1], x.z, y.z, x.w, y.w, w4.z, w4.w);
      }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s_sum[warp][g + 8 * (j >> 1)][2 * q + (j & 1)] = c[0][j] + c[1][j];
  __syncthreads();
  // two columns a thread
#pragma unroll 1
  for (int i = threadIdx.x; i < per * kFewCols / 2 * rows; i += 32 * kFewWarps) {
    const int j = i / (per * kFewCols / 2), c2 = i - j * (per * kFewCols / 2), block = c2 / (kFewCols / 2);
    const int n = blockIdx.x * per * kFewCols + 2 * c2, r = r0 + j;
    if (n >= p.N) continue;
    float2 z = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kFewWarps; ++k) {
      if (k >= slices) break;
      const float2 v = *reinterpret_cast<const float2*>(&s_sum[k * per + block][j][2 * c2 - block * kFewCols]);
      z.x += v.x;
      z.y += v.y;
    }
    if (p.bias) {
      z.x += __ldg(p.bias + static_cast<size_t>(group) * p.N + n);
      z.y += __ldg(p.bias + static_cast<size_t>(group) * p.N + n + 1);
    }
    if (p.z) *reinterpret_cast<uint32_t*>(p.z + static_cast<size_t>(r) * p.N + n) = pack_bf16x2(z.x, z.y);
    const int d = p.row_to_pair ? __ldg(p.row_to_pair + r) : r;
    if (d < 0 || d >= p.P) continue;
    float2 y = z;
    act::dispatch(p.activation, [&](auto k) {
      y = ptx::unpair(act::apply2<decltype(k)::value>(ptx::pair(__float_as_uint(z.x), __float_as_uint(z.y))));
    });
    const size_t to = static_cast<size_t>(d) * p.N + n;
    if (p.pair_weight) {
      const float f = __ldg(p.pair_weight + d);
      y.x = __fmul_rn(y.x, f);
      y.y = __fmul_rn(y.y, f);
    }
    if (p.residual) {
      const uint32_t u = *reinterpret_cast<const uint32_t*>(p.residual + to);
      y.x = __fadd_rn(y.x, __uint_as_float(u << 16));
      y.y = __fadd_rn(y.y, __uint_as_float(u & 0xFFFF0000u));
    }
    *reinterpret_cast<uint32_t*>(p.out + to) = pack_bf16x2(y.x, y.y);
  }
}

// ------------------------------------------------------------------ host side
constexpr int kLeastBlock = 64;      // rows of a tile where they are few
long long row_blocks(int P, int G, int block) {
  return G == 1 ? (static_cast<long long>(P) + block - 1) / block : P / block + (G < P ? G : P);
}
long long col_blocks(int N) { return (N + kColBlock - 1ll) / kColBlock; }
// Ranges of K for `blocks` row blocks: as many as fill the pairs, each of at least kRangeSteps
// steps.  One row of 4096 x 1024 takes 4 tiles of 64 steps: 16 ranges, 64 pairs at work.
int ranges_of(long long blocks, int K, int N) {
  const long long tiles = blocks * col_blocks(N);
  long long s = sm_count() / 2 / tiles;
  const long long most = (K + BK - 1ll) / BK / kRangeSteps;
  s = s < most ? s : most;
  s = s < kMaxRanges ? s : kMaxRanges;
  return s < 1 ? 1 : static_cast<int>(s);
}
// blocks of 16 rows of a group, at most
int few_blocks(int P, int G) {
  if (G == 1) return P / kFewRows + (P % kFewRows != 0);
  const int blocks = P / kFewRows + (G < P ? G : P);
  return blocks < P ? blocks : P;
}
// Slices of K in the kernel of few rows, or 0: the pairs' kernel.  The most slices with which all CTAs (two per SM) run at once:
// one row of 4096 x 4096 takes 7.9 us with 4 slices and 256 CTAs, 9.1 with 8 and 512, 10.7 with 2 and 128.
// Every block of 16 rows reads the weights anew, so with several of them a warp may have four batches of K, each a
// latency: 128 rows of 512 x 512 2.9 us (pairs 8.0), 64 rows of 2048 x 768 6.1 (8.5), in 8 groups 8.9 (12.4), 48 rows of
// 4096 x 1024, four batches, 9.4 (9.8); with eight batches 32 rows of 4096 x 4096 take 16.1 (13.0).  One block takes any
// K, and where a single slice leaves more CTAs than two per SM at most eight rows: 16 rows of 1024 x 32768 19 us against
// 15.5, eight 14.7.
int few_slices(int P, int K, int N, int G) {
  for (int s = kFewWarps; s; s >>= 1) {
    const long long cols = kFewCols * kFewWarps / s;
    if ((N + cols - 1) / cols * few_blocks(P, G) <= 2 * sm_count())
      return P <= kFewRows || K <= 4 * kFewFlight * 64 * s ? s : 0;
  }
  return P > 8 ? 0 : 1;
}
size_t part_bytes(int ranges, long long rows, int N) {
  return ranges < 2 ? 0 : static_cast<size_t>(ranges) * N * ((rows + 3) & ~3ll) * 4;
}

// Rows of a tile and ranges of K.  Where every tile has a pair of its own, fewer rows make the epilogue shorter (it takes
// chunks of 64 rows in turn) and save ranges, whose sums go to memory and back; but more tiles leave fewer ranges, and a
// pair more K steps.  The estimate is in ns: 350 a K step (a stage's way, with six under way), 600 a chunk, 2500 for a second
// launch, and for a range's sums 1.5 ps each (4 where groups begin at odd rows).  What it chooses: 2000 rows of 1024 x 512 in 8
// groups 128 rows and one range, 12.3 us (256 rows and two ranges: 27.6); 777 rows of 1040 x 1000 in 13 groups
// 128 rows, 12.1 (256: 13.3); 1024 rows of 4096 x 512 128 rows and four ranges, 18.0 (256 and nine 17.0, 64 and two 22.5).
void plan(Params& p) {
  double best = 0.0;
  for (int block = kRowBlock; block >= kLeastBlock; block /= 2) {
    const long long blocks = row_blocks(p.P, p.G, block), tiles = blocks * col_blocks(p.N);
    if (block < kRowBlock && tiles > sm_count() / 2) break;
    const int s = ranges_of(blocks, p.K, p.N), steps = ((p.K + BK - 1) / BK + s - 1) / s;
    const double rows = block < p.P ? block : p.P;
    const double t = 350.0 * steps + 600.0 * ((static_cast<int>(rows) + 63) / 64) +
                     (s > 1 ? 2500.0 + (p.G > 1 ? 4e-3 : 1.5e-3) * s * p.P * p.N : 0.0);
    if (block == kRowBlock || t < best) {
      best = t;
      p.row_block = block;
      p.ranges = s;
    }
  }
}

template <bool kColumns>
int launch(const char* op, const CUtensorMap (&tt)[4], const CUtensorMap& tw, Params p, cudaStream_t stream) {
  auto kern = bias_act_kernel<kColumns>;
  static std::atomic<int> configured[64] = {};
  static std::atomic<int> resident[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    dev = -1;
  }
  const bool cache = dev >= 0 && dev < 64;
  if (!cache || !configured[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::ALLOC) != cudaSuccess)
      return set_error(MOE_ERR_CUDA, "%s: cannot reserve %d bytes of shared memory: %s", op, Smem::ALLOC,
                       cudaGetErrorString(cudaGetLastError()));
    if (cache) configured[dev].store(1, std::memory_order_release);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // a pair sits in one GPC, so fewer than SMs / 2 may fit at once
  int pairs = cache ? resident[dev].load(std::memory_order_relaxed) : 0;
  if (pairs <= 0) {
    pairs = num_sms() / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Smem::ALLOC;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) == cudaSuccess && clusters > 0)
      pairs = clusters < pairs ? clusters : pairs;
    else
      cudaGetLastError();
    if (cache) resident[dev].store(pairs, std::memory_order_relaxed);
  }
  const long long work = row_blocks(p.P, p.G, p.row_block) * col_blocks(p.N) * p.ranges;
  if (work < pairs) pairs = work < 1 ? 1 : static_cast<int>(work);
  DeviceDiag diag = device_diag();
  p.status = diag.status;
  p.launches = diag.launches;
  p.wait_ns = pipeline_wait_ns();
  const int rc = launch_status(
      launch_kernel(kern, dim3(static_cast<unsigned>(2 * pairs), 1, 1), dim3(kThreads, 1, 1), Smem::ALLOC, stream,
                    attr, 1, tt[0], tt[1], tt[2], tt[3], tw, p),
      op);
  if (rc != MOE_OK || !p.part) return rc;
  return launch_status(launch_kernel(join_kernel, dim3((p.N + 31) / 32, (p.P + 31) / 32), dim3(256), 0, stream,
                                     nullptr, 0, p),
                       op);
}

}  // namespace
}  // namespace gemm
}  // namespace moe

using namespace moe;
using namespace moe::gemm;

extern "C" size_t moe_grouped_gemm_bias_act_workspace_size(int P, int K, int N, int G) {
  if (P <= 0 || K <= 0 || N <= 0 || G <= 0) return 0;
  // the most that any number of rows up to P takes, whatever the tiles: a workspace for the largest call serves all
  size_t most = 0;
  for (int block = kLeastBlock; block <= kRowBlock; block *= 2)
    for (long long b = 1; b <= row_blocks(P, G, block); ++b) {
      const int s = ranges_of(b, K, N);
      if (s < 2) break;
      const long long rows = b * block < P ? b * block : P;
      const size_t n = part_bytes(s, rows, N);
      most = n > most ? n : most;
    }
  return most;
}

extern "C" int moe_grouped_gemm_bias_act_bf16(const void* a_bf16, const void* w_bf16, int w_layout,
                                              const float* bias, int activation, void* pre_act_bf16,
                                              const float* pair_weight, const int32_t* row_to_pair,
                                              const void* residual_bf16, const int32_t* group_offsets, int P,
                                              int K, int N, int G, void* out_bf16, void* workspace,
                                              size_t ws_bytes, void* stream) {
  clear_error();
  const char* op = "moe_grouped_gemm_bias_act_bf16";
  if (P < 0 || K < 1 || N < 1) return set_error(MOE_ERR_ARG, "%s: P=%d, K=%d, N=%d", op, P, K, N);
  if (P > kMaxDim || K > kMaxDim || N > kMaxDim)
    return set_error(MOE_ERR_ARG, "%s: P=%d, K=%d or N=%d is too large", op, P, K, N);
  if (G < 1 || G > kMaxGroups) return set_error(MOE_ERR_ARG, "%s: G=%d outside [1, %d]", op, G, kMaxGroups);
  if (w_layout != MOE_W_ROWS && w_layout != MOE_W_COLUMNS)
    return set_error(MOE_ERR_ARG, "%s: w_layout=%d is not MOE_W_ROWS or MOE_W_COLUMNS", op, w_layout);
  if (activation < MOE_ACT_NONE || activation > MOE_ACT_SILU)
    return set_error(MOE_ERR_ARG, "%s: activation=%d is not a MOE_ACT_* value", op, activation);
  if (K % 8 || N % 8) return set_error(MOE_ERR_ALIGN, "%s: K=%d and N=%d must be multiples of 8", op, K, N);
  if (row_blocks(P, G, kRowBlock) * col_blocks(N) > kMaxDim)
    return set_error(MOE_ERR_ARG, "%s: P=%d and N=%d are too large together", op, P, N);
  if (P == 0) return MOE_OK;
  if (!a_bf16 || !w_bf16 || !out_bf16) return set_error(MOE_ERR_ARG, "%s: a, w or out is NULL", op);
  if (!group_offsets && G != 1) return set_error(MOE_ERR_ARG, "%s: group_offsets is NULL with G=%d", op, G);
  for (const void* q : {a_bf16, w_bf16, const_cast<const void*>(pre_act_bf16), residual_bf16,
                        const_cast<const void*>(out_bf16), const_cast<const void*>(workspace)})
    if (q && !aligned16(q))
      return set_error(MOE_ERR_ALIGN, "%s: bf16 matrices and workspace must be 16-byte aligned", op);
  for (const void* q : {static_cast<const void*>(bias), static_cast<const void*>(pair_weight),
                        static_cast<const void*>(row_to_pair), static_cast<const void*>(group_offsets)})
    if (reinterpret_cast<uintptr_t>(q) & 3u)
      return set_error(MOE_ERR_ALIGN, "%s: bias, weights and indices must be 4-byte aligned", op);
  Params p{};
  p.group_offsets = group_offsets;
  p.P = P; p.K = K; p.N = N; p.G = G;
  p.bias = bias;
  p.activation = activation;
  p.z = static_cast<uint16_t*>(pre_act_bf16);
  p.pair_weight = pair_weight;
  p.row_to_pair = row_to_pair;
  p.residual = static_cast<const uint16_t*>(residual_bf16);
  p.out = static_cast<uint16_t*>(out_bf16);
  if (w_layout == MOE_W_ROWS) {
    const int slices = few_slices(P, K, N, G), cols = kFewCols * kFewWarps / (slices ? slices : 1);
    if (slices) {
      const DeviceDiag diag = device_diag();
      p.launches = diag.launches;
      return launch_status(launch_kernel(P > 8 ? few_rows_kernel<true> : few_rows_kernel<false>,
                                         dim3((N + cols - 1) / cols, few_blocks(P, G)), dim3(32 * kFewWarps), 0,
                                         static_cast<cudaStream_t>(stream), nullptr, 0,
                                         static_cast<const uint16_t*>(a_bf16), static_cast<const uint16_t*>(w_bf16), p,
                                         slices),
                           op);
    }
  }
  p.part_rows = (P + 3) & ~3;
  plan(p);
  const size_t one = part_bytes(2, P, N) / 2, fit = workspace ? ws_bytes / one : 0;
  if (static_cast<size_t>(p.ranges) > fit) p.ranges = static_cast<int>(fit);
  if (p.ranges < 2) p.ranges = 1;
  p.part = p.ranges > 1 ? static_cast<float*>(workspace) : nullptr;
  CUtensorMap tt[4], tw;
  int rc;
  for (int i = 0; i < 4; ++i)
    if ((rc = make_tmap(&tt[i], a_bf16, P, K, 16 << i, op, "a")) != MOE_OK) return rc;
  const bool columns = w_layout == MOE_W_COLUMNS;
  if ((rc = make_tmap3(&tw, w_bf16, G, columns ? K : N, columns ? N : K, columns ? BK : 128, op, "w")) != MOE_OK)
    return rc;
  return columns ? launch<true>(op, tt, tw, p, static_cast<cudaStream_t>(stream))
                 : launch<false>(op, tt, tw, p, static_cast<cudaStream_t>(stream));
}
