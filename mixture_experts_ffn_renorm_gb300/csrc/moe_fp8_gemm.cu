// moe_fp8_gemm.cu -- the grouped products of E4M3 activations and E4M3 weights
// (moe_grouped_gemm_fp8, moe_grouped_gemm_gateup_silu_fp8) on CTA pairs.
//
// y[r,n] = sum_b (sa[r,b] sw[n,b]) p_b[r,n], p_b the product over the 128
// columns of scale block b.  The scales change with every block of the
// contraction, so the tensor core sums one block at a time: each block's MMAs
// start a fresh accumulator in tensor memory, and eight epilogue warps per CTA
// join the blocks in registers, acc += p_b * s_b, while the tensor core fills the
// next accumulators.
//
// As in moe_gemm_pair.cu a tile has weight rows on the MMA's M side (256: 128
// per SM, one tcgen05.mma.cta_group::2) and up to 256 rows of one group on its
// N side, so a group pads to 16 rows and the same tile serves single tokens.
// The round trip MMA -> join -> MMA crosses the pair and takes about as long as
// two blocks' MMAs, so the accumulators are a ring: the tile's rows go in parts
// of 128, each with an MMA sequence and one of four accumulators of its own (parts
// of 64 and eight accumulators when no group has more than 64 rows).
//
// A thread of the epilogue owns one weight row and half of every part's rows: 128
// sums.  The factors s_b[r] = sa[r,b] * sw[b] are the same for every weight row of
// a scale block, so two warps form them once per CTA and block in shared memory,
// and the epilogue reads four per 16-byte broadcast load.  They arrive on the same
// barrier as the part's MMAs, so the epilogue waits once per part.  (tcgen05.ld
// in the 16x256b shape would need a fourth of those loads and feed stmatrix, but
// moves 1024 words in 64 cycles; the 32x32b shape used here takes 18.)
//
//   warp 0      TMA producer: the CTA's weight rows and its half of each part's
//               token rows, 128 bytes (one scale block) of each per stage
//   warp 1      tensor memory; in the even CTA the one thread that issues MMAs
//   warps 2-3   the factors s_b
//   warps 4-11  block joins and the epilogue
//
// gate/up: a CTA's 128 weight rows are 64 up rows, then the 64 gate rows of the
// same features.  Both are narrowed to bf16 into a token-major staging buffer;
// four threads per row then form silu(gate) * up of 16 features each in f32.  The
// largest magnitude of a row's 128 features spans both CTAs of the pair: each
// writes its own to both through distributed shared memory, and after one
// cluster-scope barrier per tile both quantise with the same scale.
//
// The tile schedule, the bounded waits and the exit of a CTA that gives up are
// those of moe_gemm_pair.cu.
#include <atomic>

#include "fp8_common.cuh"

namespace moe {
namespace fp8 {
namespace {

using gemm::wait_bar;
using gemm::wait_bar_spin;

// Bounded wait (see gemm::wait_bar) for the loops that run once per scale block and
// warp, where every instruction counts: the probe without a time hint (the one with a
// hint is a software loop around it), and no result.  A wait that gives up raises the
// status and the CTA's abort flag; its warp goes on with what is there, its later waits
// end at once, and it stops at the tile's vote.
__device__ __forceinline__ void wait_lean(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          unsigned int* status, unsigned long long limit_ns) {
  if (!ptx::mbar_try_wait(bar, parity)) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(bar, parity) && !*abort_flag) {
      if (ptx::globaltimer_ns() - t0 > limit_ns) {
        if (status) atomicOr(status, static_cast<unsigned int>(MOE_STATUS_TIMEOUT));
        *abort_flag = 1;
      }
    }
  }
  __syncwarp();
}

// The accumulator of part r of block kb of a tile of np parts: every tile begins with
// accumulator 0, and blocks of one parity, whose factors share a slot, share
// accumulators.
__device__ __forceinline__ int acc_of(int kb, int r, int np, bool small) {
  return small ? kb & 7 : 2 * (kb & 1) + (np == 2 ? r : (kb >> 1) & 1);
}

constexpr int kThreads = 384;
constexpr int kAuxRegs = 72, kEpiRegs = 216;
// the split draws on the registers the block was launched with (168 a thread)
static_assert(128 * kAuxRegs + 256 * kEpiRegs <= 384 * 168, "register split");
constexpr int kTokBlock = 256;              // rows per tile at most (MMA N)
constexpr int kPart = 128;                  // rows per accumulator
constexpr int kSmallPart = 64;              // the same in launches without larger groups
constexpr int kMaxAcc = 512 / kSmallPart;
constexpr int kStages = 6;
constexpr int kStageBytes = 128 * 128;      // one operand's stage per CTA, at most
constexpr int kMaxGroupsLaunch = 512;       // groups of one launch (schedule in shared memory)
constexpr int kMmaK = 32;                   // K per tcgen05.mma of 8-bit types
constexpr unsigned long long kCopyGraceNs = 100000ull;  // see moe_gemm_pair.cu

template <bool kGU>
struct Smem {
  static constexpr int kVecs = kGU ? 3 : 1;   // factor vectors per block: rows, or gate, up, up of the next block
  static constexpr int kSlots = 2;            // blocks the factors run ahead: at most the ring's, see below
  static constexpr int kSlotBytes = kVecs * kTokBlock * 4;
  static constexpr int W = 0;
  static constexpr int T = W + kStages * kStageBytes;
  static constexpr int EPI = T + kStages * kStageBytes;         // two of [32 rows][128 features] bf16
  static constexpr int FAC = EPI + 2 * 8192;                    // factor ring
  static constexpr int META = FAC + kSlots * kSlotBytes;        // dst and weight, or row maxima
  static constexpr int BARS = META + 4096;
  // full, empty [kStages], tfull, tempty [kMaxAcc], sempty [kSlots], drain, maxima [2]
  static constexpr int NBARS = 2 * kStages + 2 * kMaxAcc + kSlots + 3;
  static constexpr int MISC = BARS + NBARS * 8;                 // tmem slot, abort flag, scan
  static constexpr int TILE_START = MISC + 96;
  static constexpr int GOFF = TILE_START + (kMaxGroupsLaunch + 1) * 4;
  static constexpr int ALLOC = GOFF + (kMaxGroupsLaunch + 1) * 4 + 1024;
  static_assert(ALLOC <= 227 * 1024, "shared memory");
};

struct KernelParams {
  GemmParams g;
  int rows_per_group;            // weight rows of a group
  unsigned long long wait_ns;
  unsigned int* status;
  unsigned long long* launches;
};

struct Tile {
  int g, r0, n_tok, n0;
};

__device__ __forceinline__ Tile tile_at(int tile, const int* tile_start, const int* goff, int G,
                                        int n_fb, int fb_cols) {
  int lo = 0, hi = G;  // tile_start[lo] <= tile < tile_start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile_start[mid] <= tile) lo = mid; else hi = mid;
  }
  const int local = tile - tile_start[lo];
  const int m = local / n_fb;
  Tile t;
  t.g = lo;
  t.r0 = goff[lo] + m * kTokBlock;
  t.n_tok = min(goff[lo + 1], t.r0 + kTokBlock) - t.r0;
  t.n0 = (local - m * n_fb) * fb_cols;
  return t;
}

__device__ __forceinline__ int group_tiles(int rows, int n_fb) {
  return rows > 0 ? (rows + kTokBlock - 1) / kTokBlock * n_fb : 0;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

template <bool kGU>
__global__ void __launch_bounds__(kThreads, 1)
fp8_pair_kernel(const __grid_constant__ CUtensorMap tmT16, const __grid_constant__ CUtensorMap tmT32,
                const __grid_constant__ CUtensorMap tmT64, const __grid_constant__ CUtensorMap tmW,
                const KernelParams kp) {
  using S = Smem<kGU>;
  const GemmParams& p = kp.g;
  constexpr int kFbCols = kGU ? 128 : 256;   // output features per tile (both CTAs)
  constexpr int kWBox = kGU ? 64 : 128;      // weight rows per TMA box
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::MISC + 4);
  int* scan_tmp = reinterpret_cast<int*>(smem + S::MISC + 8);   // one int per warp
  int* tile_start = reinterpret_cast<int*>(smem + S::TILE_START);
  int* goff = reinterpret_cast<int*>(smem + S::GOFF);

  // opaque, so that the inner loops hold them in registers instead of reading them anew
  int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("" : "+r"(warp), "+r"(lane));
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0;
  const int unit = static_cast<int>(blockIdx.x >> 1);
  const int n_units = static_cast<int>(gridDim.x >> 1);
  const uint32_t bars = sbase + S::BARS;
  auto bar_full = [&](int s) { return bars + 8u * s; };
  auto bar_empty = [&](int s) { return bars + 8u * (kStages + s); };
  auto bar_tfull = [&](int a) { return bars + 8u * (2 * kStages + a); };
  auto bar_tempty = [&](int a) { return bars + 8u * (2 * kStages + kMaxAcc + a); };
  auto bar_sempty = [&](int s) { return bars + 8u * (2 * kStages + 2 * kMaxAcc + s); };
  const uint32_t bar_drain = bars + 8u * (S::NBARS - 3);
  auto bar_max = [&](int h) { return bars + 8u * (S::NBARS - 2 + h); };

  count_launch(kp.launches, p.kid);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(bar_full(s), 1);    // the even CTA's expect-tx arrive
      ptx::mbar_init(bar_empty(s), 1);   // the pair's MMA commit
    }
    for (int a = 0; a < kMaxAcc; ++a) {
      ptx::mbar_init(bar_tfull(a), 3);    // the pair's MMA commit and the CTA's factor warps
      ptx::mbar_init(bar_tempty(a), 16);  // one arrive per epilogue warp of both CTAs
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(bar_sempty(s), 8);   // the epilogue warps
      ptx::mbar_init(bar_max(s), 8);      // a group's four warps in both CTAs
    }
    ptx::mbar_init(bar_drain, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::tma_prefetch_desc(&tmT16);
    ptx::tma_prefetch_desc(&tmT32);
    ptx::tma_prefetch_desc(&tmT64);
    ptx::tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    ptx::tmem_alloc2(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish2();
  }

  grid_dep_wait();
  grid_dep_launch();

  // ---- device-side tile schedule (every CTA computes the same one)
  const int G = p.G;
  for (int g = threadIdx.x; g <= G; g += kThreads)
    goff[g] = p.group_offsets ? max(0, min(p.P, __ldg(p.group_offsets + g))) : (g == 0 ? 0 : p.P);
  __syncthreads();
  const int n_fb = (p.N + kFbCols - 1) / kFbCols;
  const int chunk = (G + kThreads - 1) / kThreads;
  const int g_lo = min(G, static_cast<int>(threadIdx.x) * chunk);
  const int g_hi = min(G, g_lo + chunk);
  int local = 0, rows_max = 0;
  for (int g = g_lo; g < g_hi; ++g) {
    const int rows = goff[g + 1] - goff[g];
    local += group_tiles(rows, n_fb);
    rows_max = max(rows_max, rows);
  }
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan_tmp[warp] = incl;
  const bool small = __syncthreads_or(rows_max > kSmallPart) == 0;
  int warp_base = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    const int v = scan_tmp[w];
    if (w < warp) warp_base += v;
    total += v;
  }
  int run = warp_base + incl - local;
  for (int g = g_lo; g < g_hi; ++g) {
    tile_start[g] = run;
    run += group_tiles(goff[g + 1] - goff[g], n_fb);
  }
  if (threadIdx.x == 0) tile_start[G] = total;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // the peer's barriers exist before any remote arrive or copy
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int nk = blocks_of(p.K);
  const int part = small ? kSmallPart : kPart;
  auto tile_of = [&](int tile) { return tile_at(tile, tile_start, goff, G, n_fb, kFbCols); };

  bool mma_any = false;

  if (warp < 4) {
    ptx::setmaxnreg_dec<kAuxRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer
      // lane 0 the first weight box (up rows, or all), lane 1 the gate rows, lanes 2
      // and 3 the CTA's half of the tokens of the tile's one or two parts
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = unit; ok && tile < total; tile += n_units) {
        const Tile t = tile_of(tile);
        const int np = t.n_tok > kPart ? 2 : 1;
        auto half_of = [&](int s) { return ((min(kPart, t.n_tok - kPart * s) + 15) & ~15) >> 1; };
        auto box_of = [&](int half) { return half <= 16 ? 16 : (half <= 32 ? 32 : 64); };
        const int box0 = box_of(half_of(0)), box1 = np == 2 ? box_of(half_of(1)) : 0;
        const uint32_t bytes = kStageBytes + (box0 + box1) * 128;
        const int wrow = t.g * kp.rows_per_group + t.n0 + static_cast<int>(rank) * (kFbCols / 2);
        const int s = lane == 3 ? 1 : 0;
        const int tbox = s ? box1 : box0;
        const bool issues = lane == 0 || lane == 2 || (kGU && lane == 1) || (np == 2 && lane == 3);
        const CUtensorMap* mbox =
            lane < 2 ? &tmW : (tbox == 16 ? &tmT16 : (tbox == 32 ? &tmT32 : &tmT64));
        const int ybox = lane >= 2 ? t.r0 + kPart * s + static_cast<int>(rank) * half_of(s)
                                   : (kGU && lane == 0 ? wrow + p.N : wrow);
        const uint32_t dbox = lane >= 2 ? S::T + s * (kStageBytes / 2) : S::W + (lane == 1 ? kWBox * 128 : 0);
        for (int kb = 0; kb < nk; ++kb) {
          bool got = true;
          if (lane == 0) {
            // spinning: the producer's reaction time is part of the ring's round trip
            got = wait_bar_spin(bar_empty(stage), phase ^ 1u, abort_flag, kp.status, kp.wait_ns);
            if (got && leader) ptx::mbar_arrive_expect_tx(bar_full(stage), 2 * bytes);
          }
          if (!__shfl_sync(0xffffffffu, got ? 1 : 0, 0)) {
            ok = false;
            break;
          }
          // the maps see pairs of codes as 2-byte elements: 64 of them per scale block
          if (issues)
            ptx::tma_load_2d_pair(sbase + dbox + stage * kStageBytes, mbox, kb * 64, ybox,
                                  ptx::mapa_shared(bar_full(stage), 0));
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer (even CTA)
      if (leader && ptx::elect_one()) {
        int stage = 0;
        uint32_t phase = 0, free_mask = 0;   // a bit per accumulator: parity of its next release
        bool ok = true;
        for (int tile = unit; ok && tile < total; tile += n_units) {
          const Tile t = tile_of(tile);
          const int np = t.n_tok > kPart ? 2 : 1;
          for (int kb = 0; ok && kb < nk; ++kb) {
            ok = wait_bar(bar_full(stage), phase, abort_flag, kp.status, kp.wait_ns);
            for (int r = 0; ok && r < np; ++r) {
              const int acc = acc_of(kb, r, np, small);
              ok = wait_bar<true>(bar_tempty(acc), ((free_mask >> acc) & 1u) ^ 1u, abort_flag,
                                  kp.status, kp.wait_ns);
              if (!ok) break;
              free_mask ^= 1u << acc;
              ptx::tc_fence_after();
              const uint32_t idesc = ptx::idesc_e4m3_f32(256, (min(kPart, t.n_tok - kPart * r) + 15) & ~15);
              const uint64_t dw = ptx::desc_kmajor_sw128(sbase + S::W + stage * kStageBytes);
              const uint64_t dt =
                  ptx::desc_kmajor_sw128(sbase + S::T + stage * kStageBytes + r * (kStageBytes / 2));
              const uint32_t d = tmem_base + static_cast<uint32_t>(acc * part);
#pragma unroll
              for (int k = 0; k < kBlk / kMmaK; ++k)   // a fresh sum per scale block
                ptx::mma_e4m3_pair(d, dw + 2ull * k, dt + 2ull * k, idesc, k != 0 ? 1u : 0u);
              mma_any = true;
              ptx::mma_commit_pair(bar_tfull(acc), 3);     // the part's sums are ready in both
            }
            if (!ok) break;
            ptx::mma_commit_pair(bar_empty(stage), 3);     // frees the stage in both CTAs
            if (++stage == kStages) { stage = 0; phase ^= 1u; }
          }
        }
      }
    } else {
      // ---------------------------------------------------------- factors
      // 64 threads, rows st, st + 64, ... of the tile; the scales are loaded two
      // blocks ahead.  A slot is written again once the epilogue has passed its last
      // block; the accumulators of a slot's blocks are its own, so they are then in
      // their next turn and an arrive on a part's barrier never meets the turn before.
      const int st = static_cast<int>(threadIdx.x) - 64;
      const int rb = blocks_of(kp.rows_per_group);
      uint32_t free_mask = 0;   // a bit per slot: parity of its next release
      for (int tile = unit; !*abort_flag && tile < total; tile += n_units) {
        const Tile t = tile_of(tile);
        const int np = t.n_tok > kPart ? 2 : 1;
        const int first = t.n0 + static_cast<int>(rank) * (kFbCols / 2);
        const float* sw = p.sw + static_cast<size_t>(t.g) * rb * nk;
        int w_at[S::kVecs];
        w_at[0] = min(first / kBlk, rb - 1) * nk;
        if (kGU) {
          w_at[S::kVecs > 1 ? 1 : 0] = min((p.N + first) / kBlk, rb - 1) * nk;
          w_at[S::kVecs > 2 ? 2 : 0] = min((p.N + first) / kBlk + 1, rb - 1) * nk;
        }
        const float* sa = p.sa + static_cast<size_t>(t.r0) * nk;
        int a_at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a_at[i] = min(st + 64 * i, t.n_tok - 1) * nk;
        auto load = [&](int kb, float (&a)[4], float (&w)[S::kVecs]) {
          const int k = min(kb, nk - 1);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (64 * i < t.n_tok) a[i] = __ldg(sa + a_at[i] + k);
#pragma unroll
          for (int v = 0; v < S::kVecs; ++v) w[v] = __ldg(sw + w_at[v] + k);
        };
        float a0[4] = {}, w0[S::kVecs], a1[4] = {}, w1[S::kVecs];
        load(0, a0, w0);
        load(1, a1, w1);
        for (int kb = 0; kb < nk; ++kb) {
          float ca[4], cw[S::kVecs];
#pragma unroll
          for (int i = 0; i < 4; ++i) { ca[i] = a0[i]; a0[i] = a1[i]; }
#pragma unroll
          for (int v = 0; v < S::kVecs; ++v) { cw[v] = w0[v]; w0[v] = w1[v]; }
          load(kb + 2, a1, w1);
          const int slot = kb & 1;
          wait_lean(bar_sempty(slot), ((free_mask >> slot) & 1u) ^ 1u, abort_flag, kp.status, kp.wait_ns);
          free_mask ^= 1u << slot;
          const uint32_t at = sbase + S::FAC + slot * S::kSlotBytes + st * 4;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (64 * i < t.n_tok)
#pragma unroll
              for (int v = 0; v < S::kVecs; ++v)
                ptx::st_shared_f32(at + v * (kTokBlock * 4) + i * 256, __fmul_rn(ca[i], cw[v]));
          __syncwarp();
          if (lane < np) ptx::mbar_arrive(bar_tfull(acc_of(kb, lane, np, small)));
        }
      }
    }
  } else {
    // ------------------------------------------------------------ joins and epilogue
    // Two groups of four warps: group h takes columns 64 h .. + 63 of every part
    // (32 h .. + 31 of parts of 64).
    ptx::setmaxnreg_inc<kEpiRegs>();
    const int h = (warp - 4) >> 2;
    const int et = (static_cast<int>(threadIdx.x) - 128) & 127;  // thread of its group
    const int ea = static_cast<int>(threadIdx.x) - 128;          // 0..255 over both
    const int q = warp & 3;                                      // TMEM lane quarter
    const int f = q * 32 + lane;                                 // weight row within the CTA
    const int width = part >> 1;                                 // the group's columns of a part
    const uint32_t tmem_lane = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + h * width;
    const uint32_t ost = sbase + S::EPI + h * 8192;              // [32 rows][128 features] bf16
    // this thread's 16-bit place in staging row j: 16-byte pieces XOR-swizzled by the row
    const uint32_t place = ost + ((f >> 3) << 4) + (f & 7) * 2;
    const uint32_t tempty_leader = ptx::mapa_shared(bar_tempty(0), 0);
    uint32_t full_mask = 0, tphase = 0;   // full_mask: a bit per accumulator, parity of its next sums
    int parity = 0;                       // of the tile: META's half
    auto dst_of = [&](const Tile& nt) {
      const int r = nt.r0 + ea;
      return ea < nt.n_tok ? (p.row_to_pair ? __ldg(p.row_to_pair + r) : r) : -1;
    };
    int nd = -1;
    if (!kGU && unit < total) nd = dst_of(tile_of(unit));
    for (int tile = unit; tile < total; tile += n_units, parity ^= 1) {
      const Tile t = tile_of(tile);
      const int first = t.n0 + static_cast<int>(rank) * (kFbCols / 2);   // the CTA's first column
      int* dst_t = reinterpret_cast<int*>(smem + S::META) + parity * kTokBlock;            // plain
      float* w_t = reinterpret_cast<float*>(smem + S::META + 2048) + parity * kTokBlock;
      if (!kGU) {
        // destination rows and weights of this tile, the next tile's rows a tile ahead; the last
        // readers of this half (two tiles ago) passed the previous tile's vote
        const int d = nd >= 0 && nd < p.P ? nd : -1;
        dst_t[ea] = d;
        w_t[ea] = p.pair_weight && d >= 0 ? __ldg(p.pair_weight + d) : 1.0f;
        if (tile + n_units < total) nd = dst_of(tile_of(tile + n_units));
      }
      // the factor vector of this thread's weight row
      int vec = 0;
      if (kGU && f < 64) vec = (p.N + first + f) / kBlk == (p.N + first) / kBlk ? 1 : 2;
      const uint32_t fac0 = sbase + S::FAC + vec * (kTokBlock * 4) + h * width * 4;
      // sum[r][i]: row 128 r + 64 h + i of the tile (32 h + i in small launches)
      float sum[2][64];
#pragma unroll
      for (int i = 0; i < 64; ++i) sum[0][i] = sum[1][i] = 0.0f;

      // one part of one block: its sums times their factors
      auto join = [&](float (&to)[64], int acc, uint32_t fac, uint32_t parity_bit) {
        wait_lean(bar_tfull(acc), parity_bit, abort_flag, kp.status, kp.wait_ns);
        ptx::tc_fence_after();
        const uint32_t taddr = tmem_lane + acc * part;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c == 0 || !small) {
            uint32_t v[32];
            ptx::tmem_ld_32x32b_x32(taddr + 32 * c, v);
            ptx::tmem_ld_wait();
            if (c == 1 || small) {     // the last of the accumulator: free it
              ptx::tc_fence_before();
              if (lane == 0) ptx::mbar_arrive_remote_relaxed(tempty_leader + 8u * acc);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 s4 = ptx::ld_shared_v4(fac + c * 128 + i * 16);
              float* s = to + 32 * c + 4 * i;
              s[0] = fmaf(__uint_as_float(v[4 * i]), __uint_as_float(s4.x), s[0]);
              s[1] = fmaf(__uint_as_float(v[4 * i + 1]), __uint_as_float(s4.y), s[1]);
              s[2] = fmaf(__uint_as_float(v[4 * i + 2]), __uint_as_float(s4.z), s[2]);
              s[3] = fmaf(__uint_as_float(v[4 * i + 3]), __uint_as_float(s4.w), s[3]);
            }
          }
        }
      };
      auto pass_slot = [&](int slot) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_sempty(slot));
      };
      if (t.n_tok > kPart) {
        for (int kb = 0; kb < nk; kb += 2) {
          join(sum[0], 0, fac0, full_mask & 1u);
          join(sum[1], 1, fac0 + 512, (full_mask >> 1) & 1u);
          pass_slot(0);
          full_mask ^= 3u;
          if (kb + 1 < nk) {
            join(sum[0], 2, fac0 + S::kSlotBytes, (full_mask >> 2) & 1u);
            join(sum[1], 3, fac0 + S::kSlotBytes + 512, (full_mask >> 3) & 1u);
            pass_slot(1);
            full_mask ^= 12u;
          }
        }
      } else {
        for (int kb = 0; kb < nk; ++kb) {
          const int acc = acc_of(kb, 0, 1, small);
          join(sum[0], acc, fac0 + (kb & 1) * S::kSlotBytes, (full_mask >> acc) & 1u);
          full_mask ^= 1u << acc;
          pass_slot(kb & 1);
        }
      }
      // one decision for the eight warps; the barrier also publishes dst_t / w_t
      if (!ptx::bar_and(3, 256, *abort_flag == 0)) break;
      // 32 rows of the group at a time through its staging buffer
      const int tok = et >> 2, quad = et & 3;    // gate/up: row of the 32, 16 features of it
      const int col = first + 16 * quad;
      const bool in = col < p.N;                 // N % 16 == 0
      const uint32_t s_max = sbase + S::META + (parity * 2 + h) * 1024 + tok * 4;   // [2][2 groups][2 CTAs][128]
      float act[4][16];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int j0 = (c >> 1) * kPart + h * width + (c & 1) * 32;
        if (j0 >= t.n_tok || (small && c > 0)) continue;   // the same for the whole group
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = sum[c >> 1][32 * (c & 1) + 4 * i + k];
          if (!kGU && p.pair_weight) {           // one f32 multiply, then the one bf16 rounding
            const uint4 w4 = ptx::ld_shared_v4(ptx::smem_u32(w_t) + 4 * j0 + 16 * i);
            x[0] = __fmul_rn(x[0], __uint_as_float(w4.x));
            x[1] = __fmul_rn(x[1], __uint_as_float(w4.y));
            x[2] = __fmul_rn(x[2], __uint_as_float(w4.z));
            x[3] = __fmul_rn(x[3], __uint_as_float(w4.w));
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {          // gate/up: narrowed before the activation
            const uint32_t pk = gemm::pack_bf16x2(x[2 * k], x[2 * k + 1]);
            const int j = 4 * i + 2 * k;
            ptx::st_shared_u16((place ^ ((j & 15) << 4)) + j * 256, static_cast<uint16_t>(pk));
            ptx::st_shared_u16((place ^ (((j + 1) & 15) << 4)) + (j + 1) * 256,
                               static_cast<uint16_t>(pk >> 16));
          }
        }
        ptx::bar_sync(1 + h, 128);
        if (!kGU) {
          // sixteen threads store one row's 256 bytes
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int idx = et + 128 * i;
            const int j = idx >> 4, k = idx & 15;
            const int cc = first + 8 * k;
            if (j0 + j < t.n_tok && cc < p.N) {
              const int d = dst_t[j0 + j];
              const uint4 val = ptx::ld_shared_v4(ost + j * 256 + ((k ^ (j & 15)) << 4));
              if (d >= 0) *reinterpret_cast<uint4*>(p.out + static_cast<size_t>(d) * p.N + cc) = val;
            }
          }
        } else {
          const uint32_t row = ost + tok * 256;
          const uint4 u0 = ptx::ld_shared_v4(row + (((2 * quad) ^ (tok & 15)) << 4));
          const uint4 u1 = ptx::ld_shared_v4(row + (((2 * quad + 1) ^ (tok & 15)) << 4));
          const uint4 g0 = ptx::ld_shared_v4(row + (((2 * quad + 8) ^ (tok & 15)) << 4));
          const uint4 g1 = ptx::ld_shared_v4(row + (((2 * quad + 9) ^ (tok & 15)) << 4));
          if (p.out && in && j0 + tok < t.n_tok) {
            uint16_t* o = p.out + static_cast<size_t>(t.r0 + j0 + tok) * 2 * p.N + col;
            reinterpret_cast<uint4*>(o)[0] = g0;
            reinterpret_cast<uint4*>(o)[1] = g1;
            reinterpret_cast<uint4*>(o + p.N)[0] = u0;
            reinterpret_cast<uint4*>(o + p.N)[1] = u1;
          }
          float g[16], u[16], m = 0.0f;
          widen16(g0, g1, g);
          widen16(u0, u1, u);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            // SiLU is tolerance-checked: the fast exponential and division serve
            act[c][i] = __fdividef(g[i], 1.0f + __expf(-g[i])) * u[i];
            m = fmaxf(m, fabsf(act[c][i]));
          }
          if (!in) m = 0.0f;
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          if (quad == 0) {
            const uint32_t at = s_max + rank * 512 + c * 128;
            ptx::st_shared_f32(at, m);
            ptx::st_cluster_f32(ptx::mapa_shared(at, rank ^ 1u), m);
          }
        }
        ptx::bar_sync(1 + h, 128);
      }
      if (kGU) {
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive_remote(ptx::mapa_shared(bar_max(h), rank));
          ptx::mbar_arrive_remote(ptx::mapa_shared(bar_max(h), rank ^ 1u));
        }
        // a warp that gives up here stops at the next tile's vote: the named barriers stay matched
        const bool ok = wait_bar<true>(bar_max(h), tphase, abort_flag, kp.status, kp.wait_ns);
        tphase ^= 1u;
        if (ok) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int j = (c >> 1) * kPart + h * width + (c & 1) * 32 + tok;
            if (j >= t.n_tok || (small && c > 0)) continue;
            const float m = fmaxf(ptx::ld_shared_f32(s_max + c * 128), ptx::ld_shared_f32(s_max + 512 + c * 128));
            float d, id;
            block_scale(m, d, id);
            const size_t r = static_cast<size_t>(t.r0 + j);
            if (in) *reinterpret_cast<uint4*>(p.act + r * p.N + col) = codes16(act[c], id);
            if (quad == 0 && leader) p.act_scale[r * blocks_of(p.N) + t.n0 / kBlk] = d;
          }
        }
      }
    }
  }

  // ---- exit: if either CTA of the pair gave up, drain before freeing memory
  __syncthreads();
  ptx::cluster_sync();
  const bool gave_up =
      *abort_flag != 0 ||
      ld_cluster_u32(ptx::mapa_shared(sbase + S::MISC + 4, rank ^ 1u)) != 0;
  if (gave_up) {
    if (warp == 1 && lane == 0 && leader && mma_any) {
      ptx::mma_commit_pair(bar_drain, 1);
      gemm::spin_bounded(bar_drain, 0);
    }
    if (warp == 0 && lane == 0) {
      const uint64_t t0 = ptx::globaltimer_ns();
      while (ptx::globaltimer_ns() - t0 < kCopyGraceNs) {
      }
    }
  }
  __syncthreads();
  ptx::cluster_sync();  // the peer may still use this CTA's shared memory or TMEM until here
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc2(tmem_base, 512);
  }
}

template <bool kGU>
int launch_range(const char* op, const CUtensorMap (&tt)[3], const CUtensorMap& tw, KernelParams kp,
                 cudaStream_t stream) {
  auto kern = fp8_pair_kernel<kGU>;
  const int smem = Smem<kGU>::ALLOC;
  static std::atomic<int> pairs_dev[64] = {};   // resident clusters, once the kernel is configured
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    dev = -1;
  }
  const bool cache = dev >= 0 && dev < 64;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  int max_pairs = cache ? pairs_dev[dev].load(std::memory_order_acquire) : 0;
  if (max_pairs <= 0) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return set_error(MOE_ERR_CUDA, "%s: cannot reserve %d bytes of shared memory: %s", op, smem,
                       cudaGetErrorString(cudaGetLastError()));
    // a pair must sit in one GPC, so fewer than SMs / 2 pairs may fit at once
    max_pairs = sm_count() / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * max_pairs), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) == cudaSuccess && clusters > 0)
      max_pairs = clusters < max_pairs ? clusters : max_pairs;
    else
      cudaGetLastError();
    if (cache) pairs_dev[dev].store(max_pairs, std::memory_order_release);
  }
  const GemmParams& p = kp.g;
  const int fb_cols = kGU ? 128 : 256;
  long long pairs = (p.P + kTokBlock - 1) / kTokBlock + (p.G < p.P ? p.G : p.P);
  pairs *= (p.N + fb_cols - 1) / fb_cols;       // an upper bound on the tiles
  if (pairs > max_pairs) pairs = max_pairs;
  return launch_status(launch_kernel(kern, dim3(static_cast<unsigned>(2 * pairs), 1, 1),
                                     dim3(kThreads, 1, 1), smem, stream, attr, 1, tt[0], tt[1],
                                     tt[2], tw, kp),
                       op);
}

}  // namespace

int launch_product(const char* op, const GemmParams& p0, bool gateup, cudaStream_t stream) {
  GemmParams p = p0;
  const int rows = gateup ? 2 * p.N : p.N;
  CUtensorMap tt[3], tw;
  int rc;
  // pairs of codes as 2-byte elements (K is a multiple of 16): the same bytes and the same
  // 128-byte swizzle as a bf16 operand's box
  for (int i = 0; i < 3; ++i)
    if ((rc = gemm::make_tmap(&tt[i], p.a, p.P, p.K / 2, 16 << i, op, "a_codes")) != MOE_OK) return rc;
  if ((rc = gemm::make_tmap(&tw, p.w, static_cast<long long>(p.G) * rows, p.K / 2, gateup ? 64 : 128,
                            op, "weights")) != MOE_OK)
    return rc;
  DeviceDiag diag = device_diag();
  KernelParams kp{p, rows, gemm::pipeline_wait_ns(), diag.status, diag.launches};
  if (p.G <= kMaxGroupsLaunch)
    return gateup ? launch_range<true>(op, tt, tw, kp, stream) : launch_range<false>(op, tt, tw, kp, stream);
  // more groups than a launch's schedule holds: one launch per range of groups
  for (int g0 = 0; g0 < p0.G; g0 += kMaxGroupsLaunch) {
    GemmParams& q = kp.g;
    q = p0;
    q.G = p0.G - g0 < kMaxGroupsLaunch ? p0.G - g0 : kMaxGroupsLaunch;
    q.group_offsets = p0.group_offsets + g0;
    q.w = p0.w + static_cast<size_t>(g0) * rows * p0.K;
    q.sw = p0.sw + static_cast<size_t>(g0) * blocks_of(rows) * blocks_of(p0.K);
    if ((rc = gemm::make_tmap(&tw, q.w, static_cast<long long>(q.G) * rows, q.K / 2, gateup ? 64 : 128,
                              op, "weights")) != MOE_OK)
      return rc;
    rc = gateup ? launch_range<true>(op, tt, tw, kp, stream) : launch_range<false>(op, tt, tw, kp, stream);
    if (rc != MOE_OK) return rc;
  }
  return MOE_OK;
}

}  // namespace fp8
}  // namespace moe
