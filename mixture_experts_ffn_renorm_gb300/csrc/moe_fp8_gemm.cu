// moe_fp8_gemm.cu -- the grouped products of E4M3 activations and E4M3 weights
// (moe_grouped_gemm_fp8, moe_grouped_gemm_gateup_silu_fp8).
//
// y[r,n] = sum_b (sa[r,b] sw[n,b]) p_b[r,n], p_b the product over the 128
// columns of scale block b.  The scales change with every block of the
// contraction, so the tensor core sums one block at a time: each block's MMAs
// start a fresh accumulator in tensor memory, and sixteen epilogue warps join the
// blocks in registers, acc += p_b * s_b, while the tensor core fills the next
// accumulators.
//
// A tile has 256 weight rows (256 output columns, or 128 features' up and gate
// rows) in two parts of 128, each with its MMAs, its issuing thread and its half of
// the epilogue warps.  Two kinds of tile:
//   rows tiles     (blocks of more than 64 rows of a group): 128 token rows on the
//                  MMA's M side, a part's 128 weight rows on N.  A thread owns one
//                  token row and 64 of the columns, so the factor s_b is one
//                  register: one fused multiply-add per product and block.
//   weights tiles  (blocks of up to 64 rows): a part's 128 weight rows on M, the
//                  token rows on N, padded to 16.  A thread owns one weight row and
//                  32 of the token rows, whose scales its warp keeps in shared memory.
// Rows tiles need no transpose and no scale loads per product, and pad to 128 rows;
// weights tiles pad to 16 rows, which is what ragged and decode-sized groups need.
//
// What bounds it: a block's joins.  A part's eight warps each wait for its accumulator, read
// 64 columns in four steps and add them up, about 740 cycles a block against 512 of MMA work
// (with the multiply-adds left out a block takes 530; with the accumulators released before
// they are read, as long as before).  The joins use paired multiply-adds, whose issue slots
// were the bound before (845 cycles), and the scales come through shared memory: a warp
// that reads its 32 rows' scales itself touches 32 cache lines a block, and from 32 blocks a
// row on took 1600.  A tile costs about 4600 cycles besides (launch and fill of an eight-tile
// call spread over its tiles included 5700): the vote, the packing, the stores, and the first
// block's scales and accumulator, while the MMAs run two blocks ahead and then wait.
// Times of 9728 x 4096 x 2048, 74.2 us as built; tried and not kept, each against the step it
// was tried on: CTA pairs (256 x 256 tiles; the trip to the peer costs what the shared weight
// rows save: 78.5 against 78.7), one MMA of N = 256 for both parts (83.0 against 78.7: its one
// issuer waits for both parts' joins), tiles left in staging and stored during the next one
// (81.4 against 78.7), three operand stages and 64 KB of staging (80.8 against 74.2).
//
//   warp 0      TMA producer: 256 weight rows and up to 128 token rows of one scale
//               block (128 bytes a row) per stage
//   warps 1-2   tensor memory (1); the two threads that issue MMAs, one per part
//   warp 3      the tiles' descriptions and the scales, ahead of the epilogue
//   warps 4-19  block joins and the epilogue; part 0 the first eight, part 1 the others
//
// gate/up: a part holds the up rows and then the gate rows of 64 features.  Gate and up are
// narrowed to bf16, silu(gate) * up is formed in f32 and a row's 128 features are quantised
// with one scale.
//   rows tiles: a thread's 64 columns are up and gate of 32 features; the row's largest
//     magnitude is that of four threads.
//   weights tiles: the bf16 results are transposed through shared memory, and sixteen
//     threads form a row's 128 activations.
//
// The tile schedule and the bounded waits are those of moe_gemm.cu; a CTA that gives
// up drains its MMAs and copies before it frees tensor memory.
#include <atomic>

#include "fp8_common.cuh"

namespace moe {
namespace fp8 {
namespace {

using gemm::wait_bar_spin;

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t ld_shared_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t pack_bf16(uint64_t v) {
  const float2 f = ptx::unpair(v);
  return gemm::pack_bf16x2(f.x, f.y);
}

constexpr int kEpiWarps = 16;
constexpr int kThreads = 128 + 32 * kEpiWarps;   // a warpgroup of the other roles
constexpr int kAuxRegs = 64, kEpiRegs = 104;
// the split draws on the registers the block was launched with (96 a thread)
static_assert(128 * kAuxRegs + 32 * kEpiWarps * kEpiRegs <= kThreads * 96, "register split");
constexpr int kTokBlock = 128;              // rows per rows tile
// Rows of a weights tile at most, the size of the epilogue's halves.  64 groups of 2048 x 1536
// as weights tiles against rows tiles: 24 rows each 38.3 us against 40.1, 40 rows 40.2 against
// 40.9, 56 and 64 rows the same (42.0, 42.2).
constexpr int kTail = 64;
constexpr int kStages = 4;
constexpr int kWBytes = 256 * 128;          // a stage's weight rows
constexpr int kTBytes = 128 * 128;          // a stage's token rows, at most
constexpr int kMaxAcc = 8;
constexpr int kMmaK = 32;                   // K per tcgen05.mma of 8-bit types

// Scales of 8 blocks: the rows' as [block][128 rows], 16 bytes of padding per block (so that
// the four rows x 8 blocks of one copy instruction meet 32 banks); then up to three weight
// scale blocks' as [which][8].  which, plain: the two 128-row parts; gate/up: the gate rows,
// and the up rows, which of I not a multiple of 128 lie in two scale blocks.
constexpr int kChunk = 8, kRowStride = 128 * 4 + 16;
constexpr int kChunkW = kChunk * kRowStride, kChunkBytes = kChunkW + 3 * kChunk * 4;

struct Smem {
  static constexpr int W = 0;
  static constexpr int T = W + kStages * kWBytes;
  static constexpr int EPI = T + kStages * kTBytes;             // 16 KB of staging
  static constexpr int SCALE = EPI + 16384;                     // two chunks of scales
  static constexpr int META = SCALE + 2 * kChunkBytes;          // two tiles' destinations and weights, or row maxima
  static constexpr int INFO = META + 2048;                      // two tiles
  static constexpr int BARS = INFO + 32;
  // full, empty [kStages], tfull, tempty [kMaxAcc], drain [2], ifull, iempty [2],
  // sfull, sempty [2]
  static constexpr int NBARS = 2 * kStages + 2 * kMaxAcc + 10;
  static constexpr int MISC = (BARS + NBARS * 8 + 15) & ~15;                 // tmem slot, then:
  static constexpr int kAbort = 4, kSmall = 8, kStatus = 16, kLimit = 24, kScan = 32;
  static constexpr int ROWS_START = (MISC + kScan + 8 * (kThreads / 32) + 15) & ~15;
  static constexpr int TAIL_START = ROWS_START + (kMaxGroupsLaunch + 1) * 4;
  static constexpr int GOFF = TAIL_START + (kMaxGroupsLaunch + 1) * 4;
  static constexpr int ALLOC = GOFF + (kMaxGroupsLaunch + 1) * 4 + 1024;
};
static_assert(Smem::ALLOC <= 227 * 1024, "shared memory");

// Bounded wait (see gemm::wait_bar) for the loops that run once per scale block, where
// every instruction and register counts: the probe without a time hint (the one with a
// hint is a software loop around it), and the limit and the status word's address from
// shared memory (`misc`).  A wait that gives up raises the status and the CTA's abort flag.
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, uint32_t misc) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (ld_shared_u32(misc + Smem::kAbort) != 0) return false;
    if (ptx::globaltimer_ns() - t0 > ld_shared_u64(misc + Smem::kLimit)) {
      unsigned int* status = reinterpret_cast<unsigned int*>(ld_shared_u64(misc + Smem::kStatus));
      if (status) atomicOr(status, static_cast<unsigned int>(MOE_STATUS_TIMEOUT));
      asm volatile("st.shared.u32 [%0], 1;" ::"r"(misc + Smem::kAbort) : "memory");
    }
  }
  return true;
}
// the same for a whole warp, which after a wait that gives up goes on with what is there:
// its later waits end at once, and it stops at the tile's vote
__device__ __forceinline__ void wait_lean(uint32_t bar, uint32_t parity, uint32_t misc) {
  wait_one(bar, parity, misc);
  __syncwarp();
}

struct KernelParams {
  GemmParams g;
  int rows_per_group;            // weight rows of a group
  unsigned long long wait_ns;
  unsigned int* status;
  unsigned long long* launches;
};

// What an epilogue thread is, worked out anew where it is needed: the loops over the
// scale blocks have no registers left to carry it through.
struct Ids {
  int e, h, set, f, et, ht;
  __device__ __forceinline__ Ids() {
    int tid;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
    const int warp = tid >> 5, lane = tid & 31;
    e = warp - 4;                      // 0..15
    h = (e >> 2) & 1;                  // half of the columns of a part
    set = e >> 3;                      // the part
    f = (warp & 3) * 32 + lane;        // TMEM lane
    et = e * 32 + lane;                // 0..511
    ht = (set << 7) | f;               // thread among those of its half of the columns
  }
  // the thread's column of accumulator 0: tensor memory's lane quarter is the warp's
  __device__ __forceinline__ uint32_t tmem(uint32_t base) const {
    return base + (static_cast<uint32_t>(f & ~31) << 16);
  }
};

struct Tile {
  int g, r0, n_tok, n0;          // n_tok > kTail: a rows tile
};

// rows tiles first, then weights tiles; each kind by group, block of rows, columns
struct Schedule {
  // [G + 1] words each in shared memory: first rows tile of a group; first weights tile,
  // counted from the number of rows tiles; group offsets.  32-bit addresses: the epilogue
  // warps have no registers to spare.
  uint32_t base;
  int G, N, fb_cols;
  __device__ __forceinline__ int word(uint32_t at, int i) const { return ld_shared_u32(base + at + 4 * i); }
  __device__ __forceinline__ int total() const { return word(Smem::ROWS_START, G) + word(Smem::TAIL_START, G); }
  __device__ __forceinline__ Tile at(int tile) const {
    // opaque: what it works out for a tile is not kept in registers across the tile's loop
    asm volatile("" : "+r"(tile));
    const int n_fb = (N + fb_cols - 1) / fb_cols;
    const int n_rows = word(Smem::ROWS_START, G);
    const bool tail = tile >= n_rows;
    const uint32_t start = tail ? Smem::TAIL_START : Smem::ROWS_START;
    if (tail) tile -= n_rows;
    int lo = 0, hi = G;  // start[lo] <= tile < start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (word(start, mid) <= tile) lo = mid; else hi = mid;
    }
    const int local = tile - word(start, lo);
    const int r0 = word(Smem::GOFF, lo), r1 = word(Smem::GOFF, lo + 1);
    const int m = tail ? (r1 - r0 - 1) / kTokBlock : local / n_fb;
    Tile t;
    t.g = lo;
    t.r0 = r0 + m * kTokBlock;
    t.n_tok = min(r1, t.r0 + kTokBlock) - t.r0;
    t.n0 = (tail ? local : local - m * n_fb) * fb_cols;
    return t;
  }
};

// blocks of a group that take rows tiles, and whether its last one takes weights tiles
__device__ __forceinline__ int rows_blocks(int rows) {
  return rows > 0 ? rows / kTokBlock + (rows % kTokBlock > kTail ? 1 : 0) : 0;
}
__device__ __forceinline__ int tail_blocks(int rows) {
  return rows > 0 && rows % kTokBlock != 0 && rows % kTokBlock <= kTail ? 1 : 0;
}

template <bool kGU>
__global__ void __launch_bounds__(kThreads, 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmT16, const __grid_constant__ CUtensorMap tmT32,
                const __grid_constant__ CUtensorMap tmT64, const __grid_constant__ CUtensorMap tmT128,
                const __grid_constant__ CUtensorMap tmW, const KernelParams kp) {
  using S = Smem;
  const GemmParams& p = kp.g;
  constexpr int kFbCols = kGU ? 128 : 256;   // output features per tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::MISC + S::kAbort);
  int2* scan_tmp = reinterpret_cast<int2*>(smem + S::MISC + S::kScan);   // one pair per warp
  int* rows_start = reinterpret_cast<int*>(smem + S::ROWS_START);
  int* tail_start = reinterpret_cast<int*>(smem + S::TAIL_START);
  int* goff = reinterpret_cast<int*>(smem + S::GOFF);

  // opaque, so that the inner loops hold them in registers instead of reading them anew
  int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("" : "+r"(warp), "+r"(lane));
  const int unit = static_cast<int>(blockIdx.x);
  const int n_units = static_cast<int>(gridDim.x);
  const uint32_t bars = sbase + S::BARS;
  auto bar_full = [&](int s) { return bars + 8u * s; };
  auto bar_empty = [&](int s) { return bars + 8u * (kStages + s); };
  auto bar_tfull = [&](int a) { return bars + 8u * (2 * kStages + a); };
  auto bar_tempty = [&](int a) { return bars + 8u * (2 * kStages + kMaxAcc + a); };
  auto bar_drain = [&](int i) { return bars + 8u * (2 * kStages + 2 * kMaxAcc + i); };
  auto bar_ifull = [&](int i) { return bars + 8u * (2 * kStages + 2 * kMaxAcc + 2 + i); };
  auto bar_iempty = [&](int i) { return bars + 8u * (2 * kStages + 2 * kMaxAcc + 4 + i); };
  auto bar_sfull = [&](int i) { return bars + 8u * (2 * kStages + 2 * kMaxAcc + 6 + i); };
  auto bar_sempty = [&](int i) { return bars + 8u * (2 * kStages + 2 * kMaxAcc + 8 + i); };

  count_launch(kp.launches, p.kid);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(bar_full(s), 1);    // the producer's expect-tx arrive
      ptx::mbar_init(bar_empty(s), 2);   // the two issuers' MMA commits
    }
    for (int a = 0; a < kMaxAcc; ++a) {
      ptx::mbar_init(bar_tfull(a), 1);    // the issuer's MMA commit
      ptx::mbar_init(bar_tempty(a), 8);   // the epilogue warps of its part
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar_drain(i), 1);
      ptx::mbar_init(bar_ifull(i), 32);          // warp 3
      ptx::mbar_init(bar_iempty(i), kEpiWarps);
      ptx::mbar_init(bar_sfull(i), 32);          // warp 3's copies
      ptx::mbar_init(bar_sempty(i), kEpiWarps);
    }
    *abort_flag = 0;
    *reinterpret_cast<unsigned int**>(smem + S::MISC + S::kStatus) = kp.status;
    *reinterpret_cast<unsigned long long*>(smem + S::MISC + S::kLimit) = kp.wait_ns;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::tma_prefetch_desc(&tmT16);
    ptx::tma_prefetch_desc(&tmT32);
    ptx::tma_prefetch_desc(&tmT64);
    ptx::tma_prefetch_desc(&tmT128);
    ptx::tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
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
  int n_big = 0, n_tail = 0, rows_max = 0;
  for (int g = g_lo; g < g_hi; ++g) {
    const int rows = goff[g + 1] - goff[g];
    n_big += rows_blocks(rows) * n_fb;
    n_tail += tail_blocks(rows) * n_fb;
    rows_max = max(rows_max, rows);
  }
  int incl_b = n_big, incl_t = n_tail;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int b = __shfl_up_sync(0xffffffffu, incl_b, o), t = __shfl_up_sync(0xffffffffu, incl_t, o);
    if (lane >= o) {
      incl_b += b;
      incl_t += t;
    }
  }
  if (lane == 31) scan_tmp[warp] = make_int2(incl_b, incl_t);
  const bool small = __syncthreads_or(rows_max > kTail) == 0;   // eight accumulators of kTail columns
  int run_b = incl_b - n_big, run_t = incl_t - n_tail;
  int all_b = 0, all_t = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    const int2 v = scan_tmp[w];
    if (w < warp) {
      run_b += v.x;
      run_t += v.y;
    }
    all_b += v.x;
    all_t += v.y;
  }
  for (int g = g_lo; g < g_hi; ++g) {
    const int rows = goff[g + 1] - goff[g];
    rows_start[g] = run_b;
    tail_start[g] = run_t;
    run_b += rows_blocks(rows) * n_fb;
    run_t += tail_blocks(rows) * n_fb;
  }
  if (threadIdx.x == 0) {
    *reinterpret_cast<int*>(smem + S::MISC + S::kSmall) = small;
    rows_start[G] = all_b;
    tail_start[G] = all_t;
  }
  const Schedule sch{sbase, G, p.N, kFbCols};
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int nk = blocks_of(p.K);
  const int total = sch.total();

  bool mma_any = false;
  uint32_t loads = 0;   // stages the producer has filled

  if (warp < 4) {
    ptx::setmaxnreg_dec<kAuxRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer
      // one lane per box: the two parts' 128 weight rows each (gate/up: 64 up rows, then the 64
      // gate rows of the same features), the token rows
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = unit; ok && tile < total; tile += n_units) {
        const Tile t = sch.at(tile);
        const int tbox = t.n_tok > 64 ? 128 : (t.n_tok > 32 ? 64 : (t.n_tok > 16 ? 32 : 16));
        const uint32_t bytes = kWBytes + tbox * 128;
        const int wrow = t.g * kp.rows_per_group + t.n0;
        constexpr int kTokLane = kGU ? 4 : 2;
        const CUtensorMap* mbox = lane < kTokLane ? &tmW
                                  : (tbox == 16 ? &tmT16 : (tbox == 32 ? &tmT32 : (tbox == 64 ? &tmT64 : &tmT128)));
        const int ybox = lane == kTokLane ? t.r0
                         : (kGU ? wrow + 64 * (lane >> 1) + (lane & 1 ? 0 : p.N) : wrow + 128 * lane);
        const uint32_t dbox = lane == kTokLane ? S::T : S::W + lane * (kWBytes / kTokLane);
        const uint32_t dstep = lane == kTokLane ? kTBytes : kWBytes;
        for (int kb = 0; kb < nk; ++kb) {
          bool got = true;
          if (lane == 0) {
            // spinning: the producer's reaction time is part of the ring's round trip
            got = wait_bar_spin(bar_empty(stage), phase ^ 1u, abort_flag, kp.status, kp.wait_ns);
            if (got) ptx::mbar_arrive_expect_tx(bar_full(stage), bytes);
          }
          if (!__shfl_sync(0xffffffffu, got ? 1 : 0, 0)) {
            ok = false;
            break;
          }
          ++loads;
          // the maps see pairs of codes as 2-byte elements: 64 of them per scale block
          if (lane <= kTokLane) ptx::tma_load_2d(sbase + dbox + stage * dstep, mbox, kb * 64, ybox, bar_full(stage));
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
    } else if (warp < 3) {
      // ---------------------------------------------------------- MMA issuers
      // One thread takes about 400 cycles a part for its waits, MMAs and commits, more than
      // the MMAs run, so there is one for each part.
      if (ptx::elect_one()) {
        const uint32_t me = warp - 1;
        const int acc_shift = small ? 3 : 2;   // log2 of the accumulators in the ring
        const uint32_t acc_mask = (1u << acc_shift) - 1u, acc_cols = 512u >> acc_shift;
        int stage = 0;
        uint32_t phase = 0, parts = me;    // the part's place among the accumulators taken so far
        bool ok = true;
        for (int tile = unit; ok && tile < total; tile += n_units) {
          const Tile t = sch.at(tile);
          const bool big = t.n_tok > kTail;
          const uint32_t idesc = ptx::idesc_e4m3_f32(128, big ? 128 : (t.n_tok + 15) & ~15);
          for (int kb = 0; kb < nk; ++kb, parts += 2) {
            const uint32_t acc = parts & acc_mask;
            const uint64_t dw = ptx::desc_kmajor_sw128(sbase + S::W + stage * kWBytes + me * (kWBytes / 2));
            const uint64_t dt = ptx::desc_kmajor_sw128(sbase + S::T + stage * kTBytes);
            const uint32_t d = tmem_base + acc * acc_cols;
            const uint64_t da = big ? dt : dw, db = big ? dw : dt;   // rows tiles: tokens on M
            // the accumulator last: its release is what the round trip waits for
            if (!wait_one(bar_full(stage), phase, sbase + S::MISC) ||
                !wait_one(bar_tempty(acc), ((parts >> acc_shift) & 1u) ^ 1u, sbase + S::MISC)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
#pragma unroll
            for (int k = 0; k < kBlk / kMmaK; ++k)   // a fresh sum per scale block
              ptx::mma_e4m3(d, da + 2ull * k, db + 2ull * k, idesc, k != 0 ? 1u : 0u);
            mma_any = true;
            ptx::mma_commit(bar_tfull(acc));         // the part's sums are ready
            ptx::mma_commit(bar_empty(stage));       // frees the stage, with the other part's
            if (++stage == kStages) { stage = 0; phase ^= 1u; }
          }
        }
      }
    } else {
      // ---------------------------------------------------------- tiles and scales
      // Warp 3 works ahead of the epilogue: chunks of scales, the tile, and its rows'
      // destinations and weights, which cost a binary search and two dependent loads.
      uint32_t n = 0, q = 0;     // tiles and chunks so far
      bool ok = true;
      for (int tile = unit; ok && tile < total; tile += n_units, ++n) {
        const Tile t = sch.at(tile);
        const int rb = blocks_of(kp.rows_per_group);
        // this lane copies block `blk` of rows sub, sub + 4, ..., and of weight scale block `sub`
        const int blk = lane & 7, sub = lane >> 3;
        const int wb = kGU && sub > 0 ? (p.N + t.n0) / kBlk + sub - 1 : t.n0 / kBlk + sub;
        const float* sa = p.sa + static_cast<size_t>(t.r0 + sub) * nk + blk;
        const float* sw = p.sw + (static_cast<size_t>(t.g) * rb + min(wb, rb - 1)) * nk + blk;
        auto copy = [&](int kb) {
          ok = __all_sync(0xffffffffu, wait_one(bar_sempty(q & 1), ((q >> 1) & 1u) ^ 1u, sbase + S::MISC));
          if (!ok) return;
          const uint32_t at = sbase + S::SCALE + (q & 1) * kChunkBytes;
          if (kb + blk < nk) {
            uint32_t to = at + blk * kRowStride + sub * 4;
            const float* from = sa + kb;
            for (int r = sub; r < t.n_tok; r += 4, to += 16, from += 4 * nk) ptx::cp_async_4(to, from);
            if (sub < (kGU ? 3 : 2)) ptx::cp_async_4(at + kChunkW + (sub * kChunk + blk) * 4, sw + kb);
          }
          ptx::cp_async_arrive_noinc(bar_sfull(q & 1));
          ++q;
        };
        copy(0);
        if (!ok) break;
        int d[4];
        float w[4];
        if (!kGU) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = lane + 32 * i;
            d[i] = j < t.n_tok ? (p.row_to_pair ? __ldg(p.row_to_pair + t.r0 + j) : t.r0 + j) : -1;
            if (d[i] >= p.P) d[i] = -1;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = p.pair_weight && d[i] >= 0 ? __ldg(p.pair_weight + d[i]) : 1.0f;
        }
        if (!__all_sync(0xffffffffu, wait_one(bar_iempty(n & 1), ((n >> 1) & 1u) ^ 1u, sbase + S::MISC))) break;
        if (!kGU) {
          const uint32_t at = sbase + S::META + (n & 1) * 1024 + lane * 4;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ptx::st_shared_f32(at + 128 * i, __int_as_float(d[i]));
            ptx::st_shared_f32(at + 512 + 128 * i, w[i]);
          }
        }
        if (lane == 0) ptx::st_shared_v4(sbase + S::INFO + (n & 1) * 16, t.g, t.r0, t.n_tok, t.n0);
        ptx::mbar_arrive(bar_ifull(n & 1));
        for (int kb = kChunk; ok && kb < nk; kb += kChunk) copy(kb);
      }
      ptx::cp_async_wait_all();
    }
  } else {
    // ------------------------------------------------------------ joins and epilogue
    ptx::setmaxnreg_inc<kEpiRegs>();
    // this role's own copies: what is carried over from before the register split is spilled,
    // and reloaded in the loops
    uint32_t sbase = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    asm volatile("" : "+r"(sbase));
    const uint32_t tmem_base = ld_shared_u32(sbase + S::MISC);
    const int nk = blocks_of(p.K);
    const Schedule sch{sbase, p.G, p.N, kFbCols};
    auto bar_tfull = [&](int a) { return sbase + S::BARS + 8u * (2 * kStages + a); };
    auto bar_tempty = [&](int a) { return sbase + S::BARS + 8u * (2 * kStages + kMaxAcc + a); };
    auto bar_ifull = [&](int i) { return sbase + S::BARS + 8u * (2 * kStages + 2 * kMaxAcc + 2 + i); };
    auto bar_iempty = [&](int i) { return sbase + S::BARS + 8u * (2 * kStages + 2 * kMaxAcc + 4 + i); };
    auto bar_sfull = [&](int i) { return sbase + S::BARS + 8u * (2 * kStages + 2 * kMaxAcc + 6 + i); };
    auto bar_sempty = [&](int i) { return sbase + S::BARS + 8u * (2 * kStages + 2 * kMaxAcc + 8 + i); };
    // the n-th tile of this CTA
    auto wait_info = [&](uint32_t n) {
      return __all_sync(0xffffffffu, wait_one(bar_ifull(n & 1), (n >> 1) & 1u, sbase + S::MISC)) != 0;
    };
    auto info = [&](uint32_t n) {
      const uint4 v = ptx::ld_shared_v4(sbase + S::INFO + (n & 1) * 16);
      Tile t;
      t.g = v.x;
      t.r0 = v.y;
      t.n_tok = v.z;
      t.n0 = v.w;
      return t;
    };
    uint32_t parts = Ids().set;   // the part's place among the accumulators passed so far
    uint32_t n = 0, q = 0;              // tiles and chunks passed
    int tile = blockIdx.x;
    bool on = true;
    // ------------------------------------------------------------ rows tiles
    for (; tile < sch.word(Smem::ROWS_START, G); tile += gridDim.x, ++n) {
      if (!wait_info(n)) {
        ptx::bar_and(5, 32 * kEpiWarps, false);
        on = false;
        break;
      }
      uint64_t sum[32];   // 64 columns; gate/up: 32 features' up, then their gate
#pragma unroll
      for (int i = 0; i < 32; ++i) sum[i] = 0;
      uint32_t taddr0, w_at, to_u0 = 0, to_u1 = 0;   // w_at: within a chunk; the others from there
      {
        const Ids id;
        taddr0 = id.tmem(tmem_base) + (kGU ? 32 : 64) * id.h;
        w_at = kChunkW + (kGU ? 0 : id.set * kChunk * 4);
        if (kGU) {
          const int up = p.N + info(n).n0, ur = up + 64 * id.set + 32 * id.h;
          to_u0 = (1 + ur / kBlk - up / kBlk) * kChunk * 4;
          to_u1 = (1 + (ur + 16) / kBlk - up / kBlk) * kChunk * 4;
        }
      }
#pragma unroll 1
      for (int left = nk; left > 0; left -= kChunk) {
      wait_lean(bar_sfull(q & 1), (q >> 1) & 1u, sbase + S::MISC);
      uint32_t row_at = sbase + S::SCALE + (q & 1) * kChunkBytes;
      uint32_t wt_at = row_at + w_at;
      row_at += Ids().f * 4;
#pragma unroll 1
      for (const uint32_t end = wt_at + 4 * min(left, kChunk); wt_at != end; wt_at += 4, row_at += kRowStride) {
        const float a0 = ptx::ld_shared_f32(row_at);
        const float s0 = __fmul_rn(a0, ptx::ld_shared_f32(wt_at));
        const float s1 = kGU ? __fmul_rn(a0, ptx::ld_shared_f32(wt_at + to_u0)) : 0.0f;
        const float s2 = kGU ? __fmul_rn(a0, ptx::ld_shared_f32(wt_at + to_u1)) : 0.0f;
        const uint32_t acc = parts & 3u;
        wait_lean(bar_tfull(acc), (parts >> 2) & 1u, sbase + S::MISC);
        ptx::tc_fence_after();
        const uint32_t taddr = taddr0 + acc * 128;
        // Gate/up, whose three scales leave fewer registers, reads 8 columns at a time with the
        // next 8 on their way; plain tiles read 16.  (9728 x 4096 x 2048: gate/up 71.1 us
        // instead of 74.1, plain 80.2 instead of 74.2.)
        if constexpr (kGU) {
          uint32_t v[2][8];
          ptx::tmem_ld_32x32b_x8(taddr, v[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            ptx::tmem_ld_wait();
            if (c < 7) {
              ptx::tmem_ld_32x32b_x8(taddr + 64 * ((c + 1) >> 2) + 8 * ((c + 1) & 3), v[(c + 1) & 1]);
            } else {                               // the warp has read all of it
              ptx::tc_fence_before();
              if (ptx::elect_one()) ptx::mbar_arrive(bar_tempty(acc));
            }
            const uint64_t s = ptx::pair(c > 3 ? s0 : (c < 2 ? s1 : s2));
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sum[4 * c + i] = ptx::fma2(ptx::pair(v[c & 1][2 * i], v[c & 1][2 * i + 1]), s, sum[4 * c + i]);
          }
        } else {
          const uint64_t s = ptx::pair(s0);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[16];
            ptx::tmem_ld_32x32b_x16(taddr + 16 * c, v);
            ptx::tmem_ld_wait();
            if (c == 3) {
              ptx::tc_fence_before();
              if (ptx::elect_one()) ptx::mbar_arrive(bar_tempty(acc));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[8 * c + i] = ptx::fma2(ptx::pair(v[2 * i], v[2 * i + 1]), s, sum[8 * c + i]);
          }
        }
        parts += 2;
      }
      __syncwarp();
      if (ptx::elect_one()) ptx::mbar_arrive(bar_sempty(q & 1));
      ++q;
      }
      // one decision for the sixteen warps
      if (!ptx::bar_and(5, 32 * kEpiWarps, ld_shared_u32(sbase + S::MISC + S::kAbort) == 0)) {
        on = false;
        break;
      }
      const Ids id;
      const int h = id.h, set = id.set, f = id.f, lane = f & 31;
      const Tile t = info(n);
      uint32_t pk[32];                             // the 64 results in bf16
      int d = -1;                                  // the destination row
      if (!kGU) {
        const uint32_t at = sbase + S::META + (n & 1) * 1024 + f * 4;
        d = static_cast<int>(ld_shared_u32(at));
        const float w = ptx::ld_shared_f32(at + 512);
#pragma unroll
        for (int i = 0; i < 32; ++i)               // one f32 multiply, then the one bf16 rounding
          pk[i] = pack_bf16(ptx::mul2(sum[i], ptx::pair(w)));
      } else {
        if (f < t.n_tok) d = t.r0 + f;
#pragma unroll
        for (int i = 0; i < 32; ++i) pk[i] = pack_bf16(sum[i]);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar_iempty(n & 1));
      // Sixteen rows and 32 columns at a time through the warp's 1 KB, so that four lanes store
      // 64 bytes of a row.  (A 16-byte shared store takes its passes whether 8 or 16 lanes are
      // active: eight rows of 128 bytes at a time took 78.7 us where this takes 74.2, all 32 rows
      // of 32 bytes 79.6, 32-byte stores straight from registers 79.6.)
      const int col = kGU ? t.n0 + 64 * set + 32 * h : t.n0 + 128 * set + 64 * h;
      const uint32_t st = sbase + S::EPI + ((id.e & 3) * 4 + 2 * set + h) * 1024;
      if (!kGU || p.out) {
        const int row_stride = kGU ? 2 * p.N : p.N;
        // this lane's pieces: of row `lane`, and to be stored, of row 8 i + lane / 4
        const uint32_t mine = st + (lane & 15) * 64, swz = (lane >> 1) & 3;
        const uint32_t from = st + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {              // q & 1: half of the columns (gate/up: up, gate)
          const int cc = col + 8 * (lane & 3) + (kGU ? 0 : 32 * (q & 1));
          if ((lane >> 4) == (q >> 1)) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int k = 16 * (q & 1) + 4 * c;
              ptx::st_shared_v4(mine + ((c ^ swz) << 4), pk[k], pk[k + 1], pk[k + 2], pk[k + 3]);
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 val = ptx::ld_shared_v4(from + i * 512);
            const int dr = __shfl_sync(0xffffffffu, d, 16 * (q >> 1) + 8 * i + (lane >> 2));
            if (dr >= 0 && cc < p.N)
              *reinterpret_cast<uint4*>(p.out + static_cast<size_t>(dr) * row_stride + cc + (kGU && q % 2 == 0 ? p.N : 0)) = val;
          }
          __syncwarp();
        }
      }
      if (kGU) {
        float act[32], m = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          act[2 * i] = silu_mul(__uint_as_float(pk[16 + i] << 16), __uint_as_float(pk[i] << 16));
          act[2 * i + 1] = silu_mul(__uint_as_float(pk[16 + i] & 0xFFFF0000u), __uint_as_float(pk[i] & 0xFFFF0000u));
        }
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (col + (i & 16) < p.N) m = fmaxf(m, fabsf(act[i]));        // N % 16 == 0
        // the four threads of a row, in four warps of the same rows
        const uint32_t s_max = sbase + S::META + f * 4;                 // [4][128 rows]
        ptx::st_shared_f32(s_max + (2 * set + h) * 512, m);
        ptx::bar_sync(6 + (f >> 5), 128);
#pragma unroll
        for (int i = 0; i < 4; ++i) m = fmaxf(m, ptx::ld_shared_f32(s_max + i * 512));
        float dd, inv;
        block_scale(m, dd, inv);
        if (h + set == 0 && d >= 0) p.act_scale[static_cast<size_t>(d) * blocks_of(p.N) + t.n0 / kBlk] = dd;
        // the four warps' 4 KB hold their rows' codes; eight lanes store a row's 128 bytes
        const uint32_t rows = sbase + S::EPI + (f >> 5) * 4096;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) x[k] = act[16 * i + k];
          const uint4 c = codes16(x, inv);
          ptx::st_shared_v4(rows + lane * 128 + (((4 * set + 2 * h + i) ^ (lane & 7)) << 4), c.x, c.y, c.z, c.w);
        }
        ptx::bar_sync(6 + (f >> 5), 128);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = (2 * set + h) * 8 + 4 * i + (lane >> 3), piece = lane & 7;
          const uint4 val = ptx::ld_shared_v4(rows + row * 128 + ((piece ^ (row & 7)) << 4));
          const int dr = __shfl_sync(0xffffffffu, d, row), cc = t.n0 + 16 * piece;
          if (dr >= 0 && cc < p.N) *reinterpret_cast<uint4*>(p.act + static_cast<size_t>(dr) * p.N + cc) = val;
        }
      }
    }
    // ------------------------------------------------------------ weights tiles
    const int total = sch.total();
    for (; on && tile < total; tile += gridDim.x, ++n) {
      if (!wait_info(n)) {
        ptx::bar_and(5, 32 * kEpiWarps, false);
        break;
      }
      const Ids id;
      const int h = id.h, set = id.set, f = id.f, ht = id.ht, lane = f & 31;
      const Tile t = info(n);
      const uint32_t dst_t = sbase + S::META + (n & 1) * 1024, w_t = dst_t + 512;   // plain
      // half h joins the rows 32 h .. of the tile; where the second half has none, the first
      // one's warps arrive on the accumulators' barriers for both
      uint64_t sum[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[i] = 0;
      if (32 * h < t.n_tok) {
        const int acc_shift = ld_shared_u32(sbase + S::MISC + S::kSmall) ? 3 : 2;
        const uint32_t acc_mask = (1u << acc_shift) - 1u, acc_cols = 512u >> acc_shift;
        const uint32_t n_arrive = t.n_tok > 32 ? 1 : 2;
        const bool wide = t.n_tok > 32 * h + 16;
        const uint32_t taddr0 = id.tmem(tmem_base) + 32 * h;
        uint32_t w_at = kChunkW + set * kChunk * 4;
        if (kGU) {
          const int up = p.N + t.n0;
          w_at = kChunkW + (f < 64 ? 1 + (up + 64 * set + f) / kBlk - up / kBlk : 0) * kChunk * 4;
        }
        uint32_t sc = 0;
        for (int kb = 0; kb < nk; ++kb) {
          if ((kb & (kChunk - 1)) == 0) {
            if (kb > 0) {
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(bar_sempty(q & 1));
              ++q;
            }
            wait_lean(bar_sfull(q & 1), (q >> 1) & 1u, sbase + S::MISC);
            sc = sbase + S::SCALE + (q & 1) * kChunkBytes;
          }
          const uint32_t fk = sc + (kb & (kChunk - 1)) * kRowStride + 128 * h;
          const uint64_t s2 = ptx::pair(ptx::ld_shared_f32(sc + w_at + (kb & (kChunk - 1)) * 4));
          const uint32_t acc = parts & acc_mask;
          wait_lean(bar_tfull(acc), (parts >> acc_shift) & 1u, sbase + S::MISC);
          ptx::tc_fence_after();
          uint32_t v[32];
          ptx::tmem_ld_32x32b_x32(taddr0 + acc * acc_cols, v);
          ptx::tmem_ld_wait();
          ptx::tc_fence_before();
          if (lane == 0) ptx::mbar_arrive_n(bar_tempty(acc), n_arrive);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (i < 4 || wide) {
              const uint4 a4 = ptx::ld_shared_v4(fk + 16 * i);
              const uint64_t lo = ptx::mul2(ptx::pair(a4.x, a4.y), s2), hi = ptx::mul2(ptx::pair(a4.z, a4.w), s2);
              sum[2 * i] = ptx::fma2(ptx::pair(v[4 * i], v[4 * i + 1]), lo, sum[2 * i]);
              sum[2 * i + 1] = ptx::fma2(ptx::pair(v[4 * i + 2], v[4 * i + 3]), hi, sum[2 * i + 1]);
            }
          }
          parts += 2;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_sempty(q & 1));
        ++q;
      } else {
        parts += 2 * nk;
        for (int kb = 0; kb < nk; kb += kChunk, ++q) {   // every phase is seen, every chunk released
          wait_lean(bar_sfull(q & 1), (q >> 1) & 1u, sbase + S::MISC);
          if (lane == 0) ptx::mbar_arrive(bar_sempty(q & 1));
        }
      }
      // one decision for the sixteen warps (and those without rows wait for the others)
      if (!ptx::bar_and(5, 32 * kEpiWarps, ld_shared_u32(sbase + S::MISC + S::kAbort) == 0)) break;
      // 16 rows of the half at a time through its 8 KB of staging: [16 rows][256 weight rows] bf16,
      // 16-byte pieces XOR-swizzled by the row
      const uint32_t ost = sbase + S::EPI + h * 8192;
      const uint32_t place = ost + ((ht >> 3) << 4) + (ht & 7) * 2;
      const int tok = ht >> 4, oct = ht & 15;    // gate/up: row of the 16, 8 features of it
      const int col = t.n0 + 8 * oct;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int j0 = 32 * h + 16 * c;
        if (j0 >= t.n_tok) continue;             // the same for the whole half
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint64_t x[2] = {sum[8 * c + 2 * i], sum[8 * c + 2 * i + 1]};
          if (!kGU && p.pair_weight) {           // one f32 multiply, then the one bf16 rounding
            const uint4 w4 = ptx::ld_shared_v4(w_t + 4 * j0 + 16 * i);
            x[0] = ptx::mul2(x[0], ptx::pair(w4.x, w4.y));
            x[1] = ptx::mul2(x[1], ptx::pair(w4.z, w4.w));
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {          // gate/up: narrowed before the activation
            const uint32_t pk = pack_bf16(x[k]);
            const int jj = 4 * i + 2 * k;
            ptx::st_shared_u16((place ^ (jj << 4)) + jj * 512, static_cast<uint16_t>(pk));
            ptx::st_shared_u16((place ^ ((jj + 1) << 4)) + (jj + 1) * 512, static_cast<uint16_t>(pk >> 16));
          }
        }
        ptx::bar_sync(1 + h, 256);
        if (!kGU) {
          // a warp stores one row's 512 bytes
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int jj = (ht >> 5) + 8 * i;
            const int cc = t.n0 + 8 * lane;
            if (j0 + jj < t.n_tok && cc < p.N) {
              const int d = static_cast<int>(ld_shared_u32(dst_t + 4 * (j0 + jj)));
              const uint4 val = ptx::ld_shared_v4(ost + jj * 512 + ((lane ^ jj) << 4));
              if (d >= 0) *reinterpret_cast<uint4*>(p.out + static_cast<size_t>(d) * p.N + cc) = val;
            }
          }
        } else {
          // sixteen threads hold a row; 8 pieces of up, 8 of gate, and the other 64 features' ones
          const uint32_t row = ost + tok * 512;
          const int piece = (oct >> 3) * 16 + (oct & 7);
          const uint4 u4 = ptx::ld_shared_v4(row + ((piece ^ tok) << 4));
          const uint4 g4 = ptx::ld_shared_v4(row + (((piece + 8) ^ tok) << 4));
          const bool in = col < p.N;             // N % 16 == 0
          const bool live = j0 + tok < t.n_tok;
          const size_t r = static_cast<size_t>(t.r0 + j0 + tok);
          if (p.out && in && live) {
            uint16_t* o = p.out + r * 2 * p.N + col;
            *reinterpret_cast<uint4*>(o) = g4;
            *reinterpret_cast<uint4*>(o + p.N) = u4;
          }
          float g[8], u[8], act[8], m = 0.0f;
          widen8(g4, g);
          widen8(u4, u);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            act[i] = silu_mul(g[i], u[i]);
            m = fmaxf(m, fabsf(act[i]));
          }
          if (!in) m = 0.0f;
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          float d, inv;
          block_scale(m, d, inv);
          if (in && live)
            *reinterpret_cast<uint2*>(p.act + r * p.N + col) = make_uint2(
                codes4(__fmul_rn(act[0], inv), __fmul_rn(act[1], inv), __fmul_rn(act[2], inv), __fmul_rn(act[3], inv)),
                codes4(__fmul_rn(act[4], inv), __fmul_rn(act[5], inv), __fmul_rn(act[6], inv), __fmul_rn(act[7], inv)));
          if (oct == 0 && live) p.act_scale[r * blocks_of(p.N) + t.n0 / kBlk] = d;
        }
        ptx::bar_sync(1 + h, 256);
      }
      if (lane == 0) ptx::mbar_arrive(bar_iempty(n & 1));
    }
  }

  // ---- exit: a CTA that gave up drains its MMAs and copies before it frees memory
  __syncthreads();
  if (*abort_flag != 0) {
    if (mma_any) {   // the issuing threads
      ptx::mma_commit(bar_drain(warp - 1));
      gemm::spin_bounded(bar_drain(warp - 1), 0);
    }
    // the producer's copies: the last kStages fills may still be on their way
    if (warp == 0 && lane == 0)
      for (uint32_t i = loads < kStages ? 0 : loads - kStages; i < loads; ++i)
        gemm::spin_bounded(bar_full(i % kStages), (i / kStages) & 1u);
  }
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, 512);
  }
}

template <bool kGU>
int launch_range(const char* op, const CUtensorMap (&tt)[4], const CUtensorMap& tw, KernelParams kp,
                 cudaStream_t stream) {
  auto kern = fp8_gemm_kernel<kGU>;
  const int smem = Smem::ALLOC;
  static std::atomic<int> ready_dev[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    dev = -1;
  }
  const bool cache = dev >= 0 && dev < 64;
  if (!cache || !ready_dev[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return set_error(MOE_ERR_CUDA, "%s: cannot reserve %d bytes of shared memory: %s", op, smem,
                       cudaGetErrorString(cudaGetLastError()));
    if (cache) ready_dev[dev].store(1, std::memory_order_release);
  }
  const GemmParams& p = kp.g;
  const int fb_cols = kGU ? 128 : 256;
  long long tiles = (p.P + kTokBlock - 1) / kTokBlock + (p.G < p.P ? p.G : p.P);
  tiles *= (p.N + fb_cols - 1) / fb_cols;       // an upper bound
  const long long sms = sm_count();
  if (tiles > sms) tiles = sms;
  return launch_status(launch_kernel(kern, dim3(static_cast<unsigned>(tiles), 1, 1), dim3(kThreads, 1, 1),
                                     smem, stream, nullptr, 0, tt[0], tt[1], tt[2], tt[3], tw, kp),
                       op);
}

}  // namespace

int launch_product(const char* op, const GemmParams& p0, bool gateup, cudaStream_t stream) {
  GemmParams p = p0;
  const int rows = gateup ? 2 * p.N : p.N;
  if (p.P <= kFewRows && static_cast<long long>(p.P) * rows <= kFewProducts) return launch_few(op, p, gateup, stream);
  CUtensorMap tt[4], tw;
  int rc;
  // pairs of codes as 2-byte elements (K is a multiple of 16): the same bytes and the same
  // 128-byte swizzle as a bf16 operand's box
  for (int i = 0; i < 4; ++i)
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
