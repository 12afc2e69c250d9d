// moe_route_grad.cu -- moe_route_logits_backward: the gradients of the router's
// logits product l = x W^T + bias, given dl [T,E] in f32:
//   dx[t,:] = sum_e dl[t,e] W[e,:]     dW[e,:] = sum_t dl[t,e] x[t,:]     db[e] = sum_t dl[t,e]
//
// x and W are bf16 and dl is f32.  The tensor core multiplies bf16, so dl enters as
// a sum of bf16 values, dl = hi + mid + lo (8 + 8 + 8 significand bits: exact), and
// every product is exact in f32.  Both products take all three parts: the rows of a
// softmax router's dl sum to zero, so what the rows of W have in common cancels in dx, and
// what is left can lie below the 16 bits of hi + mid (which took dx 15.5 us instead of
// 18.7).  x and W are read as they lie in memory: their contiguous dimension is an output
// dimension of both products, so they go to the tensor core as MN-major operands straight
// from TMA boxes.
//
// The floor is the bytes: x read and dx written once (67 MB at T = 8192, H = 2048,
// E = 128: 9.9 us), against 6 + 6 FLOP per element and expert on the tensor core
// (26 GFLOP: 14 us of it at most).
//
//   dW  CTA: 128 experts x 128 columns of H x a range of tokens, 64 tokens a step.
//       Eight warps load dl, split it and write the three parts as MN-major operand
//       tiles; a ninth loads x by TMA and issues the MMAs.  hi is summed in one
//       accumulator and mid + lo in another; every 256 tokens both are added to f32 sums
//       in registers while a second pair of accumulators fills, so no chain of
//       tensor-core additions (which may truncate) is longer than 32.  (With chains of
//       1024 tokens dW was more than 1.5 times as far from the 64-bit result as an f32
//       product.)  The ranges' sums go to the workspace and a second kernel adds them in
//       range order.  The CTAs of the first column block also sum dl for db.
//       26 us at the sizes above with the second kernel.  A step takes about 1800 cycles:
//       its MMAs read 128 bytes of operands a cycle from shared memory for 770 of them, the
//       parts of dl and x are written there (500), and dl's loads pass through the same
//       memory (600: a timing copy without them takes 1250 a step).  Sixteen converting
//       warps instead of eight took 28.4 us, so it is not the conversion's latency.
//   dx  CTA: 128 tokens x 256 columns of H, 64 experts a step; dl is split into three
//       K-major operand tiles.  Two CTAs share an SM and fill each other's gaps.  18.7 us
//       alone for 34 MB written, in 1.7 rounds of CTAs that each load, split, multiply and
//       store in turn; dW starts beside its last ones.
#include <atomic>

#include "gemm_common.cuh"
#include "sm100_ptx_fp8.cuh"

namespace moe {
namespace rgrad {
namespace {

constexpr int kConv = 256;              // converting (and epilogue) threads: warps 0-7
constexpr int kThreads = kConv + 32;    // warp 8: TMA and MMA
constexpr int kStepT = 64;              // tokens per step of dW
constexpr int kChunk = 4;               // steps between two additions to the f32 sums
constexpr int kBStages = 4;             // steps of x on their way (its first touch is in DRAM)
constexpr int kBlk = 64 * 128;          // one operand block: 64 K rows (or 64 rows) of 128 bytes

struct WsLimits {
  unsigned long long wait_ns;
  unsigned int* status;
};

// hi, mid and lo of 8 values, packed, by cutting off: a part is the upper half of the rest's
// word.  A value that is not finite is all in hi.
__device__ __forceinline__ void split8(const float (&v)[8], uint4& hi, uint4& mid, uint4& lo) {
  uint32_t part[3][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool fin = fabsf(v[i]) < INFINITY;
    // the upper half of a NaN's word may read as an infinity
    part[0][i] = v[i] != v[i] ? 0x7FFF0000u : __float_as_uint(v[i]) & 0xFFFF0000u;
    const float r = fin ? __fsub_rn(v[i], __uint_as_float(part[0][i])) : 0.0f;   // exact
    part[1][i] = __float_as_uint(r) & 0xFFFF0000u;
    part[2][i] = __float_as_uint(__fsub_rn(r, __uint_as_float(part[1][i])));
  }
  uint32_t w[3][4];
#pragma unroll
  for (int p = 0; p < 3; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[p][i] = __byte_perm(part[p][2 * i], part[p][2 * i + 1], 0x7632);
  hi = make_uint4(w[0][0], w[0][1], w[0][2], w[0][3]);
  mid = make_uint4(w[1][0], w[1][1], w[1][2], w[1][3]);
  lo = make_uint4(w[2][0], w[2][1], w[2][2], w[2][3]);
}

// The same in paired instructions where all 8 values are finite.
__device__ __forceinline__ void cut8(const float (&v)[8], uint4& hi, uint4& mid, uint4& lo) {
  uint32_t h[4], m[4], l[4];
  uint64_t finite = 0;                   // 0 times every rest: NaN where a value is not finite
  const uint64_t minus = ptx::pair(-1.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = __float_as_uint(v[2 * i]), b = __float_as_uint(v[2 * i + 1]);
    h[i] = __byte_perm(a, b, 0x7632);
    const uint64_t r = ptx::fma2(ptx::pair(a & 0xFFFF0000u, b & 0xFFFF0000u), minus, ptx::pair(a, b));
    finite = ptx::fma2(r, 0, finite);
    const float2 f = ptx::unpair(r);
    const uint32_t ra = __float_as_uint(f.x), rb = __float_as_uint(f.y);
    m[i] = __byte_perm(ra, rb, 0x7632);
    const float2 g = ptx::unpair(ptx::fma2(ptx::pair(ra & 0xFFFF0000u, rb & 0xFFFF0000u), minus, r));
    l[i] = __byte_perm(__float_as_uint(g.x), __float_as_uint(g.y), 0x7632);
  }
  const float2 z = ptx::unpair(finite);
  if (z.x + z.y != 0.0f) return split8(v, hi, mid, lo);   // NaN != 0
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  mid = make_uint4(m[0], m[1], m[2], m[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// dl[t, e0 .. e0 + 7], zeros outside [0,T) x [0,E); whole vectors when the row allows it
__device__ __forceinline__ void load_dl8(const float* __restrict__ dl, int t, int e0, int T, int E,
                                         bool vec, float (&v)[8]) {
  const float* p = dl + static_cast<size_t>(t) * E + e0;
  if (t < T && vec && e0 + 8 <= E) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = t < T && e0 + i < E ? __ldg(p + i) : 0.0f;
  }
}

// Bounded wait of any thread (see gemm::wait_bar; the probe without a time hint wakes
// sooner); false once it gives up (the status is raised and the CTA's abort flag set).
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                     const WsLimits& lim) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (ptx::globaltimer_ns() - t0 > lim.wait_ns) {
      if (lim.status) atomicOr(lim.status, static_cast<unsigned int>(MOE_STATUS_TIMEOUT));
      *abort_flag = 1;
    }
  }
  return true;
}

// ------------------------------------------------------------------ dW
struct DwSmem {
  static constexpr int A = 0;                          // 2 stages x 3 parts x 2 blocks of 64 experts
  static constexpr int B = A + 2 * 6 * kBlk;           // kBStages x 2 blocks of 64 columns
  static constexpr int DB = B + kBStages * 2 * kBlk;   // db: [16 token rows][128] f32
  static constexpr int BARS = DB + 16 * 128 * 4;       // fullA, empty, done [2], fullB [kBStages], drain
  static constexpr int MISC = BARS + 48 + 8 * (kBStages + 1);
  static constexpr int ALLOC = MISC + 16 + 1024;
};

struct DwParams {
  const float* dl;
  int T, H, E, steps;          // steps of 64 tokens per range
  float* out;                  // [ranges][E][H] or null (db alone)
  float* db;                   // [ranges][E] or null
  int behind_dx;               // launched right behind route_dx_kernel
  WsLimits lim;
  unsigned long long* launches;
};

__global__ void __launch_bounds__(kThreads, 1)
route_dw_kernel(const __grid_constant__ CUtensorMap tmX, const DwParams p) {
  using S = DwSmem;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = ptx::smem_u32(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto full_a = [&](int s) { return sb + S::BARS + 8u * s; };
  auto empty = [&](int s) { return sb + S::BARS + 16 + 8u * s; };
  auto done = [&](int a) { return sb + S::BARS + 32 + 8u * a; };
  auto full_b = [&](int s) { return sb + S::BARS + 48 + 8u * s; };
  const uint32_t drain = full_b(kBStages);
  count_launch(p.launches, MOE_KID_ROUTE_DW);
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(full_a(s), kConv);
      ptx::mbar_init(empty(s), 1);
    }
    for (int s = 0; s < kBStages; ++s) ptx::mbar_init(full_b(s), 1);
    for (int a = 0; a < 2; ++a) ptx::mbar_init(done(a), 1);
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 8 && lane == 0) ptx::tma_prefetch_desc(&tmX);
  // Behind dx of the same call nothing here waits for it: dx let this kernel start once all
  // earlier work was complete, the two share no output, and the wait comes at the end, so
  // that what follows finds both done.
  if (!p.behind_dx) grid_dep_wait();
  if (warp == 8) {
    ptx::tmem_alloc(sb + S::MISC, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  grid_dep_launch();
  const uint32_t tmem = *reinterpret_cast<uint32_t*>(smem + S::MISC);
  const int h0 = blockIdx.x * 128, e0 = blockIdx.y * 128;
  const size_t range = blockIdx.z;
  const int t0 = static_cast<int>(range) * p.steps * kStepT;
  const int steps = min(p.steps, (p.T - t0 + kStepT - 1) / kStepT);
  const bool mul = p.out != nullptr;
  uint32_t issued = 0;
  if (warp == 8) {
    // ------------------------------------------------------------ TMA and MMA
    if (mul && ptx::elect_one()) {
      constexpr uint32_t idesc = ptx::idesc_bf16_f32_mn(128, 128, true, true);
      auto load = [&](int i) {
        const int s = i % kBStages;
        ptx::mbar_arrive_expect_tx(full_b(s), 2 * kBlk);
        for (int b = 0; b < 2; ++b)
          ptx::tma_load_2d(sb + S::B + (s * 2 + b) * kBlk, &tmX, h0 + 64 * b, t0 + i * kStepT, full_b(s));
        ++issued;
      };
      bool ok = true;
      for (int i = 0; i < kBStages - 1 && i < steps; ++i) load(i);
      for (int i = 0; ok && i < steps; ++i) {
        const int s = i & 1;
        // x of a later step, into the stage that the step before this one has been multiplied from
        if (i + kBStages - 1 < steps) {
          ok = i == 0 || wait(empty(s ^ 1), ((i - 1) >> 1) & 1, abort_flag, p.lim);
          if (!ok) break;
          load(i + kBStages - 1);
        }
        ok = wait(full_b(i % kBStages), (i / kBStages) & 1, abort_flag, p.lim) &&
             wait(full_a(s), (i >> 1) & 1, abort_flag, p.lim);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint64_t db = ptx::desc_mnmajor_sw128(sb + S::B + (i % kBStages) * 2 * kBlk, kBlk);
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          const uint64_t da = ptx::desc_mnmajor_sw128(sb + S::A + (s * 6 + part * 2) * kBlk, kBlk);
#pragma unroll
          for (int k = 0; k < kStepT / 16; ++k)   // a fresh sum per chunk of steps; mid and lo share one
            ptx::mma_bf16(tmem + ((i / kChunk) & 1) * 256u + (part ? 128u : 0u), da + 128ull * k, db + 128ull * k, idesc,
                          i % kChunk != 0 || k != 0 || part == 2 ? 1u : 0u);
        }
        ptx::mma_commit(empty(s));
        if (i % kChunk == kChunk - 1 || i == steps - 1) ptx::mma_commit(done((i / kChunk) & 1));
      }
    }
  } else {
    // ------------------------------------------------------------ conversion and epilogue
    const int o = threadIdx.x & 15, r = threadIdx.x >> 4;      // 8 experts of the 128, token of 16
    const int e = e0 + 8 * o;
    const bool vec = (p.E & 3) == 0 && (reinterpret_cast<uintptr_t>(p.dl) & 15) == 0;
    // this thread's 16 bytes of row t of a block of 64 experts, swizzled by the row
    const uint32_t at = (o >> 3) * kBlk + (((o & 7) ^ (r & 7)) << 4);
    float colsum[8] = {};
    float sum[64];                 // expert e0 + TMEM lane, columns 64 (warp / 4) + 0 .. 63
#pragma unroll
    for (int k = 0; k < 64; ++k) sum[k] = 0.0f;
    // a thread that gives up (ok) still meets the others at the chunks' ends, where all of
    // them leave together (on)
    bool ok = true, on = true;
    // adds chunk c's accumulators to the sums; the issuer takes them again two chunks on, after
    // this thread's arrive on that chunk's first operands
    auto take = [&](int c) {
      if (ok && !wait(done(c & 1), (c >> 1) & 1, abort_flag, p.lim)) ok = false;
      ok = ptx::bar_and(1, kConv, ok);
      if (!ok) return;
      ptx::tc_fence_after();
      const uint32_t ta = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (c & 1) * 256 + (warp >> 2) * 64;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t a[16], b[16];
        ptx::tmem_ld_32x32b_x16(ta + 16 * k, a);
        ptx::tmem_ld_32x32b_x16(ta + 128 + 16 * k, b);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) sum[16 * k + j] += __uint_as_float(a[j]) + __uint_as_float(b[j]);
      }
      ptx::tc_fence_before();
    };
    float v[4][8];   // this step's values, replaced by the next step's as they are split
#pragma unroll
    for (int j = 0; j < 4; ++j) load_dl8(p.dl, t0 + r + 16 * j, e, p.T, p.E, vec, v[j]);
    for (int i = 0; i < steps; ++i) {
      const int s = i & 1;
      if (mul && ok && i >= 2 && !wait(empty(s), ((i - 2) >> 1) & 1, abort_flag, p.lim)) ok = false;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (p.db && blockIdx.x == 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) colsum[k] += v[j][k];
        }
        if (mul && ok) {
          uint4 x[3];
          cut8(v[j], x[0], x[1], x[2]);
          const uint32_t dst = sb + S::A + s * 6 * kBlk + at + (r + 16 * j) * 128;
#pragma unroll
          for (int part = 0; part < 3; ++part)
            ptx::st_shared_v4(dst + part * 2 * kBlk, x[part].x, x[part].y, x[part].z, x[part].w);
        }
        if (i + 1 < steps) load_dl8(p.dl, t0 + (i + 1) * kStepT + r + 16 * j, e, p.T, p.E, vec, v[j]);
      }
      if (!mul) continue;
      if (ok) {
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(full_a(s));
      }
      // the chunk before, while this one is multiplied
      if (i % kChunk == 0 && i > 0) {
        take(i / kChunk - 1);
        if (!ok) {                 // in all of them
          on = false;
          break;
        }
      }
    }
    if (mul && on) take((steps - 1) / kChunk);
    if (mul && ok) {
      // [128 experts][128 columns] through the operands' memory, whose MMAs are done: 512 bytes
      // a row, 16-byte pieces XOR-swizzled by the row; then a warp stores one row at a time
      // (each thread its own row took 4700 cycles, a fifth of the kernel)
      const int row = (warp & 3) * 32 + lane;
#pragma unroll
      for (int k = 0; k < 16; ++k)
        ptx::st_shared_v4(sb + S::A + row * 512 + ((((warp >> 2) * 16 + k) ^ lane) << 4),
                          __float_as_uint(sum[4 * k]), __float_as_uint(sum[4 * k + 1]),
                          __float_as_uint(sum[4 * k + 2]), __float_as_uint(sum[4 * k + 3]));
      ptx::bar_sync(1, kConv);
      const int h = h0 + 4 * lane;
      for (int j = warp; j < 128 && e0 + j < p.E; j += 8)
        if (h < p.H)                     // H % 8 == 0
          *reinterpret_cast<uint4*>(p.out + (range * p.E + e0 + j) * p.H + h) =
              ptx::ld_shared_v4(sb + S::A + j * 512 + ((lane ^ (j & 31)) << 4));
    }
    if (p.db && blockIdx.x == 0) {
      // the 16 threads of an expert octet, in row order
      float* red = reinterpret_cast<float*>(smem + S::DB);     // [16][128]
#pragma unroll
      for (int k = 0; k < 8; ++k) red[r * 128 + 8 * o + k] = colsum[k];
      ptx::bar_sync(1, kConv);
      if (threadIdx.x < 128 && e0 + static_cast<int>(threadIdx.x) < p.E) {
        float sum = 0.0f;
        for (int k = 0; k < 16; ++k) sum += red[k * 128 + threadIdx.x];
        p.db[range * p.E + e0 + threadIdx.x] = sum;
      }
    }
  }
  // ---- exit: a CTA that gave up drains its copies and MMAs first
  __syncthreads();
  if (*abort_flag != 0 && issued != 0) {
    ptx::mma_commit(drain);
    gemm::spin_bounded(drain, 0);
    for (uint32_t i = issued < kBStages ? 0 : issued - kBStages; i < issued; ++i)
      gemm::spin_bounded(full_b(i % kBStages), (i / kBStages) & 1);
  }
  __syncthreads();
  if (warp == 8) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
  if (p.behind_dx) grid_dep_wait();
}

// the ranges' sums in range order: dW as vectors of four, then db
__global__ void __launch_bounds__(256)
route_reduce_kernel(const float* __restrict__ part_w, const float* __restrict__ part_b, int ranges,
                    long long n4, int E, float* __restrict__ dw, float* __restrict__ db,
                    unsigned long long* launches) {
  count_launch(launches, MOE_KID_ROUTE_REDUCE);
  grid_dep_wait();
  grid_dep_launch();
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (dw && i < n4) {
    const float4* p = reinterpret_cast<const float4*>(part_w) + i;
    float4 s = p[0];
    for (int r = 1; r < ranges; ++r) {
      const float4 v = p[r * n4];
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    reinterpret_cast<float4*>(dw)[i] = s;
  }
  if (db && i < E) {
    float s = part_b[i];
    for (int r = 1; r < ranges; ++r) s += part_b[static_cast<size_t>(r) * E + i];
    db[i] = s;
  }
}

// ------------------------------------------------------------------ dx
struct DxSmem {
  static constexpr int A = 0;                          // 3 parts x 128 tokens x 128 bytes (64 experts)
  static constexpr int B = A + 3 * 2 * kBlk;           // 4 blocks of 64 columns x 64 experts
  static constexpr int BARS = B + 4 * kBlk;            // fullA, fullB, done, drain
  static constexpr int MISC = BARS + 32;
  static constexpr int ALLOC = MISC + 16 + 1024;
};

struct DxParams {
  const float* dl;
  int T, H, E;
  uint16_t* dx;
  WsLimits lim;
  unsigned long long* launches;
};

__global__ void __launch_bounds__(kThreads, 2)
route_dx_kernel(const __grid_constant__ CUtensorMap tmW, const DxParams p) {
  using S = DxSmem;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = ptx::smem_u32(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t full_a = sb + S::BARS, full_b = sb + S::BARS + 8, done = sb + S::BARS + 16, drain = sb + S::BARS + 24;
  count_launch(p.launches, MOE_KID_ROUTE_DX);
  if (threadIdx.x == 0) {
    ptx::mbar_init(full_a, kConv);
    ptx::mbar_init(full_b, 1);
    ptx::mbar_init(done, 1);
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 8 && lane == 0) ptx::tma_prefetch_desc(&tmW);
  // Tensor memory is taken after the wait and before the next kernel may start: these CTAs
  // share SMs, and none that waits for another kernel holds what that kernel needs.
  grid_dep_wait();
  if (warp == 8) {
    ptx::tmem_alloc(sb + S::MISC, 256);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  grid_dep_launch();
  const uint32_t tmem = *reinterpret_cast<uint32_t*>(smem + S::MISC);
  const int h0 = blockIdx.x * 256, t0 = blockIdx.y * 128;
  const int steps = (p.E + 63) / 64;
  uint32_t issued = 0;
  if (warp == 8) {
    if (ptx::elect_one()) {
      constexpr uint32_t idesc = ptx::idesc_bf16_f32_mn(128, 256, false, true);
      bool ok = true;
      for (int i = 0; ok && i < steps; ++i) {
        // the step before has been multiplied: its operands may be overwritten
        ok = i == 0 || wait(done, (i - 1) & 1, abort_flag, p.lim);
        if (!ok) break;
        ptx::mbar_arrive_expect_tx(full_b, 4 * kBlk);
        for (int b = 0; b < 4; ++b)
          ptx::tma_load_2d(sb + S::B + b * kBlk, &tmW, h0 + 64 * b, 64 * i, full_b);
        ++issued;
        ok = wait(full_b, i & 1, abort_flag, p.lim) && wait(full_a, i & 1, abort_flag, p.lim);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint64_t db = ptx::desc_mnmajor_sw128(sb + S::B, kBlk);
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          const uint64_t da = ptx::desc_kmajor_sw128(sb + S::A + part * 2 * kBlk);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            ptx::mma_bf16(tmem, da + 2ull * k, db + 128ull * k, idesc, (i | part | k) != 0 ? 1u : 0u);
        }
        ptx::mma_commit(done);
      }
    }
  } else {
    const int o = threadIdx.x & 7, r = threadIdx.x >> 3;       // 8 experts of 64, token of 32
    const bool vec = (p.E & 3) == 0 && (reinterpret_cast<uintptr_t>(p.dl) & 15) == 0;
    bool ok = true;
    float next[4][8];
    auto fetch = [&](int i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) load_dl8(p.dl, t0 + r + 32 * j, 64 * i + 8 * o, p.T, p.E, vec, next[j]);
    };
    fetch(0);
    for (int i = 0; ok && i < steps; ++i) {
      float v[4][8];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] = next[j][k];
      if (i + 1 < steps) fetch(i + 1);   // on its way while this step is split
      if (i > 0 && !wait(done, (i - 1) & 1, abort_flag, p.lim)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4 hi, mid, lo;
        cut8(v[j], hi, mid, lo);
        const int row = r + 32 * j;
        const uint32_t dst = sb + S::A + row * 128 + ((o ^ (row & 7)) << 4);
        ptx::st_shared_v4(dst, hi.x, hi.y, hi.z, hi.w);
        ptx::st_shared_v4(dst + 2 * kBlk, mid.x, mid.y, mid.z, mid.w);
        ptx::st_shared_v4(dst + 4 * kBlk, lo.x, lo.y, lo.z, lo.w);
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(full_a);
    }
    if (ok && !wait(done, (steps - 1) & 1, abort_flag, p.lim)) ok = false;
    if (ptx::bar_and(1, kConv, ok)) {
      // [128 tokens][256 columns] bf16 through the operands' memory: 512 bytes a row, 16-byte
      // pieces XOR-swizzled by the row; then a warp stores one row at a time
      ptx::tc_fence_after();
      const int row = (warp & 3) * 32 + lane;
      const uint32_t ta = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (warp >> 2) * 128;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t a[32];
        ptx::tmem_ld_32x32b_x32(ta + 32 * c, a);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int piece = (warp >> 2) * 16 + 4 * c + k;
          uint32_t w[4];
#pragma unroll
          for (int m = 0; m < 4; ++m)
            w[m] = gemm::pack_bf16x2(__uint_as_float(a[8 * k + 2 * m]), __uint_as_float(a[8 * k + 2 * m + 1]));
          ptx::st_shared_v4(sb + row * 512 + ((piece ^ (row & 31)) << 4), w[0], w[1], w[2], w[3]);
        }
      }
      ptx::tc_fence_before();
      ptx::bar_sync(1, kConv);
      for (int j = warp; j < 128; j += 8) {
        const int t = t0 + j, h = h0 + 8 * lane;
        if (t < p.T && h < p.H)
          *reinterpret_cast<uint4*>(p.dx + static_cast<size_t>(t) * p.H + h) =
              ptx::ld_shared_v4(sb + j * 512 + ((lane ^ (j & 31)) << 4));
      }
    }
  }
  __syncthreads();
  if (*abort_flag != 0 && issued != 0) {
    ptx::mma_commit(drain);
    gemm::spin_bounded(drain, 0);
    gemm::spin_bounded(full_b, (issued - 1) & 1);
  }
  __syncthreads();
  if (warp == 8) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 256);
  }
}

static_assert(DxSmem::ALLOC * 2 <= 227 * 1024, "two dx CTAs per SM");
static_assert(DwSmem::ALLOC <= 227 * 1024, "shared memory");

// steps of 64 tokens per range: enough ranges to give every SM a CTA, but at least six
// steps in each, since a range costs a pass over its [E,H] sums and more than one a launch
struct Ranges {
  int steps, count;
  int bound;   // no smaller for more tokens, never below count: what the workspace is sized by
};
Ranges ranges_of(int T, int H, int E) {
  const int total = T / kStepT + (T % kStepT != 0);
  const long long tiles = (H / 128 + (H % 128 != 0)) * ((E - 1) / 128 + 1ll);
  int want = static_cast<int>(sm_count() / tiles);
  if (want > total / 6) want = total / 6;
  if (want > 32) want = 32;
  if (want < 1) want = 1;
  Ranges r;
  r.bound = want;
  // whole steps: fewer tokens can make more ranges (54 steps in nine ranges, 55 in eight)
  r.steps = (total + want - 1) / want;
  r.count = (total + r.steps - 1) / r.steps;
  return r;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

template <typename K>
int reserve(const char* op, K kern, int smem, std::atomic<int>* ready) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    dev = -1;
  }
  const bool cache = dev >= 0 && dev < 64;
  if (cache && ready[dev].load(std::memory_order_acquire)) return MOE_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "%s: cannot reserve %d bytes of shared memory: %s", op, smem,
                     cudaGetErrorString(cudaGetLastError()));
  if (cache) ready[dev].store(1, std::memory_order_release);
  return MOE_OK;
}

}  // namespace
}  // namespace rgrad
}  // namespace moe

using namespace moe;
using namespace moe::rgrad;

extern "C" {

size_t moe_route_logits_backward_workspace_size(int T, int H, int E) {
  if (T <= 0 || H <= 0 || E <= 0) return 0;
  const Ranges r = ranges_of(T, H, E);
  if (r.bound == 1) return 0;
  return static_cast<size_t>(r.bound) * E * (static_cast<size_t>(H) + 1) * sizeof(float);
}

int moe_route_logits_backward(const float* grad_logits, const void* x_bf16, const void* w_router_bf16,
                              int T, int H, int E, void* grad_x_bf16, float* grad_w_router,
                              float* grad_bias, void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  const char* op = "moe_route_logits_backward";
  if (T < 0 || H <= 0) return set_error(MOE_ERR_ARG, "%s: bad sizes T=%d H=%d", op, T, H);
  if (E < 1 || E > 1024) return set_error(MOE_ERR_ARG, "%s: E=%d outside [1, 1024]", op, E);
  if (H % 8 != 0) return set_error(MOE_ERR_ALIGN, "%s: H=%d is not a multiple of 8", op, H);
  if (T > 128 * 65535) return set_error(MOE_ERR_ARG, "%s: T=%d is too large", op, T);   // the grid's y
  if (H > kMaxDim) return set_error(MOE_ERR_ARG, "%s: H=%d is too large", op, H);
  if (!grad_x_bf16 && !grad_w_router && !grad_bias)
    return set_error(MOE_ERR_ARG, "%s: no output requested", op);
  if (T > 0 && (!grad_logits || (grad_x_bf16 && !w_router_bf16) || (grad_w_router && !x_bf16)))
    return set_error(MOE_ERR_ARG, "%s: NULL operand", op);
  if (!aligned16(x_bf16) || !aligned16(w_router_bf16) || !aligned16(grad_x_bf16) ||
      !aligned16(grad_w_router))
    return set_error(MOE_ERR_ALIGN, "%s: x, w_router, grad_x and grad_w_router must be 16-byte aligned",
                     op);
  if (!aligned4(grad_logits) || !aligned4(grad_bias))
    return set_error(MOE_ERR_ALIGN, "%s: grad_logits and grad_bias must be 4-byte aligned", op);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {   // sums over no token
    if (grad_w_router &&
        cudaMemsetAsync(grad_w_router, 0, static_cast<size_t>(E) * H * sizeof(float), s) != cudaSuccess)
      return check_launch(op);
    if (grad_bias && cudaMemsetAsync(grad_bias, 0, E * sizeof(float), s) != cudaSuccess)
      return check_launch(op);
    return MOE_OK;
  }
  const bool sums = grad_w_router || grad_bias;
  const Ranges rg = ranges_of(T, H, E);
  if (sums && rg.count > 1) {
    if (!workspace || ws_bytes < moe_route_logits_backward_workspace_size(T, H, E))
      return set_error(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", op, ws_bytes,
                       moe_route_logits_backward_workspace_size(T, H, E));
    if (!aligned16(workspace)) return set_error(MOE_ERR_ALIGN, "%s: workspace must be 16-byte aligned", op);
  }
  DeviceDiag diag = device_diag();
  const WsLimits lim{gemm::pipeline_wait_ns(), diag.status};
  static std::atomic<int> ready_dx[64] = {}, ready_dw[64] = {};
  int rc;
  if (grad_x_bf16) {
    if ((rc = reserve(op, route_dx_kernel, DxSmem::ALLOC, ready_dx)) != MOE_OK) return rc;
    CUtensorMap tm;
    if ((rc = gemm::make_tmap(&tm, w_router_bf16, E, H, 64, op, "w_router")) != MOE_OK) return rc;
    DxParams p{grad_logits, T, H, E, static_cast<uint16_t*>(grad_x_bf16), lim, diag.launches};
    rc = launch_status(launch_kernel(route_dx_kernel, dim3((H + 255) / 256, (T + 127) / 128), dim3(kThreads),
                                     DxSmem::ALLOC, s, nullptr, 0, tm, p),
                       op);
    if (rc != MOE_OK) return rc;
  }
  if (sums) {
    if ((rc = reserve(op, route_dw_kernel, DwSmem::ALLOC, ready_dw)) != MOE_OK) return rc;
    CUtensorMap tm{};
    if (grad_w_router && (rc = gemm::make_tmap(&tm, x_bf16, T, H, kStepT, op, "x")) != MOE_OK) return rc;
    float* part_w = rg.count > 1 ? static_cast<float*>(workspace) : grad_w_router;
    float* part_b = rg.count > 1 ? static_cast<float*>(workspace) + static_cast<size_t>(rg.count) * E * H : grad_bias;
    DwParams p{grad_logits, T, H, E, rg.steps, grad_w_router ? part_w : nullptr,
               grad_bias ? part_b : nullptr, grad_x_bf16 && pdl_enabled() ? 1 : 0, lim, diag.launches};
    rc = launch_status(launch_kernel(route_dw_kernel,
                                     dim3(grad_w_router ? (H + 127) / 128 : 1, (E + 127) / 128, rg.count),
                                     dim3(kThreads), DwSmem::ALLOC, s, nullptr, 0, tm, p),
                       op);
    if (rc != MOE_OK) return rc;
    if (rg.count > 1) {
      const long long n4 = static_cast<long long>(E) * H / 4;
      const long long n = grad_w_router ? (n4 > E ? n4 : E) : E;
      rc = launch_status(launch_kernel(route_reduce_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256),
                                       0, s, nullptr, 0, static_cast<const float*>(part_w),
                                       static_cast<const float*>(part_b), rg.count, n4, E, grad_w_router,
                                       grad_bias, diag.launches),
                         op);
      if (rc != MOE_OK) return rc;
    }
  }
  return MOE_OK;
}

}  // extern "C"
