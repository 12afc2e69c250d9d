// moe_fp8_few.cu -- the FP8 products of a call with few rows in all (a decoded token).
//
// Every weight of a row's group is used once, so the product is a read of the weights:
// what bounds it is how many SMs read, and how soon.  The tiles of moe_fp8_gemm.cu give a
// row's group to an SM per 256 weight rows (4 SMs for one row of 1024 columns); here a
// warp takes 4 output columns (gate/up: 4 features' gate and up rows) of one row, every
// lane 16 codes of each per step, and all loads of a step are in flight together.
//
//   y[r,n] = sum over pieces of 16 columns: (sum of the piece's products) sa sw,
//
// in f32: products of two E4M3 values are exact (both operands as f16, the multiply-add
// widens), and the lanes' sums are joined by a butterfly, in one order.  Two steps of 512
// columns are loaded before either is used: with one, each waited for memory anew (9.9 us
// instead of 7.8 for the gate/up products of 8 rows, 2048 x 768), and with four the idle
// lanes of short rows cost more.  A row of 4096 x 1024 takes 5.0 us, on tiles 13.8.
#include "fp8_common.cuh"

namespace moe {
namespace fp8 {
namespace {

constexpr int kWarps = 8, kCols = 4;          // columns (gate/up: features) per warp
constexpr int kCta = kWarps * kCols;          // and per CTA: a quarter of a scale block

__device__ __forceinline__ void st_cluster_f32(uint32_t cluster_addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 16 codes as pairs of f16, which hold every E4M3 value
__device__ __forceinline__ void decode16(const uint4& c, __half2 (&v)[8]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3));
}
// c + a b, the product exact
__device__ __forceinline__ float fma_half(__half a, __half b, float c) {
  float d;
  asm("fma.rn.f32.f16 %0, %1, %2, %3;"
      : "=f"(d) : "h"(__half_as_ushort(a)), "h"(__half_as_ushort(b)), "f"(c));
  return d;
}

// the group of row r (all lanes of a warp), or -1: the last one that starts at or before r
__device__ __forceinline__ int group_of(const int32_t* __restrict__ off, int G, int r, int lane) {
  if (!off) return 0;
  int n = 0;
  for (int i = lane; i <= G; i += 32) n += __ldg(off + i) <= r ? 1 : 0;
  n = __reduce_add_sync(0xffffffffu, n);
  return n >= 1 && n <= G ? n - 1 : -1;
}

// kRows dot products of the codes a[K] with rows of w at w0 + i * step (one weight scale
// block for each run of kCols of them), summed over the warp
template <int kRows>
__device__ __forceinline__ void dots(const uint8_t* __restrict__ a, const float* __restrict__ sa,
                                     const uint8_t* const (&w)[kRows / kCols], const float* const (&sw)[kRows / kCols],
                                     int K, int lane, float (&acc)[kRows]) {
#pragma unroll
  for (int i = 0; i < kRows; ++i) acc[i] = 0.0f;
  constexpr int kSteps = 2;      // 512 columns each, loaded together
  for (int k0 = lane * 16; k0 < K; k0 += 512 * kSteps) {
    uint4 ar[kSteps], raw[kSteps][kRows];
    float s[kSteps][kRows / kCols];
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      const int k = min(k0 + 512 * t, K - 16);
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        raw[t][i] = __ldg(reinterpret_cast<const uint4*>(w[i / kCols] + static_cast<size_t>(i % kCols) * K + k));
      ar[t] = __ldg(reinterpret_cast<const uint4*>(a + k));
      const float d = __ldg(sa + k / kBlk);
#pragma unroll
      for (int i = 0; i < kRows / kCols; ++i) s[t][i] = __fmul_rn(d, __ldg(sw[i] + k / kBlk));
    }
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      if (k0 + 512 * t >= K) break;
      __half2 x[8];
      decode16(ar[t], x);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        __half2 y[8];
        float p = 0.0f;
        decode16(raw[t][i], y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          p = fma_half(__low2half(x[j]), __low2half(y[j]), p);
          p = fma_half(__high2half(x[j]), __high2half(y[j]), p);
        }
        acc[i] = fmaf(p, s[t][i / kCols], acc[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
}

// grid (columns / 32, rows)
__global__ void __launch_bounds__(32 * kWarps)
few_rows_kernel(const GemmParams p, unsigned long long* launches) {
  count_launch(launches, p.kid);
  count_launch(launches, MOE_KID_GEMM_FP8_FEW);
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.y;
  const int n0 = blockIdx.x * kCta + warp * kCols;
  if (n0 >= p.N) return;         // N % 8 == 0: four columns are in or out together
  const int d = p.row_to_pair ? __ldg(p.row_to_pair + r) : r;
  const int g = group_of(p.group_offsets, p.G, r, lane);
  if (g < 0 || d < 0 || d >= p.P) return;
  const float weight = p.pair_weight ? __ldg(p.pair_weight + d) : 1.0f;
  const int nk = blocks_of(p.K);
  const uint8_t* w[1] = {p.w + (static_cast<size_t>(g) * p.N + n0) * p.K};
  const float* sw[1] = {p.sw + (static_cast<size_t>(g) * blocks_of(p.N) + n0 / kBlk) * nk};
  float acc[kCols];
  dots<kCols>(p.a + static_cast<size_t>(r) * p.K, p.sa + static_cast<size_t>(r) * nk, w, sw, p.K, lane, acc);
  if (lane == 0)                 // one f32 multiply, then the one bf16 rounding
    *reinterpret_cast<uint2*>(p.out + static_cast<size_t>(d) * p.N + n0) =
        make_uint2(gemm::pack_bf16x2(__fmul_rn(acc[0], weight), __fmul_rn(acc[1], weight)),
                   gemm::pack_bf16x2(__fmul_rn(acc[2], weight), __fmul_rn(acc[3], weight)));
}

// gate/up: a cluster of four CTAs holds a row's 128 features and joins their largest
// magnitude through distributed shared memory.  grid (4 * blocks of 128 features, rows)
__global__ void __launch_bounds__(32 * kWarps)
few_rows_gateup_kernel(const GemmParams p, unsigned long long* launches) {
  __shared__ float s_max[4 * kWarps];
  cluster_arrive();              // waited for before the first store to another CTA
  count_launch(launches, p.kid);
  count_launch(launches, MOE_KID_GEMM_FP8_FEW);
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.y;
  const int n0 = blockIdx.x * kCta + warp * kCols;
  const bool in = n0 < p.N;      // N % 16 == 0
  const int g = group_of(p.group_offsets, p.G, r, lane);
  if (g < 0) {                   // the whole cluster: it has one row
    cluster_wait();
    return;
  }
  const int nk = blocks_of(p.K), rb = blocks_of(2 * p.N);
  float act[kCols] = {}, m = 0.0f;
  if (in) {
    const uint8_t* base = p.w + static_cast<size_t>(g) * 2 * p.N * p.K;
    const float* sbase = p.sw + static_cast<size_t>(g) * rb * nk;
    const uint8_t* w[2] = {base + static_cast<size_t>(n0) * p.K, base + static_cast<size_t>(p.N + n0) * p.K};
    const float* sw[2] = {sbase + static_cast<size_t>(n0 / kBlk) * nk,
                          sbase + static_cast<size_t>((p.N + n0) / kBlk) * nk};
    float acc[2 * kCols];
    dots<2 * kCols>(p.a + static_cast<size_t>(r) * p.K, p.sa + static_cast<size_t>(r) * nk, w, sw, p.K, lane, acc);
    uint32_t pk[kCols];          // gate, then up, narrowed before the activation
#pragma unroll
    for (int i = 0; i < kCols; ++i) pk[i] = gemm::pack_bf16x2(acc[2 * i], acc[2 * i + 1]);
    if (p.out && lane == 0) {
      uint16_t* o = p.out + static_cast<size_t>(r) * 2 * p.N + n0;
      *reinterpret_cast<uint2*>(o) = make_uint2(pk[0], pk[1]);
      *reinterpret_cast<uint2*>(o + p.N) = make_uint2(pk[2], pk[3]);
    }
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const uint32_t gw = pk[i / 2], uw = pk[2 + i / 2];
      const float gv = __uint_as_float(i & 1 ? gw & 0xFFFF0000u : gw << 16);
      const float uv = __uint_as_float(i & 1 ? uw & 0xFFFF0000u : uw << 16);
      act[i] = silu_mul(gv, uv);
      m = fmaxf(m, fabsf(act[i]));
    }
  }
  // every warp's largest magnitude to the four CTAs, slot by CTA and warp
  const uint32_t rank = ptx::cluster_ctarank();
  cluster_wait();
  if (lane < 4)
    st_cluster_f32(ptx::mapa_shared(ptx::smem_u32(s_max) + (rank * kWarps + warp) * 4, lane), m);
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  m = s_max[lane];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!in || lane != 0) return;
  float d, inv;
  block_scale(m, d, inv);
  *reinterpret_cast<uint32_t*>(p.act + static_cast<size_t>(r) * p.N + n0) =
      codes4(__fmul_rn(act[0], inv), __fmul_rn(act[1], inv), __fmul_rn(act[2], inv), __fmul_rn(act[3], inv));
  if (n0 % kBlk == 0) p.act_scale[static_cast<size_t>(r) * blocks_of(p.N) + n0 / kBlk] = d;
}

}  // namespace

int launch_few(const char* op, const GemmParams& p, bool gateup, cudaStream_t stream) {
  DeviceDiag diag = device_diag();
  if (!gateup)
    return launch_status(launch_kernel(few_rows_kernel, dim3((p.N + kCta - 1) / kCta, p.P), dim3(32 * kWarps),
                                       0, stream, nullptr, 0, p, diag.launches),
                         op);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kBlk / kCta;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  return launch_status(launch_kernel(few_rows_gateup_kernel, dim3(blocks_of(p.N) * (kBlk / kCta), p.P),
                                     dim3(32 * kWarps), 0, stream, attr, 1, p, diag.launches),
                       op);
}

}  // namespace fp8
}  // namespace moe
