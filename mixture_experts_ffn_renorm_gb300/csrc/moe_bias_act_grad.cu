// moe_bias_act_grad.cu -- the gradient of the products' epilogue (moe_gemm_bias_act.cu):
//
//   dy[r] = dout[dst] * pair_weight[dst],  s = dy act'(z):  dz = bf16(s),
//   grad_bias[g] = sum of s over g's rows,  grad_pair_weight[dst] = sum_n dout[dst,n] act(z[r,n])
//
// One pass over dout and z: what bounds it is HBM (6 bytes an element), with GELU the instructions.  A CTA takes 256
// columns of a range of rows, three CTAs an SM, one wave of them; a warp every eighth row, a lane 8 columns, so that its column sums are
// 8 registers and its row sums one butterfly each.  A warp's next eight rows are always under way to its own
// shared memory (cp.async, no barrier): 192 KB an SM.
// 32768 x 768 with bias and row weights takes 43.2 us with GELU (3.5 TB/s), 38 with GELU by tanh, 34 with SiLU, 33 with
// ReLU or none (HBM 22).  A warp spends 286 instructions on a row's 256 columns with GELU, 195 with SiLU and 179 with ReLU,
// which has next to no arithmetic: copies, widening, packing, the row's sum and addresses are most of them.  The second
// kernel takes 6 us by itself.  (Blocks of 64 rows, three rows of a warp in registers, 2.5 waves: 42.6, 37.8 and
// 37.  A CTA for all columns of 64 rows: 48.  All 64 rows of a block asked for at once: 43.6 and 39.)
// A CTA's rows may meet several groups: at
// each group's end the warps' column sums are joined through shared memory in warp order and
// leave as one partial row.  Block c and group g meet in partial row c + g: along the rows
// either index or both step up, so no two meetings share one, and the second kernel finds a
// group's rows from its offsets alone.  It adds them in block order: fixed order, no atomics.
#include <atomic>

#include "activation.cuh"
#include "gemm_common.cuh"

namespace moe {
namespace gemm {
namespace {

constexpr int kCols = 256;           // columns of a CTA: 8 per lane
constexpr int kWarps = 8;
constexpr int kCtas = 3;             // per SM
constexpr int kLeast = 16;           // rows of a CTA, at least
constexpr int kAhead = 8;            // rows of a warp whose copies are under way
constexpr int kBytes = kWarps * kAhead * kCols * 2 * 2;        // dout's and z's

struct BackParams {
  const uint16_t* dout;
  const uint16_t* z;
  int activation;
  const float* pair_weight;
  const int32_t* row_to_pair;
  const int32_t* group_offsets;
  int P, N, G, rows;
  uint16_t* dz;
  float* part_b;                     // [blocks + G][N] column sums, or null
  float* part_w;                     // [column blocks][P] row sums by row (one block: by dst), or null
  unsigned long long* launches;
};

__device__ __forceinline__ int offset_at(const int32_t* off, int i, int P) {
  return off ? min(max(__ldg(off + i), 0), P) : (i == 0 ? 0 : P);
}

// 8 bf16 values as four pairs of f32
__device__ __forceinline__ void widen(const uint4& u, uint64_t (&v)[4]) {
  const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = ptx::pair(q[i] << 16, q[i] & 0xFFFF0000u);
}

// 16 bytes to shared memory on their own, or zeros
__device__ __forceinline__ void copy16(uint4* to, const uint16_t* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(to)), "l"(from), "r"(there ? 16 : 0)
               : "memory");
}
template <int kAct>
__global__ void __launch_bounds__(32 * kWarps, kCtas)
bias_act_backward_kernel(const BackParams p) {
  extern __shared__ uint4 s_rows[];  // [warp][own row modulo kAhead][dout, z][lane]
  __shared__ float s_sum[kWarps][kCols];
  count_launch(p.launches, MOE_KID_BIAS_ACT_BACKWARD);
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int block = blockIdx.x, r_lo = block * p.rows, r_hi = r_lo + min(p.rows, p.P - r_lo);
  const int n = blockIdx.y * kCols + lane * 8;
  const bool live = n < p.N;
  // This warp's rows r_lo + warp + 8 i, i < own.  Destinations and weights of the 32 around row i, lane i % 32, and of
  // the 32 after them.
  const int own = (r_hi - r_lo - warp + kWarps - 1) / kWarps;
  int d_now = -1, d_next = -1;
  float w_now = 1.0f, w_next = 1.0f;
  auto look_up = [&](int i, int& d, float& w) {
    d = -1;
    w = 1.0f;
    if (i >= own) return;
    const int r = r_lo + warp + kWarps * i;
    d = p.row_to_pair ? __ldg(p.row_to_pair + r) : r;
    if (d < 0 || d >= p.P) d = -1;
    else if (p.pair_weight) w = __ldg(p.pair_weight + d);
  };
  look_up(lane, d_now, w_now);
  look_up(32 + lane, d_next, w_next);
  // The copies of row j, for i = the row that is worked on; a group for every row, also behind the last.  A row without a
  // destination comes as zeros, of z too.
  uint4* mine = s_rows + warp * (2 * kAhead * 32) + lane;
  const size_t first = static_cast<size_t>(r_lo + warp) * p.N + (live ? n : 0), stride = static_cast<size_t>(kWarps) * p.N;
  const uint16_t *z = p.z ? p.z + first : nullptr, *dout = p.dout + (live ? n : 0);
  uint16_t* dz = p.dz + first;
  auto bring = [&](int j, int i) {
    const int d = __shfl_sync(0xffffffffu, (j >> 5) == (i >> 5) ? d_now : d_next, j & 31);
    if (j < own) {
      const bool there = live && d >= 0;
      uint4* to = mine + (j % kAhead) * 64;
      if (z) copy16(to + 32, z, there);
      copy16(to, dout + (there ? static_cast<size_t>(d) * p.N : 0), there);
    }
    if (z) z += stride;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int j = 0; j < kAhead; ++j) bring(j, 0);
  int i = 0;                         // the next row
  auto step = [&]() {
    bring(i + kAhead, i);
    dz += stride;
    if ((++i & 31) == 0) {
      d_now = d_next;
      w_now = w_next;
      look_up(i + 32 + lane, d_next, w_next);
    }
  };
  // the last group that starts at or before the block's first row
  int before = 0;
  for (int g0 = 0; g0 < p.G; g0 += 32 * kWarps) {
    const int g = g0 + static_cast<int>(threadIdx.x);
    before += __syncthreads_count(g < p.G && offset_at(p.group_offsets, g, p.P) <= r_lo);
  }
  int g = max(before - 1, 0);
  for (int r0 = max(r_lo, offset_at(p.group_offsets, g, p.P)); g < p.G; ++g) {
    const int r1 = min(r_hi, offset_at(p.group_offsets, g + 1, p.P));
    if (r1 > r0) {
      uint64_t sum[4] = {};
#pragma unroll 1
      while (i < own && r_lo + warp + kWarps * i < r0) step();       // rows of no group
#pragma unroll 1
      for (; i < own && r_lo + warp + kWarps * i < r1; step()) {
        const float w = __shfl_sync(0xffffffffu, w_now, i & 31);
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        uint64_t dy[4], zz[4] = {}, dots = 0;
        uint32_t out[4];
        const uint4* from = mine + (i % kAhead) * 64;
        widen(from[0], dy);
        if (p.z) widen(from[32], zz);
        const uint64_t w2 = ptx::pair(w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint64_t y, s;
          act::slope2<kAct>(zz[j], y, s);
          dots = ptx::fma2(dy[j], y, dots);
          const uint64_t v = ptx::mul2(ptx::mul2(dy[j], w2), s);
          sum[j] = act::add2(sum[j], v);
          const float2 u = ptx::unpair(v);
          out[j] = pack_bf16x2(u.x, u.y);
        }
        if (live)
          *reinterpret_cast<uint4*>(dz) = make_uint4(out[0], out[1], out[2], out[3]);
        if (p.part_w) {
          const float2 u = ptx::unpair(dots);
          float dot = u.x + u.y;
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
          // several column blocks: by row, for the sum; one: the gradient itself, by destination
          if (lane == (i & 31) && d_now >= 0)
            p.part_w[gridDim.y > 1 ? static_cast<size_t>(blockIdx.y) * p.P + r_lo + warp + kWarps * i
                                   : static_cast<size_t>(d_now)] = dot;
        }
      }
      if (p.part_b) {
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint64_t*>(&s_sum[warp][lane * 8 + 2 * j]) = sum[j];
        __syncthreads();
        const int at = blockIdx.y * kCols + static_cast<int>(threadIdx.x);
        if (at < p.N) {
          float s = s_sum[0][threadIdx.x];
#pragma unroll
          for (int k = 1; k < kWarps; ++k) s += s_sum[k][threadIdx.x];
          p.part_b[(static_cast<size_t>(block) + g) * p.N + at] = s;
        }
        __syncthreads();
      }
      r0 = r1;
    }
    if (r0 >= r_hi) break;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// grad_bias: kSlices threads share a group's blocks of four columns, their sums joined in order; a CTA
// of the first G * bias_ctas takes one group and 64 x 4 columns.  grad_pair_weight: the CTAs behind
// them, a thread a row.
constexpr int kSlices = 4;

__global__ void __launch_bounds__(256)
bias_act_reduce_kernel(const BackParams p, float* __restrict__ grad_bias, float* __restrict__ grad_w, int bias_ctas,
                       int col_blocks) {
  __shared__ float4 s_part[kSlices][64];
  count_launch(p.launches, MOE_KID_BIAS_ACT_REDUCE);
  const int id = blockIdx.x;
  const bool bias = id < p.G * bias_ctas;
  const int g = bias ? id / bias_ctas : 0;
  // the offsets are older than the kernel before, which started after what it waited for
  const int r0 = offset_at(p.group_offsets, g, p.P), r1 = offset_at(p.group_offsets, bias ? g + 1 : p.G, p.P);
  grid_dep_wait();
  grid_dep_launch();
  if (bias) {
    const int x = threadIdx.x & 63, slice = threadIdx.x >> 6;
    const int c = 4 * ((id - g * bias_ctas) * 64 + x);
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (r1 > r0 && c < p.N) {
      const float* q = p.part_b + static_cast<size_t>(g) * p.N + c;
      const int b0 = r0 / p.rows, n = (r1 - 1) / p.rows - b0 + 1;
#pragma unroll 8
      for (int b = b0 + n * slice / kSlices; b < b0 + n * (slice + 1) / kSlices; ++b) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(q + static_cast<size_t>(b) * p.N));
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
      }
    }
    s_part[slice][x] = s;
    __syncthreads();
    if (slice == 0 && c < p.N) {
#pragma unroll
      for (int i = 1; i < kSlices; ++i) {
        const float4 v = s_part[i][x];
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
      }
      *reinterpret_cast<float4*>(grad_bias + static_cast<size_t>(g) * p.N + c) = s;
    }
    return;
  }
  const long long i = static_cast<long long>(id - p.G * bias_ctas) * 256 + threadIdx.x;
  // rows outside every group, and destinations that no row has, keep what they hold
  if (!grad_w || i < r0 || i >= r1) return;
  const int d = p.row_to_pair ? __ldg(p.row_to_pair + i) : static_cast<int>(i);
  if (d < 0 || d >= p.P) return;
  float s = __ldcg(p.part_w + i);
#pragma unroll 4
  for (int b = 1; b < col_blocks; ++b) s += __ldcg(p.part_w + static_cast<size_t>(b) * p.P + i);
  grad_w[d] = s;
}

int blocks_of(int n, int size) { return n / size + (n % size != 0); }
size_t pad(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
// Row ranges of a call: one wave of CTAs
int ranges_of(int P, int N) {
  const int all = kCtas * sm_count() / blocks_of(N, kCols), most = blocks_of(P, kLeast);
  return all < 1 ? 1 : all < most ? all : most;
}
size_t bias_bytes(int P, int N, int G) {
  return pad((static_cast<size_t>(ranges_of(P, N)) + G) * N * 4);
}

}  // namespace
}  // namespace gemm
}  // namespace moe

using namespace moe;
using namespace moe::gemm;

extern "C" size_t moe_bias_act_backward_workspace_size(int P, int N, int G) {
  if (P <= 0 || N <= 0 || G <= 0) return 0;
  const size_t cb = blocks_of(N, kCols);
  return bias_bytes(P, N, G) + (cb > 1 ? pad(cb * P * 4) : 0);
}

extern "C" int moe_bias_act_backward(const void* dout_bf16, const void* z_bf16, int activation,
                                     const float* pair_weight, const int32_t* row_to_pair,
                                     const int32_t* group_offsets, int P, int N, int G, void* dz_bf16,
                                     float* grad_bias, float* grad_pair_weight, void* workspace,
                                     size_t ws_bytes, void* stream) {
  clear_error();
  const char* op = "moe_bias_act_backward";
  if (P < 0 || N < 1) return set_error(MOE_ERR_ARG, "%s: P=%d, N=%d", op, P, N);
  if (P > kMaxDim || N > kMaxDim) return set_error(MOE_ERR_ARG, "%s: P=%d or N=%d is too large", op, P, N);
  if (blocks_of(N, kCols) > 65535) return set_error(MOE_ERR_ARG, "%s: N=%d is too large", op, N);
  if (G < 1 || G > kMaxGroups) return set_error(MOE_ERR_ARG, "%s: G=%d outside [1, %d]", op, G, kMaxGroups);
  if (activation < MOE_ACT_NONE || activation > MOE_ACT_SILU)
    return set_error(MOE_ERR_ARG, "%s: activation=%d is not a MOE_ACT_* value", op, activation);
  if (N % 8) return set_error(MOE_ERR_ALIGN, "%s: N=%d must be a multiple of 8", op, N);
  if (!group_offsets && G != 1) return set_error(MOE_ERR_ARG, "%s: group_offsets is NULL with G=%d", op, G);
  if (P > 0 && (!dout_bf16 || !dz_bf16)) return set_error(MOE_ERR_ARG, "%s: dout or dz is NULL", op);
  if (P > 0 && !z_bf16 && (activation != MOE_ACT_NONE || grad_pair_weight))
    return set_error(MOE_ERR_ARG, "%s: an activation or grad_pair_weight needs z", op);
  for (const void* q : {dout_bf16, z_bf16, const_cast<const void*>(dz_bf16), static_cast<const void*>(grad_bias),
                        const_cast<const void*>(workspace)})
    if (q && !aligned16(q))
      return set_error(MOE_ERR_ALIGN, "%s: dout, z, dz, grad_bias and workspace must be 16-byte aligned", op);
  for (const void* q : {static_cast<const void*>(pair_weight), static_cast<const void*>(row_to_pair),
                        static_cast<const void*>(group_offsets), static_cast<const void*>(grad_pair_weight)})
    if (reinterpret_cast<uintptr_t>(q) & 3u)
      return set_error(MOE_ERR_ALIGN, "%s: weights and indices must be 4-byte aligned", op);
  if (P == 0 && !grad_bias) return MOE_OK;
  const int cb = blocks_of(N, kCols);
  const bool rows = grad_pair_weight && cb > 1 && P > 0;   // row sums of several column blocks to join
  const size_t need = (grad_bias && P > 0 ? bias_bytes(P, N, G) : 0) + (rows ? pad(static_cast<size_t>(cb) * P * 4) : 0);
  if (need > 0 && (!workspace || ws_bytes < need))
    return set_error(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes is smaller than the %zu needed", op,
                     workspace ? ws_bytes : 0, need);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  BackParams p{};
  p.dout = static_cast<const uint16_t*>(dout_bf16);
  p.z = static_cast<const uint16_t*>(z_bf16);
  p.activation = activation;
  p.pair_weight = pair_weight;
  p.row_to_pair = row_to_pair;
  p.group_offsets = group_offsets;
  p.P = P; p.N = N; p.G = G;
  p.rows = P > 0 ? blocks_of(P, ranges_of(P, N)) : 1;
  p.dz = static_cast<uint16_t*>(dz_bf16);
  p.part_b = grad_bias ? static_cast<float*>(workspace) : nullptr;
  float* joined = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + (grad_bias ? bias_bytes(P, N, G) : 0));
  p.part_w = rows ? joined : grad_pair_weight;
  p.launches = device_diag().launches;
  if (P > 0) {
    void (*const kernels[])(BackParams) = {
        bias_act_backward_kernel<MOE_ACT_NONE>, bias_act_backward_kernel<MOE_ACT_RELU>,
        bias_act_backward_kernel<MOE_ACT_RELU2>, bias_act_backward_kernel<MOE_ACT_GELU>,
        bias_act_backward_kernel<MOE_ACT_GELU_TANH>, bias_act_backward_kernel<MOE_ACT_SILU>};
    static std::atomic<int> configured[6][64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
      cudaGetLastError();
      dev = -1;
    }
    const bool cache = dev >= 0 && dev < 64;
    if (!cache || !configured[activation][dev].load(std::memory_order_acquire)) {
      if (cudaFuncSetAttribute(kernels[activation], cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes) != cudaSuccess)
        return set_error(MOE_ERR_CUDA, "%s: cannot reserve %d bytes of shared memory: %s", op, kBytes,
                         cudaGetErrorString(cudaGetLastError()));
      if (cache) configured[activation][dev].store(1, std::memory_order_release);
    }
    const int rc = launch_status(launch_kernel(kernels[activation], dim3(blocks_of(P, p.rows), cb), dim3(32 * kWarps), kBytes,
                                               s, nullptr, 0, p),
                                 op);
    if (rc != MOE_OK) return rc;
  }
  if (!grad_bias && !rows) return MOE_OK;
  const int bias_ctas = grad_bias ? blocks_of(N, 256) : 0, row_ctas = rows ? blocks_of(P, 256) : 0;
  return launch_status(launch_kernel(bias_act_reduce_kernel, dim3(G * bias_ctas + row_ctas), dim3(256), 0, s, nullptr, 0, p,
                                     grad_bias, rows ? grad_pair_weight : nullptr, bias_ctas, cb),
                       op);
}
