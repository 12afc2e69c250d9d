// moe_backward.cu -- gradients of the combine and of the router.
//
// Combine, out[t,:] = rs sum_k w[t,k] eo[t,k,:]:
//   dw[t,k] = rs <eo[t,k,:], dout[t,:]>,   deo[t,k,:] = (rs w[t,k]) dout[t,:]
// Router weights to logits: see moe.h (moe_route_backward).  The products behind
// the logits are in moe_route_grad.cu.
#include "moe_common.cuh"

namespace moe {
namespace bwd {
namespace {

// 8 consecutive values of a row as they lie in memory, and widened
template <bool kBf16>
struct Raw8 {
  uint4 a[kBf16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* base, size_t i) {
    const uint4* p = reinterpret_cast<const uint4*>(
        kBf16 ? static_cast<const void*>(static_cast<const uint16_t*>(base) + i)
              : static_cast<const void*>(static_cast<const float*>(base) + i));
#pragma unroll
    for (int j = 0; j < (kBf16 ? 1 : 2); ++j) a[j] = __ldg(p + j);
  }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    if (kBf16) {
      const uint32_t w[4] = {a[0].x, a[0].y, a[0].z, a[0].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    } else {
      const uint4 b = a[kBf16 ? 0 : 1];
      const uint32_t w[8] = {a[0].x, a[0].y, a[0].z, a[0].w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
    }
  }
};
template <bool kBf16>
__device__ __forceinline__ void store8(void* base, size_t i, const float (&v)[8]) {
  if (kBf16) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// ------------------------------------------------------------------ combine
// A block takes one token and up to 8 of its expert rows; a thread owns 8 channels
// (and strides over the rest), so dout is read once and the rows' loads are all in
// flight together.  Bound by bytes: 285 MB at 4096 tokens of 8 bf16 rows of 2048 with
// both gradients, 42 us at the copy rate; it takes 45.8.
constexpr int kCbThreads = 256;
constexpr int kCbRows = 8;

template <bool kEoBf16, bool kDoBf16, bool kDeoBf16>
__global__ void __launch_bounds__(kCbThreads)
combine_backward_kernel(const void* __restrict__ eo, const float* __restrict__ w,
                        const void* __restrict__ dout, float rs, int K, int H,
                        float* __restrict__ dw, void* __restrict__ deo,
                        unsigned long long* launches) {
  __shared__ float red[kCbThreads / 32][kCbRows];
  count_launch(launches, MOE_KID_COMBINE_BACKWARD);
  grid_dep_wait();
  grid_dep_launch();
  const int kc = (K + kCbRows - 1) / kCbRows;
  const size_t t = blockIdx.x / kc;
  const int k0 = static_cast<int>(blockIdx.x % kc) * kCbRows;
  const int kn = min(kCbRows, K - k0);
  float acc[kCbRows], f[kCbRows];
#pragma unroll
  for (int j = 0; j < kCbRows; ++j) {
    acc[j] = 0.0f;
    f[j] = w && j < kn ? __fmul_rn(__ldg(w + t * K + k0 + j), rs) : rs;
  }
  for (int c = threadIdx.x * 8; c < H; c += kCbThreads * 8) {
    Raw8<kDoBf16> rd;
    rd.load(dout, t * H + c);
    float d[8];
    if (dw) {
      Raw8<kEoBf16> re[kCbRows];
#pragma unroll
      for (int j = 0; j < kCbRows; ++j) re[j].load(eo, (t * K + k0 + min(j, kn - 1)) * H + c);
      rd.widen(d);
#pragma unroll
      for (int j = 0; j < kCbRows; ++j) {
        float e[8];
        re[j].widen(e);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j] = fmaf(e[i], d[i], acc[j]);
      }
    } else {
      rd.widen(d);
    }
    if (deo) {
#pragma unroll
      for (int j = 0; j < kCbRows; ++j) {
        if (j < kn) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = __fmul_rn(d[i], f[j]);
          store8<kDeoBf16>(deo, (t * K + k0 + j) * H + c, o);
        }
      }
    }
  }
  if (!dw) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < kCbRows; ++j) {
    acc[j] = warp_sum(acc[j]);
    if (lane == 0) red[warp][j] = acc[j];
  }
  __syncthreads();
  if (threadIdx.x < kn) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kCbThreads / 32; ++i) s += red[i][threadIdx.x];
    dw[t * K + k0 + threadIdx.x] = __fmul_rn(s, rs);
  }
}

// ------------------------------------------------------------------ router: logits
constexpr int kRtWarps = 8;   // tokens per block

int route_blocks(int T) { return T / kRtWarps + (T % kRtWarps != 0); }

struct RouteParams {
  const float* logits;
  const int32_t* ids;
  const float* grad_w;
  const int32_t* offsets;
  int T, E, K, renormalize, scoring;
  float balance, z;           // coefficients; the balance term needs offsets
  float* dl;
  float* partial;             // [blocks, 2] sums of q and lse^2 over a block's tokens, or null
  float* losses;              // [2] or null
  unsigned int* status;
  unsigned long long* launches;
};

// s = sigmoid(l) and its slope s (1 - s).  Through exp(-|l|) <= 1, so that neither
// 1 - s near 1 nor a large exponential costs the slope its leading bits.
__device__ __forceinline__ float sigmoid_slope(float l, float& slope) {
  const float e = expf(-fabsf(l));
  const float r = 1.0f / (1.0f + e);
  slope = e * r * r;
  return l >= 0.0f ? r : e * r;
}

// One warp per token; lane i holds the logits of experts i, i + 32, ... in registers, so
// a row is read once and every exponential is taken once.  The chosen experts' terms are
// added in the registers of the lanes that hold them.  8.4 MB at 8192
// tokens and 128 experts take 9.6 us with the losses' launch, bound by issue (55 % active)
// and the latency of the two launches.
template <int kPer>
__global__ void __launch_bounds__(32 * kRtWarps)
route_backward_kernel(const RouteParams p) {
  __shared__ float red[kRtWarps][2];
  count_launch(p.launches, MOE_KID_ROUTE_BACKWARD);
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRtWarps + warp;
  const bool aux = p.balance != 0.0f || p.z != 0.0f;
  float tok_q = 0.0f, tok_z = 0.0f;
  if (t < p.T) {
    const float* row = p.logits + static_cast<size_t>(t) * p.E;
    const float inv_t = 1.0f / static_cast<float>(p.T);
    float l[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) l[i] = lane + 32 * i < p.E ? __ldg(row + lane + 32 * i) : -INFINITY;
    // the chosen experts: lane j holds rank j (K <= 32)
    int id = -1;
    float lj = -INFINITY, gj = 0.0f;
    if (lane < p.K) {
      id = __ldg(p.ids + static_cast<size_t>(t) * p.K + lane);
      if (id < 0 || id >= p.E) {
        if (p.status) atomicOr(p.status, static_cast<unsigned int>(MOE_STATUS_BAD_ID));
        id = -1;
      } else {
        lj = __ldg(row + id);
        if (p.grad_w) gj = __ldg(p.grad_w + static_cast<size_t>(t) * p.K + lane);
      }
    }
    const bool sel = id >= 0;
    const bool dense = aux || (p.scoring == 0 && !p.renormalize);
    // the row's softmax, where it enters
    float pe[kPer], sum = 0.0f, lse = 0.0f, base = 0.0f;
    if (dense) {
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < kPer; ++i) top = fmaxf(top, l[i]);
      top = warp_max(top);
      base = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        pe[i] = lane + 32 * i < p.E ? expf(l[i] - base) : 0.0f;
        sum += pe[i];
      }
      sum = warp_sum(sum);
      lse = base + logf(sum);
    }
    const bool empty = dense && sum == 0.0f;     // every logit is -inf: no gradient
    const float inv_sum = dense && !empty ? 1.0f / sum : 0.0f;
    // the gradient at the chosen experts
    float add = 0.0f, dot = 0.0f;
    if (p.scoring == 0 && p.renormalize) {
      float m = warp_max(sel ? lj : -INFINITY);
      if (m == -INFINITY) m = 0.0f;
      const float e = sel ? expf(lj - m) : 0.0f;
      const float S = warp_sum(e);
      const float w = S > 0.0f || S != S ? e / S : 0.0f;
      add = w * (gj - warp_sum(gj * w));
    } else if (p.scoring == 0) {
      const float w = sel ? expf(lj - base) * inv_sum : 0.0f;
      dot = warp_sum(gj * w);
      add = w * gj;
    } else {
      float slope = 0.0f;
      float s = sigmoid_slope(lj, slope);
      if (!sel) s = slope = 0.0f;
      float gs = gj;
      if (p.renormalize) {
        const float S = warp_sum(s);
        gs = S == 0.0f ? 0.0f : (gj - warp_sum(gj * (s / S))) / S;
      }
      add = gs * slope;
    }
    // the balance term's load share q
    const bool bal = p.balance != 0.0f && !empty;
    float f[kPer], slope[kPer], q = 0.0f, S_all = 0.0f;
    if (bal) {
      const float fscale = static_cast<float>(p.E) / (static_cast<float>(p.K) * static_cast<float>(p.T));
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        f[i] = e < p.E ? static_cast<float>(__ldg(p.offsets + e + 1) - __ldg(p.offsets + e)) * fscale : 0.0f;
        float share = e < p.E ? pe[i] : 0.0f;
        slope[i] = 0.0f;
        if (p.scoring && e < p.E) share = sigmoid_slope(l[i], slope[i]);
        q += f[i] * share;
        S_all += share;
      }
      q = warp_sum(q);
      S_all = warp_sum(S_all);
      q = S_all == 0.0f ? 0.0f : q / S_all;
    }
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      v[i] = 0.0f;
      if (dense && !empty) {
        const float pi = pe[i] * inv_sum;
        if (p.scoring == 0 && !p.renormalize) v[i] -= pi * dot;
        if (bal && S_all != 0.0f)
          v[i] += p.scoring ? p.balance * inv_t * (f[i] - q) / S_all * slope[i] : p.balance * inv_t * pi * (f[i] - q);
        if (p.z != 0.0f) v[i] += 2.0f * p.z * inv_t * lse * pi;
      }
    }
    for (int j = 0; j < p.K; ++j) {
      const int ej = __shfl_sync(0xffffffffu, id, j);
      const float aj = __shfl_sync(0xffffffffu, add, j);
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (lane + 32 * i == ej) v[i] += aj;
    }
    float* dl = p.dl + static_cast<size_t>(t) * p.E;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < p.E) dl[lane + 32 * i] = v[i];
    tok_q = q;
    tok_z = empty || p.z == 0.0f ? 0.0f : lse * lse;
  }
  if (p.partial) {
    if (lane == 0) {
      red[warp][0] = tok_q;
      red[warp][1] = tok_z;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
      float s = 0.0f;
      for (int i = 0; i < kRtWarps; ++i) s += red[i][threadIdx.x];
      p.partial[2 * static_cast<size_t>(blockIdx.x) + threadIdx.x] = s;
    }
  } else if (p.losses && blockIdx.x == 0 && threadIdx.x < 2) {
    p.losses[threadIdx.x] = 0.0f;   // no auxiliary loss
  }
}

// the blocks' partial sums in a fixed order
__global__ void __launch_bounds__(256)
route_losses_kernel(const float* __restrict__ partial, int n, float balance, float z,
                    float* __restrict__ losses, unsigned long long* launches) {
  __shared__ float red[8][2];
  count_launch(launches, MOE_KID_ROUTE_LOSSES);
  grid_dep_wait();
  grid_dep_launch();
  float a = 0.0f, b = 0.0f;
  for (int i = threadIdx.x; i < n; i += 256) {
    a += partial[2 * i];
    b += partial[2 * i + 1];
  }
  a = warp_sum(a);
  b = warp_sum(b);
  if ((threadIdx.x & 31) == 0) {
    red[threadIdx.x >> 5][0] = a;
    red[threadIdx.x >> 5][1] = b;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    float s = 0.0f;
    for (int i = 0; i < 8; ++i) s += red[i][threadIdx.x];
    losses[threadIdx.x] = s * (threadIdx.x ? z : balance);
  }
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_dtype(const char* op, const char* what, int dt) {
  if (dt == MOE_F32 || dt == MOE_BF16) return MOE_OK;
  return set_error(MOE_ERR_DTYPE, "%s: %s dtype %s is not supported (f32 or bf16)", op, what,
                   dt == MOE_F16 ? "f16" : "unknown");
}

}  // namespace
}  // namespace bwd
}  // namespace moe

using namespace moe;
using namespace moe::bwd;

extern "C" {

int moe_combine_backward(const void* expert_out, int eo_dtype, const float* w, const void* dout,
                         int do_dtype, float routed_scale, int T, int K, int H, float* dw,
                         void* d_expert_out, int deo_dtype, void* stream) {
  clear_error();
  const char* op = "moe_combine_backward";
  int rc;
  if ((rc = check_dtype(op, "expert_out", eo_dtype)) != MOE_OK) return rc;
  if ((rc = check_dtype(op, "dout", do_dtype)) != MOE_OK) return rc;
  if ((rc = check_dtype(op, "d_expert_out", deo_dtype)) != MOE_OK) return rc;
  if (T < 0 || H <= 0) return set_error(MOE_ERR_ARG, "%s: bad sizes T=%d H=%d", op, T, H);
  if (K < 1 || K > 64) return set_error(MOE_ERR_ARG, "%s: K=%d outside [1, 64]", op, K);
  if (H % 8 != 0) return set_error(MOE_ERR_ALIGN, "%s: H=%d is not a multiple of 8", op, H);
  if (H > kMaxDim) return set_error(MOE_ERR_ARG, "%s: H=%d is too large", op, H);
  if (!dw && !d_expert_out) return set_error(MOE_ERR_ARG, "%s: no output requested", op);
  if (T == 0) return MOE_OK;
  if (!dout || (dw && !expert_out)) return set_error(MOE_ERR_ARG, "%s: NULL operand", op);
  if (!aligned16(expert_out) || !aligned16(dout) || !aligned16(d_expert_out))
    return set_error(MOE_ERR_ALIGN, "%s: expert_out, dout and d_expert_out must be 16-byte aligned",
                     op);
  if (!aligned4(w) || !aligned4(dw)) return set_error(MOE_ERR_ALIGN, "%s: w and dw must be 4-byte aligned", op);
  const long long blocks = static_cast<long long>(T) * ((K + kCbRows - 1) / kCbRows);
  if (blocks > 0x7FFFFFFFLL) return set_error(MOE_ERR_ARG, "%s: T*K is too large", op);
  auto go = [&](auto kern) {
    return launch_status(launch_kernel(kern, dim3(static_cast<unsigned>(blocks)), dim3(kCbThreads), 0,
                                       static_cast<cudaStream_t>(stream), nullptr, 0, expert_out, w,
                                       dout, routed_scale, K, H, dw, d_expert_out,
                                       device_diag().launches),
                         op);
  };
  const int arm = (eo_dtype == MOE_BF16 ? 4 : 0) | (do_dtype == MOE_BF16 ? 2 : 0) |
                  (deo_dtype == MOE_BF16 ? 1 : 0);
  switch (arm) {
    case 0: return go(combine_backward_kernel<false, false, false>);
    case 1: return go(combine_backward_kernel<false, false, true>);
    case 2: return go(combine_backward_kernel<false, true, false>);
    case 3: return go(combine_backward_kernel<false, true, true>);
    case 4: return go(combine_backward_kernel<true, false, false>);
    case 5: return go(combine_backward_kernel<true, false, true>);
    case 6: return go(combine_backward_kernel<true, true, false>);
    default: return go(combine_backward_kernel<true, true, true>);
  }
}

size_t moe_route_backward_workspace_size(int T, int E) {
  if (T <= 0 || E <= 0) return 0;
  return static_cast<size_t>(route_blocks(T)) * 2 * sizeof(float);
}

int moe_route_backward(const float* logits, const int32_t* topk_ids, const float* grad_w,
                       const int32_t* expert_offsets, int T, int E, int K, int renormalize,
                       int scoring, float balance_coef, float z_coef, float* grad_logits,
                       float* losses, void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  const char* op = "moe_route_backward";
  if (scoring != 0 && scoring != 1)
    return set_error(MOE_ERR_UNSUPPORTED, "%s: scoring=%d (0 softmax, 1 sigmoid)", op, scoring);
  if (T < 0) return set_error(MOE_ERR_ARG, "%s: T=%d < 0", op, T);
  if (E < 1 || E > 1024) return set_error(MOE_ERR_ARG, "%s: E=%d outside [1, 1024]", op, E);
  if (K < 1 || K > 32 || K > E) return set_error(MOE_ERR_ARG, "%s: K=%d outside [1, min(E, 32)]", op, K);
  if (renormalize != 0 && renormalize != 1)
    return set_error(MOE_ERR_ARG, "%s: renormalize must be 0 or 1", op);
  if (balance_coef != 0.0f && !expert_offsets)
    return set_error(MOE_ERR_ARG, "%s: the balance loss needs expert_offsets", op);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (losses && cudaMemsetAsync(losses, 0, 2 * sizeof(float), s) != cudaSuccess)
      return check_launch(op);
    return MOE_OK;
  }
  if (!logits || !topk_ids || !grad_logits) return set_error(MOE_ERR_ARG, "%s: NULL operand", op);
  if (!aligned4(logits) || !aligned4(topk_ids) || !aligned4(grad_w) || !aligned4(expert_offsets) ||
      !aligned4(grad_logits) || !aligned4(losses))
    return set_error(MOE_ERR_ALIGN, "%s: operands must be 4-byte aligned", op);
  if (losses) {
    if (!workspace || ws_bytes < moe_route_backward_workspace_size(T, E))
      return set_error(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", op, ws_bytes,
                       moe_route_backward_workspace_size(T, E));
    if (!aligned16(workspace)) return set_error(MOE_ERR_ALIGN, "%s: workspace must be 16-byte aligned", op);
  }
  DeviceDiag diag = device_diag();
  const bool sum_losses = losses && (balance_coef != 0.0f || z_coef != 0.0f);
  RouteParams p{logits, topk_ids, grad_w, expert_offsets, T, E, K, renormalize, scoring, balance_coef,
                z_coef, grad_logits, sum_losses ? static_cast<float*>(workspace) : nullptr, losses,
                diag.status, diag.launches};
  const int blocks = route_blocks(T);
  auto go = [&](auto kern) {
    return launch_status(launch_kernel(kern, dim3(blocks), dim3(32 * kRtWarps), 0, s, nullptr, 0, p), op);
  };
  int rc;
  if (E <= 64) rc = go(route_backward_kernel<2>);
  else if (E <= 128) rc = go(route_backward_kernel<4>);
  else if (E <= 256) rc = go(route_backward_kernel<8>);
  else if (E <= 512) rc = go(route_backward_kernel<16>);
  else rc = go(route_backward_kernel<32>);
  if (rc != MOE_OK || !sum_losses) return rc;
  const float inv_t = 1.0f / static_cast<float>(T);
  return launch_status(launch_kernel(route_losses_kernel, dim3(1), dim3(256), 0, s, nullptr, 0,
                                     static_cast<const float*>(workspace), blocks,
                                     balance_coef * inv_t, z_coef * inv_t, losses, diag.launches),
                       op);
}

}  // extern "C"
