// route_device.cuh -- device pieces of the router that moe_route.cu and the few-token
// layer (moe_layer_few.cu) share, so that both give the same logits, choice and weights.
#pragma once

#include <stdint.h>

#include "moe_common.cuh"

namespace moe {
namespace route {

constexpr int kMaxGroups = 64;   // n_group limit of the grouped router

// Order-preserving 32-bit key of a logit for the selection: larger key = ranks
// higher.  -0 and +0 share a key (they compare equal), every NaN gets key 0
// (below -inf, whose key is 0x007FFFFF), and equal keys go to the lower expert
// id -- the order "descending value, ties to the lower id, NaN last".
__device__ __forceinline__ uint32_t rank_key(float v) {
  if (v != v) return 0u;
  uint32_t u = __float_as_uint(v);
  if ((u & 0x7FFFFFFFu) == 0u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Does key a (expert ia) rank above key b (expert ib): larger first, ties to
// the lower index, NaN last (the order of rank_key).
__device__ __forceinline__ bool ranks_above(float a, int ia, float b, int ib) {
  const uint32_t ka = rank_key(a), kb = rank_key(b);
  return ka > kb || (ka == kb && ia < ib);
}

// Router logits of small batches on CUDA cores: one warp adds one weight row's
// products with kTokWarp tokens (the first nt of them live).  Lane l owns the
// 8-element chunks l, l + 32, ... of H.  For each block of kChunks chunks the lane
// loads the weights and the tokens' inputs all at once (one memory round trip), and
// adds each token's products into its f32 sum by fused multiply-adds in index order.
// The warp adds its 32 lane sums by a butterfly: every lane returns them.
constexpr int kChunks = 8;     // 16-byte chunks per lane and block: 2048 of H
constexpr int kTokWarp = 2;    // tokens per warp

__device__ __forceinline__ void small_logits(const uint16_t* __restrict__ x,
                                             const uint16_t* __restrict__ wrow, int H, int t0,
                                             int nt, int lane, float (&sum)[kTokWarp]) {
#pragma unroll
  for (int u = 0; u < kTokWarp; ++u) sum[u] = 0.0f;
  for (int hb = 0; hb < H; hb += 256 * kChunks) {
    uint4 w4[kChunks];
    uint4 x4[kTokWarp][kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int h = hb + 256 * c + 8 * lane;
      w4[c] = h < H ? __ldg(reinterpret_cast<const uint4*>(wrow + h)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int u = 0; u < kTokWarp; ++u)
        x4[u][c] = (h < H && u < nt)
                       ? __ldg(reinterpret_cast<const uint4*>(x + static_cast<size_t>(t0 + u) * H + h))
                       : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kTokWarp; ++u)
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const uint32_t xw[4] = {x4[u][c].x, x4[u][c].y, x4[u][c].z, x4[u][c].w};
        const uint32_t ww[4] = {w4[c].x, w4[c].y, w4[c].z, w4[c].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          sum[u] = __fmaf_rn(__uint_as_float(xw[q] << 16), __uint_as_float(ww[q] << 16), sum[u]);
          sum[u] = __fmaf_rn(__uint_as_float(xw[q] & 0xFFFF0000u),
                             __uint_as_float(ww[q] & 0xFFFF0000u), sum[u]);
        }
      }
  }
#pragma unroll
  for (int u = 0; u < kTokWarp; ++u)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], o);
}

}  // namespace route
}  // namespace moe
