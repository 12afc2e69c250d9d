// fp8_common.cuh -- block-scaled E4M3 rows: the scale and code arithmetic that
// the quantiser and the products share, and the products' arguments.
#pragma once

#include <cuda_fp8.h>

#include "gemm_common.cuh"
#include "sm100_ptx_fp8.cuh"

namespace moe {
namespace fp8 {

constexpr int kBlk = 128;   // columns per activation scale, rows and columns per weight scale

__host__ __device__ constexpr int blocks_of(int n) { return (n + kBlk - 1) / kBlk; }

// d and 1 / d of a block whose largest magnitude is amax: every step one binary32
// operation, so codes and scales are the same bits everywhere.  The floor keeps
// 1 / d finite for blocks of zeros and of the smallest subnormals.
__device__ __forceinline__ void block_scale(float amax, float& d, float& id) {
  d = fmaxf(__fdiv_rn(amax, 448.0f), 0x1p-126f);
  id = __frcp_rn(d);
}

// four values as E4M3 codes (nearest even, saturating; NaN stays NaN), lowest first
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// 8 bf16 values of a 16-byte vector
__device__ __forceinline__ void widen8(const uint4& a, float (&v)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// 16 bf16 values of two 16-byte vectors
__device__ __forceinline__ void widen16(const uint4& a, const uint4& b, float (&v)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 codes16(const float (&v)[16], float id) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = codes4(__fmul_rn(v[4 * i], id), __fmul_rn(v[4 * i + 1], id), __fmul_rn(v[4 * i + 2], id),
                  __fmul_rn(v[4 * i + 3], id));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 values, as pairs, times id as E4M3 codes
__device__ __forceinline__ uint4 codes16(const uint64_t (&v)[8], float id) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 lo = ptx::unpair(ptx::mul2(v[2 * i], ptx::pair(id))), hi = ptx::unpair(ptx::mul2(v[2 * i + 1], ptx::pair(id)));
    w[i] = codes4(lo.x, lo.y, hi.x, hi.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// silu(g) u; tolerance-checked: the fast exponential and division serve
__device__ __forceinline__ float silu_mul(float g, float u) {
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

constexpr int kMaxGroupsLaunch = 512;       // groups of one launch of the tiles (schedule in shared memory)

struct GemmParams {
  const uint8_t* a;
  const float* sa;               // [P, blocks(K)]
  const uint8_t* w;              // [G, rows, K]
  const float* sw;               // [G, blocks(rows), blocks(K)]
  const int32_t* group_offsets;  // [G + 1], or null: one group of P rows
  int P, K, N, G;                // N: output columns (I for gate/up)
  const float* pair_weight;
  const int32_t* row_to_pair;
  uint16_t* out;                 // bf16 [P, N]; gate/up: bf16 [P, 2N] or null
  uint8_t* act;                  // gate/up: codes [P, N]
  float* act_scale;              // gate/up: [P, blocks(N)]
  int kid;
};

// the products on the tensor cores (moe_fp8_gemm.cu); gateup: SiLU-mul and
// quantised activations.  Arguments already checked.
int launch_product(const char* op, const GemmParams& p, bool gateup, cudaStream_t stream);

// the same for calls of few dot products (rows times weight rows), where a warp per 4 columns
// reads the weights (moe_fp8_few.cu).  Its time grows with the products, that of the tiles
// with the columns of a row: 7.8 us against 11.5 (12288 products of 2048), 4.6 against 6.9
// (16384 of 768), 9.1 against 13.9 (16384 of 4096); 7.8 against 7.8 (32768 of 768), 8.9
// against 9.4 (32768 of 2048), 17.3 against 14.5 (24576 of 2048 with gate/up).
constexpr int kFewRows = 16, kFewProducts = 16384;
int launch_few(const char* op, const GemmParams& p, bool gateup, cudaStream_t stream);

}  // namespace fp8
}  // namespace moe
