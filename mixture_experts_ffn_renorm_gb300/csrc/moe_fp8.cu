// moe_fp8.cu -- the expert products in 8-bit floating point: activations and
// weights are E4M3 codes with one f32 scale per 128 columns of an activation
// row and per 128 x 128 block of a weight matrix (the block-scaled format that
// the FP8-weight calls of moe.h describe), and the data gradient of those
// products through frozen weights.
//
// For row r of group g and output column n, with K cut into blocks b of 128:
//   y[r,n] = sum_b  sa[r,b] * sw[g,n/128,b] * ( sum_{k in b} a[r,k] * w[g,n,k] )
// The inner sums run on E4M3 values; the scaled joins of the blocks are f32.
#include "fp8_common.cuh"

namespace moe {
namespace fp8 {
namespace {

// ------------------------------------------------------------------ quantiser
// A lane owns 16 consecutive columns of one token, 8 lanes a scale block, so a
// warp covers 512 columns: one 32-byte read per lane, then one 16-byte store per
// lane for each of the token's K destination rows.  Bound by its stores: 8192 tokens
// of 2048 to 8 rows each, 172 MB in all, take 27.7 us (6.2 TB/s).  Without row weights the
// codes are formed once, in 32 registers instead of the 64 of a kernel for both, so twice as
// many warps are resident: 8192 rows of 4096 take 17.6 us instead of 24.0.  With row weights the
// codes are formed anew for each of the K rows: 4096 tokens of 2048 to 8 rows each, 86 MB, take
// 20.1 us (4.3 TB/s), 14.1 without.  A row factor f scales every
// value, and rounding is monotone, so the block's largest magnitude is
// f32(amax(|x|) * |f|): it is reduced over the lanes once, not once per row.
template <bool kWeighted>
__global__ void __launch_bounds__(256)
quant_rows_kernel(const uint16_t* __restrict__ x, int T, int H, int K,
                  const int32_t* __restrict__ pair_to_row, const float* __restrict__ pair_weight,
                  float routed_scale, uint8_t* __restrict__ codes, float* __restrict__ scales,
                  unsigned long long* launches) {
  count_launch(launches, MOE_KID_QUANT_FP8);
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int chunks = (H + 511) / 512;
  const long long item = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  if (item >= static_cast<long long>(T) * chunks) return;
  const int t = static_cast<int>(item / chunks);
  const int col = static_cast<int>(item % chunks) * 512 + lane * 16;
  const bool live = col < H;   // H % 16 == 0
  uint4 a = make_uint4(0, 0, 0, 0), b = a;
  if (live) {
    const uint4* src = reinterpret_cast<const uint4*>(x + static_cast<size_t>(t) * H + col);
    a = __ldg(src);
    b = __ldg(src + 1);
  }
  const uint32_t raw[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint64_t v[8];
  __nv_bfloat162 top = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = ptx::pair(raw[i] << 16, raw[i] & 0xFFFF0000u);
    top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&raw[i])));   // skips NaN
  }
  float amax = fmaxf(__low2float(top), __high2float(top));
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (!live) return;
  const int P = T * K;
  const int nb = blocks_of(H);
  uint4 same = make_uint4(0, 0, 0, 0);
  float same_d = 0.0f;
  if (!kWeighted) {   // one factor for all rows: one set of codes
    uint64_t w[8];
    float id;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = ptx::mul2(v[i], ptx::pair(routed_scale));
    block_scale(__fmul_rn(amax, fabsf(routed_scale)), same_d, id);
    same = codes16(w, id);
  }
  for (int j = 0; j < K; ++j) {
    const int p = t * K + j;
    const int row = pair_to_row ? __ldg(pair_to_row + p) : p;
    if (row < 0 || row >= P) continue;
    uint4 out = same;
    float d = same_d;
    if (kWeighted) {
      const float f = __fmul_rn(__ldg(pair_weight + p), routed_scale);
      uint64_t w[8];
      float id;
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = ptx::mul2(v[i], ptx::pair(f));
      block_scale(__fmul_rn(amax, fabsf(f)), d, id);
      out = codes16(w, id);
    }
    *reinterpret_cast<uint4*>(codes + static_cast<size_t>(row) * H + col) = out;
    if ((lane & 7) == 0) scales[static_cast<size_t>(row) * nb + col / kBlk] = d;
  }
}

// ------------------------------------------------------------------ SiLU-mul backward
// a = silu(g) u with s = sigmoid(g):  dg = da u s (1 + g (1 - s)),  du = da g s.
// The gradient row (dg, then du: 2I columns) is quantised in blocks of 128 of its
// own columns straight from binary32.  Lanes own 16 columns as in the quantiser.
__global__ void __launch_bounds__(256)
silu_mul_backward_kernel(const uint16_t* __restrict__ gu, const uint16_t* __restrict__ dact, int P,
                         int I, uint8_t* __restrict__ codes, float* __restrict__ scales,
                         unsigned long long* launches) {
  count_launch(launches, MOE_KID_SILU_BACKWARD);
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int W = 2 * I;
  const int chunks = (W + 511) / 512;
  const long long item = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  if (item >= static_cast<long long>(P) * chunks) return;
  const size_t r = static_cast<size_t>(item / chunks);
  const int col = static_cast<int>(item % chunks) * 512 + lane * 16;
  const bool live = col < W;
  float v[16];
  float amax = 0.0f;
  if (live) {
    const bool is_up = col >= I;             // I % 16 == 0: a lane's columns are all gate or all up
    const int c = is_up ? col - I : col;
    float g[16], u[16], da[16];
    const uint4* pg = reinterpret_cast<const uint4*>(gu + r * W + c);
    const uint4* pu = reinterpret_cast<const uint4*>(gu + r * W + I + c);
    const uint4* pd = reinterpret_cast<const uint4*>(dact + r * I + c);
    widen16(__ldg(pg), __ldg(pg + 1), g);
    widen16(__ldg(pu), __ldg(pu + 1), u);
    widen16(__ldg(pd), __ldg(pd + 1), da);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float s = __fdividef(1.0f, 1.0f + __expf(-g[i]));
      v[i] = is_up ? da[i] * g[i] * s : da[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
      amax = fmaxf(amax, fabsf(v[i]));
    }
  }
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (!live) return;
  float d, id;
  block_scale(amax, d, id);
  *reinterpret_cast<uint4*>(codes + r * W + col) = codes16(v, id);
  if ((lane & 7) == 0) scales[r * blocks_of(W) + col / kBlk] = d;
}

// The same where I is a multiple of 128: gate and up columns of a feature then lie in
// blocks of the same 128 features, so a lane forms both halves of its 16 features from
// one read of g, u and da and one sigmoid.  Bound by bytes: 203 MB at 32768 rows of
// I = 768, 34.0 us (6.0 TB/s).
__global__ void __launch_bounds__(256)
silu_mul_backward_paired_kernel(const uint16_t* __restrict__ gu, const uint16_t* __restrict__ dact,
                                int P, int I, uint8_t* __restrict__ codes, float* __restrict__ scales,
                                unsigned long long* launches) {
  count_launch(launches, MOE_KID_SILU_BACKWARD);
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int W = 2 * I;
  const int pieces = I / 16;   // a multiple of 8: the 8 lanes of a block stay together
  const long long item = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const bool live = item < static_cast<long long>(P) * pieces;
  const size_t r = static_cast<size_t>(item / pieces);
  const int c = static_cast<int>(item % pieces) * 16;
  float dg[16], du[16], mg = 0.0f, mu = 0.0f;
  if (live) {
    const uint4* pg = reinterpret_cast<const uint4*>(gu + r * W + c);
    const uint4* pu = reinterpret_cast<const uint4*>(gu + r * W + I + c);
    const uint4* pd = reinterpret_cast<const uint4*>(dact + r * I + c);
    const uint4 g0 = __ldg(pg), g1 = __ldg(pg + 1), u0 = __ldg(pu), u1 = __ldg(pu + 1);
    const uint4 d0 = __ldg(pd), d1 = __ldg(pd + 1);
    float g[16], u[16], da[16];
    widen16(g0, g1, g);
    widen16(u0, u1, u);
    widen16(d0, d1, da);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float s = __fdividef(1.0f, 1.0f + __expf(-g[i]));
      dg[i] = da[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
      du[i] = da[i] * g[i] * s;
      mg = fmaxf(mg, fabsf(dg[i]));
      mu = fmaxf(mu, fabsf(du[i]));
    }
  }
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) {
    mg = fmaxf(mg, __shfl_xor_sync(0xffffffffu, mg, o));
    mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, o));
  }
  if (!live) return;
  float d, id;
  block_scale(mg, d, id);
  *reinterpret_cast<uint4*>(codes + r * W + c) = codes16(dg, id);
  if ((lane & 7) == 0) scales[r * (W / kBlk) + c / kBlk] = d;
  block_scale(mu, d, id);
  *reinterpret_cast<uint4*>(codes + r * W + I + c) = codes16(du, id);
  if ((lane & 7) == 0) scales[r * (W / kBlk) + (I + c) / kBlk] = d;
}

// ------------------------------------------------------------------ weight transpose
// 64 x 64 codes per block through shared memory (rows padded to 68 bytes).  A block's codes are
// transposed once, when it is built, so this is short rather than fast: 128 x 1536 x 2048 take
// 272 us (3.0 TB/s).
__global__ void __launch_bounds__(256)
transpose_codes_kernel(const uint8_t* __restrict__ w, const float* __restrict__ scale, int R, int C,
                       uint8_t* __restrict__ out, float* __restrict__ out_scale,
                       unsigned long long* launches) {
  __shared__ __align__(4) uint8_t tile[64][68];   // stored as words
  count_launch(launches, MOE_KID_TRANSPOSE_FP8);
  grid_dep_wait();
  grid_dep_launch();
  const size_t g = blockIdx.z;
  const int c0 = blockIdx.x * 64, r0 = blockIdx.y * 64;
  const int q = threadIdx.x & 15, y = threadIdx.x >> 4;
  for (int i = y; i < 64; i += 16) {
    const int r = r0 + i, c = c0 + 4 * q;
    if (r < R && c < C)   // C % 16 == 0
      *reinterpret_cast<uint32_t*>(&tile[i][4 * q]) =
          __ldg(reinterpret_cast<const uint32_t*>(w + (g * R + r) * C + c));
  }
  __syncthreads();
  for (int i = y; i < 64; i += 16) {
    const int c = c0 + i, r = r0 + 4 * q;
    if (c < C && r < R) {
      const uint32_t v = tile[4 * q][i] | (tile[4 * q + 1][i] << 8) | (tile[4 * q + 2][i] << 16) |
                         (static_cast<uint32_t>(tile[4 * q + 3][i]) << 24);
      *reinterpret_cast<uint32_t*>(out + (g * C + c) * R + r) = v;
    }
  }
  // the scale of a 128 x 128 block, by the block of threads at its first corner
  if (threadIdx.x == 0 && c0 % kBlk == 0 && r0 % kBlk == 0) {
    const int rb = blocks_of(R), cb = blocks_of(C);
    out_scale[(g * cb + c0 / kBlk) * rb + r0 / kBlk] =
        __ldg(scale + (g * rb + r0 / kBlk) * cb + c0 / kBlk);
  }
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// the checks the two products share; K is the contraction length, N the output columns, with
// their names in the call; a group has rows_per_col * N weight rows
int check_product(const char* op, const void* a, const void* sa, const void* w, const void* sw,
                  const void* group_offsets, int P, int K, const char* k_name, int N,
                  const char* n_name, int rows_per_col, int G) {
  if (P < 0) return set_error(MOE_ERR_ARG, "%s: P=%d < 0", op, P);
  if (K <= 0 || N <= 0) return set_error(MOE_ERR_ARG, "%s: dimensions must be positive", op);
  if (G < 1 || G > gemm::kMaxGroups)
    return set_error(MOE_ERR_ARG, "%s: G=%d outside [1, %d]", op, G, gemm::kMaxGroups);
  if (P > kMaxDim) return set_error(MOE_ERR_ARG, "%s: P=%d is too large", op, P);
  if (K > kMaxDim) return set_error(MOE_ERR_ARG, "%s: %s=%d is too large", op, k_name, K);
  if (N > kMaxDim / rows_per_col) return set_error(MOE_ERR_ARG, "%s: %s=%d is too large", op, n_name, N);
  const long long rows = static_cast<long long>(G < kMaxGroupsLaunch ? G : kMaxGroupsLaunch) * rows_per_col * N;
  if (rows > kMaxDim) return set_error(MOE_ERR_ARG, "%s: %lld weight rows are too large a number", op, rows);
  if (P == 0) return MOE_OK;
  if (!a || !sa || !w || !sw) return set_error(MOE_ERR_ARG, "%s: NULL operand or scales", op);
  if (!group_offsets && G > 1)
    return set_error(MOE_ERR_ARG, "%s: group_offsets is NULL with G=%d", op, G);
  if (!aligned16(a) || !aligned16(w))
    return set_error(MOE_ERR_ALIGN, "%s: codes must be 16-byte aligned", op);
  if (!aligned4(sa) || !aligned4(sw) || !aligned4(group_offsets))
    return set_error(MOE_ERR_ALIGN, "%s: scales and group_offsets must be 4-byte aligned", op);
  return MOE_OK;
}

}  // namespace
}  // namespace fp8
}  // namespace moe

using namespace moe;
using namespace moe::fp8;

extern "C" {

int moe_quantize_act_fp8(const void* x_bf16, int T, int H, int K, const int32_t* pair_to_row,
                         const float* pair_weight, float routed_scale, uint8_t* codes,
                         float* scales, void* stream) {
  clear_error();
  const char* op = "moe_quantize_act_fp8";
  if (T < 0 || H <= 0) return set_error(MOE_ERR_ARG, "%s: bad sizes T=%d H=%d", op, T, H);
  if (K < 1 || K > 64) return set_error(MOE_ERR_ARG, "%s: K=%d outside [1, 64]", op, K);
  if (H > kMaxDim) return set_error(MOE_ERR_ARG, "%s: H=%d is too large", op, H);
  if (static_cast<long long>(T) * K > 0x7FFFFFFFLL)
    return set_error(MOE_ERR_ARG, "%s: T*K is too large", op);
  if (H % 16 != 0) return set_error(MOE_ERR_ALIGN, "%s: H=%d is not a multiple of 16", op, H);
  if (T == 0) return MOE_OK;
  if (!x_bf16 || !codes || !scales) return set_error(MOE_ERR_ARG, "%s: NULL operand", op);
  if (!aligned16(x_bf16) || !aligned16(codes))
    return set_error(MOE_ERR_ALIGN, "%s: x and codes must be 16-byte aligned", op);
  if (!aligned4(scales) || !aligned4(pair_to_row) || !aligned4(pair_weight))
    return set_error(MOE_ERR_ALIGN, "%s: scales, pair_to_row and pair_weight must be 4-byte aligned",
                     op);
  const long long warps = static_cast<long long>(T) * ((H + 511) / 512);
  const long long blocks = (warps + 7) / 8;
  if (blocks > 0x7FFFFFFFLL) return set_error(MOE_ERR_ARG, "%s: T*H is too large", op);
  return launch_status(
      launch_kernel(pair_weight ? quant_rows_kernel<true> : quant_rows_kernel<false>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                    static_cast<cudaStream_t>(stream), nullptr, 0,
                    static_cast<const uint16_t*>(x_bf16), T, H, K, pair_to_row, pair_weight,
                    routed_scale, codes, scales, device_diag().launches),
      op);
}

int moe_grouped_gemm_fp8(const uint8_t* a_codes, const float* a_scales, const uint8_t* w_e4m3,
                         const float* w_scale, const int32_t* group_offsets,
                         const float* pair_weight, const int32_t* row_to_pair, int P, int K, int N,
                         int G, void* out_bf16, void* stream) {
  clear_error();
  const char* op = "moe_grouped_gemm_fp8";
  int rc = check_product(op, a_codes, a_scales, w_e4m3, w_scale, group_offsets, P, K, "K", N, "N",
                         1, G);
  if (rc != MOE_OK) return rc;
  if (K % 16 != 0 || N % 8 != 0)
    return set_error(MOE_ERR_ALIGN, "%s: K=%d must be a multiple of 16 and N=%d of 8", op, K, N);
  if (P == 0) return MOE_OK;
  if (!out_bf16) return set_error(MOE_ERR_ARG, "%s: NULL out", op);
  if (!aligned16(out_bf16)) return set_error(MOE_ERR_ALIGN, "%s: out must be 16-byte aligned", op);
  if (!aligned4(pair_weight) || !aligned4(row_to_pair))
    return set_error(MOE_ERR_ALIGN, "%s: pair_weight and row_to_pair must be 4-byte aligned", op);
  GemmParams p{};
  p.a = a_codes;
  p.sa = a_scales;
  p.w = w_e4m3;
  p.sw = w_scale;
  p.group_offsets = group_offsets;
  p.P = P;
  p.K = K;
  p.N = N;
  p.G = G;
  p.pair_weight = pair_weight;
  p.row_to_pair = row_to_pair;
  p.out = static_cast<uint16_t*>(out_bf16);
  p.kid = MOE_KID_GEMM_FP8;
  return launch_product(op, p, false, static_cast<cudaStream_t>(stream));
}

int moe_grouped_gemm_gateup_silu_fp8(const uint8_t* a_codes, const float* a_scales,
                                     const uint8_t* w13_e4m3, const float* w13_scale,
                                     const int32_t* group_offsets, int P, int H, int I, int G,
                                     void* gate_up_bf16, uint8_t* act_codes, float* act_scales,
                                     void* stream) {
  clear_error();
  const char* op = "moe_grouped_gemm_gateup_silu_fp8";
  int rc = check_product(op, a_codes, a_scales, w13_e4m3, w13_scale, group_offsets, P, H, "H", I,
                         "I", 2, G);
  if (rc != MOE_OK) return rc;
  if (H % 16 != 0 || I % 16 != 0)
    return set_error(MOE_ERR_ALIGN, "%s: H=%d and I=%d must be multiples of 16", op, H, I);
  if (P == 0) return MOE_OK;
  if (!act_codes || !act_scales) return set_error(MOE_ERR_ARG, "%s: NULL act_codes or act_scales", op);
  if (!aligned16(act_codes) || !aligned16(gate_up_bf16) || !aligned4(act_scales))
    return set_error(MOE_ERR_ALIGN,
                     "%s: act_codes and gate_up must be 16-byte aligned, act_scales 4-byte", op);
  GemmParams p{};
  p.a = a_codes;
  p.sa = a_scales;
  p.w = w13_e4m3;
  p.sw = w13_scale;
  p.group_offsets = group_offsets;
  p.P = P;
  p.K = H;
  p.N = I;
  p.G = G;
  p.out = static_cast<uint16_t*>(gate_up_bf16);
  p.act = act_codes;
  p.act_scale = act_scales;
  p.kid = MOE_KID_GEMM_FP8_GATEUP;
  return launch_product(op, p, true, static_cast<cudaStream_t>(stream));
}

int moe_silu_mul_backward_fp8(const void* gate_up_bf16, const void* dact_bf16, int P, int I,
                              uint8_t* codes, float* scales, void* stream) {
  clear_error();
  const char* op = "moe_silu_mul_backward_fp8";
  if (P < 0 || I <= 0) return set_error(MOE_ERR_ARG, "%s: bad sizes P=%d I=%d", op, P, I);
  if (I > kMaxDim / 2) return set_error(MOE_ERR_ARG, "%s: I=%d is too large", op, I);
  if (I % 16 != 0) return set_error(MOE_ERR_ALIGN, "%s: I=%d is not a multiple of 16", op, I);
  if (P == 0) return MOE_OK;
  if (!gate_up_bf16 || !dact_bf16 || !codes || !scales)
    return set_error(MOE_ERR_ARG, "%s: NULL operand", op);
  if (!aligned16(gate_up_bf16) || !aligned16(dact_bf16) || !aligned16(codes) || !aligned4(scales))
    return set_error(MOE_ERR_ALIGN,
                     "%s: gate_up, dact and codes must be 16-byte aligned, scales 4-byte", op);
  const bool paired = I % kBlk == 0;   // I = 768, 32768 rows: 45.3 us unpaired, 34.0 paired
  const long long threads = static_cast<long long>(P) * (paired ? I / 16 : (2 * I + 511) / 512 * 32);
  const long long blocks = (threads + 255) / 256;
  if (blocks > 0x7FFFFFFFLL) return set_error(MOE_ERR_ARG, "%s: P*I is too large", op);
  return launch_status(
      launch_kernel(paired ? silu_mul_backward_paired_kernel : silu_mul_backward_kernel,
                    dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                    static_cast<cudaStream_t>(stream), nullptr, 0,
                    static_cast<const uint16_t*>(gate_up_bf16),
                    static_cast<const uint16_t*>(dact_bf16), P, I, codes, scales,
                    device_diag().launches),
      op);
}

int moe_transpose_fp8w(const uint8_t* w_e4m3, const float* w_scale, int G, int R, int C,
                       uint8_t* out_e4m3, float* out_scale, void* stream) {
  clear_error();
  const char* op = "moe_transpose_fp8w";
  if (G < 1 || G > gemm::kMaxGroups)
    return set_error(MOE_ERR_ARG, "%s: G=%d outside [1, %d]", op, G, gemm::kMaxGroups);
  if (R <= 0 || C <= 0) return set_error(MOE_ERR_ARG, "%s: bad sizes R=%d C=%d", op, R, C);
  if (R % 16 != 0 || C % 16 != 0)
    return set_error(MOE_ERR_ALIGN, "%s: R=%d and C=%d must be multiples of 16", op, R, C);
  if (R > 64 * 65535) return set_error(MOE_ERR_ARG, "%s: R=%d is too large", op, R);   // the grid's y
  if (C > kMaxDim) return set_error(MOE_ERR_ARG, "%s: C=%d is too large", op, C);
  if (!w_e4m3 || !w_scale || !out_e4m3 || !out_scale)
    return set_error(MOE_ERR_ARG, "%s: NULL operand", op);
  if (!aligned16(w_e4m3) || !aligned16(out_e4m3) || !aligned4(w_scale) || !aligned4(out_scale))
    return set_error(MOE_ERR_ALIGN, "%s: codes must be 16-byte aligned, scales 4-byte", op);
  return launch_status(
      launch_kernel(transpose_codes_kernel,
                    dim3(static_cast<unsigned>((C + 63) / 64), static_cast<unsigned>((R + 63) / 64),
                         static_cast<unsigned>(G)),
                    dim3(256), 0, static_cast<cudaStream_t>(stream), nullptr, 0, w_e4m3, w_scale, R,
                    C, out_e4m3, out_scale, device_diag().launches),
      op);
}

}  // extern "C"
