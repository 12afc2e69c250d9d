// moe_layer_few.cu -- a whole MoE layer for a few tokens (decode) in one kernel.
//
// For T <= 16 tokens every expert that a token chooses is read once and used for one or two
// rows, so the layer is a read of weights: 3 H I values per touched expert against two
// operations a value and token.  What bounds it is HBM, and around it the latencies that the
// separate launches of the layer expose one by one: each launch drains before the next one's
// first load.  Here one persistent CTA per SM keeps a ring of bulk copies in flight from the
// choice of experts to the last row, and no phase waits for an empty memory system:
//
//   logits    a warp per (expert, two tokens), as in the router's small batches; grid barrier
//   choice    every CTA selects the experts of all tokens (the router's order and bits) and
//             groups the T K pairs by expert
//   gate/up   the features of the touched experts, in one line, cut evenly over the CTAs:
//             act[p, n] = silu(gate) up in f32 to the workspace; grid barrier
//   down      a CTA owns H / CTAs output columns for all experts: it sums routed_scale w y
//             over a token's experts in shared memory, so no partial sums cross CTAs
//
// The barrier between gate/up and down costs no bandwidth: the producer thread runs ahead of it
// and fills the ring with the down rows, which do not depend on it.
//
// A chunk of the ring holds whole weight rows.  A consumer group of eight warps takes every
// second chunk; a warp takes 8 rows x 256 columns (a lane 8 columns), keeps the tokens' 8
// columns in registers, and sums 8 rows x up to 4 tokens over its lanes by a transposing
// butterfly; the segments of a row are then added in order through shared memory.  All sums
// are f32 in a fixed order, nothing between the weights and the output is narrowed, and no
// atomics touch data.  CUDA cores suffice: a touched expert has 1.5 tokens on average at T = 16,
// and with f32 activations a tensor-core product would need them split into bf16 parts.
#include <atomic>

#include "fp8_common.cuh"
#include "route_device.cuh"

namespace moe {
namespace few {
namespace {

constexpr int kMaxT = 16;          // tokens: one warp of a group per token in the choice
constexpr int kMaxDim = 8192;      // H, I, I_shared: a gate and an up row fit a ring slot
constexpr int kMaxE = 1024;
constexpr int kMaxPairs = kMaxT * 32;
constexpr int kGroupWarps = 8;     // warps of a consumer group
constexpr int kConsumers = 2 * 32 * kGroupWarps;
constexpr int kThreads = kConsumers + 32;
constexpr int kSeg = 256;          // columns of a segment: 8 per lane
constexpr int kMaxSlots = 16;
constexpr int kItems = 32;         // items (8 rows x a segment) of a chunk, at most
constexpr int kMaxRows = 64;       // rows of a chunk, at most
constexpr int kBarAll = 1, kBarGroup = 2;   // named barriers: both groups; one group (+ its index)

static_assert(kMaxDim / kSeg == kItems, "eight rows of any width are a chunk");

struct Params {
  const uint16_t* x;
  const uint16_t* w_router;
  const float* logit_bias;
  const float* select_bias;
  const void* w13;                 // bf16 or E4M3 codes
  const float* s13;                // scales of 128 x 128 blocks (FP8)
  const void* w2;
  const float* s2;
  const uint16_t* w_gate;          // shared expert's gate, or null: ungated
  const uint16_t* w13s;
  const uint16_t* w2s;
  const uint16_t* residual;
  int T, H, I, E, K, Is;
  int renormalize, scoring, n_group, topk_group, group_score;
  float routed_scale;
  int32_t* ids;                    // outputs, or null
  float* w;
  uint16_t* out;
  unsigned int* barrier;           // [0] arrivals, [1] generation
  float* logits;                   // [T, E]
  float* gate;                     // [T]
  float* act;                      // [T K, I]
  float* act_s;                    // [T, Is]
  int slot_bytes, n_slots, rows_max;
  unsigned long long wait_ns;
  unsigned int* status;
  unsigned long long* launches;
};

// Shared memory: the fixed part, then the output sums, then the ring (which first holds the
// choice's scores)
struct alignas(16) Fixed {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  float red[2][2][kItems * 8 * 4]; // [group][buffer][item][row of 8][token of 4]
  float weight[kMaxPairs];         // routing weight of a pair, times routed_scale
  float gate[kMaxT];               // sigmoid of the shared expert's gate
  uint32_t mask[kMaxE];            // tokens that chose an expert
  uint16_t pair[kMaxPairs + kMaxT];    // pairs by expert; then the shared expert's tokens
  uint16_t token[kMaxPairs + kMaxT];   // their tokens
  int16_t expert[kMaxPairs + 1];   // touched experts, ascending
  int16_t first[kMaxPairs + 3];    // their first pair
  int16_t slot[kMaxT][32];         // chosen experts of a token, by rank
  int n_groups;                    // touched experts, without the shared one
  int abort_flag;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Bounded wait; false, at once, when this CTA has given up.  Callers go on either way: every
// loop is finite, so a CTA that gave up runs to its end without waiting again.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                     const Params& p) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (ptx::globaltimer_ns() - t0 > p.wait_ns) {
      if (p.status) atomicOr(p.status, static_cast<unsigned int>(MOE_STATUS_TIMEOUT));
      *abort_flag = 1;
      return false;
    }
  }
}

// One thread's part of the grid barrier: the last CTA to arrive resets the count and starts the
// next generation.  Every CTA arrives exactly once per barrier, also one that has given up.
__device__ __forceinline__ void grid_barrier(volatile int* abort_flag, const Params& p) {
  const uint32_t gen = *reinterpret_cast<volatile uint32_t*>(p.barrier + 1);
  __threadfence();
  if (atomicAdd(p.barrier, 1u) == gridDim.x - 1) {
    atomicSub(p.barrier, gridDim.x);   // not a store: a CTA that gave up may arrive again at any time
    __threadfence();
    ptx::st_release_gpu_u32(p.barrier + 1, gen + 1u);
    return;
  }
  const uint64_t t0 = ptx::globaltimer_ns();
  while (ptx::ld_acquire_gpu_u32(p.barrier + 1) == gen) {
    if (*abort_flag) return;
    if (ptx::globaltimer_ns() - t0 > p.wait_ns) {
      if (p.status) atomicOr(p.status, static_cast<unsigned int>(MOE_STATUS_TIMEOUT));
      *abort_flag = 1;
      return;
    }
  }
  __threadfence();
}

// The pairs of a token: one warp picks the K experts in the router's order and forms their
// weights with the router's arithmetic.  v and key: E values of shared memory each.
__device__ void choose(const Params& p, Fixed& f, int t, int lane, float* v, float* key) {
  const int E = p.E, K = p.K;
  for (int e = lane; e < E; e += 32) {
    const float l = __ldcg(p.logits + static_cast<size_t>(t) * E + e);
    const float s = p.scoring ? sigmoid_f32(l) : l;
    v[e] = s;
    key[e] = p.select_bias ? __fadd_rn(s, __ldg(p.select_bias + e)) : s;
  }
  __syncwarp();
  uint32_t taken = 0;              // bit i: entry lane + 32 i is not eligible any more
  if (p.n_group > 1) {
    const int gs = E / p.n_group;
    uint32_t gkey[2], gtaken = 0, open[2] = {0u, 0u};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int g = lane + 32 * q;
      gkey[q] = 0u;
      if (g < p.n_group) {
        int b0 = -1, b1 = -1;
        for (int e = g * gs; e < g * gs + gs; ++e) {
          if (b0 < 0 || route::ranks_above(key[e], e, key[b0], b0)) {
            b1 = b0;
            b0 = e;
          } else if (b1 < 0 || route::ranks_above(key[e], e, key[b1], b1)) {
            b1 = e;
          }
        }
        gkey[q] = route::rank_key(p.group_score ? __fadd_rn(key[b0], key[b1]) : key[b0]);
      }
    }
    for (int j = 0; j < p.topk_group; ++j) {
      uint32_t bk = 0u, bid = 0xFFFFFFFFu;
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (lane + 32 * q < p.n_group && !((gtaken >> q) & 1u) &&
            (bid == 0xFFFFFFFFu || gkey[q] > bk)) {
          bk = gkey[q];
          bid = static_cast<uint32_t>(lane + 32 * q);
        }
      const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
      const uint32_t win =
          __reduce_min_sync(0xffffffffu, bid != 0xFFFFFFFFu && bk == top ? bid : 0xFFFFFFFFu);
      if (static_cast<int>(win & 31u) == lane) gtaken |= 1u << (win >> 5);
      if (win >> 5) open[1] |= 1u << (win & 31u);
      else open[0] |= 1u << win;
    }
    for (int i = 0; lane + 32 * i < E; ++i) {
      const int g = (lane + 32 * i) / gs;
      const uint32_t bits = g >> 5 ? open[1] : open[0];
      if (!((bits >> (g & 31)) & 1u)) taken |= 1u << i;
    }
  }
  // a lane's best entry is looked for again only after it was taken
  uint32_t bk = 0u, bid = 0xFFFFFFFFu;
  auto rescan = [&]() {
    bk = 0u;
    bid = 0xFFFFFFFFu;
    for (int i = 0; lane + 32 * i < E; ++i) {
      if ((taken >> i) & 1u) continue;
      const uint32_t k = route::rank_key(key[lane + 32 * i]);
      if (bid == 0xFFFFFFFFu || k > bk) {
        bk = k;
        bid = static_cast<uint32_t>(lane + 32 * i);
      }
    }
  };
  rescan();
  float sel = 0.0f;
  int id = 0;
  for (int j = 0; j < K; ++j) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
    const uint32_t win =
        __reduce_min_sync(0xffffffffu, bid != 0xFFFFFFFFu && bk == top ? bid : 0xFFFFFFFFu);
    if (lane == j) {
      id = static_cast<int>(win);
      sel = v[win];
    }
    if (static_cast<int>(win & 31u) == lane) {
      taken |= 1u << (win >> 5);
      rescan();
    }
  }
  float num = sel, den = 1.0f;
  if (p.scoring) {
    if (p.renormalize) {
      den = 0.0f;
      for (int j = 0; j < K; ++j) den = __fadd_rn(den, __shfl_sync(0xffffffffu, sel, j));
    }
  } else {
    const float m = __shfl_sync(0xffffffffu, sel, 0);
    const float d = __fsub_rn(sel, m);
    num = (lane == 0 && d == 0.0f) ? 1.0f : exp_f32(d);
    den = 0.0f;
    if (p.renormalize) {
      for (int j = 0; j < K; ++j) den = __fadd_rn(den, __shfl_sync(0xffffffffu, num, j));
    } else {
      // the sum over all experts, in id order
      for (int e = lane; e < E; e += 32) key[e] = exp_f32(__fsub_rn(v[e], m));
      __syncwarp();
#pragma unroll 8
      for (int e = 0; e < E; ++e) den = __fadd_rn(den, key[e]);
    }
  }
  if (lane < K) {
    const float w = p.scoring && !p.renormalize ? num : __fdiv_rn(num, den);
    f.slot[t][lane] = static_cast<int16_t>(id);
    f.weight[t * K + lane] = __fmul_rn(w, p.routed_scale);
    atomicOr(&f.mask[id], 1u << t);
    if (blockIdx.x == 0) {
      if (p.ids) p.ids[t * K + lane] = id;
      if (p.w) p.w[t * K + lane] = w;
    }
  }
}

// Touched experts in ascending order with their pairs (tokens ascending), then the shared
// expert's tokens.  One warp scans the experts; then a thread per pair places it.
__device__ void group_experts(const Params& p, Fixed& f, int lane) {
  const int per = (p.E + 31) / 32, lo = min(p.E, lane * per), hi = min(p.E, lo + per);
  int n = 0;                       // touched experts, and their pairs in the upper half
  for (int e = lo; e < hi; ++e)
    if (f.mask[e]) n += 1 + (__popc(f.mask[e]) << 16);
  int incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  int run = incl - n;
  for (int e = lo; e < hi; ++e) {
    const uint32_t m = f.mask[e];
    if (!m) continue;
    f.expert[run & 0xFFFF] = static_cast<int16_t>(e);
    f.first[run & 0xFFFF] = static_cast<int16_t>(run >> 16);
    f.mask[e] = m | (static_cast<uint32_t>(run >> 16) << 16);   // tokens below, first pair above
    run += 1 + (__popc(m) << 16);
  }
  if (lane == 31) {
    const int D = run & 0xFFFF, P = run >> 16;
    f.n_groups = D;
    f.first[D] = static_cast<int16_t>(P);
    f.first[D + 1] = static_cast<int16_t>(P + p.T);
  }
}

// One consumer group's or the producer's walk over a phase's chunks, in the same order
struct Chunk {
  int d;          // touched expert, or D: the shared expert
  int n0, cnt;    // first feature (gate/up) or output column (down), and how many
};

// rows of `bytes` that a chunk takes, at most: what a slot holds, in at most kItems items
__device__ __forceinline__ int chunk_rows(const Params& p, int bytes, int cols) {
  const int nseg = (cols + kSeg - 1) / kSeg;       // at most kMaxDim / kSeg = kItems
  return min(min(p.slot_bytes / bytes, kMaxRows), kItems / nseg * 8);
}

template <bool kFp8>
struct GateUpWalk {
  int d, n, left, sh, sh_end, D, I, per, per_s;
  __device__ GateUpWalk(const Params& p, const Fixed& f) {
    // all features in one line, a shared expert's bf16 feature beside FP8 ones counted twice
    constexpr int kCost = kFp8 ? 2 : 1;
    D = f.n_groups;
    I = p.I;
    const long long routed = static_cast<long long>(D) * I, all = routed + kCost * p.Is;
    const long long f0 = all * blockIdx.x / gridDim.x, f1 = all * (blockIdx.x + 1) / gridDim.x;
    const long long r0 = f0 < routed ? f0 : routed, r1 = f1 < routed ? f1 : routed;
    d = static_cast<int>(r0 / I);
    n = static_cast<int>(r0 - static_cast<long long>(d) * I);
    left = static_cast<int>(r1 - r0);
    sh = static_cast<int>(((f0 > routed ? f0 - routed : 0) + kCost - 1) / kCost);
    sh_end = static_cast<int>(((f1 > routed ? f1 - routed : 0) + kCost - 1) / kCost);
    per_s = max(1, chunk_rows(p, 2 * p.H, p.H) / 2);
    per = kFp8 ? max(1, chunk_rows(p, p.H, p.H) / 2) : per_s;
  }
  __device__ bool next(Chunk& c) {
    if (left > 0) {
      c.d = d;
      c.n0 = n;
      c.cnt = min(per, min(I - n, left));
      left -= c.cnt;
      n += c.cnt;
      if (n == I) {
        n = 0;
        ++d;
      }
      return true;
    }
    if (sh >= sh_end) return false;
    c.d = D;
    c.n0 = sh;
    c.cnt = min(per_s, sh_end - sh);
    sh += c.cnt;
    return true;
  }
};

template <bool kFp8>
struct DownWalk {
  int d, n, r0, r1, groups, D, per, per_s;
  // first output column of a CTA
  static __device__ int column(int H, unsigned cta) {
    return static_cast<int>(static_cast<long long>(H) * cta / gridDim.x);
  }
  __device__ DownWalk(const Params& p, const Fixed& f) {
    r0 = column(p.H, blockIdx.x);
    r1 = column(p.H, blockIdx.x + 1);
    D = f.n_groups;
    groups = r1 > r0 ? D + (p.Is > 0 ? 1 : 0) : 0;
    d = 0;
    n = r0;
    // even parts of the CTA's columns
    auto even = [&](int cap) {
      const int parts = (r1 - r0 + cap - 1) / cap;
      return parts > 0 ? (r1 - r0 + parts - 1) / parts : 1;
    };
    per = even(chunk_rows(p, (kFp8 ? 1 : 2) * p.I, p.I));
    per_s = p.Is > 0 ? even(chunk_rows(p, 2 * p.Is, p.Is)) : 1;
  }
  __device__ bool next(Chunk& c) {
    if (d >= groups) return false;
    c.d = d;
    c.n0 = n;
    c.cnt = min(d == D ? per_s : per, r1 - n);
    n += c.cnt;
    if (n == r1) {
      n = r0;
      ++d;
    }
    return true;
  }
};

// 8 weights of a row at shared address a, as f32
template <bool kFp8>
__device__ __forceinline__ void load8(uint32_t a, float (&w)[8]) {
  if (kFp8) {
    uint32_t u[2];
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(u[0]), "=r"(u[1]) : "r"(a) : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>(u[i >> 1] >> (16 * (i & 1))), __NV_E4M3));
      w[2 * i] = __low2float(h);
      w[2 * i + 1] = __high2float(h);
    }
  } else {
    const uint4 u = ptx::ld_shared_v4(a);
    const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[2 * i] = __uint_as_float(q[i] << 16);
      w[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
    }
  }
}

// Sums v[n] over the warp's lanes, n = 8 NT a power of two up to 32: lane l ends with the sum
// of value l * n / 32.  Each step halves the values a lane keeps, so 32 take 31 exchanges.
template <int kN>
__device__ __forceinline__ float transpose_sum(float (&v)[kN], int lane) {
#pragma unroll
  for (int o = 16, n = kN; o >= 1; o >>= 1) {
    if (n > 1) {
      n >>= 1;
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) {
        if (i >= n) break;
        const float keep = lane & o ? v[i + n] : v[i], give = lane & o ? v[i] : v[i + n];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
  return v[0];
}

// A group's work on one chunk and NT tokens (n_tok of them live): every warp sums its items of
// 8 rows x 256 columns into red[(item * 8 + row) * 4 + token], items ordered by row batch, then
// segment.  kDown: the tokens' rows are f32 activations, else bf16 tokens.
template <int NT, bool kFp8, bool kDown>
__device__ __forceinline__ void chunk_sums(const Params& p, const void* const (&src)[NT],
                                           const float* scale0, const float* scale1, int scale_off0,
                                           int scale_off1, int half, int rows, int cols,
                                           uint32_t at, uint32_t full, uint32_t parity, bool first,
                                           volatile int* abort_flag, int warp, int lane,
                                           float* red) {
  const int nseg = (cols + kSeg - 1) / kSeg, items = nseg * ((rows + 7) >> 3);
  const int row_bytes = cols * (kFp8 ? 1 : 2), nblk = (cols + 127) >> 7;
  bool waited = !first;
  for (int it = warp; it < items || !waited; it += kGroupWarps) {
    const bool live = it < items;
    const int b = live ? it / nseg : 0, col = (live ? it - b * nseg : nseg) * kSeg + lane * 8;
    const bool in = live && col < cols;
    float x[NT][8];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (!in) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[t][i] = 0.0f;
      } else if (kDown) {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(src[t]) + col);
        const float4 u = __ldcg(s), w = __ldcg(s + 1);
        x[t][0] = u.x; x[t][1] = u.y; x[t][2] = u.z; x[t][3] = u.w;
        x[t][4] = w.x; x[t][5] = w.y; x[t][6] = w.z; x[t][7] = w.w;
      } else {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src[t]) + col));
        const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[t][2 * i] = __uint_as_float(q[i] << 16);
          x[t][2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
        }
      }
    }
    float sc[8];
    if (kFp8 && in) {
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int row = min(8 * b + r, rows - 1);   // rows [half, 2 half) are up rows
        const bool up = !kDown && row >= half;
        const int at_row = up ? scale_off1 + row - half : scale_off0 + row;
        sc[r] = __ldg((up ? scale1 : scale0) + static_cast<size_t>(at_row >> 7) * nblk + (col >> 7));
      }
    }
    if (!waited) {
      wait(full, parity, abort_flag, p);
      waited = true;
    }
    if (!live) break;
    float acc[8 * NT];
#pragma unroll
    for (int i = 0; i < 8 * NT; ++i) acc[i] = 0.0f;
    const uint32_t a = at + static_cast<uint32_t>(8 * b) * row_bytes + col * (kFp8 ? 1 : 2);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      if (8 * b + r >= rows) break;
      if (!in) continue;
      float w[8];
      load8<kFp8>(a + r * row_bytes, w);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float s = x[t][0] * w[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) s = fmaf(x[t][i], w[i], s);
        acc[r * NT + t] = kFp8 ? s * sc[r] : s;
      }
    }
    const float s = transpose_sum<8 * NT>(acc, lane);
    constexpr int kRep = 32 / (8 * NT);   // lanes that hold the same sum
    const int idx = lane / kRep;
    if (lane % kRep == 0) red[(it * 8 + idx / NT) * 4 + idx % NT] = s;
  }
}

// value of (row, token) of a chunk: its segments in order
__device__ __forceinline__ float row_sum(const float* red, int nseg, int row, int t) {
  const float* q = red + ((row >> 3) * nseg * 8 + (row & 7)) * 4 + t;
  float s = q[0];
  for (int i = 1; i < nseg; ++i) s += q[i * 32];
  return s;
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
layer_few_kernel(const Params p) {
  extern __shared__ uint8_t smem_raw[];
  Fixed& f = *reinterpret_cast<Fixed*>(smem_raw);
  float* out_sum = reinterpret_cast<float*>(smem_raw + sizeof(Fixed));   // [2][T][rows_max]
  const uint32_t ring_off = (sizeof(Fixed) + 2u * p.T * p.rows_max * 4u + 127u) & ~127u;
  uint8_t* ring = smem_raw + ring_off;
  volatile int* abort_flag = &f.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = p.T, H = p.H, E = p.E, K = p.K;

  count_launch(p.launches, MOE_KID_LAYER_FEW);
  if (tid == 0) {
    for (int s = 0; s < p.n_slots; ++s) {
      ptx::mbar_init(ptx::smem_u32(&f.full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&f.empty[s]), kGroupWarps);
    }
    f.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  for (int e = tid; e < E; e += kThreads) f.mask[e] = 0u;
  for (int i = tid; i < 2 * T * p.rows_max; i += kThreads) out_sum[i] = 0.0f;
  grid_dep_wait();
  grid_dep_launch();

  // ---- logits, and the shared expert's gate logits as one more row
  if (warp < 2 * kGroupWarps) {
    const int rows = E + (p.w_gate ? 1 : 0), halves = (T + route::kTokWarp - 1) / route::kTokWarp;
    for (int task = blockIdx.x + gridDim.x * warp; task < rows * halves;
         task += gridDim.x * 2 * kGroupWarps) {
      const int e = task % rows, t0 = task / rows * route::kTokWarp;
      float sum[route::kTokWarp];
      route::small_logits(p.x, e < E ? p.w_router + static_cast<size_t>(e) * H : p.w_gate, H, t0,
                          min(route::kTokWarp, T - t0), lane, sum);
#pragma unroll
      for (int u = 0; u < route::kTokWarp; ++u)
        if (lane == 0 && t0 + u < T) {
          if (e < E)
            p.logits[static_cast<size_t>(t0 + u) * E + e] =
                p.logit_bias ? __fadd_rn(sum[u], __ldg(p.logit_bias + e)) : sum[u];
          else
            p.gate[t0 + u] = sum[u];
        }
    }
  }
  __syncthreads();
  if (tid == 0) grid_barrier(abort_flag, p);
  __syncthreads();

  // ---- choice of experts
  if (warp < T) {
    float* v = reinterpret_cast<float*>(ring) + static_cast<size_t>(warp) * 2 * E;
    choose(p, f, warp, lane, v, v + E);
  }
  if (warp == 2 * kGroupWarps && lane < T)
    f.gate[lane] = p.w_gate ? sigmoid_f32(__ldcg(p.gate + lane)) : 1.0f;
  __syncthreads();
  if (warp == 0) group_experts(p, f, lane);
  __syncthreads();
  for (int i = tid; i < T * K + T; i += kThreads) {
    const int t = i < T * K ? i / K : i - T * K;
    int at = i;
    if (i < T * K) {
      const uint32_t m = f.mask[f.slot[t][i - t * K]];
      at = static_cast<int>(m >> 16) + __popc(m & ((1u << t) - 1u));
    }
    f.pair[at] = static_cast<uint16_t>(i);
    f.token[at] = static_cast<uint16_t>(t);
  }
  ptx::fence_proxy_async_smem();   // the scores in the ring, before copies overwrite them
  __syncthreads();

  const int D = f.n_groups;
  const int col0 = DownWalk<kFp8>::column(H, blockIdx.x);   // this CTA's output columns
  if (warp == 2 * kGroupWarps) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int s = 0;
      uint32_t issued = 0, phase = 1;
      // one chunk of `cnt` rows at src (and at src2), of `bytes` each
      auto put = [&](const uint8_t* src, const uint8_t* src2, uint32_t bytes) {
        if (!wait(ptx::smem_u32(&f.empty[s]), phase, abort_flag, p)) return false;
        const uint32_t bar = ptx::smem_u32(&f.full[s]);
        const uint32_t dst = ptx::smem_u32(ring) + static_cast<uint32_t>(s) * p.slot_bytes;
        ptx::mbar_arrive_expect_tx(bar, src2 ? 2 * bytes : bytes);
        bulk_load(dst, src, bytes, bar);
        if (src2) bulk_load(dst + bytes, src2, bytes, bar);
        ++issued;
        if (++s == p.n_slots) {
          s = 0;
          phase ^= 1u;
        }
        return true;
      };
      Chunk c;
      bool ok = true;
      for (GateUpWalk<kFp8> walk(p, f); ok && walk.next(c);) {
        const bool q = kFp8 && c.d < D;          // E4M3 rows
        const int I = c.d < D ? p.I : p.Is;
        const size_t row = static_cast<size_t>(H) * (q ? 1 : 2);
        const uint8_t* w = c.d < D ? static_cast<const uint8_t*>(p.w13) +
                                         static_cast<size_t>(f.expert[c.d]) * 2 * I * row
                                   : reinterpret_cast<const uint8_t*>(p.w13s);
        ok = put(w + c.n0 * row, w + (static_cast<size_t>(I) + c.n0) * row,
                 static_cast<uint32_t>(c.cnt * row));
      }
      for (DownWalk<kFp8> walk(p, f); ok && walk.next(c);) {
        const bool q = kFp8 && c.d < D;
        const size_t row = static_cast<size_t>(c.d < D ? p.I : p.Is) * (q ? 1 : 2);
        const uint8_t* w = c.d < D ? static_cast<const uint8_t*>(p.w2) +
                                         static_cast<size_t>(f.expert[c.d]) * H * row
                                   : reinterpret_cast<const uint8_t*>(p.w2s);
        ok = put(w + c.n0 * row, nullptr, static_cast<uint32_t>(c.cnt * row));
      }
      // a CTA that gave up lets its copies land before it ends
      const uint32_t n = p.n_slots;
      for (uint32_t i = issued > n ? issued - n : 0; i < issued; ++i)
        gemm::spin_bounded(ptx::smem_u32(&f.full[i % n]), (i / n) & 1u);
    }
    return;
  }

  // ------------------------------------------------------------ consumers
  const int group = warp / kGroupWarps, gwarp = warp - group * kGroupWarps;
  const int gtid = tid - group * 32 * kGroupWarps;
  int index = 0;                   // of the chunk, over both phases
  int s = 0;
  uint32_t phase = 0;
  int buffer = 0;
  auto advance = [&]() {
    ++index;
    if (++s == p.n_slots) {
      s = 0;
      phase ^= 1u;
    }
  };
  // sums of one chunk for up to 4 of its expert's tokens; returns the buffer they are in
  auto sums = [&](auto down, auto fp8, const Chunk& c, int i0, int nt, bool first) {
    constexpr bool kDown = decltype(down)::value, kQ = decltype(fp8)::value;
    const bool shared = c.d == D;
    const int I = shared ? p.Is : p.I, cols = kDown ? I : H, rows = kDown ? c.cnt : 2 * c.cnt;
    const uint32_t at = ptx::smem_u32(ring) + static_cast<uint32_t>(s) * p.slot_bytes;
    const uint32_t full = ptx::smem_u32(&f.full[s]);
    float* red = f.red[group][buffer];
    const float *sc0 = nullptr, *sc1 = nullptr;
    int so0 = 0, so1 = 0;
    if (kQ) {
      const int nblk = (cols + 127) >> 7, R = kDown ? H : 2 * I;
      sc0 = (kDown ? p.s2 : p.s13) + static_cast<size_t>(f.expert[c.d]) * ((R + 127) >> 7) * nblk;
      sc1 = sc0;
      so0 = c.n0;
      so1 = I + c.n0;
    }
    const int first_pair = f.first[c.d] + i0;
    auto src_of = [&](int i) -> const void* {
      const int at_pair = first_pair + min(i, nt - 1);
      if (!kDown) return p.x + static_cast<size_t>(f.token[at_pair]) * H;
      if (shared) return p.act_s + static_cast<size_t>(f.token[at_pair]) * I;
      return p.act + static_cast<size_t>(f.pair[at_pair]) * I;
    };
    if (nt == 1) {
      const void* const src[1] = {src_of(0)};
      chunk_sums<1, kQ, kDown>(p, src, sc0, sc1, so0, so1, c.cnt, rows, cols, at, full, phase, first,
                               abort_flag, gwarp, lane, red);
    } else if (nt == 2) {
      const void* const src[2] = {src_of(0), src_of(1)};
      chunk_sums<2, kQ, kDown>(p, src, sc0, sc1, so0, so1, c.cnt, rows, cols, at, full, phase, first,
                               abort_flag, gwarp, lane, red);
    } else {
      const void* const src[4] = {src_of(0), src_of(1), src_of(2), src_of(3)};
      chunk_sums<4, kQ, kDown>(p, src, sc0, sc1, so0, so1, c.cnt, rows, cols, at, full, phase, first,
                               abort_flag, gwarp, lane, red);
    }
  };
  auto chunk = [&](auto down, const Chunk& c) {
    constexpr bool kDown = decltype(down)::value;
    const bool shared = c.d == D;
    const int I = shared ? p.Is : p.I, nseg = ((kDown ? I : H) + kSeg - 1) / kSeg;
    const int n_tok = f.first[c.d + 1] - f.first[c.d];
    for (int i0 = 0; i0 < n_tok; i0 += 4) {
      const int nt = min(4, n_tok - i0);
      if (kFp8 && !shared) sums(down, std::true_type{}, c, i0, nt, i0 == 0);
      else sums(down, std::false_type{}, c, i0, nt, i0 == 0);
      if (i0 + 4 >= n_tok) {       // this warp's last read of the slot
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&f.empty[s]));
      }
      ptx::bar_sync(kBarGroup + group, 32 * kGroupWarps);
      const float* red = f.red[group][buffer];
      buffer ^= 1;                 // the other half is free: its readers have passed this barrier
      for (int i = gtid; i < c.cnt * nt; i += 32 * kGroupWarps) {
        const int t = i / c.cnt, r = i - t * c.cnt, pair = f.first[c.d] + i0 + t;
        if (kDown) {
          const float y = row_sum(red, nseg, r, t);
          const int tok = f.token[pair];
          const float w = shared ? f.gate[tok] : f.weight[f.pair[pair]];
          float* o = out_sum + (group * T + tok) * p.rows_max + c.n0 + r - col0;
          *o = fmaf(w, y, *o);
        } else {
          const float g = row_sum(red, nseg, r, t), u = row_sum(red, nseg, c.cnt + r, t);
          const float a = g / (1.0f + __expf(-g)) * u;
          if (shared) p.act_s[static_cast<size_t>(f.token[pair]) * I + c.n0 + r] = a;
          else p.act[static_cast<size_t>(f.pair[pair]) * I + c.n0 + r] = a;
        }
      }
    }
  };
  Chunk c;
  for (GateUpWalk<kFp8> walk(p, f); walk.next(c); advance())
    if ((index & 1) == group) chunk(std::false_type{}, c);
  ptx::bar_sync(kBarAll, kConsumers);
  if (tid == 0) grid_barrier(abort_flag, p);
  ptx::bar_sync(kBarAll, kConsumers);
  for (DownWalk<kFp8> walk(p, f); walk.next(c); advance())
    if ((index & 1) == group) chunk(std::true_type{}, c);
  ptx::bar_sync(kBarAll, kConsumers);

  // ---- both groups' sums, the residual, one rounding
  const int rows = DownWalk<kFp8>::column(H, blockIdx.x + 1) - col0;
  for (int i = tid; i < T * rows; i += kConsumers) {
    const int t = i / rows, r = i - t * rows;
    float v = out_sum[t * p.rows_max + r] + out_sum[(T + t) * p.rows_max + r];
    const size_t at = static_cast<size_t>(t) * H + col0 + r;
    if (p.residual) v += bf16_bits_to_f32(p.residual[at]);
    p.out[at] = f32_to_bf16_bits(v);
  }
}

// ------------------------------------------------------------------ host side
size_t pad(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

struct Layout {
  size_t logits, gate, act, act_s, bytes;
};
Layout layout_of(int T, int I, int E, int K, int Is) {
  Layout l;
  l.logits = 256;                  // the barrier's words before it
  l.gate = l.logits + pad(static_cast<size_t>(T) * E * 4);
  l.act = l.gate + pad(static_cast<size_t>(T) * 4);
  l.act_s = l.act + pad(static_cast<size_t>(T) * K * I * 4);
  l.bytes = l.act_s + pad(static_cast<size_t>(T) * Is * 4);
  return l;
}

int check(const char* op, const Params& p, bool fp8, const void* workspace, size_t ws_bytes) {
  if (p.T < 0 || p.T > kMaxT) return set_error(MOE_ERR_ARG, "%s: T=%d outside [0, %d]", op, p.T, kMaxT);
  if (p.E < 1 || p.E > kMaxE) return set_error(MOE_ERR_ARG, "%s: E=%d outside [1, %d]", op, p.E, kMaxE);
  if (p.K < 1 || p.K > p.E || p.K > 32)
    return set_error(MOE_ERR_ARG, "%s: K=%d outside [1, min(E, 32)]", op, p.K);
  if (p.H < 1 || p.H > kMaxDim) return set_error(MOE_ERR_ARG, "%s: H=%d outside [1, %d]", op, p.H, kMaxDim);
  if (p.I < 1 || p.I > kMaxDim) return set_error(MOE_ERR_ARG, "%s: I=%d outside [1, %d]", op, p.I, kMaxDim);
  if (p.Is < 0 || p.Is > kMaxDim)
    return set_error(MOE_ERR_ARG, "%s: I_shared=%d outside [0, %d]", op, p.Is, kMaxDim);
  if (p.renormalize != 0 && p.renormalize != 1)
    return set_error(MOE_ERR_ARG, "%s: renormalize must be 0 or 1", op);
  if (p.scoring != 0 && p.scoring != 1)
    return set_error(MOE_ERR_UNSUPPORTED, "%s: scoring=%d is not 0 (softmax) or 1 (sigmoid)", op, p.scoring);
  if (p.select_bias && p.scoring != 1)
    return set_error(MOE_ERR_UNSUPPORTED, "%s: a selection bias is implemented for sigmoid scores only", op);
  if (p.n_group < 1 || p.n_group > route::kMaxGroups || p.E % p.n_group != 0)
    return set_error(MOE_ERR_ARG, "%s: n_group=%d must divide E=%d and be at most %d", op, p.n_group, p.E,
                     route::kMaxGroups);
  if (p.topk_group < 1 || p.topk_group > p.n_group)
    return set_error(MOE_ERR_ARG, "%s: topk_group=%d outside [1, n_group=%d]", op, p.topk_group, p.n_group);
  if (p.group_score != 0 && p.group_score != 1)
    return set_error(MOE_ERR_ARG, "%s: group_score=%d is not 0 (best) or 1 (two best)", op, p.group_score);
  if (p.group_score == 1 && p.E / p.n_group < 2)
    return set_error(MOE_ERR_ARG, "%s: two-best group scores need groups of two experts", op);
  if (p.K > p.topk_group * (p.E / p.n_group))
    return set_error(MOE_ERR_ARG, "%s: K=%d exceeds the %d experts of the eligible groups", op, p.K,
                     p.topk_group * (p.E / p.n_group));
  const int step = fp8 ? 16 : 8;
  if (p.H % step || p.I % step || p.Is % 8)
    return set_error(MOE_ERR_ALIGN, "%s: H=%d and I=%d must be multiples of %d, I_shared=%d of 8", op, p.H, p.I,
                     step, p.Is);
  if (p.T == 0) return MOE_OK;
  if (!p.x || !p.w_router || !p.w13 || !p.w2 || !p.out)
    return set_error(MOE_ERR_ARG, "%s: x, w_router, the expert weights or out is NULL", op);
  if (fp8 && (!p.s13 || !p.s2)) return set_error(MOE_ERR_ARG, "%s: the weights' scales are NULL", op);
  if (p.Is > 0 && (!p.w13s || !p.w2s))
    return set_error(MOE_ERR_ARG, "%s: I_shared=%d without w13_shared or w2_shared", op, p.Is);
  if (p.Is == 0 && (p.w_gate || p.w13s || p.w2s))
    return set_error(MOE_ERR_ARG, "%s: shared expert's weights with I_shared=0", op);
  for (const void* q : {static_cast<const void*>(p.x), static_cast<const void*>(p.w_router), p.w13, p.w2,
                        static_cast<const void*>(p.w_gate), static_cast<const void*>(p.w13s),
                        static_cast<const void*>(p.w2s), workspace})
    if (q && !aligned16(q))
      return set_error(MOE_ERR_ALIGN, "%s: x, weights and workspace must be 16-byte aligned", op);
  for (const void* q : {static_cast<const void*>(p.logit_bias), static_cast<const void*>(p.select_bias),
                        static_cast<const void*>(p.s13), static_cast<const void*>(p.s2),
                        static_cast<const void*>(p.ids), static_cast<const void*>(p.w)})
    if (reinterpret_cast<uintptr_t>(q) & 3u)
      return set_error(MOE_ERR_ALIGN, "%s: biases, scales, topk_ids and topk_w must be 4-byte aligned", op);
  if ((reinterpret_cast<uintptr_t>(p.residual) & 1u) || (reinterpret_cast<uintptr_t>(p.out) & 1u))
    return set_error(MOE_ERR_ALIGN, "%s: residual and out must be 2-byte aligned", op);
  const size_t need = layout_of(p.T, p.I, p.E, p.K, p.Is).bytes;
  if (!workspace || ws_bytes < need)
    return set_error(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes is smaller than the %zu needed", op,
                     workspace ? ws_bytes : 0, need);
  return MOE_OK;
}

template <bool kFp8>
int launch(const char* op, Params p, void* workspace, cudaStream_t stream) {
  const Layout l = layout_of(p.T, p.I, p.E, p.K, p.Is);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.barrier = reinterpret_cast<unsigned int*>(ws);
  p.logits = reinterpret_cast<float*>(ws + l.logits);
  p.gate = reinterpret_cast<float*>(ws + l.gate);
  p.act = reinterpret_cast<float*>(ws + l.act);
  p.act_s = reinterpret_cast<float*>(ws + l.act_s);
  const int ctas = sm_count();
  p.rows_max = (p.H + ctas - 1) / ctas;
  // a slot holds a feature's gate and up row and a down row
  int slot = 16384;
  auto grow = [&](int bytes) { slot = bytes > slot ? bytes : slot; };
  grow(2 * p.H * (kFp8 ? 1 : 2));
  grow(p.I * (kFp8 ? 1 : 2));
  if (p.Is > 0) {
    grow(4 * p.H);
    grow(2 * p.Is);
  }
  p.slot_bytes = (slot + 127) & ~127;
  const int fixed = (static_cast<int>(sizeof(Fixed)) + 2 * p.T * p.rows_max * 4 + 127) & ~127;
  constexpr int kSmem = 227 * 1024;
  p.n_slots = (kSmem - fixed) / p.slot_bytes;
  if (p.n_slots > kMaxSlots) p.n_slots = kMaxSlots;
  int ring = p.n_slots * p.slot_bytes;
  if (ring < 2 * p.T * p.E * 4) ring = 2 * p.T * p.E * 4;   // the scores of the choice
  const int smem = fixed + ring;
  if (p.n_slots < 2 || smem > kSmem)
    return set_error(MOE_ERR_CUDA, "%s: %d SMs leave no room for the ring", op, ctas);
  auto kern = layer_few_kernel<kFp8>;
  static std::atomic<int> configured[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    dev = -1;
  }
  const bool cache = dev >= 0 && dev < 64;
  if (!cache || !configured[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
      return set_error(MOE_ERR_CUDA, "%s: cannot reserve %d bytes of shared memory: %s", op, kSmem,
                       cudaGetErrorString(cudaGetLastError()));
    if (cache) configured[dev].store(1, std::memory_order_release);
  }
  DeviceDiag diag = device_diag();
  p.status = diag.status;
  p.launches = diag.launches;
  p.wait_ns = gemm::pipeline_wait_ns();
  // cooperative: the CTAs wait for one another, so all of them start together or none does
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  return launch_status(launch_kernel(kern, dim3(ctas), dim3(kThreads), smem, stream, attr, 1, p), op);
}

}  // namespace
}  // namespace few
}  // namespace moe

using namespace moe;

extern "C" size_t moe_layer_few_workspace_size(int T, int H, int I, int E, int K, int I_shared) {
  (void)H;
  if (T <= 0 || I <= 0 || E <= 0 || K <= 0 || I_shared < 0) return 0;
  return few::layout_of(T, I, E, K, I_shared).bytes;
}

namespace moe {
namespace few {
namespace {
template <bool kFp8>
int run(const char* op, const void* x, const void* w_router, const float* logit_bias, const float* select_bias,
        const void* w13, const float* s13, const void* w2, const float* s2, const void* w_gate, const void* w13s,
        const void* w2s, const void* residual, int T, int H, int I, int E, int K, int Is, int renormalize,
        int scoring, int n_group, int topk_group, int group_score, float routed_scale, int32_t* ids, float* w,
        void* out, void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  Params p{};
  p.x = static_cast<const uint16_t*>(x);
  p.w_router = static_cast<const uint16_t*>(w_router);
  p.logit_bias = logit_bias;
  p.select_bias = select_bias;
  p.w13 = w13;
  p.s13 = s13;
  p.w2 = w2;
  p.s2 = s2;
  p.w_gate = static_cast<const uint16_t*>(w_gate);
  p.w13s = static_cast<const uint16_t*>(w13s);
  p.w2s = static_cast<const uint16_t*>(w2s);
  p.residual = static_cast<const uint16_t*>(residual);
  p.T = T; p.H = H; p.I = I; p.E = E; p.K = K; p.Is = Is;
  p.renormalize = renormalize; p.scoring = scoring; p.n_group = n_group;
  p.topk_group = topk_group; p.group_score = group_score;
  p.routed_scale = routed_scale;
  p.ids = ids;
  p.w = w;
  p.out = static_cast<uint16_t*>(out);
  const int rc = check(op, p, kFp8, workspace, ws_bytes);
  if (rc != MOE_OK || T == 0) return rc;
  return launch<kFp8>(op, p, workspace, static_cast<cudaStream_t>(stream));
}
}  // namespace
}  // namespace few
}  // namespace moe

extern "C" int moe_layer_few_bf16(const void* x_bf16, const void* w_router_bf16, const float* logit_bias,
                                  const float* select_bias, const void* w13_bf16, const void* w2_bf16,
                                  const void* w_shared_gate_bf16, const void* w13_shared_bf16,
                                  const void* w2_shared_bf16, const void* residual_bf16, int T, int H, int I, int E,
                                  int K, int I_shared, int renormalize, int scoring, int n_group, int topk_group,
                                  int group_score, float routed_scale, int32_t* topk_ids, float* topk_w,
                                  void* out_bf16, void* workspace, size_t ws_bytes, void* stream) {
  return few::run<false>("moe_layer_few_bf16", x_bf16, w_router_bf16, logit_bias, select_bias, w13_bf16, nullptr,
                         w2_bf16, nullptr, w_shared_gate_bf16, w13_shared_bf16, w2_shared_bf16, residual_bf16, T, H,
                         I, E, K, I_shared, renormalize, scoring, n_group, topk_group, group_score, routed_scale,
                         topk_ids, topk_w, out_bf16, workspace, ws_bytes, stream);
}

extern "C" int moe_layer_few_fp8w(const void* x_bf16, const void* w_router_bf16, const float* logit_bias,
                                  const float* select_bias, const uint8_t* w13_e4m3, const float* w13_scale,
                                  const uint8_t* w2_e4m3, const float* w2_scale, const void* w_shared_gate_bf16,
                                  const void* w13_shared_bf16, const void* w2_shared_bf16,
                                  const void* residual_bf16, int T, int H, int I, int E, int K, int I_shared,
                                  int renormalize, int scoring, int n_group, int topk_group, int group_score,
                                  float routed_scale, int32_t* topk_ids, float* topk_w, void* out_bf16,
                                  void* workspace, size_t ws_bytes, void* stream) {
  return few::run<true>("moe_layer_few_fp8w", x_bf16, w_router_bf16, logit_bias, select_bias, w13_e4m3, w13_scale,
                        w2_e4m3, w2_scale, w_shared_gate_bf16, w13_shared_bf16, w2_shared_bf16, residual_bf16, T, H,
                        I, E, K, I_shared, renormalize, scoring, n_group, topk_group, group_score, routed_scale,
                        topk_ids, topk_w, out_bf16, workspace, ws_bytes, stream);
}
