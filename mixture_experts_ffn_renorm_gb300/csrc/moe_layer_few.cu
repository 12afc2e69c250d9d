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
//   gate/up   blocks of four features of the touched experts, each taken by the first warp of the grid that is
//             free: w[p] act[p, n] to the workspace; grid barrier
//   down      a CTA owns H / CTAs output columns for all experts, so no partial sums cross CTAs
//
// The barrier between gate/up and down costs no bandwidth: the copies run ahead of it, since
// the down rows do not depend on it.
//
// Every warp is a stream of its own: two slots of 8 KB that it refills as soon as it has read them, and
// no warp waits for another.  A slot is one TMA box, swizzled over 128 bytes, one of whose dimensions
// steps along the rows: one instruction.  (Copies of single rows reach the same 7.0 TB/s in a loop of
// copies alone, but each costs its warp about 200 cycles to issue, 1700 a slot.)
// The products are mma.sync: a few tokens leave tcgen05's 128 rows empty, and what counts is
// instructions per byte of weights.  Weight rows are the M side, tokens the N side; a lane reads 16 bytes of a row
// and the same columns of a token, which permutes the columns of a step alike on both sides.  Columns of
// the N side without a token repeat another's, and their sums are dropped.
//   gate/up   4 gate rows and the 4 up rows of the same features at two places of the contraction, against
//             four tokens at the same two: exact products, f32 sums; silu(gate) up times routing weight in f32
//   down      16 output columns.  The f32 activations are kept as three bf16 parts that add up
//             to them (8 bits each, rounded to nearest, 24 in all), so their products stay exact too; two
//             tokens' parts are six columns.  A token's sums over its experts never leave the registers.
// FP8 weights are widened to bf16, exactly, and a block's sums take its scale in f32.
// All sums are f32 in a fixed order, nothing between the weights and the output is narrowed, and
// no atomics touch data.
//
// What it measured (2048 x 768, 128 experts, 8 of them chosen; bf16): one token 27.0 us, of which 3.2 until
// the logits have crossed the grid, 3 the choice, 15 gate/up (7.4 of them the weights' way), 1 the second barrier, 3.5 down;
// 16 tokens 130 us at 6.0 TB/s.  Steps on the way, us for one token and for 16:
//   chunks shared by eight warps, a group barrier after each      80  681   13000 cycles a chunk of index arithmetic
//   a ring per warp, single rows and multiply-adds                37  319   an expert of many tokens held all SMs up
//   mma.sync, three parts, one loop for both phases               33  186   (140 KB of code had to come from L2)
//   TMA boxes, a piece's token loads in flight together           28  187   (680 cycles each, in turn, before)
//   features dealt by their experts' tokens                       28  158
//   sorted heads in the choice, tokens to L1 beside it            27  151
//   blocks taken in turn, not dealt                               27  130   (SMs differed by a third)
#include <atomic>

#include "fp8_common.cuh"
#include "route_device.cuh"

namespace moe {
namespace few {
namespace {

constexpr int kMaxT = MOE_LAYER_FEW_MAX_TOKENS;    // one warp per token in the choice
constexpr int kMaxDim = MOE_LAYER_FEW_MAX_DIM;     // H, I, I_shared
constexpr int kMaxE = 1024;
constexpr int kMaxPairs = kMaxT * 32;
constexpr int kWarps = 12;
constexpr int kThreads = 32 * kWarps;
constexpr int kSlots = 2;          // per warp (the loop's two cursors)
// A slot, in blocks of 128 bytes of a row: gate/up 8 blocks x 4 features' gate rows and their up rows;
// down 4 blocks x 16 rows
constexpr int kFeat = 4;
constexpr int kGuBlocks = 8, kDnBlocks = 4;
constexpr int kSlotBytes = 8192;
static_assert(2 * kFeat * kGuBlocks * 128 == kSlotBytes && 16 * kDnBlocks * 128 == kSlotBytes, "slot");
constexpr int kRing = kWarps * kSlots * kSlotBytes;

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
  unsigned long long* barrier;     // arrivals of all launches
  unsigned int* turns;             // blocks of gate/up that were asked for
  float* logits;                   // [T, E]
  float* gate;                     // [T]
  uint16_t* act;                   // [3][T K, I], then [3][T, Is]: parts of the weighted activations
  unsigned long long wait_ns;
  unsigned int* status;
  unsigned long long* launches;
};

// A weight matrix: boxes of a slot's whole blocks, and single blocks
struct Matrix {
  CUtensorMap slot, block;
};
struct Maps {
  Matrix w13, w2, w13s, w2s;
};

// Shared memory: the fixed part, then the ring, which first holds the choice's scratch and last
// the warps' sums
struct alignas(16) Fixed {
  uint64_t full[kWarps][kSlots];
  float weight[kMaxPairs];         // routing weight of a pair, times routed_scale
  float gate[kMaxT];               // sigmoid of the shared expert's gate
  uint16_t pair[kMaxPairs + kMaxT];    // pairs by expert; then the shared expert's tokens
  uint16_t token[kMaxPairs + kMaxT];   // their tokens
  int16_t expert[kMaxPairs + 1];   // touched experts, ascending
  int16_t first[kMaxPairs + 3];    // their first pair
  int n_groups;                    // touched experts, without the shared one
  int abort_flag;
};
struct Scratch {
  uint32_t mask[kMaxE];            // tokens that chose an expert, then its first pair above
  int16_t slot[kMaxT][32];         // chosen experts of a token, by rank
  float scores[1];                 // [T][2 E]
};

// a box of an [expert][row half][row][column] matrix, seen as blocks of 128 bytes of a row
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* m, int row, int block, int expert, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %2, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(0), "r"(row), "r"(block), "r"(expert), "r"(bar)
      : "memory");
}

// a block of 128 bytes of the rows from any column on, what lies behind their end as zeros
__device__ __forceinline__ void block_load(uint32_t dst, const CUtensorMap* m, int row, int col, int expert, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(col), "r"(row), "r"(0), "r"(expert), "r"(bar)
      : "memory");
}

// Bounded wait; false when it ran out or this CTA has given up.  Callers go on either way: every
// loop is finite, so a warp that gave up runs to its end without waiting again.
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

// The grid barrier counts arrivals and is never reset: `target` is the count that this CTA's arrival
// belongs to, a multiple of the CTAs.  One thread's part: its release covers the CTA's writes, which
// it has seen through the block barrier before it, its acquire those of all others.
__device__ __forceinline__ void grid_barrier(unsigned long long target, volatile int* abort_flag, const Params& p) {
  asm volatile("fence.acq_rel.gpu;" ::: "memory");
  asm volatile("red.relaxed.gpu.global.add.u64 [%0], 1;" ::"l"(p.barrier) : "memory");
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
    unsigned long long n;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(n) : "l"(p.barrier) : "memory");
    if (n >= target) return;
    if (ptx::globaltimer_ns() - t0 > p.wait_ns) {
      if (p.status) atomicOr(p.status, static_cast<unsigned int>(MOE_STATUS_TIMEOUT));
      *abort_flag = 1;
      return;
    }
  }
}

// one copy of the router's exponential: what runs once per call costs its instructions' way
// from memory (the kernel of one token spent a third of its time waiting for code)
__device__ __noinline__ float exp_once(float v) { return exp_f32(v); }
__device__ __forceinline__ float sigmoid_once(float v) { return __fdiv_rn(1.0f, __fadd_rn(1.0f, exp_once(-v))); }

// The K best of a token's E keys in the router's order (descending, ties to the lower id, NaN last)
// among those whose bit of `taken` is clear: the j-th id in lane j.  A lane holds entries lane +
// 32 i, sorted once; a pick compares the lanes' heads, and the winning lane's next entry moves up.
template <int kPer>
__device__ __forceinline__ int pick(const float* key, int E, int K, int lane, uint32_t taken) {
  uint32_t k[kPer], id[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    const bool out = e >= E || (taken >> i & 1u);            // below every expert, and never reached
    k[i] = out ? 0u : route::rank_key(key[e]);
    id[i] = out ? 0xFFFFFFFFu : static_cast<uint32_t>(e);
  }
#pragma unroll
  for (int r = 0; r < kPer; ++r)                             // odd-even transposition
#pragma unroll
    for (int i = r & 1; i + 1 < kPer; i += 2) {
      const bool turn = k[i + 1] > k[i] || (k[i + 1] == k[i] && id[i + 1] < id[i]);
      const uint32_t k0 = k[i], i0 = id[i];
      k[i] = turn ? k[i + 1] : k0;
      id[i] = turn ? id[i + 1] : i0;
      k[i + 1] = turn ? k0 : k[i + 1];
      id[i + 1] = turn ? i0 : id[i + 1];
    }
  int mine = 0;
#pragma unroll 1
  for (int j = 0; j < K; ++j) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, k[0]);
    const uint32_t win = __reduce_min_sync(0xffffffffu, k[0] == top ? id[0] : 0xFFFFFFFFu);
    if (lane == j) mine = static_cast<int>(win);
    if ((win & 31u) == static_cast<uint32_t>(lane)) {
#pragma unroll
      for (int i = 0; i + 1 < kPer; ++i) {
        k[i] = k[i + 1];
        id[i] = id[i + 1];
      }
      k[kPer - 1] = 0u;
      id[kPer - 1] = 0xFFFFFFFFu;
    }
  }
  return mine;
}

// The same for many experts: a lane looks through its entries again for every pick
__device__ __forceinline__ int pick_many(const float* key, int E, int K, int lane, uint32_t taken) {
  int mine = 0;
#pragma unroll 1
  for (int j = 0; j < K; ++j) {
    uint32_t bk = 0u, bid = 0xFFFFFFFFu;
#pragma unroll 4
    for (int i = 0; i < (E + 31) / 32; ++i) {
      const int e = lane + 32 * i;
      const uint32_t k = e < E ? route::rank_key(key[e]) : 0u;
      if (e < E && !(taken >> i & 1u) && (bid == 0xFFFFFFFFu || k > bk)) {
        bk = k;
        bid = static_cast<uint32_t>(e);
      }
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
    const uint32_t win = __reduce_min_sync(0xffffffffu, bk == top ? bid : 0xFFFFFFFFu);
    if ((win & 31u) == static_cast<uint32_t>(lane)) taken |= 1u << (win >> 5);
    if (lane == j) mine = static_cast<int>(win);
  }
  return mine;
}

// The pairs of a token: one warp picks the K experts in the router's order and forms their
// weights with the router's arithmetic.
__device__ __forceinline__ void choose(const Params& p, Fixed& f, Scratch& x, int t, int lane) {
  const int E = p.E, K = p.K;
  float *v = x.scores + static_cast<size_t>(t) * 2 * E, *key = v + E;
#pragma unroll 1
  for (int e0 = lane; e0 < E; e0 += 256) {
    float l[8];                    // in flight together
#pragma unroll
    for (int i = 0; i < 8; ++i)
      l[i] = e0 + 32 * i < E ? __ldcg(p.logits + static_cast<size_t>(t) * E + e0 + 32 * i) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = e0 + 32 * i;
      if (e >= E) break;
      const float s = p.scoring ? sigmoid_once(l[i]) : l[i];
      v[e] = s;
      key[e] = p.select_bias ? __fadd_rn(s, __ldg(p.select_bias + e)) : s;
    }
  }
  __syncwarp();
  uint32_t taken = 0;              // bit i: entry lane + 32 i is not eligible
  if (p.n_group > 1) {
    // A group is scored by its best key or two: `sub` lanes look through its experts, each keeping two,
    // and join them.  A key and its value are one 64-bit number, so that the larger is the better.
    // Lane g then has the keys of groups g and g + 32; the topk_group best stay open.
    const int gs = E / p.n_group;
    const int sub = p.n_group > 16 ? 1 : p.n_group > 8 ? 2 : p.n_group > 4 ? 4 : 8;
    uint32_t gkey[2] = {0u, 0u}, open[2] = {0u, 0u}, gtaken = 0;
#pragma unroll 1
    for (int q = 0; q < (p.n_group > 32 ? 2 : 1); ++q) {
      const int g = 32 * q + lane / sub;
      unsigned long long b0 = 0, b1 = 0;
      if (g < p.n_group)
#pragma unroll 2
        for (int e = g * gs + lane % sub; e < g * gs + gs; e += sub) {
          const unsigned long long k =
              (route::rank_key(key[e]) + 1ull) << 32 | __float_as_uint(key[e]);
          b1 = max(b1, min(b0, k));
          b0 = max(b0, k);
        }
#pragma unroll 1
      for (int o = 1; o < sub; o <<= 1) {
        const unsigned long long c0 = __shfl_xor_sync(0xffffffffu, b0, o), c1 = __shfl_xor_sync(0xffffffffu, b1, o);
        b1 = max(min(b0, c0), max(b1, c1));
        b0 = max(b0, c0);
      }
      const float best = __uint_as_float(static_cast<uint32_t>(b0)), next = __uint_as_float(static_cast<uint32_t>(b1));
      const uint32_t k = route::rank_key(p.group_score ? __fadd_rn(best, next) : best);
      if (q) gkey[1] = __shfl_sync(0xffffffffu, k, lane * sub & 31);
      else gkey[0] = __shfl_sync(0xffffffffu, k, lane * sub & 31);
    }
#pragma unroll 1
    for (int j = 0; j < p.topk_group; ++j) {
      uint32_t bk = 0u, bid = 0xFFFFFFFFu;
#pragma unroll
      for (int q = 0; q < 2; ++q)
        if (lane + 32 * q < p.n_group && !((gtaken >> q) & 1u) && (bid == 0xFFFFFFFFu || gkey[q] > bk)) {
          bk = gkey[q];
          bid = static_cast<uint32_t>(lane + 32 * q);
        }
      const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
      const uint32_t win = __reduce_min_sync(0xffffffffu, bk == top ? bid : 0xFFFFFFFFu);
      if ((win & 31u) == static_cast<uint32_t>(lane)) gtaken |= 1u << (win >> 5);
      if (win >> 5) open[1] |= 1u << (win & 31u);
      else open[0] |= 1u << win;
    }
#pragma unroll 1
    for (int i = 0; lane + 32 * i < E; ++i) {
      const int g = (lane + 32 * i) / gs;
      if (!((g >> 5 ? open[1] : open[0]) >> (g & 31) & 1u)) taken |= 1u << i;
    }
  }
  const int id = E <= 128   ? pick<4>(key, E, K, lane, taken)
                 : E <= 256 ? pick<8>(key, E, K, lane, taken)
                            : pick_many(key, E, K, lane, taken);
  const float sel = v[id];
  float num = sel, den = 0.0f;
  const float m = __shfl_sync(0xffffffffu, sel, 0);
  if (!p.scoring) {
    const float d = __fsub_rn(sel, m);
    num = (lane == 0 && d == 0.0f) ? 1.0f : exp_once(d);
  }
  if (p.renormalize) {
#pragma unroll 1
    for (int j = 0; j < K; ++j) den = __fadd_rn(den, __shfl_sync(0xffffffffu, num, j));
  } else if (!p.scoring) {
    // the sum over all experts, in id order
    __syncwarp();
#pragma unroll 1
    for (int e = lane; e < E; e += 32) key[e] = exp_once(__fsub_rn(v[e], m));
    __syncwarp();
#pragma unroll 4
    for (int e = 0; e < E; ++e) den = __fadd_rn(den, key[e]);
  }
  if (lane < K) {
    const float w = p.scoring && !p.renormalize ? num : __fdiv_rn(num, den);
    x.slot[t][lane] = static_cast<int16_t>(id);
    f.weight[t * K + lane] = __fmul_rn(w, p.routed_scale);
    atomicOr(&x.mask[id], 1u << t);
    if (blockIdx.x == 0) {
      if (p.ids) p.ids[t * K + lane] = id;
      if (p.w) p.w[t * K + lane] = w;
    }
  }
}

// Touched experts in ascending order with their pairs (tokens ascending), then the shared
// expert's tokens.  One warp scans the experts; then a thread per pair places it.
__device__ __forceinline__ void group_experts(const Params& p, Fixed& f, Scratch& x, int lane) {
  const int per = (p.E + 31) / 32, lo = min(p.E, lane * per), hi = min(p.E, lo + per);
  int n = 0;                       // touched experts, and their pairs in the upper half
#pragma unroll 1
  for (int e = lo; e < hi; ++e)
    if (x.mask[e]) n += 1 + (__popc(x.mask[e]) << 16);
  int incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  int run = incl - n;
#pragma unroll 1
  for (int e = lo; e < hi; ++e) {
    const uint32_t m = x.mask[e];
    if (!m) continue;
    const int tokens = __popc(m);
    f.expert[run & 0xFFFF] = static_cast<int16_t>(e);
    f.first[run & 0xFFFF] = static_cast<int16_t>(run >> 16);
    x.mask[e] = m | (static_cast<uint32_t>(run >> 16) << 16);
    run += 1 + (tokens << 16);
  }
  if (lane == 31) {
    const int D = run & 0xFFFF, P = run >> 16;
    f.n_groups = D;
    f.first[D] = static_cast<int16_t>(P);
    f.first[D + 1] = static_cast<int16_t>(P + p.T);
  }
}

// The pieces of a warp's stream, in order: its blocks of features of gate/up, piece by piece, then
// its (expert, piece) units of down.  Two cursors walk it, the copies' ahead of the sums'.
struct Cursor {
  int phase;      // 0 gate/up, 1 down, 2 end
  int i;          // gate/up: block of all touched experts'; down: unit among the row block's
  int d, n;       // touched expert (D: the shared one); gate/up: its features [n, n + 4)
  int k;          // column of the piece
};

template <bool kFp8>
struct Stream {
  const Params& p;
  const Fixed& f;
  const Maps& maps;
  int D, warp, lane;
  // gate/up: blocks of features, the shared expert's first; the warp's next one is known by its turn
  int shared_blocks, blocks;
  unsigned turn;
  // down: output columns [col0, col0 + cols) of the CTA, [row0, row0 + rows) of this warp's row block
  int col0, cols, row_blocks, row0, rows, unit0, unit_step, pieces, units;
  unsigned per_inv, pieces_inv;    // of I / 4 and of pieces

  __device__ Stream(const Params& p_, const Fixed& f_, const Maps& maps_, int warp_, int lane_)
      : p(p_), f(f_), maps(maps_), warp(warp_), lane(lane_) {
    D = f.n_groups;
    // The blocks in one line.  A warp's first is its place in the grid, the SMs' first warps before their second
    // ones; every further one is the next that nobody has.
    const unsigned cta = blockIdx.x;
    const int per = p.I / kFeat;                             // I % 8 == 0
    per_inv = 0xFFFFFFFFu / per + 1u;
    shared_blocks = p.Is / kFeat;
    blocks = shared_blocks + D * per;
    turn = blocks;
    take_turn();
    const unsigned H = p.H;
    col0 = static_cast<int>(H / gridDim.x * cta + min(cta, H % gridDim.x));
    cols = static_cast<int>(H / gridDim.x + (cta < H % gridDim.x ? 1u : 0u));
    // even blocks of at most 16 rows; the warps take blocks in turn, and share a block's units
    row_blocks = (cols + 15) >> 4;
    const int rb_i = row_blocks ? warp % row_blocks : 0;
    row0 = row_blocks ? cols * rb_i / row_blocks : 0;
    rows = row_blocks ? cols * (rb_i + 1) / row_blocks - row0 : 0;
    unit0 = row_blocks ? warp / row_blocks : 0;
    unit_step = row_blocks ? (kWarps - 1 - rb_i) / row_blocks + 1 : 1;
    pieces = (p.I + dn_cols(0) - 1) / dn_cols(0);
    pieces_inv = 0xFFFFFFFFu / pieces + 1u;
    units = rows > 0 ? D * pieces + (p.Is + dn_cols(D) - 1) / dn_cols(D) : 0;
  }
  __device__ bool quant(int d) const { return kFp8 && d < D; }
  __device__ int inner(int d) const { return d < D ? p.I : p.Is; }
  __device__ int shift(int d) const { return quant(d) ? 7 : 6; }               // columns of a block of 128 bytes
  __device__ int gu_cols(int d) const { return kGuBlocks << shift(d); }        // of a piece
  __device__ int dn_cols(int d) const { return kDnBlocks << shift(d); }

  // j / n for inv = ceil(2^32 / n) modulo 2^32: exact while j n < 2^32 (here below 2^31); 0 stands for n = 1
  static __device__ int divided(int j, unsigned inv) {
    return inv ? static_cast<int>(__umulhi(static_cast<unsigned>(j), inv)) : j;
  }
  __device__ void locate(Cursor& c) const {
    if (c.phase == 0) {
      if (c.i < blocks) {
        const int j = c.i - shared_blocks, of = divided(max(j, 0), per_inv);
        c.d = j < 0 ? D : of;
        c.n = kFeat * (j < 0 ? c.i : j - of * (p.I / kFeat));
        return;
      }
      c.phase = 1;
      c.i = unit0;
    }
    if (c.i >= units) {
      c.phase = 2;
    } else if (c.i < D * pieces) {
      c.d = divided(c.i, pieces_inv);
      c.k = (c.i - c.d * pieces) * dn_cols(0);
    } else {
      c.d = D;
      c.k = (c.i - D * pieces) * dn_cols(D);
    }
  }
  // asks for the block after the next (one lane), while the next is worked on: an answer takes as long as a load
  __device__ void take_turn() {
    const int warps = static_cast<int>(gridDim.x) * kWarps;
    if (blocks > warps && lane == 0) turn = warps + atomicAdd(p.turns, 1u);
  }
  __device__ Cursor begin() const {
    Cursor c{0, static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) * warp, 0, 0, 0};
    locate(c);
    return c;
  }
  __device__ void next(Cursor& c) {
    if (c.phase == 0) {
      c.k += gu_cols(c.d);
      if (c.k < p.H) return;
      c.k = 0;
      c.i = static_cast<int>(__shfl_sync(0xffffffffu, turn, 0));
      if (c.i < blocks) take_turn();
    } else {
      c.i += unit_step;
    }
    locate(c);
  }
  // The copy of a piece (one lane): one box, or where the row ends inside a block (whose rest in memory is
  // the next row's) blocks one by one.  What lies behind the row, and rows behind the expert's, are zeros;
  // rows of the next CTA are not used.
  __device__ void issue(const Cursor& c, uint32_t slot, uint32_t bar) const {
    const int sh = shift(c.d), left = (c.phase == 0 ? p.H : inner(c.d)) - c.k, n = c.phase == 0 ? kGuBlocks : kDnBlocks;
    const int expert = c.d < D ? f.expert[c.d] : 0, row = c.phase == 0 ? c.n : col0 + row0;
    const Matrix& m = c.phase == 0 ? (c.d < D ? maps.w13 : maps.w13s) : (c.d < D ? maps.w2 : maps.w2s);
    ptx::mbar_arrive_expect_tx(bar, kSlotBytes);
    if (left >= n << sh || !(left & ((1 << sh) - 1))) {
      box_load(slot, &m.slot, row, c.k >> sh, expert, bar);
    } else {
#pragma unroll 1
      for (int i = 0; i < n; ++i) block_load(slot + i * (kSlotBytes / n), &m.block, row, c.k + (i << sh), expert, bar);
    }
  }
};

// four E4M3 codes as bf16, exactly
__device__ __forceinline__ void widen4(uint32_t c, uint32_t& lo, uint32_t& hi) {
  const __half2 a = __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3));
  const __half2 b = __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c >> 16), __NV_E4M3));
  lo = gemm::pack_bf16x2(__low2float(a), __high2float(a));
  hi = gemm::pack_bf16x2(__low2float(b), __high2float(b));
}

// two steps' weights of a lane, 16 bytes each, as MMA operands: bf16 for 2 x 16 columns, or codes for 4 x 16
template <bool kQ>
struct Row {
  uint32_t v[kQ ? 4 : 2][2];       // [MMA][first and second 8 columns]
  __device__ __forceinline__ explicit Row(const uint4& w) {
    if (kQ) {
      widen4(w.x, v[0][0], v[0][1]);
      widen4(w.y, v[1][0], v[1][1]);
      widen4(w.z, v[kQ ? 2 : 0][0], v[kQ ? 2 : 0][1]);
      widen4(w.w, v[kQ ? 3 : 0][0], v[kQ ? 3 : 0][1]);
    } else {
      v[0][0] = w.x;
      v[0][1] = w.y;
      v[1][0] = w.z;
      v[1][1] = w.w;
    }
  }
};

// c[0] += the first MMAs' products, c[1] the second's (two sums, two chains): rows 0-7 lo, 8-15 hi
template <bool kQ>
__device__ __forceinline__ void products(float (&c)[2][4], const Row<kQ>& lo, const Row<kQ>& hi, const uint4 (&u)[kQ ? 2 : 1]) {
#pragma unroll
  for (int j = 0; j < (kQ ? 4 : 2); ++j) {
    const uint4& b = u[kQ ? j >> 1 : 0];
    // rows of weights x columns of tokens
    ptx::mma_m16n8k16(c[j & 1], lo.v[j][0], hi.v[j][0], lo.v[j][1], hi.v[j][1], j & 1 ? b.z : b.x, j & 1 ? b.w : b.y);
  }
}
// c += the two sums, with FP8 times the scales of rows 0-7 and 8-15; and clears them
template <bool kQ>
__device__ __forceinline__ void join(float (&sum)[2][4], float lo, float hi, float (&c)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float v = sum[0][j] + sum[1][j];
    c[j] = kQ ? fmaf(v, j < 2 ? lo : hi, c[j]) : c[j] + v;
    sum[0][j] = sum[1][j] = 0.0f;
  }
}

// A lane's token values of a piece: in each of four blocks of 128 bytes of weights vectors 2 q and 2 q + 1.
// x: the token's values of the piece's first of the four blocks, 16 bytes a vector; `vecs` of them are left of the
// token (the others' products are with zeros).  All loads are in flight together: they are the latency of a
// piece (680 cycles from L2; in turn with the multiplications four times that).
template <bool kQ>
struct Tokens {
  static constexpr int kVec = kQ ? 2 : 1;        // token vectors to a weight vector
  uint4 u[4][2][kVec];
  template <bool kFinal>                         // not written while the kernel runs
  __device__ __forceinline__ void load(const uint4* x, int q, int vecs) {
    x += 2 * q * kVec;
    vecs -= 2 * q * kVec;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          const int at = (i * 8 + h) * kVec + v;
          u[i][h][v] = at < vecs ? (kFinal ? __ldg(x + at) : x[at]) : make_uint4(0, 0, 0, 0);
        }
  }
};

// One piece of a block of gate/up for four of the expert's tokens, added to c.  The 8 rows (4 features'
// gate rows, then their up rows) fill both halves of the MMA's rows, its first with the blocks 0-3 of 128
// bytes of the piece, its second with 4-7; the MMA's columns 0-3 are the tokens at the first blocks'
// columns, 4-7 the same tokens at the second's.  What counts of c is rows 0-7 of columns 0-3 and rows
// 8-15 of columns 4-7.  at: row g of the slot; d: this lane's row's scales, block by block.
template <bool kQ>
__device__ __forceinline__ void gate_up(const uint8_t* at, int g, int q, const Tokens<kQ>& x, const float (&d)[8],
                                        float (&c)[4]) {
  float sum[2][4] = {};
  at += ((2 * q) ^ g) << 4;                      // vector 2 q; 2 q + 1 is 16 bytes to either side
  const int odd = (g & 1) ? -16 : 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t* v = at + (h ? odd : 0) + i * 1024;
      products<kQ>(sum, Row<kQ>(*reinterpret_cast<const uint4*>(v)), Row<kQ>(*reinterpret_cast<const uint4*>(v + 4096)),
                   x.u[i][h]);
    }
    if (kQ) join<kQ>(sum, d[i], d[i + 4], c);    // a block is a scale block
  }
  if (!kQ) join<kQ>(sum, 1.0f, 1.0f, c);
}

// One unit of down for two of the expert's tokens, added to c: 16 output columns' rows (this lane's rows
// g and g + 8, their scales d[0-3] and d[4-7]); the MMA's columns 2 j and 2 j + 1 are the two tokens' part j.
template <bool kQ>
__device__ __forceinline__ void down(const uint8_t* at, int g, int q, const Tokens<kQ>& x, const float (&d)[8],
                                     float (&c)[4]) {
  float sum[2][4] = {};
  at += ((2 * q) ^ g) << 4;
  const int odd = (g & 1) ? -16 : 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t* v = at + (h ? odd : 0) + i * 2048;
      products<kQ>(sum, Row<kQ>(*reinterpret_cast<const uint4*>(v)), Row<kQ>(*reinterpret_cast<const uint4*>(v + 1024)),
                   x.u[i][h]);
    }
    if (kQ) join<kQ>(sum, d[i], d[i + 4], c);
  }
  if (!kQ) join<kQ>(sum, 1.0f, 1.0f, c);
}

// v as three bf16 parts that add up to it (an infinity or NaN as its first part alone)
__device__ __forceinline__ void cut3(float v, uint16_t (&part)[3]) {
  part[0] = f32_to_bf16_bits(v);
  const float r = v - bf16_bits_to_f32(part[0]);
  const bool fine = fabsf(r) < __int_as_float(0x7f800000);   // false for NaN
  part[1] = fine ? f32_to_bf16_bits(r) : 0;
  part[2] = fine ? f32_to_bf16_bits(r - bf16_bits_to_f32(part[1])) : 0;
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
layer_few_kernel(const __grid_constant__ Maps maps, const Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the ring at a multiple of 1024 bytes, the swizzle's period, the fixed part behind it
  uint8_t* slots = smem_raw + (-ptx::smem_u32(smem_raw) & 1023u);
  Fixed& f = *reinterpret_cast<Fixed*>(slots + kRing);
  Scratch& x = *reinterpret_cast<Scratch*>(slots);
  volatile int* abort_flag = &f.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = p.T, H = p.H, E = p.E, K = p.K;

  count_launch(p.launches, MOE_KID_LAYER_FEW);
  if (lane < kSlots) ptx::mbar_init(ptx::smem_u32(&f.full[warp][lane]), 1);
  if (tid == 0) {
    f.abort_flag = 0;
    ptx::tma_prefetch_desc(&maps.w13.slot);
    ptx::tma_prefetch_desc(&maps.w2.slot);
  }
  ptx::fence_mbar_init();
  for (int e = tid; e < E; e += kThreads) x.mask[e] = 0u;
  grid_dep_wait();
  grid_dep_launch();
  // the arrivals of earlier launches are a multiple of the CTAs, and before this CTA's own nobody passes
  unsigned long long arrivals = 0;
  if (tid == 0) arrivals = (*reinterpret_cast<volatile unsigned long long*>(p.barrier) / gridDim.x + 1) * gridDim.x;

  // ---- logits, and the shared expert's gate logits as one more row
  {
    const int rows = E + (p.w_gate ? 1 : 0), halves = (T + route::kTokWarp - 1) / route::kTokWarp;
#pragma unroll 1
    for (int task = blockIdx.x + gridDim.x * warp; task < rows * halves; task += gridDim.x * kWarps) {
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
  if (tid == 0) {
    if (blockIdx.x == 0) *p.turns = 0u;          // nobody asks before the barrier
    grid_barrier(arrivals, abort_flag, p);
  }
  __syncthreads();

  // ---- choice of experts
#pragma unroll 1
  for (int t = warp; t < T; t += kWarps) choose(p, f, x, t, lane);
  // Meanwhile the other warps bring the tokens to L1, where the barrier's acquire has left nothing, if
  // they fit into the 24 KB that the ring leaves: loads of their 32-byte sectors whose values nobody waits for
  if (warp >= T && T * H <= 12 * 1024) {
    float unused;
#pragma unroll 1
    for (int i = (warp - T) * 32 + lane; i < T * H / 16; i += (kWarps - T) * 32)
      asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(unused) : "l"(p.x + static_cast<size_t>(i) * 16));
  }
  if (tid < T) f.gate[tid] = p.w_gate ? sigmoid_once(__ldcg(p.gate + tid)) : 1.0f;
  __syncthreads();
  if (warp == 0) group_experts(p, f, x, lane);
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < T * K + T; i += kThreads) {
    const int t = i < T * K ? i / K : i - T * K;
    int at = i;
    if (i < T * K) {
      const uint32_t m = x.mask[x.slot[t][i - t * K]];
      at = static_cast<int>(m >> 16) + __popc(m & ((1u << t) - 1u));
    }
    f.pair[at] = static_cast<uint16_t>(i);
    f.token[at] = static_cast<uint16_t>(t);
  }
  ptx::fence_proxy_async_smem();   // the scratch in the ring, before copies overwrite it
  __syncthreads();

  // ---- the experts.  One loop over the pieces of both phases, so that their code is there once:
  // wait for the slot, multiply, refill the slot
  Stream<kFp8> st(p, f, maps, warp, lane);
  const int D = st.D, g = lane >> 2, q = lane & 3;
  const uint32_t ring = ptx::smem_u32(slots) + warp * kSlots * kSlotBytes, bars = ptx::smem_u32(&f.full[warp][0]);
  Cursor c[kSlots], ahead = st.begin();          // of the pieces in the slots, the oldest first
  int s = 0;
  uint32_t parity = 0;
  // A warp whose wait ran out neither waits nor copies again: the slot's barrier is a phase behind from
  // there on, where a wait would return at once and a copy would arm the same phase twice.
  bool gave_up = false;
  uint32_t armed = 0;              // bit s: parity of slot s's last copy; bit s + 2: it has had one
  auto arm = [&](int slot) {
    if (ahead.phase == 2) return;
    if (lane == 0) st.issue(ahead, ring + slot * kSlotBytes, bars + 8 * slot);
    armed = (armed >> (slot + 2) & 1u ? armed ^ 1u << slot : armed) | 4u << slot;
  };
#pragma unroll 1
  for (int i = 0; i < kSlots; ++i) {
    arm(i);
    c[0] = c[1];
    c[1] = ahead;
    if (ahead.phase < 2) st.next(ahead);
  }
  // gate/up: sums of the expert's tokens, four by four; down: of tokens 0-7 and 8-15
  float sum[4][4] = {};
  auto turn = [&]() {                            // the next four's sums first
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float t = sum[0][j];
      sum[0][j] = sum[1][j];
      sum[1][j] = sum[2][j];
      sum[2][j] = sum[3][j];
      sum[3][j] = t;
    }
  };
#pragma unroll 1
  for (int phase = 0; phase < 2; ++phase) {
#pragma unroll 1
    while (c[0].phase == phase) {
      const int d = c[0].d, k = c[0].k, first = f.first[d], n_tok = f.first[d + 1] - first, I = st.inner(d);
      const bool quant = st.quant(d), shared = d == D;
      const int expert = shared ? 0 : f.expert[d];
      const uint8_t* at = slots + (warp * kSlots + s) * kSlotBytes;
      bool landed = false, waited = false;
      auto take = [&]() {
        if (waited) return;
        waited = true;
        landed = !gave_up && __all_sync(0xffffffffu, wait(bars + 8 * s, parity, abort_flag, p));
        gave_up = !landed;
      };
      const int sh = st.shift(d), cols = 1 << sh;
      if (phase == 0) {
        const int n = min(kGuBlocks * cols, H - k), last = (n - 1) >> sh;    // columns, last block
        // this lane's row: feature g & 3, gate or up
        const int row = (g < kFeat ? 0 : I) + c[0].n + (g & 3);
        const float* sc = nullptr;
        if (kFp8 && quant)
          sc = p.s13 + (expert * ((2 * I + 127) >> 7) + (row >> 7)) * static_cast<size_t>((H + 127) >> 7) + (k >> 7);
        const uint8_t* mine = at + g * 128;
        const int fours = n_tok > 4 ? 4 : 1;     // of tokens, in the sums' four places
        float scale[8];
        if (kFp8 && quant) {
#pragma unroll
          for (int i = 0; i < 8; ++i) scale[i] = __ldg(sc + min(i, last));
        }
        auto token = [&](int i0) {
          return p.x + static_cast<size_t>(f.token[first + min(i0 + (g & 3), n_tok - 1)]) * H + k;
        };
        auto load = [&](int i0, auto& u) {
          const int from = (g >> 2) * 4 * cols;
          u.template load<true>(reinterpret_cast<const uint4*>(token(i0) + from), q, (n - from) >> 3);
        };
        auto multiply = [&](int i0, auto u) {
          load(i0, u);
          take();
          gate_up(mine, g, q, u, scale, sum[0]);
        };
#pragma unroll 1
        for (int i0 = 0; i0 < 4 * fours; i0 += 4) {
          if (i0 < n_tok) {
            if (kFp8 && quant) multiply(i0, Tokens<kFp8>());
            else multiply(i0, Tokens<false>());
          }
          if (fours > 1) turn();
        }
        if (k + n == H) {
          // the features' last piece: silu(gate) up, weighted, in parts for the down product
#pragma unroll 1
          for (int i0 = 0; i0 < 4 * fours; i0 += 4) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              // both halves of the columns; then lanes q < 2 hold tokens 2 q + j of rows g
              const float v = sum[0][j] + __shfl_xor_sync(0xffffffffu, sum[0][2 + j], 2);
              const float up = __shfl_down_sync(0xffffffffu, v, 4 * kFeat);
              const int i = i0 + 2 * q + j;
              if (q < 2 && g < kFeat && i < n_tok) {              // gate rows
                const int pair = f.pair[first + i], tok = f.token[first + i], to_row = shared ? tok : pair;
                const float a = v / (1.0f + __expf(-v)) * up * (shared ? f.gate[tok] : f.weight[pair]);
                uint16_t part[3];
                cut3(a, part);
                const size_t step = static_cast<size_t>(shared ? T : T * K) * I;
                uint16_t* to = p.act + (shared ? 3 * static_cast<size_t>(T) * K * p.I : 0) +
                               static_cast<size_t>(to_row) * I + c[0].n + g;
                to[0] = part[0];
                to[step] = part[1];
                to[2 * step] = part[2];
              }
            }
            if (fours > 1) turn();
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[0][j] = sum[1][j] = sum[2][j] = sum[3][j] = 0.0f;
        }
      } else {
        const int n = min(kDnBlocks * cols, I - k), last = (n - 1) >> sh;
        // this lane's rows
        const int r0 = min(st.col0 + st.row0 + g, H - 1), r1 = min(r0 + 8, H - 1);
        const float *sc0 = nullptr, *sc1 = nullptr;
        if (kFp8 && quant) {
          const size_t nblk = (I + 127) >> 7;
          const float* s2 = p.s2 + expert * ((H + 127) >> 7) * nblk + (k >> 7);
          sc0 = s2 + (r0 >> 7) * nblk;
          sc1 = s2 + (r1 >> 7) * nblk;
        }
        const uint16_t* act = p.act + (shared ? 3 * static_cast<size_t>(T) * K * p.I : 0) +
                              min(g >> 1, 2) * (static_cast<size_t>(shared ? T : T * K) * I) + k;
        float scale[8];
        if (kFp8 && quant) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            scale[i] = __ldg(sc0 + min(i, last));
            scale[i + 4] = __ldg(sc1 + min(i, last));
          }
        }
        auto token = [&](int i0) {
          const int i = first + min(i0 + (g & 1), n_tok - 1);
          return act + static_cast<size_t>(shared ? f.token[i] : f.pair[i]) * I;
        };
        auto load = [&](int i0, auto& u) { u.template load<false>(reinterpret_cast<const uint4*>(token(i0)), q, n >> 3); };
        auto multiply = [&](int i0, auto u, float (&v)[4]) {
          load(i0, u);
          take();
          down(at + g * 128, g, q, u, scale, v);
        };
#pragma unroll 1
        for (int i0 = 0; i0 < n_tok; i0 += 2) {
          float v[4] = {};
          if (kFp8 && quant) multiply(i0, Tokens<kFp8>(), v);
          else multiply(i0, Tokens<false>(), v);
          // the three parts, in lanes q = 0, 1, 2; then to the sums of the lane that keeps the token
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (q == 3) v[j] = 0.0f;
            v[j] += __shfl_xor_sync(0xffffffffu, v[j], 1);
            v[j] += __shfl_xor_sync(0xffffffffu, v[j], 2);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (i0 + e >= n_tok) break;
            const int t = f.token[first + i0 + e];
            if ((t >> 1 & 3) == q) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                if (t == 2 * q + j) {
                  sum[0][j] += v[e];
                  sum[0][2 + j] += v[2 + e];
                } else if (t == 8 + 2 * q + j) {
                  sum[1][j] += v[e];
                  sum[1][2 + j] += v[2 + e];
                }
              }
            }
          }
        }
      }
      __syncwarp();                              // all lanes have read the slot
      if (landed) arm(s);
      c[0] = c[1];
      c[1] = ahead;
      if (ahead.phase < 2) st.next(ahead);
      s ^= 1;
      parity ^= s ? 0u : 1u;
    }
    __syncthreads();
    if (phase == 0) {
      if (tid == 0) grid_barrier(arrivals + gridDim.x, abort_flag, p);
      __syncthreads();
    }
  }

  // ---- the warps' sums in warp order, the residual, one rounding
  float* sums = reinterpret_cast<float*>(slots);                 // [warp][row of 16][token of 16]
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float* to = sums + (warp * 16 + g + 8 * (j >> 1)) * 16 + 2 * q + (j & 1);
    to[0] = sum[0][j];
    to[8] = sum[1][j];
  }
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < T * st.cols; i += kThreads) {
    const int t = i / st.cols, r = i - t * st.cols;
    // the row block of column r: the last one that starts at or before it
    int rb = r * st.row_blocks / st.cols;
    if (rb + 1 < st.row_blocks && st.cols * (rb + 1) / st.row_blocks <= r) ++rb;
    const int row = r - st.cols * rb / st.row_blocks;
    float v = 0.0f;
#pragma unroll 1
    for (int w = rb; w < kWarps; w += st.row_blocks) v += sums[(w * 16 + row) * 16 + t];
    const size_t at = static_cast<size_t>(t) * H + st.col0 + r;
    if (p.residual) v += bf16_bits_to_f32(p.residual[at]);
    p.out[at] = f32_to_bf16_bits(v);
  }
  // a warp that gave up lets its copies land before it ends
  if (gave_up)
    for (int i = 0; i < kSlots; ++i)
      if (armed >> (i + 2) & 1u) gemm::spin_bounded(bars + 8 * i, armed >> i & 1u);
}

// ------------------------------------------------------------------ host side
size_t pad(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

struct Layout {
  size_t logits, gate, act, bytes;
};
Layout layout_of(int T, int I, int E, int K, int Is) {
  Layout l;
  l.logits = 256;                  // the barrier's count before it
  l.gate = l.logits + pad(static_cast<size_t>(T) * E * 4);
  l.act = l.gate + pad(static_cast<size_t>(T) * 4);
  l.bytes = l.act + pad(6 * static_cast<size_t>(T) * (static_cast<size_t>(K) * I + Is));
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

// [experts][halves][rows][cols] bf16 values or codes, boxes of box_rows rows of every half; rows without a whole
// block of 128 bytes have no boxes of several
int make_maps(Matrix* m, const void* base, bool codes, int experts, int halves, int rows, int cols, int box_rows,
              int box_blocks, const char* op, const char* what) {
  const int rc = gemm::make_tmap_block(&m->block, base, codes, experts, halves, rows, cols, box_rows, op, what);
  if (rc != MOE_OK || cols < (codes ? 128 : 64)) return rc;
  return gemm::make_tmap_blocks(&m->slot, base, codes, experts, halves, rows, cols, box_rows, box_blocks, op, what);
}

template <bool kFp8>
int launch(const char* op, Params p, void* workspace, cudaStream_t stream) {
  const Layout l = layout_of(p.T, p.I, p.E, p.K, p.Is);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.barrier = reinterpret_cast<unsigned long long*>(ws);
  p.turns = reinterpret_cast<unsigned int*>(ws + 64);
  p.logits = reinterpret_cast<float*>(ws + l.logits);
  p.gate = reinterpret_cast<float*>(ws + l.gate);
  p.act = reinterpret_cast<uint16_t*>(ws + l.act);
  const int ctas = sm_count();
  if (p.H > 16ll * kWarps * ctas)      // row blocks of the down product: a warp has one
    return set_error(MOE_ERR_CUDA, "%s: H=%d on %d SMs", op, p.H, ctas);
  constexpr int kSmem = kRing + static_cast<int>(sizeof(Fixed)) + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(sizeof(Scratch) + 2 * kMaxT * kMaxE * 4 <= kRing && kWarps * 1024 <= kRing, "what the ring holds besides");
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
  Maps maps{};
  int rc;
  if ((rc = make_maps(&maps.w13, p.w13, kFp8, p.E, 2, p.I, p.H, kFeat, kGuBlocks, op, "w13")) != MOE_OK) return rc;
  if ((rc = make_maps(&maps.w2, p.w2, kFp8, p.E, 1, p.H, p.I, 16, kDnBlocks, op, "w2")) != MOE_OK) return rc;
  if (p.Is > 0) {
    if ((rc = make_maps(&maps.w13s, p.w13s, false, 1, 2, p.Is, p.H, kFeat, kGuBlocks, op, "w13_shared")) != MOE_OK)
      return rc;
    if ((rc = make_maps(&maps.w2s, p.w2s, false, 1, 1, p.H, p.Is, 16, kDnBlocks, op, "w2_shared")) != MOE_OK) return rc;
  }
  // cooperative: the CTAs wait for one another, so all of them start together or none does
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  return launch_status(launch_kernel(kern, dim3(ctas), dim3(kThreads), kSmem, stream, attr, 1, maps, p), op);
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
