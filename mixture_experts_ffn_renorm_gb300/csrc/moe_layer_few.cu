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
// The barrier between gate/up and down costs no bandwidth: the copies run ahead of it, since
// the down rows do not depend on it.
//
// Every warp is a stream of its own: three 4 KB slots that its lanes refill as soon as they have
// read them, so 192 KB an SM are in flight and no warp waits for another.  A slot holds up to 2 KB of two
// rows: a feature's gate and up row, or two output columns' rows of an expert.  A lane takes 8
// columns of each 256; bf16 weights meet bf16 tokens in the multiply-add that widens (exact
// products, f32 sums), FP8 weights and the f32 activations are widened first.  After the last
// piece of a row the sums of two rows x up to 16 tokens are joined over the lanes by a
// transposing butterfly.  A down row's sums are added to its tokens' outputs in expert order by the one
// warp that owns it, experts of even and of odd place apart (two rows share an activation's load).
// All sums are f32 in a fixed order, nothing between the weights and the output is narrowed, and
// no atomics touch data.  CUDA cores suffice: a touched expert has 1.5 tokens on average at T = 16,
// and with f32 activations a tensor-core product would need them split into bf16 parts.
//
// Chunks shared by eight warps, with a group barrier after each, took 80 us for one token (2048 x 768,
// 128 experts, 8 of them chosen): 13000 cycles a chunk of index arithmetic and barriers.
#include <atomic>

#include "fp8_common.cuh"
#include "route_device.cuh"

namespace moe {
namespace few {
namespace {

constexpr int kMaxT = 16;          // tokens: one warp per token in the choice
constexpr int kMaxDim = 8192;      // H, I, I_shared
constexpr int kMaxE = 1024;
constexpr int kMaxPairs = kMaxT * 32;
constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kSeg = 256;          // columns of a segment: 8 per lane
constexpr int kSlots = 3;          // per warp
constexpr int kPiece = 2048;       // bytes of a row in a slot, at most
constexpr int kSlotBytes = 2 * kPiece;
constexpr unsigned long long kCopyGraceNs = 100000ull;
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
  unsigned int* barrier;           // [0] arrivals, [1] generation
  float* logits;                   // [T, E]
  float* gate;                     // [T]
  float* act;                      // [T K, I]
  float* act_s;                    // [T, Is]
  int rows_max;                    // output columns of a CTA, at most
  unsigned long long wait_ns;
  unsigned int* status;
  unsigned long long* launches;
};

// Shared memory: the fixed part, then the output sums, then the ring (which first holds the
// choice's scores)
struct alignas(16) Fixed {
  uint64_t full[kWarps][kSlots];
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

// The pieces of a warp's stream, in order: its features of gate/up, then its rows of down.  Two
// cursors walk it, the copies' ahead of the sums'.
struct Cursor {
  int phase;      // 0 gate/up, 1 down, 2 end
  int i;          // gate/up: feature among the CTA's; down: first of the two rows among the CTA's
  int d, n;       // touched expert (D: the shared one); feature of the expert
  int k;          // column of the piece
};

template <bool kFp8>
struct Stream {
  const Params& p;
  const Fixed& f;
  int D, warp, lane;
  long long f0;                    // the CTA's first feature among the routed ones in one line
  int nr, ns, s0;                  // its routed and shared features, the first shared one
  int col0, cols;                  // its output columns

  __device__ Stream(const Params& p_, const Fixed& f_, int warp_, int lane_) : p(p_), f(f_), warp(warp_), lane(lane_) {
    D = f.n_groups;
    // all features in one line, a shared expert's bf16 feature beside FP8 ones counted twice
    constexpr int kCost = kFp8 ? 2 : 1;
    const long long routed = static_cast<long long>(D) * p.I, all = routed + kCost * p.Is;
    const long long a = all * blockIdx.x / gridDim.x, b = all * (blockIdx.x + 1) / gridDim.x;
    f0 = a < routed ? a : routed;
    nr = static_cast<int>((b < routed ? b : routed) - f0);
    s0 = static_cast<int>(((a > routed ? a - routed : 0) + kCost - 1) / kCost);
    ns = static_cast<int>(((b > routed ? b - routed : 0) + kCost - 1) / kCost) - s0;
    col0 = static_cast<int>(static_cast<long long>(p.H) * blockIdx.x / gridDim.x);
    cols = static_cast<int>(static_cast<long long>(p.H) * (blockIdx.x + 1) / gridDim.x) - col0;
  }
  __device__ bool quant(int d) const { return kFp8 && d < D; }
  __device__ int inner(int d) const { return d < D ? p.I : p.Is; }
  // columns of a row, and of a piece of it
  __device__ int row_cols(const Cursor& c) const { return c.phase == 0 ? p.H : inner(c.d); }
  __device__ int piece_cols(int d) const { return quant(d) ? kPiece : kPiece / 2; }

  __device__ void feature(Cursor& c) const {
    if (c.i < nr) {
      const unsigned at = static_cast<unsigned>(f0 + c.i);      // below 512 * 8192
      c.d = static_cast<int>(at / static_cast<unsigned>(p.I));
      c.n = static_cast<int>(at - static_cast<unsigned>(c.d) * static_cast<unsigned>(p.I));
    } else if (c.i < nr + ns) {
      c.d = D;
      c.n = s0 + c.i - nr;
    } else {                       // down: experts of this half of the warps, two rows a warp
      c.phase = 1;
      c.d = warp >> 3;
      c.i = 2 * (warp & 7);
      if (c.i >= cols || c.d >= groups()) c.phase = 2;
    }
  }
  __device__ int groups() const { return D + (p.Is > 0 ? 1 : 0); }
  __device__ Cursor begin() const {
    Cursor c{0, warp, 0, 0, 0};
    feature(c);
    return c;
  }
  // the next feature or pair of rows
  __device__ void next_item(Cursor& c) const {
    c.k = 0;
    if (c.phase == 0) {
      c.i += kWarps;
      feature(c);
    } else {
      c.i += kWarps;               // eight warps, two rows each
      if (c.i >= cols) {
        c.i = 2 * (warp & 7);
        c.d += 2;
        if (c.d >= groups()) c.phase = 2;
      }
    }
  }
  __device__ void next_piece(Cursor& c) const {
    c.k += piece_cols(c.d);
    if (c.k >= row_cols(c)) next_item(c);
  }
  // the copies of a piece: lanes 0 and 1 a row each
  __device__ void issue(const Cursor& c, uint32_t slot, uint32_t bar) const {
    if (c.phase == 2) return;
    const bool q = quant(c.d);
    const int C = row_cols(c), I = inner(c.d);
    const uint32_t bytes = static_cast<uint32_t>(min(piece_cols(c.d), C - c.k)) * (q ? 1 : 2);
    const int rows = c.phase == 0 || c.i + 1 < cols ? 2 : 1;
    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, bytes * rows);
    if (lane < rows) {
      const size_t row_bytes = static_cast<size_t>(C) * (q ? 1 : 2);
      const uint8_t* w;
      size_t row;
      if (c.phase == 0) {
        w = static_cast<const uint8_t*>(c.d < D ? p.w13 : p.w13s);
        row = (c.d < D ? static_cast<size_t>(f.expert[c.d]) * 2 * I : 0) + c.n + (lane ? I : 0);
      } else {
        w = static_cast<const uint8_t*>(c.d < D ? p.w2 : p.w2s);
        row = (c.d < D ? static_cast<size_t>(f.expert[c.d]) * p.H : 0) + col0 + c.i + lane;
      }
      bulk_load(slot + lane * kPiece, w + row * row_bytes + static_cast<size_t>(c.k) * (q ? 1 : 2), bytes, bar);
    }
  }
};

// two exact bf16 products added to an f32 sum, low halves first
__device__ __forceinline__ float fma_bf16x2(uint32_t a, uint32_t b, float c) {
  float d;
  asm("{\n\t.reg .b16 al, ah, bl, bh;\n\t.reg .f32 t;\n\t"
      "mov.b32 {al, ah}, %1;\n\tmov.b32 {bl, bh}, %2;\n\t"
      "fma.rn.f32.bf16 t, al, bl, %3;\n\tfma.rn.f32.bf16 %0, ah, bh, t;\n\t}"
      : "=f"(d) : "r"(a), "r"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void widen_bf16(const uint4& u, float (&w)[8]) {
  const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[2 * i] = __uint_as_float(q[i] << 16);
    w[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void load_e4m3(uint32_t a, float (&w)[8]) {
  uint32_t u[2];
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(u[0]), "=r"(u[1]) : "r"(a) : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(u[i >> 1] >> (16 * (i & 1))), __NV_E4M3));
    w[2 * i] = __low2float(h);
    w[2 * i + 1] = __high2float(h);
  }
}

// Sums v[n] over the warp's lanes, n a power of two up to 32: lane l ends with the sum
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

// A warp's ring
struct Ring {
  uint32_t slots, bars;            // shared addresses of slot 0 and its barrier
  int s;
  uint32_t phase;
};

// One item: a feature (kDown false: rows gate and up) or two output columns (kDown) of one
// expert, for its NT tokens (padded by repeating the last): all pieces of the two rows.  Returns the
// sum of row r and token t, value 2 t + r, in lane (2 t + r) * 16 / NT.
template <int NT, bool kQ, bool kDown, bool kFp8>
__device__ __forceinline__ float item(const Stream<kFp8>& st, Ring& ring, Cursor& c, Cursor& ahead, int n_tok,
                                      volatile int* abort_flag) {
  const Params& p = st.p;
  const Fixed& f = st.f;
  const int lane = st.lane, C = st.row_cols(c), per = kQ ? kPiece : kPiece / 2;
  // the tokens' rows (tokens, or f32 activations)
  const int first = f.first[c.d];
  const uint8_t* src[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int at = first + min(t, n_tok - 1);
    if (!kDown) src[t] = reinterpret_cast<const uint8_t*>(p.x + static_cast<size_t>(f.token[at]) * C);
    else if (c.d < st.D) src[t] = reinterpret_cast<const uint8_t*>(p.act + static_cast<size_t>(f.pair[at]) * C);
    else src[t] = reinterpret_cast<const uint8_t*>(p.act_s + static_cast<size_t>(f.token[at]) * C);
  }
  const float *sc0 = nullptr, *sc1 = nullptr;
  if (kQ) {
    const int nblk = (C + 127) >> 7, R = kDown ? p.H : 2 * p.I;
    const float* base = (kDown ? p.s2 : p.s13) + static_cast<size_t>(f.expert[c.d]) * ((R + 127) >> 7) * nblk;
    const int r0 = kDown ? st.col0 + c.i : c.n, r1 = kDown ? min(r0 + 1, p.H - 1) : p.I + c.n;
    sc0 = base + static_cast<size_t>(r0 >> 7) * nblk;
    sc1 = base + static_cast<size_t>(r1 >> 7) * nblk;
  }
  float acc[2 * NT];
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) acc[i] = 0.0f;
  for (int k = 0; k < C; k += per) {
    const int n = min(per, C - k);
    const bool landed = __all_sync(0xffffffffu, wait(ring.bars + 8 * ring.s, ring.phase, abort_flag, p));
    const uint32_t at = ring.slots + ring.s * kSlotBytes + lane * (kQ ? 8 : 16);
#pragma unroll(NT <= 2 ? 4 : NT <= 4 ? 2 : 1)
    for (int c0 = 0; c0 < n; c0 += kSeg) {
      const int col = c0 + lane * 8;
      if (col >= n) break;
      const uint32_t a = at + c0 * (kQ ? 1 : 2);
      if (!kQ && !kDown) {
        const uint4 g = ptx::ld_shared_v4(a), u = ptx::ld_shared_v4(a + kPiece);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(src[t]) + ((k + col) >> 3));
          acc[2 * t] = fma_bf16x2(x.x, g.x, acc[2 * t]);
          acc[2 * t + 1] = fma_bf16x2(x.x, u.x, acc[2 * t + 1]);
          acc[2 * t] = fma_bf16x2(x.y, g.y, acc[2 * t]);
          acc[2 * t + 1] = fma_bf16x2(x.y, u.y, acc[2 * t + 1]);
          acc[2 * t] = fma_bf16x2(x.z, g.z, acc[2 * t]);
          acc[2 * t + 1] = fma_bf16x2(x.z, u.z, acc[2 * t + 1]);
          acc[2 * t] = fma_bf16x2(x.w, g.w, acc[2 * t]);
          acc[2 * t + 1] = fma_bf16x2(x.w, u.w, acc[2 * t + 1]);
        }
      } else {
        float w0[8], w1[8];
        float d0 = 1.0f, d1 = 1.0f;
        if (kQ) {
          load_e4m3(a, w0);
          load_e4m3(a + kPiece, w1);
          d0 = __ldg(sc0 + ((k + col) >> 7));
          d1 = __ldg(sc1 + ((k + col) >> 7));
        } else {
          widen_bf16(ptx::ld_shared_v4(a), w0);
          widen_bf16(ptx::ld_shared_v4(a + kPiece), w1);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float x[8];
          if (kDown) {             // written by other SMs before the grid barrier: not the read-only path
            const float4* q = reinterpret_cast<const float4*>(src[t]) + ((k + col) >> 2);
            const float4 lo = q[0], hi = q[1];
            x[0] = lo.x; x[1] = lo.y; x[2] = lo.z; x[3] = lo.w;
            x[4] = hi.x; x[5] = hi.y; x[6] = hi.z; x[7] = hi.w;
          } else {
            widen_bf16(__ldg(reinterpret_cast<const uint4*>(src[t]) + ((k + col) >> 3)), x);
          }
          float s0 = kQ ? 0.0f : acc[2 * t], s1 = kQ ? 0.0f : acc[2 * t + 1];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            s0 = fmaf(x[i], w0[i], s0);
            s1 = fmaf(x[i], w1[i], s1);
          }
          acc[2 * t] = kQ ? fmaf(s0, d0, acc[2 * t]) : s0;
          acc[2 * t + 1] = kQ ? fmaf(s1, d1, acc[2 * t + 1]) : s1;
        }
      }
    }
    __syncwarp();                  // all lanes have read the slot
    if (landed) st.issue(ahead, ring.slots + ring.s * kSlotBytes, ring.bars + 8 * ring.s);
    if (ahead.phase < 2) st.next_piece(ahead);
    if (++ring.s == kSlots) {
      ring.s = 0;
      ring.phase ^= 1u;
    }
  }
  return transpose_sum<2 * NT>(acc, lane);
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
layer_few_kernel(const Params p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Fixed& f = *reinterpret_cast<Fixed*>(smem_raw);
  float* out_sum = reinterpret_cast<float*>(smem_raw + sizeof(Fixed));   // [2][T][rows_max]
  const uint32_t ring_off = (sizeof(Fixed) + 2u * p.T * p.rows_max * 4u + 127u) & ~127u;
  uint8_t* slots = smem_raw + ring_off;
  volatile int* abort_flag = &f.abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = p.T, H = p.H, E = p.E, K = p.K;

  count_launch(p.launches, MOE_KID_LAYER_FEW);
  if (lane < kSlots) ptx::mbar_init(ptx::smem_u32(&f.full[warp][lane]), 1);
  if (tid == 0) f.abort_flag = 0;
  ptx::fence_mbar_init();
  for (int e = tid; e < E; e += kThreads) f.mask[e] = 0u;
  for (int i = tid; i < 2 * T * p.rows_max; i += kThreads) out_sum[i] = 0.0f;
  grid_dep_wait();
  grid_dep_launch();

  // ---- logits, and the shared expert's gate logits as one more row
  {
    const int rows = E + (p.w_gate ? 1 : 0), halves = (T + route::kTokWarp - 1) / route::kTokWarp;
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
  if (tid == 0) grid_barrier(abort_flag, p);
  __syncthreads();

  // ---- choice of experts
  if (warp < T) {
    float* v = reinterpret_cast<float*>(slots) + static_cast<size_t>(warp) * 2 * E;
    choose(p, f, warp, lane, v, v + E);
  }
  if (tid < T) f.gate[tid] = p.w_gate ? sigmoid_f32(__ldcg(p.gate + tid)) : 1.0f;
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

  // ---- the experts
  const Stream<kFp8> st(p, f, warp, lane);
  const int D = st.D;
  Ring ring{ptx::smem_u32(slots) + warp * kSlots * kSlotBytes, ptx::smem_u32(&f.full[warp][0]), 0, 0u};
  Cursor c = st.begin(), ahead = c;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    st.issue(ahead, ring.slots + s * kSlotBytes, ring.bars + 8 * s);
    if (ahead.phase < 2) st.next_piece(ahead);
  }
  // an item for tokens [0, n_tok) of its expert; lane (2 t + r) * 16 / NT gets row r, token t
  auto run = [&](auto down, auto nt, int n_tok) {
    constexpr bool kDown = decltype(down)::value;
    constexpr int NT = decltype(nt)::value;
    const float v = kFp8 && c.d < D ? item<NT, kFp8, kDown>(st, ring, c, ahead, n_tok, abort_flag)
                                    : item<NT, false, kDown>(st, ring, c, ahead, n_tok, abort_flag);
    constexpr int kRep = 16 / NT;            // lanes that hold the same sum
    const int t = lane / (2 * kRep), r = lane / kRep & 1, pair = f.first[c.d] + t;
    if (kDown) {
      if (lane % kRep == 0 && t < n_tok && c.i + r < st.cols) {
        const int tok = f.token[pair];
        const float w = c.d < D ? f.weight[f.pair[pair]] : f.gate[tok];
        float* o = out_sum + ((warp >> 3) * T + tok) * p.rows_max + c.i + r;
        *o = fmaf(w, v, *o);
      }
    } else {
      const float up = __shfl_down_sync(0xffffffffu, v, kRep);
      if (lane % (2 * kRep) == 0 && t < n_tok) {
        const float a = v / (1.0f + __expf(-v)) * up;
        if (c.d < D) p.act[static_cast<size_t>(f.pair[pair]) * p.I + c.n] = a;
        else p.act_s[static_cast<size_t>(f.token[pair]) * p.Is + c.n] = a;
      }
    }
  };
  auto each = [&](auto down) {
    const int n_tok = f.first[c.d + 1] - f.first[c.d];
    if (n_tok == 1) run(down, std::integral_constant<int, 1>{}, n_tok);
    else if (n_tok == 2) run(down, std::integral_constant<int, 2>{}, n_tok);
    else if (n_tok <= 4) run(down, std::integral_constant<int, 4>{}, n_tok);
    else if (n_tok <= 8) run(down, std::integral_constant<int, 8>{}, n_tok);
    else run(down, std::integral_constant<int, 16>{}, n_tok);
    st.next_item(c);
  };
  while (c.phase == 0) each(std::false_type{});
  __syncthreads();
  if (tid == 0) grid_barrier(abort_flag, p);
  __syncthreads();
  while (c.phase == 1) each(std::true_type{});
  __syncthreads();

  // ---- both halves' sums, the residual, one rounding
  for (int i = tid; i < T * st.cols; i += kThreads) {
    const int t = i / st.cols, r = i - t * st.cols;
    float v = out_sum[t * p.rows_max + r] + out_sum[(T + t) * p.rows_max + r];
    const size_t at = static_cast<size_t>(t) * H + st.col0 + r;
    if (p.residual) v += bf16_bits_to_f32(p.residual[at]);
    p.out[at] = f32_to_bf16_bits(v);
  }
  // a CTA that gave up lets its copies land before it ends
  if (*abort_flag) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - t0 < kCopyGraceNs) {
    }
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
  const int fixed = (static_cast<int>(sizeof(Fixed)) + 2 * p.T * p.rows_max * 4 + 127) & ~127;
  constexpr int kSmem = 227 * 1024;
  const int scores = 2 * p.T * p.E * 4;      // of the choice, in the ring
  const int smem = fixed + (scores > kRing ? scores : kRing);
  if (smem > kSmem) return set_error(MOE_ERR_CUDA, "%s: %d SMs leave no room for the ring", op, ctas);
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
