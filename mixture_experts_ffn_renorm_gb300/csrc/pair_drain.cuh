// pair_drain.cuh -- how a CTA pair that gave up lets its copies land before it ends.
//
// Both CTAs of a pair copy their own half of a stage, and both halves are counted on the even CTA's
// barrier of the stage, which the even CTA arms for all of the bytes as it issues its own.  When a wait
// ran out, one CTA may have issued copies for uses of the ring that the other never came to: such a
// use's barrier would count bytes that nobody brings, or was never armed for those that are under way.
// Once both CTAs have left their loops, the even one settles these accounts, so that a barrier's phase
// ends exactly when the last copy under way has landed, and waits for it.
//
// A use of a stage (numbered from 0 through the launch; use i is of stage i % stages) waits for the use before it
// of the same stage to be consumed, in either CTA, and that takes everything which arrives on its barrier.  So no role is more
// than `stages` uses ahead of another, and only the last `stages` uses can be unfinished.
#pragma once

#include "gemm_common.cuh"

namespace moe {
namespace gemm {

struct StageDebt {
  bool open;            // copies of this use may be under way
  uint32_t expect;      // bytes to arm the barrier with, one arrival; 0: it is armed
  uint32_t complete;    // armed bytes that nobody will bring
};

// use i of a pair whose CTAs issued the uses below `even` and `odd`, `bytes` of them each a use
__host__ __device__ __forceinline__ StageDebt stage_debt(uint32_t i, uint32_t even, uint32_t odd, uint32_t bytes) {
  StageDebt d;
  d.open = i < even || i < odd;
  d.expect = d.open && i >= even ? bytes : 0u;
  d.complete = d.open && i >= odd ? bytes : 0u;
  return d;
}

// Rows that are gathered: besides the arming arrival a use's barrier counts one of each thread of the even CTA's two
// gatherer warps and one of the odd CTA's relay.  Those that use i lacks, of roles that came through so many uses:
__host__ __device__ __forceinline__ uint32_t gather_debt(uint32_t i, uint32_t warp0, uint32_t warp1, uint32_t relay) {
  return (i >= warp0 ? 32u : 0u) + (i >= warp1 ? 32u : 0u) + (i >= relay ? 1u : 0u);
}

// One thread of the even CTA, after both CTAs' roles have ended.  bar(s): stage s's barrier; bytes(i): one CTA's
// bytes of use i; arrivals(i): arrivals besides the arming one that use i's barrier still lacks.
template <int kStages, typename Bar, typename Bytes, typename Arrivals>
__device__ __forceinline__ void drain_pair_copies(uint32_t even, uint32_t odd, Bar&& bar, Bytes&& bytes,
                                                  Arrivals&& arrivals) {
  const uint32_t n = even > odd ? even : odd, first = n < kStages ? 0u : n - kStages;
#pragma unroll 1
  for (uint32_t i = first; i < n; ++i) {
    const StageDebt d = stage_debt(i, even, odd, bytes(i));
    const uint32_t b = bar(i % kStages);
    if (d.complete) ptx::mbar_complete_tx(b, d.complete);
    if (d.expect) ptx::mbar_arrive_expect_tx(b, d.expect);
    for (uint32_t k = arrivals(i); k > 0; --k) ptx::mbar_arrive(b);
  }
#pragma unroll 1
  for (uint32_t i = first; i < n; ++i) spin_bounded(bar(i % kStages), (i / kStages) & 1u);
}

}  // namespace gemm
}  // namespace moe
