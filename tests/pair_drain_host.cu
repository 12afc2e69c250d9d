// Host build of stage_debt and gather_debt (csrc/pair_drain.cuh) for tests/test_pair_drain_host.py.
#include "pair_drain.cuh"

extern "C" void stage_debt_host(unsigned i, unsigned even, unsigned odd, unsigned bytes, unsigned* out) {
  const moe::gemm::StageDebt d = moe::gemm::stage_debt(i, even, odd, bytes);
  out[0] = d.open ? 1u : 0u;
  out[1] = d.expect;
  out[2] = d.complete;
}

extern "C" unsigned gather_debt_host(unsigned i, unsigned warp0, unsigned warp1, unsigned relay) {
  return moe::gemm::gather_debt(i, warp0, warp1, relay);
}
