"""CTA pairs whose waits ran out: each launch ends promptly, which it does only where the accounts of both
CTAs' copies are settled so that every stage's barrier still completes (a barrier that did not would be waited
for a second), and leaves the next calls their bits.  Limits from 1 to 30 us end the roles at different
places of the ring."""
from __future__ import annotations

import time

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m

from .gpu_util import DEV
from .test_gpu_bias_act import Product, offsets

pytestmark = pytest.mark.gpu

FULL_LIMIT_NS = 10**9


@pytest.fixture(autouse=True)
def _restore_limit():
    m.lib()
    m.moe_device_status(clear=True)
    yield
    m.moe_set_wait_limit_ns(FULL_LIMIT_NS)
    m.moe_device_status(clear=True)


def run_out(call, outs):
    call()
    torch.cuda.synchronize()
    assert m.moe_device_status() == 0
    want = [o.clone() for o in outs]
    gave_up = 0
    for limit in (1000, 1500, 2000, 3000, 5000, 10000, 30000):
        for _ in range(6):
            torch.zeros(1 << 28, dtype=torch.uint8, device=DEV)     # the inputs leave L2
            torch.cuda.synchronize()
            m.moe_set_wait_limit_ns(limit)
            t0 = time.perf_counter()
            call()
            torch.cuda.synchronize()
            assert time.perf_counter() - t0 < 0.5, limit
            gave_up += bool(m.moe_device_status(clear=True) & m.STATUS_TIMEOUT)
            m.moe_set_wait_limit_ns(FULL_LIMIT_NS)
        for o in outs:
            o.zero_()
        call()
        torch.cuda.synchronize()
        assert m.moe_device_status() == 0
        for o, w in zip(outs, want):
            assert torch.equal(o, w), limit
    assert gave_up >= 6


@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("sizes", [None, [700, 0, 3, 900, 33, 1400, 257, 64]])      # boxes of every height
def test_product(columns, sizes):
    P = 4000 if sizes is None else sum(sizes)
    c = Product(P, 2048, 4096, len(sizes) if sizes else 1, offsets(sizes) if sizes else None, columns, residual=True, pre=True)
    run_out(c.call, (c.out, c.pre))


def test_product_in_ranges_of_k():
    c = Product(500, 8192, 1024, columns=True, residual=True)       # and their join
    run_out(c.call, (c.out,))


class Experts:
    """gate/up and down of the block's experts, [group][rows] of x taken as they lie."""

    def __init__(self, sizes, H, I):
        g = torch.Generator(device=DEV).manual_seed(len(sizes))
        n = lambda *s, std=1.0: (torch.randn(s, generator=g, device=DEV) * std).to(torch.bfloat16)
        self.G, self.P, self.H, self.I = len(sizes), sum(sizes), H, I
        self.off = offsets(sizes)
        self.x, self.w13, self.w2 = n(self.P, H), n(self.G, 2 * I, H, std=H ** -0.5), n(self.G, H, I, std=I ** -0.5)
        self.act, self.rows, self.out = n(self.P, I), n(self.P, H), n(self.P, H)
        self.ident = torch.arange(self.P, dtype=torch.int32, device=DEV)
        self.ws = torch.zeros(m.moe_gateup_staged_workspace_size(self.P), dtype=torch.uint8, device=DEV)

    def gateup(self, gather=None):
        m.moe_grouped_gemm_gateup_silu_bf16(self.x, self.P, gather, 1, self.w13, self.off, self.P, self.H, self.I, self.G, self.act)

    def gathered(self):
        self.gateup(self.ident)

    def staged(self):
        m.moe_grouped_gemm_gateup_silu_bf16_staged(self.x, self.P, self.ident, 1, self.rows, self.w13, self.off, self.P,
                                                   self.H, self.I, self.G, self.act, self.ws, self.ws.numel())

    def down(self):
        m.moe_grouped_gemm_down_bf16(self.act, self.w2, self.off, None, None, self.P, self.I, self.H, self.G, self.out)


@pytest.mark.parametrize("call", ["gateup", "gathered", "staged", "down"])
@pytest.mark.parametrize("sizes", [[1024] * 8, [900, 0, 7, 1400, 33, 257, 30, 64, 2000, 129]], ids=["even", "ragged"])
def test_experts(sizes, call):
    prev = m.moe_set_gemm_pairing(m.GEMM_PAIR)
    try:
        e = Experts(sizes, 2048, 2048)
        run_out(getattr(e, call), (e.out,) if call == "down" else (e.act,))
    finally:
        m.moe_set_gemm_pairing(prev)
