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
