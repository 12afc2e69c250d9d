"""The bounded waits of the FP8 products and of the router's gradient, made to run out.

At a limit of 1 us a launch over large inputs cannot finish: the first tiles alone take longer to
arrive from memory.  Each kernel must still end, raise MOE_STATUS_TIMEOUT and leave the device
usable: with the limit restored, the same calls give the same bits as before.
"""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m

from .gpu_util import DEV, launched_since, launches

pytestmark = pytest.mark.gpu

FULL_LIMIT_NS = 10**9


@pytest.fixture(autouse=True)
def _restore_limit():
    m.lib()
    m.moe_device_status(clear=True)
    yield
    m.moe_set_wait_limit_ns(FULL_LIMIT_NS)
    m.moe_device_status(clear=True)


def fp8_calls(rows):
    """gate/up and down of 8 groups of `rows` rows (rows and weights tiles)"""
    g = torch.Generator(device=DEV).manual_seed(rows)
    G, H, I = 8, 2048, 2048
    P = G * rows
    off = torch.arange(0, P + 1, rows, dtype=torch.int32, device=DEV)
    code = lambda *s: torch.randint(0, 0x70, s, generator=g, device=DEV, dtype=torch.uint8)
    ones = lambda *s: torch.rand(s, generator=g, device=DEV) * 1e-3
    a, asc, w13, s13 = code(P, H), ones(P, H // 128), code(G, 2 * I, H), ones(G, 2 * I // 128, H // 128)
    w2, s2 = code(G, H, I), ones(G, H // 128, I // 128)
    act, act_s = torch.zeros_like(a), torch.zeros_like(asc)
    gu = torch.zeros((P, 2 * I), dtype=torch.bfloat16, device=DEV)
    y = torch.zeros((P, H), dtype=torch.bfloat16, device=DEV)
    return {
        "gemm_fp8_gateup": (lambda: m.moe_grouped_gemm_gateup_silu_fp8(a, asc, w13, s13, off, P, H, I, G, gu, act, act_s),
                            (act, act_s, gu)),
        "gemm_fp8": (lambda: m.moe_grouped_gemm_fp8(a, asc, w2, s2, off, None, None, P, I, H, G, y), (y,)),
    }


def route_calls(T):
    g = torch.Generator(device=DEV).manual_seed(T)
    H, E = 2048, 256
    dl = torch.randn((T, E), generator=g, device=DEV)
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn((E, H), generator=g, device=DEV).to(torch.bfloat16)
    ws = torch.zeros(m.moe_route_logits_backward_workspace_size(T, H, E), dtype=torch.uint8, device=DEV)
    dx = torch.zeros_like(x)
    dw = torch.zeros((E, H), device=DEV)
    db = torch.zeros((E,), device=DEV)
    call = lambda *o: m.moe_route_logits_backward(dl, x, w, T, H, E, *o, ws, ws.numel())
    return {"route_dx": (lambda: call(dx, None, None), (dx,)), "route_dw": (lambda: call(None, dw, db), (dw, db))}


@pytest.mark.parametrize("calls,size", [(fp8_calls, 1024), (fp8_calls, 48), (route_calls, 8192)],
                         ids=["fp8-rows", "fp8-weights", "route"])
def test_expiry_is_reported_and_the_device_stays_usable(calls, size):
    cold = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    for kid, (call, outs) in calls(size).items():
        call()
        assert m.moe_device_status() == 0
        want = [o.clone() for o in outs]
        m.moe_set_wait_limit_ns(1000)
        cold.zero_()                            # the inputs leave the L2
        torch.cuda.synchronize()
        before = launches()
        assert call() == m.OK                   # the launch itself is accepted
        torch.cuda.synchronize()                # and the kernel ends
        assert launched_since(before, kid) >= 1
        assert m.moe_device_status(clear=True) & m.STATUS_TIMEOUT, kid
        m.moe_set_wait_limit_ns(FULL_LIMIT_NS)
        for o in outs:
            o.zero_()
        call()
        assert m.moe_device_status() == 0
        for o, v in zip(outs, want):
            assert torch.equal(o, v), kid
