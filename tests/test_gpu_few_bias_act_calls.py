"""Calls around the few-token layer and the products with an epilogue that their other tests do not make:
graphs that share a workspace, programmatic launch off, weights of experts that nobody chose, no tokens."""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m
from mixture_experts_ffn_renorm_gb300 import workloads as W
from mixture_experts_ffn_renorm_gb300.layer import MoeBlock, MoeMlpBlock, _dev_bf16

from .gpu_util import DEV
from .test_gpu_bias_act import Back, Product, Wgrad, offsets, ws_of
from .test_gpu_layer_few import Case

pytestmark = pytest.mark.gpu


def captured(call):
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    return g


def test_graphs_that_share_a_workspace():
    cases = [Case(1, 1032, 400, 60, 6), Case(16, 2048, 768, 128, 8), Case(5, 264, 72, 12, 3, Is=64)]
    ws = torch.zeros(max(c.ws.numel() for c in cases), dtype=torch.uint8, device=DEV)
    for c in cases:
        c.ws = ws
    products = [Product(20, 4096, 520, columns=True, residual=True, seed=1), Product(100, 2048, 264, columns=True, seed=2)]
    shared = ws_of(max(p.ws.numel() for p in products))
    for p in products:
        p.ws = shared
    both = cases + products
    want = [c.call().clone() for c in both]
    graphs = [captured(c.call) for c in both]
    for k in range(5):
        for c in both:
            c.out.zero_()
        for i in ([4, 0, 3, 1, 2], [0, 1, 2, 3, 4])[k % 2]:
            graphs[i].replay()
        cases[k % 3].call()                          # and a call of its own in between
        for c, w in zip(both, want):
            assert torch.equal(c.out, w)
    assert m.moe_device_status() == 0


def test_programmatic_launch_off_gives_the_same_bits():
    layer, few, pair = (Case(7, 1032, 400, 60, 6, Is=64), Product(3, 520, 264),
                        Product(40, 2048, 264, columns=True, residual=True))
    back = Back(900, 520, 3, offsets([100, 0, 800]), scatter=True, weight=True)
    grad = Wgrad(300, 136, 264, 2, offsets([170, 130]), add=True)
    one = Wgrad(3000, 136, 264, 1)                   # ranges of rows
    calls = [(layer.call, (layer.out, layer.ids, layer.w)), (few.call, (few.out,)), (pair.call, (pair.out,)),
             (back.call, (back.dz, back.db, back.dpw)), (grad.call, (grad.dw,)), (one.call, (one.dw,))]
    for call, _ in calls:
        call()
    want = [[o.clone() for o in outs] for _, outs in calls]
    try:
        m.moe_set_pdl(False)
        for call, outs in calls:
            for o in outs:
                o.zero_()
            call()
    finally:
        m.moe_set_pdl(True)
    torch.cuda.synchronize()
    for (_, outs), w in zip(calls, want):
        for o, v in zip(outs, w):
            assert torch.equal(o, v)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("size", [(3, 1040, 400, 16, 2), (1, 144, 48, 9, 1), (9, 16, 16, 30, 1)], ids=str)
def test_weights_of_experts_that_nobody_chose_are_not_used(fp8, size):
    # rows end inside a block of 128 bytes: what lies behind them is the next row's
    c = Case(*size, fp8=fp8, Is=72)
    c.call()
    torch.cuda.synchronize()
    want = c.out.clone()
    idle = torch.ones(size[3], dtype=torch.bool, device=DEV)
    idle[c.ids.flatten().long()] = False
    assert idle.any()
    bad = 0x7F if fp8 else float("nan")
    c.w13[idle] = bad
    c.w2[idle] = bad
    c.call()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want)


def test_a_nan_row_of_weights_stays_in_its_column():
    # output column 5 of the expert's second product, and a token that did not choose the expert
    c = Case(2, 136, 72, 8, 1, residual=False, bias=False)
    c.call()
    torch.cuda.synchronize()
    want, e = c.out.clone(), int(c.ids[0, 0])
    c.w2[e, 5] = float("nan")
    c.call()
    torch.cuda.synchronize()
    hit = (c.ids == e).any(1)
    assert c.out[hit, 5].isnan().all()
    keep = torch.ones_like(c.out, dtype=torch.bool)
    keep[hit, 5] = False
    assert torch.equal(c.out[keep], want[keep])


def test_no_tokens():
    cfg = W.TINY
    d = W.layer_inputs(cfg)
    blk = MoeBlock(cfg.H, cfg.I, cfg.E, cfg.K, d, max_tokens=4, device=DEV, I_shared=cfg.I_shared, few=True)
    x = _dev_bf16(d["x"], DEV)[:4].contiguous()
    assert blk.forward(x[:0]).shape == (0, cfg.H)
    assert blk.forward(x).isfinite().all()
    g = torch.Generator(device=DEV).manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g, device=DEV).to(torch.bfloat16)
    mlp = MoeMlpBlock(64, 32, 4, 2, {"w_router": n(4, 64), "w1": n(4, 32, 64), "w2": n(4, 64, 32)}, max_tokens=8,
                      device=DEV, training=True)
    x = n(8, 64)
    mlp.forward(x)
    for bad in (x[:0], n(9, 64)):
        with pytest.raises(ValueError, match="tokens, outside"):
            mlp.forward(bad)
    assert mlp.backward(x, x)["grad_x"].isfinite().all()     # of the last forward that ran
    assert m.moe_device_status() == 0
