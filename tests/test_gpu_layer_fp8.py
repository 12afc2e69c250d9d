"""The MoE block with FP8 activations: forward, and the gradients of router and tokens.

forward() is compared bit for bit with its own calls made one by one, and with a 64-bit layer on
the same routing and the dequantised weights.  An E4M3 rounding is at most 2^-4 of a value, with
a mean square of about (2^-5)^2 over a binade; a forward rounds two operands (tokens, activations),
so its relative error in the 2-norm stays under 2 * 2^-4 = 0.125 even if all roundings conspired,
and the gradient of the tokens, which rounds two more (0.25 in all), under 0.375.  The gradient of
the routing weights sees the forward's two roundings (0.125), and the router's gradients are exact
functions of it.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m
from mixture_experts_ffn_renorm_gb300 import workloads as W
from mixture_experts_ffn_renorm_gb300.layer import MoeBlock

from . import ref_fp8 as R
from .gpu_util import DEV, to_dev

pytestmark = pytest.mark.gpu


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def problem(T, H, I, E, K, training, seed=0, scale=1.0):
    cfg = W.LayerConfig("fp8", T=T, H=H, I=I, E=E, K=K, seed=seed)
    d = W.layer_inputs(cfg)
    d["logit_bias"] = np.linspace(-0.3, 0.3, E).astype(np.float32)
    d["w13_e4m3"], d["w13_scale"] = W.quantize_fp8_block(d["w13"])
    d["w2_e4m3"], d["w2_scale"] = W.quantize_fp8_block(d["w2"])
    blk = MoeBlock(H, I, E, K, d, max_tokens=T + 3, fp8_weights=True, fp8_acts=True, training=training,
                   routed_scale=scale)
    return blk, to_dev(d["x"]), d


def layer64(blk, x, ids):
    """(out, leaves) of the block in f64 on given expert ids, differentiable."""
    x = x.double().cpu().requires_grad_()
    wr = blk.w_router.double().cpu().requires_grad_()
    bias = blk.logit_bias.double().cpu().requires_grad_()
    l = x @ wr.t() + bias
    ids = ids.long().cpu()
    w = torch.softmax(l.gather(1, ids), 1)
    w.retain_grad()
    w13 = R.weight_values(blk.w13_q.cpu(), blk.w13_s.cpu())
    w2 = R.weight_values(blk.w2_q.cpu(), blk.w2_s.cpu())
    out = torch.zeros_like(x)
    for e in range(blk.E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            g, u = (x[t] @ w13[e].t()).split(blk.I, 1)
            y = (torch.nn.functional.silu(g) * u) @ w2[e].t()
            out = out.index_add(0, t, y * w[t, j][:, None] * blk.routed_scale)
    return out, l, w, (x, wr, bias)


@pytest.mark.parametrize("T,H,I,E,K", [(1, 128, 64, 8, 2), (16, 256, 128, 16, 4), (70, 272, 144, 5, 3),
                                       (300, 512, 256, 12, 2)])
@pytest.mark.parametrize("training", [False, True])
def test_forward(T, H, I, E, K, training):
    blk, x, _ = problem(T, H, I, E, K, training, scale=0.5)
    m.moe_device_status(clear=True)
    out = blk.forward(x).clone()
    want, l, w, _ = layer64(blk, x, blk.topk_ids[:T])
    assert rel(out.cpu(), want.detach()) < 0.125
    # again, one call at a time
    P = T * K
    xq, xs = torch.empty_like(blk.x_q), torch.empty_like(blk.x_s)
    m.moe_quantize_act_fp8(x, T, H, K, blk.pair_to_row, None, 1.0, xq, xs)
    aq, as_ = torch.empty_like(blk.act_q), torch.empty_like(blk.act_s)
    m.moe_grouped_gemm_gateup_silu_fp8(xq, xs, blk.w13_q, blk.w13_s, blk.expert_offsets, P, H, I, E, None, aq, as_)
    y = torch.empty_like(blk.expert_out)
    m.moe_grouped_gemm_fp8(aq, as_, blk.w2_q, blk.w2_s, blk.expert_offsets, None if training else blk.topk_w,
                           blk.sorted_pair, P, I, H, E, y)
    again = torch.empty_like(out)
    m.moe_combine(y, m.BF16, blk.topk_w if training else None, None, m.BF16, 0.5, T, K, H, again, m.BF16)
    assert torch.equal(out, again)
    # and replayed from a CUDA graph
    blk.capture(x)
    assert torch.equal(blk.replay(), out)
    assert m.moe_device_status() == 0


@pytest.mark.parametrize("T,H,I,E,K", [(1, 128, 64, 8, 2), (70, 272, 144, 5, 3), (300, 512, 256, 12, 2)])
def test_backward(T, H, I, E, K):
    blk, x, _ = problem(T, H, I, E, K, True, scale=0.5)
    g = torch.Generator().manual_seed(T)
    dout = (torch.randn((T, H), generator=g) * 0.1).to(torch.bfloat16).to(DEV)
    bal, z = 0.02, 0.003
    blk.forward(x)
    got = {k: v.clone().cpu() for k, v in blk.backward(x, dout, bal, z).items()}
    out, l, w, (xl, wr, bias) = layer64(blk, x, blk.topk_ids[:T])
    ids = blk.topk_ids[:T].long().cpu()
    _, lb, lz = R.route(l, ids, 1, 0, blk.expert_offsets.cpu(), bal, z)
    ((out * dout.double().cpu()).sum() + lb + lz).backward()
    if T * K > 2:
        assert rel(got["grad_topk_w"], w.grad) < 0.125
        assert rel(got["grad_w_router"], wr.grad) < 0.125
        assert rel(got["grad_logit_bias"], bias.grad) < 0.125
    assert rel(got["grad_x"], xl.grad) < 0.375
    assert torch.allclose(got["losses"].double(), torch.stack([lb, lz]).detach(), rtol=1e-4)
    # the router's part is exact given the routing weights' gradient
    ld = blk.logits[:T].cpu().double().requires_grad_()
    w64, lb, lz = R.route(ld, ids, 1, 0, blk.expert_offsets.cpu(), bal, z)
    (dl,) = torch.autograd.grad((w64 * got["grad_topk_w"].double()).sum() + lb + lz, ld)
    assert rel(got["grad_w_router"], dl.t() @ x.double().cpu()) < 1e-5
    assert rel(got["grad_logit_bias"], dl.sum(0)) < 1e-5
    # the same bits again, with other work on the device's other streams
    blk.forward(x)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        junk = torch.randn(1 << 20, device=DEV)
        for _ in range(20):
            junk = junk * 1.0001
    again = blk.backward(x, dout, bal, z)
    for k, v in got.items():
        assert torch.equal(again[k].cpu(), v), k


@pytest.mark.parametrize("T", [3, 80])
def test_shared_expert_beside_fp8_activations(T):
    # the shared expert stays bf16: the block's output is the routed part plus the gated shared rows
    cfg = W.LayerConfig("s", T=T, H=256, I=128, E=8, K=2, I_shared=64)
    d = W.layer_inputs(cfg)
    d["w13_e4m3"], d["w13_scale"] = W.quantize_fp8_block(d["w13"])
    d["w2_e4m3"], d["w2_scale"] = W.quantize_fp8_block(d["w2"])
    blk = MoeBlock(256, 128, 8, 2, d, I_shared=64, max_tokens=T, fp8_weights=True, fp8_acts=True)
    x = to_dev(d["x"])
    out = blk.forward(x)
    blk.logit_bias = torch.zeros(8, device=DEV)
    want, *_ = layer64(blk, x, blk.topk_ids[:T])
    xd = x.double().cpu()
    g, u = (xd @ blk.w13_shared[0].double().cpu().t()).split(64, 1)
    y = (torch.nn.functional.silu(g) * u) @ blk.w2_shared[0].double().cpu().t()
    gate = torch.sigmoid(xd @ blk.w_shared_gate.double().cpu().reshape(-1, 1))
    assert rel(out.cpu(), (want + gate * y).detach()) < 0.125


def test_block_refuses_what_it_lacks():
    cfg = W.LayerConfig("r", T=4, H=64, I=32, E=4, K=2)
    d = W.layer_inputs(cfg)
    d["w13_e4m3"], d["w13_scale"] = W.quantize_fp8_block(d["w13"])
    d["w2_e4m3"], d["w2_scale"] = W.quantize_fp8_block(d["w2"])
    make = lambda **k: MoeBlock(64, 32, 4, 2, d, max_tokens=4, **k)
    for bad in (dict(fp8_acts=True), dict(training=True), dict(fp8_weights=True, training=True)):
        with pytest.raises(ValueError):
            make(**bad)
    blk = make(fp8_weights=True, fp8_acts=True)
    x = to_dev(d["x"])
    blk.forward(x)
    with pytest.raises(ValueError, match="training"):
        blk.backward(x, x)


def test_router_tuning_example_learns():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import tune_router as ex

    cfg = W.LayerConfig("tune", T=512, H=256, I=128, E=16, K=4, seed=3)
    blk, x, target = ex.build(cfg, cfg.T)
    errors = [e for e, _, _ in ex.tune(blk, x, target, 40, 0.02)]
    assert errors[-1] < 0.7 * errors[0], errors
