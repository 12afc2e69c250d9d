"""MoeMlpBlock: forward and all gradients against autograd in 64 bits, and MoeBlock(few=True) against
the block's separate launches."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m
from mixture_experts_ffn_renorm_gb300 import workloads as W
from mixture_experts_ffn_renorm_gb300.layer import ACTIVATIONS, MoeBlock, MoeMlpBlock, _dev_bf16

from . import ref_bias_act as R
from .gpu_util import DEV, launched_since, launches

pytestmark = pytest.mark.gpu

# A value passes at most 8 roundings to bf16 on its way (x W1, act, W2, rows; back: rows, dz2, dhidden,
# dz1, rows, output), each off by at most 2^-8: relative to the norm of a result
BOUND = 10 * 2.0 ** -8


def mlp(T, H, I, E, K, activation, seed=0, bias=True, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed + T)
    n = lambda *s, std=1.0, dt=torch.bfloat16: (torch.randn(s, generator=g, device=DEV) * std).to(dt)
    w = {"w_router": n(E, H, std=H ** -0.5), "w1": n(E, I, H, std=H ** -0.5), "w2": n(E, H, I, std=I ** -0.5),
         "logit_bias": n(E, std=0.3, dt=torch.float32) if bias else None,
         "b1": n(E, I, std=0.5, dt=torch.float32) if bias else None,
         "b2": n(E, H, std=0.5, dt=torch.float32) if bias else None}
    blk = MoeMlpBlock(H, I, E, K, w, max_tokens=T, activation=activation, device=DEV, routed_scale=scale, training=True)
    return blk, w, n(T, H), n(T, H, std=0.5), n(T, H)


def reference(blk, w, x, dout, residual, activation, scale):
    """Output and gradients in 64 bits, the choice of experts taken from the block."""
    d = {k: (None if v is None else v.double().requires_grad_()) for k, v in w.items()}
    xd = x.double().requires_grad_()
    T, K = x.shape[0], blk.K
    l = xd @ d["w_router"].t() + (d["logit_bias"] if d["logit_bias"] is not None else 0.0)
    ids = blk.topk_ids[:T].long()
    pick = torch.softmax(l.gather(1, ids), 1)
    pick.retain_grad()
    out = torch.zeros_like(xd) if residual is None else residual.double()
    for j in range(K):
        e = ids[:, j]
        z = torch.einsum("th,tih->ti", xd, d["w1"][e])
        if d["b1"] is not None:
            z = z + d["b1"][e]
        y = torch.einsum("ti,thi->th", R.act(z, ACTIVATIONS[activation]), d["w2"][e])
        if d["b2"] is not None:
            y = y + d["b2"][e]
        out = out + scale * pick[:, j:j + 1] * y
    out.backward(dout.double())
    grads = {"grad_x": xd.grad, "grad_w_router": d["w_router"].grad, "grad_topk_w": pick.grad, "grad_w1": d["w1"].grad,
             "grad_w2": d["w2"].grad}
    for k, n in (("grad_b1", "b1"), ("grad_b2", "b2"), ("grad_logit_bias", "logit_bias")):
        if d[n] is not None:
            grads[k] = d[n].grad
    return out.detach(), grads


def near(got, want, what):
    off = (got.double() - want).norm() / want.norm()
    assert off <= BOUND, f"{what}: {off.item():.2e} of its norm"


@pytest.mark.parametrize("activation", sorted(ACTIVATIONS))
@pytest.mark.parametrize("size", [(1, 64, 32, 4, 2), (33, 136, 72, 6, 3), (300, 264, 392, 5, 2)], ids=lambda s: "x".join(map(str, s)))
def test_forward_and_gradients(size, activation):
    blk, w, x, dout, residual = mlp(*size, activation, bias=size[0] != 33, scale=1.5)
    res = residual if size[0] != 1 else None
    out = blk.forward(x, residual=res)
    grads = {k: v.clone() for k, v in blk.backward(x, dout).items()}
    want, wanted = reference(blk, w, x, dout, res, activation, 1.5)
    near(out, want, "out")
    for k, v in wanted.items():
        near(grads[k], v, k)
    again = blk.backward(x, dout)                 # what the forward kept is still there
    torch.cuda.synchronize()
    for k in wanted:
        assert torch.equal(again[k], grads[k]), k


def test_gradients_against_differences():
    # the loss sum(out * dout) along random directions, from forwards whose bf16 roundings are
    # averaged away by many tokens: the difference quotient of a step h errs by the roundings over h
    blk, w, x, dout, _ = mlp(256, 64, 48, 4, 2, "silu", seed=3)
    blk.forward(x)
    grads = {k: v.clone() for k, v in blk.backward(x, dout).items()}
    g = torch.Generator(device=DEV).manual_seed(5)
    for name, key in (("b1", "grad_b1"), ("b2", "grad_b2")):
        p = getattr(blk, name)
        keep, step = p.clone(), 0.25
        # towards the gradient, so that the derivative is large against the roundings
        v = grads[key] / grads[key].norm()
        vals = []
        for s in (step, -step):
            p.copy_(keep + s * v)
            vals.append((blk.forward(x).double() * dout.double()).sum().item())
        p.copy_(keep)
        slope = (vals[0] - vals[1]) / (2 * step)
        want = (grads[key].double() * v.double()).sum().item()
        # out's rounding: 2^-8 of 0.5 * |out| a value, at random over T H of them, twice, over 2 step
        noise = 2.0 ** -8 * blk.out.double().norm().item() * 0.5 * 2 / (2 * step)
        assert abs(slope - want) <= 0.05 * abs(want) + noise, (name, slope, want, noise)


def test_mlp_block_in_a_graph_and_its_refusals():
    blk, w, x, dout, residual = mlp(40, 136, 72, 6, 3, "gelu")
    with pytest.raises(ValueError, match="before it"):
        blk.backward(x, dout)
    want = blk.forward(x, residual=residual).clone()
    grads = {k: v.clone() for k, v in blk.backward(x, dout).items()}
    with pytest.raises(ValueError, match="took 40"):
        blk.backward(x[:3].contiguous(), dout[:3].contiguous())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = blk.forward(x, residual=residual)
        got = blk.backward(x, dout)
    for _ in range(3):
        for v in (out, *got.values()):
            v.zero_()
        g.replay()
        assert torch.equal(out, want)
        for k in grads:
            assert torch.equal(got[k], grads[k]), k
    assert m.moe_device_status() == 0
    with pytest.raises(ValueError, match="activation"):
        MoeMlpBlock(64, 32, 4, 2, w, 4, activation="swish", device=DEV)
    with pytest.raises(ValueError, match="multiples of 8"):
        MoeMlpBlock(60, 32, 4, 2, w, 4, device=DEV)
    serve = MoeMlpBlock(136, 72, 6, 3, w, 64, device=DEV)      # a larger workspace, no training buffers
    assert torch.equal(serve.forward(x, residual=residual), want)
    with pytest.raises(ValueError, match="training"):
        serve.backward(x, dout)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shared", [0, 64])
def test_few_tokens_block_agrees_with_its_launches(fp8, shared):
    cfg = W.LayerConfig("few", T=48, H=512, I=256, E=16, K=4, I_shared=shared, seed=5)
    d = W.layer_inputs(cfg)
    if fp8:
        d["w13_e4m3"], d["w13_scale"] = W.quantize_fp8_block(d["w13"])
        d["w2_e4m3"], d["w2_scale"] = W.quantize_fp8_block(d["w2"])
    mk = lambda **kw: MoeBlock(cfg.H, cfg.I, cfg.E, cfg.K, d, max_tokens=cfg.T, device=DEV, I_shared=shared,
                               fp8_weights=fp8, **kw)
    plain, few = mk(), mk(few=True)
    x = _dev_bf16(d["x"], DEV)
    for T in (1, 7, 16, 17, 48):
        before = launches()
        got = few.forward(x[:T].contiguous()).clone()
        assert launched_since(before, "layer_few") == (1 if T <= 16 else 0)
        want = plain.forward(x[:T].contiguous())
        assert torch.equal(few.topk_ids[:T], plain.topk_ids[:T]) and torch.equal(few.topk_w[:T], plain.topk_w[:T])
        if T > 16:
            assert torch.equal(got, want)
        else:
            near(got, want.double(), f"T={T}")
    xs = x[:5].contiguous()
    want = few.forward(xs).clone()
    few.capture(xs)
    assert torch.equal(few.replay(), want)
    hosts = [torch.from_numpy(np.ascontiguousarray(d["x"][i:i + 3]).view(np.int16)).view(torch.bfloat16).pin_memory() for i in (0, 3, 6)]
    outs = [torch.empty_like(h).pin_memory() for h in hosts]
    few.run_host_batches(hosts, outs)
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o.to(DEV), few.forward(x[3 * i:3 * i + 3].contiguous()))


def test_few_refuses_what_it_does_not_have():
    cfg = W.TINY
    d = W.layer_inputs(cfg)
    with pytest.raises(ValueError, match="few"):
        MoeBlock(cfg.H, cfg.I, cfg.E, cfg.K, {**d, "w13_e4m3": None}, max_tokens=4, device=DEV, fp8_weights=True,
                 fp8_acts=True, few=True)
