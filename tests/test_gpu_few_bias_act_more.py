"""More calls around the few-token layer and MoeMlpBlock: layers in place one behind the other, two at once,
first calls inside a capture, the router's losses through the block."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m

from .gpu_util import DEV
from .test_gpu_layer_few import Case
from .test_gpu_layer_mlp import BOUND, mlp

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("pdl", [True, False])
@pytest.mark.parametrize("size", [(1, 2048, 768, 128, 8), (4, 1024, 256, 16, 4), (16, 512, 64, 8, 2)], ids=str)
def test_layers_in_place_in_a_row(size, pdl):
    # out is x and the residual: each layer reads what the one before wrote to the same addresses
    c = Case(*size, scale=0.5)
    x0 = c.x.clone()

    def chain(in_place, n=12):
        x = x0.clone()
        for _ in range(n):
            c.x = x
            x = c.call(out=x if in_place else torch.empty_like(x), residual=x)
        torch.cuda.synchronize()
        return x.clone()

    m.moe_set_pdl(pdl)
    try:
        want = chain(False)
        for _ in range(20):
            assert torch.equal(chain(True), want)
    finally:
        m.moe_set_pdl(True)
    assert want.isfinite().all() and m.moe_device_status() == 0


def test_two_layers_at_once():
    # on streams and workspaces of their own, bf16 and FP8
    a, b = Case(16, 2048, 768, 128, 8), Case(3, 1040, 400, 60, 6, Is=208, fp8=True)
    want = [a.call().clone(), b.call().clone()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(30):
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                c.out.zero_()
                for _ in range(3):
                    c.call(stream=s)
        torch.cuda.synchronize()
        assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])
    assert m.moe_device_status() == 0


def test_first_calls_inside_a_capture():
    # a fresh process whose first call of each kernel is captured
    code = """
import torch
import mixture_experts_ffn_renorm_gb300 as m
from tests.test_gpu_bias_act import Back, Product, Wgrad, offsets
from tests.test_gpu_layer_few import Case
calls = []
for c in (Case(2, 264, 72, 12, 3), Case(2, 272, 80, 12, 3, fp8=True)):
    calls.append((c, (c.out, c.ids, c.w)))
for c in (Product(3, 520, 264), Product(20, 520, 264), Product(300, 264, 520), Product(300, 2048, 520, columns=True)):
    calls.append((c, (c.out,)))
c = Back(300, 520, 2, offsets([100, 200]), scatter=True, weight=True)
calls.append((c, (c.dz, c.db, c.dpw)))
for c in (Wgrad(300, 136, 264, 2, offsets([170, 130]), add=True), Wgrad(3000, 136, 264, 1), Wgrad(1300, 136, 264, 1, add=True)):
    calls.append((c, (c.dw,)))
torch.cuda.synchronize()
for c, outs in calls:
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    g.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    c.call()
    torch.cuda.synchronize()
    for o, v in zip(outs, got):
        assert torch.equal(o, v), type(c)
assert m.moe_device_status() == 0
print("captured", len(calls))
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env={**os.environ, "PYTHONPATH": ROOT}, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "captured 10" in r.stdout, r.stdout + r.stderr


def test_the_routers_losses_through_the_block():
    balance, z_coef = 0.5, 0.25
    blk, w, x, dout, _ = mlp(120, 136, 72, 6, 3, "gelu", seed=4)
    blk.forward(x)
    plain = {k: v.clone() for k, v in blk.backward(x, dout).items()}
    got = {k: v.clone() for k, v in blk.backward(x, dout, balance_coef=balance, z_coef=z_coef).items()}
    torch.cuda.synchronize()
    wr, lb, xd = (t.double().requires_grad_() for t in (w["w_router"], w["logit_bias"], x))
    T, K, E = 120, 3, 6
    l = xd @ wr.t() + lb
    f = E * torch.bincount(blk.topk_ids.flatten().long(), minlength=E).double() / (K * T)
    losses = torch.stack([balance * (f * torch.softmax(l, 1).mean(0)).sum(), z_coef * (torch.logsumexp(l, 1) ** 2).mean()])
    gx, gw, gb = torch.autograd.grad(losses.sum(), (xd, wr, lb))
    assert not plain["losses"].any()
    assert (got["losses"].double() - losses).abs().max() <= 1e-5 * losses.abs().max()
    for k, v in (("grad_w_router", gw), ("grad_logit_bias", gb), ("grad_x", gx)):
        # what the losses add, beside the roundings of what they are added to (f32; grad_x is bf16)
        bound = BOUND * v.norm() + (2.0 ** -8 * 2 if k == "grad_x" else 2.0 ** -20) * plain[k].double().norm()
        assert (got[k].double() - plain[k].double() - v).norm() <= bound, k
    for k in ("grad_w1", "grad_w2", "grad_b1", "grad_b2", "grad_topk_w"):
        assert torch.equal(got[k], plain[k]), k
