"""The workspace of the router's product gradients: a size queried for many tokens serves fewer.

The ranges of tokens that the sums are split into are rounded to whole steps, so fewer tokens can
take more ranges than more tokens do; the query must bound them all.
"""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m
from mixture_experts_ffn_renorm_gb300 import workloads as W
from mixture_experts_ffn_renorm_gb300.layer import MoeBlock

from .gpu_util import DEV, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,E", [(8, 1), (128, 16), (1024, 64), (2048, 128), (2048, 256), (1032, 300), (4096, 1024)])
def test_size_never_falls_as_tokens_grow(H, E):
    m.lib()
    torch.cuda.current_stream()
    tokens = sorted({max(1, 64 * i + j) for i in range(0, 300) for j in (-1, 0, 1)})
    sizes = [m.moe_route_logits_backward_workspace_size(T, H, E) for T in tokens]
    falls = [(a, b) for a, b, s, t in zip(tokens, tokens[1:], sizes, sizes[1:]) if s > t]
    assert not falls, falls[:3]


@pytest.mark.parametrize("T,most,H,E", [(4000, 4096, 2048, 128), (3400, 3500, 2048, 128), (12288, 12352, 128, 16)])
def test_fewer_tokens_in_a_workspace_for_more(T, most, H, E):
    g = torch.Generator(device=DEV).manual_seed(T)
    dl = torch.randn((T, E), generator=g, device=DEV)
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn((E, H), generator=g, device=DEV).to(torch.bfloat16)
    n = m.moe_route_logits_backward_workspace_size(most, H, E)
    ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
    got = [torch.empty_like(x), torch.empty((E, H), device=DEV), torch.empty((E,), device=DEV)]
    m.moe_route_logits_backward(dl, x, w, T, H, E, *got, ws, n)
    assert (ws[n:] == 0x5A).all()
    own = torch.empty(m.moe_route_logits_backward_workspace_size(T, H, E), dtype=torch.uint8, device=DEV)
    want = [torch.empty_like(t) for t in got]
    m.moe_route_logits_backward(dl, x, w, T, H, E, *want, own, own.numel())
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_block_takes_fewer_tokens_than_it_was_built_for():
    T, most, H, I, E, K = 12288, 12352, 128, 16, 16, 1
    d = W.layer_inputs(W.LayerConfig("ws", T=T, H=H, I=I, E=E, K=K))
    d["w13_e4m3"], d["w13_scale"] = W.quantize_fp8_block(d["w13"])
    d["w2_e4m3"], d["w2_scale"] = W.quantize_fp8_block(d["w2"])
    x = to_dev(d["x"])
    dout = torch.randn((T, H), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    grads = []
    for tokens in (most, T):
        blk = MoeBlock(H, I, E, K, d, max_tokens=tokens, fp8_weights=True, fp8_acts=True, training=True)
        blk.forward(x)
        grads.append(blk.backward(x, dout, 0.01, 0.001))
    for k, v in grads[0].items():
        assert torch.equal(v, grads[1][k]), k
