"""MoeBlock(few=True) at the one launch's largest sizes and past them, where the separate launches serve."""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m
from mixture_experts_ffn_renorm_gb300 import workloads as W
from mixture_experts_ffn_renorm_gb300.layer import MoeBlock, _dev_bf16

from .gpu_util import DEV, launched_since, launches
from .test_gpu_layer_mlp import near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,I,shared,one", [
    (64, 8192, 0, True), (64, 8208, 0, False), (8192, 32, 0, True), (8208, 32, 0, False),
    (64, 32, 8192, True), (64, 32, 8200, False),
])
def test_sizes_past_the_one_launchs(H, I, shared, one, fp8):
    cfg = W.LayerConfig("few", T=20, H=H, I=I, E=4, K=2, I_shared=shared, seed=9)
    d = W.layer_inputs(cfg)
    if fp8:
        d["w13_e4m3"], d["w13_scale"] = W.quantize_fp8_block(d["w13"])
        d["w2_e4m3"], d["w2_scale"] = W.quantize_fp8_block(d["w2"])
    mk = lambda **kw: MoeBlock(H, I, cfg.E, cfg.K, d, max_tokens=cfg.T, device=DEV, I_shared=shared, fp8_weights=fp8, **kw)
    plain, few = mk(), mk(few=True)
    assert m.LAYER_FEW_MAX_DIM == 8192 and plain.few_tokens == 0
    x = _dev_bf16(d["x"], DEV)
    for T in (1, 16, 17):
        before = launches()
        got = few.forward(x[:T].contiguous()).clone()
        assert launched_since(before, "layer_few") == (1 if one and T <= 16 else 0)
        want = plain.forward(x[:T].contiguous())
        if one and T <= 16:
            near(got, want.double(), f"T={T}")
        else:
            assert torch.equal(got, want)
