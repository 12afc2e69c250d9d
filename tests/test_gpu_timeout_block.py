"""MoeBlock(few=True) after a wait of its one launch ran out: the block's next calls, on the workspace as the
timed-out ones left it, give their bits again -- every CTA arrives at both grid barriers also when it gave up."""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m
from mixture_experts_ffn_renorm_gb300 import workloads as W
from mixture_experts_ffn_renorm_gb300.layer import MoeBlock, _dev_bf16

from .gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
def test_the_next_calls(fp8):
    cfg = W.LayerConfig("few", T=16, H=2048, I=1024, E=32, K=8, I_shared=256, seed=2)
    d = W.layer_inputs(cfg)
    if fp8:
        d["w13_e4m3"], d["w13_scale"] = W.quantize_fp8_block(d["w13"])
        d["w2_e4m3"], d["w2_scale"] = W.quantize_fp8_block(d["w2"])
    blk = MoeBlock(cfg.H, cfg.I, cfg.E, cfg.K, d, max_tokens=16, device=DEV, I_shared=cfg.I_shared, fp8_weights=fp8, few=True)
    x = _dev_bf16(d["x"], DEV)
    want = {T: blk.forward(x[:T].contiguous()).clone() for T in (1, 7, 16)}
    torch.cuda.synchronize()
    m.moe_device_status(clear=True)
    gave_up = 0
    try:
        for limit in (1000, 1000, 2000, 5000, 10000, 20000):
            for T in want:
                torch.zeros(1 << 28, dtype=torch.uint8, device=DEV)      # the weights leave L2
                m.moe_set_wait_limit_ns(limit)
                blk.forward(x[:T].contiguous())
                torch.cuda.synchronize()
                gave_up += bool(m.moe_device_status(clear=True) & m.STATUS_TIMEOUT)
                m.moe_set_wait_limit_ns(10**9)
                for t, w in want.items():
                    assert torch.equal(blk.forward(x[:t].contiguous()), w), (limit, T, t)
                assert m.moe_device_status() == 0
    finally:
        m.moe_set_wait_limit_ns(10**9)
        m.moe_device_status(clear=True)
    assert gave_up >= 6
