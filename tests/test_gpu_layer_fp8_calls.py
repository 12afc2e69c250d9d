"""MoeBlock.backward as a program calls it: more than once after a forward, and not for tokens
that no forward has seen."""
from __future__ import annotations

import pytest
import torch

from mixture_experts_ffn_renorm_gb300 import workloads as W
from mixture_experts_ffn_renorm_gb300.layer import MoeBlock

from .gpu_util import DEV, to_dev

pytestmark = pytest.mark.gpu


def problem(T, H, I, E, K):
    d = W.layer_inputs(W.LayerConfig("calls", T=T, H=H, I=I, E=E, K=K))
    d["w13_e4m3"], d["w13_scale"] = W.quantize_fp8_block(d["w13"])
    d["w2_e4m3"], d["w2_scale"] = W.quantize_fp8_block(d["w2"])
    blk = MoeBlock(H, I, E, K, d, max_tokens=T + 2, fp8_weights=True, fp8_acts=True, training=True,
                   routed_scale=0.5)
    g = torch.Generator().manual_seed(T)
    douts = [(torch.randn((T, H), generator=g) * 0.1).to(torch.bfloat16).to(DEV) for _ in range(2)]
    return blk, to_dev(d["x"]), douts


def taken(grads):
    return {k: v.clone() for k, v in grads.items()}


@pytest.mark.parametrize("T,H,I,E,K", [(1, 128, 64, 8, 2), (70, 272, 144, 5, 3), (300, 512, 256, 12, 2)])
def test_second_backward_sees_the_same_forward(T, H, I, E, K):
    blk, x, (first, second) = problem(T, H, I, E, K)
    want = []
    for dout in (first, second):
        out = blk.forward(x).clone()
        want.append(taken(blk.backward(x, dout, 0.02, 0.003)))
    assert torch.equal(blk.forward(x), out)
    for i, dout in ((0, first), (1, second), (1, second), (0, first)):
        got = blk.backward(x, dout, 0.02, 0.003)
        for k, v in want[i].items():
            assert torch.equal(got[k], v), (i, k)


def test_backward_is_of_the_last_forward():
    blk, x, (dout, _) = problem(40, 128, 64, 8, 2)
    with pytest.raises(ValueError, match="forward"):
        blk.backward(x, dout)
    blk.forward(x)
    for n in (39, 1):
        with pytest.raises(ValueError, match="40"):
            blk.backward(x[:n], dout[:n])
    want = taken(blk.backward(x, dout))
    blk.forward(x[:7])
    with pytest.raises(ValueError, match="7"):
        blk.backward(x, dout)
    few = taken(blk.backward(x[:7], dout[:7]))
    # a replayed forward is the last one too
    blk.capture(x)
    blk.forward(x[:7])
    for k, v in few.items():
        assert torch.equal(blk.backward(x[:7], dout[:7])[k], v), k
    blk.replay()
    got = blk.backward(x, dout)
    for k, v in want.items():
        assert torch.equal(got[k], v), k


def test_no_tokens():
    blk, x, (dout, _) = problem(5, 128, 64, 8, 2)
    blk.forward(x)
    blk.backward(x, dout, 0.1, 0.1)
    assert blk.forward(x[:0]).shape == (0, 128)
    got = blk.backward(x[:0], dout[:0], 0.1, 0.1)      # sums over no token, in place of the call before's
    assert got["grad_x"].shape == (0, 128) and got["grad_topk_w"].shape == (0, 2)
    for k in ("grad_w_router", "grad_logit_bias", "losses"):
        assert (got[k] == 0).all(), k
