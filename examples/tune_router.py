"""Tune the router of an MoE block whose experts are frozen in FP8.

    python examples/tune_router.py [--tokens 2048] [--steps 60]

The experts of a block are quantised to block-scaled FP8 (weights and activations) and its
router is replaced by a perturbed one.  Gradient descent on the bf16 output of the original
router then moves the router back: each step runs the FP8 forward, the gradients of the
combine, of the router and of the tokens (MoeBlock.backward), and updates an f32 copy of the
router weight, with a balance loss and a z-loss.  Prints the output error and the losses; every
step is replayed from CUDA graphs.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixture_experts_ffn_renorm_gb300 import workloads as W  # noqa: E402
from mixture_experts_ffn_renorm_gb300.layer import MoeBlock, _dev_bf16  # noqa: E402


def build(cfg, tokens, device="cuda"):
    """(the FP8 block with a perturbed router, the tokens, the original router's output)."""
    d = W.layer_inputs(cfg)
    d["w13_e4m3"], d["w13_scale"] = W.quantize_fp8_block(d["w13"])
    d["w2_e4m3"], d["w2_scale"] = W.quantize_fp8_block(d["w2"])
    blk = MoeBlock(cfg.H, cfg.I, cfg.E, cfg.K, d, max_tokens=tokens, device=device,
                   fp8_weights=True, fp8_acts=True, training=True)
    x = _dev_bf16(d["x"], device)[:tokens].contiguous()
    target = blk.forward(x).float().clone()
    g = torch.Generator(device=device).manual_seed(cfg.seed + 1)
    noise = torch.randn(blk.w_router.shape, generator=g, device=device) * 0.01
    blk.w_router.copy_(blk.w_router.float() + noise)
    return blk, x, target


def tune(blk, x, target, steps, lr, balance=1e-4, z=1e-5):
    """Plain gradient descent with momentum on the mean squared error of the output; yields
    (error, balance loss, z-loss) before each step."""
    master = blk.w_router.float()
    speed = torch.zeros_like(master)
    dout = torch.empty_like(x)
    err = torch.zeros((), device=x.device)

    def step():
        diff = blk.forward(x).float() - target
        err.copy_(diff.square().mean() / target.square().mean())
        # the error's gradient, scaled so that its elements are of order one
        dout.copy_(diff / target.square().mean().sqrt())
        grads = blk.backward(x, dout, balance, z)
        speed.mul_(0.9).add_(grads["grad_w_router"] / x.shape[0])
        master.sub_(lr * speed)
        blk.w_router.copy_(master)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = master.clone()
    with torch.cuda.stream(side):        # once outside the graph, then undone
        step()
        master.copy_(keep)
        speed.zero_()
        blk.w_router.copy_(master)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(steps):
        graph.replay()
        b, zl = blk.losses.tolist()
        yield float(err), b, zl


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--lr", type=float, default=0.02)
    args = ap.parse_args()
    cfg = W.LayerConfig("tune", T=args.tokens, H=1024, I=512, E=64, K=6, seed=3)
    blk, x, target = build(cfg, args.tokens)
    for i, (err, b, z) in enumerate(tune(blk, x, target, args.steps, args.lr)):
        if i % 10 == 0 or i == args.steps - 1:
            print(f"step {i:4d}  relative output error {err:.5f}  balance {b:.6f}  z {z:.6f}")


if __name__ == "__main__":
    main()
