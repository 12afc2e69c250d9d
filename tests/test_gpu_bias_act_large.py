"""The products with an epilogue and their gradients where element counts pass 2^31: the last rows and
groups against their formulas."""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m

from . import ref_bias_act as R
from .gpu_util import DEV

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
P, N, K = 70000, 32768, 16          # P N = 2.3e9


def normal(g, *s, std=1.0, dt=BF):
    return (torch.randn(s, generator=g, device=DEV) * std).to(dt)


def test_product_and_its_epilogue_gradient():
    g = torch.Generator(device=DEV).manual_seed(1)
    off = torch.tensor([0, 3, 69990, P], dtype=torch.int32, device=DEV)
    a, w, bias = normal(g, P, K), normal(g, 3, N, K, std=K ** -0.5), normal(g, 3, N, dt=torch.float32)
    out, z = torch.empty((P, N), dtype=BF, device=DEV), torch.empty((P, N), dtype=BF, device=DEV)
    m.moe_grouped_gemm_bias_act_bf16(a, w, m.W_ROWS, bias, m.ACT_SILU, z, None, None, None, off, P, K, N, 3, out)
    tail = torch.tensor([0, 8], dtype=torch.int32)              # the last 8 rows are of the last group
    rows = slice(P - 8, P)
    zz, dz, y, dy = R.product(a[rows], w[2:], False, bias[2:], R.SILU, tail, 1)
    R.check(out[rows], y, dy + R.UBF * (y.abs() + dy), None, "out")
    R.check(z[rows], zz, dz + R.UBF * (zz.abs() + dz), None, "pre_act")
    dout, grad = out, torch.empty((P, N), dtype=BF, device=DEV)   # any gradient serves
    db, dpw = torch.empty((3, N), device=DEV), torch.empty((P,), device=DEV)
    ws = torch.empty(m.moe_bias_act_backward_workspace_size(P, N, 3), dtype=torch.uint8, device=DEV)
    m.moe_bias_act_backward(dout, z, m.ACT_SILU, None, None, off, P, N, 3, grad, db, dpw, ws, ws.numel())
    zd, d = z[rows].double(), dout[rows].double()
    want = d * R.slope(zd, R.SILU)
    err = d.abs() * (4 * R.U32 + R.REL + R.PHI * (1 + zd.abs()))
    R.check(grad[rows], want, err + R.UBF * (want.abs() + err), None, "dz")
    zd, d = z[69990:].double(), dout[69990:].double()
    want = d * R.slope(zd, R.SILU)
    err = d.abs() * (4 * R.U32 + R.REL + R.PHI * (1 + zd.abs()))
    R.check(db[2], want.sum(0), (err + 50 * R.U32 * want.abs()).sum(0), None, "grad_bias")
    y = R.act(zd, R.SILU)
    R.check(dpw[69990:], (d * y).sum(1), (d.abs() * (R.REL * y.abs() + R.PHI * zd.abs() + (N / 32 + 140) * R.U32 * y.abs())).sum(1),
            None, "grad_pair_weight")


def test_weight_gradient():
    g = torch.Generator(device=DEV).manual_seed(2)
    G, n, k = 3, 32768, 24576           # 2.4e9 sums
    off = torch.tensor([0, 20, 20, 53], dtype=torch.int32, device=DEV)
    dz, a = normal(g, 53, n), normal(g, 53, k)
    dw = torch.full((G, n, k), float("nan"), device=DEV)
    ws = torch.empty(max(16, m.moe_grouped_gemm_wgrad_workspace_size(53, n, k, G)), dtype=torch.uint8, device=DEV)
    m.moe_grouped_gemm_wgrad_bf16(dz, a, off, 53, n, k, G, None, dw, ws, ws.numel())
    d, x = dz[20:, -64:].double(), a[20:].double()
    R.check(dw[2, -64:], d.t() @ x, 40 * R.U32 * (d.abs().t() @ x.abs()), None, "grad_w")
    assert not dw[1].any()
    assert dw[0].isfinite().all()
