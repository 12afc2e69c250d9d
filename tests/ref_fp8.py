"""Plain 64-bit implementations of the FP8 products and of the gradients, for the tests.

Inputs and results are CPU tensors.  Quantisation is defined by operations that are each
rounded to binary32, so that part is computed in binary32 (codes and scales are compared bit
for bit); everything else is float64.
"""
from __future__ import annotations

import torch

BLOCK = 128
E4M3 = torch.float8_e4m3fn


def blocks(n):
    return -(-n // BLOCK)


def quantise(v):
    """f32 rows [R, C] -> (codes uint8 [R, C], scales f32 [R, blocks])."""
    R, C = v.shape
    codes = torch.empty((R, C), dtype=torch.uint8)
    scales = torch.empty((R, blocks(C)))
    for b in range(blocks(C)):
        part = v[:, b * BLOCK:(b + 1) * BLOCK]
        amax = torch.nan_to_num(part.abs(), nan=0.0, posinf=float("inf")).amax(1)
        d = torch.maximum(amax / torch.full_like(amax, 448.0), torch.tensor(2.0 ** -126))
        q = part * torch.reciprocal(d)[:, None]
        q = torch.where(q.isnan(), q, q.clamp(-448.0, 448.0))
        codes[:, b * BLOCK:(b + 1) * BLOCK] = q.to(E4M3).view(torch.uint8)
        scales[:, b] = d
    return codes, scales


def row_values(codes, scales):
    s = scales.double().repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]
    return codes.view(E4M3).double() * s


def weight_values(codes, scale):
    R, C = codes.shape[1:]
    s = scale.double().repeat_interleave(BLOCK, 1)[:, :R].repeat_interleave(BLOCK, 2)[:, :, :C]
    return codes.view(E4M3).double() * s


def grouped(a, w, off):
    """(a [P, K] x w [G, N, K]^T per group, and the same of the magnitudes), f64 [P, N]."""
    y = torch.zeros((a.shape[0], w.shape[1]), dtype=torch.float64)
    mag = torch.zeros_like(y)
    for g in range(w.shape[0]):
        lo, hi = int(off[g]), int(off[g + 1])
        y[lo:hi] = a[lo:hi] @ w[g].t()
        mag[lo:hi] = a[lo:hi].abs() @ w[g].abs().t()
    return y, mag


def bf16_between(y, tol):
    """The bf16 roundings of y - tol and y + tol (rounding is monotone), as f64."""
    return (y - tol).float().to(torch.bfloat16).double(), (y + tol).float().to(torch.bfloat16).double()


def silu_mul_backward(g, u, da):
    s = torch.sigmoid(g)
    dg, du = da * u * s * (1 + g * (1 - s)), da * g * s
    mag = torch.cat([(da * u * s).abs() * (1 + (g * (1 - s)).abs()), du.abs()], 1)
    return torch.cat([dg, du], 1), mag


def e4m3_half_step(q):
    """Half the spacing of E4M3 values at magnitude q (f64): subnormal spacing is 2^-9."""
    e = torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6)))
    return torch.exp2(e - 4)


def route(l, ids, renormalize, scoring, offsets, balance, z):
    """Routing weights [T, K] and the two losses, differentiable, f64."""
    score = torch.sigmoid(l) if scoring else torch.softmax(l, 1)
    if scoring == 0 and renormalize:
        w = torch.softmax(l.gather(1, ids), 1)
    else:
        w = score.gather(1, ids)
        w = w / w.sum(1, keepdim=True) if renormalize else w
    T, E = l.shape
    loss_b = loss_z = l.sum() * 0
    if balance:
        f = offsets.double().diff() * E / (ids.shape[1] * T)
        loss_b = balance * (f * (score / score.sum(1, keepdim=True)).mean(0)).sum()
    if z:
        loss_z = z * torch.logsumexp(l, 1).square().mean()
    return w, loss_b, loss_z
