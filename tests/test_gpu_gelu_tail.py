"""GELU of the products' epilogue and its gradient far below zero, where z Phi(z) and its slope are small
beside z: a bound relative to the value, not to z.

Bounds: Phi(z) is off by at most 2^-14 of itself below -4 (3e-7 above), the density's exponential by 2^-15
(its argument, at most 121, is rounded twice: 2 x 2^-24 x 121 ln 2 < 2^-16, and 2^-22 for the fast 2^x);
a rounding to bf16 by 2^-8, one to f32 by 2^-24."""
from __future__ import annotations

import math

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m

from .gpu_util import DEV
from .test_gpu_bias_act import Back, Product

pytestmark = pytest.mark.gpu

U32, UBF = 2.0 ** -24, 2.0 ** -8


def phi(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2.0))


def phi_bound(z):
    return torch.where(z < -4.0, 2.0 ** -14 * phi(z), torch.full_like(z, 3e-7))


# the kernel of few rows, the join of ranges of K, a tile's own epilogue
@pytest.mark.parametrize("P,K,columns", [(1, 8, False), (20, 2048, True), (600, 256, True)])
def test_gelu_of_negative_values(P, K, columns):
    N = 1296
    c = Product(P, K, N, columns=columns, kind=m.ACT_GELU)
    c.a.zero_()                                   # z is the bias
    c.bias[0] = torch.linspace(-12.9, -0.01, N, device=DEV)
    c.call()
    torch.cuda.synchronize()
    z = c.bias[0].double()
    y = z * phi(z)
    bound = phi_bound(z) * z.abs() + U32 * y.abs()
    off = (c.out.double() - y).abs() - (bound + UBF * (y.abs() + bound))
    assert (off <= 0).all(), f"first at z = {z[(off > 0).any(0)][:3].tolist()}"


def test_gelus_slope_of_negative_values():
    c = Back(1, 1296, kind=m.ACT_GELU, weight=True)
    c.z[0] = torch.linspace(-12.9, 4.0, c.N, device=DEV).to(torch.bfloat16)
    c.dout.fill_(1.0)
    c.pw.fill_(1.0)
    c.call()
    torch.cuda.synchronize()
    z = c.z[0].double()
    density = z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    s = phi(z) + density
    bound = phi_bound(z) + (2.0 ** -15 + 4 * U32) * density.abs() + 2 * U32 * s.abs()
    assert ((c.db[0].double() - s).abs() <= bound).all()                       # f32, one row: the slope itself
    assert ((c.dz[0].double() - s).abs() <= bound + UBF * (s.abs() + bound)).all()
    y = z * phi(z)
    sum_bound = (phi_bound(z) * z.abs() + (c.N / 32 + 10) * U32 * y.abs()).sum()
    assert (c.dpw[0].double() - y.sum()).abs() <= sum_bound
