"""grad_x of the router's product where the sum over experts cancels: every bit of the f32
logits' gradient counts.

The rows of a softmax router's gradient sum to zero, so what all rows of the router weight have in
common drops out of grad_x and a small rest is left.  The cases below are built of powers of two,
so that every product and every partial sum is exact in binary32 and grad_x is exactly the bf16
rounding of the true sum (tolerance 0).
"""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m

from .gpu_util import DEV

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def dx(dl, w):
    T, E = dl.shape
    H = w.shape[1]
    out = torch.empty((T, H), dtype=BF, device=DEV)
    m.moe_route_logits_backward(dl.to(DEV), None, w.to(DEV), T, H, E, out, None, None, None, 0)
    return out.cpu()


@pytest.mark.parametrize("T,H,E", [(1, 8, 2), (130, 264, 128), (3, 520, 300), (5, 8, 1024)])
@pytest.mark.parametrize("tail", [2.0 ** -20, -2.0 ** -20])
def test_cancelling_rows_keep_the_last_bits(T, H, E, tail):
    # pairs of experts: 1 + 2^-10 + tail against -(1 + 2^-10); a pair adds `tail` to each column
    dl = torch.zeros((T, E))
    dl[:, 0:E - E % 2:2] = 1.0 + 2.0 ** -10 + tail
    dl[:, 1::2] = -(1.0 + 2.0 ** -10)
    scale = torch.exp2((torch.arange(T) % 5).float())           # a power of two per token
    dl = dl * scale[:, None]
    w = torch.exp2(-(torch.arange(H) % 7).float()).to(BF).expand(E, H).contiguous()
    want = (dl.double() @ w.double()).to(BF)
    assert (want != 0).all()
    assert torch.equal(dx(dl, w), want)


def test_large_values_stay_finite():
    # beyond the largest bf16 value, whose rounding to bf16 would be infinite
    top = torch.finfo(torch.float32).max
    dl = torch.tensor([[top, 0.0, 0.0], [0.0, -top, 0.0]])
    w = torch.full((3, 16), 2.0 ** -3).to(BF)
    want = (dl.double() @ w.double()).to(BF)
    assert torch.equal(dx(dl, w), want)


def test_infinities_and_nan_stay_in_their_rows():
    dl = torch.randn((4, 70), generator=torch.Generator().manual_seed(1))
    clean = dl.clone()
    dl[1, 3] = float("inf")
    dl[2, 69] = float("nan")
    w = torch.rand((70, 24), generator=torch.Generator().manual_seed(2)).add(0.5).to(BF)
    got, want = dx(dl, w), dx(clean, w)
    assert torch.equal(got[[0, 3]], want[[0, 3]])
    assert not got[1].isfinite().any() and got[2].isnan().all()
