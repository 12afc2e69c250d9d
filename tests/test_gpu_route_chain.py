"""Steps of the router's gradient one behind the other, without a synchronisation: the products
start beside one another under programmatic launch and must read this step's logits' gradient,
not the one that lay in the same buffer a step before."""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m

from .gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _pdl_on():
    m.moe_set_pdl(True)
    yield
    m.moe_set_pdl(True)


@pytest.mark.parametrize("T,H,E,K", [(1, 64, 8, 2), (40, 128, 16, 2), (300, 1032, 60, 6), (1500, 256, 128, 8),
                                     (4096, 512, 128, 8)])
def test_every_step_reads_its_own_gradient(T, H, E, K):
    steps = 60
    g = torch.Generator(device=DEV).manual_seed(T)
    logits = torch.randn((T, E), generator=g, device=DEV)
    ids = logits.topk(K, 1).indices.int()
    gws = torch.randn((steps, T, K), generator=g, device=DEV)
    xs = torch.randn((4, T, H), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn((E, H), generator=g, device=DEV).to(torch.bfloat16)
    n = max(16, m.moe_route_logits_backward_workspace_size(T, H, E))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    dl, x = torch.empty((T, E), device=DEV), torch.empty((T, H), dtype=torch.bfloat16, device=DEV)

    def run():
        outs = [(torch.empty_like(x), torch.empty((E, H), device=DEV), torch.empty(E, device=DEV)) for _ in range(steps)]
        torch.cuda.synchronize()
        for i in range(steps):
            if i % 3 == 0:
                x.copy_(xs[i % 4])
            m.moe_route_backward(logits, ids, gws[i], None, T, E, K, 1, 0, 0.0, 0.0, dl, None, None, 0)
            m.moe_route_logits_backward(dl, x, w, T, H, E, *outs[i], ws, n)
        torch.cuda.synchronize()
        return outs
    got = run()
    m.moe_set_pdl(False)
    want = run()
    for i in range(steps):
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b), i
