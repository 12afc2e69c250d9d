"""The bounded waits of the few-token layer, of the products with an epilogue and of the weights'
gradient, made to run out: at a limit of 1 us a launch over large inputs cannot finish.  Each kernel
must still end, raise MOE_STATUS_TIMEOUT and leave the device usable: with the limit restored, the
same calls give the same bits as before."""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m

from .gpu_util import DEV
from .test_gpu_bias_act import Product, Wgrad, offsets
from .test_gpu_layer_few import Case

pytestmark = pytest.mark.gpu

FULL_LIMIT_NS = 10**9


@pytest.fixture(autouse=True)
def _restore_limit():
    m.lib()
    m.moe_device_status(clear=True)
    yield
    m.moe_set_wait_limit_ns(FULL_LIMIT_NS)
    m.moe_device_status(clear=True)


def runs_out(call, outs, reset=lambda: None):
    call()
    torch.cuda.synchronize()
    assert m.moe_device_status() == 0
    want = [o.clone() for o in outs]
    torch.zeros(1 << 29, dtype=torch.uint8, device=DEV)     # the inputs leave L2
    m.moe_set_wait_limit_ns(1000)
    call()
    assert m.moe_device_status(clear=True) & m.STATUS_TIMEOUT
    m.moe_set_wait_limit_ns(FULL_LIMIT_NS)
    reset()
    for o in outs:
        o.zero_()
    call()
    torch.cuda.synchronize()
    assert m.moe_device_status() == 0
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 16])
def test_layer(T, fp8):
    c = Case(T, 4096, 1024, 32, 8, Is=1024, fp8=fp8)
    runs_out(c.call, (c.out, c.ids, c.w), reset=c.ws.zero_)     # as its description asks


@pytest.mark.parametrize("columns", [False, True])
def test_product(columns):
    c = Product(4000, 4096, 4096, 1, None, columns, residual=True)
    runs_out(c.call, (c.out,))


@pytest.mark.parametrize("add,rows", [(False, 512), (True, 512), (True, 576)])
def test_weight_gradient(add, rows):
    # a tile per SM and group, 60 MB of rows: its first sums are 9 us of HBM away
    G = 152
    c = Wgrad(rows * G, 128, 256, G, offsets([rows] * G), add=add)
    runs_out(c.call, (c.dw,))
