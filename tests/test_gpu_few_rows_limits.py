"""Which calls of the product with an epilogue the kernel of few rows takes, on either side of each of its
limits as they follow from this GPU's SMs, and that both sides give the same product."""
from __future__ import annotations

import pytest
import torch

from . import ref_bias_act as R
from .gpu_util import DEV, launched_since, launches
from .test_gpu_bias_act import Product

pytestmark = pytest.mark.gpu

SMS = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 152
WAVE = 128 * SMS           # columns of two CTAs an SM, 64 to a CTA with one slice of K


@pytest.mark.parametrize("P,K,N,few", [
    (16, 136, WAVE, True), (16, 136, WAVE + 8, False),             # one wave of one block of 16 rows
    (8, 136, WAVE + 8, True), (9, 136, WAVE + 8, False),           # past it at most eight rows
    (16, 8192, 264, True),                                         # one block takes any K
    (17, 8192, 264, True), (17, 8200, 264, False),                 # more of them four batches of 64 K by eight slices
    (17, 72, WAVE // 2, True), (17, 72, WAVE // 2 + 8, False),     # two blocks, one wave
    (16, 136, 264, True),
])
@pytest.mark.parametrize("columns", [False, True])
def test_limits(P, K, N, few, columns):
    c = Product(P, K, N, columns=columns, kind=R.SILU, pre=True, residual=True)
    before = launches()
    c.run()
    assert launched_since(before, "gemm_bias_act") == 1
    assert launched_since(before, "bias_act_few") == int(few and not columns)
