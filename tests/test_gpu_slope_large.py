"""The activations' slopes at values up to bf16's largest: their limits, no overflow on the way."""
from __future__ import annotations

import pytest
import torch

from . import ref_bias_act as R
from .gpu_util import DEV
from .test_gpu_bias_act import Back

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", range(6))
def test_slopes_of_large_values(kind):
    v = [s * x for x in (30.0, 1e4, 1e10, 1.8e19, 1.9e19, 1e25, 1e30, 1e38, 1.6e38, 3.38e38) for s in (1.0, -1.0)]
    c = Back(1, 24, kind=kind)
    c.z.zero_()
    c.z[0, :len(v)] = torch.tensor(v, device=DEV).to(torch.bfloat16)
    c.dout.fill_(1.0)
    c.call()
    torch.cuda.synchronize()
    z = c.z.double()
    want = R.slope(z, kind)                       # close to 0, 1 or 2 z
    assert want.isfinite().all()
    want = want.float().double()                  # infinite where 2 z is beyond f32
    # a slope below 2^-126 may be 0; the exponentials' arguments, at most 30 / ln 2 where it is not, are rounded twice:
    # 2 x 2^-24 x 30 and the fast forms' few 2^-22, together below 2^-17
    assert torch.allclose(c.db.double(), want, rtol=2.0 ** -17, atol=2.0 ** -126)
    assert torch.allclose(c.dz.double(), want, rtol=2.0 ** -17 + 2.0 ** -8, atol=2.0 ** -126)
