"""Infinite logits and NaN in the router's gradient: where they enter, and where they do not."""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m

from . import ref_fp8 as R
from .test_gpu_backward import magnitudes, problem, run_route

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _clear_status():
    m.lib()
    m.moe_device_status(clear=True)
    yield
    assert m.moe_device_status() == 0


@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("balance", [0.0, 0.5])
def test_sigmoid_of_plus_infinity_is_one_with_slope_zero(renorm, balance):
    T, E, K = 5, 40, 4
    l, _, off, gw = problem(T, E, K, 11)
    l[1, 9] = INF                                      # chosen below: the largest
    ids = l.topk(K, 1).indices
    assert 9 in ids[1]
    got, losses = run_route(l, ids, gw, off if balance else None, renorm, 1, balance, 0.0)
    assert float(got[1, 9]) == 0.0 and got.isfinite().all() and losses.isfinite().all()
    ld = l.double()
    ld[1, 9] = 1e3                                     # the limit, differentiable
    ld.requires_grad_()
    w, lb, _ = R.route(ld, ids, renorm, 1, off, balance, 0)
    (want,) = torch.autograd.grad((w * gw.double()).sum() + lb, ld)
    mag = magnitudes(ld.detach(), ids, gw.double(), off, renorm, 1, balance, 0.0)
    assert ((got.double() - want).abs() <= 2.0 ** -16 * mag + 1e-37).all()


@pytest.mark.parametrize("bad", [INF, NAN])
@pytest.mark.parametrize("renorm,scoring,z,enters", [(1, 0, 0.0, False), (0, 0, 0.0, True), (1, 1, 0.0, False),
                                                     (0, 1, 0.0, False), (1, 0, 0.25, True), (1, 1, 0.25, True)])
def test_a_bad_logit_that_is_not_chosen(bad, renorm, scoring, z, enters):
    T, E, K = 5, 40, 4
    l, ids, off, gw = problem(T, E, K, 12)
    clean, _ = run_route(l, ids, gw, None, renorm, scoring, 0.0, z)
    e = next(e for e in range(E) if e not in ids[2])
    l[2, e] = bad
    got, _ = run_route(l, ids, gw, None, renorm, scoring, 0.0, z)
    keep = [0, 1, 3, 4] if enters else list(range(T))
    assert torch.equal(got[keep], clean[keep])
    assert not enters or got[2].isnan().any()


@pytest.mark.parametrize("renorm,scoring", [(1, 0), (0, 0)])
def test_a_chosen_infinity_of_a_softmax_makes_its_row_nan(renorm, scoring):
    T, E, K = 4, 24, 3
    l, ids, off, gw = problem(T, E, K, 13)
    clean, _ = run_route(l, ids, gw, None, renorm, scoring, 0.0, 0.0)
    l[1, ids[1, 0]] = INF
    got, _ = run_route(l, ids, gw, None, renorm, scoring, 0.0, 0.0)
    assert got[1, ids[1]].isnan().all() and torch.equal(got[[0, 2, 3]], clean[[0, 2, 3]])
