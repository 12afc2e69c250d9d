"""Gradients of the combine and of the router against plain 64-bit forms and differences.

Tolerances, derived from the definitions (u = 2^-24):
  dw of the combine   sums of H products in f32: at most H u of the sum of magnitudes
  deo                 two rounded products and one store rounding: bit-exact
  grad_logits         2^-16 of the sum of the magnitudes of its terms: the exponentials' arguments
                      are exact to u |l| (under 2^-18 here), sums of at most 1024 terms are trees
  grad_x              the bf16 rounding of a value within 2^-14 of the magnitudes (16-bit logits'
                      gradient, sums of at most 1024 terms)
  grad_w, grad_bias   2^-16 of the magnitudes: chains of at most 128 additions that may truncate
"""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m

from . import ref_fp8 as R
from .gpu_util import launched_since, launches

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _clear_status():
    m.lib()
    m.moe_device_status(clear=True)
    yield
    m.moe_device_status(clear=True)


def normal(seed, shape, std=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std


DT = {"f32": (torch.float32, m.F32), "bf16": (BF, m.BF16)}


# ------------------------------------------------------------------ combine
@pytest.mark.parametrize("T,K,H", [(1, 1, 8), (3, 8, 264), (37, 3, 520), (5, 64, 1032), (65, 9, 2048)])
@pytest.mark.parametrize("eo,do,deo", [(a, b, c) for a in DT for b in DT for c in DT])
def test_combine_backward(T, K, H, eo, do, deo):
    e, d = normal(T, (T, K, H)).to(DT[eo][0]), normal(H, (T, H), 0.1).to(DT[do][0])
    w = normal(K, (T, K))
    rs = 0.7
    dw = torch.full((T * K + 16,), 5.0, device=DEV)
    rows = torch.full((T * K * H + 64,), 5.0, dtype=DT[deo][0], device=DEV)
    before = launches()
    call = lambda w_, dw_, rows_: m.moe_combine_backward(
        e.to(DEV), DT[eo][1], None if w_ is None else w_.to(DEV), d.to(DEV), DT[do][1], rs, T, K, H, dw_, rows_,
        DT[deo][1])
    call(w, dw, rows)
    assert launched_since(before, "combine_backward") == 1
    assert (dw[T * K:] == 5.0).all() and (rows[T * K * H:] == 5.0).all()
    prod = e.double() * d.double()[:, None, :]
    rs32 = float(torch.tensor(rs))
    err = (dw[:T * K].cpu().double().view(T, K) - rs32 * prod.sum(2)).abs()
    assert (err <= (H + 2) * 2.0 ** -24 * rs32 * prod.abs().sum(2) + 1e-38).all()
    f = w * torch.tensor(rs)
    assert torch.equal(rows[:T * K * H].cpu().view(T, K, H), (d.float()[:, None, :] * f[:, :, None]).to(DT[deo][0]))
    # each output alone, and without weights; the same bits
    dw2, rows2 = torch.empty_like(dw), torch.empty_like(rows)
    call(w, dw2, None)
    call(w, None, rows2)
    assert torch.equal(dw2[:T * K], dw[:T * K]) and torch.equal(rows2[:T * K * H], rows[:T * K * H])
    call(None, None, rows2)
    want = (d.float()[:, None, :] * torch.tensor(rs)).to(DT[deo][0]).expand(T, K, H)
    assert torch.equal(rows2[:T * K * H].cpu().view(T, K, H), want)


# ------------------------------------------------------------------ router: logits
def problem(T, E, K, seed, spread=1.0):
    l = normal(seed, (T, E), spread)
    ids = l.topk(K, 1).indices
    off = torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(ids.reshape(-1), minlength=E).cumsum(0)])
    return l, ids, off.int(), normal(seed + 1, (T, K))


def run_route(l, ids, gw, off, renorm, scoring, balance, z, losses=True):
    T, E = l.shape
    K = ids.shape[1]
    dl = torch.full((T * E + 64,), 5.0, device=DEV)
    ls = torch.full((3,), 5.0, device=DEV)
    ws = torch.empty(max(16, m.moe_route_backward_workspace_size(T, E)), dtype=torch.uint8, device=DEV)
    m.moe_route_backward(l.to(DEV), ids.int().to(DEV), None if gw is None else gw.to(DEV),
                         None if off is None else off.to(DEV), T, E, K, renorm, scoring, balance, z, dl,
                         ls if losses else None, ws if losses else None, ws.numel() if losses else 0)
    torch.cuda.synchronize()
    assert (dl[T * E:] == 5.0).all() and float(ls[2]) == 5.0
    return dl[:T * E].cpu().view(T, E), ls[:2].cpu()


def magnitudes(l, ids, gw, off, renorm, scoring, balance, z):
    """The sum of the magnitudes of the terms of each grad_logits entry."""
    T, E = l.shape
    K = ids.shape[1]
    s = torch.sigmoid(l) if scoring else torch.softmax(l, 1)
    slope = s * torch.sigmoid(-l) if scoring else s
    picked = s.gather(1, ids)
    tot = picked.sum(1, keepdim=True)
    w = picked / tot if renorm else picked
    ga = gw.abs()
    if scoring:
        at = (ga + (ga * w).sum(1, keepdim=True)) / tot if renorm else ga
        mag = torch.zeros_like(l).scatter(1, ids, at * slope.gather(1, ids))
    else:
        mag = torch.zeros_like(l).scatter(1, ids, w * (ga + (ga * w).sum(1, keepdim=True)))
        if not renorm:
            mag = mag + s * (ga * w).sum(1, keepdim=True)
    if balance:
        f = off.double().diff() * E / (K * T)
        share = s.sum(1, keepdim=True)
        q = (f * s).sum(1, keepdim=True) / share
        mag = mag + balance / T * (f + q) * (slope / share if scoring else s)
    return mag + 2 * z / T * torch.logsumexp(l, 1, keepdim=True).abs() * torch.softmax(l, 1)


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 128, 8), (7, 3, 2), (33, 60, 6), (50, 1024, 32), (300, 257, 5)])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("scoring", [0, 1])
@pytest.mark.parametrize("balance,z", [(0.0, 0.0), (0.5, 0.0), (0.25, 0.125)])
def test_route_backward(T, E, K, renorm, scoring, balance, z):
    l, ids, off, gw = problem(T, E, K, T + E, 3.0)
    got, losses = run_route(l, ids, gw, off, renorm, scoring, balance, z)
    ld = l.double().requires_grad_()
    w, lb, lz = R.route(ld, ids, renorm, scoring, off, balance, z)
    (want,) = torch.autograd.grad((w * gw.double()).sum() + lb + lz, ld)
    mag = magnitudes(l.double(), ids, gw.double(), off, renorm, scoring, balance, z)
    assert ((got.double() - want).abs() <= 2.0 ** -16 * mag + 1e-37).all()
    for a, b in zip(losses.double(), (lb, lz)):
        assert abs(float(a) - float(b.detach())) <= 2.0 ** -16 * abs(float(b.detach())) + 1e-37
    # against differences along a random direction, token by token
    h, v = 1e-5, normal(9, (T, E)).double()

    def per_token(x):
        w, _, _ = R.route(x, ids, renorm, scoring, off, 0, 0)
        out = (w * gw.double()).sum(1)
        if balance:
            s = torch.sigmoid(x) if scoring else torch.softmax(x, 1)
            out = out + balance / T * ((off.double().diff() * E / (K * T)) * s).sum(1) / s.sum(1)
        return out + (z / T * torch.logsumexp(x, 1).square() if z else 0)
    num = (per_token(l.double() + h * v) - per_token(l.double() - h * v)) / (2 * h)
    err = ((got.double() * v).sum(1) - num).abs()
    assert (err <= 2.0 ** -16 * (mag * v.abs()).sum(1) + 1e-7 * (1 + num.abs())).all()
    again, l2 = run_route(l, ids, gw, off, renorm, scoring, balance, z)
    assert torch.equal(again, got) and torch.equal(l2, losses)
    alone, _ = run_route(l, ids, gw, off if balance else None, renorm, scoring, balance, z, losses=False)
    assert torch.equal(alone, got)


@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("scoring", [0, 1])
def test_route_backward_masked_rows(renorm, scoring):
    # row 0: some experts masked with -inf; row 1: all of them, also the chosen ones; row 2: masked by the
    # lowest f32; row 3: a NaN; row 4: very large logits; row 5 as usual
    T, E, K = 6, 40, 4
    l, _, off, gw = problem(T, E, K, 3)
    l[0, 2:] = float("-inf")                          # fewer finite logits than K
    l[1] = float("-inf")
    l[2, 5:] = torch.finfo(torch.float32).min
    l[4] = l[4] * 0 + 80 + torch.arange(E) * 0.01
    ids = torch.nan_to_num(l, neginf=-3e38).topk(K, 1).indices
    l[3, 7] = float("nan")
    got, losses = run_route(l, ids, gw, off, renorm, scoring, 0.5, 0.25)
    assert got[3].isnan().any() and torch.isnan(losses).all()
    assert (got[1] == 0).all()
    assert (got[0, 2:] == 0).all()
    for t in (0, 2, 4, 5):
        ld = l[t:t + 1].double()
        if t == 0:
            ld[0, 2:] = -1e30                         # the limit, differentiable
        ld.requires_grad_()
        w, _, lz = R.route(ld, ids[t:t + 1], renorm, scoring, off, 0, 0.25)
        s = torch.sigmoid(ld) if scoring else torch.softmax(ld, 1)
        lb = 0.5 / T * ((off.double().diff() * E / (K * T)) * s).sum() / s.sum()
        (want,) = torch.autograd.grad((w * gw[t:t + 1].double()).sum() + lb + lz / T, ld)
        tol = 2.0 ** -15 * (gw[t].abs().sum().double() + 1 + ld.detach()[0, :2].abs().max())
        assert ((got[t].double() - want[0]).abs() <= tol).all(), t
    # the fully masked token adds nothing to the losses
    keep = [0, 2, 4, 5]
    only, l1 = run_route(l[keep + [1]], ids[keep + [1]], gw[keep + [1]], off, renorm, scoring, 0.5, 0.25)
    assert torch.isfinite(l1).all() and torch.isfinite(only).all()


def test_route_backward_bad_ids_are_skipped_and_reported():
    T, E, K = 5, 16, 3
    l, ids, off, gw = problem(T, E, K, 8)
    ids = ids.clone()
    ids[2, 1], ids[3, 0] = E, -1
    got, _ = run_route(l, ids, gw, off, 0, 1, 0.0, 0.0)
    assert m.moe_device_status(clear=True) == m.STATUS_BAD_ID
    assert int((got[2] != 0).sum()) == K - 1 and int((got[3] != 0).sum()) == K - 1


def test_route_backward_without_tokens():
    losses = torch.full((2,), 5.0, device=DEV)
    m.moe_route_backward(None, None, None, losses, 0, 8, 2, 1, 0, 0.5, 0.5, None, losses, None, 0)
    assert (losses == 0).all()


# ------------------------------------------------------------------ router: products
@pytest.mark.parametrize("T,H,E", [(1, 8, 1), (1, 2048, 128), (130, 264, 3), (300, 1032, 60), (2050, 136, 128),
                                   (513, 520, 257), (64, 64, 1024), (5000, 128, 16)])
def test_route_logits_backward(T, H, E):
    dl = normal(T, (T, E), 0.1)
    dl[:, ::3] *= 1e-4                                # columns of very different sizes
    x, w = normal(H, (T, H)).to(BF), normal(E, (E, H), 0.05).to(BF)
    n = m.moe_route_logits_backward_workspace_size(T, H, E)
    ws = torch.empty(max(16, n), dtype=torch.uint8, device=DEV)

    def call(dx, dw, db):
        m.moe_route_logits_backward(dl.to(DEV), x.to(DEV), w.to(DEV), T, H, E, dx, dw, db, ws, ws.numel())
        torch.cuda.synchronize()
    dx = torch.full((T * H + 64,), 5.0, dtype=BF, device=DEV)
    dw = torch.full((E * H + 64,), 5.0, device=DEV)
    db = torch.full((E + 16,), 5.0, device=DEV)
    call(dx, dw, db)
    assert (dx[T * H:] == 5.0).all() and (dw[E * H:] == 5.0).all() and (db[E:] == 5.0).all()
    d, xd, wd = dl.double(), x.double(), w.double()
    y, mag = d @ wd, d.abs() @ wd.abs()
    lo, hi = R.bf16_between(y, 2.0 ** -14 * mag + 1e-38)
    got = dx[:T * H].cpu().double().view(T, H)
    assert ((lo <= got) & (got <= hi)).all()
    y, mag = d.t() @ xd, d.abs().t() @ xd.abs()
    assert ((dw[:E * H].cpu().double().view(E, H) - y).abs() <= 2.0 ** -16 * mag + 1e-38).all()
    assert ((db[:E].cpu().double() - d.sum(0)).abs() <= 2.0 ** -16 * d.abs().sum(0) + 1e-38).all()
    # any one output alone, and again: the same bits
    dx2, dw2, db2 = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
    call(dx2, None, None)
    call(None, dw2, None)
    call(None, None, db2)
    assert torch.equal(dx2[:T * H], dx[:T * H]) and torch.equal(dw2[:E * H], dw[:E * H])
    assert torch.equal(db2[:E], db[:E])


def test_route_logits_backward_without_tokens():
    H, E = 64, 8
    dw, db = torch.ones((E, H), device=DEV), torch.ones((E,), device=DEV)
    m.moe_route_logits_backward(None, None, None, 0, H, E, None, dw, db, None, 0)
    assert (dw == 0).all() and (db == 0).all()
