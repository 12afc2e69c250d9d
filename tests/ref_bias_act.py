"""The grouped products with bias, activation and residual, and their gradients, in 64 bits, with
bounds on what 32-bit arithmetic and the roundings of the outputs may add.

Bounds: a rounding to bf16 is off by at most 2^-8 of the value, one to f32 by 2^-24.  The tensor
core adds 16 products at a time to an f32 accumulator and may cut bits off there: 2^-23 of the
sum of magnitudes for each of those steps, which also covers f32 additions of the sums.
APPROX: the fast exponential, reciprocal and Phi of the activations, absolute error in units of
|z| (Phi: 0.75e-7 from its series, twice that with its own roundings) plus relative error.
"""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24
UBF = 2.0 ** -8
REL = 2.0 ** -19
PHI = 2.0e-7
NONE, RELU, RELU2, GELU, GELU_TANH, SILU = range(6)


def act(z, kind):
    f = torch.nn.functional
    return [lambda v: v, torch.relu, lambda v: torch.relu(v) ** 2, f.gelu,
            lambda v: f.gelu(v, approximate="tanh"), f.silu][kind](z)


def slope(z, kind):
    z = z.detach().clone().requires_grad_()
    (s,) = torch.autograd.grad(act(z, kind).sum(), z)
    return s


def groups(off, P, G):
    off = [0, P] if off is None else off.tolist()
    lo = [min(max(o, 0), P) for o in off]
    return [(g, lo[g], lo[g + 1]) for g in range(G) if lo[g] < lo[g + 1]]


def product(a, w, columns, bias, kind, off, G):
    """(z, bound of its f32 value, y, bound) [P, N] in row order; NaN in rows of no group."""
    P, N = a.shape[0], w.shape[2] if columns else w.shape[1]
    K = a.shape[1]
    z = torch.full((P, N), float("nan"), dtype=torch.float64, device=a.device)
    dz = z.clone()
    for g, lo, hi in groups(off, P, G):
        wg = w[g].double() if columns else w[g].double().t()
        z[lo:hi] = a[lo:hi].double() @ wg
        mag = a[lo:hi].double().abs() @ wg.abs()
        if bias is not None:
            z[lo:hi] += bias[g].double()
            mag += bias[g].double().abs()
        dz[lo:hi] = (math.ceil(K / 16) + 32) * 2 * U32 * mag
    y = act(z, kind)
    lip = 2.0 * (z.abs() + dz) if kind == RELU2 else 1.0 if kind in (NONE, RELU) else 1.2
    dy = lip * dz + (0 if kind == NONE else REL * y.abs() + PHI * z.abs())
    return z, dz, y, dy


def placed(y, dy, dst, pw, residual):
    """Rows at their destinations with weight and residual, and the bound of the bf16 result; rows
    that nothing reaches are NaN."""
    P = y.shape[0]
    out, bound = torch.full_like(y, float("nan")), torch.full_like(y, float("nan"))
    rows = torch.arange(P, device=y.device)
    to = rows if dst is None else dst.long()
    ok = (to >= 0) & (to < P) & ~y.isnan().all(1)
    w = torch.ones(P, dtype=torch.float64, device=y.device) if pw is None else pw.double()
    out[to[ok]] = y[ok] * w[to[ok], None]
    bound[to[ok]] = (dy[ok] + 2 * U32 * y[ok].abs()) * w[to[ok], None].abs()
    if residual is not None:
        out = out + residual.double()
        bound = bound + U32 * out.abs()
    return out, bound + UBF * (out.abs() + bound)


def check(got, want, bound, keep, what=""):
    """got within bound where want is a number, untouched (equal to keep) elsewhere."""
    none = want.isnan()
    off = (got.double() - want).abs()
    bad = ~none & ~(off <= bound)
    assert not bad.any(), f"{what}: off by {(off / bound)[bad].max().item():.2f} of the bound at {bad.nonzero()[:4].tolist()}"
    if keep is not None:
        assert torch.equal(got[none], keep[none]), f"{what}: rows that no group has were written"
