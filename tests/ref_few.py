"""The few-token MoE layer and the grouped products with bias and activation in 64 bits, with
bounds on what 32-bit arithmetic and the roundings of the outputs may add.

Bounds: a rounding to bf16 is off by at most 2^-8 of the value (half of torch's eps), one to f32
by 2^-24.  A sum of n products in f32, in any order, is off by at most n 2^-24 times the sum of
their magnitudes; the kernels add at most CHAIN terms one after the other (8 columns of a lane or
16 of an MMA, a butterfly, then segments or K steps), so CHAIN stands for n.
"""
from __future__ import annotations

import torch

U32 = 2.0 ** -24
UBF = 2.0 ** -8
CHAIN = 128          # longest chain of f32 additions behind one value of the tested sizes
EXP = 2.0 ** -20     # relative error of the fast exponential and division in silu, generously


def dequant(codes, scale):
    R, C = codes.shape[-2:]
    s = scale.double().repeat_interleave(128, -2)[..., :R, :].repeat_interleave(128, -1)[..., :C]
    return codes.view(torch.float8_e4m3fn).double() * s


def swiglu(x, w13, w2):
    """(y, bound of |f32 y - y|) of one expert, x [H], w13 [2I, H], w2 [H, I], all f64."""
    g, u = (w13 @ x).chunk(2)
    mg, mu = (w13.abs() @ x.abs()).chunk(2)
    dg, du = CHAIN * U32 * mg, CHAIN * U32 * mu
    sg = g * torch.sigmoid(g)
    act = sg * u
    # |silu'| <= 1.1
    dact = 1.1 * dg * (u.abs() + du) + sg.abs() * du + EXP * act.abs()
    y = w2 @ act
    return y, w2.abs() @ dact + CHAIN * U32 * (w2.abs() @ (act.abs() + dact))


def layer(x, ids, w, w13, w2, scale, shared=None, residual=None):
    """Output and its bound [T, H], given the choice.  w13(e), w2(e): f64 weights of expert e.
    shared: (w_gate or None, w13, w2)."""
    T, H = x.shape
    out = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(out)
    for t in range(T):
        xt = x[t].double()
        terms = []
        for j in range(ids.shape[1]):
            y, d = swiglu(xt, w13(int(ids[t, j])), w2(int(ids[t, j])))
            f = float(w[t, j]) * scale
            terms.append((f * y, abs(f) * (d + 4 * U32 * y.abs())))
        if shared is not None:
            y, d = swiglu(xt, shared[1].double(), shared[2].double())
            gate = 1.0
            dg = 0.0
            if shared[0] is not None:
                wg = shared[0].double()
                gate = float(torch.sigmoid(wg @ xt))
                dg = CHAIN * U32 * float(wg.abs() @ xt.abs()) + 4 * U32
            terms.append((gate * y, gate * d + dg * y.abs()))
        if residual is not None:
            terms.append((residual[t].double(), torch.zeros_like(out[t])))
        v = sum(a for a, _ in terms)
        mag = sum(a.abs() for a, _ in terms)
        err = sum(b for _, b in terms) + len(terms) * U32 * mag
        out[t] = v
        bound[t] = err + UBF * (v.abs() + err)
    return out, bound
