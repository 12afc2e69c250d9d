"""FP8 expert products and their data gradient against plain 64-bit forms.

The quantiser and the transpose are bit-exact.  A product's tolerance is derived from its
definition: with A = sum of the magnitudes of the terms, out is the bf16 rounding of a value
within 2^-15 A of y, so it lies between the roundings of y - 2^-15 A and y + 2^-15 A.  That
bounds the f32 accumulation: within a block of 128 columns at most 128
additions, each losing at most 2^-23 of A's share (2^-16 A), and the at most 32 joins of blocks
2^-18 A more.  Codes formed from f32 values inside a kernel (the SiLU paths) have to lie within
half a step of E4M3 of the 64-bit value, plus 2^-17 of its magnitude for the fast exponential
(under 2^-19 for the arguments here), the division and the scale.
"""
from __future__ import annotations

import numpy as np
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
    assert m.moe_device_status() == 0


def rows(seed, shape, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std)


def weights(seed, G, N, K):
    w = rows(seed, (G, R.blocks(N) * 128, R.blocks(K) * 128), 0.05)
    w = w.view(G, R.blocks(N), 128, R.blocks(K), 128)
    s = w.abs().amax((2, 4)) / 448.0
    c = (w / s[:, :, None, :, None]).to(R.E4M3).view(torch.uint8)
    return c.reshape(G, R.blocks(N) * 128, R.blocks(K) * 128)[:, :N, :K].contiguous(), s.contiguous()


def offsets(sizes):
    return torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32)


def guarded(shape, dtype, fill):
    """A tensor with 64 guard rows of `fill` behind it (and filled itself)."""
    full = torch.full((shape[0] + 64, *shape[1:]), fill, dtype=dtype, device=DEV)
    return full, full[:shape[0]]


def check_product(out, y, mag, what=""):
    lo, hi = R.bf16_between(y, 2.0 ** -15 * mag + 1e-38)
    bad = ((out.double() < lo) | (out.double() > hi) | out.isnan()).nonzero()
    assert bad.numel() == 0, f"{what}: {bad.shape[0]} off, first {bad[0].tolist()}: " \
        f"{out[tuple(bad[0])]} for {y[tuple(bad[0])]}"


def check_codes(codes, scales, v, mag):
    """codes/scales hold v (f64) as nearest E4M3 values of v / d, d from the row's blocks."""
    C = v.shape[1]
    for b in range(R.blocks(C)):
        c = slice(128 * b, min(C, 128 * b + 128))
        d = scales[:, b].double()
        want = torch.maximum(v[:, c].abs().amax(1) / 448.0, torch.tensor(2.0 ** -126, dtype=torch.float64))
        slack = 2.0 ** -17 * mag[:, c].amax(1) / 448.0 + 2.0 ** -22 * want
        assert ((d - want).abs() <= slack).all()
        q = v[:, c] / d[:, None]
        got = codes[:, c].view(R.E4M3).double()
        tol = R.e4m3_half_step(q) + 2.0 ** -17 * mag[:, c] / d[:, None]
        assert ((got - q).abs() <= tol).all()


# ------------------------------------------------------------------ quantiser
@pytest.mark.parametrize("T,H,K", [(1, 16, 1), (1, 2048, 8), (3, 144, 2), (37, 1040, 3), (5, 512, 64),
                                   (300, 2064, 1)])
@pytest.mark.parametrize("form", ["plain", "placed", "weighted"])
def test_quantiser_is_bit_exact(T, H, K, form):
    x = rows(T + H, (T, H)).to(BF)
    x[0, :16] = 0                                     # a block of zeros where H = 16
    x[-1] *= 1e-38                                    # subnormal blocks meet the scale's floor
    P = T * K
    g = torch.Generator().manual_seed(K)
    place = torch.randperm(P, generator=g).int() if form != "plain" else None
    pw = (torch.rand(P, generator=g) - 0.3) if form == "weighted" else None
    rs = 0.7 if form == "weighted" else 1.0
    v = x.float().repeat_interleave(K, 0)
    f = torch.full((P,), rs) if pw is None else pw * torch.tensor(rs)
    want_c, want_s = R.quantise(v * f[:, None])
    if place is not None:
        inv = torch.argsort(place.long())
        want_c, want_s = want_c[inv], want_s[inv]
    full_c, c = guarded((P, H), torch.uint8, 0x5A)
    full_s, s = guarded((P, R.blocks(H)), torch.float32, 7.0)
    before = launches()
    m.moe_quantize_act_fp8(x.to(DEV), T, H, K, None if place is None else place.to(DEV),
                           None if pw is None else pw.to(DEV), rs, c, s)
    assert launched_since(before, "quant_fp8") == 1
    assert torch.equal(s.cpu(), want_s)
    assert torch.equal(c.cpu(), want_c)
    assert (full_c[P:] == 0x5A).all() and (full_s[P:] == 7.0).all()


def test_quantiser_special_values_and_rows_outside():
    # NaN becomes a NaN code and leaves its block's scale to the others; an infinity makes the
    # scale infinite and the row NaN; destinations outside [0, T*K) are skipped
    x = rows(1, (4, 256)).to(BF)
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    place = torch.tensor([0, 1, 2, 4], dtype=torch.int32)
    full_c, c = guarded((4, 256), torch.uint8, 0x5A)
    full_s, s = guarded((4, 2), torch.float32, 7.0)
    m.moe_quantize_act_fp8(x.to(DEV), 4, 256, 1, place.to(DEV), None, 1.0, c, s)
    want_c, want_s = R.quantise(x.float())
    assert torch.equal(s.cpu()[:2], want_s[:2])
    got = c.cpu().view(R.E4M3).float()
    assert got[1, 5].isnan() and not got[1, :5].isnan().any()
    assert torch.equal(got[0], want_c.view(R.E4M3).float()[0])
    assert s[2, 1].isinf() and got[2, 200].isnan() and not got[2, :128].isnan().any()
    assert (full_c[3:] == 0x5A).all() and (full_s[3:] == 7.0).all()


# ------------------------------------------------------------------ products
SHAPES = [
    # sizes of the groups, K, N
    ([1], 2048, 136),
    ([1], 16, 8),
    ([0, 3, 0, 1, 0], 144, 264),
    ([17, 130, 5], 272, 200),
    ([300, 0, 31, 33, 2], 1040, 120),
    ([513], 128, 392),
    ([64, 64, 64, 64], 384, 256),
    ([1500, 700], 256, 520),
    ([2] * 40, 528, 128),
    # several tiles per SM pair, tiles of one and of two parts in turn, 6 and 3 scale blocks
    ([300, 90] * 20, 768, 1032),
    ([129, 500, 30] * 12, 384, 1544),
]


@pytest.mark.parametrize("sizes,K,N", SHAPES)
@pytest.mark.parametrize("form", ["plain", "down"])
def test_product(sizes, K, N, form):
    G, P = len(sizes), sum(sizes) + 3                # three rows outside every group
    a, sa = R.quantise(rows(P, (P, K)))
    w, sw = weights(N, G, N, K)
    off = offsets(sizes)
    y, mag = R.grouped(R.row_values(a, sa), R.weight_values(w, sw), off)
    g = torch.Generator().manual_seed(K)
    dst = torch.randperm(P, generator=g).int() if form == "down" else None
    pw = torch.rand(P, generator=g) if form == "down" else None
    full, out = guarded((P, N), BF, 3.0)
    before = launches()
    args = (a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), off.to(DEV), None if pw is None else pw.to(DEV),
            None if dst is None else dst.to(DEV), P, K, N, G)
    m.moe_grouped_gemm_fp8(*args, out)
    assert launched_since(before, "gemm_fp8") >= 1
    n = int(off[-1])
    got = out.cpu()
    assert (full[P:] == 3.0).all()
    if dst is None:
        assert (got[n:] == 3.0).all()
    else:
        assert (got[dst[n:].long()] == 3.0).all()
        got = got[dst.long()]
        y, mag = (t * pw[dst.long()].double()[:, None] for t in (y, mag))
    check_product(got[:n], y[:n], mag[:n], f"{sizes} {K} {N} {form}")
    again = torch.empty_like(out)
    m.moe_grouped_gemm_fp8(*args, again)
    rows_written = torch.arange(n) if dst is None else dst[:n].long()
    assert torch.equal(again.cpu()[rows_written], out.cpu()[rows_written])


def test_product_of_one_group_without_offsets_on_another_stream():
    P, K, N = 70, 400, 336
    a, sa = R.quantise(rows(2, (P, K)))
    w, sw = weights(3, 1, N, K)
    y, mag = R.grouped(R.row_values(a, sa), R.weight_values(w, sw), [0, P])
    d = [t.to(DEV) for t in (a, sa, w, sw)]
    out = torch.empty((P, N), dtype=BF, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    m.moe_grouped_gemm_fp8(*d, None, None, None, P, K, N, 1, out, stream=s)
    s.synchronize()
    check_product(out.cpu(), y, mag)


def test_product_keeps_a_bad_row_to_itself():
    # a NaN code makes its own row NaN, an infinite scale its own row not finite; rows of zeros give
    # zeros; a destination outside [0, P) is skipped; offsets beyond P are clamped
    P, K, N, G = 40, 256, 128, 2
    a, sa = R.quantise(rows(4, (P, K)))
    a[3, 77] = 0x7F
    sa[20, 1] = float("inf")
    a[30] = 0
    w, sw = weights(5, G, N, K)
    off = torch.tensor([0, 25, P + 1000], dtype=torch.int32)
    dst = torch.arange(P, dtype=torch.int32)
    dst[7] = P
    dst[8] = -1
    full, out = guarded((P, N), BF, 3.0)
    m.moe_grouped_gemm_fp8(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), off.to(DEV), None, dst.to(DEV),
                           P, K, N, G, out)
    got = out.cpu()
    assert got[3].isnan().all() and not got[20].isfinite().any() and (got[30] == 0).all()
    assert (got[7:9] == 3.0).all() and (full[P:] == 3.0).all()
    y, mag = R.grouped(R.row_values(a, sa), R.weight_values(w, sw), [0, 25, P])
    keep = [i for i in range(P) if i not in (3, 20, 7, 8)]
    check_product(got[keep], y[keep], mag[keep])


@pytest.mark.parametrize("sizes,H,I", [([1], 2048, 16), ([5, 0, 40], 144, 208), ([17, 130, 5], 272, 400),
                                       ([300, 33], 1040, 128), ([2] * 20, 528, 48), ([700], 256, 1024),
                                       ([300, 90] * 12, 768, 1040), ([129, 500, 30] * 8, 384, 912)])
@pytest.mark.parametrize("keep", [True, False])
def test_gateup(sizes, H, I, keep):
    G, P = len(sizes), sum(sizes) + 2
    a, sa = R.quantise(rows(P, (P, H)))
    w, sw = weights(I, G, 2 * I, H)
    off = offsets(sizes)
    y, mag = R.grouped(R.row_values(a, sa), R.weight_values(w, sw), off)
    full_c, c = guarded((P, I), torch.uint8, 0x5A)
    full_s, s = guarded((P, R.blocks(I)), torch.float32, 7.0)
    full_g, gu = guarded((P, 2 * I), BF, 3.0)
    d = [t.to(DEV) for t in (a, sa, w, sw, off)]
    before = launches()
    m.moe_grouped_gemm_gateup_silu_fp8(*d, P, H, I, G, gu, c, s)
    assert launched_since(before, "gemm_fp8_gateup") >= 1
    n = int(off[-1])
    assert (full_g[n:] == 3.0).all() and (full_c[n:] == 0x5A).all() and (full_s[n:] == 7.0).all()
    gate_up = gu.cpu()[:n]
    check_product(gate_up, y[:n], mag[:n])
    # the activation of the narrowed gate and up rows, as codes
    g, u = gate_up.double().split(I, 1)
    v = g * torch.sigmoid(g) * u
    check_codes(c.cpu()[:n], s.cpu()[:n], v, v.abs())
    if not keep:   # the same codes without the gate and up rows
        c2, s2 = torch.empty_like(c), torch.empty_like(s)
        m.moe_grouped_gemm_gateup_silu_fp8(*d, P, H, I, G, None, c2, s2)
        assert torch.equal(c2[:n], c[:n]) and torch.equal(s2[:n], s[:n])


# ------------------------------------------------------------------ data gradient
@pytest.mark.parametrize("P,I", [(1, 16), (3, 144), (37, 400), (130, 768), (9, 1024)])
def test_silu_mul_backward(P, I):
    gu = rows(P, (P, 2 * I), 2.0).to(BF)
    da = rows(I, (P, I), 0.1).to(BF)
    gu[0, :3] = torch.tensor([90.0, -90.0, 0.0])      # the sigmoid's ends
    full_c, c = guarded((P, 2 * I), torch.uint8, 0x5A)
    full_s, s = guarded((P, R.blocks(2 * I)), torch.float32, 7.0)
    m.moe_silu_mul_backward_fp8(gu.to(DEV), da.to(DEV), P, I, c, s)
    v, mag = R.silu_mul_backward(*gu.double().split(I, 1), da.double())
    check_codes(c.cpu(), s.cpu(), v, mag)
    assert (full_c[P:] == 0x5A).all() and (full_s[P:] == 7.0).all()
    # against differences of the forward activation
    g, u = gu.double().split(I, 1)
    f = lambda g, u: (g * torch.sigmoid(g) * u * da.double())
    h = 1e-5
    num = torch.cat([f(g + h, u) - f(g - h, u), f(g, u + h) - f(g, u - h)], 1) / (2 * h)
    assert ((num - v).abs() <= 1e-8 * (1 + v.abs())).all()
    got = R.row_values(c.cpu(), s.cpu())
    assert float((got - num).norm() / num.norm()) < 2.0 ** -4   # half a step of E4M3 at most


@pytest.mark.parametrize("G,Rr,C", [(1, 16, 16), (3, 144, 272), (2, 400, 128), (5, 256, 1040)])
def test_transpose(G, Rr, C):
    w, s = weights(C, G, Rr, C)
    full_w, wt = guarded((G, C, Rr), torch.uint8, 0x5A)
    full_s, st = guarded((G, R.blocks(C), R.blocks(Rr)), torch.float32, 7.0)
    m.moe_transpose_fp8w(w.to(DEV), s.to(DEV), G, Rr, C, wt, st)
    assert torch.equal(wt.cpu(), w.transpose(1, 2)) and torch.equal(st.cpu(), s.transpose(1, 2))
    assert (full_w[G:] == 0x5A).all() and (full_s[G:] == 7.0).all()


@pytest.mark.parametrize("sizes,K,N", [([4, 0, 0, 5, 7], 4096, 1024), ([0] * 40 + [1] + [0] * 90 + [2], 1040, 392),
                                       ([16], 528, 1000), ([17], 528, 960), ([9], 2048, 1816), ([1] * 700, 144, 128)])
def test_few_rows_and_the_tiles_beyond(sizes, K, N):
    # either side of the bounds on rows and products, and more groups than one launch of the tiles holds
    test_product(sizes, K, N, "down")
    if N % 16 == 0:
        test_gateup(sizes, K, N // 2 // 16 * 16, True)


def test_empty_calls_launch_nothing():
    before = launches()
    assert m.moe_quantize_act_fp8(None, 0, 64, 2, None, None, 1.0, None, None) == m.OK
    assert m.moe_grouped_gemm_fp8(None, None, None, None, None, None, None, 0, 64, 64, 3, None) == m.OK
    assert m.moe_grouped_gemm_gateup_silu_fp8(None, None, None, None, None, 0, 64, 64, 3, None, None,
                                              None) == m.OK
    assert m.moe_silu_mul_backward_fp8(None, None, 0, 64, None, None) == m.OK
    assert launches() == before
