"""FP8 products of few rows, where a warp reads the weights, against the same 64-bit forms as the
tiles; either side of the rule that chooses; and long contractions on tiles.

The bound of the tiles' products (test_gpu_fp8.py) holds for few rows too: 16 exact products in a
chain of 16 f32 additions, at most 9 joins a lane and 5 across the lanes, a scale and a weight:
under 40 * 2^-24 of the sum of magnitudes, far below 2^-15.
"""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m

from . import ref_fp8 as R
from .gpu_util import launched_since, launches
from .test_gpu_fp8 import BF, DEV, check_codes, check_product, guarded, offsets, rows, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_status():
    m.lib()
    m.moe_device_status(clear=True)
    yield
    assert m.moe_device_status() == 0


def product(sizes, K, N, extra, form, few):
    G, P = len(sizes), sum(sizes) + extra
    a, sa = R.quantise(rows(P + K, (P, K)))
    w, sw = weights(N, G, N, K)
    off = offsets(sizes)
    y, mag = R.grouped(R.row_values(a, sa), R.weight_values(w, sw), off)
    g = torch.Generator().manual_seed(K)
    dst = torch.randperm(P, generator=g).int() if form == "down" else None
    pw = torch.rand(P, generator=g) if form == "down" else None
    full, out = guarded((P, N), BF, 3.0)
    before = launches()
    m.moe_grouped_gemm_fp8(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), off.to(DEV),
                           None if pw is None else pw.to(DEV), None if dst is None else dst.to(DEV), P, K, N, G, out)
    assert launched_since(before, "gemm_fp8") >= 1 and launched_since(before, "gemm_fp8_few") == int(few)
    n, got = sum(sizes), out.cpu()
    assert (full[P:] == 3.0).all()
    if dst is not None:
        got = got[dst.long()]
        y, mag = (t * pw[dst.long()].double()[:, None] for t in (y, mag))
    assert (got[n:] == 3.0).all()
    check_product(got[:n], y[:n], mag[:n], f"{sizes} {K} {N} {form}")


def gateup(sizes, H, I, extra, few):
    G, P = len(sizes), sum(sizes) + extra
    a, sa = R.quantise(rows(P + H, (P, H)))
    w, sw = weights(I, G, 2 * I, H)
    off = offsets(sizes)
    y, mag = R.grouped(R.row_values(a, sa), R.weight_values(w, sw), off)
    full_c, c = guarded((P, I), torch.uint8, 0x5A)
    full_s, s = guarded((P, R.blocks(I)), torch.float32, 7.0)
    full_g, gu = guarded((P, 2 * I), BF, 3.0)
    d = [t.to(DEV) for t in (a, sa, w, sw, off)]
    before = launches()
    m.moe_grouped_gemm_gateup_silu_fp8(*d, P, H, I, G, gu, c, s)
    assert launched_since(before, "gemm_fp8_gateup") >= 1 and launched_since(before, "gemm_fp8_few") == int(few)
    n = sum(sizes)
    assert (full_g[n:] == 3.0).all() and (full_c[n:] == 0x5A).all() and (full_s[n:] == 7.0).all()
    gate_up = gu.cpu()[:n]
    check_product(gate_up, y[:n], mag[:n])
    g, u = gate_up.double().split(I, 1)
    v = g * torch.sigmoid(g) * u
    check_codes(c.cpu()[:n], s.cpu()[:n], v, v.abs())
    c2, s2 = torch.empty_like(c), torch.empty_like(s)
    m.moe_grouped_gemm_gateup_silu_fp8(*d, P, H, I, G, None, c2, s2)
    assert torch.equal(c2[:n], c[:n]) and torch.equal(s2[:n], s[:n])


@pytest.mark.parametrize("sizes,K,N,extra,few", [
    ([1], 16, 8, 0, True),
    ([1], 4096, 1024, 0, True),
    ([1], 4096, 16384, 0, True),                       # 16384 products, and one row of columns more
    ([1], 144, 16392, 0, False),
    ([16], 528, 1000, 0, True),
    ([16], 528, 1024, 0, True),                        # 16384 products
    ([16], 528, 1032, 0, False),
    ([17], 528, 960, 0, False),
    ([9], 2048, 1816, 0, True),
    ([9], 2048, 1824, 0, False),
    ([4, 0, 0, 5, 7], 4096, 1024, 0, True),
    ([0, 3, 0, 1, 0], 144, 264, 2, True),              # rows outside every group
    ([0] * 40 + [1] + [0] * 90 + [2], 1040, 392, 0, True),
    ([1] * 16, 1552, 120, 0, True),
    ([0] * 700 + [2, 0, 1], 80, 136, 1, True),
])
@pytest.mark.parametrize("form", ["plain", "down"])
def test_product_of_few_rows(sizes, K, N, extra, few, form):
    product(sizes, K, N, extra, form, few)


@pytest.mark.parametrize("sizes,H,I,extra,few", [
    ([1], 16, 16, 0, True),
    ([1, 0, 2], 144, 208, 0, True),                    # the up rows begin inside a scale block
    ([3], 2064, 208, 1, True),
    ([2, 0, 1, 5], 1040, 768, 0, True),                # six clusters of features a row
    ([1] * 8, 2048, 768, 0, True),
    ([5], 528, 1040, 2, True),
    ([16], 272, 512, 0, True),                         # 16384 products
    ([16], 272, 528, 0, False),
    ([17], 272, 400, 0, False),
    ([1], 4112, 4096 * 2, 0, True),
    ([0] * 40 + [1] + [0] * 90 + [2], 400, 144, 0, True),
])
def test_gateup_of_few_rows(sizes, H, I, extra, few):
    gateup(sizes, H, I, extra, few)


def test_few_rows_keep_a_bad_row_to_themselves():
    # as on tiles: a NaN code makes its own row NaN, an infinite scale its own row not finite, rows of
    # zeros give zeros, a destination outside [0, P) is skipped, offsets beyond P are clamped
    P, K, N, G = 12, 256, 128, 2
    a, sa = R.quantise(rows(4, (P, K)))
    a[3, 77] = 0x7F
    sa[5, 1] = float("inf")
    a[10] = 0
    w, sw = weights(5, G, N, K)
    off = torch.tensor([0, 6, P + 1000], dtype=torch.int32)
    dst = torch.arange(P, dtype=torch.int32)
    dst[7] = P
    dst[8] = -1
    full, out = guarded((P, N), BF, 3.0)
    before = launches()
    m.moe_grouped_gemm_fp8(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), off.to(DEV), None, dst.to(DEV),
                           P, K, N, G, out)
    assert launched_since(before, "gemm_fp8_few") == 1
    got = out.cpu()
    assert got[3].isnan().all() and not got[5].isfinite().any() and (got[10] == 0).all()
    assert (got[7:9] == 3.0).all() and (full[P:] == 3.0).all()
    y, mag = R.grouped(R.row_values(a, sa), R.weight_values(w, sw), [0, 6, P])
    keep = [i for i in range(P) if i not in (3, 5, 7, 8)]
    check_product(got[keep], y[keep], mag[keep])


@pytest.mark.parametrize("P", [7, 40, 200])
def test_gateup_keeps_a_bad_row_to_itself(P):
    # few rows, weights tiles and rows tiles: a NaN code makes every activation of its row a NaN code,
    # and the scale of a block that holds nothing else is the floor
    H, I = 256, 144
    a, sa = R.quantise(rows(P, (P, H)))
    clean = a.clone()
    a[3, 77] = 0x7F
    w, sw = weights(6, 1, 2 * I, H)
    outs = []
    for x in (a, clean):
        gu = torch.empty((P, 2 * I), dtype=BF, device=DEV)
        c, s = torch.empty((P, I), dtype=torch.uint8, device=DEV), torch.empty((P, 2), device=DEV)
        before = launches()
        m.moe_grouped_gemm_gateup_silu_fp8(x.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), None, P, H, I, 1, gu, c, s)
        assert launched_since(before, "gemm_fp8_few") == int(P == 7)
        outs.append((gu.cpu(), c.cpu(), s.cpu()))
    (gu, c, s), want = outs
    assert gu[3].isnan().all() and c[3].view(R.E4M3).float().isnan().all() and (s[3] == 2.0 ** -126).all()
    keep = [i for i in range(P) if i != 3]
    assert all(torch.equal(x[keep], y[keep]) for x, y in zip((gu, c, s), want))


# 18 to 32 scale blocks a row: the tiles' two chunks of eight blocks' scales wrap within a tile
@pytest.mark.parametrize("sizes,K,N", [([300, 90], 2320, 520), ([129, 70], 4096, 264), ([33, 5, 64], 2320, 264),
                                       ([130] * 30, 2576, 1032)])
@pytest.mark.parametrize("form", ["plain", "down"])
def test_product_of_long_rows(sizes, K, N, form):
    product(sizes, K, N, 3, form, False)


@pytest.mark.parametrize("sizes,H,I", [([300, 33], 2320, 208), ([129], 4096, 128), ([40, 7, 64], 2576, 400),
                                       ([130] * 20, 2320, 912)])
def test_gateup_of_long_rows(sizes, H, I):
    gateup(sizes, H, I, 2, False)
