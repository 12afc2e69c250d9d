"""moe_grouped_gemm_bias_act_bf16, moe_bias_act_backward and moe_grouped_gemm_wgrad_bf16 against
their formulas in 64 bits."""
from __future__ import annotations

import math

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m

from . import ref_bias_act as R
from .gpu_util import DEV, launched_since, launches

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rng(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, shape, std=1.0, dt=BF):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dt)


def offsets(sizes, first=0):
    return torch.tensor([first] + sizes, device=DEV).cumsum(0).to(torch.int32)


def ws_of(size):
    return torch.full((max(16, size),), 0xFF, dtype=torch.uint8, device=DEV)     # NaN: nothing is assumed of it


class Product:
    def __init__(self, P, K, N, G=1, off=None, columns=False, bias=True, kind=0, pre=False, scatter=False,
                 weight=False, residual=False, seed=0):
        g = rng(P * 7 + K * 3 + N + seed)
        self.P, self.K, self.N, self.G, self.off, self.columns, self.kind = P, K, N, G, off, columns, kind
        self.a = normal(g, (P, K))
        self.w = normal(g, (G, K, N) if columns else (G, N, K), K ** -0.5)
        self.bias = normal(g, (G, N), 0.5, torch.float32) if bias else None
        self.dst = torch.randperm(P, generator=g, device=DEV).to(torch.int32) if scatter else None
        self.pw = torch.rand((P,), generator=g, device=DEV) + 0.25 if weight else None
        self.res = normal(g, (P, N)) if residual else None
        self.out = normal(g, (P, N))
        self.pre = normal(g, (P, N)) if pre else None
        self.ws = ws_of(m.moe_grouped_gemm_bias_act_workspace_size(P, K, N, G))

    def call(self, out=None, ws=True, stream=None, residual=None):
        out = self.out if out is None else out
        ws = self.ws if ws is True else ws
        m.moe_grouped_gemm_bias_act_bf16(
            self.a, self.w, m.W_COLUMNS if self.columns else m.W_ROWS, self.bias, self.kind, self.pre, self.pw, self.dst,
            self.res if residual is None else residual, self.off, self.P, self.K, self.N, self.G, out, ws,
            0 if ws is None else ws.numel(), stream)
        return out

    def run(self):
        keep, keep_z = self.out.clone(), None if self.pre is None else self.pre.clone()
        self.call()
        torch.cuda.synchronize()
        self.check(self.out, keep, keep_z)

    def check(self, out, keep=None, keep_z=None):
        z, dz, y, dy = R.product(self.a, self.w, self.columns, self.bias, self.kind, self.off, self.G)
        want, bound = R.placed(y, dy, self.dst, self.pw, self.res)
        R.check(out, want, bound, keep, "out")
        if self.pre is not None:
            R.check(self.pre, z, dz + R.UBF * (z.abs() + dz), keep_z, "pre_act")


SHAPES = [
    # P, K, N, sizes of the groups
    (1, 8, 8, None),
    (1, 4096, 1024, None),
    (5, 72, 264, None),
    (64, 4096, 512, None),
    (300, 136, 1000, None),
    (1000, 1040, 776, None),
    (777, 1040, 1000, [0, 1, 300, 0, 17, 255, 204, 0]),
    (600, 64, 256, [256, 257, 87]),
    (40, 200, 328, [3, 0, 5, 32]),
]


@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:3])) + ("g" if s[3] else ""))
def test_product(shape, columns):
    P, K, N, sizes = shape
    Product(P, K, N, len(sizes) if sizes else 1, offsets(sizes) if sizes else None, columns).run()


@pytest.mark.parametrize("kind", range(6))
@pytest.mark.parametrize("P", [3, 700])
@pytest.mark.parametrize("pre,weight,residual", [(False, False, False), (True, True, False), (False, True, True),
                                                 (True, False, True)])
def test_epilogue(kind, P, pre, weight, residual):
    Product(P, 264, 392, 2, offsets([P // 3, P - P // 3]), kind=kind, pre=pre, scatter=weight, weight=weight,
            residual=residual).run()
    Product(P, 1024, 392, kind=kind, pre=pre, scatter=residual, weight=weight, residual=residual).run()


def test_rows_of_no_group_and_the_largest_group_count():
    Product(500, 72, 136, 3, offsets([100, 0, 250], first=37), scatter=True, pre=True).run()
    sizes = [(i * 7) % 3 for i in range(1024)]
    Product(sum(sizes) + 9, 72, 136, 1024, offsets(sizes, first=4), pre=True).run()
    Product(20, 4096, 136, 1, offsets([11], first=6), scatter=True, pre=True, residual=True, weight=True).run()


def test_offsets_are_clamped_and_destinations_outside_are_skipped():
    c = Product(90, 136, 264, 2, torch.tensor([-5, 40, 200], dtype=torch.int32, device=DEV), scatter=True, residual=True)
    c.dst[7], c.dst[50] = -1, 90
    c.run()
    c = Product(9, 2048, 264, scatter=True, pre=True)
    c.dst[3], c.dst[5] = -2147483648, 2147483647
    c.run()


@pytest.mark.parametrize("columns", [False, True])
def test_a_groups_end_reads_zeros_and_not_its_neighbour(columns):
    # K and N end inside a box, and every group but one has NaN weights
    c = Product(130, 72, 136, 3, offsets([40, 50, 40]), columns, bias=False)
    c.w[0] = float("nan")
    c.w[2] = float("nan")
    c.a[:40] = float("nan")
    c.call()
    torch.cuda.synchronize()
    z, dz, y, dy = R.product(c.a, c.w, columns, None, 0, c.off, 3)
    assert (c.out[40:90].double() - y[40:90]).abs().le(dy[40:90] + R.UBF * (y[40:90].abs() + dy[40:90])).all()
    assert c.out[:40].isnan().all() and c.out[90:].isnan().all()


def test_infinities_and_nan_through_the_activations():
    v = torch.tensor([float("inf"), float("-inf"), float("nan"), 0.0, -0.0, 30.0, -30.0, 1e-30], device=DEV)
    for kind in range(6):
        for P, columns in ((1, False), (20, True), (600, True)):     # the few rows' epilogue, the join's and the tile's own
            c = Product(P, 2048 if P < 600 else 256, 8, columns=columns, kind=kind)
            c.a.zero_()
            c.bias[0] = v
            c.call()
            torch.cuda.synchronize()
            want = R.act(v.double(), kind).float()
            got = c.out[0].float()
            assert torch.equal(got.isnan(), want.isnan()), (kind, got, want)
            ok = ~want.isnan()
            assert torch.allclose(got[ok], want[ok], rtol=2.0 ** -8, atol=1e-20), (kind, got, want)


def test_few_rows_split_k_and_no_workspace_only_costs_speed():
    c = Product(200, 4096, 1024, residual=True)
    before = launches()
    c.run()
    assert launched_since(before, "bias_act_join") == 1
    for size in (None, c.ws[: 2 * 1024 * 200 * 4], c.ws[: 1024]):
        before = launches()
        c.out.fill_(0)
        c.call(ws=size)
        torch.cuda.synchronize()
        c.check(c.out)
        assert launched_since(before, "bias_act_join") == (1 if size is not None and size.numel() > 30000 else 0)


@pytest.mark.parametrize("P,K,N,sizes", [
    (1, 8, 8, None), (7, 64, 72, None), (8, 1032, 1000, None), (9, 72, 40, None), (16, 520, 2048, None),
    (8, 72, 40000, None), (16, 136, 19456, None), (16, 136, 19464, None),       # one slice; eight rows' and more rows' limit
    (16, 264, 392, [1] * 16), (16, 264, 392, [0, 9, 0, 0, 7]), (13, 200, 136, [0] * 40 + [1, 0, 8] + [0] * 70 + [2]),
    (16, 72, 1288, [1] * 16 + [0] * 1008), (5, 72, 136, [0, 0, 0]),
    (17, 520, 264, None), (129, 136, 520, None), (100, 264, 136, [0, 33, 1, 0, 16, 17, 31]),     # several blocks of 16 rows
    (300, 72, 72, [1, 0] * 40 + [100, 0, 90, 60]), (64, 2048, 768, None),
])
def test_few_rows(P, K, N, sizes):
    # one launch, without a workspace; rows of no group stay as they were
    c = Product(P, K, N, len(sizes) if sizes else 1, offsets(sizes) if sizes else None, kind=R.GELU, pre=True, scatter=True,
                weight=True, residual=True)
    before = launches()
    c.ws = None
    c.run()
    if (P, N) != (16, 19464):
        assert launched_since(before, "gemm_bias_act") == 1 and launched_since(before, "bias_act_join") == 0


def test_few_rows_read_no_other_group_and_spread_no_nan():
    c = Product(12, 200, 136, 3, offsets([3, 4, 5]), bias=False, kind=R.SILU, pre=True)
    c.w[0] = float("nan")
    c.w[2] = float("inf")
    c.a[:3] = float("nan")
    c.a[5, 7] = float("nan")
    c.call()
    torch.cuda.synchronize()
    z, dz, y, dy = R.product(c.a, c.w, False, None, R.SILU, c.off, 3)
    ok = torch.tensor([3, 4, 6], device=DEV)
    assert (c.out[ok].double() - y[ok]).abs().le(dy[ok] + R.UBF * (y[ok].abs() + dy[ok])).all()
    assert c.out[:3].isnan().all() and c.out[5].isnan().all() and not c.out[7:].isfinite().any()


def test_a_workspace_of_the_most_rows_serves_fewer():
    for K, N, G in ((4096, 1024, 1), (512, 8, 1), (2048, 768, 3)):
        most = m.moe_grouped_gemm_bias_act_workspace_size(8192, K, N, G)
        for P in (1, 2, 16, 100, 256, 257, 1000, 2048, 8000):
            assert m.moe_grouped_gemm_bias_act_workspace_size(P, K, N, G) <= most


@pytest.mark.parametrize("columns", [False, True])
@pytest.mark.parametrize("P,K,N,sizes", [
    (2000, 1024, 512, [300, 0, 700, 1, 499, 63, 64, 373]), (1024, 4096, 512, None), (130, 520, 264, None),
    (65, 72, 4096, None), (300, 264, 1000, [129, 127, 44]),
])
def test_tiles_of_fewer_rows(P, K, N, sizes, columns):
    # 64 and 128 rows a tile, with and without ranges of K
    c = Product(P, K, N, len(sizes) if sizes else 1, offsets(sizes) if sizes else None, columns, kind=R.SILU, pre=True,
                scatter=True, weight=True, residual=True)
    c.run()
    c.call(ws=None)
    torch.cuda.synchronize()
    c.check(c.out)


def test_out_may_be_residual():
    for P, columns in ((2, False), (20, True), (500, False)):
        c = Product(P, 2048, 264, columns=columns, scatter=True, residual=True, kind=R.SILU)
        want = c.call().clone()
        res = c.res.clone()
        c.call(out=res, residual=res)
        torch.cuda.synchronize()
        assert torch.equal(res, want)


def test_same_bits_each_time_in_graphs_and_on_other_streams():
    for P, columns in ((4, False), (20, True), (900, False)):
        c = Product(P, 2048, 776, columns=columns, kind=R.GELU, residual=True)
        want = c.call().clone()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call()
        for _ in range(5):
            c.out.zero_()
            g.replay()
            assert torch.equal(c.out, want)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        c.out.zero_()
        s.wait_stream(torch.cuda.current_stream())
        c.call(stream=s)
        s.synchronize()
        assert torch.equal(c.out, want)
    assert m.moe_device_status() == 0


# ------------------------------------------------------------------ the epilogue's gradient
class Back:
    def __init__(self, P, N, G=1, off=None, kind=3, scatter=False, weight=False, seed=0):
        g = rng(P * 11 + N + kind + seed)
        self.P, self.N, self.G, self.off, self.kind = P, N, G, off, kind
        self.dout, self.z = normal(g, (P, N)), normal(g, (P, N), 1.5)
        self.dst = torch.randperm(P, generator=g, device=DEV).to(torch.int32) if scatter else None
        self.pw = torch.rand((P,), generator=g, device=DEV) + 0.25 if weight else None
        self.dz = normal(g, (P, N))
        self.db = normal(g, (G, N), 1.0, torch.float32)
        self.dpw = normal(g, (P,), 1.0, torch.float32)
        self.ws = ws_of(m.moe_bias_act_backward_workspace_size(P, N, G))

    def call(self, dz=None, db=True, dpw=True, z=True, ws=True):
        dz = self.dz if dz is None else dz
        ws = self.ws if ws is True else ws
        m.moe_bias_act_backward(self.dout, self.z if z else None, self.kind, self.pw, self.dst, self.off, self.P, self.N,
                                self.G, dz, self.db if db else None, self.dpw if dpw else None, ws,
                                0 if ws is None else ws.numel())

    def run(self, **kw):
        keep = [t.clone() for t in (self.dz, self.db, self.dpw)]
        self.call(**kw)
        torch.cuda.synchronize()
        P, N = self.P, self.N
        z = self.z.double()
        s, y = R.slope(z, self.kind), R.act(z, self.kind)
        to = torch.arange(P, device=DEV) if self.dst is None else self.dst.long()
        ok = (to >= 0) & (to < P)
        d = torch.zeros_like(z)
        d[ok] = self.dout[to[ok]].double()
        w = torch.ones(P, dtype=torch.float64, device=DEV)
        if self.pw is not None:
            w[ok] = self.pw[to[ok]].double()
        dz, mag = d * w[:, None] * s, (d * w[:, None]).abs()
        err = mag * (4 * U(1) + (0 if self.kind < 3 else R.REL + R.PHI * (1 + z.abs())))
        want, bound = torch.full_like(z, float("nan")), torch.full_like(z, float("nan"))
        db, db_err = torch.zeros((self.G, N), dtype=torch.float64, device=DEV), torch.zeros((self.G, N), dtype=torch.float64, device=DEV)
        dpw = torch.full((P,), float("nan"), dtype=torch.float64, device=DEV)
        dpw_err = dpw.clone()
        for g, lo, hi in R.groups(self.off, P, self.G):
            want[lo:hi], bound[lo:hi] = dz[lo:hi], err[lo:hi] + R.UBF * (dz[lo:hi].abs() + err[lo:hi])
            db[g] = dz[lo:hi].sum(0)
            db_err[g] = (err[lo:hi] + (hi - lo + 40) * R.U32 * (dz[lo:hi].abs() + err[lo:hi])).sum(0)
            i = torch.arange(lo, hi, device=DEV)[ok[lo:hi]]
            dpw[to[i]] = (d[i] * y[i]).sum(1)
            yerr = 0 if self.kind == 0 else R.REL * y[i].abs() + R.PHI * z[i].abs()
            dpw_err[to[i]] = (d[i].abs() * (yerr + (N / 32 + 8) * R.U32 * y[i].abs())).sum(1)
        R.check(self.dz if kw.get("dz") is None else kw["dz"], want, bound, keep[0] if kw.get("dz") is None else None, "dz")
        if kw.get("db", True):
            R.check(self.db, db, db_err, None, "grad_bias")
        if kw.get("dpw", True):
            R.check(self.dpw, dpw, dpw_err, keep[2], "grad_pair_weight")


def U(n):
    return n * R.U32


@pytest.mark.parametrize("kind", range(6))
@pytest.mark.parametrize("shape", [(1, 8, None), (37, 264, [10, 0, 27]), (700, 1032, [0, 650, 1, 2, 3, 44, 0]), (65, 2304, None)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_backward(kind, shape):
    P, N, sizes = shape
    for scatter, weight in ((False, False), (True, True), (True, False)):
        Back(P, N, len(sizes) if sizes else 1, offsets(sizes) if sizes else None, kind, scatter, weight).run()


def test_backward_of_many_small_groups_and_rows_of_none():
    sizes = [(i * 5) % 4 for i in range(1024)]
    Back(sum(sizes) + 21, 72, 1024, offsets(sizes, first=13), scatter=True, weight=True).run()
    c = Back(300, 1100 // 8 * 8, 3, offsets([100, 0, 150], first=20), scatter=True, weight=True)
    c.dst[30], c.dst[200] = -1, 300
    c.run()


@pytest.mark.parametrize("P", [900, 2500, 5001])     # few and many rows to a CTA, the last with fewer
def test_backward_of_every_block_height(P):
    sizes = [P // 3, 0, 1, 15, 16, 17, 63, 64, 65]
    sizes += [5, P - sum(sizes) - 9]
    c = Back(P, 1032, len(sizes), offsets(sizes), kind=R.GELU, scatter=True, weight=True)
    c.dst[P - 3], c.dst[P // 2] = -7, P          # of a group's row, and of one in no group
    c.run()


def test_backward_workspace_of_the_most_rows_serves_fewer():
    for N, G in ((8, 1), (768, 3), (4096, 7), (40000, 1)):
        most = m.moe_bias_act_backward_workspace_size(40000, N, G)
        sizes = [m.moe_bias_act_backward_workspace_size(P, N, G) for P in range(1, 40001, 13)]
        assert max(sizes) <= most and sizes == sorted(sizes)


def test_backward_without_outputs_or_z():
    c = Back(100, 264, 2, offsets([60, 40]), kind=0)
    c.run(z=False, dpw=False)
    c.run(db=False, dpw=False, ws=None)          # no sums: no workspace
    c.run(db=False)
    Back(100, 136, 2, offsets([60, 40])).run(db=False)
    Back(100, 2056, 2, offsets([60, 40]), kind=5).run(db=False)
    Back(100, 2056, 2, offsets([60, 40]), kind=5).run(dpw=False)
    c = Back(100, 264, 2, offsets([60, 40]), kind=4)
    z = c.z.clone()
    c.call()
    c.z.copy_(z)
    want = c.dz.clone()
    c.call(dz=c.z)                               # dz may be z
    torch.cuda.synchronize()
    assert torch.equal(c.z, want)


def test_no_rows_gives_zero_sums():
    c = Back(8, 264, 3, offsets([0, 0, 0]))
    c.P = 0
    c.call(dpw=False)
    torch.cuda.synchronize()
    assert not c.db.any()
    w = Wgrad(8, 72, 136, 3, offsets([0, 0, 0]), add=True)
    w.P = 0
    w.call()
    torch.cuda.synchronize()
    assert torch.equal(w.dw, w.add)


# ------------------------------------------------------------------ the weights' gradient
class Wgrad:
    def __init__(self, P, N, K, G=1, off=None, add=False, seed=0):
        g = rng(P * 13 + N * 3 + K + seed)
        self.P, self.N, self.K, self.G, self.off = P, N, K, G, off
        self.dz, self.a = normal(g, (P, N)), normal(g, (P, K))
        self.add = normal(g, (G, N, K), 1.0, torch.float32) if add else None
        self.dw = torch.full((G, N, K), float("nan"), device=DEV)
        self.ws = ws_of(m.moe_grouped_gemm_wgrad_workspace_size(P, N, K, G))

    def call(self, out=None, add=None):
        m.moe_grouped_gemm_wgrad_bf16(self.dz, self.a, self.off, self.P, self.N, self.K, self.G,
                                      self.add if add is None else add, self.dw if out is None else out, self.ws,
                                      self.ws.numel())

    def run(self):
        self.call()
        torch.cuda.synchronize()
        want = torch.zeros((self.G, self.N, self.K), dtype=torch.float64, device=DEV)
        bound = torch.zeros_like(want)
        for g, lo, hi in R.groups(self.off, self.P, self.G):
            d, a = self.dz[lo:hi].double(), self.a[lo:hi].double()
            want[g] = d.t() @ a
            n = hi - lo
            bound[g] = (math.ceil(min(n, 512) / 16) + math.ceil(n / 512) + 17) * 2 * R.U32 * (d.abs().t() @ a.abs())
        if self.add is not None:
            want += self.add.double()
            bound += R.U32 * (want.abs() + bound)
        R.check(self.dw, want, bound, None, "grad_w")


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("shape", [(1, 8, 8, None), (17, 136, 264, None), (64, 128, 256, None), (777, 400, 1040, [0, 1, 300, 0, 17, 255, 204, 0]),
                                   (2000, 264, 520, None), (5000, 72, 136, [4000, 1000]), (9000, 8, 24, [0, 8990, 1])],
                         ids=lambda s: "x".join(map(str, s[:3])) + ("g" if s[3] else ""))
def test_wgrad(shape, add):
    P, N, K, sizes = shape
    Wgrad(P, N, K, len(sizes) if sizes else 1, offsets(sizes) if sizes else None, add).run()


def test_wgrad_does_not_touch_rows_of_no_group():
    # NaN rows before the first group, behind the last one and in another group stay where they are
    c = Wgrad(500, 136, 264, 3, offsets([100, 33, 250], first=21))
    for t in (c.dz, c.a):
        t[:21] = float("nan")
        t[404:] = float("nan")
    c.run()
    c.dz[121:154] = float("nan")
    c.a[121:154] = float("inf")
    c.dw.zero_()
    c.call()
    torch.cuda.synchronize()
    assert c.dw[0].isfinite().all() and c.dw[2].isfinite().all() and not c.dw[1].isfinite().any()


def test_wgrad_ranges_add_in_place_and_same_bits():
    for P, N, K, G in ((6000, 136, 264, 1), (3000, 264, 512, 2), (100, 72, 72, 1)):
        c = Wgrad(P, N, K, G, offsets([P // G] * G), add=True)
        before = launches()
        c.run()
        assert launched_since(before, "wgrad_reduce") == (1 if P > 1024 else 0)
        want = c.dw.clone()
        acc = c.add.clone()
        c.call(out=acc, add=acc)
        c.call()
        torch.cuda.synchronize()
        assert torch.equal(acc, want) and torch.equal(c.dw, want)
    assert m.moe_device_status() == 0


def test_wgrad_adds_in_place_over_many_tiles():
    # 320 tiles, several an SM; N and K end inside a box; groups without rows and of more than one accumulator
    sizes = [0, 1100, 3, 0, 17, 64, 0, 513] * 5
    c = Wgrad(sum(sizes), 136, 776, len(sizes), offsets(sizes), add=True)
    c.run()
    want = c.dw.clone()
    for _ in range(3):
        held = c.add.clone()
        c.call(out=held, add=held)
        torch.cuda.synchronize()
        assert torch.equal(held, want)
    c = Wgrad(100, 2560, 2560, 3, offsets([50, 0, 50]), add=True)
    c.run()


def test_wgrad_adds_to_groups_of_many_rows():
    # more than 512 rows a group on average: 180 tiles, some of them empty
    sizes = [1500, 0, 700, 17, 1600]
    c = Wgrad(sum(sizes), 1040, 776, 5, offsets(sizes), add=True)
    c.run()
    want = c.dw.clone()
    for _ in range(3):
        held = c.add.clone()
        c.call(out=held, add=held)
        torch.cuda.synchronize()
        assert torch.equal(held, want)
