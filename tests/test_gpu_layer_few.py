"""moe_layer_few_bf16 / moe_layer_few_fp8w against the layer in 64 bits, and their choice of
experts against the router's entry points, bit for bit."""
from __future__ import annotations

import pytest
import torch

import mixture_experts_ffn_renorm_gb300 as m

from . import ref_few as R
from .gpu_util import DEV, launched_since, launches

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Case:
    def __init__(self, T, H, I, E, K, Is=0, fp8=False, gate=True, residual=True, bias=True, scoring=0, renorm=1,
                 n_group=1, topk_group=1, group_score=0, select=False, scale=1.0, seed=0, same=False):
        g = torch.Generator(device=DEV).manual_seed(1000 * T + 10 * H + E + seed)
        n = lambda *s, std=1.0, dt=BF: (torch.randn(s, generator=g, device=DEV) * std).to(dt)
        self.T, self.H, self.I, self.E, self.K, self.Is, self.fp8 = T, H, I, E, K, Is, fp8
        self.route = (renorm, scoring, n_group, topk_group, group_score)
        self.scale = scale
        self.x = n(T, H)
        if same:                      # every token alike: all choose the same experts
            self.x[:] = self.x[:1].clone()
        self.wr = n(E, H, std=H ** -0.5)
        self.bias = n(E, std=0.3, dt=torch.float32) if bias else None
        self.select = n(E, std=0.1, dt=torch.float32) if select else None
        if fp8:
            code = lambda *s: torch.randn(s, generator=g, device=DEV).mul_(100).clamp_(-448, 448).to(
                torch.float8_e4m3fn).view(torch.uint8)
            sc = lambda r, c, std: (torch.rand((E, -(-r // 128), -(-c // 128)), generator=g, device=DEV) + 0.5) * std / 100
            self.w13, self.s13 = code(E, 2 * I, H), sc(2 * I, H, H ** -0.5)
            self.w2, self.s2 = code(E, H, I), sc(H, I, I ** -0.5)
        else:
            self.w13, self.w2 = n(E, 2 * I, H, std=H ** -0.5), n(E, H, I, std=I ** -0.5)
        self.wg = n(H, std=H ** -0.5) if Is and gate else None
        self.w13s, self.w2s = (n(2 * Is, H, std=H ** -0.5), n(H, Is, std=Is ** -0.5)) if Is else (None, None)
        self.res = n(T, H) if residual else None
        self.out = torch.full((T, H), float("nan"), dtype=BF, device=DEV)
        self.ids = torch.full((T, K), -1, dtype=torch.int32, device=DEV)
        self.w = torch.full((T, K), float("nan"), device=DEV)
        self.ws = torch.zeros(m.moe_layer_few_workspace_size(T, H, I, E, K, Is), dtype=torch.uint8, device=DEV)

    def call(self, out=None, ws=None, stream=None, **other):
        out = self.out if out is None else out
        ws = self.ws if ws is None else ws
        rest = (self.wg, self.w13s, self.w2s, other.get("residual", self.res), self.T, self.H, self.I, self.E,
                self.K, self.Is, *self.route, self.scale, other.get("ids", self.ids), other.get("w", self.w), out, ws,
                ws.numel(), stream)
        if self.fp8:
            m.moe_layer_few_fp8w(self.x, self.wr, self.bias, self.select, self.w13, self.s13, self.w2, self.s2, *rest)
        else:
            m.moe_layer_few_bf16(self.x, self.wr, self.bias, self.select, self.w13, self.w2, *rest)
        return out

    def routed(self):
        """ids and weights from the router's entry points."""
        T, H, E, K = self.T, self.H, self.E, self.K
        renorm, scoring, n_group, topk_group, group_score = self.route
        ids, w = torch.empty_like(self.ids), torch.empty_like(self.w)
        ws = torch.empty(max(256, m.moe_route_topk_workspace_size(T, E, K)), dtype=torch.uint8, device=DEV)
        m.moe_route_topk_ex(self.x, self.wr, self.bias, self.select, None, None, T, H, E, K, renorm, scoring, n_group,
                            topk_group, group_score, ids, w, None, None, ws, ws.numel())
        return ids, w

    def check(self, out=None):
        out = self.out if out is None else out
        ids, w = self.routed()
        torch.cuda.synchronize()
        assert torch.equal(ids, self.ids) and torch.equal(w.view(torch.int32), self.w.view(torch.int32))
        if self.fp8:
            w13, w2 = (lambda e: R.dequant(self.w13[e], self.s13[e])), (lambda e: R.dequant(self.w2[e], self.s2[e]))
        else:
            w13, w2 = (lambda e: self.w13[e].double()), (lambda e: self.w2[e].double())
        want, bound = R.layer(self.x, ids.cpu(), w.cpu(), w13, w2, self.scale,
                              (self.wg, self.w13s, self.w2s) if self.Is else None, self.res)
        off = (out.double() - want).abs()
        assert (off <= bound).all(), f"off by {(off / bound).max().item():.2f} of the bound"


SIZES = [
    # T, H, I, E, K
    (1, 2048, 768, 128, 8),
    (16, 2048, 768, 128, 8),
    (1, 64, 32, 8, 2),
    (4, 64, 32, 8, 2),
    (2, 8, 8, 1, 1),             # the smallest sizes, one expert
    (16, 264, 72, 40, 32),       # as many pairs as there can be
    (3, 1032, 400, 60, 6),
    (7, 520, 1040, 5, 5),        # every expert chosen by every token
    (5, 8192, 16, 4, 2),         # the widest rows
    (2, 16, 8192, 4, 3),
    (13, 296, 120, 1024, 3),     # the most experts
]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_bf16(size):
    c = Case(*size)
    c.call()
    c.check()


@pytest.mark.parametrize("size", [(1, 2048, 768, 128, 8), (16, 1040, 400, 60, 6), (2, 16, 16, 3, 1), (5, 8192, 16, 4, 2),
                                  (3, 16, 8192, 4, 3), (4, 144, 272, 12, 4)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("Is", [0, 208])
def test_fp8(size, Is):
    c = Case(*size, Is=Is, fp8=True, residual=Is > 0)
    c.call()
    c.check()


@pytest.mark.parametrize("Is,gate", [(32, True), (8, False), (1024, True), (8192, True)])
@pytest.mark.parametrize("T", [1, 6, 16])
def test_shared_expert(T, Is, gate):
    c = Case(T, 520, 136, 16, 4, Is=Is, gate=gate)
    c.call()
    c.check()


@pytest.mark.parametrize("scoring,renorm", [(0, 0), (0, 1), (1, 0), (1, 1)])
@pytest.mark.parametrize("groups", [(1, 1, 0), (4, 2, 0), (4, 2, 1), (16, 3, 1), (64, 40, 0)])
def test_router_forms(scoring, renorm, groups):
    c = Case(5, 264, 40, 64 if groups[0] == 64 else 192, 6, scoring=scoring, renorm=renorm, n_group=groups[0],
             topk_group=groups[1], group_score=groups[2], select=scoring == 1, scale=2.5)
    c.call()
    c.check()


@pytest.mark.parametrize("T", [2, 3, 5, 16])
def test_tokens_of_one_expert(T):
    c = Case(T, 512, 96, 24, 3, same=True)
    c.call()
    c.check()


def test_no_optional_outputs_and_operands():
    c = Case(3, 264, 72, 12, 4, residual=False, bias=False)
    c.call()
    c.check()
    want = c.out.clone()
    c.out.zero_()
    c.call(ids=None, w=None)
    torch.cuda.synchronize()
    assert torch.equal(c.out, want)


def test_out_may_be_residual_or_x():
    c = Case(6, 1032, 400, 60, 6)
    c.call()
    torch.cuda.synchronize()
    want = c.out.clone()
    res = c.res.clone()
    c.call(out=res, residual=res)
    keep = c.x.clone()
    torch.cuda.synchronize()
    assert torch.equal(res, want)
    a = c.call(residual=c.x, out=torch.empty_like(c.out)).clone()
    c.call(residual=c.x, out=c.x)
    torch.cuda.synchronize()
    assert torch.equal(c.x, a) and not torch.equal(c.x, keep)


def test_one_workspace_for_calls_of_many_sizes_and_the_same_bits_each_time():
    cases = [Case(*s, seed=1) for s in SIZES[:6]]
    ws = torch.zeros(max(c.ws.numel() for c in cases), dtype=torch.uint8, device=DEV)
    first = [c.call(ws=ws).clone() for c in cases]
    for _ in range(20):
        for c, want in zip(cases, first):
            c.out.fill_(float("nan"))
            c.call(ws=ws)
            assert torch.equal(c.out, want)
    assert m.moe_device_status() == 0


def test_one_launch_and_no_tokens():
    c = Case(2, 64, 32, 8, 2)
    before = launches()
    c.call()
    assert launched_since(before, "layer_few") == 1
    c.T = 0
    before = launches()
    c.call()
    assert launched_since(before, "layer_few") == 0


def test_captured_and_replayed_on_another_stream():
    c = Case(4, 1032, 400, 60, 6, Is=64)
    c.call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    keep = c.x.clone()
    for k in range(3):
        c.x.copy_(keep.roll(k, 0))
        c.out.fill_(float("nan"))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g.replay()
        torch.cuda.current_stream().wait_stream(s)
        c.check()


def test_two_calls_at_once_with_a_workspace_each():
    a, b = Case(3, 1032, 400, 60, 6), Case(16, 2048, 768, 128, 8)
    want = [c.call().clone() for c in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(30):
        for c, s in zip((a, b), streams):
            c.call(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])
    assert m.moe_device_status() == 0


def test_nan_token_stays_in_its_row_and_infinite_weights_in_theirs():
    c = Case(4, 264, 72, 12, 3, bias=False)
    c.call()
    torch.cuda.synchronize()
    want = c.out.clone()
    c.x[2, 5] = float("nan")
    c.call()
    torch.cuda.synchronize()
    keep = [0, 1, 3]
    assert torch.equal(c.out[keep], want[keep]) and c.out[2].isnan().all()
    c.x[2] = c.x[1]
    c.call()
    torch.cuda.synchronize()
    e = int(c.ids[0, 0])
    c.w2[e, 17, 3] = float("inf")
    c.call()
    torch.cuda.synchronize()
    hit = (c.ids == e).any(1)
    assert not c.out[hit, 17].isfinite().any()
    rest = torch.ones_like(c.out, dtype=torch.bool)
    rest[hit, 17] = False
    assert c.out[rest].isfinite().all()
