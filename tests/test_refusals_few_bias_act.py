"""Refusals of the few-token layer, the products with an epilogue and their gradients: by name and
before any CUDA call (no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest

import mixture_experts_ffn_renorm_gb300 as m
from mixture_experts_ffn_renorm_gb300 import build as moe_build

BUF = (ctypes.c_uint8 * 4096)()
BASE = (ctypes.addressof(BUF) + 15) & ~15
A = ctypes.c_void_p(BASE)
ODD = ctypes.c_void_p(BASE + 2)       # 2-byte aligned
BYTE = ctypes.c_void_p(BASE + 1)
BIG = 1 << 40
TOP = 0x7FFFFFFF


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return m.lib()


def refused(rc, code, text):
    assert rc == code and text in m.last_error(), (rc, m.last_error())


# ------------------------------------------------------------------ the layer
BF16 = ["x", "w_router", "logit_bias", "select_bias", "w13", "w2", "w_gate", "w13s", "w2s", "residual"]
FP8 = ["x", "w_router", "logit_bias", "select_bias", "w13", "s13", "w2", "s2", "w_gate", "w13s", "w2s", "residual"]


def layer(lib, fp8=False, **kw):
    p = dict.fromkeys(FP8 if fp8 else BF16, A)
    p.update(dict.fromkeys(["logit_bias", "select_bias", "w_gate", "w13s", "w2s", "residual"]))
    s = dict(T=2, H=64, I=32, E=8, K=2, Is=0, renorm=1, scoring=0, n_group=1, topk_group=1, group_score=0)
    o = dict(scale=1.0, ids=A, w=A, out=A, ws=A, bytes=BIG)
    for k, v in kw.items():
        next(d for d in (p, s, o) if k in d)[k] = v
    f = lib.moe_layer_few_fp8w if fp8 else lib.moe_layer_few_bf16
    return f(*p.values(), *s.values(), o["scale"], o["ids"], o["w"], o["out"], o["ws"], o["bytes"], None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,code,text", [
    (dict(T=-1), m.ERR_ARG, "T=-1"), (dict(T=17), m.ERR_ARG, "T=17"), (dict(E=0, K=0), m.ERR_ARG, "E=0"),
    (dict(E=1025), m.ERR_ARG, "E=1025"), (dict(K=0), m.ERR_ARG, "K=0"), (dict(K=9), m.ERR_ARG, "K=9"),
    (dict(E=64, K=33), m.ERR_ARG, "K=33"), (dict(H=0), m.ERR_ARG, "H=0"), (dict(H=8208), m.ERR_ARG, "H=8208"),
    (dict(I=0), m.ERR_ARG, "I=0"), (dict(I=TOP), m.ERR_ARG, "I="), (dict(Is=-8), m.ERR_ARG, "I_shared"),
    (dict(Is=8200, w13s=A, w2s=A), m.ERR_ARG, "I_shared"), (dict(renorm=2), m.ERR_ARG, "renormalize"),
    (dict(scoring=2), m.ERR_UNSUPPORTED, "scoring=2"), (dict(select_bias=A), m.ERR_UNSUPPORTED, "sigmoid"),
    (dict(n_group=3), m.ERR_ARG, "n_group=3"), (dict(E=128, n_group=128), m.ERR_ARG, "n_group"),
    (dict(n_group=4, topk_group=5), m.ERR_ARG, "topk_group=5"), (dict(group_score=2), m.ERR_ARG, "group_score"),
    (dict(n_group=8, topk_group=8, group_score=1), m.ERR_ARG, "two experts"),
    (dict(n_group=8, topk_group=1), m.ERR_ARG, "K=2 exceeds"), (dict(H=68), m.ERR_ALIGN, "multiples"),
    (dict(I=36), m.ERR_ALIGN, "multiples"), (dict(Is=12, w13s=A, w2s=A), m.ERR_ALIGN, "multiples"),
    (dict(x=None), m.ERR_ARG, "NULL"), (dict(w_router=None), m.ERR_ARG, "NULL"), (dict(w13=None), m.ERR_ARG, "NULL"),
    (dict(w2=None), m.ERR_ARG, "NULL"), (dict(out=None), m.ERR_ARG, "NULL"),
    (dict(Is=32), m.ERR_ARG, "without w13_shared"), (dict(Is=32, w13s=A), m.ERR_ARG, "without w13_shared"),
    (dict(w13s=A), m.ERR_ARG, "I_shared=0"), (dict(w_gate=A), m.ERR_ARG, "I_shared=0"),
    (dict(x=ODD), m.ERR_ALIGN, "16-byte"), (dict(w13=ODD), m.ERR_ALIGN, "16-byte"), (dict(ws=ODD), m.ERR_ALIGN, "16-byte"),
    (dict(logit_bias=ODD), m.ERR_ALIGN, "4-byte"), (dict(ids=ODD), m.ERR_ALIGN, "4-byte"), (dict(w=ODD), m.ERR_ALIGN, "4-byte"),
    (dict(out=BYTE), m.ERR_ALIGN, "2-byte"), (dict(residual=BYTE), m.ERR_ALIGN, "2-byte"),
    (dict(ws=None), m.ERR_WORKSPACE, "workspace"), (dict(bytes=256), m.ERR_WORKSPACE, "workspace"),
], ids=str)
def test_layer(lib, fp8, kw, code, text):
    refused(layer(lib, fp8, **kw), code, text)


def test_layer_fp8_only(lib):
    refused(layer(lib, True, H=72), m.ERR_ALIGN, "multiples of 16")
    refused(layer(lib, True, I=24), m.ERR_ALIGN, "multiples of 16")
    refused(layer(lib, True, s13=None), m.ERR_ARG, "scales")
    refused(layer(lib, True, s2=None), m.ERR_ARG, "scales")
    refused(layer(lib, True, s2=ODD), m.ERR_ALIGN, "4-byte")


def test_layer_no_tokens_and_workspace_sizes(lib):
    assert layer(lib, T=0, x=None, w13=None, out=None, ws=None, bytes=0) == m.OK
    assert layer(lib, True, T=0, x=None, s13=None, ws=None, bytes=0) == m.OK
    size = m.moe_layer_few_workspace_size
    assert size(0, 64, 32, 8, 2, 0) == 0 and size(1, 64, 32, 8, 0, 0) == 0 and size(1, 64, 32, 8, 2, -1) == 0
    # never smaller for more tokens: one for the most serves every call
    sizes = [size(t, 2048, 768, 128, 8, 64) for t in range(1, 17)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    need = size(2, 64, 32, 8, 2, 0)
    refused(layer(lib, bytes=need - 1), m.ERR_WORKSPACE, str(need))


# ------------------------------------------------------------------ the product
def product(lib, **kw):
    p = dict(a=A, w=A, layout=0, bias=None, act=0, pre=None, pw=None, dst=None, res=None, off=A, P=4, K=16, N=16, G=2,
             out=A, ws=None, bytes=0)
    p.update(kw)
    return lib.moe_grouped_gemm_bias_act_bf16(*p.values(), None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(P=-1), m.ERR_ARG, "P=-1"), (dict(K=0), m.ERR_ARG, "K=0"), (dict(N=0), m.ERR_ARG, "N=0"),
    (dict(P=TOP), m.ERR_ARG, "too large"), (dict(K=TOP - 7), m.ERR_ARG, "too large"), (dict(N=TOP - 7), m.ERR_ARG, "too large"),
    (dict(P=1 << 30, N=1 << 30, G=1), m.ERR_ARG, "too large together"), (dict(G=0), m.ERR_ARG, "G=0"),
    (dict(G=1025), m.ERR_ARG, "G=1025"), (dict(layout=2), m.ERR_ARG, "w_layout=2"), (dict(act=6), m.ERR_ARG, "activation=6"),
    (dict(act=-1), m.ERR_ARG, "activation=-1"), (dict(K=20), m.ERR_ALIGN, "multiples of 8"), (dict(N=20), m.ERR_ALIGN, "multiples of 8"),
    (dict(a=None), m.ERR_ARG, "NULL"), (dict(w=None), m.ERR_ARG, "NULL"), (dict(out=None), m.ERR_ARG, "NULL"),
    (dict(off=None), m.ERR_ARG, "group_offsets"), (dict(a=ODD), m.ERR_ALIGN, "16-byte"), (dict(w=ODD), m.ERR_ALIGN, "16-byte"),
    (dict(pre=ODD), m.ERR_ALIGN, "16-byte"), (dict(res=ODD), m.ERR_ALIGN, "16-byte"), (dict(out=ODD), m.ERR_ALIGN, "16-byte"),
    (dict(ws=ODD), m.ERR_ALIGN, "16-byte"), (dict(bias=ODD), m.ERR_ALIGN, "4-byte"), (dict(pw=ODD), m.ERR_ALIGN, "4-byte"),
    (dict(dst=ODD), m.ERR_ALIGN, "4-byte"), (dict(off=ODD), m.ERR_ALIGN, "4-byte"),
], ids=str)
def test_product(lib, kw, code, text):
    refused(product(lib, **kw), code, text)


def test_product_no_rows(lib):
    assert product(lib, P=0, a=None, w=None, off=None, out=None) == m.OK
    assert m.moe_grouped_gemm_bias_act_workspace_size(0, 64, 64, 1) == 0
    assert m.moe_grouped_gemm_bias_act_workspace_size(4, 64, 64, 0) == 0


# ------------------------------------------------------------------ the epilogue's gradient
def backward(lib, **kw):
    p = dict(dout=A, z=A, act=3, pw=None, dst=None, off=A, P=4, N=16, G=2, dz=A, db=A, dpw=A, ws=A, bytes=BIG)
    p.update(kw)
    return lib.moe_bias_act_backward(*p.values(), None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(P=-1), m.ERR_ARG, "P=-1"), (dict(N=0), m.ERR_ARG, "N=0"), (dict(P=TOP), m.ERR_ARG, "too large"),
    (dict(N=TOP - 7), m.ERR_ARG, "too large"), (dict(N=256 * 65536), m.ERR_ARG, "too large"), (dict(G=0), m.ERR_ARG, "G=0"),
    (dict(G=1025), m.ERR_ARG, "G=1025"), (dict(act=6), m.ERR_ARG, "activation=6"), (dict(N=20), m.ERR_ALIGN, "multiple of 8"),
    (dict(off=None), m.ERR_ARG, "group_offsets"), (dict(dout=None), m.ERR_ARG, "NULL"), (dict(dz=None), m.ERR_ARG, "NULL"),
    (dict(z=None), m.ERR_ARG, "needs z"), (dict(z=None, act=0), m.ERR_ARG, "needs z"), (dict(dout=ODD), m.ERR_ALIGN, "16-byte"),
    (dict(z=ODD), m.ERR_ALIGN, "16-byte"), (dict(dz=ODD), m.ERR_ALIGN, "16-byte"), (dict(db=ODD), m.ERR_ALIGN, "16-byte"),
    (dict(ws=ODD), m.ERR_ALIGN, "16-byte"), (dict(pw=ODD), m.ERR_ALIGN, "4-byte"), (dict(dst=ODD), m.ERR_ALIGN, "4-byte"),
    (dict(off=ODD), m.ERR_ALIGN, "4-byte"), (dict(dpw=ODD), m.ERR_ALIGN, "4-byte"), (dict(ws=None), m.ERR_WORKSPACE, "workspace"),
    (dict(bytes=16), m.ERR_WORKSPACE, "workspace"), (dict(db=None, N=512, bytes=16), m.ERR_WORKSPACE, "workspace"),
], ids=str)
def test_backward(lib, kw, code, text):
    refused(backward(lib, **kw), code, text)


def test_backward_no_rows_and_workspace_sizes(lib):
    assert backward(lib, P=0, dout=None, z=None, dz=None, db=None, ws=None, bytes=0) == m.OK
    size = m.moe_bias_act_backward_workspace_size
    assert size(0, 64, 1) == 0 and size(4, 64, 0) == 0
    sizes = [size(p, 1024, 8) for p in (1, 31, 64, 65, 1000, 100000)]
    assert sizes == sorted(sizes) and sizes[0] > 0


# ------------------------------------------------------------------ the weights' gradient
def wgrad(lib, **kw):
    p = dict(dz=A, a=A, off=A, P=4, N=16, K=16, G=2, add=None, dw=A, ws=None, bytes=0)
    p.update(kw)
    return lib.moe_grouped_gemm_wgrad_bf16(*p.values(), None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(P=-1), m.ERR_ARG, "P=-1"), (dict(N=0), m.ERR_ARG, "N=0"), (dict(K=0), m.ERR_ARG, "K=0"), (dict(P=TOP), m.ERR_ARG, "too large"),
    (dict(N=TOP - 7), m.ERR_ARG, "too large"), (dict(K=TOP - 7), m.ERR_ARG, "too large"), (dict(G=0), m.ERR_ARG, "G=0"),
    (dict(G=1025), m.ERR_ARG, "G=1025"), (dict(N=12), m.ERR_ALIGN, "multiples of 8"), (dict(K=12), m.ERR_ALIGN, "multiples of 8"),
    (dict(N=1 << 20, K=1 << 20), m.ERR_ARG, "too large together"), (dict(dw=None), m.ERR_ARG, "grad_w is NULL"),
    (dict(off=None), m.ERR_ARG, "group_offsets"), (dict(dz=None), m.ERR_ARG, "NULL"), (dict(a=None), m.ERR_ARG, "NULL"),
    (dict(dz=ODD), m.ERR_ALIGN, "16-byte"), (dict(a=ODD), m.ERR_ALIGN, "16-byte"), (dict(add=ODD), m.ERR_ALIGN, "16-byte"),
    (dict(dw=ODD), m.ERR_ALIGN, "16-byte"), (dict(ws=ODD), m.ERR_ALIGN, "16-byte"), (dict(off=ODD), m.ERR_ALIGN, "4-byte"),
], ids=str)
def test_wgrad(lib, kw, code, text):
    refused(wgrad(lib, **kw), code, text)


def test_wgrad_workspace_sizes(lib):
    assert m.moe_grouped_gemm_wgrad_workspace_size(0, 64, 64, 1) == 0
    sizes = [m.moe_grouped_gemm_wgrad_workspace_size(p, 64, 64, 1) for p in (1, 1000, 5000, 100000)]
    assert sizes == sorted(sizes)
