"""Argument checks of the FP8 products and of the gradients: every refusal names what is wrong
and returns before any CUDA call (no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest

import mixture_experts_ffn_renorm_gb300 as m
from mixture_experts_ffn_renorm_gb300 import build as moe_build

BUF = (ctypes.c_uint8 * 4096)()
A = ctypes.c_void_p((ctypes.addressof(BUF) + 15) & ~15)      # 16-byte aligned
B = ctypes.c_void_p(A.value + 4)                              # 4-byte aligned
C = ctypes.c_void_p(A.value + 2)                              # 2-byte aligned


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return m.lib()


def refused(rc, code, text):
    assert rc == code and text in m.last_error(), (rc, m.last_error())


@pytest.mark.parametrize("args,code,text", [
    ((A, -1, 64, 1, None, None, 1.0, A, A), m.ERR_ARG, "T=-1"),
    ((A, 1, 0, 1, None, None, 1.0, A, A), m.ERR_ARG, "H=0"),
    ((A, 1, 64, 0, None, None, 1.0, A, A), m.ERR_ARG, "K=0"),
    ((A, 1, 64, 65, None, None, 1.0, A, A), m.ERR_ARG, "K=65"),
    ((A, 1 << 30, 64, 4, None, None, 1.0, A, A), m.ERR_ARG, "too large"),
    ((A, 1, 72, 1, None, None, 1.0, A, A), m.ERR_ALIGN, "16"),
    ((None, 1, 64, 1, None, None, 1.0, A, A), m.ERR_ARG, "NULL"),
    ((B, 1, 64, 1, None, None, 1.0, A, A), m.ERR_ALIGN, "16-byte"),
    ((A, 1, 64, 1, None, None, 1.0, B, A), m.ERR_ALIGN, "16-byte"),
    ((A, 1, 64, 1, None, None, 1.0, A, C), m.ERR_ALIGN, "4-byte"),
    ((A, 1, 64, 1, C, None, 1.0, A, A), m.ERR_ALIGN, "4-byte"),
])
def test_quantiser(lib, args, code, text):
    refused(lib.moe_quantize_act_fp8(*args, None), code, text)


@pytest.mark.parametrize("args,code,text", [
    ((A, A, A, A, A, None, None, -1, 64, 64, 1, A), m.ERR_ARG, "P=-1"),
    ((A, A, A, A, A, None, None, 4, 0, 64, 1, A), m.ERR_ARG, "positive"),
    ((A, A, A, A, A, None, None, 4, 64, 64, 0, A), m.ERR_ARG, "G=0"),
    ((A, A, A, A, A, None, None, 4, 64, 64, 1025, A), m.ERR_ARG, "G=1025"),
    ((A, A, A, A, A, None, None, 4, 72, 64, 1, A), m.ERR_ALIGN, "K=72"),
    ((A, A, A, A, A, None, None, 4, 64, 60, 1, A), m.ERR_ALIGN, "N=60"),
    ((A, None, A, A, A, None, None, 4, 64, 64, 1, A), m.ERR_ARG, "scales"),
    ((A, A, A, A, None, None, None, 4, 64, 64, 2, A), m.ERR_ARG, "group_offsets"),
    ((A, A, A, A, A, None, None, 4, 64, 64, 1, None), m.ERR_ARG, "out"),
    ((B, A, A, A, A, None, None, 4, 64, 64, 1, A), m.ERR_ALIGN, "codes"),
    ((A, C, A, A, A, None, None, 4, 64, 64, 1, A), m.ERR_ALIGN, "scales"),
    ((A, A, A, A, A, C, None, 4, 64, 64, 1, A), m.ERR_ALIGN, "pair_weight"),
    ((A, A, A, A, A, None, None, 4, 64, 64, 1, B), m.ERR_ALIGN, "out"),
])
def test_product(lib, args, code, text):
    refused(lib.moe_grouped_gemm_fp8(*args, None), code, text)


@pytest.mark.parametrize("args,code,text", [
    ((A, A, A, A, A, 4, 72, 64, 1, None, A, A), m.ERR_ALIGN, "H=72"),
    ((A, A, A, A, A, 4, 64, 72, 1, None, A, A), m.ERR_ALIGN, "I=72"),
    ((A, A, A, A, A, 4, 64, 64, 1, None, None, A), m.ERR_ARG, "act_codes"),
    ((A, A, A, A, A, 4, 64, 64, 1, None, A, None), m.ERR_ARG, "act_scales"),
    ((A, A, A, A, A, 4, 64, 64, 1, B, A, A), m.ERR_ALIGN, "gate_up"),
    ((A, A, A, A, None, 4, 64, 64, 3, None, A, A), m.ERR_ARG, "group_offsets"),
])
def test_gateup(lib, args, code, text):
    refused(lib.moe_grouped_gemm_gateup_silu_fp8(*args, None), code, text)


def test_data_gradient(lib):
    f = lib.moe_silu_mul_backward_fp8
    refused(f(A, A, -1, 64, A, A, None), m.ERR_ARG, "P=-1")
    refused(f(A, A, 1, 72, A, A, None), m.ERR_ALIGN, "I=72")
    refused(f(A, None, 1, 64, A, A, None), m.ERR_ARG, "NULL")
    refused(f(A, B, 1, 64, A, A, None), m.ERR_ALIGN, "16-byte")
    f = lib.moe_transpose_fp8w
    refused(f(A, A, 0, 64, 64, A, A, None), m.ERR_ARG, "G=0")
    refused(f(A, A, 1, 0, 64, A, A, None), m.ERR_ARG, "R=0")
    refused(f(A, A, 1, 64, 72, A, A, None), m.ERR_ALIGN, "C=72")
    refused(f(A, None, 1, 64, 64, A, A, None), m.ERR_ARG, "NULL")
    refused(f(A, A, 1, 64, 64, B, A, None), m.ERR_ALIGN, "16-byte")


@pytest.mark.parametrize("args,code,text", [
    ((A, m.F16, A, A, m.BF16, 1.0, 1, 1, 8, A, None, m.BF16), m.ERR_DTYPE, "f16"),
    ((A, m.BF16, A, A, 9, 1.0, 1, 1, 8, A, None, m.BF16), m.ERR_DTYPE, "dout"),
    ((A, m.BF16, A, A, m.BF16, 1.0, 1, 1, 8, A, None, 9), m.ERR_DTYPE, "d_expert_out"),
    ((A, m.BF16, A, A, m.BF16, 1.0, -1, 1, 8, A, None, m.BF16), m.ERR_ARG, "T=-1"),
    ((A, m.BF16, A, A, m.BF16, 1.0, 1, 65, 8, A, None, m.BF16), m.ERR_ARG, "K=65"),
    ((A, m.BF16, A, A, m.BF16, 1.0, 1, 1, 12, A, None, m.BF16), m.ERR_ALIGN, "H=12"),
    ((A, m.BF16, A, A, m.BF16, 1.0, 1, 1, 8, None, None, m.BF16), m.ERR_ARG, "output"),
    ((None, m.BF16, A, A, m.BF16, 1.0, 1, 1, 8, A, None, m.BF16), m.ERR_ARG, "NULL"),
    ((A, m.BF16, A, B, m.BF16, 1.0, 1, 1, 8, A, None, m.BF16), m.ERR_ALIGN, "16-byte"),
    ((A, m.BF16, C, A, m.BF16, 1.0, 1, 1, 8, A, None, m.BF16), m.ERR_ALIGN, "4-byte"),
])
def test_combine_backward(lib, args, code, text):
    refused(lib.moe_combine_backward(*args, None), code, text)


@pytest.mark.parametrize("args,code,text", [
    ((A, A, A, A, 1, 8, 2, 1, 2, 0.0, 0.0, A, None, None, 0), m.ERR_UNSUPPORTED, "scoring"),
    ((A, A, A, A, -1, 8, 2, 1, 0, 0.0, 0.0, A, None, None, 0), m.ERR_ARG, "T=-1"),
    ((A, A, A, A, 1, 1025, 2, 1, 0, 0.0, 0.0, A, None, None, 0), m.ERR_ARG, "E=1025"),
    ((A, A, A, A, 1, 8, 9, 1, 0, 0.0, 0.0, A, None, None, 0), m.ERR_ARG, "K=9"),
    ((A, A, A, A, 1, 64, 33, 1, 0, 0.0, 0.0, A, None, None, 0), m.ERR_ARG, "K=33"),
    ((A, A, A, A, 1, 8, 2, 2, 0, 0.0, 0.0, A, None, None, 0), m.ERR_ARG, "renormalize"),
    ((A, A, A, None, 1, 8, 2, 1, 0, 0.5, 0.0, A, None, None, 0), m.ERR_ARG, "expert_offsets"),
    ((A, A, A, A, 1, 8, 2, 1, 0, 0.0, 0.0, None, None, None, 0), m.ERR_ARG, "NULL"),
    ((C, A, A, A, 1, 8, 2, 1, 0, 0.0, 0.0, A, None, None, 0), m.ERR_ALIGN, "4-byte"),
    ((A, A, A, A, 1, 8, 2, 1, 0, 0.0, 0.0, A, A, None, 0), m.ERR_WORKSPACE, "workspace"),
    ((A, A, A, A, 1, 8, 2, 1, 0, 0.0, 0.0, A, A, A, 4), m.ERR_WORKSPACE, "workspace"),
])
def test_route_backward(lib, args, code, text):
    refused(lib.moe_route_backward(*args, None), code, text)


@pytest.mark.parametrize("args,code,text", [
    ((A, A, A, -1, 8, 8, A, A, A, A, 4096), m.ERR_ARG, "T=-1"),
    ((A, A, A, 1, 8, 1025, A, A, A, A, 4096), m.ERR_ARG, "E=1025"),
    ((A, A, A, 1, 12, 8, A, A, A, A, 4096), m.ERR_ALIGN, "H=12"),
    ((A, A, A, 1, 8, 8, None, None, None, A, 4096), m.ERR_ARG, "output"),
    ((A, None, A, 1, 8, 8, None, A, None, A, 4096), m.ERR_ARG, "NULL"),
    ((A, A, None, 1, 8, 8, A, None, None, A, 4096), m.ERR_ARG, "NULL"),
    ((A, B, A, 1, 8, 8, A, A, A, A, 4096), m.ERR_ALIGN, "16-byte"),
    ((C, A, A, 1, 8, 8, A, A, A, A, 4096), m.ERR_ALIGN, "4-byte"),
])
def test_route_logits_backward(lib, args, code, text):
    refused(lib.moe_route_logits_backward(*args, None), code, text)


def test_workspace_queries(lib):
    assert m.moe_route_backward_workspace_size(0, 8) == 0
    assert m.moe_route_backward_workspace_size(100, 8) >= 8
    assert m.moe_route_logits_backward_workspace_size(0, 64, 8) == 0
