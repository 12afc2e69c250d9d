"""Sizes near the end of int: the FP8 products and the gradients refuse what their 32-bit tile
arithmetic cannot hold, by name and before any CUDA call (no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest

import mixture_experts_ffn_renorm_gb300 as m
from mixture_experts_ffn_renorm_gb300 import build as moe_build

BUF = (ctypes.c_uint8 * 4096)()
A = ctypes.c_void_p((ctypes.addressof(BUF) + 15) & ~15)
TOP = 0x7FFFFFFF
HUGE = 1 << 62


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return m.lib()


def refused(rc, text):
    assert rc == m.ERR_ARG and text in m.last_error() and "too large" in m.last_error(), (rc, m.last_error())


@pytest.mark.parametrize("H", [TOP - 15, TOP - 511])
def test_quantiser(lib, H):
    H = H // 16 * 16
    refused(lib.moe_quantize_act_fp8(A, 1, H, 1, None, None, 1.0, A, A, None), f"H={H}")


@pytest.mark.parametrize("P,K,N,text", [(TOP, 16, 8, f"P={TOP}"), (TOP - 126, 16, 8, "P="), (1, TOP - 15, 8, "K="),
                                        (1, 16, TOP - 7, "N=")])
def test_product(lib, P, K, N, text):
    refused(lib.moe_grouped_gemm_fp8(A, A, A, A, A, None, None, P, K, N, 1, A, None), text)


@pytest.mark.parametrize("P,H,I,text", [(TOP, 16, 16, "P="), (1, TOP - 15, 16, "H="), (1, 16, 1 << 30, "I="),
                                        (1, 16, TOP - 15, "I=")])
def test_gateup(lib, P, H, I, text):
    refused(lib.moe_grouped_gemm_gateup_silu_fp8(A, A, A, A, A, P, H, I, 1, None, A, A, None), text)


def test_weight_rows_of_all_groups(lib):
    # the rows of a launch's groups are counted in int
    refused(lib.moe_grouped_gemm_fp8(A, A, A, A, A, None, None, 17, 16, 1 << 22, 512, A, None), "weight rows")
    refused(lib.moe_grouped_gemm_gateup_silu_fp8(A, A, A, A, A, 17, 16, 1 << 21, 1024, None, A, A, None), "weight rows")


@pytest.mark.parametrize("I", [(1 << 30) - 16, 1 << 30])
def test_silu_mul_backward(lib, I):
    refused(lib.moe_silu_mul_backward_fp8(A, A, 1, I, A, A, None), f"I={I}")


@pytest.mark.parametrize("R,C,text", [(TOP - 15, 16, "R="), (16, TOP - 15, "C="), (16 << 20, 16, "R=")])
def test_transpose(lib, R, C, text):
    refused(lib.moe_transpose_fp8w(A, A, 1, R, C, A, A, None), text)


def test_combine_backward(lib):
    H = TOP - 7
    refused(lib.moe_combine_backward(A, m.BF16, A, A, m.BF16, 1.0, 1, 1, H, A, None, m.BF16, None), f"H={H}")


@pytest.mark.parametrize("T", [TOP, TOP - 126, 65535 * 128 + 1])
def test_route_logits_backward_tokens(lib, T):
    refused(lib.moe_route_logits_backward(A, A, A, T, 8, 8, A, A, A, A, HUGE, None), f"T={T}")


def test_route_logits_backward_columns(lib):
    H = TOP - 7
    refused(lib.moe_route_logits_backward(A, A, A, 1, H, 8, A, A, A, A, HUGE, None), f"H={H}")


def test_route_backward_workspace_of_the_most_tokens(lib):
    assert lib.moe_route_backward_workspace_size(TOP, 8) == (1 << 28) * 8
    assert lib.moe_route_backward_workspace_size(9, 8) == 16
