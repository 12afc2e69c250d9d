"""The blocks refuse tensors of other sizes than theirs before any kernel sees their addresses (no GPU
needed: the blocks here are built without their constructors)."""
from __future__ import annotations

import pytest
import torch

from mixture_experts_ffn_renorm_gb300.layer import MoeBlock, MoeMlpBlock

H, I, E, K = 64, 32, 4, 2


def rows(T, n=H, dt=torch.bfloat16):
    return torch.zeros((T, n), dtype=dt)


def block(cls):
    b = cls.__new__(cls)
    b.H, b.I, b.E, b.K, b.max_tokens, b.training, b._tokens, b.workspace, b.few_tokens = H, I, E, K, 8, True, 4, None, 0
    return b


WRONG = [rows(4, 32), rows(4, 72), torch.zeros((4, H, 1), dtype=torch.bfloat16), torch.zeros((4,), dtype=torch.bfloat16)]
TYPES = [rows(4, dt=torch.float32), rows(4, 2 * H)[:, ::2]]


@pytest.mark.parametrize("x", WRONG, ids=lambda t: str(list(t.shape)))
@pytest.mark.parametrize("cls", [MoeBlock, MoeMlpBlock])
def test_rows_of_another_width(cls, x):
    with pytest.raises(ValueError, match=f"x must be contiguous bf16 rows of {H}"):
        block(cls).forward(x)
    with pytest.raises(ValueError, match="out must be"):
        block(cls).forward(rows(4), out=x)


@pytest.mark.parametrize("t", TYPES, ids=["f32", "strided"])
def test_other_types_and_strides(t):
    b = block(MoeMlpBlock)
    for call in (lambda: b.forward(t), lambda: b.forward(rows(4), residual=t), lambda: b.forward(rows(4), out=t),
                 lambda: b.backward(t, rows(4)), lambda: b.backward(rows(4), t)):
        with pytest.raises(ValueError, match="must be contiguous bf16 rows"):
            call()
    with pytest.raises(ValueError, match="out must be"):
        block(MoeBlock).forward(rows(4), out=t)


def test_rows_of_another_number():
    with pytest.raises(ValueError, match="out has 3 rows for 4 tokens"):
        block(MoeBlock).forward(rows(4), out=rows(3))
    b = block(MoeMlpBlock)
    for kw, what in ((dict(out=rows(3)), "out"), (dict(residual=rows(5)), "residual")):
        with pytest.raises(ValueError, match=f"{what} has . rows for 4 tokens"):
            b.forward(rows(4), **kw)
    with pytest.raises(ValueError, match="dout has 3 rows"):
        b.backward(rows(4), rows(3))
    with pytest.raises(ValueError, match="dout must be"):
        b.backward(rows(4), rows(4, 72))
    with pytest.raises(ValueError, match="x must be"):
        b.backward(rows(4, 72), rows(4, 72))
    with pytest.raises(ValueError, match="x must be"):
        block(MoeBlock).backward(rows(4, 72), rows(4, 72))


GOOD = dict(w_router=(E, H), w1=(E, I, H), w2=(E, H, I), b1=(E, I), b2=(E, H), logit_bias=(E,))


def weights(**kw):
    shapes = {**GOOD, **kw}
    return {k: None if s is None else torch.zeros(s, dtype=torch.bfloat16 if k.startswith("w") else torch.float32)
            for k, s in shapes.items()}


@pytest.mark.parametrize("key,shape", [
    ("w_router", (E, H + 8)), ("w_router", None), ("w1", (E, H, I)), ("w1", (E, 2 * I, H)), ("w2", (E, I, H)),
    ("w2", (E - 1, H, I)), ("b1", (E, H)), ("b2", (H,)), ("logit_bias", (E + 1,)),
])
def test_weights_of_another_shape(key, shape):
    with pytest.raises(ValueError, match=f"{key} must be"):
        MoeMlpBlock(H, I, E, K, weights(**{key: shape}), max_tokens=4)


def test_weights_of_another_type():
    w = weights()
    w["w1"] = w["w1"].float()
    with pytest.raises(ValueError, match="w1 must be bf16"):
        MoeMlpBlock(H, I, E, K, w, max_tokens=4)
