"""What the layer for a few tokens, and the product with bias, activation and residual and its
gradients compute, and at which sizes they are measured.

Five kinds of case:
  layer         a whole MoE layer for at most 16 tokens: router, chosen experts, an optional shared
                expert behind its gate, the weighted sum and the residual; bf16 or FP8 weights
  product       rows in groups times their group's weights, plus bias, through an activation,
                times a row weight, scattered, plus a residual
  product_dx    the same product over the weights' other axis: the rows' gradient
  act_grad      the gradient of bias, activation and row weight
  weight_grad   the gradient of the groups' weights
"""
import math

import torch

own = False

BLOCK = 128
NONE, RELU, RELU2, GELU, GELU_TANH, SILU = range(6)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token of a chat, bf16 experts: the latency of a layer
        dict(name="layer T1", kind="layer", T=1, H=2048, I=768, E=128, K=8, Is=0, fp8=False, scoring=0, renormalize=1,
             groups=1, residual=False),
        # a decode batch: most experts serve one or two tokens, the weight stream counts
        dict(name="layer T16", kind="layer", T=16, H=2048, I=768, E=128, K=8, Is=0, fp8=False, scoring=0,
             renormalize=1, groups=1, residual=True),
        # two tokens through the wide layer with a gated shared expert
        dict(name="layer T2 wide", kind="layer", T=2, H=4096, I=1024, E=256, K=8, Is=1024, fp8=False, scoring=0,
             renormalize=1, groups=1, residual=True),
        # FP8 weights, sigmoid scores, expert groups, sizes off every tile edge
        dict(name="layer T5 fp8", kind="layer", T=5, H=1040, I=400, E=60, K=6, Is=208, fp8=True, scoring=1,
             renormalize=1, groups=4, residual=True),
        # one row through a dense projection of the wide layer, added to the residual stream
        dict(name="product 1 row", kind="product", P=1, C=4096, N=1024, G=1, skew=0.0, scatter=False, bias=False,
             act=NONE, residual=True, pre=False),
        # a decode batch through a dense layer's first projection
        dict(name="product 64 rows", kind="product", P=64, C=4096, N=4096, G=1, skew=0.0, scatter=False, bias=True,
             act=GELU_TANH, residual=False, pre=False),
        # the second projection of a prompt's experts: ragged groups, weighted and scattered rows
        dict(name="product ragged", kind="product", P=777, C=1040, N=1000, G=13, skew=1.5, scatter=True, bias=True,
             act=NONE, residual=False, pre=False),
        # the first projection of a training batch's experts, what the gradient needs kept
        dict(name="product 65536 rows", kind="product", P=65536, C=2048, N=768, G=128, skew=0.5, scatter=False,
             bias=True, act=GELU, residual=False, pre=True),
        # the rows' gradient through the second projection of a training batch's experts
        dict(name="product_dx 32768 rows", kind="product_dx", P=32768, C=2048, N=768, G=128, skew=0.5),
        # activation's gradient of the same batch, with bias and routing weights
        dict(name="act_grad 32768 rows", kind="act_grad", P=32768, N=768, G=128, skew=0.5, act=GELU, scatter=True),
        # weight gradient of small odd experts, some of them empty
        dict(name="weight_grad ragged", kind="weight_grad", P=777, C=1040, N=400, G=13, skew=1.5, add=True),
        # weight gradient of a training batch's experts
        dict(name="weight_grad 32768 rows", kind="weight_grad", P=32768, C=2048, N=768, G=128, skew=0.5, add=False),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], uniform in its logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(hi // step * step, max(step, lo, v))


def draw(rng):
    kind = rng.choice(["layer", "layer", "product", "product", "product_dx", "act_grad", "weight_grad"])
    skew = round(rng.uniform(0.0, 1.0), 2)
    if kind == "layer":
        fp8 = rng.random() < 0.5
        step = 16 if fp8 else 8
        T, H, I = rng.randint(1, 16), _spread(rng, 64, 4096, step), _spread(rng, 32, 1024, step)
        groups = rng.choice([1, 1, 2, 4])
        E = groups * _spread(rng, 4, 256 // groups)
        while E * H * I > 128 * 2048 * 1024:
            E = groups * max(4, E // 2 // groups)
        scoring = rng.randint(0, 1)
        return dict(kind=kind, T=T, H=H, I=I, E=E, K=rng.randint(1, min(8, max(1, groups // 2) * (E // groups))),
                    Is=rng.choice([0, _spread(rng, 32, 1024, 8)]), fp8=fp8, scoring=scoring,
                    renormalize=rng.randint(0, 1), groups=groups, residual=rng.random() < 0.5)
    G = _spread(rng, 1, 128)
    C, N = _spread(rng, 64, 4096, 8), _spread(rng, 64, 4096, 8)
    while G * C * N > 128 * 2048 * 768:
        G = max(1, G // 2)
    P = _spread(rng, 1, 65536)
    while P * C * N > 32768 * 2048 * 768:
        P = max(1, P // 2)
    c = dict(kind=kind, P=P, C=C, N=N, G=G, skew=skew)
    if kind == "product":
        c.update(scatter=rng.random() < 0.5, bias=rng.random() < 0.5, act=rng.randrange(6),
                 residual=rng.random() < 0.5, pre=rng.random() < 0.5)
    elif kind == "act_grad":
        del c["C"]
        c.update(act=rng.randrange(6), scatter=rng.random() < 0.5)
    elif kind == "weight_grad":
        c["add"] = rng.random() < 0.5
    return c


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    k = case["kind"]
    if k == "layer":
        T, H, I, E, K, Is = (case[n] for n in ("T", "H", "I", "E", "K", "Is"))
        touched = E * (1.0 - (1.0 - K / E) ** T)   # experts that T tokens' choices meet
        w = touched * 3 * H * I * (1 if case["fp8"] else 2)
        if case["fp8"]:
            w += 4 * touched * (_blocks(2 * I) + _blocks(I)) * _blocks(H)
        rows = 2 * T * H * (3 if case["residual"] else 2) + 8 * T * K
        shared = (6 * H * Is + 2 * H) if Is else 0
        return {"bytes": int(w + rows + shared + 2 * E * H), "flops": T * (6 * H * (K * I + Is) + 2 * H * E)}
    P, N, G = case["P"], case["N"], min(case["G"], case["P"])
    if k == "product":
        C = case["C"]
        rows = 2 * P * C + 2 * P * N * (1 + case["residual"] + case["pre"]) + (8 * P if case["scatter"] else 0)
        return {"bytes": rows + G * (2 * C * N + (4 * N if case["bias"] else 0)), "flops": 2 * P * C * N}
    if k == "product_dx":
        C = case["C"]
        return {"bytes": 2 * P * C + 2 * P * N + 2 * G * C * N, "flops": 2 * P * C * N}
    if k == "act_grad":
        return {"bytes": 2 * P * N * (3 if case["act"] or case["scatter"] else 2) + 4 * case["G"] * N + (12 * P if case["scatter"] else 0),
                "flops": 12 * P * N}
    C = case["C"]
    return {"bytes": 2 * P * (C + N) + 4 * case["G"] * C * N * (1 + case["add"]), "flops": 2 * P * C * N}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, std, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _fp8_weights(g, G, R, C, std):
    """Trained-like weights as E4M3 codes [G, R, C] and a scale per 128 x 128 block."""
    rb, cb = _blocks(R), _blocks(C)
    w = torch.zeros((G, rb * BLOCK, cb * BLOCK), device="cuda")
    w[:, :R, :C] = torch.randn((G, R, C), generator=g, device="cuda") * std
    w = w.view(G, rb, BLOCK, cb, BLOCK)
    scale = (w.abs().amax((2, 4)) / 448.0).clamp_min(2.0 ** -126)
    codes = (w / scale[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(G, rb * BLOCK, cb * BLOCK)[:, :R, :C].contiguous(), scale


def _grouping(g, P, G, skew):
    """Rows in groups of uneven sizes: offsets, a destination for every row, the largest group."""
    rank = torch.randperm(G, generator=g, device="cuda") + 1
    u = torch.rand((P, G), generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)
    group = (-torch.log(-torch.log(u)) - skew * torch.log(rank.float())).argmax(1)
    counts = torch.bincount(group, minlength=G)
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return off.int(), torch.argsort(group, stable=True).int(), int(counts.max())


def prepare(case, seed):
    g = _gen(seed)
    k = case["kind"]
    s = dict(case)
    bf = torch.bfloat16
    if k == "layer":
        T, H, I, E, K, Is = (case[n] for n in ("T", "H", "I", "E", "K", "Is"))
        s["x"] = _normal(g, (T, H), 1.0, bf)
        s["wr"] = _normal(g, (E, H), H ** -0.5, bf)
        s["bias"] = _normal(g, (E,), 0.3)
        s["select"] = _normal(g, (E,), 0.1) if case["scoring"] else None
        std = (H ** -0.5, I ** -0.5)
        if case["fp8"]:
            s["w13"], s["w13s"] = _fp8_weights(g, E, 2 * I, H, std[0])
            s["w2"], s["w2s"] = _fp8_weights(g, E, H, I, std[1])
        else:
            s["w13"], s["w2"] = _normal(g, (E, 2 * I, H), std[0], bf), _normal(g, (E, H, I), std[1], bf)
        if Is:
            s["wg"] = _normal(g, (H,), H ** -0.5, bf)
            s["w13_sh"], s["w2_sh"] = _normal(g, (2 * Is, H), std[0], bf), _normal(g, (H, Is), Is ** -0.5, bf)
        s["res"] = _normal(g, (T, H), 1.0, bf) if case["residual"] else None
        s["scale"] = 2.5 if case["scoring"] else 1.0
        s["ids"] = torch.empty((T, K), dtype=torch.int32, device="cuda")
        s["w"] = torch.empty((T, K), device="cuda")
        s["out"] = torch.empty((T, H), dtype=bf, device="cuda")
        return s
    P, N, G = case["P"], case["N"], case["G"]
    s["off"], order, s["cap"] = _grouping(g, P, G, case["skew"])
    s["dst"] = order if case.get("scatter") else None
    s["pw"] = torch.rand((P,), generator=g, device="cuda") if case.get("scatter") else None
    if k == "act_grad":
        s["z"] = _normal(g, (P, N), 1.0, bf)
        s["dout"] = _normal(g, (P, N), 0.1, bf)
        s["dz"] = torch.empty((P, N), dtype=bf, device="cuda")
        s["db"] = torch.empty((G, N), device="cuda")
        s["dpw"] = torch.empty((P,), device="cuda") if case["scatter"] else None
        return s
    C = case["C"]
    if k == "weight_grad":
        s["dz"] = _normal(g, (P, N), 0.1, bf)
        s["a"] = _normal(g, (P, C), 1.0, bf)
        s["sum"] = _normal(g, (G, N, C), 1.0) if case["add"] else None   # of the batches before
        s["dw"] = torch.empty((G, N, C), device="cuda")
        return s
    s["a"] = _normal(g, (P, C), 1.0, bf)
    # product: [G, N, C], a row per output column; product_dx: [G, C, N], the layer's own weights
    s["wt"] = _normal(g, (G, N, C) if k == "product" else (G, C, N), C ** -0.5, bf)
    s["b"] = _normal(g, (G, N), 0.5) if case.get("bias") else None
    s["res"] = _normal(g, (P, N), 1.0, bf) if case.get("residual") else None
    s["out"] = torch.empty((P, N), dtype=bf, device="cuda")
    s["z"] = torch.empty((P, N), dtype=bf, device="cuda") if case.get("pre") else None
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return (_own if own else _plain)[state["kind"]](state)


def _kept(state, size):
    """The workspace that a program keeps with its buffers: zero-filled once."""
    if "ws" not in state:
        state["ws"] = torch.zeros(max(16, size), dtype=torch.uint8, device="cuda")
    return state["ws"]


def _top_groups(groups):
    return max(1, groups // 2)


def _own_layer(s):
    import mixture_experts_ffn_renorm_gb300 as m

    T, H, I, E, K, Is = (s[n] for n in ("T", "H", "I", "E", "K", "Is"))
    ws = _kept(s, m.moe_layer_few_workspace_size(T, H, I, E, K, Is))
    shared = (s["wg"], s["w13_sh"], s["w2_sh"]) if Is else (None, None, None)
    rest = (*shared, s["res"], T, H, I, E, K, Is, s["renormalize"], s["scoring"], s["groups"], _top_groups(s["groups"]),
            0, s["scale"], s["ids"], s["w"], s["out"], ws, ws.numel())
    if s["fp8"]:
        m.moe_layer_few_fp8w(s["x"], s["wr"], s["bias"], s["select"], s["w13"], s["w13s"], s["w2"], s["w2s"], *rest)
    else:
        m.moe_layer_few_bf16(s["x"], s["wr"], s["bias"], s["select"], s["w13"], s["w2"], *rest)
    return {"out": s["out"], "ids": s["ids"], "w": s["w"]}


def _own_product(s):
    import mixture_experts_ffn_renorm_gb300 as m

    P, C, N, G = s["P"], s["C"], s["N"], s["G"]
    ws = _kept(s, m.moe_grouped_gemm_bias_act_workspace_size(P, C, N, G))
    m.moe_grouped_gemm_bias_act_bf16(s["a"], s["wt"], m.W_ROWS, s["b"], s["act"], s["z"], s["pw"], s["dst"], s["res"],
                                     s["off"], P, C, N, G, s["out"], ws, ws.numel())
    return {"out": s["out"], "z": s["z"]}


def _own_product_dx(s):
    import mixture_experts_ffn_renorm_gb300 as m

    P, C, N, G = s["P"], s["C"], s["N"], s["G"]
    ws = _kept(s, m.moe_grouped_gemm_bias_act_workspace_size(P, C, N, G))
    m.moe_grouped_gemm_bias_act_bf16(s["a"], s["wt"], m.W_COLUMNS, None, NONE, None, None, None, None, s["off"], P, C, N,
                                     G, s["out"], ws, ws.numel())
    return s["out"]


def _own_act_grad(s):
    import mixture_experts_ffn_renorm_gb300 as m

    P, N, G = s["P"], s["N"], s["G"]
    ws = _kept(s, m.moe_bias_act_backward_workspace_size(P, N, G))
    m.moe_bias_act_backward(s["dout"], s["z"], s["act"], s["pw"], s["dst"], s["off"], P, N, G, s["dz"], s["db"],
                            s["dpw"], ws, ws.numel())
    return {"dz": s["dz"], "dbias": s["db"], "dweight": s["dpw"]}


def _own_weight_grad(s):
    import mixture_experts_ffn_renorm_gb300 as m

    P, C, N, G = s["P"], s["C"], s["N"], s["G"]
    ws = _kept(s, m.moe_grouped_gemm_wgrad_workspace_size(P, N, C, G))
    m.moe_grouped_gemm_wgrad_bf16(s["dz"], s["a"], s["off"], P, N, C, G, s["sum"], s["dw"], ws, ws.numel())
    return s["dw"]


_own = {"layer": _own_layer, "product": _own_product, "product_dx": _own_product_dx, "act_grad": _own_act_grad,
        "weight_grad": _own_weight_grad}


# the plain forms: binary32 arithmetic on torch's elementary operations; logits, whose order
# decides whole numbers, in binary64
def _expanded(codes, scale):
    R, C = codes.shape[-2:]
    s = scale.repeat_interleave(BLOCK, -2)[..., :R, :].repeat_interleave(BLOCK, -1)[..., :C]
    return codes.view(torch.float8_e4m3fn).float() * s


def _chosen(s):
    """Ids and weights of the chosen experts, in binary64."""
    E, K, n = s["E"], s["K"], s["groups"]
    l = s["x"].double() @ s["wr"].double().t() + s["bias"].double()
    score = 1.0 / (1.0 + torch.exp(-l)) if s["scoring"] else l
    key = score + s["select"].double() if s["scoring"] else score
    if n > 1:
        best = key.view(-1, n, E // n).amax(2)
        rank = torch.argsort(torch.argsort(-best, dim=1, stable=True), dim=1)
        out = (rank >= _top_groups(n)).repeat_interleave(E // n, 1)
        key = key.masked_fill(out, -math.inf)
    ids = torch.argsort(-key, dim=1, stable=True)[:, :K]
    if s["scoring"]:
        w = score.gather(1, ids)
        total = w.sum(1, keepdim=True) if s["renormalize"] else 1.0
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        w = e.gather(1, ids)
        total = (w if s["renormalize"] else e).sum(1, keepdim=True)
    return ids, w / total


def _swiglu(x, w13, w2, I):
    """x [B, H], w13 [B, 2I, H], w2 [B, H, I]: one expert per row."""
    gu = torch.bmm(w13, x[:, :, None])[:, :, 0]
    gate, up = gu[:, :I], gu[:, I:]
    act = gate / (1.0 + torch.exp(-gate)) * up
    return torch.bmm(w2, act[:, :, None])[:, :, 0]


def _plain_layer(s):
    T, H, I, K = s["T"], s["H"], s["I"], s["K"]
    ids, w = _chosen(s)
    x, e = s["x"].float(), ids.reshape(-1)
    if s["fp8"]:
        w13, w2 = _expanded(s["w13"][e], s["w13s"][e]), _expanded(s["w2"][e], s["w2s"][e])
    else:
        w13, w2 = s["w13"][e].float(), s["w2"][e].float()
    y = _swiglu(x.repeat_interleave(K, 0), w13, w2, I).view(T, K, H)
    out = (y * w.float()[:, :, None]).sum(1) * s["scale"]
    if s["Is"]:
        Is = s["Is"]
        gu = x @ s["w13_sh"].float().t()
        act = gu[:, :Is] / (1.0 + torch.exp(-gu[:, :Is])) * gu[:, Is:]
        gate = 1.0 / (1.0 + torch.exp(-(x @ s["wg"].float())))
        out = out + gate[:, None] * (act @ s["w2_sh"].float().t())
    if s["residual"]:
        out = out + s["res"].float()
    return {"out": out.to(torch.bfloat16), "ids": ids.int(), "w": w.float()}


def _group_of(off, P):
    r = torch.arange(P, device="cuda")
    return (r[:, None] >= off.long()[None, 1:]).sum(1)


def _padded(a, off, cap):
    """Rows of a [P, C] as [G, cap, C], zeros behind each group's rows."""
    off = off.long()
    at = off[:-1, None] + torch.arange(cap, device="cuda")
    return a[at.clamp_max(a.shape[0] - 1)] * (at < off[1:, None])[:, :, None]


def _grouped(a, w, off, cap):
    """Rows of a [P, C] in groups off [G + 1] times w [G, C, N]: f32 [P, N]."""
    if w.shape[0] == 1:
        return a @ w[0]
    y = torch.bmm(_padded(a, off, cap), w)
    group = _group_of(off, a.shape[0])
    return y[group, torch.arange(a.shape[0], device="cuda") - off.long()[group]]


def _activated(z, act):
    if act == RELU:
        return z.clamp_min(0.0)
    if act == RELU2:
        return z.clamp_min(0.0).square()
    if act == GELU:
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == GELU_TANH:
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == SILU:
        return z / (1.0 + torch.exp(-z))
    return z


def _slope(z, act):
    if act == RELU:
        return (z > 0.0).to(z.dtype)
    if act == RELU2:
        return 2.0 * z.clamp_min(0.0)
    if act == GELU:
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == GELU_TANH:
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if act == SILU:
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _plain_product(s):
    z = _grouped(s["a"].float(), s["wt"].float().transpose(1, 2), s["off"], s["cap"])
    if s["bias"]:
        z = z + s["b"][_group_of(s["off"], s["P"])]
    y = _activated(z, s["act"])
    if s["scatter"]:
        dst = s["dst"].long()
        y = torch.empty_like(y).index_copy_(0, dst, y * s["pw"][dst, None])
    if s["residual"]:
        y = y + s["res"].float()
    return {"out": y.to(torch.bfloat16), "z": z.to(torch.bfloat16) if s["pre"] else None}


def _plain_product_dx(s):
    return _grouped(s["a"].float(), s["wt"].float(), s["off"], s["cap"]).to(torch.bfloat16)


def _plain_act_grad(s):
    d, z = s["dout"].float(), s["z"].float()
    dpw = None
    if s["scatter"]:
        dst = s["dst"].long()
        d = d[dst]
        dpw = torch.empty_like(s["pw"]).index_copy_(0, dst, (d * _activated(z, s["act"])).sum(1))
        d = d * s["pw"][dst, None]
    dz = d * _slope(z, s["act"])
    db = torch.zeros_like(s["db"]).index_add_(0, _group_of(s["off"], s["P"]), dz)
    return {"dz": dz.to(torch.bfloat16), "dbias": db, "dweight": dpw}


def _plain_weight_grad(s):
    dz, a = s["dz"].float(), s["a"].float()
    if s["G"] == 1:
        y = (dz.t() @ a)[None]
    else:
        y = torch.bmm(_padded(dz, s["off"], s["cap"]).transpose(1, 2), _padded(a, s["off"], s["cap"]))
    return s["sum"] + y if s["add"] else y


_plain = {"layer": _plain_layer, "product": _plain_product, "product_dx": _plain_product_dx,
          "act_grad": _plain_act_grad, "weight_grad": _plain_weight_grad}


# ------------------------------------------------------------------ in 64 bits
def _exact_weights(codes, scale):
    if scale is None:
        return codes.double()
    i, j = torch.arange(codes.shape[0], device="cuda") // BLOCK, torch.arange(codes.shape[1], device="cuda") // BLOCK
    return codes.view(torch.float8_e4m3fn).double() * scale.double()[i[:, None], j[None, :]]


def _exact_expert(x, w13, w2):
    gate, up = (w13 @ x).chunk(2)
    return w2 @ (torch.nn.functional.silu(gate) * up)


def _exact_layer(s):
    T, E, K, n = s["T"], s["E"], s["K"], s["groups"]
    out = torch.zeros((T, s["H"]), dtype=torch.float64, device="cuda")
    w = torch.zeros((T, K), dtype=torch.float64, device="cuda")
    ids = torch.zeros((T, K), dtype=torch.int32, device="cuda")
    logits = torch.einsum("th,eh->te", s["x"].double(), s["wr"].double()) + s["bias"].double()
    for t in range(T):
        l = logits[t]
        p = torch.sigmoid(l) if s["scoring"] else torch.softmax(l, 0)
        key = (p + s["select"].double() if s["scoring"] else l).tolist()
        best = sorted(range(n), key=lambda j: (-max(key[j * E // n:(j + 1) * E // n]), j))[:_top_groups(n)]
        pick = sorted((e for e in range(E) if e * n // E in best), key=lambda e: (-key[e], e))[:K]
        total = p[pick].sum() if s["renormalize"] else 1.0
        x = s["x"][t].double()
        for j, e in enumerate(pick):
            ids[t, j], w[t, j] = e, p[e] / total
            y = _exact_expert(x, _exact_weights(s["w13"][e], s["w13s"][e] if s["fp8"] else None),
                              _exact_weights(s["w2"][e], s["w2s"][e] if s["fp8"] else None))
            out[t] += s["scale"] * w[t, j] * y
        if s["Is"]:
            out[t] += torch.sigmoid(s["wg"].double() @ x) * _exact_expert(x, s["w13_sh"].double(), s["w2_sh"].double())
        if s["residual"]:
            out[t] += s["res"][t].double()
    return {"out": out, "ids": ids, "w": w}


def _torch_act(z, act):
    f = torch.nn.functional
    return [lambda v: v, torch.relu, lambda v: torch.relu(v) ** 2, f.gelu, lambda v: f.gelu(v, approximate="tanh"),
            f.silu][act](z)


def exact(case, seed):
    s = prepare(case, seed)
    k = case["kind"]
    if k == "layer":
        return _exact_layer(s)
    off, P, N, G = s["off"].tolist(), case["P"], case["N"], case["G"]
    if k == "act_grad":
        z = s["z"].double().requires_grad_()
        d = s["dout"].double()
        if case["scatter"]:
            pw = s["pw"].double().requires_grad_()
            y = _torch_act(z, case["act"]) * pw[s["dst"].long(), None]
            dz, dpw = torch.autograd.grad(y, (z, pw), d[s["dst"].long()])
        else:
            (dz,), dpw = torch.autograd.grad(_torch_act(z, case["act"]), (z,), d), None
        db = torch.stack([dz[off[i]:off[i + 1]].sum(0) for i in range(G)])
        return {"dz": dz, "dbias": db, "dweight": dpw}
    if k == "weight_grad":
        dw = s["sum"].double() if case["add"] else torch.zeros((G, N, case["C"]), dtype=torch.float64, device="cuda")
        for i in range(G):
            dw[i] += torch.einsum("rn,rc->nc", s["dz"][off[i]:off[i + 1]].double(), s["a"][off[i]:off[i + 1]].double())
        return dw
    z = torch.empty((P, N), dtype=torch.float64, device="cuda")
    for i in range(G):
        w = s["wt"][i].double()
        z[off[i]:off[i + 1]] = s["a"][off[i]:off[i + 1]].double() @ (w.t() if k == "product" else w)
        if case.get("bias"):
            z[off[i]:off[i + 1]] += s["b"][i].double()
    if k == "product_dx":
        return z
    y = _torch_act(z, case["act"])
    if case["scatter"]:
        y = torch.zeros_like(y).index_copy_(0, s["dst"].long(), y) * s["pw"].double()[:, None]
    if case["residual"]:
        y = y + s["res"].double()
    return {"out": y, "z": z if case["pre"] else None}
