"""What the FP8 expert products, their data gradient, and the gradients of the
combine and of the router compute, and at which sizes they are measured.

Five kinds of case:
  product       rows quantised to E4M3 (a scale per row and 128 columns), times grouped E4M3
                weights (a scale per 128 x 128 block), optional row weight and scatter
  experts       the routed experts of one MoE layer in FP8: quantise the routed rows, gate/up
                with SiLU-mul, down with the routing weight, rows in (token, slot) order
  experts_grad  the gradient of that path with respect to its input rows, weights frozen
  combine_grad  the gradient of the weighted top-k sum: routing weights and expert rows
  route_grad    the gradient of the router: its logits (with the balance loss and the z-loss),
                the tokens, the router weight and the logit bias
"""
import math

import torch

own = False

BLOCK = 128
F32, BF16 = 0, 1


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token of a chat: eight experts, each with one row; latency of the calls
        dict(name="experts T1", kind="experts", T=1, H=2048, I=768, E=128, K=8, skew=0.5, train=False),
        # a decode batch: most experts hold one or two rows, the weight stream counts
        dict(name="experts T16", kind="experts", T=16, H=2048, I=768, E=128, K=8, skew=0.5, train=False),
        # prefill of a long prompt with an uneven load
        dict(name="experts T8192", kind="experts", T=8192, H=2048, I=768, E=128, K=8, skew=0.5, train=False),
        # one row through a dense projection of the wide layer
        dict(name="product 1 row", kind="product", P=1, C=4096, N=1024, G=1, skew=0.0, scatter=False),
        # ragged groups, some of them empty, sizes off every tile edge, weighted and scattered
        dict(name="product ragged", kind="product", P=777, C=1040, N=1000, G=13, skew=1.5, scatter=True),
        # a dense projection of a training batch
        dict(name="product 8192 rows", kind="product", P=8192, C=4096, N=2048, G=1, skew=0.0, scatter=False),
        # backward through small odd experts
        dict(name="experts_grad T128", kind="experts_grad", T=128, H=1040, I=400, E=12, K=3, skew=1.0),
        # backward of a training batch
        dict(name="experts_grad T4096", kind="experts_grad", T=4096, H=2048, I=768, E=128, K=8, skew=0.5),
        # backward of the combine: f32 rows, few tokens, the routing weights' gradient alone
        dict(name="combine_grad T37 f32", kind="combine_grad", T=37, K=3, H=520, bf16=False, rows=False),
        # the same of a training batch in bf16, with the expert rows' gradient
        dict(name="combine_grad T4096", kind="combine_grad", T=4096, K=8, H=2048, bf16=True, rows=True),
        # sigmoid router of a small layer, no auxiliary losses, an expert count off every tile
        dict(name="route_grad T300", kind="route_grad", T=300, H=1032, E=60, K=6, scoring=1, renormalize=1,
             balance=0.0, z=0.0),
        # softmax router of a training batch with both auxiliary losses
        dict(name="route_grad T8192", kind="route_grad", T=8192, H=2048, E=128, K=8, scoring=0, renormalize=1,
             balance=0.01, z=0.001),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], uniform in its logarithm (and not 3072)."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    v = min(hi // step * step, max(step, lo, v))
    return v if v != 3072 else v - step


def draw(rng):
    kind = rng.choice(["experts", "product", "experts_grad", "combine_grad", "route_grad"])
    skew = round(rng.uniform(0.0, 1.0), 2)
    if kind in ("experts", "experts_grad"):
        H, I = _spread(rng, 64, 4096, 16), _spread(rng, 32, 1024, 16)
        E = _spread(rng, 4, 256)
        while E * H * I > 128 * 2048 * 768:
            E = max(4, E // 2)
        K = rng.randint(1, min(8, E))
        T = _spread(rng, 1, 8192 if kind == "experts" else 4096)
        while T * K * H * I > 4096 * 8 * 2048 * 768:
            T = max(1, T // 2)
        c = dict(kind=kind, T=T, H=H, I=I, E=E, K=K, skew=skew)
        if kind == "experts":
            c["train"] = rng.random() < 0.5
        return c
    if kind == "product":
        G = _spread(rng, 1, 64)
        C, N = _spread(rng, 64, 4096, 16), _spread(rng, 64, 4096, 8)
        P = _spread(rng, 1, 8192)
        return dict(kind=kind, P=P, C=C, N=N, G=G, skew=skew, scatter=rng.random() < 0.5)
    if kind == "combine_grad":
        return dict(kind=kind, T=_spread(rng, 1, 4096), K=rng.randint(1, 8), H=_spread(rng, 64, 4096, 8),
                    bf16=rng.random() < 0.7, rows=rng.random() < 0.5)
    E = _spread(rng, 4, 512)
    aux = rng.random() < 0.5
    return dict(kind=kind, T=_spread(rng, 1, 8192), H=_spread(rng, 64, 4096, 8), E=E, K=rng.randint(1, min(8, E)),
                scoring=rng.randint(0, 1), renormalize=rng.randint(0, 1), balance=0.01 if aux else 0.0,
                z=0.001 if aux else 0.0)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    k = case["kind"]
    if k == "product":
        P, C, N, G = case["P"], case["C"], case["N"], case["G"]
        g = min(G, P)
        return {"bytes": 2 * P * C + g * (C * N + 4 * _blocks(C) * _blocks(N)) + 2 * P * N, "flops": 2 * P * C * N}
    if k in ("experts", "experts_grad"):
        T, H, I, E, K = (case[n] for n in "THIEK")
        P = T * K
        g = min(E, P)
        w = g * (3 * H * I + 4 * (_blocks(2 * I) + _blocks(I)) * _blocks(H))
        rows = 2 * P * H + 2 * T * H + 12 * P  # out, x (or the output's gradient), plan and weights
        if k == "experts_grad" or case.get("train"):
            rows += 4 * P * I  # gate and up, read by the gradient, written for it
        return {"bytes": w + rows, "flops": 6 * P * H * I}
    if k == "combine_grad":
        T, K, H = (case[n] for n in "TKH")
        e = 2 if case["bf16"] else 4
        return {"bytes": e * T * H * (K + 1 + (K if case["rows"] else 0)) + 8 * T * K,
                "flops": T * K * H * (3 if case["rows"] else 2)}
    T, H, E, K = (case[n] for n in "THEK")
    return {"bytes": 8 * T * E + 8 * T * K + 4 * T * H + 6 * E * H, "flops": 4 * T * E * H + 16 * T * E}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, std, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _weights(g, G, R, C, std):
    """Trained-like weights as E4M3 codes [G, R, C] and a scale per 128 x 128 block."""
    rb, cb = _blocks(R), _blocks(C)
    w = torch.zeros((G, rb * BLOCK, cb * BLOCK), device="cuda")
    w[:, :R, :C] = torch.randn((G, R, C), generator=g, device="cuda") * std
    w = w.view(G, rb, BLOCK, cb, BLOCK)
    scale = (w.abs().amax((2, 4)) / 448.0).clamp_min(2.0 ** -126)
    codes = (w / scale[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(G, rb * BLOCK, cb * BLOCK)[:, :R, :C].contiguous(), scale


def _plan(group, G):
    """Stable grouping of rows by `group`: offsets, the row order and its inverse."""
    order = torch.argsort(group, stable=True)
    inverse = torch.empty_like(order)
    inverse[order] = torch.arange(order.numel(), device="cuda")
    counts = torch.bincount(group, minlength=G)
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return off.int(), order.int(), inverse.int(), int(counts.max())


def _uneven(g, n, E, skew):
    """Scores whose best entries favour some of the E experts by rank ** -skew."""
    rank = torch.randperm(E, generator=g, device="cuda") + 1
    u = torch.rand((n, E), generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)
    return -torch.log(-torch.log(u)) - skew * torch.log(rank.float())


def prepare(case, seed):
    g = _gen(seed)
    k = case["kind"]
    s = dict(case)
    bf = torch.bfloat16
    if k == "product":
        P, C, N, G = case["P"], case["C"], case["N"], case["G"]
        group = _uneven(g, P, G, case["skew"]).argmax(1)
        s["off"], order, _, s["cap"] = _plan(group, G)
        s["x"] = _normal(g, (P, C), 1.0, bf)
        s["w"], s["ws"] = _weights(g, G, N, C, 0.02)
        s["dst"] = order if case["scatter"] else None
        s["pw"] = torch.rand((P,), generator=g, device="cuda") if case["scatter"] else None
        s["codes"] = torch.empty((P, C), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty((P, _blocks(C)), device="cuda")
        s["out"] = torch.empty((P, N), dtype=bf, device="cuda")
    elif k in ("experts", "experts_grad"):
        T, H, I, E, K = (case[n] for n in "THIEK")
        P = T * K
        top = _uneven(g, T, E, case["skew"]).topk(K, dim=1)
        s["off"], s["sorted_pair"], s["pair_to_row"], s["cap"] = _plan(top.indices.reshape(-1), E)
        s["pw"] = torch.softmax(top.values, 1).reshape(-1)
        s["x"] = _normal(g, (T, H), 1.0 if k == "experts" else 0.1, bf)  # the tokens, or the output's gradient
        w13, w13s = _weights(g, E, 2 * I, H, 0.02)
        w2, w2s = _weights(g, E, H, I, 0.02)
        if k == "experts":
            s["w13"], s["w13s"], s["w2"], s["w2s"] = w13, w13s, w2, w2s
            s["gu"] = torch.empty((P, 2 * I), dtype=bf, device="cuda") if case["train"] else None
            s["mid"] = torch.empty((P, I), dtype=torch.uint8, device="cuda")
            s["mids"] = torch.empty((P, _blocks(I)), device="cuda")
        else:  # the copies that a backward pass keeps, contraction along their rows
            s["w13"], s["w13s"] = w13.transpose(1, 2).contiguous(), w13s.transpose(1, 2).contiguous()
            s["w2"], s["w2s"] = w2.transpose(1, 2).contiguous(), w2s.transpose(1, 2).contiguous()
            s["gu"] = _normal(g, (P, 2 * I), 1.0, bf)
            s["dact"] = torch.empty((P, I), dtype=bf, device="cuda")
            s["mid"] = torch.empty((P, 2 * I), dtype=torch.uint8, device="cuda")
            s["mids"] = torch.empty((P, _blocks(2 * I)), device="cuda")
        s["codes"] = torch.empty((P, H), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty((P, _blocks(H)), device="cuda")
        s["out"] = torch.empty((P, H), dtype=bf, device="cuda")
    elif k == "combine_grad":
        T, K, H = (case[n] for n in "TKH")
        dt = bf if case["bf16"] else torch.float32
        s["eo"] = _normal(g, (T, K, H), 1.0, dt)
        s["dout"] = _normal(g, (T, H), 0.1, dt)
        s["pw"] = torch.softmax(_normal(g, (T, K), 1.0), 1)
        s["dw"] = torch.empty((T, K), device="cuda")
        s["deo"] = torch.empty((T, K, H), dtype=dt, device="cuda") if case["rows"] else None
    else:
        T, H, E, K = (case[n] for n in "THEK")
        s["x"] = _normal(g, (T, H), 1.0, bf)
        s["wr"] = _normal(g, (E, H), 0.02, bf)
        s["logits"] = s["x"].float() @ s["wr"].float().t() + _normal(g, (E,), 0.3)
        ids = s["logits"].topk(K, dim=1).indices
        s["ids"] = ids.int()
        s["off"] = _plan(ids.reshape(-1), E)[0]
        s["gw"] = _normal(g, (T, K), 0.1)
        s["dl"] = torch.empty((T, E), device="cuda")
        s["losses"] = torch.empty((2,), device="cuda")
        s["dx"] = torch.empty((T, H), dtype=bf, device="cuda")
        s["dwr"] = torch.empty((E, H), device="cuda")
        s["db"] = torch.empty((E,), device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return (_own if own else _plain)[state["kind"]](state)


def _own_product(s):
    import mixture_experts_ffn_renorm_gb300 as m

    P, C, N, G = s["P"], s["C"], s["N"], s["G"]
    m.moe_quantize_act_fp8(s["x"], P, C, 1, None, None, 1.0, s["codes"], s["scales"])
    m.moe_grouped_gemm_fp8(s["codes"], s["scales"], s["w"], s["ws"], s["off"], s["pw"], s["dst"], P, C, N, G, s["out"])
    return s["out"]


def _own_experts(s):
    import mixture_experts_ffn_renorm_gb300 as m

    T, H, I, E, K = (s[n] for n in "THIEK")
    P = T * K
    m.moe_quantize_act_fp8(s["x"], T, H, K, s["pair_to_row"], None, 1.0, s["codes"], s["scales"])
    m.moe_grouped_gemm_gateup_silu_fp8(s["codes"], s["scales"], s["w13"], s["w13s"], s["off"], P, H, I, E, s["gu"],
                                       s["mid"], s["mids"])
    m.moe_grouped_gemm_fp8(s["mid"], s["mids"], s["w2"], s["w2s"], s["off"], s["pw"], s["sorted_pair"], P, I, H, E,
                           s["out"])
    return {"out": s["out"], "gate_up": s["gu"]}


def _own_experts_grad(s):
    import mixture_experts_ffn_renorm_gb300 as m

    T, H, I, E, K = (s[n] for n in "THIEK")
    P = T * K
    m.moe_quantize_act_fp8(s["x"], T, H, K, s["pair_to_row"], s["pw"], 1.0, s["codes"], s["scales"])
    m.moe_grouped_gemm_fp8(s["codes"], s["scales"], s["w2"], s["w2s"], s["off"], None, None, P, H, I, E, s["dact"])
    m.moe_silu_mul_backward_fp8(s["gu"], s["dact"], P, I, s["mid"], s["mids"])
    m.moe_grouped_gemm_fp8(s["mid"], s["mids"], s["w13"], s["w13s"], s["off"], None, s["sorted_pair"], P, 2 * I, H, E,
                           s["out"])
    return s["out"]


def _own_combine_grad(s):
    import mixture_experts_ffn_renorm_gb300 as m

    dt = BF16 if s["bf16"] else F32
    m.moe_combine_backward(s["eo"], dt, s["pw"], s["dout"], dt, 0.7, s["T"], s["K"], s["H"], s["dw"], s["deo"], dt)
    return {"dw": s["dw"], "rows": s["deo"]}


def _own_route_grad(s):
    import mixture_experts_ffn_renorm_gb300 as m

    T, H, E, K = (s[n] for n in "THEK")
    ws = torch.empty(max(m.moe_route_backward_workspace_size(T, E), m.moe_route_logits_backward_workspace_size(T, H, E)),
                     dtype=torch.uint8, device="cuda")
    m.moe_route_backward(s["logits"], s["ids"], s["gw"], s["off"], T, E, K, s["renormalize"], s["scoring"], s["balance"],
                         s["z"], s["dl"], s["losses"], ws, ws.numel())
    m.moe_route_logits_backward(s["dl"], s["x"], s["wr"], T, H, E, s["dx"], s["dwr"], s["db"], ws, ws.numel())
    return {"dlogits": s["dl"], "losses": s["losses"], "dx": s["dx"], "dw": s["dwr"], "dbias": s["db"]}


_own = {"product": _own_product, "experts": _own_experts, "experts_grad": _own_experts_grad,
        "combine_grad": _own_combine_grad, "route_grad": _own_route_grad}


# the plain forms: binary32 arithmetic on torch's elementary operations
def _quantised(v):
    """The values that rows of E4M3 codes and their scales stand for, v f32 [R, C]."""
    R, C = v.shape
    b = torch.zeros((R, _blocks(C) * BLOCK), device=v.device)
    b[:, :C] = v
    b = b.view(R, -1, BLOCK)
    amax = b.abs().amax(2, keepdim=True)
    d = (amax / torch.full_like(amax, 448.0)).clamp_min(2.0 ** -126)  # a division by a number would multiply
    q = (b * (1.0 / d)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    return (q * d).view(R, -1)[:, :C]


def _expanded(codes, scale):
    R, C = codes.shape[1:]
    s = scale.repeat_interleave(BLOCK, 1)[:, :R].repeat_interleave(BLOCK, 2)[:, :, :C]
    return codes.view(torch.float8_e4m3fn).float() * s


def _grouped(a, w, off, cap):
    """Rows of a [P, C] in groups off [G + 1] times w [G, N, C]: f32 [P, N]. Groups are padded to `cap` rows."""
    P = a.shape[0]
    off = off.long()
    at = off[:-1, None] + torch.arange(cap, device=a.device)
    live = at < off[1:, None]
    padded = a[at.clamp_max(P - 1)] * live[:, :, None]
    y = torch.bmm(padded, w.transpose(1, 2))
    r = torch.arange(P, device=a.device)
    group = (r[:, None] >= off[None, 1:]).sum(1)
    return y[group, r - off[group]]


def _placed(y, weight, dst):
    """Row r of y to row dst[r], times that row's weight, in bf16."""
    if dst is None:
        return (y if weight is None else y * weight[:, None]).to(torch.bfloat16)
    out = torch.empty(y.shape, dtype=torch.bfloat16, device=y.device)
    dst = dst.long()
    out[dst] = (y if weight is None else y * weight[dst, None]).to(torch.bfloat16)
    return out


def _plain_product(s):
    y = _grouped(_quantised(s["x"].float()), _expanded(s["w"], s["ws"]), s["off"], s["cap"])
    return _placed(y, s["pw"], s["dst"])


def _plain_experts(s):
    I, K = s["I"], s["K"]
    row = s["sorted_pair"].long()
    a = _quantised(s["x"].float())[row // K]
    gu = _grouped(a, _expanded(s["w13"], s["w13s"]), s["off"], s["cap"]).to(torch.bfloat16)
    gate, up = gu.float().split(I, 1)
    act = gate / (1.0 + torch.exp(-gate)) * up
    y = _grouped(_quantised(act), _expanded(s["w2"], s["w2s"]), s["off"], s["cap"])
    return {"out": _placed(y, s["pw"], s["sorted_pair"]), "gate_up": gu if s["train"] else None}


def _plain_experts_grad(s):
    I, K = s["I"], s["K"]
    row = s["sorted_pair"].long()
    dy = _quantised(s["x"].float()[row // K] * s["pw"][row, None])
    dact = _grouped(dy, _expanded(s["w2"], s["w2s"]), s["off"], s["cap"]).to(torch.bfloat16).float()
    gate, up = s["gu"].float().split(I, 1)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    dgu = torch.cat([dact * up * sig * (1.0 + gate * (1.0 - sig)), dact * gate * sig], 1)
    y = _grouped(_quantised(dgu), _expanded(s["w13"], s["w13s"]), s["off"], s["cap"])
    return _placed(y, None, s["sorted_pair"])


def _plain_combine_grad(s):
    d = s["dout"].float()
    dw = (s["eo"].float() * d[:, None, :]).sum(2) * 0.7
    rows = (d[:, None, :] * (s["pw"] * 0.7)[:, :, None]).to(s["eo"].dtype) if s["rows"] else None
    return {"dw": dw, "rows": rows}


def _plain_route_grad(s):
    T, E, K = s["T"], s["E"], s["K"]
    l, ids, gw = s["logits"], s["ids"].long(), s["gw"]
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - top)
    total = e.sum(1, keepdim=True)
    p, lse = e / total, top + torch.log(total)
    if s["scoring"]:
        score = 1.0 / (1.0 + torch.exp(-l))
        slope = score * (1.0 - score)
        picked = score.gather(1, ids)
        if s["renormalize"]:
            S = picked.sum(1, keepdim=True)
            gs = (gw - (gw * picked / S).sum(1, keepdim=True)) / S
        else:
            gs = gw
        dl = torch.zeros_like(l).scatter_(1, ids, gs) * slope
        share, all_ = score, score.sum(1, keepdim=True)
    elif s["renormalize"]:
        picked = l.gather(1, ids)
        w = torch.exp(picked - picked.amax(1, keepdim=True))
        w = w / w.sum(1, keepdim=True)
        dl = torch.zeros_like(l).scatter_(1, ids, w * (gw - (gw * w).sum(1, keepdim=True)))
    else:
        dl = p * (torch.zeros_like(l).scatter_(1, ids, gw) - (gw * p.gather(1, ids)).sum(1, keepdim=True))
    f = (s["off"][1:] - s["off"][:-1]).float() * (E / (K * T))
    if s["scoring"]:
        q = (share * f).sum(1, keepdim=True) / all_
        dl = dl + s["balance"] / T * (f - q) / all_ * slope
    else:
        q = (p * f).sum(1, keepdim=True)
        dl = dl + s["balance"] / T * p * (f - q)
    dl = dl + (2.0 * s["z"] / T) * lse * p
    losses = torch.stack([q.sum() * (s["balance"] / T), lse.square().sum() * (s["z"] / T)])
    return {"dlogits": dl, "losses": losses, "dx": (dl @ s["wr"].float()).to(torch.bfloat16), "dw": dl.t() @ s["x"].float(),
            "dbias": dl.sum(0)}


_plain = {"product": _plain_product, "experts": _plain_experts, "experts_grad": _plain_experts_grad,
          "combine_grad": _plain_combine_grad, "route_grad": _plain_route_grad}


# ------------------------------------------------------------------ in 64 bits
def _exact_rows(v):
    """Rows as their E4M3 codes and 32-bit scales stand for them, block by block. The operator is
    defined by operations that are each rounded to 32 bits; the codes, which a tie decides, need them."""
    out = torch.empty_like(v)
    v = v.float().double()
    for c in range(0, v.shape[1], BLOCK):
        b = v[:, c:c + BLOCK]
        d = (b.abs().amax(1, keepdim=True) / 448.0).clamp_min(2.0 ** -126).float().double()
        q = (b * (1.0 / d).float().double()).float().clamp(-448.0, 448.0)
        out[:, c:c + BLOCK] = q.to(torch.float8_e4m3fn).double() * d
    return out


def _exact_product(rows, codes, scale, off):
    off = off.tolist()
    R, C = codes.shape[1:]
    out = torch.zeros((rows.shape[0], R), dtype=torch.float64, device="cuda")
    i, j = torch.arange(R, device="cuda") // BLOCK, torch.arange(C, device="cuda") // BLOCK
    for g in range(len(off) - 1):
        if off[g] < off[g + 1]:
            w = codes[g].view(torch.float8_e4m3fn).double() * scale[g].double()[i[:, None], j[None, :]]
            out[off[g]:off[g + 1]] = rows[off[g]:off[g + 1]] @ w.t()
    return out


def _exact_scatter(y, dst):
    out = torch.zeros_like(y)
    out.index_copy_(0, dst.long(), y)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    k = case["kind"]
    if k == "product":
        y = _exact_product(_exact_rows(s["x"].double()), s["w"], s["ws"], s["off"])
        return _exact_scatter(y, s["dst"]) * s["pw"].double()[:, None] if case["scatter"] else y
    if k == "experts":
        t = s["sorted_pair"].long() // case["K"]
        y = _exact_product(_exact_rows(s["x"].double())[t], s["w13"], s["w13s"], s["off"])
        n = y.to(torch.bfloat16).double()
        act = torch.nn.functional.silu(n[:, :case["I"]]) * n[:, case["I"]:]
        out = _exact_scatter(_exact_product(_exact_rows(act), s["w2"], s["w2s"], s["off"]), s["sorted_pair"])
        return {"out": out * s["pw"].double()[:, None], "gate_up": y if case["train"] else None}
    if k == "experts_grad":
        row = s["sorted_pair"].long()
        dy = _exact_rows(s["x"].double()[row // case["K"]] * s["pw"].double()[row, None])
        dact = _exact_product(dy, s["w2"], s["w2s"], s["off"]).to(torch.bfloat16).double()
        gu = s["gu"].double().requires_grad_()
        gate, up = gu.split(case["I"], 1)
        (dgu,) = torch.autograd.grad(torch.nn.functional.silu(gate) * up, gu, dact)
        return _exact_scatter(_exact_product(_exact_rows(dgu), s["w13"], s["w13s"], s["off"]), s["sorted_pair"])
    if k == "combine_grad":
        eo, w = s["eo"].double().requires_grad_(), s["pw"].double().requires_grad_()
        deo, dw = torch.autograd.grad(0.7 * torch.einsum("tkh,tk->th", eo, w), (eo, w), s["dout"].double())
        return {"dw": dw, "rows": deo if case["rows"] else None}
    T, E, K = case["T"], case["E"], case["K"]
    l = s["logits"].double().requires_grad_()
    score = torch.sigmoid(l) if case["scoring"] else torch.softmax(l, 1)
    w = score.gather(1, s["ids"].long())
    w = w / w.sum(1, keepdim=True) if case["renormalize"] else w
    f = s["off"].double().diff() * E / (K * T)
    balance = case["balance"] * (f * (score / score.sum(1, keepdim=True)).mean(0)).sum()
    z = case["z"] * torch.logsumexp(l, 1).square().mean()
    (dl,) = torch.autograd.grad((w * s["gw"].double()).sum() + balance + z, l)
    return {"dlogits": dl, "losses": torch.stack([balance.detach(), z.detach()]), "dx": dl @ s["wr"].double(),
            "dw": dl.t() @ s["x"].double(), "dbias": dl.sum(0)}
