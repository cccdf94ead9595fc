"""Timing cases of the operators around the MoE finalize: expert routing and its gradient, the dispatch of token
rows into expert order, the gradient of the finalize, and the per-head RMSNorm with position rotation of queries
and keys and its gradient.

``listed()`` gives the fixed cases and ``draw(rng)`` one more of the same ranges; ``prepare`` makes a case's inputs
and output buffers on the GPU, ``run`` makes one pass, ``work`` counts what a pass cannot do without and ``exact``
evaluates the definition in 64 bits.  With ``own`` false, ``run`` computes the operators from elementary torch
operations; with ``own`` true it calls this package.
"""
import math

import numpy as np
import torch

own = False

ACT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
INF = float("inf")


# ------------------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------------------

def _route(name, T, E, K, score, renorm, logits="fp32", scale="fp32", bias=False, G=1, Gk=1, top2=False, align=1,
           factor=1.0, masked=False):
    return dict(name=name, op="route", T=T, E=E, K=K, score=score, renorm=renorm, logits=logits, scale=scale,
                bias=bias, G=G, Gk=Gk, top2=top2, align=align, factor=factor, masked=masked)


def _route_grad(name, T, E, K, score, renorm, logits="fp32", scale="fp32", factor=1.0, masked=False):
    return dict(name=name, op="route_grad", T=T, E=E, K=K, score=score, renorm=renorm, logits=logits, scale=scale,
                factor=factor, masked=masked)


def _dispatch(name, T, H, K, E, act="bf16", masked=False):
    return dict(name=name, op="dispatch", T=T, H=H, K=K, E=E, act=act, masked=masked)


def _finalize_grad(name, T, H, K, E, act="bf16", scale="fp32", factor=1.0, masked=False):
    return dict(name=name, op="finalize_grad", T=T, H=H, K=K, E=E, act=act, scale=scale, factor=factor, masked=masked)


def _heads(op, name, T, Hq, Hk, D, rot, style="half", act="bf16", base=10000.0, packed=True, padded=False):
    return dict(name=name, op=op, T=T, Hq=Hq, Hk=Hk, D=D, rot=rot, style=style, act=act, base=base, packed=packed,
                padded=padded)


def listed():
    return [
        # one decode token of the 256-expert top-8 layer: latency
        _route("route decode token", 1, 256, 8, "softmax", True, scale="bf16"),
        # a long prompt of the same layer with a balance bias and expert groups, rows of an expert padded to GEMM tiles
        _route("route prompt groups", 16384, 256, 8, "sigmoid", True, bias=True, G=8, Gk=4, top2=True, align=128,
               factor=2.5),
        # a small ragged training batch of the 512-expert top-22 layer
        _route_grad("route grad ragged", 333, 512, 22, "sigmoid", True, logits="bf16", factor=2.5, masked=True),
        # a training batch of the 256-expert layer; every expert's logit gets a gradient
        _route_grad("route grad batch", 16384, 256, 8, "softmax", False),
        # a decode batch of 16 tokens, hidden size 6144
        _dispatch("dispatch decode batch", 16, 6144, 8, 256),
        # a prompt, hidden size 7168, a quarter of the routes masked (experts of other ranks)
        _dispatch("dispatch prompt masked", 4096, 7168, 8, 256, act="fp16", masked=True),
        # a small batch of the top-16 layer
        _finalize_grad("finalize grad small", 65, 3584, 16, 896, scale="fp32"),
        # a training batch, hidden size 7168, top-8, a quarter of the routes masked
        _finalize_grad("finalize grad batch", 4096, 7168, 8, 256, scale="bf16", factor=2.5, masked=True),
        # one decode token: 48 query heads of 128 are the hidden size 6144, 8 key heads
        _heads("head_norm", "head norm decode token", 1, 48, 8, 128, 128),
        # a long prompt of the same heads, read from the packed projection
        _heads("head_norm", "head norm prompt", 16384, 48, 8, 128, 128),
        # a ragged training batch of small heads, interleaved pairs, half of each head rotated, padding at the end
        _heads("head_norm_grad", "head norm grad ragged", 517, 32, 4, 64, 32, style="interleaved", act="fp16",
               padded=True),
        # a training batch of the heads above
        _heads("head_norm_grad", "head norm grad batch", 8192, 48, 8, 128, 128, base=1000000.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "dispatch", "finalize_grad", "head_norm", "head_norm_grad"])
    if op in ("route", "route_grad"):
        score = rng.choice(["softmax", "sigmoid"])
        E = rng.choice([8, 60, 64, 128, 160, 256, 384, 512, 896, rng.randint(9, 1000)])
        T = _log_int(rng, 1, min(16384, 16384 * 256 // E))
        K = rng.randint(1, min(E, 22 if E > 256 else 10))
        kw = dict(logits=rng.choice(["fp32", "fp32", "bf16", "fp16"]), scale=rng.choice(["fp32", "bf16", "fp16"]),
                  factor=rng.choice([1.0, 2.5]), masked=rng.random() < 0.25)
        if op == "route_grad":
            return _route_grad(None, T, E, K, score, rng.random() < 0.6, **kw) | {"name": "drawn"}
        G = rng.choice([g for g in (1, 1, 4, 8) if E % g == 0 and E // g >= 2] or [1])
        Gk = rng.randint(max(1, -(-K * G // E)), G) if G > 1 else 1
        return _route(None, T, E, K, score, rng.random() < 0.6, bias=rng.random() < 0.5, G=G, Gk=Gk,
                      top2=G > 1 and rng.random() < 0.5, align=rng.choice([1, 16, 128]), **kw) | {"name": "drawn"}
    if op in ("dispatch", "finalize_grad"):
        H = rng.choice([256, 2048, 3584, 4096, 6144, 7168, 8 * rng.randint(16, 896)])
        E, K = rng.choice([(8, 2), (64, 6), (256, 8), (256, 10), (512, 22), (896, 16)])
        T = _log_int(rng, 1, max(1, 4096 * 8 * 7168 // (K * H)))
        kw = dict(act=rng.choice(["bf16", "fp16"]), masked=rng.random() < 0.5)
        if op == "dispatch":
            return _dispatch(None, T, H, K, E, **kw) | {"name": "drawn"}
        return _finalize_grad(None, T, H, K, E, scale=rng.choice(["fp32", "bf16", "fp16"]),
                              factor=rng.choice([1.0, 2.5]), **kw) | {"name": "drawn"}
    D = rng.choice([64, 80, 96, 128, 128, 192, 256])
    Hk = rng.choice([1, 2, 4, 8, 5])
    Hq = Hk * rng.choice([1, 4, 6, 8])
    T = _log_int(rng, 1, (16384 if op == "head_norm" else 8192) * 56 * 128 // ((Hq + Hk) * D))
    rot = rng.choice([D, D, D // 32 * 16])
    return _heads(op, None, T, Hq, Hk, D, rot, style=rng.choice(["half", "interleaved"]),
                  act=rng.choice(["bf16", "fp16"]), base=rng.choice([10000.0, 1000000.0]),
                  packed=rng.random() < 0.7, padded=rng.random() < 0.3) | {"name": "drawn"}


# ------------------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------------------

def _capacity(T, K, E, align):
    """The most rows that T*K routes fill when each expert's rows are padded to a multiple of ``align``."""
    n = T * K
    return (n + min(E, n) * (align - 1)) // align * align


def _random_routes(T, K, E, masked, g, dev):
    """Distinct random experts for each token, their expert-sorted row numbers and the rows' routes; with ``masked``
    a quarter of the routes is -1 and their rows belong to no route."""
    ids = torch.rand(T, E, generator=g, device=dev).topk(K, dim=1).indices
    order = torch.sort(ids.reshape(-1), stable=True).indices
    perm = torch.empty_like(order)
    perm[order] = torch.arange(T * K, device=dev)
    row_route = order.clone()
    if masked and T * K >= 4:
        off = torch.randperm(T * K, generator=g, device=dev)[: T * K // 4]
        row_route[perm[off]] = -1
        perm[off] = -1
    return perm.view(T, K).int(), row_route.int()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    s = {"case": case}
    op, T = case["op"], case["T"]
    if op in ("route", "route_grad"):
        E, K = case["E"], case["K"]
        logits = normal(T, E, dtype=ACT[case["logits"]])
        if case["masked"]:  # experts that a token cannot take, and a token in the middle that can take none
            logits[torch.rand(T, E, generator=g, device=dev) < 0.25] = -INF
            logits[T // 2] = -INF
        s["logits"] = logits
        if op == "route":
            rows = _capacity(T, K, E, case["align"])
            s["bias"] = normal(E, std=0.05) if case["bias"] else None
            s["expert_ids"] = torch.empty(T, K, dtype=torch.int32, device=dev)
            s["expert_scale"] = torch.empty(T, K, dtype=ACT[case["scale"]], device=dev)
            s["perm_idx"] = torch.empty(T, K, dtype=torch.int32, device=dev)
            s["row_route"] = torch.empty(rows, dtype=torch.int32, device=dev)
            s["expert_offsets"] = torch.empty(E + 1, dtype=torch.int32, device=dev)
            s["expert_counts"] = torch.empty(E, dtype=torch.int32, device=dev)
        else:
            top = logits.float().topk(K, dim=1)
            s["expert_ids"] = torch.where(top.values > -INF, top.indices, -1).int()
            s["d_scale"] = normal(T, K, dtype=ACT[case["scale"]])
            s["d_logits"] = torch.empty_like(logits)
    elif op in ("dispatch", "finalize_grad"):
        H, K, act = case["H"], case["K"], ACT[case["act"]]
        s["perm_idx"], s["row_route"] = _random_routes(T, K, case["E"], case["masked"], g, dev)
        if op == "dispatch":
            s["x"] = normal(T, H, dtype=act)
            s["rows"] = torch.empty(T * K, H, dtype=act, device=dev)
        else:
            s["gemm2"] = normal(T * K, H, std=0.05, dtype=act)
            s["gemm2"][s["row_route"] < 0] = float("nan")  # rows of no route hold anything
            w = torch.rand(T, K, generator=g, device=dev) + 0.1
            s["scale"] = (w / w.sum(1, keepdim=True)).to(ACT[case["scale"]])
            s["d_out"] = normal(T, H, dtype=act)
            s["d_gemm2"] = torch.empty(T * K, H, dtype=act, device=dev)
            s["d_scale"] = torch.empty(T, K, dtype=ACT[case["scale"]], device=dev)
    else:
        Hq, Hk, D, act = case["Hq"], case["Hk"], case["D"], ACT[case["act"]]

        def pair(fill):
            if case["packed"]:  # the packed projection's output: queries, keys, values
                t = fill(T, (Hq + 2 * Hk) * D)
                return t[:, :Hq * D].view(T, Hq, D), t[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
            return fill(T, Hq, D), fill(T, Hk, D)

        s["q"], s["k"] = pair(lambda *n: normal(*n, dtype=act))
        s["wq"], s["wk"] = (normal(D, std=0.1) + 1.0).to(act), (normal(D, std=0.1) + 1.0).to(act)
        start = int(torch.randint(0, 100000, (1,), generator=g, device=dev))
        s["positions"] = torch.arange(start, start + T, device=dev, dtype=torch.int32)
        if case["padded"]:
            s["positions"][T - T // 8:] = -1
        s["inv_freq"] = (1.0 / case["base"] ** (torch.arange(0, case["rot"], 2, device=dev).double() / case["rot"])).float()
        s["q_out"], s["k_out"] = pair(lambda *n: torch.zeros(*n, dtype=act, device=dev))
        if op == "head_norm_grad":
            s["d_q_out"], s["d_k_out"] = pair(lambda *n: normal(*n, dtype=act))
            s["d_wq"], s["d_wk"] = (torch.empty(D, dtype=torch.float32, device=dev) for _ in range(2))
    return s


# ------------------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s, s["case"])
    return {"route": _plain_route, "route_grad": _plain_route_grad, "dispatch": _plain_dispatch,
            "finalize_grad": _plain_finalize_grad, "head_norm": _plain_head_norm,
            "head_norm_grad": _plain_head_norm_grad}[op](s, s["case"])


def _own(op, s, c):
    import moe_finalize_residual_gb300 as mfr

    if op == "route":
        out = mfr.Routing(s["expert_ids"], s["expert_scale"], s["perm_idx"], s["row_route"], s["expert_offsets"],
                          s["expert_counts"])
        mfr.moe_route(s["logits"], c["K"], score=c["score"], bias=s["bias"], num_groups=c["G"], topk_groups=c["Gk"],
                      group_score="top2" if c["top2"] else "max", renormalize=c["renorm"], scale=c["factor"],
                      row_align=c["align"], out=out)
        return {"expert_ids": out.expert_ids, "expert_scale": out.expert_scale, "perm_idx": out.perm_idx,
                "row_route": out.row_route, "expert_offsets": out.expert_offsets, "expert_counts": out.expert_counts}
    if op == "route_grad":
        return {"d_logits": mfr.moe_route_backward(s["d_scale"], s["logits"], s["expert_ids"], score=c["score"],
                                                   renormalize=c["renorm"], scale=c["factor"], out=s["d_logits"])}
    if op == "dispatch":
        return {"rows": mfr.moe_dispatch(s["x"], s["perm_idx"], row_route=s["row_route"], out=s["rows"])}
    if op == "finalize_grad":
        part = mfr.Partial(s["gemm2"], s["perm_idx"], s["scale"])
        d_gemm2, d_scale = mfr.moe_finalize_routed_backward(s["d_out"], part, routed_scaling_factor=c["factor"],
                                                            row_route=s["row_route"], d_gemm2=s["d_gemm2"],
                                                            d_scale=s["d_scale"])
        return {"d_gemm2": d_gemm2, "d_scale": d_scale}
    if op == "head_norm":
        q, k = mfr.head_norm_rotary(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"], style=c["style"],
                                    q_out=s["q_out"], k_out=s["k_out"])
        return {"q": q, "k": k}
    d_q, d_k, d_wq, d_wk = mfr.head_norm_rotary_backward(
        s["d_q_out"], s["d_k_out"], s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"], style=c["style"],
        d_q=s["q_out"], d_k=s["k_out"], d_q_weight=s["d_wq"], d_k_weight=s["d_wk"])
    return {"d_q": d_q, "d_k": d_k, "d_wq": d_wq, "d_wk": d_wk}


def _plain_route(s, c):
    """Scores in 64 bits: which expert comes first must not depend on how a score near another's was rounded."""
    T, E, K, G = c["T"], c["E"], c["K"], c["G"]
    x = s["logits"].double()
    dev = x.device
    can = x > -INF
    top = x.amax(1, keepdim=True).clamp(min=-1e308)
    if c["score"] == "softmax":
        e = torch.exp(x - top) * can
        score = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    choice = score + s["bias"].double() if s["bias"] is not None else x  # without a bias the score orders as the logit
    choice = torch.where(can, choice, -INF)
    if G > 1:
        of_group = (score if c["top2"] and s["bias"] is None else choice).where(can, -INF).view(T, G, E // G)
        if c["top2"]:
            two = of_group.topk(2, dim=2).values
            group = torch.where(two[..., 0] > -INF, two[..., 0] + two[..., 1].where(two[..., 1] > -INF, 0.0), -INF)
        else:
            group = of_group.amax(2)
        rank = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :c["Gk"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=dev).scatter_(1, rank, True)
        choice = torch.where(kept.repeat_interleave(E // G, dim=1), choice, -INF)
    values, ids = (v[:, :K] for v in torch.sort(choice, dim=1, descending=True, stable=True))
    taken = values > -INF
    if c["renorm"] and c["score"] == "softmax":
        xk = x.gather(1, ids).where(taken, -INF)
        w = torch.exp(xk - xk.amax(1, keepdim=True).clamp(min=-1e308))
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        w = score.gather(1, ids) * taken
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    w = (w * c["factor"]).to(s["expert_scale"].dtype)
    ids = torch.where(taken, ids, -1)
    # rows in expert order, each expert's rows from a multiple of the alignment on
    flat = torch.where(taken, ids, E).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = (flat[:, None] == torch.arange(E + 1, device=dev)).sum(0) if T * K * E < 1 << 24 else \
        torch.zeros(E + 1, dtype=torch.long, device=dev).index_add_(0, flat, torch.ones_like(flat))
    first = counts.cumsum(0) - counts
    padded = (counts[:E] + c["align"] - 1) // c["align"] * c["align"]
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    at = torch.arange(T * K, device=dev) - first[flat[order]] + offsets[flat[order].clamp(max=E - 1)]
    at = torch.where(flat[order] < E, at, -1)
    perm = torch.empty_like(at)
    perm[order] = at
    rows = s["row_route"].numel()
    route = torch.full((rows + 1,), -1, dtype=torch.long, device=dev)
    route[torch.where(at >= 0, at, rows)] = order
    return {"expert_ids": ids.int(), "expert_scale": w, "perm_idx": perm.view(T, K).int(),
            "row_route": route[:rows].int(), "expert_offsets": offsets.int(), "expert_counts": counts[:E].int()}


def _plain_route_grad(s, c):
    x = s["logits"].float()
    ids = s["expert_ids"].long()
    taken = ids >= 0
    dw = s["d_scale"].float() * c["factor"] * taken
    xk = x.gather(1, ids.clamp(min=0)).where(taken, -INF)
    if c["score"] == "softmax":
        over = xk if c["renorm"] else x
        top = over.amax(1, keepdim=True).clamp(min=-3e38)
        total = torch.exp(over - top).sum(1, keepdim=True).clamp(min=1e-30)
        p = torch.exp(xk - top) / total
        inner = (dw * p).sum(1, keepdim=True)
        if c["renorm"]:
            grad = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), p * (dw - inner) * taken)
        else:
            grad = -torch.exp(x - top) / total * inner
            grad = grad.scatter_add_(1, ids.clamp(min=0), p * dw)
    else:
        sk = 1.0 / (1.0 + torch.exp(-xk))
        if c["renorm"]:
            p = sk / sk.sum(1, keepdim=True).clamp(min=1e-30)
            dk = p * (1.0 - sk) * (dw - (dw * p).sum(1, keepdim=True))
        else:
            dk = sk * (1.0 - sk) * dw
        grad = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), dk * taken)
    return {"d_logits": grad.to(s["logits"].dtype)}


def _plain_dispatch(s, c):
    route = s["row_route"].long()
    rows = s["x"][route.clamp(min=0) // c["K"]]
    return {"rows": torch.where((route >= 0)[:, None], rows, torch.zeros_like(rows))}


def _plain_finalize_grad(s, c):
    perm = s["perm_idx"].long()
    taken = perm >= 0
    d_out = s["d_out"].float()
    rows = s["gemm2"][perm.clamp(min=0)].float().where(taken[..., None], 0.0)
    d_scale = (rows * d_out[:, None, :]).sum(2) * c["factor"]
    route = s["row_route"].long()
    weight = (s["scale"].float() * c["factor"]).reshape(-1)[route.clamp(min=0)] * (route >= 0)
    d_gemm2 = d_out[route.clamp(min=0) // c["K"]] * weight[:, None]
    return {"d_gemm2": d_gemm2.to(s["gemm2"].dtype), "d_scale": d_scale.to(s["scale"].dtype)}


def _cos_sin(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()  # 64 bits: far positions
    return torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]


def _rotate(v, cos, sin, c):
    """Rotate the pairs of the first ``rot`` elements of each head; the rest passes."""
    rot = c["rot"]
    if c["style"] == "half":
        a, b, rest = v[..., :rot // 2], v[..., rot // 2:rot], v[..., rot:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], dim=2)
    a, b, rest = v[..., 0:rot:2], v[..., 1:rot:2], v[..., rot:]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], dim=3).flatten(2), rest], dim=2)


def _plain_head_norm(s, c):
    cos, sin = _cos_sin(s)
    live = (s["positions"] >= 0)[:, None, None]
    out = {}
    for n in ("q", "k"):
        x = s[n].float()
        v = x * torch.rsqrt((x * x).mean(2, keepdim=True) + 1e-6) * s["w" + n].float()
        out[n] = torch.where(live, _rotate(v, cos, sin, c).to(s[n].dtype), s[n + "_out"])
    return out


def _plain_head_norm_grad(s, c):
    cos, sin = _cos_sin(s)
    live = (s["positions"] >= 0)[:, None, None]
    out = {}
    for n in ("q", "k"):
        x, w = s[n].float(), s["w" + n].float()
        r = torch.rsqrt((x * x).mean(2, keepdim=True) + 1e-6)
        dv = _rotate(s["d_%s_out" % n].float(), cos, -sin, c).where(live, 0.0)  # the inverse rotation
        u = dv * w
        d = r * (u - x * (r * r) * (u * x).mean(2, keepdim=True))
        out["d_" + n] = d.to(s[n].dtype)
        out["d_w" + n] = (dv * x * r).sum((0, 1), dtype=torch.float64).float()
    return out


# ------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ------------------------------------------------------------------------------------------------------------

def work(case):
    c, op, T = case, case["op"], case["T"]
    if op in ("route", "route_grad"):
        E, K = c["E"], c["K"]
        logits, scales = T * E * SIZE[c["logits"]], T * K * SIZE[c["scale"]]
        if op == "route":
            rows = _capacity(T, K, E, c["align"])
            full = c["bias"] or c["top2"] or not (c["renorm"] and c["score"] == "softmax")
            return {"bytes": logits + (4 * E if c["bias"] else 0) + scales + 8 * T * K + 4 * rows + 4 * (2 * E + 1),
                    "flops": T * (E * (5 if full else 1) + 6 * K)}
        dense = c["score"] == "softmax" and not c["renorm"]
        read = logits if dense else T * K * SIZE[c["logits"]]
        return {"bytes": read + logits + scales + 4 * T * K, "flops": T * (E * (5 if dense else 0) + 10 * K)}
    if op in ("dispatch", "finalize_grad"):
        H, K = c["H"], c["K"]
        row = 2 * H
        live = T * K - (T * K // 4 if c["masked"] and T * K >= 4 else 0)
        if op == "dispatch":
            return {"bytes": T * row + T * K * row + 8 * T * K, "flops": T * K * H}
        return {"bytes": T * row + live * row + T * K * row + T * K * (8 + 2 * SIZE[c["scale"]]), "flops": 3 * live * H}
    heads = T * (c["Hq"] + c["Hk"])
    live = heads - (T // 8 * (c["Hq"] + c["Hk"]) if c["padded"] else 0)
    each = heads * c["D"] * 2
    if op == "head_norm":
        return {"bytes": 2 * live * c["D"] * 2 + 4 * T, "flops": live * (4 * c["D"] + 3 * c["rot"])}
    return {"bytes": 2 * live * c["D"] * 2 + each + 4 * T, "flops": live * (12 * c["D"] + 3 * c["rot"])}


# ------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return {"expert_ids": None, "expert_scale": _exact_route(s, case), "perm_idx": None, "row_route": None,
                "expert_offsets": None, "expert_counts": None}
    if op == "route_grad":
        return {"d_logits": _exact_route_grad(s, case)}
    if op == "dispatch":  # a copy: token t's row at the row of each of its routes, zeros elsewhere
        rows = torch.zeros(case["T"] * case["K"], case["H"], dtype=torch.float64, device=s["x"].device)
        t, k = torch.nonzero(s["perm_idx"] >= 0, as_tuple=True)
        rows[s["perm_idx"][t, k].long()] = s["x"].double()[t]
        return {"rows": rows}
    if op == "finalize_grad":
        return _exact_finalize_grad(s, case)
    return _exact_heads(s, case)


def _exact_route(s, c):
    """The weights, token by token, in numpy."""
    x = s["logits"].double().cpu().numpy()
    b = None if s["bias"] is None else s["bias"].double().cpu().numpy()
    T, E, K, G = c["T"], c["E"], c["K"], c["G"]
    out = np.zeros((T, K))
    for t in range(T):
        can = np.flatnonzero(x[t] > -np.inf)
        if not can.size:
            continue
        v = x[t, can]
        p = np.exp(v - v.max()) if c["score"] == "softmax" else 1.0 / (1.0 + np.exp(-v))
        p = p / p.sum() if c["score"] == "softmax" else p
        choice = v if b is None else p + b[can]
        if G > 1:
            value = p if c["top2"] and b is None else choice
            best = np.full(G, -np.inf)
            for q in range(G):
                of = np.sort(value[can // (E // G) == q])[::-1]
                if of.size:
                    best[q] = of[:2].sum() if c["top2"] else of[0]
            keep = np.argsort(-best, kind="stable")[:c["Gk"]]
            ok = np.isin(can // (E // G), keep)
            p, choice = p[ok], choice[ok]
        w = p[np.argsort(-choice, kind="stable")[:K]]
        out[t, :w.size] = (w / w.sum() if c["renorm"] else w) * c["factor"]
    return torch.from_numpy(out)


def _exact_route_grad(s, c):
    """By automatic differentiation of the weights in 64 bits."""
    ids = s["expert_ids"].long()
    taken = ids >= 0
    dead = ~taken.any(1, keepdim=True)
    x = s["logits"].double().masked_fill(dead, 0.0).requires_grad_()
    p = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
    w = p.gather(1, ids.clamp(min=0)).where(taken, 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).where(~dead, 1.0)
    (w * c["factor"] * s["d_scale"].double().where(taken, 0.0)).sum().backward()
    return x.grad.masked_fill(dead, 0.0)


def _exact_finalize_grad(s, c):
    """By automatic differentiation of out[t] = factor * sum_k scale[t, k] * row[perm[t, k]], token blocks at a time."""
    T, K = c["T"], c["K"]
    d_gemm2 = torch.zeros(s["gemm2"].shape, dtype=torch.float64, device=s["gemm2"].device)
    d_scale = torch.zeros(T, K, dtype=torch.float64, device=d_gemm2.device)
    for t0 in range(0, T, 512):
        perm = s["perm_idx"][t0:t0 + 512].long()
        t, k = torch.nonzero(perm >= 0, as_tuple=True)
        rows = s["gemm2"][perm[t, k]].double().requires_grad_()
        scale = s["scale"][t0:t0 + 512].double().requires_grad_()
        out = torch.zeros(perm.shape[0], c["H"], dtype=torch.float64, device=rows.device)
        out = out.index_add(0, t, rows * scale[t, k][:, None]) * c["factor"]
        (out * s["d_out"][t0:t0 + 512].double()).sum().backward()
        d_gemm2[perm[t, k]] = rows.grad
        d_scale[t0:t0 + 512] = scale.grad
    return {"d_gemm2": d_gemm2, "d_scale": d_scale}


def _exact_heads(s, c):
    """Pairs as complex numbers; the gradients by automatic differentiation."""
    live = s["positions"] >= 0
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle)[live][:, None, :]
    rot = c["rot"]
    out = {}
    for n in ("q", "k"):
        x = s[n].double().requires_grad_()
        w = s["w" + n].double().requires_grad_()
        v = x[live]
        v = v / (v.pow(2).mean(2, keepdim=True) + 1e-6).sqrt() * w
        if c["style"] == "half":
            z = torch.complex(v[..., :rot // 2], v[..., rot // 2:rot]) * turn
            y = torch.cat([z.real, z.imag, v[..., rot:]], 2)
        else:
            z = torch.view_as_complex(v[..., :rot].reshape(*v.shape[:2], rot // 2, 2).contiguous()) * turn
            y = torch.cat([torch.view_as_real(z).flatten(2), v[..., rot:]], 2)
        if c["op"] == "head_norm":
            out[n] = torch.zeros(s[n].shape, dtype=torch.float64, device=x.device).index_put((live,), y.detach())
        else:
            (y * s["d_%s_out" % n].double()[live]).sum().backward()
            out["d_" + n], out["d_w" + n] = x.grad, w.grad
    return out
