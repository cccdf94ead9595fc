"""Timing cases of the experts' products between the dispatch and the finalize: matrix products grouped by expert with
ragged sizes and their gradients, the gradient of the gate between the two products, NVFP4 quantisation and its
inverse, and the product of NVFP4 rows with NVFP4 weights.

``listed()`` gives the fixed cases and ``draw(rng)`` one more of the same ranges; ``prepare`` makes a case's inputs
and output buffers on the GPU, ``run`` makes one pass, ``work`` counts what a pass cannot do without and ``exact``
evaluates the definition in 64 bits.  With ``own`` false, ``run`` computes the operators from elementary torch
operations; with ``own`` true it calls this package.
"""
import math

import torch

own = False

ACT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------------------

def _matmul(name, T, E, K, n_in, n_out, gated=False, save=False, act="bf16", align=1, masked=False):
    """``n_out`` values a row; with ``gated`` the weights hold 2 * n_out rows, and ``save`` keeps what the gate reads."""
    return dict(name=name, op="matmul", T=T, E=E, K=K, n_in=n_in, n_out=n_out, gated=gated, save=save, act=act,
                align=align, masked=masked)


def _matmul_grad(name, T, E, K, n_in, n_out, act="bf16", align=1, masked=False):
    return dict(name=name, op="matmul_grad", T=T, E=E, K=K, n_in=n_in, n_out=n_out, act=act, align=align, masked=masked)


def _gate_grad(name, T, E, K, F, act="bf16", masked=False):
    return dict(name=name, op="gate_grad", T=T, E=E, K=K, F=F, act=act, masked=masked)


def _quantize(name, rows, H, act="bf16", swizzled=False, masked=False):
    return dict(name=name, op="quantize", rows=rows, H=H, act=act, swizzled=swizzled, masked=masked)


def _matmul4(name, T, E, K, n_in, n_out, gated=False, act="bf16", align=1, masked=False):
    return dict(name=name, op="matmul4", T=T, E=E, K=K, n_in=n_in, n_out=n_out, gated=gated, act=act, align=align,
                masked=masked)


def listed():
    return [
        # one decode token of the 256-expert top-8 layer, hidden size 6144, first product with the gate
        _matmul("matmul token gated", 1, 256, 8, 6144, 1024, gated=True),
        # a decode batch of the same layer, second product
        _matmul("matmul decode", 64, 256, 8, 1024, 6144),
        # a small ragged training batch, odd sizes, a quarter of the routes on other ranks, the gate's inputs kept
        _matmul("matmul ragged", 333, 60, 4, 3584, 1288, gated=True, save=True, act="fp16", masked=True),
        # a long prompt, hidden size 7168, first product with the gate, each expert's rows from a multiple of 128 on
        _matmul("matmul prompt gated", 8192, 64, 6, 7168, 2048, gated=True, align=128),
        # a ragged training batch of a small layer
        _matmul_grad("matmul grad ragged", 77, 8, 2, 1000, 520, act="fp16", masked=True),
        # a training batch, hidden size 4096
        _matmul_grad("matmul grad batch", 4096, 64, 6, 4096, 4096, align=128),
        # a ragged batch of the top-16 layer
        _gate_grad("gate grad small", 65, 896, 16, 1000, act="fp16", masked=True),
        # a training batch
        _gate_grad("gate grad batch", 4096, 64, 8, 2048),
        # a decode batch, hidden size 7168, in the tiled layout of the scales
        _quantize("nvfp4 decode batch", 16, 7168, act="fp16", swizzled=True),
        # a prompt's rows in expert order, hidden size 7168, some of them padding
        _quantize("nvfp4 prompt", 32768, 7168, masked=True),
        # a decode batch, hidden size 7168, first product with the gate
        _matmul4("nvfp4 matmul decode", 16, 256, 8, 7168, 1024, gated=True),
        # a long prompt of the layer above that has 64 experts
        _matmul4("nvfp4 matmul prompt", 8192, 64, 6, 7168, 2048, gated=True, align=128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul_grad", "gate_grad", "quantize", "matmul4"])
    act = rng.choice(["bf16", "fp16"])
    masked = rng.random() < 0.4
    if op == "quantize":
        H = rng.choice([256, 2048, 4096, 7168, 16 * rng.randint(4, 448)])
        rows = _log_int(rng, 1, 32768 * 7168 // max(H, 1024))
        return _quantize("drawn", rows, H, act, swizzled=rng.random() < 0.5, masked=masked)
    E, K = rng.choice([(8, 2), (60, 4), (64, 6), (256, 8), (256, 10), (512, 22), (896, 16)])
    if op == "gate_grad":
        F = rng.choice([512, 1024, 2048, 8 * rng.randint(8, 320)])
        return _gate_grad("drawn", _log_int(rng, 1, 4096 * 8 * 2048 // (K * max(F, 512))), E, K, F, act, masked)
    align = rng.choice([1, 1, 8, 128])
    gated = rng.random() < 0.5
    if op == "matmul4":
        n_in = rng.choice([512, 1024, 2048, 4096, 7168, 64 * rng.randint(4, 112)])
        n_out = 128 * rng.randint(1, 16) if gated else 8 * rng.randint(16, 512)
    else:
        n_in = rng.choice([512, 1024, 2048, 3584, 4096, 8 * rng.randint(16, 896)])
        n_out = rng.choice([512, 1024, 2048, 8 * rng.randint(16, 512 if not gated else 256)])
    wide = n_out * (2 if gated else 1)
    while E * wide * n_in > 3 << 30:  # weights of a few GB
        E, K = E // 2, min(K, E // 2)
    flops = 4.0e11 if op == "matmul_grad" else 1.4e12
    T = _log_int(rng, 1, max(1, int(flops / (2.0 * K * wide * n_in))))
    if op == "matmul":
        return _matmul("drawn", T, E, K, n_in, n_out, gated, gated and rng.random() < 0.4, act, align, masked)
    if op == "matmul_grad":
        return _matmul_grad("drawn", T, E, K, n_in, wide, act, align, masked)
    return _matmul4("drawn", T, E, K, n_in, n_out, gated, act, align, masked)


# ------------------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------------------

def _capacity(T, K, E, align):
    """The most rows that T*K routes fill when each expert's rows are padded to a multiple of ``align``."""
    n = T * K
    return (n + min(E, n) * (align - 1)) // align * align


def _order(s, T, E, K, align, masked, g, dev):
    """The expert order of random routes, some experts chosen more often than others: where each expert's rows start,
    how many it has, and each row's route (-1: a row of no route)."""
    popular = 0.5 * torch.randn(E, generator=g, device=dev)
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=dev).clamp(1e-6, 1 - 1e-6)))
    ids = (noise + popular).topk(K, dim=1).indices.reshape(-1)
    if masked and T * K >= 4:  # a quarter of the routes belongs to other ranks
        ids[torch.randperm(T * K, generator=g, device=dev)[: T * K // 4]] = E
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=E + 1)[:E]
    padded = (counts + align - 1) // align * align
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    live = order[: int(counts.sum())]
    of = ids[live]
    at = torch.arange(live.numel(), device=dev) - (counts.cumsum(0) - counts)[of] + offsets[of]
    route = torch.full((_capacity(T, K, E, align),), -1, dtype=torch.int32, device=dev)
    route[at] = live.int()
    s["row_route"], s["offsets"], s["counts"] = route, offsets.int(), counts.int()
    s["most"] = max(1, int(counts.max()))     # rows of the busiest expert
    s["busy"] = min(E, T * K)                 # experts that can have rows at all


def _e2m1(a):
    """The codes of non-negative values: the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    up = (a > 0.25).to(torch.uint8)
    for limit, tie in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        up += (a >= limit) if tie else (a > limit)
    return up


def _nvfp4(x, g):
    """Codes [.., H/2] and block scales [.., H/16] of FP32 values, ``g`` the global scale (a tensor of one value)."""
    block = x.unflatten(-1, (-1, 16))
    sf = torch.clamp(block.abs().amax(-1) / torch.full_like(g, 6.0) * g, max=448.0).to(torch.float8_e4m3fn)
    wide = sf.float()
    y = (block * torch.where(wide > 0, g / wide, 0.0)[..., None]).flatten(-2)
    code = _e2m1(y.abs()) | (torch.signbit(y).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4), sf


def _decoded(codes, sf, table):
    """The values that codes and block scales stand for, without the global scale."""
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], dim=-1).flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * sf.float()[..., None]).flatten(-2)


def _tiled(sf, rows, cols):
    """Block scales [.., rows, cols] in tiles of 128 rows and 4 columns, zeros behind the ends: row r of a tile at
    (r % 32) * 16 + r // 32 * 4, tiles row by row."""
    up, across = -(-rows // 128), -(-cols // 4)
    b = sf.view(torch.uint8)
    b = torch.nn.functional.pad(b, (0, across * 4 - cols, 0, up * 128 - rows))
    b = b.unflatten(-1, (across, 4)).unflatten(-3, (up, 4, 32))          # [.., up, 4, 32, across, 4]
    return b.movedim(-2, -4).transpose(-3, -2).flatten(-5).contiguous()  # [.., up, across, 32, 4, 4]


def _table(dev):
    half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=dev)
    return torch.cat([half, -half])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        out = torch.empty(*shape, dtype=dtype, device=dev)
        step = max(1, (1 << 28) // max(1, out[0].numel()))
        for i in range(0, shape[0], step):
            out[i:i + step] = torch.randn(*out[i:i + step].shape, generator=g, device=dev) * std
        return out

    s = {"case": case}
    op, act = case["op"], ACT[case["act"]]
    if op == "quantize":
        rows, H = case["rows"], case["H"]
        s["x"] = normal(rows, H, dtype=act)
        s["x"][:, :: 97] *= 30.0                                    # some channels are far larger than the others
        s["scale"] = torch.tensor([448.0 * 6.0 / 200.0], device=dev)  # a calibrated range
        s["row_route"] = None
        if case["masked"]:  # rows of no route hold anything
            s["row_route"] = torch.arange(rows, dtype=torch.int32, device=dev)
            s["row_route"][torch.rand(rows, generator=g, device=dev) < 0.125] = -1
            s["x"][s["row_route"] < 0] = float("nan")
        s["table"] = _table(dev)
        s["codes"] = torch.empty(rows, H // 2, dtype=torch.uint8, device=dev)
        s["sf"] = torch.zeros(-(-rows // 128) * 128 * -(-H // 64) * 4 if case["swizzled"] else rows * (H // 16),
                              dtype=torch.uint8, device=dev)
        s["values"] = torch.empty(rows, H, dtype=act, device=dev)
        return s
    T, E, K = case["T"], case["E"], case["K"]
    _order(s, T, E, K, case.get("align", 1), case["masked"], g, dev)
    R = s["row_route"].numel()
    dead = s["row_route"] < 0
    if op == "gate_grad":
        F = case["F"]
        s["gate_up"], s["d_out"] = normal(R, 2 * F, dtype=act), normal(R, F, dtype=act)
        s["gate_up"][dead] = float("nan")
        s["d_gate_up"], s["act"] = torch.empty_like(s["gate_up"]), torch.empty_like(s["d_out"])
        return s
    n_in, n_out = case["n_in"], case["n_out"]
    wide = n_out * (2 if case.get("gated") else 1)
    if op == "matmul4":
        s["table"] = _table(dev)
        s["gx"], s["gw"] = torch.tensor([448.0 * 6.0 / 8.0], device=dev), torch.tensor([448.0 * 6.0 * n_in ** 0.5 / 8.0], device=dev)
        s["codes"], sf = _nvfp4(normal(R, n_in), s["gx"])
        s["codes"][dead] = 0x77
        s["sf"] = sf.view(torch.uint8)
        s["sf"][dead] = 0x7f                                        # not a number
        s["w_codes"] = torch.empty(E, wide, n_in // 2, dtype=torch.uint8, device=dev)
        s["w_sf"] = torch.empty(E, wide, n_in // 16, dtype=torch.uint8, device=dev)
        step = max(1, (1 << 27) // (wide * n_in))
        for e in range(0, E, step):
            c, f = _nvfp4(normal(min(step, E - e), wide, n_in, std=n_in ** -0.5), s["gw"])
            s["w_codes"][e:e + step], s["w_sf"][e:e + step] = c, f.view(torch.uint8)
        s["w_sf_tiled"] = _tiled(s["w_sf"], wide, n_in // 16)       # the weights are laid out once
        s["alpha"] = (1.0 / (s["gx"].double() * s["gw"].double())).float().expand(E).contiguous()
    else:
        s["rows"] = normal(R, n_in, dtype=act)
        s["rows"][dead] = float("nan")                              # rows of no route hold anything
        s["weight"] = normal(E, wide, n_in, std=n_in ** -0.5, dtype=act)
    if op == "matmul_grad":
        s["d_out"] = normal(R, wide, dtype=act)
        s["d_out"][dead] = float("nan")
        s["d_rows"] = torch.zeros(R, n_in, dtype=act, device=dev)
        s["d_weight"] = torch.empty_like(s["weight"])
    else:
        s["out"] = torch.zeros(R, n_out, dtype=act, device=dev)
        s["gate_up"] = torch.zeros(R, wide, dtype=act, device=dev) if case.get("save") else None
    return s


# ------------------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s, s["case"])
    return {"matmul": _plain_matmul, "matmul_grad": _plain_matmul_grad, "gate_grad": _plain_gate_grad,
            "quantize": _plain_quantize, "matmul4": _plain_matmul4}[op](s, s["case"])


def _own(op, s, c):
    import moe_finalize_residual_gb300 as mfr

    if op == "matmul":
        mfr.moe_expert_matmul(s["rows"], s["weight"], s["offsets"], s["counts"], gated=c["gated"], gate_up=s["gate_up"],
                              out=s["out"])
        return {"out": s["out"], "gate_up": s["gate_up"]}
    if op == "matmul_grad":
        d_rows, d_weight = mfr.moe_expert_matmul_backward(s["d_out"], s["rows"], s["weight"], s["offsets"], s["counts"],
                                                          d_rows=s["d_rows"], d_weight=s["d_weight"])
        return {"d_rows": d_rows, "d_weight": d_weight}
    if op == "gate_grad":
        d_gate_up, act = mfr.moe_swiglu_backward(s["d_out"], s["gate_up"], row_route=s["row_route"],
                                                 d_gate_up=s["d_gate_up"], act=s["act"])
        return {"d_gate_up": d_gate_up, "act": act}
    if op == "quantize":  # there and back: the values that the codes stand for
        layout = "swizzled_128x4" if c["swizzled"] else "row_major"
        codes, sf = mfr.nvfp4_quantize(s["x"], s["scale"], sf_layout=layout, row_route=s["row_route"], codes=s["codes"],
                                       sf=s["sf"])
        values = mfr.nvfp4_dequantize(codes, sf, s["scale"], sf_layout=layout, out=s["values"])
        return {"values": values, "sf": sf.view(torch.float8_e4m3fn)}
    return {"out": mfr.moe_expert_matmul_nvfp4(s["codes"], s["sf"], s["w_codes"], s["w_sf_tiled"], s["offsets"],
                                               s["counts"], alpha=s["alpha"], gated=c["gated"], out=s["out"])}


def _by_expert(s):
    """The experts that can have rows, busiest first; for each place of each of them its row, and whether it has one."""
    counts, experts = torch.sort(s["counts"].long(), descending=True, stable=True)
    counts, experts = counts[:s["busy"]], experts[:s["busy"]]
    place = torch.arange(s["most"], device=counts.device)
    live = place < counts[:, None]
    row = torch.where(live, s["offsets"].long()[experts][:, None] + place, 0)
    return experts, row, live


def _back(y, row, live, R):
    """Places back to rows; zeros in rows of no route."""
    out = y.new_zeros(R + 1, y.shape[2])
    out[torch.where(live, row, R).reshape(-1)] = y.reshape(-1, y.shape[2])
    return out[:R]


def _gate(y):
    gate, up = y.chunk(2, dim=-1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_matmul(s, c):
    experts, row, live = _by_expert(s)
    x = s["rows"].float()[row].where(live[..., None], 0.0)
    y = _back(torch.bmm(x, s["weight"][experts].float().transpose(1, 2)), row, live, s["rows"].shape[0])
    dt = s["rows"].dtype
    return {"out": (_gate(y) if c["gated"] else y).to(dt), "gate_up": y.to(dt) if c["save"] else None}


def _plain_matmul_grad(s, c):
    experts, row, live = _by_expert(s)
    x = s["rows"].float()[row].where(live[..., None], 0.0)
    d = s["d_out"].float()[row].where(live[..., None], 0.0)
    d_rows = _back(torch.bmm(d, s["weight"][experts].float()), row, live, s["rows"].shape[0])
    d_weight = torch.zeros_like(s["weight"])
    d_weight[experts] = torch.bmm(d.transpose(1, 2), x).to(d_weight.dtype)
    return {"d_rows": d_rows.to(s["rows"].dtype), "d_weight": d_weight}


def _plain_gate_grad(s, c):
    live = (s["row_route"] >= 0)[:, None]
    gate, up = s["gate_up"].float().chunk(2, dim=1)
    d = s["d_out"].float()
    p = 1.0 / (1.0 + torch.exp(-gate))
    both = torch.cat([d * up * p * (1.0 + gate * (1.0 - p)), d * gate * p], dim=1).where(live, 0.0)
    return {"d_gate_up": both.to(s["gate_up"].dtype), "act": (gate * p * up).where(live, 0.0).to(s["d_out"].dtype)}


def _plain_quantize(s, c):
    x = s["x"].float()
    if s["row_route"] is not None:
        x = x.where((s["row_route"] >= 0)[:, None], 0.0)
    codes, sf = _nvfp4(x, s["scale"])
    v = torch.stack([s["table"][(codes & 15).int()], s["table"][(codes >> 4).int()]], dim=-1).flatten(-2)
    v = (v.unflatten(-1, (-1, 16)) * (sf.float() / s["scale"])[..., None]).flatten(-2)
    out = _tiled(sf, *sf.shape).view(torch.float8_e4m3fn) if c["swizzled"] else sf.reshape(-1)
    return {"values": v.to(s["x"].dtype), "sf": out}


def _plain_matmul4(s, c):
    experts, row, live = _by_expert(s)
    x = _decoded(s["codes"], s["sf"].view(torch.float8_e4m3fn), s["table"])[row].where(live[..., None], 0.0)
    w = _decoded(s["w_codes"][experts], s["w_sf"][experts].view(torch.float8_e4m3fn), s["table"])
    y = torch.bmm(x, w.transpose(1, 2)) * s["alpha"][experts][:, None, None]
    y = _back(y, row, live, s["codes"].shape[0])
    return {"out": (_gate(y) if c["gated"] else y).to(s["out"].dtype)}


# ------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ------------------------------------------------------------------------------------------------------------

def work(case):
    c, op = case, case["op"]
    if op == "quantize":
        rows, H = c["rows"], c["H"]
        live = rows * 7 // 8 if c["masked"] else rows
        # read the values, write codes and scales; read those, write the values
        return {"bytes": live * H * 2 + 2 * rows * (H // 2 + H // 16) + rows * H * 2 + 4 * rows * bool(c["masked"]), "flops": 4 * live * H}
    T, E, K = c["T"], c["E"], c["K"]
    live = T * K - (T * K // 4 if c["masked"] and T * K >= 4 else 0)
    if op == "gate_grad":
        R = _capacity(T, K, E, 1)
        return {"bytes": live * c["F"] * 6 + R * c["F"] * 6 + 4 * R, "flops": live * c["F"] * 12}
    busy = min(E * (1.0 - (1.0 - live / (T * E)) ** T), live)  # experts that have rows, were all alike
    wide = c["n_out"] * (2 if c.get("gated") else 1)
    product = 2 * live * wide * c["n_in"]
    if op == "matmul":
        return {"bytes": 2 * (live * c["n_in"] + busy * wide * c["n_in"] + live * (c["n_out"] + (wide if c["save"] else 0))),
                "flops": product}
    if op == "matmul4":
        return {"bytes": (live + busy * wide) * c["n_in"] * 9 / 16 + 2 * live * c["n_out"], "flops": product}
    return {"bytes": 2 * (live * (2 * c["n_in"] + wide) + busy * wide * c["n_in"] + E * wide * c["n_in"]), "flops": 2 * product}


# ------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    w = work(case)
    if w["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    return {"matmul": _exact_matmul, "matmul_grad": _exact_matmul_grad, "gate_grad": _exact_gate_grad,
            "quantize": _exact_quantize, "matmul4": _exact_matmul4}[case["op"]](s, case)


def _spans(s):
    at, n = s["offsets"].tolist(), s["counts"].tolist()
    return [(e, slice(at[e], at[e] + n[e])) for e in range(len(n)) if n[e]]


def _silu(x):
    return torch.nn.functional.silu(x)


def _exact_matmul(s, c):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    kept = None if s["gate_up"] is None else torch.zeros(s["gate_up"].shape, dtype=torch.float64, device=out.device)
    for e, at in _spans(s):
        y = s["rows"][at].double() @ s["weight"][e].double().T
        if kept is not None:
            kept[at] = y
        out[at] = _silu(y[:, :c["n_out"]]) * y[:, c["n_out"]:] if c["gated"] else y
    return {"out": out, "gate_up": kept}


def _exact_matmul_grad(s, c):
    """By automatic differentiation of each expert's product."""
    d_rows = torch.zeros(s["rows"].shape, dtype=torch.float64, device=s["rows"].device)
    d_weight = torch.zeros(s["weight"].shape, dtype=torch.float64, device=d_rows.device)
    for e, at in _spans(s):
        x, w = s["rows"][at].double().requires_grad_(), s["weight"][e].double().requires_grad_()
        (x @ w.T).backward(s["d_out"][at].double())
        d_rows[at], d_weight[e] = x.grad, w.grad
    return {"d_rows": d_rows, "d_weight": d_weight}


def _exact_gate_grad(s, c):
    live = s["row_route"] >= 0
    x = s["gate_up"][live].double().requires_grad_()
    y = _silu(x[:, :c["F"]]) * x[:, c["F"]:]
    y.backward(s["d_out"][live].double())
    out = {"d_gate_up": torch.zeros(s["gate_up"].shape, dtype=torch.float64, device=x.device),
           "act": torch.zeros(s["d_out"].shape, dtype=torch.float64, device=x.device)}
    out["d_gate_up"][live], out["act"][live] = x.grad, y.detach()
    return out


def _nearest(v, least, most, bits, top):
    """Non-negative 64-bit values to the nearest of a binary format, ties to even: exponents from ``least`` to ``most``,
    ``bits`` bits behind the point, ``top`` the largest value."""
    e = torch.floor(torch.log2(v.clamp(min=1e-300))).clamp(least, most)
    step = torch.exp2(e - bits)
    return torch.clamp(torch.round(v / step) * step, max=top)


def _exact_quantize(s, c):
    """The recipe's three FP32 roundings, each of one operation in 64 bits; blocks of rows at a time."""
    g = s["scale"].double()

    def single(v):
        return v.float().double()

    values = torch.empty(s["x"].shape, dtype=torch.float64, device=s["x"].device)
    scales = torch.empty(c["rows"], c["H"] // 16, dtype=torch.float64, device=values.device)
    for r in range(0, c["rows"], 4096):
        x = s["x"][r:r + 4096].double()
        if s["row_route"] is not None:
            x[s["row_route"][r:r + 4096] < 0] = 0.0
        x = x.view(x.shape[0], -1, 16)
        sf = _nearest(single(single(x.abs().amax(2) / 6.0) * g), -6, 8, 3, 448.0)
        y = single(x * torch.where(sf > 0, single(g / sf), 0.0)[..., None])
        scales[r:r + 4096] = sf
        values[r:r + 4096] = (torch.sign(y) * _nearest(y.abs(), 0, 2, 1, 6.0) * sf[..., None] / g).flatten(1)
    if not c["swizzled"]:
        return {"values": values, "sf": scales.reshape(-1)}
    rows, cols = scales.shape
    tiled = torch.zeros(s["sf"].numel(), dtype=torch.float64, device=values.device)
    r, k = torch.arange(rows, device=values.device)[:, None], torch.arange(cols, device=values.device)
    tiled[(r // 128 * -(-cols // 4) + k // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + k % 4] = scales
    return {"values": values, "sf": tiled}


def _exact_matmul4(s, c):
    def value(codes, sf):
        """Sign, exponent and mantissa of each code, times its block's scale."""
        v = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).double()
        sign, v = 1.0 - 2.0 * (v >= 8), v % 8
        e, m = v // 2, v % 2
        v = sign * torch.where(e > 0, torch.exp2(e - 1) * (1.0 + m / 2), m / 2)
        return (v.unflatten(-1, (-1, 16)) * sf.view(torch.float8_e4m3fn).double()[..., None]).flatten(-2)

    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    over = s["gx"].double() * s["gw"].double()
    for e, at in _spans(s):
        y = value(s["codes"][at], s["sf"][at]) @ value(s["w_codes"][e], s["w_sf"][e]).T / over
        out[at] = _silu(y[:, :c["n_out"]]) * y[:, c["n_out"]:] if c["gated"] else y
    return {"out": out}
