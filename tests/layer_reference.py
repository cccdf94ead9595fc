"""The operators around the finalize by their definitions, in 64 bits on the CPU, one token or head at a time."""
from __future__ import annotations

from decimal import Decimal, getcontext

import numpy as np
import torch


def step(dtype) -> float:
    """The most a rounding to the type is off, relative to the value."""
    return torch.finfo(dtype).eps / 2


def smallest(dtype) -> float:
    """Half the spacing of the type's subnormals."""
    f = torch.finfo(dtype)
    return f.tiny * f.eps / 2


def choose(x, K, score, bias=None, G=1, Gk=1, top2=False):
    """Ids (numpy int64 [T, K], -1 for none) and scores ([T, E]) of logits x (float64 numpy [T, E])."""
    T, E = x.shape
    ids = np.full((T, K), -1, dtype=np.int64)
    scores = np.zeros((T, E))
    for t in range(T):
        can = x[t] > -np.inf  # False for NaN
        if not can.any():
            continue
        v = np.where(can, x[t], -np.inf)
        if score == "softmax":
            m = v.max()
            e = np.where(v == m, 1.0, np.exp(np.minimum(v, 1e300) - (m if np.isfinite(m) else 0.0)) if np.isfinite(m) else 0.0)
            e = np.where(can, e, 0.0)
            s = e / e.sum()
        else:
            with np.errstate(over="ignore"):
                s = np.where(can, 1.0 / (1.0 + np.exp(-v)), 0.0)
        scores[t] = s
        c = np.where(can, s + bias, -np.inf) if bias is not None else v
        c = np.where(c > -np.inf, c, -np.inf)
        if G > 1:
            by = s if top2 and bias is None else c
            group = np.full(G, -np.inf)
            for g in range(G):
                of = by[g * (E // G):(g + 1) * (E // G)]
                of = np.sort(of[c[g * (E // G):(g + 1) * (E // G)] > -np.inf])[::-1]
                if of.size:
                    group[g] = of[:2].sum() if top2 else of[0]
            kept = [g for g in np.argsort(-group, kind="stable")[:Gk] if group[g] > -np.inf]
            c = np.where(np.isin(np.arange(E) // (E // G), kept), c, -np.inf)
        order = np.argsort(-c, kind="stable")[:K]
        order = order[c[order] > -np.inf]
        ids[t, :order.size] = order
    return ids, scores


def weights(x, ids, scores, score, renorm, scale):
    """Weights [T, K] in float64; renormalised ones from logarithms, so that they hold for tiny scores."""
    T, K = ids.shape
    w = np.zeros((T, K))
    for t in range(T):
        n = int((ids[t] >= 0).sum())
        if not n:
            continue
        v = x[t, ids[t, :n]]
        if renorm:
            l = v if score == "softmax" else np.minimum(v, 0.0) - np.log1p(np.exp(-np.abs(v)))
            m = l.max()
            e = np.where(l == m, 1.0, np.exp(l - m) if np.isfinite(m) else 0.0)
            w[t, :n] = e / e.sum()
        else:
            w[t, :n] = scores[t, ids[t, :n]]
    return w * scale


def order(ids, E, align, rows):
    """perm_idx, row_route, expert_offsets, expert_counts by walking the experts and their routes."""
    T, K = ids.shape
    perm = np.full((T, K), -1, dtype=np.int32)
    route = np.full(rows, -1, dtype=np.int32)
    offsets, counts, at = np.zeros(E + 1, np.int32), np.zeros(E, np.int32), 0
    for e in range(E):
        offsets[e] = at
        t, k = np.nonzero(ids == e)  # token-major: the order of the routes
        counts[e] = t.size
        perm[t, k] = at + np.arange(t.size)
        route[at:at + t.size] = t * K + k
        at += -(-t.size // align) * align
    offsets[E] = at
    return perm, route, offsets, counts


def route_weights_torch(x, ids, score, renorm, scale):
    """The weights as a differentiable function of float64 logits; ids < 0 weigh 0."""
    taken = ids >= 0
    dead = ~taken.any(1, keepdim=True)
    y = torch.where(dead, torch.zeros_like(x), x)
    p = torch.softmax(y, 1) if score == "softmax" else torch.sigmoid(y)
    w = p.gather(1, ids.clamp(min=0)) * taken
    if renorm:
        w = w / torch.where(dead, torch.ones_like(w[:, :1]), w.sum(1, keepdim=True))
    return w * scale


def finalize(rows, perm, scale, rsf):
    """out[t] = rsf * sum_k scale * row, float64, differentiable; routes outside the rows are skipped."""
    ok = (perm >= 0) & (perm < rows.shape[0])
    picked = rows[perm.clamp(0, rows.shape[0] - 1).long()]
    picked = torch.where(ok[..., None], picked, torch.zeros_like(picked))
    return rsf * (picked * (scale * ok)[..., None]).sum(1)


def head_norm(x, w, pos, inv_freq, style, eps, rotary_scale):
    """Per-head RMSNorm and rotation, float64, differentiable: x [T, heads, D], w [D] or None, pos [T] (all live)."""
    D, rot = x.shape[2], 2 * inv_freq.numel()
    v = x / (x.pow(2).mean(2, keepdim=True) + eps).sqrt()
    if w is not None:
        v = v * w
    # the exact angle modulo 2 pi: integers times the float's exact value, in Python's big integers
    frac = [[_angle(int(p), float(f)) for f in inv_freq] for p in pos]
    a = torch.tensor(frac, dtype=torch.float64).reshape(len(pos), 1, rot // 2)
    c, s = torch.cos(a) * rotary_scale, torch.sin(a) * rotary_scale
    if style == "half":
        p, q = v[..., :rot // 2], v[..., rot // 2:rot]
        return torch.cat([p * c - q * s, q * c + p * s, v[..., rot:]], 2)
    p, q = v[..., 0:rot:2], v[..., 1:rot:2]
    return torch.cat([torch.stack([p * c - q * s, q * c + p * s], 3).flatten(2), v[..., rot:]], 2)


def _angle(p: int, f: float) -> float:
    """p * f modulo 2 pi, both taken exactly."""
    getcontext().prec = 60
    two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257")
    v = Decimal(p) * Decimal(f)  # Decimal(float) is exact
    return float(v - two_pi * (v / two_pi).to_integral_value())
