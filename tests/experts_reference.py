"""Definitions in 64 bits of the experts' products, the random cases of their tests, and how far FP32 sums may be off."""
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -126}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def order(counts, align=1, free=0):
    """Where each expert's rows start, and all rows: each expert's from a multiple of ``align`` on, ``free`` rows behind."""
    at, offsets = 0, [0]
    for n in counts:
        at += -(-n // align) * align
        offsets.append(at)
    return torch.tensor(offsets, dtype=torch.int32), at + free


def spans(offsets, counts):
    return [(e, slice(int(offsets[e]), int(offsets[e]) + int(n))) for e, n in enumerate(counts)]


def free_rows(offsets, counts, R):
    free = torch.ones(R, dtype=torch.bool)
    for _, s in spans(offsets, counts):
        free[s] = False
    return free


def silu(g):
    return torch.where(g >= 0, g / (1 + torch.exp(-g)), g * torch.exp(g) / (1 + torch.exp(g)))


def summed(a, b):
    """a @ b.T in 64 bits, and how far a sum of the products in FP32 may be from it: each of n additions in 32 bits is off by at
    most 2^-23 of the largest partial sum (tensor cores may cut where a rounding would go to the nearest)."""
    a, b = a.double(), b.double()
    return a @ b.T, max(1, a.shape[1]) * 2.0 ** -23 * (a.abs() @ b.abs().T)


def gate(g, u, dg=0.0, du=0.0):
    """silu(g) * u, and its error from those of g and u (silu's slope is at most 1.1), of the exponential (its relative
    error is at most (|g| + 4) * 2^-23 in FP32) and of three more FP32 operations."""
    s = silu(g)
    y = s * u
    off = (s.abs() + 1.1 * dg) * (u.abs() + du) - y.abs() + 2.0 ** -23 * (g.abs() + 8) * (s.abs() + 1.1 * dg) * (u.abs() + du)
    return y, off


def close(name, got, want, off, extra=0.0):
    """One rounding to got's type of a value that is at most ``off`` from ``want``."""
    got, u, tiny = got.double(), U[got.dtype], TINY[got.dtype]
    assert torch.isfinite(got).all(), f"{name} is not finite"
    allowed = off + u * (want.abs() + off) + tiny + extra
    bad = (got - want).abs() > allowed
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got - want).abs() / allowed).max()):.3g} times the bound"


def e4m3(v):
    """The nearest E4M3 values of non-negative numbers, ties to even, at most 448."""
    e = torch.floor(torch.log2(v.clamp(min=1e-300))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return torch.clamp(torch.round(v / step) * step, max=448.0)


def e2m1_codes(y):
    """Codes of the nearest E2M1 values, ties to the even code, the sign of a zero kept."""
    a = y.abs()
    table = torch.tensor(E2M1, dtype=torch.float64, device=y.device)
    up = torch.zeros_like(a, dtype=torch.long)
    for c in range(7):
        mid = (table[c] + table[c + 1]) / 2
        up += (a > mid) if c % 2 == 0 else (a >= mid)
    return (up + 8 * torch.signbit(y).long()).to(torch.uint8)


def quantize(x, scale):
    """Codes (one a byte), block scales as E4M3 values: the recipe's FP32 roundings, each of one operation in 64 bits."""
    single = lambda v: v.float().double()  # noqa: E731
    g = single(torch.as_tensor(scale, dtype=torch.float64))
    b = x.double().unflatten(-1, (-1, 16))
    sf = e4m3(single(single(b.abs().amax(-1) / 6.0) * g))
    es = torch.where(sf > 0, single(g / sf), torch.zeros((), dtype=torch.float64))
    return e2m1_codes(single(b * es[..., None])).flatten(-2), sf


def values(codes):
    """The values of codes, two a byte."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=codes.device)
    return torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)


def tile_at(rows, cols):
    """Where the scale of (row, block) lies in tiles of 128 x 4."""
    r, k = torch.arange(rows)[:, None], torch.arange(cols)
    return (r // 128 * -(-cols // 4) + k // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + k % 4
