"""The operators around the finalize against their definitions in 64 bits, at the sizes and values where they can go
wrong, alone and together.

Tolerances count roundings: half a step of the output type (``step``) on the value, plus the FP32 arithmetic before
it, derived beside each test.  u = 2^-24 is half a step of FP32.
"""
import math

import numpy as np
import pytest
import torch

import layer_reference as ref
from layer_reference import smallest, step

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = float("inf")
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def mfr():
    import moe_finalize_residual_gb300 as m
    return m


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def within(got, want, dtype, rel=0.0, extra=0.0):
    """|got - want| at most: the FP32 error before the rounding (``rel`` of the value and ``extra``), and half a step
    of the type on the value that it rounds."""
    got, want = torch.as_tensor(got).double().cpu(), torch.as_tensor(want).double()
    before = rel * want.abs() + extra
    bound = before + step(dtype) * (want.abs() + before) + smallest(dtype)
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}: {got[bad][0]} for {want[bad][0]}"


# ------------------------------------------------------------------------------------------------------------
# Routing
# ------------------------------------------------------------------------------------------------------------

# Weights in FP32: expf is at most 1 ulp (2 u) off and its argument, a difference of logits up to 20 apart, 20 u; the
# sum of up to 64 weights or 1024 fast exponentials 3.4e-6 (derived in the kernel); log1pf and the products a few u.
W_REL = 3.4e-6 + 40 * U


def check_route(mfr, x, K, *, score, bias=None, G=1, Gk=1, top2=False, renorm=True, scale=1.0, scale_dtype=torch.float32,
                align=1, spare=0, **kw):
    T, E = x.shape
    dev = torch.device("cuda")
    xd = x.to(dev)
    bd = None if bias is None else bias.to(dev)
    out = mfr.moe_route(xd, K, score=score, bias=bd, num_groups=G, topk_groups=Gk, group_score="top2" if top2 else "max",
                        renormalize=renorm, scale=scale, scale_dtype=scale_dtype, row_align=align, **kw)
    torch.cuda.synchronize()
    x64 = x.double().numpy()
    ids, s = ref.choose(x64, K, score, None if bias is None else bias.double().numpy(), G, Gk, top2)
    got = out.expert_ids.cpu().numpy()
    assert np.array_equal(got, ids), f"ids differ in tokens {np.unique(np.nonzero(got != ids)[0])[:5]}"
    w = ref.weights(x64, ids, s, score, renorm, scale)
    within(out.expert_scale, torch.from_numpy(w), scale_dtype, rel=W_REL, extra=1e-37)
    assert (out.expert_scale.cpu()[torch.from_numpy(ids) < 0] == 0).all()
    perm, route, offsets, counts = ref.order(ids, E, align, out.row_route.numel())
    assert np.array_equal(out.perm_idx.cpu().numpy(), perm)
    assert np.array_equal(out.row_route.cpu().numpy(), route)
    assert np.array_equal(out.expert_offsets.cpu().numpy(), offsets)
    assert np.array_equal(out.expert_counts.cpu().numpy(), counts)
    return out


ROUTES = [  # T, E, K, score, renorm, logits, biased, G, Gk, top2, align
    (1, 1, 1, "softmax", True, "fp32", False, 1, 1, False, 1),
    (1, 256, 8, "softmax", True, "fp32", False, 1, 1, False, 1),
    (4, 8, 2, "softmax", True, "bf16", False, 1, 1, False, 16),
    (3, 7, 7, "sigmoid", True, "fp32", True, 1, 1, False, 1),
    (63, 33, 5, "softmax", False, "fp32", False, 1, 1, False, 1),
    (64, 60, 4, "sigmoid", False, "fp16", True, 4, 2, True, 8),
    (65, 64, 6, "softmax", True, "fp32", True, 8, 3, False, 16),
    (65, 256, 8, "sigmoid", True, "fp32", True, 8, 4, True, 128),
    (129, 896, 16, "softmax", False, "bf16", False, 1, 1, False, 1),
    (152, 512, 22, "sigmoid", True, "fp32", True, 16, 5, True, 16),
    (153, 512, 22, "softmax", False, "fp32", True, 8, 8, False, 1),
    (300, 1000, 64, "softmax", True, "fp32", False, 8, 7, True, 1),
    (257, 1024, 32, "sigmoid", True, "fp16", False, 32, 4, True, 128),
    (640, 257, 33, "sigmoid", False, "fp32", True, 1, 1, False, 32),
    (1000, 160, 6, "softmax", False, "fp32", False, 8, 3, False, 1),
    (1000, 128, 1, "sigmoid", False, "bf16", True, 2, 1, True, 64),
    (2500, 96, 3, "softmax", True, "fp32", True, 3, 2, True, 1),  # groups of one lane and a third
    (20000, 16, 2, "softmax", True, "fp32", False, 1, 1, False, 8),  # more than one segment a chunk
    (40, 64, 20, "sigmoid", True, "fp32", True, 8, 1, True, 16),  # fewer experts in the kept groups than places
    (200, 512, 62, "sigmoid", True, "fp32", True, 4, 2, False, 1),  # nearly as many places as candidates are ranked
    (90, 1024, 40, "softmax", False, "bf16", True, 1, 1, False, 1),
    (30, 1024, 64, "sigmoid", True, "fp32", True, 1, 1, False, 16),  # one cluster of eight, at the largest sizes
    (61, 512, 22, "softmax", True, "fp32", False, 1, 1, False, 1),
    (128, 256, 8, "sigmoid", True, "fp32", True, 8, 4, True, 128),
    (129, 256, 8, "sigmoid", True, "fp32", True, 8, 4, True, 128),   # and the first batch of two launches
]


@pytest.mark.parametrize("T,E,K,score,renorm,logits,biased,G,Gk,top2,align", ROUTES)
@pytest.mark.parametrize("masked", [False, True])
def test_route(mfr, T, E, K, score, renorm, logits, biased, G, Gk, top2, align, masked):
    g = gen(T + E)
    x = torch.randn(T, E, generator=g).to(DT[logits])
    if masked:
        x[torch.rand(T, E, generator=g) < 0.3] = -INF
        x[torch.rand(T, E, generator=g) < 0.05] = float("nan")
        x[T // 2] = -INF
    bias = 0.1 * torch.randn(E, generator=g) if biased else None
    check_route(mfr, x, K, score=score, renorm=renorm, bias=bias, G=G, Gk=Gk, top2=top2, align=align, scale=2.5,
                scale_dtype=[torch.float32, torch.bfloat16, torch.float16][T % 3])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("G,Gk,top2", [(1, 1, False), (8, 4, False), (8, 4, True)])
def test_route_ties_go_to_the_lowest_expert(mfr, score, biased, G, Gk, top2):
    g = gen(1)
    x = torch.randint(-2, 3, (70, 128), generator=g).float() * 0.5  # few distinct logits
    x[3] = 0.0
    x[4, ::2] = -0.0
    bias = torch.randint(0, 2, (128,), generator=g).float() * 0.25 if biased else None
    check_route(mfr, x, 9, score=score, bias=bias, G=G, Gk=Gk, top2=top2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K,G,top2", [(64, 8, 1, False), (256, 8, 8, True), (900, 20, 4, False)])
def test_route_scores_that_fp32_cannot_tell_apart(mfr, score, E, K, G, top2):
    """Biases that even out the scores to the last bit of FP32: only 64 bits decide."""
    x = torch.randn(80, E, generator=gen(E))
    s = ref.choose(x[:1].double().numpy(), K, score)[1][0]
    bias = torch.from_numpy(0.5 - s).float()  # token 0: every choice score within a rounding of 0.5
    x[1::2] = x[0]
    check_route(mfr, x, K, score=score, bias=bias, G=G, Gk=max(1, G // 2), top2=top2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_extreme_logits(mfr, score, renorm):
    low = torch.finfo(torch.float32).min
    x = torch.randn(12, 64, generator=gen(0))
    x[0] = low
    x[1] = -INF
    x[2] = float("nan")
    x[3, 5] = INF
    x[4, [3, 9, 40]] = INF
    x[5] = 1e30 * x[5]
    x[6, 1:] = -INF
    x[7, :60] = low
    x[8] = -90.0 + 0.01 * x[8]  # sigmoids near the smallest FP32 numbers
    x[9] = 88.0 + x[9]
    x[10] = -300.0 + x[10] if renorm else -80.0 + x[10]
    out = check_route(mfr, x, 8, score=score, renorm=renorm)
    assert out.expert_ids[6].tolist() == [0] + [-1] * 7
    bias = torch.zeros(64)
    bias[7], bias[8], bias[9] = -INF, float("nan"), INF
    out = mfr.moe_route(x.cuda(), 8, score=score, bias=bias.cuda(), renormalize=renorm)
    ids = out.expert_ids.cpu()
    assert not ((ids == 7) | (ids == 8)).any()
    assert (ids[[3, 4, 5, 8, 9, 11], 0] == 9).all()


def test_route_strided_and_offset_logits(mfr):
    wide = torch.randn(40, 300, generator=gen(2)).cuda()
    for lo, E in ((0, 256), (1, 256), (3, 61), (44, 256)):
        a = mfr.moe_route(wide[:, lo:lo + E], 6)
        b = mfr.moe_route(wide[:, lo:lo + E].contiguous(), 6)
        assert torch.equal(a.expert_ids, b.expert_ids) and torch.equal(a.expert_scale, b.expert_scale)
        h = wide.half()
        a, b = mfr.moe_route(h[:, lo:lo + E], 6), mfr.moe_route(h[:, lo:lo + E].contiguous(), 6)
        assert torch.equal(a.expert_ids, b.expert_ids) and torch.equal(a.expert_scale, b.expert_scale)


@pytest.mark.parametrize("T", [5, 500])
def test_route_outputs_stay_in_their_buffers(mfr, T):
    """Canaries behind every output, spare rows behind the last one, and a call without the order."""
    x = torch.randn(T, 40, generator=gen(T)).cuda()
    rows = mfr.moe_route_max_rows(T, 4, 40, 16) + 37

    def guarded(n, dtype):
        t = torch.full((n + 64,), 77, dtype=dtype, device="cuda")
        return t, t[:n]

    bufs = [guarded(n, d) for n, d in ((T * 4, torch.int32), (T * 4, torch.float32), (T * 4, torch.int32), (rows, torch.int32),
                                       (41, torch.int32), (40, torch.int32))]
    v = [b[1] for b in bufs]
    out = mfr.Routing(v[0].view(T, 4), v[1].view(T, 4), v[2].view(T, 4), v[3], v[4], v[5])
    check = mfr.moe_route(x, 4, row_align=16)
    mfr.moe_route(x, 4, row_align=16, out=out)
    plain = mfr.moe_route(x, 4, order=False)
    torch.cuda.synchronize()
    assert all((b[0][b[1].numel():] == 77).all() for b in bufs)
    assert torch.equal(out.perm_idx, check.perm_idx) and (out.row_route[-37:] == -1).all()
    assert torch.equal(out.row_route[:-37], check.row_route)
    assert plain.perm_idx is None and torch.equal(plain.expert_ids, out.expert_ids)


def test_route_empty_batch(mfr):
    out = mfr.moe_route(torch.empty(0, 16, device="cuda"), 2, row_align=4)
    assert out.expert_ids.shape == (0, 2) and (out.expert_offsets == 0).all() and (out.expert_counts == 0).all()
    buf = mfr.Routing(out.expert_ids, out.expert_scale, out.perm_idx, torch.full((9,), 5, dtype=torch.int32, device="cuda"),
                      torch.full((17,), 5, dtype=torch.int32, device="cuda"), torch.full((16,), 5, dtype=torch.int32, device="cuda"))
    mfr.moe_route(torch.empty(0, 16, device="cuda"), 2, out=buf)
    assert (buf.row_route == -1).all() and (buf.expert_offsets == 0).all() and (buf.expert_counts == 0).all()


def _grad_case(T, E, K, logits, seed, masked):
    g = gen(seed)
    x = torch.randn(T, E, generator=g).to(DT[logits])
    if masked:
        x[torch.rand(T, E, generator=g) < 0.3] = -INF
        x[T // 2] = -INF
    ids, _ = ref.choose(x.double().numpy(), K, "softmax")
    return x, torch.from_numpy(ids), torch.randn(T, K, generator=g)


@pytest.mark.parametrize("T,E,K,logits,dw", [(1, 1, 1, "fp32", "fp32"), (3, 7, 7, "fp32", "bf16"), (130, 256, 8, "fp32", "fp32"),
                                             (33, 512, 22, "bf16", "fp32"), (17, 1000, 64, "fp16", "fp16"),
                                             (2000, 60, 4, "bf16", "bf16")])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_route_backward(mfr, T, E, K, logits, dw, score, renorm, masked):
    x, ids, d = _grad_case(T, E, K, logits, T + E, masked)
    d = d.to(DT[dw])
    got = mfr.moe_route_backward(torch.where(ids >= 0, d, float("nan")).to(DT[dw]).cuda(), x.cuda(), ids.int().cuda(), score=score,
                                 renormalize=renorm, scale=2.5)
    x64 = x.double().requires_grad_()
    w = ref.route_weights_torch(x64, ids, score, renorm, 2.5)
    d64 = torch.where(ids >= 0, d.double(), 0.0)
    (w * d64).sum().backward()
    want = torch.nan_to_num(x64.grad)
    # p (d - sum d p): the weights' relative error, on the terms before the difference, and a few roundings of each;
    # the FP32 softmax's sum over E <= 1000 in lanes: (32 + 5) u more
    mag = 2.5 * d64.abs().amax(1, keepdim=True).expand_as(want)
    within(got, want, DT[logits], extra=mag * (W_REL + 50 * U))
    assert not torch.isnan(got).any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_against_differences(mfr, score, renorm):
    x, ids, d = _grad_case(6, 20, 4, "fp32", 3, False)
    got = mfr.moe_route_backward(d.cuda(), x.cuda(), ids.int().cuda(), score=score, renormalize=renorm).double().cpu()
    h = 1e-5
    f = lambda y: (ref.route_weights_torch(y, ids, score, renorm, 1.0) * d.double()).sum(1)  # noqa: E731
    for e in range(20):
        y = x.double().clone()
        y[:, e] += h
        z = x.double().clone()
        z[:, e] -= h
        want = (f(y) - f(z)) / (2 * h)  # third derivatives of a softmax are below 1: h^2 / 6, and rounding 1e-15 / h
        assert ((got[:, e] - want).abs() <= d.abs().amax() * (W_REL + 50 * U) + 1e-9).all()


def test_route_backward_repeated_and_foreign_ids(mfr):
    """An expert named twice gets both places' gradients; ids outside the experts are skipped."""
    x = torch.randn(3, 16, generator=gen(5))
    ids = torch.tensor([[2, 2, 5], [1, -1, 16], [-7, 99, 2 ** 31 - 1]])
    d = torch.randn(3, 3, generator=gen(6))
    got = mfr.moe_route_backward(d.cuda(), x.cuda(), ids.int().cuda(), score="sigmoid", renormalize=False).double().cpu()
    s = torch.sigmoid(x.double())
    want = torch.zeros(3, 16, dtype=torch.float64)
    want[0, 2], want[0, 5], want[1, 1] = d[0, 0].double() + d[0, 1].double(), d[0, 2].double(), d[1, 0].double()
    within(got, want * s * (1 - s), torch.float32, rel=20 * U)


def test_route_backward_strided(mfr):
    x, ids, d = _grad_case(40, 64, 6, "fp32", 9, False)
    wide_x, wide_o = torch.zeros(40, 100).cuda(), torch.full((40, 90), 7.0).cuda()
    wide_x[:, 3:67] = x.cuda()
    out = mfr.moe_route_backward(d.cuda(), wide_x[:, 3:67], ids.int().cuda(), renormalize=False, out=wide_o[:, 5:69])
    want = mfr.moe_route_backward(d.cuda(), x.cuda(), ids.int().cuda(), renormalize=False)
    assert torch.equal(out, want) and (wide_o[:, :5] == 7).all() and (wide_o[:, 69:] == 7).all()


# ------------------------------------------------------------------------------------------------------------
# Dispatch and the finalize's gradient
# ------------------------------------------------------------------------------------------------------------

def routes(T, K, spare, seed, masked=True):
    """A permutation of rows with ``spare`` rows of no route, a quarter of the routes masked, and its inverse."""
    g = gen(seed)
    n = T * K + spare
    perm = torch.randperm(n, generator=g)[:T * K].int()
    route = torch.full((n,), -1, dtype=torch.int32)
    route[perm.long()] = torch.arange(T * K, dtype=torch.int32)
    if masked and T * K >= 4:
        off = torch.randperm(T * K, generator=g)[:T * K // 4]
        route[perm[off].long()] = -1
        perm[off] = torch.tensor([-1, -5, n, 2 ** 31 - 1], dtype=torch.int32)[torch.arange(off.numel()) % 4]
    return perm.view(T, K), route


@pytest.mark.parametrize("T,K,n,dtype", [(1, 1, 8, torch.bfloat16), (1, 8, 6144, torch.bfloat16), (3, 2, 16, torch.uint8),
                                         (16, 8, 6144, torch.bfloat16), (7, 64, 264, torch.float16), (65, 6, 520, torch.float32),
                                         (700, 8, 2048, torch.bfloat16), (300, 10, 448, torch.uint8), (2, 3, 32768, torch.float32)])
@pytest.mark.parametrize("zeros", [False, True])
def test_dispatch(mfr, T, K, n, dtype, zeros):
    perm, route = routes(T, K, 13, T + n)
    x = torch.randint(0, 255, (T, n), generator=gen(n), dtype=torch.uint8).to(dtype)
    rows = route.numel()
    buf = torch.full((rows + 2, n), 99, dtype=torch.uint8).to(dtype).cuda()
    out = mfr.moe_dispatch(x.cuda(), perm.cuda(), row_route=route.cuda() if zeros else None, out=buf[1:-1])
    want = torch.full((rows, n), 0 if zeros else 99, dtype=torch.uint8).to(dtype)
    live = route >= 0
    want[live] = x[(route[live] // K).long()]
    assert torch.equal(out.cpu(), want)
    assert (buf[0] == 99).all() and (buf[-1] == 99).all()
    made = mfr.moe_dispatch(x.cuda(), perm.cuda(), rows, row_route=route.cuda() if zeros else None).cpu()
    want[~live] = 0
    assert torch.equal(made, want)


def test_dispatch_without_tokens_or_rows(mfr):
    e = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    out = mfr.moe_dispatch(torch.empty(0, 64, device="cuda"), e, row_route=torch.full((5,), -1, dtype=torch.int32, device="cuda"),
                           out=torch.ones(5, 64, device="cuda"))
    assert (out == 0).all()
    assert mfr.moe_dispatch(torch.ones(3, 64, device="cuda"), torch.zeros(3, 2, dtype=torch.int32, device="cuda"), 0).shape == (0, 64)


def _finalize_case(T, K, H, act, sdt, seed, masked=True):
    perm, route = routes(T, K, 5, seed, masked)
    g = gen(seed + 1)
    rows = (0.3 * torch.randn(route.numel(), H, generator=g)).to(act)
    rows[route < 0] = float("nan")
    scale = None if sdt is None else torch.rand(T, K, generator=g).to(sdt)
    d = torch.randn(T, H, generator=g).to(act)
    return perm, route, rows, scale, d


@pytest.mark.parametrize("T,K,H", [(1, 1, 8), (1, 8, 6144), (3, 64, 264), (65, 16, 3584), (40, 22, 2048), (700, 8, 520), (400, 3, 7168),
                                   (2, 5, 32768)])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sdt", [None, torch.float32, torch.bfloat16, torch.float16])
def test_routed_backward(mfr, T, K, H, act, sdt):
    perm, route, rows, scale, d = _finalize_case(T, K, H, act, sdt, T + H)
    part = mfr.Partial(rows.cuda(), perm.cuda(), None if scale is None else scale.cuda())
    d_rows, d_scale = mfr.moe_finalize_routed_backward(d.cuda(), part, routed_scaling_factor=2.5, row_route=route.cuda())
    r64 = rows.double().requires_grad_()
    s64 = (torch.ones(T, K) if scale is None else scale).double().requires_grad_()
    (ref.finalize(r64, perm, s64, 2.5) * d.double()).sum().backward()
    want = torch.where((route >= 0)[:, None], torch.nan_to_num(r64.grad), 0.0)
    within(d_rows, want, act, rel=2.1 * U)  # (scale rsf) d: two roundings, then the output's
    ok = (perm >= 0) & (perm < rows.shape[0])
    picked = torch.where(ok[..., None], rows[perm.clamp(0, rows.shape[0] - 1).long()].double(), 0.0)
    terms = (picked * d.double()[:, None]).abs().sum(2) * 2.5
    # a thread's chain of ceil(H / 2048) * 8 fused steps, a butterfly of 5 and 8 warps, and the factor
    within(d_scale, s64.grad, d_scale.dtype, extra=terms * (-(-H // 2048) * 8 + 14) * U)
    assert d_scale.dtype == (sdt or torch.float32) and (d_scale.cpu()[~ok] == 0).all()


def test_routed_backward_one_output_and_untouched_rows(mfr):
    perm, route, rows, scale, d = _finalize_case(50, 4, 256, torch.bfloat16, torch.float32, 3)
    part = mfr.Partial(rows.cuda(), perm.cuda(), scale.cuda())
    both = mfr.moe_finalize_routed_backward(d.cuda(), part, row_route=route.cuda())
    only = mfr.moe_finalize_routed_backward(d.cuda(), part, row_route=route.cuda(), want_d_scale=False)
    assert only[1] is None and torch.equal(only[0], both[0])
    only = mfr.moe_finalize_routed_backward(d.cuda(), part, want_d_gemm2=False)
    assert only[0] is None and torch.equal(only[1], both[1])
    buf = torch.full((route.numel() + 2, 256), 9.0, dtype=torch.bfloat16, device="cuda")
    left = mfr.moe_finalize_routed_backward(d.cuda(), part, d_gemm2=buf[1:-1])[0]
    live = (route >= 0).cuda()
    assert torch.equal(left[live], both[0][live]) and (left[~live] == 9).all() and (buf[[0, -1]] == 9).all()
    assert (both[0][~live] == 0).all()
    made = mfr.moe_finalize_routed_backward(d.cuda(), part)[0]
    assert torch.equal(made, both[0])


def test_routed_backward_against_differences(mfr):
    """The scales' gradient from the library's own forward call at two scales (exact in the products: the rows are
    small whole numbers and the scales multiples of 1/8)."""
    T, K, H = 5, 3, 64
    perm, route = routes(T, K, 2, 8, masked=False)
    rows = torch.randint(-3, 4, (route.numel(), H), generator=gen(1)).half()
    d = torch.randint(-2, 3, (T, H), generator=gen(2)).half()
    scale = torch.randint(1, 8, (T, K), generator=gen(3)).float() / 8
    got = mfr.moe_finalize_routed_backward(d.cuda(), mfr.Partial(rows.cuda(), perm.cuda(), scale.cuda()))[1].cpu()
    for k in range(K):
        up, down = scale.clone(), scale.clone()
        up[:, k] += 0.125
        down[:, k] -= 0.125
        f = [mfr.moe_finalize_routed([mfr.Partial(rows.cuda(), perm.cuda(), s.cuda())]).cpu().double() for s in (up, down)]
        assert torch.equal(((f[0] - f[1]) * d.double()).sum(1) / 0.25, got[:, k].double())


def test_dispatch_gradient_is_the_finalize(mfr):
    """sum <dispatch(x), g> = sum <x, finalize(g without scales)>, exactly for small whole numbers."""
    T, K, H = 9, 4, 128
    perm, route = routes(T, K, 3, 4)
    x = torch.randint(-3, 4, (T, H), generator=gen(1)).bfloat16().cuda()
    g = torch.randint(-3, 4, (route.numel(), H), generator=gen(2)).bfloat16().cuda()
    rows = mfr.moe_dispatch(x, perm.cuda(), row_route=route.cuda())
    dx = mfr.moe_finalize_routed([mfr.Partial(g, perm.cuda())])
    assert (rows.double() * g.double()).sum() == (x.double() * dx.double()).sum()


# ------------------------------------------------------------------------------------------------------------
# Head norm and rotation
# ------------------------------------------------------------------------------------------------------------

HEADS = [  # T, Hq, Hk, D, rot, style
    (1, 1, 1, 16, 16, "half"),
    (1, 48, 8, 128, 128, "half"),
    (3, 5, 1, 64, 64, "interleaved"),
    (7, 3, 2, 80, 80, "half"),
    (5, 4, 4, 96, 32, "half"),
    (33, 6, 2, 128, 64, "half"),
    (6, 2, 1, 192, 190, "interleaved"),
    (4, 7, 3, 256, 2, "interleaved"),
    (2, 3, 1, 512, 512, "half"),
    (5, 2, 0, 64, 64, "half"),
    (5, 0, 3, 64, 16, "half"),
    (4, 3, 2, 48, 0, "half"),
    (900, 12, 3, 128, 128, "half"),
    (700, 9, 1, 32, 30, "interleaved"),
]


def _heads(T, Hq, Hk, D, rot, act, seed, packed):
    g = gen(seed)
    total = Hq + 2 * Hk + 1
    qkv = torch.randn(T, total * D, generator=g).to(act)
    q, k = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(act) for _ in range(2)]
    pos = torch.randint(0, 100000, (T,), generator=g)
    pos[0] = 0 if T > 1 else 77777
    freq = (1.0 / 10000 ** (torch.arange(0, rot, 2).double() / max(rot, 1))).float()
    return q, k, w, pos, freq


# The value before its rounding, relative to its pair's length: the mean square (two chains of 8 fused steps, their sum,
# 5 adds, a fused step) 15 u, half of it in the root, and the root itself 4 u; the element times the root u; the turn: the
# angle 1.2e-7 (2^-32 turns and a rounding of the half turn: pi 2^-25), the sine or cosine 2 u, times rotary_scale u, times
# the weight u; the products and their sum 2 u, all of it on both elements: (7.5 + 4 + 1 + 4 + 2) u = 18.5 u, and 1.2e-7.
H_REL = 22 * U + 1.2e-7


def _pair_size(v, rot, style):
    """The length of the pair that each element belongs to (its own size where it is not rotated)."""
    out = v.abs().clone()
    if style == "half":
        n = torch.hypot(v[..., :rot // 2], v[..., rot // 2:rot])
        out[..., :rot // 2] = out[..., rot // 2:rot] = n
    else:
        n = torch.hypot(v[..., 0:rot:2], v[..., 1:rot:2])
        out[..., 0:rot:2] = out[..., 1:rot:2] = n
    return out


def _on_gpu(t, packed):
    """A copy on the GPU with the same strides."""
    if not packed:
        return t.cuda()
    g = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
    return g.copy_(t)


@pytest.mark.parametrize("T,Hq,Hk,D,rot,style", HEADS)
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("packed", [False, True])
def test_head_norm(mfr, T, Hq, Hk, D, rot, style, act, packed):
    q, k, w, pos, freq = _heads(T, Hq, Hk, D, rot, act, T + D, packed)
    wide = T % 2 == 0
    scale = 1.0 if packed else 1.25
    got = mfr.head_norm_rotary(_on_gpu(q, packed), _on_gpu(k, packed), w[0].cuda(), w[1].cuda(),
                               pos.cuda() if wide else pos.int().cuda(), freq.cuda(), style=style, rotary_scale=scale)
    for x, wi, y in zip((q, k), w, got):
        v = x.double() / (x.double().pow(2).mean(2, keepdim=True) + 1e-6).sqrt() * wi.double()
        want = ref.head_norm(x.double(), wi.double(), pos.tolist(), freq, style, 1e-6, scale)
        within(y, want, act, extra=H_REL * scale * _pair_size(v, rot, style))


@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_head_norm_far_positions(mfr, style):
    """Positions up to 2^62: the angle is exact modulo a turn, whatever the position."""
    D = 64
    pos = torch.tensor([0, 1, 2 ** 24 + 1, 2 ** 31 - 1, 2 ** 33 + 5, 10 ** 15 + 7, 2 ** 62 - 3])
    freq = torch.cat([torch.tensor([1.0, 0.5, 3.25, -0.7, 0.0, 900.0, 1e-9]), torch.rand(D // 2 - 7, generator=gen(1))])
    q = torch.randn(7, 2, D, generator=gen(2)).half()
    y, _ = mfr.head_norm_rotary(q.cuda(), q.cuda(), None, None, pos.cuda(), freq.cuda(), style=style, eps=1e-5)
    v = q.double() / (q.double().pow(2).mean(2, keepdim=True) + 1e-5).sqrt()
    want = ref.head_norm(q.double(), None, pos.tolist(), freq, style, 1e-5, 1.0)
    # the held fraction of a turn is 2^-64 (1 + 900 * 2^-1) off, times the position
    far = pos.double()[:, None, None] * 2.0 ** -64 * 2 * math.pi * 500
    within(y[:5], want[:5], torch.float16, extra=(H_REL + far[:5]) * _pair_size(v, D, style)[:5])
    small = freq.abs() <= 1.0  # at 2^62 a turn is 2^-2 off: only the near ones are held to it
    near = torch.cat([small, small]) if style == "half" else small.repeat_interleave(2)
    within(y[5, :, near], want[5, :, near], torch.float16, extra=((H_REL + 1e15 * 2.0 ** -64 * 7) * _pair_size(v, D, style))[5, :, near])


def test_head_norm_small_and_large_values(mfr):
    q = torch.randn(6, 3, 64, generator=gen(4)).bfloat16()
    q[0] = 0
    q[1] *= 1e-20
    q[2] *= 1e15
    q[3, 0, 5] = INF
    q[4, 1, 7] = float("nan")
    pos, freq = torch.arange(6, dtype=torch.int32), torch.rand(32, generator=gen(5))
    y, _ = mfr.head_norm_rotary(q.cuda(), q.cuda(), None, None, pos.cuda(), freq.cuda())
    v = q.double() / (q.double().pow(2).mean(2, keepdim=True) + 1e-6).sqrt()
    want = ref.head_norm(q.double(), None, pos.tolist(), freq, "half", 1e-6, 1.0)
    fine = torch.isfinite(want).all(2)
    assert fine.sum() == 16
    within(y.cpu()[fine], want[fine], torch.bfloat16, extra=(H_REL * _pair_size(v, 64, "half"))[fine])
    assert (y.cpu()[0] == 0).all()


@pytest.mark.parametrize("Hk", [1, 4])
def test_head_norm_padding_and_in_place(mfr, Hk):
    T, Hq, D = 50, 8, 128
    q, k, w, pos, freq = _heads(T, Hq, Hk, D, D, torch.bfloat16, 7, True)
    pos[[3, 20]] = -1
    pos[44:] = -2 ** 31
    qg, kg = q.cuda().contiguous(), k.cuda().contiguous()
    qg[44:] = float("nan")
    args = (w[0].cuda(), w[1].cuda(), pos.int().cuda(), freq.cuda())
    a = mfr.head_norm_rotary(qg, kg, *args)
    pad = (pos < 0).cuda()
    assert (a[0][pad] == 0).all() and (a[1][pad] == 0).all()
    bq, bk = torch.full_like(qg, 3.0), torch.full_like(kg, 3.0)
    mfr.head_norm_rotary(qg, kg, *args, q_out=bq, k_out=bk)
    assert (bq[pad] == 3).all() and (bk[pad] == 3).all()
    assert torch.equal(bq[~pad], a[0][~pad]) and torch.equal(bk[~pad], a[1][~pad])
    q2, k2 = qg.clone(), kg.clone()
    mfr.head_norm_rotary(q2, k2, *args, q_out=q2, k_out=k2)
    assert torch.equal(q2[~pad], a[0][~pad]) and torch.equal(k2[~pad], a[1][~pad])
    assert torch.equal(q2[pad].view(torch.int16), qg[pad].view(torch.int16)) and torch.equal(k2[pad], kg[pad])


def test_head_norm_strides_and_surroundings(mfr):
    """Heads read out of and written into other layouts, with what lies between left as it was."""
    T, H, D = 11, 6, 96
    x = torch.randn(H, T, 3 * D, generator=gen(8)).half().cuda()
    q, k = x[:, :, :D].transpose(0, 1), x[:2, :, D + 8:2 * D + 8].transpose(0, 1)
    buf = torch.full((H, T, 2 * D), 5.0, dtype=torch.float16, device="cuda")
    kb = torch.full((T, 2, 2, D), 5.0, dtype=torch.float16, device="cuda")
    pos, freq = torch.arange(T, device="cuda"), torch.rand(48, generator=gen(9)).cuda()
    mfr.head_norm_rotary(q, k, None, None, pos, freq, q_out=buf[:, :, 8:D + 8].transpose(0, 1), k_out=kb[:, :, 1])
    want = mfr.head_norm_rotary(q.contiguous(), k.contiguous(), None, None, pos, freq)
    assert torch.equal(buf[:, :, 8:D + 8].transpose(0, 1), want[0]) and torch.equal(kb[:, :, 1], want[1])
    assert (buf[:, :, :8] == 5).all() and (buf[:, :, D + 8:] == 5).all() and (kb[:, :, 0] == 5).all()


def _head_grads(x, w, pos, freq, style, scale, d):
    x64 = x.double().requires_grad_()
    w64 = w.double().requires_grad_() if w is not None else None
    (ref.head_norm(x64, w64, pos, freq, style, 1e-6, scale) * d.double()).sum().backward()
    return x64.grad, None if w is None else w64.grad


@pytest.mark.parametrize("T,Hq,Hk,D,rot,style", HEADS)
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("packed", [False, True])
def test_head_norm_backward(mfr, T, Hq, Hk, D, rot, style, act, packed):
    q, k, w, pos, freq = _heads(T, Hq, Hk, D, rot, act, T + D, packed)
    g = gen(T)
    d = [torch.randn(T, h, D, generator=g).to(act) for h in (Hq, Hk)]
    scale = 1.0 if packed else 1.25
    got = mfr.head_norm_rotary_backward(d[0].cuda(), d[1].cuda(), _on_gpu(q, packed), _on_gpu(k, packed), w[0].cuda(), w[1].cuda(),
                                        pos.cuda(), freq.cuda(), style=style, rotary_scale=scale)
    for x, wi, di, dx, dw in zip((q, k), w, d, got[:2], got[2:]):
        want_x, want_w = _head_grads(x, wi, pos.tolist(), freq, style, scale, di)
        x64, w64 = x.double(), wi.double()
        r = 1 / (x64.pow(2).mean(2, keepdim=True) + 1e-6).sqrt()
        size = _pair_size(di.double(), rot, style) * max(scale, 1.0)  # of the gradient turned back
        # r (g w - x r^2 mean(g w x)): H_REL on every factor, the mean's 21 additions on the sum of its terms' sizes
        mean = (size * w64.abs() * x64.abs()).mean(2, keepdim=True)
        within(dx, want_x, act, extra=r * (H_REL * 2 * size * w64.abs() + x64.abs() * r * r * mean * (3 * H_REL + 24 * U)))
        terms = (size * x64.abs() * r).sum((0, 1))
        # each term H_REL, and sums of at most 64 items a lane, 5 + 8 + 25 in the tree above them
        within(dw, want_w, torch.float32, extra=terms * (H_REL + 102 * U))


@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_head_norm_backward_against_differences(mfr, style):
    T, H, D = 3, 2, 32
    q, k, w, pos, freq = _heads(T, H, 1, D, 16, torch.float16, 1, False)
    d = torch.randn(T, H, D, generator=gen(3)).half()
    dk = torch.zeros(T, 1, D).half()
    dx, _, dw, dkw = mfr.head_norm_rotary_backward(d.cuda(), dk.cuda(), q.cuda(), k.cuda(), w[0].cuda(), w[1].cuda(), pos.cuda(),
                                                   freq.cuda(), style=style)
    f = lambda x, wi: (ref.head_norm(x, wi, pos.tolist(), freq, style, 1e-6, 1.0) * d.double()).sum()  # noqa: E731
    h = 1e-5
    for i in range(D):
        e = torch.zeros(D, dtype=torch.float64)
        e[i] = h
        num = (f(q.double(), w[0].double() + e) - f(q.double(), w[0].double() - e)) / (2 * h)
        assert abs(num - dw[i].item()) <= 1e-5 * T * H * 10 + 1e-7  # 40 u on terms of at most 10 each
        x = torch.zeros(T, H, D, dtype=torch.float64)
        x[1, 1, i] = h
        num = (f(q.double() + x, w[0].double()) - f(q.double() - x, w[0].double())) / (2 * h)
        assert abs(num - dx[1, 1, i].item()) <= step(torch.float16) * abs(num) + 1e-4  # FP32 before it: H_REL of at most 30
    assert (dkw == 0).all()


def test_head_norm_backward_padding_in_place_and_no_weights(mfr):
    T, Hq, Hk, D = 60, 6, 2, 64
    q, k, w, pos, freq = _heads(T, Hq, Hk, D, D, torch.bfloat16, 2, False)
    pos[[0, 31]] = -5
    pos[50:] = -1
    live = pos >= 0
    g = gen(4)
    d = [torch.randn(T, h, D, generator=g).bfloat16() for h in (Hq, Hk)]
    for t in (q, k, d[0], d[1]):
        t[50:] = float("nan")
    c = lambda *ts: [t.cuda() for t in ts]  # noqa: E731
    full = mfr.head_norm_rotary_backward(*c(d[0], d[1], q, k, w[0], w[1], pos, freq))
    assert (full[0][~live.cuda()] == 0).all() and (full[1][~live.cuda()] == 0).all()
    part = mfr.head_norm_rotary_backward(*c(d[0][live], d[1][live], q[live], k[live], w[0], w[1], pos[live], freq))
    assert torch.equal(full[0][live.cuda()], part[0]) and torch.equal(full[1][live.cuda()], part[1])
    for a, b in zip(full[2:], part[2:]):  # the same terms, in other lanes
        assert ((a - b).abs() <= 204 * U * 300 * 10).all()
    bare = mfr.head_norm_rotary_backward(*c(d[0], d[1], q, k), None, None, *c(pos, freq))
    assert bare[2] is None and bare[3] is None
    none = mfr.head_norm_rotary_backward(*c(d[0], d[1], q, k, w[0], w[1], pos, freq), want_weights=False)
    assert none[2] is None and torch.equal(none[0], full[0])
    dq, dk = c(d[0].clone(), d[1].clone())
    here = mfr.head_norm_rotary_backward(dq, dk, *c(q, k, w[0], w[1], pos, freq), d_q=dq, d_k=dk)
    assert all(torch.equal(a, b) for a, b in zip(here, full))
    q2, k2 = c(q.clone(), k.clone())
    here = mfr.head_norm_rotary_backward(*c(d[0], d[1]), q2, k2, *c(w[0], w[1], pos, freq), d_q=q2, d_k=k2)
    assert all(torch.equal(a, b) for a, b in zip(here, full))


def test_head_norm_empty(mfr):
    e, p, f = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    assert mfr.head_norm_rotary(e, e, w, w, p, f)[0].shape == e.shape
    got = mfr.head_norm_rotary_backward(e, e, e, e, w, w, p, f)
    assert (got[2] == 0).all() and (got[3] == 0).all()


# ------------------------------------------------------------------------------------------------------------
# Refusals of the binding (nothing is written)
# ------------------------------------------------------------------------------------------------------------

def test_binding_refuses_bad_tensors(mfr):
    x = torch.randn(8, 32).cuda()
    ids = torch.zeros(8, 2, dtype=torch.int32).cuda()
    good = mfr.moe_route(x, 2)
    bad = [
        lambda: mfr.moe_route(x.double(), 2), lambda: mfr.moe_route(x.t(), 2), lambda: mfr.moe_route(x, 2, score="max"),
        lambda: mfr.moe_route(x, 2, bias=torch.zeros(31).cuda()), lambda: mfr.moe_route(x, 2, bias=torch.zeros(32)),
        lambda: mfr.moe_route(x, 2, bias=torch.zeros(32).half().cuda()), lambda: mfr.moe_route(x, 2, group_score="sum"),
        lambda: mfr.moe_route(x, 2, scale_dtype=torch.float64), lambda: mfr.moe_route(x, 3, out=good),
        lambda: mfr.moe_route(x, 33), lambda: mfr.moe_route(x, 0), lambda: mfr.moe_route(x, 2, num_groups=5),
        lambda: mfr.moe_route(x[:, :1].expand(8, 32), 2), lambda: mfr.moe_route(x[:1].expand(8, 32), 2),
        lambda: mfr.moe_route(x, 2, row_align=0),
        lambda: mfr.moe_route_backward(good.expert_scale, x, ids.long()), lambda: mfr.moe_route_backward(good.expert_scale[:7], x, ids),
        lambda: mfr.moe_route_backward(good.expert_scale, x, ids, out=torch.empty(8, 32, dtype=torch.float16, device="cuda")),
        lambda: mfr.moe_dispatch(x, ids), lambda: mfr.moe_dispatch(x[:, :6].contiguous(), ids, 16),
        lambda: mfr.moe_dispatch(x[:, :16], ids, 16), lambda: mfr.moe_dispatch(x, ids, 16, out=torch.empty(16, 32).half().cuda()),
        lambda: mfr.moe_dispatch(x, ids, 16, out=torch.empty(15, 32).cuda()), lambda: mfr.moe_dispatch(x, ids[:7], 16),
        lambda: mfr.moe_dispatch(x, ids, 16, row_route=torch.zeros(15, dtype=torch.int32).cuda()),
        lambda: mfr.moe_dispatch(x.flatten()[1:225].view(7, 32), ids[:7], 16),  # not on 16 bytes
        lambda: mfr.moe_finalize_routed_backward(x, mfr.Partial(x, ids)),
        lambda: mfr.moe_finalize_routed_backward(x.half(), mfr.Partial(x.bfloat16(), ids)),
        lambda: mfr.moe_finalize_routed_backward(x.half(), mfr.Partial(x.half(), ids), want_d_scale=False, want_d_gemm2=False),
        lambda: mfr.moe_finalize_routed_backward(x.half(), mfr.Partial(x.half(), ids), d_scale=torch.zeros(8, 2).half().cuda()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, mfr.MoEFinalizeError)):
            call()
            pytest.fail(f"call {i} was not refused")


def test_binding_refuses_bad_heads(mfr):
    q = torch.randn(4, 2, 64).half().cuda()
    p, f, w = torch.arange(4).cuda(), torch.ones(32).cuda(), torch.ones(64).half().cuda()
    ok = mfr.head_norm_rotary(q, q, w, w, p, f)
    wide = torch.randn(4, 2, 132).half().cuda()
    bad = [
        lambda: mfr.head_norm_rotary(q.float(), q.float(), None, None, p, f), lambda: mfr.head_norm_rotary(q, q.bfloat16(), None, None, p, f),
        lambda: mfr.head_norm_rotary(q, q[:3], None, None, p, f), lambda: mfr.head_norm_rotary(q, q, w[:32], w, p, f),
        lambda: mfr.head_norm_rotary(q, q, w.float(), w, p, f), lambda: mfr.head_norm_rotary(q, q, w, w, p.float(), f),
        lambda: mfr.head_norm_rotary(q, q, w, w, p[:3], f), lambda: mfr.head_norm_rotary(q, q, w, w, p, f.double()),
        lambda: mfr.head_norm_rotary(q, q, w, w, p, torch.ones(33).cuda()), lambda: mfr.head_norm_rotary(q, q, w, w, p, f[:5]),
        lambda: mfr.head_norm_rotary(q, q, w, w, p, f, style="pairs"), lambda: mfr.head_norm_rotary(q, q, w, w, p, f, q_out=ok[0]),
        lambda: mfr.head_norm_rotary(wide[:, :, :64], q, w, w, p, f),  # heads 132 apart
        lambda: mfr.head_norm_rotary(q, q, w, w, p, f, q_out=ok[0][:1].expand(4, 2, 64), k_out=ok[1]),
        lambda: mfr.head_norm_rotary(q.transpose(1, 2), q.transpose(1, 2), None, None, p, f),
        lambda: mfr.head_norm_rotary_backward(q, q[:, :1], q, q, w, w, p, f), lambda: mfr.head_norm_rotary_backward(q, q, q, q, w, w, p, f, d_q=ok[0]),
        lambda: mfr.head_norm_rotary_backward(q, q, q, q, w, w, p, f, d_q_weight=torch.zeros(64).half().cuda()),
        lambda: mfr.head_norm_rotary_backward(q, q, q, q, w, w, p, f, workspace=torch.zeros(16, dtype=torch.uint8).cuda()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, mfr.MoEFinalizeError)):
            call()
            pytest.fail(f"call {i} was not refused")


# ------------------------------------------------------------------------------------------------------------
# Together, as a layer uses them
# ------------------------------------------------------------------------------------------------------------

class Layer:
    """A small layer: norm_out of the fused finalize feeds a projection and the head norm; its input is routed,
    dispatched, multiplied by each row's expert and finalized."""

    def __init__(self, T, H=256, E=16, K=4, Hq=4, Hk=2, D=64, seed=0):
        g = gen(seed)
        self.T, self.H, self.E, self.K, self.Hq, self.Hk, self.D = T, H, E, K, Hq, Hk, D
        dev = "cuda"
        self.x = torch.randn(T, H, generator=g).bfloat16().to(dev)
        self.router = (torch.randn(H, E, generator=g) / H ** 0.5).to(dev)
        self.experts = (torch.randn(E, H, H, generator=g) / H ** 0.5).bfloat16().to(dev)
        self.residual = torch.randn(T, H, generator=g).bfloat16().to(dev)
        self.gamma = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().to(dev)
        self.proj = (torch.randn(H, (Hq + 2 * Hk) * D, generator=g) / H ** 0.5).bfloat16().to(dev)
        self.wq, self.wk = ((1 + 0.1 * torch.randn(D, generator=g)).bfloat16().to(dev) for _ in range(2))
        self.pos = torch.arange(T, device=dev, dtype=torch.int32)
        self.freq = (1.0 / 10000 ** (torch.arange(0, D, 2).float() / D)).to(dev)

    def forward(self, mfr, pdl=True, stream=None):
        logits = self.x.float() @ self.router
        r = mfr.moe_route(logits, self.K, bias=None, score="sigmoid", row_align=16, scale=2.5, pdl=pdl, stream=stream)
        rows = mfr.moe_dispatch(self.x, r.perm_idx, row_route=r.row_route, pdl=pdl, stream=stream)
        which = torch.searchsorted(r.expert_offsets[1:].contiguous(), torch.arange(rows.shape[0], device="cuda", dtype=torch.int32), right=True)
        y = torch.bmm(rows[:, None], self.experts[which.clamp(max=self.E - 1)])[:, 0]
        part = mfr.Partial(y, r.perm_idx, r.expert_scale)
        res, norm, _, _ = mfr.moe_finalize_fused([part], self.residual, self.gamma, pdl=pdl, stream=stream)
        qkv = norm @ self.proj
        q = qkv[:, :self.Hq * self.D].view(self.T, self.Hq, self.D)
        k = qkv[:, self.Hq * self.D:(self.Hq + self.Hk) * self.D].view(self.T, self.Hk, self.D)
        q, k = mfr.head_norm_rotary(q, k, self.wq, self.wk, self.pos, self.freq, q_out=q, k_out=k, pdl=pdl, stream=stream)
        return logits, r, rows, y, res, norm, q, k

    def step(self, mfr, pdl=True):
        """Forward through the finalize, and the gradients of <d, out> back to x, the scales' logits and the rows."""
        logits = self.x.float() @ self.router
        r = mfr.moe_route(logits, self.K, score="softmax", row_align=8, pdl=pdl)
        rows = mfr.moe_dispatch(self.x, r.perm_idx, row_route=r.row_route, pdl=pdl)
        out = mfr.moe_finalize_routed([mfr.Partial(rows, r.perm_idx, r.expert_scale)], pdl=pdl)
        d_rows, d_scale = mfr.moe_finalize_routed_backward(self.residual, mfr.Partial(rows, r.perm_idx, r.expert_scale),
                                                           row_route=r.row_route, pdl=pdl)
        d_logits = mfr.moe_route_backward(d_scale, logits, r.expert_ids, score="softmax", pdl=pdl)
        dx = mfr.moe_finalize_routed([mfr.Partial(d_rows, r.perm_idx)], pdl=pdl)
        return out, d_rows, d_scale, d_logits, dx


def test_layer_forward_against_64_bits(mfr):
    L = Layer(37)
    logits, r, rows, y, res, norm, q, k = L.forward(mfr)
    ids = r.expert_ids.cpu().long()
    x64 = logits.double().cpu().numpy()
    want_ids, s = ref.choose(x64, L.K, "sigmoid")
    assert np.array_equal(ids.numpy(), want_ids)
    w = torch.from_numpy(ref.weights(x64, want_ids, s, "sigmoid", True, 2.5))
    # experts and finalize in 64 bits from the same bf16 inputs; the library's bf16 expert products differ by half a
    # step each, so the finalized sum by half a step of the sum of sizes, and once more for its own rounding
    prod = torch.einsum("th,tkhj->tkj", L.x.double().cpu(), L.experts.double().cpu()[ids])
    out = (prod * w[..., None]).sum(1)
    bound = (prod.abs() * w[..., None]).sum(1) * (2 * step(torch.bfloat16)) + 2e-5
    total = out + L.residual.double().cpu()
    assert ((res.double().cpu() - total).abs() <= bound + 2 * step(torch.bfloat16) * (total.abs() + out.abs() + bound)).all()
    qkv = (norm @ L.proj).cpu()
    qw = ref.head_norm(qkv[:, :L.Hq * L.D].view(L.T, L.Hq, L.D).double(), L.wq.double().cpu(), L.pos.tolist(), L.freq.cpu(), "half", 1e-6, 1.0)
    kw = ref.head_norm(qkv[:, L.Hq * L.D:(L.Hq + L.Hk) * L.D].view(L.T, L.Hk, L.D).double(), L.wk.double().cpu(), L.pos.tolist(), L.freq.cpu(), "half", 1e-6, 1.0)
    within(q, qw, torch.bfloat16, extra=H_REL * 30)
    within(k, kw, torch.bfloat16, extra=H_REL * 30)


def test_layer_gradients_against_64_bits(mfr):
    """x -> dispatch -> finalize with the routed weights, in one graph of 64-bit operations."""
    L = Layer(29, H=64, E=12)
    out, d_rows, d_scale, d_logits, dx = L.step(mfr)
    x = L.x.double().cpu().requires_grad_()
    logits = (L.x.float() @ L.router).double().cpu().requires_grad_()
    ids = torch.from_numpy(ref.choose(logits.detach().numpy(), L.K, "softmax")[0])
    w = ref.route_weights_torch(logits, ids, "softmax", True, 1.0)
    y = (x[:, None, :] * w[..., None]).sum(1)
    d = L.residual.double().cpu()
    (y * d).sum().backward()
    half = step(torch.bfloat16)
    # out: the weights' FP32 error and one rounding
    assert ((out.double().cpu() - y).abs() <= half * y.abs() + 1e-5 * x.abs() + 1e-30).all()
    # dx: every row's gradient is rounded to bf16 before the sum, and the sum again
    assert ((dx.double().cpu() - x.grad).abs() <= half * (d.abs() * w.sum(1, keepdim=True)) + half * x.grad.abs() * 1.01 + 1e-5 * d.abs()).all()
    scale = (x.detach().abs() * d.abs()).sum(1, keepdim=True)
    assert ((d_logits.double().cpu() - logits.grad).abs() <= scale * (W_REL + 100 * U)).all()


@pytest.mark.parametrize("T", [1, 9, 200])
def test_layer_pdl_streams_and_repeats_are_bitwise_equal(mfr, T):
    L = Layer(T, seed=T)
    first = [t.clone() for t in _flat(L.forward(mfr)) + list(L.step(mfr))]
    for kw in (dict(pdl=False), dict()):
        again = _flat(L.forward(mfr, **kw)) + list(L.step(mfr, pdl=kw.get("pdl", True)))
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = _flat(L.forward(mfr)) + list(L.step(mfr))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def _flat(v):
    logits, r, *rest = v
    return [logits, r.expert_ids, r.expert_scale, r.perm_idx, r.row_route, r.expert_offsets, r.expert_counts, *rest]


def test_calls_on_another_stream_than_the_current(mfr):
    """Outputs and workspaces allocated by the binding for another stream are safe to use there."""
    x = torch.randn(5000, 64, generator=gen(0)).cuda()
    want = mfr.moe_route(x, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = mfr.moe_route(x, 4, stream=side)
        torch.full((5000, 64), 1e9, device="cuda")  # would land in freed memory
        side.synchronize()
        assert torch.equal(got.perm_idx, want.perm_idx) and torch.equal(got.row_route, want.row_route)


def test_two_calls_at_once(mfr):
    """The same calls on two streams, each with workspaces of its own."""
    L = [Layer(700, seed=s) for s in (1, 2)]
    want = [[t.clone() for t in _flat(x.forward(mfr)) + list(x.step(mfr))] for x in L]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [None, None]
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = _flat(L[i].forward(mfr)) + list(L[i].step(mfr))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_past_32_bits(mfr):
    """Rows, tokens and heads that lie more than 2^32 bytes apart."""
    x = torch.randint(0, 255, (2, 1 << 20), generator=gen(0), dtype=torch.uint8).cuda()
    perm = torch.tensor([[0, 4999], [4500, 2]], dtype=torch.int32, device="cuda")
    rows = mfr.moe_dispatch(x, perm, 5000)
    assert torch.equal(rows[[0, 4999]], x[[0, 0]]) and torch.equal(rows[[4500, 2]], x[[1, 1]]) and not rows[4998].any()
    del rows
    H, n = 8192, 300000
    gemm2 = torch.zeros(n, H, dtype=torch.bfloat16, device="cuda")
    d = torch.randn(2, H, generator=gen(1)).bfloat16().cuda()
    perm = torch.tensor([[n - 1, 5], [n - 2, 280001]], dtype=torch.int32, device="cuda")
    gemm2[n - 1], gemm2[280001] = 1, 2
    d_rows, d_scale = mfr.moe_finalize_routed_backward(d, mfr.Partial(gemm2, perm))
    assert torch.equal(d_rows[perm.long()], d[:, None].expand(2, 2, H)) and int((d_rows != 0).any(1).sum()) == 4
    want = torch.tensor([[1.0, 0.0], [0.0, 2.0]], device="cuda").double() * d.double().sum(1, keepdim=True)
    assert ((d_scale.double() - want).abs() <= (-(-H // 2048) * 8 + 14) * U * 2 * d.double().abs().sum(1, keepdim=True)).all()
    del gemm2, d_rows
    wide = torch.zeros(3, 1 << 30, dtype=torch.float16, device="cuda")
    q = wide[:, 8:8 + 256].view(3, 2, 128)
    q.copy_(torch.randn(3, 2, 128, generator=gen(2)))
    pos, freq = torch.arange(3, device="cuda"), torch.rand(64, generator=gen(3)).cuda()
    w = torch.ones(128, dtype=torch.float16, device="cuda")
    a, _ = mfr.head_norm_rotary(q, q, w, w, pos, freq)
    b, _ = mfr.head_norm_rotary(q.contiguous(), q.contiguous(), w, w, pos, freq)
    assert torch.equal(a, b)
    ga = mfr.head_norm_rotary_backward(q, q, q, q, w, w, pos, freq)
    c = q.contiguous()
    gb = mfr.head_norm_rotary_backward(c, c, c, c, w, w, pos, freq)
    assert all(torch.equal(x, y) for x, y in zip(ga, gb))
    logits = wide[:, 5:5 + 100]
    logits.copy_(torch.randn(3, 100, generator=gen(4)))
    a, b = mfr.moe_route(logits, 7), mfr.moe_route(logits.contiguous(), 7)
    assert torch.equal(a.expert_ids, b.expert_ids) and torch.equal(a.perm_idx, b.perm_idx)


@pytest.mark.parametrize("T", [7, 300])
def test_layer_in_two_graphs(mfr, T):
    """Captured twice, replayed in turn with new inputs, and beside an eager run of the same tensors."""
    L = Layer(T, seed=3)
    eager = _flat(L.forward(mfr)) + list(L.step(mfr))
    graphs, outs = [], []
    for _ in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            L.forward(mfr), L.step(mfr)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = _flat(L.forward(mfr)) + list(L.step(mfr))
        graphs.append(g)
        outs.append(o)
    for seed in range(4):
        L.x.copy_(torch.randn(L.x.shape, generator=gen(seed)))
        graphs[seed % 2].replay()
        graphs[1 - seed % 2].replay()
        eager = _flat(L.forward(mfr)) + list(L.step(mfr))
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, eager))
